"""The gate (routing with scores, a bias, groups and its gradient) and the
8-bit integer products with their row quantisation: what is measured of them.

Each operator has a plain form here, in elementary torch operations, and the
calls a program makes of the library. Cases stand for the layer shapes of
``combine_softmax_top_b200.workloads`` (hidden 7168, 256 experts of 2048, 8 a
token; hidden 4096, 128 experts of 1536), for shards of them (32 of the 256
experts), and for odd sizes.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one new token of a served model: sigmoid scores, a balance bias, 4 of 8 groups
        _gate("gate one token", T=1, E=256, k=8, score="sigmoid", dtype="f32", bias=True, groups=8, topk_groups=4,
              group_best=2, renorm=True, scale=2.5),
        # a prompt batch through the 256-expert layer
        _gate("gate prompt", T=8192, E=256, k=8, score="sigmoid", dtype="f32", bias=True, groups=8, topk_groups=4,
              group_best=2, renorm=True, scale=2.5),
        # the 128-expert layer's router on a training batch, bf16 logits, no bias and no groups
        _gate("gate training batch", T=32768, E=128, k=8, score="softmax", dtype="bf16", bias=False, groups=1,
              topk_groups=1, group_best=1, renorm=True, scale=1.0),
        # gradients of both kinds: renormalised sigmoid (chosen experts only) and plain softmax (every expert)
        _gate("gate backward sigmoid", back=True, T=8192, E=256, k=8, score="sigmoid", dtype="f32", bias=True, groups=8,
              topk_groups=4, group_best=2, renorm=True, scale=2.5),
        _gate("gate backward softmax", back=True, T=32768, E=128, k=8, score="softmax", dtype="bf16", bias=False,
              groups=1, topk_groups=1, group_best=1, renorm=False, scale=1.0),
        # an int8 linear layer on bf16 rows (quantise, multiply): one token, an odd size, a prompt
        _linear("linear one token", M=1, N=7168, K=2048, dtype="bf16", out="bf16"),
        _linear("linear odd", M=333, N=1001, K=1552, dtype="f32", out="f32"),
        _linear("linear prompt", M=8192, N=4096, K=7168, dtype="bf16", out="bf16"),
        # experts' products over dispatched windows, 32 of 256 experts: a decode batch of 128 tokens (4 rows an
        # expert) and a prompt batch of 8192 (256 rows an expert), gate/up with SwiGLU and down
        _experts("experts gate/up decode", E=32, pairs=128, N=2048, K=7168, swiglu=True, skew=0.0),
        _experts("experts down decode", E=32, pairs=128, N=7168, K=2048, swiglu=False, skew=0.0),
        _experts("experts gate/up prompt", E=32, pairs=8192, N=2048, K=7168, swiglu=True, skew=0.0),
        _experts("experts down skewed", E=32, pairs=8192, N=7168, K=2048, swiglu=False, skew=0.7),
    ]


def _gate(name=None, back=False, **kw):
    return _named(name, dict(op="gate_backward" if back else "gate", **kw))


def _linear(name=None, **kw):
    return _named(name, dict(op="linear", **kw))


def _experts(name=None, **kw):
    return _named(name, dict(op="experts", **kw))


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gate", "gate", "gate_backward", "linear", "linear", "experts", "experts"])
    if kind.startswith("gate"):
        back = kind == "gate_backward"
        E = rng.choice([8, 60, 64, 96, 128, 160, 256, 384, 512, 1000])
        T = max(1, min(_log(rng, 1, 32768), 4 * 1024 * 1024 // E))
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, topk_groups * (E // groups)))
        return _gate(back=back, T=T, E=E, k=k, score=score, dtype=rng.choice(["f32", "bf16"]), bias=rng.random() < 0.6,
                     groups=groups, topk_groups=topk_groups, group_best=rng.choice([1, 2]), renorm=rng.random() < 0.6,
                     scale=rng.choice([1.0, 2.5]))
    if kind == "linear":
        N, K = _log(rng, 64, 7168), 16 * _log(rng, 4, 448)
        M = max(1, min(_log(rng, 1, 8192), 8192 * 4096 * 7168 // (N * K)))
        return _linear(M=M, N=N, K=K, dtype=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
    N, K = 16 * _log(rng, 8, 448) + rng.choice([0, 0, 8, 3]), 16 * _log(rng, 8, 448)
    return _experts(E=rng.choice([1, 3, 8, 17, 32]), pairs=_log(rng, 1, 4096), N=min(N, 2048), K=K,
                    swiglu=rng.random() < 0.5, skew=rng.choice([0.0, 0.7, 1.2]))


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "linear":
        return _prepare_linear(case, g)
    if case["op"] == "experts":
        return _prepare_experts(case, g)
    T, E, k = case["T"], case["E"], case["k"]
    st = {"case": case, "logits": torch.randn(T, E, generator=g, device="cuda").to(DT[case["dtype"]])}
    st["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
    if case["op"] == "gate_backward":
        st["topk_idx"] = torch.rand(T, E, generator=g, device="cuda").add_(st["logits"]).topk(k).indices.int()
        st["grad_w"] = torch.randn(T, k, generator=g, device="cuda")
        st["grad_logits"] = torch.empty_like(st["logits"])
    else:
        st["topk_idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["topk_w"] = torch.empty(T, k, device="cuda")
    if own:  # the layer's shape, its workspace and the gate's description, kept by a program
        from combine_softmax_top_b200 import moe, workloads as W
        s = W.spec("sweep", T=T, E=E, k=k, H=128, xq=W.BF16, renorm=int(case["renorm"]))
        st["shape"] = moe.make_shape(s)
        st["ws"] = torch.empty(moe.moe_workspace_bytes(st["shape"]), dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(st["shape"], st["ws"])
        st["gate"] = moe.make_gate(score=case["score"], groups=case["groups"], topk_groups=case["topk_groups"],
                                   group_best=case["group_best"], scale=case["scale"], logits=case["dtype"])
    return st


def _int8(shape, g, std=32.0):
    # normal weights and activations rounded to 8 bits, a row's largest near 127
    return (torch.randn(shape, generator=g, device="cuda") * std).round_().clamp_(-127, 127).to(torch.int8)


def _scales(n, g, base):
    return base * (0.5 + torch.rand(n, generator=g, device="cuda"))


def _workspace():
    """Any prepared workspace: the products latch their errors there."""
    from combine_softmax_top_b200 import moe, workloads as W
    sh = moe.make_shape(W.spec("tiny"))
    ws = torch.empty(moe.moe_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(sh, ws)
    return ws


def _prepare_linear(case, g):
    M, N, K = case["M"], case["N"], case["K"]
    st = {"case": case,
          "x": torch.randn(M, K, generator=g, device="cuda").to(DT[case["dtype"]]),
          "w": _int8((N, K), g), "w_scale": _scales(N, g, 0.02 / 32),
          "xq": torch.empty(M, K, dtype=torch.int8, device="cuda"),
          "x_scale": torch.empty(M, device="cuda"),
          "y": torch.empty(M, N, dtype=DT[case["out"]], device="cuda")}
    if own:
        st["ws"] = _workspace()
    return st


def _prepare_experts(case, g):
    E, N, K, pairs = case["E"], case["N"], case["K"], case["pairs"]
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float64).pow(-case["skew"])
    p = p[torch.randperm(E, generator=g, device="cuda")]
    who = torch.multinomial(p / p.sum(), pairs, replacement=True, generator=g)
    counts = torch.bincount(who, minlength=E)
    tiles = (counts + 127) // 128
    offsets = 128 * (tiles.cumsum(0) - tiles)
    M = 128 * (-(-pairs // 128) + E)   # windows packed on 128-row tiles, at most one partial tile an expert
    st = {"case": case, "x": _int8((M, K), g), "x_scale": _scales(M, g, 1.0 / 32),
          "w": _int8((E, N, K), g), "w_scale": _scales(E * N, g, 0.02 / 32).view(E, N),
          "w_up": _int8((E, N, K), g) if case["swiglu"] else None,
          "up_scale": _scales(E * N, g, 0.02 / 32).view(E, N) if case["swiglu"] else None,
          "offsets": offsets.int(), "counts": counts.int(),
          "most": int(counts.max()),
          "y": torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")}   # rows of no expert stay as they are
    if own:
        st["ws"] = _workspace()
    return st


# -------------------------------------------------------------------- runs --

def run(state):
    op = state["case"]["op"]
    if op == "gate":
        return _run_gate(state) if own else plain_gate(state)
    if op == "gate_backward":
        return _run_gate_backward(state) if own else plain_gate_backward(state)
    if op == "linear":
        return _run_linear(state) if own else plain_linear(state)
    return _run_experts(state) if own else plain_experts(state)


def _run_gate(st):
    from combine_softmax_top_b200 import moe
    moe.moe_gate(st["shape"], st["gate"], st["logits"], st["bias"], st["topk_idx"], st["topk_w"], st["ws"])
    return st["topk_idx"], st["topk_w"]


def _run_gate_backward(st):
    from combine_softmax_top_b200 import moe
    moe.moe_gate_backward(st["shape"], st["gate"], st["logits"], st["topk_idx"], st["grad_w"], st["grad_logits"])
    return st["grad_logits"]


def _run_linear(st):
    from combine_softmax_top_b200 import moe
    moe.moe_quant_i8(st["x"], st["xq"], st["x_scale"])
    moe.moe_gemm_i8(st["xq"], st["x_scale"], st["w"], st["w_scale"], st["y"], st["ws"])
    return st["y"]


def _run_experts(st):
    from combine_softmax_top_b200 import moe
    moe.moe_gemm_i8(st["x"], st["x_scale"], st["w"], st["w_scale"], st["y"], st["ws"], w_up=st["w_up"],
                    up_scale=st["up_scale"], offsets=st["offsets"], counts=st["counts"], fill=st["case"]["pairs"])
    return st["y"]


# ------------------------------------------------------------- plain forms --

def _best(c, n):
    """Indices of the n largest of each row, ties to the lowest index."""
    return torch.sort(c, dim=-1, descending=True, stable=True).indices[..., :n]


def plain_gate(st):
    case = st["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    # choice in 64 bits: experts next to the border are told apart
    l = st["logits"].double()
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.exp(l - l.amax(dim=1, keepdim=True))
        s = s / s.sum(dim=1, keepdim=True)
    # without a bias the scores order like the logits, which order exactly
    c = s + st["bias"].double() if case["bias"] else l
    if G > 1:
        by = (c if case["group_best"] == 1 or case["bias"] else s).view(T, G, E // G)
        rank = torch.sort(by, dim=2, descending=True).values[..., :case["group_best"]].sum(dim=2)
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, _best(rank, case["topk_groups"]), True)
        c = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), c, -math.inf)
    idx = _best(c, k)
    w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.int(), (w * case["scale"]).float()


def plain_gate_backward(st):
    case = st["case"]
    l, idx = st["logits"].float(), st["topk_idx"].long()
    g = st["grad_w"] * case["scale"]
    if case["score"] == "softmax" and not case["renorm"]:
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
        dot = (g * p.gather(1, idx)).sum(dim=1, keepdim=True)
        return (p * (torch.zeros_like(l).scatter_(1, idx, g) - dot)).to(st["logits"].dtype)
    chosen = l.gather(1, idx)
    if case["score"] == "softmax":
        q = torch.exp(chosen - chosen.amax(dim=1, keepdim=True))
        rest = 1.0
    else:
        q = 1.0 / (1.0 + torch.exp(-chosen))
        rest = 1.0 / (1.0 + torch.exp(chosen))
    if case["renorm"]:
        q = q / q.sum(dim=1, keepdim=True)
        g = g - (q * g).sum(dim=1, keepdim=True)
    return torch.zeros_like(l).scatter_(1, idx, q * g * rest).to(st["logits"].dtype)


def plain_linear(st):
    x = st["x"].float()
    amax = x.abs().amax(dim=1, keepdim=True)
    scale = torch.where(amax > 0, (amax / 127.0).clamp_min(2.0 ** -126), 1.0)
    q = torch.round(x / scale)
    y = torch.matmul(q, st["w"].float().t())
    return (y * scale * st["w_scale"]).to(st["y"].dtype)


def _padded(st):
    """Row of the buffer that each (expert, place) reads, and whether it is filled."""
    at = torch.arange(st["most"], device="cuda")
    rows = st["offsets"].long()[:, None] + at
    return rows.clamp_max(st["x"].shape[0] - 1), at < st["counts"][:, None]


def plain_experts(st):
    rows, real = _padded(st)
    x = st["x"][rows].float()                     # [E, most, K]
    xs = st["x_scale"][rows][..., None]
    y = torch.bmm(x, st["w"].float().transpose(1, 2)) * xs * st["w_scale"][:, None, :]
    if st["w_up"] is not None:
        up = torch.bmm(x, st["w_up"].float().transpose(1, 2)) * xs * st["up_scale"][:, None, :]
        y = y / (1.0 + torch.exp(-y)) * up
    out = torch.zeros_like(st["y"])
    out[rows[real]] = y[real].to(out.dtype)
    return out


# -------------------------------------------------------------------- work --

def work(case):
    if case["op"] in ("gate", "gate_backward"):
        T, E, k, el = case["T"], case["E"], case["k"], SIZE[case["dtype"]]
        if case["op"] == "gate":
            return {"bytes": T * E * el + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
        every = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * el + 8 * T * k + (T * E if every else T * k) * el,
                "flops": (6 * T * E if every else 0) + 8 * T * k}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * SIZE[case["dtype"]] + N * K + 4 * N + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    E, N, K, pairs = case["E"], case["N"], case["K"], case["pairs"]
    mats = 2 if case["swiglu"] else 1
    touched = min(E, pairs)   # the most experts that can have a row
    return {"bytes": pairs * (K + 4) + mats * touched * N * (K + 4) + pairs * N * 2 + 8 * E,
            "flops": 2 * mats * pairs * N * K}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    st = prepare(case, seed)
    return {"gate": _exact_gate, "gate_backward": _exact_gate_backward, "linear": _exact_linear,
            "experts": _exact_experts}[case["op"]](case, st)


def _log_scores(case, l):
    if case["score"] == "sigmoid":
        return -torch.logaddexp(torch.zeros_like(l), -l)
    return l - torch.logsumexp(l, dim=1, keepdim=True)


def _exact_gate(case, st):
    """Experts taken one at a time, weights from logarithms of the scores."""
    l = st["logits"].double()
    ls = _log_scores(case, l)
    c = ls.exp() + st["bias"].double() if case["bias"] else l.clone()
    T, E = l.shape
    n = E // case["groups"]
    rank = (c if case["bias"] or case["group_best"] == 1 else ls.exp()).reshape(T, case["groups"], n).clone()
    worth = torch.zeros(T, case["groups"], dtype=torch.float64, device=l.device)
    for _ in range(case["group_best"]):
        v, i = rank.max(dim=2)
        worth += v
        rank.scatter_(2, i[..., None], -math.inf)
    allowed = torch.zeros(T, case["groups"], dtype=torch.bool, device=l.device)
    place = torch.arange(max(E, case["groups"]), device=l.device)
    for _ in range(case["topk_groups"]):
        top = worth.amax(dim=1, keepdim=True)
        first = torch.where(worth == top, place[:case["groups"]], E + 1).amin(dim=1, keepdim=True)
        allowed.scatter_(1, first, True)
        worth.scatter_(1, first, -math.inf)
    c[~allowed.repeat_interleave(n, dim=1)] = -math.inf
    chosen = []
    for _ in range(case["k"]):
        top = c.amax(dim=1, keepdim=True)
        first = torch.where(c == top, place[:E], E + 1).amin(dim=1, keepdim=True)
        chosen.append(first)
        c.scatter_(1, first, -math.inf)
    idx = torch.cat(chosen, dim=1)
    lw = ls.gather(1, idx)
    if case["renorm"]:
        lw = lw - torch.logsumexp(lw, dim=1, keepdim=True)
    return idx.int(), lw.exp() * case["scale"]


def _exact_gate_backward(case, st):
    """The derivative of the weights, taken by differentiation."""
    l = st["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        lw = _log_scores(case, l).gather(1, st["topk_idx"].long())
        if case["renorm"]:
            lw = lw - torch.logsumexp(lw, dim=1, keepdim=True)
        loss = (lw.exp() * case["scale"] * st["grad_w"].double()).sum()
        return torch.autograd.grad(loss, l)[0]


def _exact_linear(case, st):
    x = st["x"].double()
    amax = x.abs().amax(dim=1, keepdim=True)
    # the scale is a 32-bit number by definition, and so is the quotient that is rounded
    scale = torch.where(amax > 0, (amax / 127).float().clamp_min(2.0 ** -126), torch.ones_like(amax, dtype=torch.float32)).double()
    q = (x / scale).float().double().round()
    return (q * scale) @ (st["w"].double() * st["w_scale"].double()[:, None]).t()


def _exact_experts(case, st):
    out = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    for e, (o, c) in enumerate(zip(st["offsets"].tolist(), st["counts"].tolist())):
        if c:
            x = st["x"][o:o + c].double() * st["x_scale"][o:o + c].double()[:, None]
            y = x @ (st["w"][e].double() * st["w_scale"][e].double()[:, None]).t()
            if case["swiglu"]:
                y = y * torch.sigmoid(y) * (x @ (st["w_up"][e].double() * st["up_scale"][e].double()[:, None]).t())
            out[o:o + c] = y
    return out
