"""moe_gate and moe_gate_backward against their formulas in 64 bits.

Tolerances. A weight is scale * a / sum(a) with terms a of exp: with |l| <= D
the exponent's argument is off by at most 2 D half-units (2^-24 each, two
roundings), exp by 2 units of 2^-23, and sums, quotients and products by one
2^-24 each: sums of up to 1024 scores in a tree of depth <= 37, of topk terms
in one of depth 5. A quotient doubles what its parts carry. So weights are
within (4 D + 96) 2^-24 relative, and gradients within twice that of
q (|g| + sum q |g|), what their differences are made of, plus 2^-8 relative
where the result is rounded to bf16.
"""
import numpy as np
import pytest
import torch

from combine_softmax_top_b200 import moe
from combine_softmax_top_b200 import workloads as W

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FLT_MAX = float(np.finfo(np.float32).max)


class Case:
    def __init__(self, T, E, k, score="softmax", dtype=W.F32, bias=False, groups=1, topk_groups=1, best=1, renorm=1,
                 scale=1.0, shared=0):
        self.__dict__.update(locals())
        s = W.spec("decode", T=T, E=E, k=k, H=128, I=128, renorm=renorm, shared=shared, compact=1)
        self.shape = moe.make_shape(s)
        self.gate = moe.make_gate(score, groups, topk_groups, best, scale, dtype)
        self.ws = torch.empty(moe.moe_workspace_bytes(self.shape), dtype=torch.uint8, device="cuda")
        moe.moe_workspace_init(self.shape, self.ws)

    def logits(self, seed=0, std=2.0):
        g = torch.Generator().manual_seed(seed)
        l = torch.randn(self.T, self.E, generator=g) * std
        return l.to(torch.bfloat16 if self.dtype == W.BF16 else torch.float32).cuda()

    def make_bias(self, seed=1, std=0.2):
        return (torch.randn(self.E, generator=torch.Generator().manual_seed(seed)) * std).cuda() if self.bias else None

    def run(self, logits, bias=None, stream=None):
        ks = self.k + self.shared
        idx = torch.full((self.T, ks), -7, dtype=torch.int32, device="cuda")
        w = torch.full((self.T, ks), -7.0, device="cuda")
        moe.moe_gate(self.shape, self.gate, logits, bias, idx, w, self.ws, stream)
        return idx, w

    def back(self, logits, idx, gw):
        out = torch.full_like(logits, float("nan"))
        moe.moe_gate_backward(self.shape, self.gate, logits, idx, gw, out)
        return out


def log_scores(c, l):
    """Logarithms of the scores, 64 bits: nothing underflows."""
    if c.score == "sigmoid":
        return -torch.logaddexp(torch.zeros_like(l), -l)
    return l - torch.logsumexp(l, dim=1, keepdim=True)


def choose(c, logits, bias):
    """Expert choice by the definition, 64 bits on the host, ties to the lowest index."""
    l = logits.double().cpu()
    s = log_scores(c, l).exp()
    ch = s + bias.double().cpu() if bias is not None else l
    T, E = l.shape
    if c.groups > 1:
        r = s if bias is None and c.best == 2 else ch
        worth = r.view(T, c.groups, -1).sort(dim=2, descending=True).values[..., :c.best].sum(2)
        keep = torch.argsort(-worth, dim=1, stable=True)[:, :c.topk_groups]
        open_ = torch.zeros(T, c.groups, dtype=torch.bool).scatter_(1, keep, True)
        ch = ch.masked_fill(~open_.repeat_interleave(E // c.groups, 1), -np.inf)
    return torch.argsort(-ch, dim=1, stable=True)[:, :c.k]


def weights(c, l, idx):
    # renormalised softmax: the sum over all experts cancels, and is left out so
    # that the others' derivative is 0 and not a rounding
    ls = l if c.renorm and c.score == "softmax" else log_scores(c, l)
    lw = ls.gather(1, idx.long())
    if c.renorm:
        lw = lw - torch.logsumexp(lw, 1, keepdim=True)
    return lw.exp() * c.scale


def tol(l):
    return (4 * float(l.abs().max()) + 96) * U


def check(c, logits, bias=None, stream=None):
    idx, w = c.run(logits, bias, stream)
    torch.cuda.synchronize()
    assert moe.moe_poll_status(c.ws) == 0
    ref = choose(c, logits, bias)
    assert torch.equal(idx[:, :c.k].cpu().long(), ref)
    l = logits.double().cpu()
    want = weights(c, l, ref)
    err = (w[:, :c.k].double().cpu() - want).abs()
    # 2^-126: scores that are not renormalised may underflow
    assert bool((err <= tol(l.clamp(-100, 100)) * want + 2.0 ** -126).all()), float((err / want).max())
    if c.shared:
        assert bool((idx[:, c.k] == c.E).all()) and bool((w[:, c.k] == 1).all())
    return idx, w


FORMS = [
    dict(E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4, best=2, scale=2.5),
    dict(E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=3, best=1, renorm=0),
    dict(E=128, k=8, dtype=W.BF16),
    dict(E=128, k=6, groups=8, topk_groups=3, scale=16.0, renorm=0),
    dict(E=160, k=6, groups=8, topk_groups=3, best=2, dtype=W.BF16),
    dict(E=160, k=6, score="sigmoid", groups=4, topk_groups=2, best=2),
    dict(E=384, k=8, score="sigmoid", bias=True, scale=2.827, shared=1),
    dict(E=64, k=6, bias=True, renorm=0, dtype=W.BF16),
    dict(E=1000, k=32, score="sigmoid", bias=True, groups=20, topk_groups=7, best=2),
    dict(E=1024, k=31, bias=True, shared=1, groups=32, topk_groups=32),
    dict(E=60, k=4, dtype=W.BF16, score="sigmoid"),
    dict(E=13, k=13, score="sigmoid", bias=True),
    dict(E=7, k=1, dtype=W.BF16, renorm=0),
    dict(E=1, k=1, score="sigmoid", renorm=0),
    dict(E=2, k=2, groups=2, topk_groups=2),
    dict(E=512, k=10, groups=1, topk_groups=1, best=2, bias=True),
    # plain softmax: the gradient's row in registers, a quarter warp or a warp a token
    dict(E=128, k=8, renorm=0, dtype=W.BF16),
    dict(E=200, k=3, renorm=0, scale=2.0),
    dict(E=256, k=8, renorm=0, dtype=W.BF16, bias=True),
    dict(E=384, k=8, renorm=0, dtype=W.BF16),
    dict(E=1024, k=8, renorm=0),
    dict(E=516, k=12, renorm=0),
    dict(E=1000, k=7, renorm=0, dtype=W.BF16),
    dict(E=1002, k=7, renorm=0, dtype=W.BF16),
]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(f"{k}{v}" for k, v in f.items()))
@pytest.mark.parametrize("T", [1, 3, 257, 8195])
def test_gate_matches_the_formulas(form, T):
    c = Case(T, **form)
    check(c, c.logits(T), c.make_bias())


@pytest.mark.parametrize("T", [64, 32769])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_choice_at_a_border_binary32_cannot_see(dtype, T):
    """Choice scores that all lie within 2^-24 of one value: their order is
    only there in binary64."""
    c = Case(T, E=128, k=8, score="sigmoid", bias=True, dtype=dtype)
    logits = c.logits(5)
    logits[:] = logits[0]
    flips = torch.arange(T, device="cuda") % 2 == 1
    logits[flips] = logits[flips] * (1 + 2.0 ** -7)     # another value of either type
    bias = (0.75 - torch.sigmoid(logits[0].double())).float()
    check(c, logits, bias)
    # and groups whose two best sum to nearly the same
    c = Case(T, E=128, k=8, score="sigmoid", bias=True, dtype=dtype, groups=8, topk_groups=4, best=2)
    check(c, logits, bias)
    # softmax scores of the same kind
    c = Case(T, E=128, k=8, bias=True, dtype=dtype, groups=8, topk_groups=4)
    check(c, logits, (0.5 - torch.softmax(logits[0].double(), 0)).float())


@pytest.mark.parametrize("T,k", [(48, 8), (32771, 8), (8195, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("near", [2, 9, 20, 31, 32, 33, 60])
def test_few_candidates_at_a_border(score, near, T, k):
    """`near` experts within 2^-24 of one another around the last slot, the
    others clearly above (three) or below."""
    E = 256 if k == 8 else 96
    c = Case(T, E=E, k=k, score=score, bias=True, renorm=0)
    logits = c.logits(near)
    logits[:] = logits[0]
    s = torch.sigmoid(logits[0].double()) if score == "sigmoid" else torch.softmax(logits[0].double(), 0)
    gen = torch.Generator().manual_seed(near)
    order = torch.randperm(E, generator=gen)
    target = torch.full((E,), 0.25, dtype=torch.float64)
    target[order[:3]] = torch.tensor([1.5, 1.25, 1.125], dtype=torch.float64)
    target[order[3:3 + near]] = 0.75
    bias = (target.cuda() - s).float()
    # the same bits in another order of rows: each row moves one logit by a unit
    t = torch.arange(T)
    logits[t, order[3 + t % near]] *= 1 + 2.0 ** -23
    check(c, logits, bias)
    # and on the logits themselves: neighbouring binary32 numbers
    c = Case(T, E=E, k=k, score=score)
    l = torch.full((T, E), -1.0)
    l[:, order[:3]] = 2.0
    steps = torch.randint(0, 8, (T, near), generator=gen).float()
    l[:, order[3:3 + near]] = 1 + steps * 2.0 ** -23
    check(c, l.cuda())


@pytest.mark.parametrize("T", [1, 41, 16390])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("E,G,Kg,k", [(256, 8, 4, 8), (96, 3, 1, 8), (160, 8, 3, 6), (128, 32, 5, 12), (1024, 16, 2, 8)])
def test_groups_at_the_border_of_the_open_ones(E, G, Kg, k, score, bias, dtype, T):
    """Some rows where the first closed group has the experts of the last open
    one in another order, the best moved by one unit (a tie where the type has
    no such unit); the others with groups far apart, one of them not finite."""
    if T > 41 and E > 256:
        T = 41
    c = Case(T, E=E, k=k, score=score, dtype=dtype, bias=bias, groups=G, topk_groups=Kg, best=2)
    flat = torch.full((E,), 0.125, device="cuda") if bias else None
    logits = c.logits(E + T, 1.0)
    n = E // G
    l = logits.double().cpu()
    worth = log_scores(c, l).exp().view(T, G, n).sort(dim=2, descending=True).values[..., :2].sum(2)
    order = torch.argsort(-worth, dim=1, stable=True)
    rows = range(0, T, 5)
    for i, t in enumerate(list(rows)[:40]):
        a, b = int(order[t, Kg - 1]), int(order[t, Kg])
        v = logits[t, a * n:(a + 1) * n].flip(0)
        if i % 3:
            v[v.argmax()] *= 1 + (2.0 ** -23 if i % 3 == 1 else -2.0 ** -23)
        logits[t, b * n:(b + 1) * n] = v
    check(c, logits, flat)
    if T > 3:
        logits[3, E - 1] = float("nan")
        idx, w = c.run(logits, flat)
        assert moe.moe_poll_status(c.ws) != 0
        want = choose(c, torch.nan_to_num(logits), flat)
        keep = torch.arange(T) != 3
        assert torch.equal(idx.cpu().long()[keep], want[keep])
        assert bool(torch.isnan(w[3]).all()) and torch.equal(idx[3].cpu(), torch.arange(k, dtype=torch.int32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_equal_candidates_go_to_the_lowest_index(score, bias):
    c = Case(5, E=96, k=8, score=score, bias=bias, groups=4, topk_groups=2, best=2)
    logits = torch.zeros(5, 96, device="cuda")
    logits[1] = -0.0
    logits[1, ::2] = 0.0                       # the two zeros are one value
    logits[2, 50:] = 1.0                       # two equal groups above two
    logits[3] = -FLT_MAX                       # a row masked throughout
    logits[4] = -FLT_MAX
    logits[4, 30:33] = torch.tensor([1.0, 2.0, 1.0], device="cuda")
    idx, w = c.run(logits, torch.zeros(96, device="cuda") if bias else None)
    assert torch.equal(idx.cpu().long(), choose(c, logits, torch.zeros(96) if bias else None))
    assert torch.equal(idx[0].cpu(), torch.arange(8, dtype=torch.int32))
    assert bool(torch.isfinite(w).all())
    # renormalised over equal scores: 1/8 each, also where every score underflows
    assert torch.allclose(w[3].cpu(), torch.full((8,), 0.125), rtol=96 * U, atol=0)


def test_bias_of_the_lowest_value_closes_experts():
    c = Case(33, E=64, k=6, score="sigmoid", bias=True, groups=8, topk_groups=2, best=2)
    bias = torch.full((64,), -FLT_MAX, device="cuda")
    bias[40:48] = 0.1
    logits = c.logits(3)
    check(c, logits, bias)
    check(c, logits, torch.full((64,), -FLT_MAX, device="cuda"))   # nothing left to choose by: lowest indices


def test_weights_where_scores_underflow():
    """sigmoid(l) is 0 in binary32 below about -104; shares of a sum are not."""
    c = Case(4, E=32, k=4, score="sigmoid")
    logits = -200.0 + torch.arange(32, device="cuda").float().repeat(4, 1) * 0.25
    logits[1] -= 3e4
    logits[2] += 300.0
    logits[3, 5] = 90.0
    idx, w = c.run(logits)
    l = logits.double().cpu()
    want = weights(c, l, choose(c, logits, None))
    # arguments up to 3e4 - 8 apart only by small differences: exact in binary32
    assert torch.allclose(w.double().cpu(), want, rtol=(4 * 100 + 96) * U, atol=2.0 ** -126)


def test_shape_without_tokens():
    c = Case(0, E=64, k=4)
    z = torch.empty(0, 64, device="cuda")
    c.run(z)
    c.back(z, torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda"))


@pytest.mark.parametrize("T", [3, 8193])
@pytest.mark.parametrize("where", ["logit", "bias"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_values_are_latched(where, value, T):
    c = Case(T, E=64, k=4, score="sigmoid", bias=True, groups=4, topk_groups=2, best=2)
    logits, bias = c.logits(), c.make_bias()
    if where == "logit":
        logits[1, 63] = value
    else:
        bias[17] = value
    idx, w = c.run(logits, bias)
    assert moe.moe_poll_status(c.ws) == 6
    bad = torch.zeros(T, dtype=torch.bool) if where == "logit" else torch.ones(T, dtype=torch.bool)
    bad[1] = True
    assert bool((idx.cpu()[bad] == torch.arange(4)).all()) and bool(torch.isnan(w.cpu()[bad]).all())
    assert bool(torch.isfinite(w.cpu()[~bad]).all())
    assert moe.moe_poll_status(c.ws) == 0      # read once


def _grad_formula(c, logits, idx, gw):
    """(gradient, what its differences are made of), 64 bits, by differentiation."""
    l = logits.double().cpu().requires_grad_(True)
    g = gw.double().cpu()
    w = weights(c, l, idx.cpu())
    grad = torch.autograd.grad((w * g).sum(), l)[0]
    w = w.detach().abs()
    share = w / abs(c.scale) if c.renorm or c.score == "softmax" else torch.zeros_like(w)
    size = torch.zeros_like(l.detach()).scatter_add_(1, idx.cpu().long(), w * g.abs())
    part = (share * g.abs()).sum(1, keepdim=True)
    if c.renorm:
        size.scatter_add_(1, idx.cpu().long(), w * part)
    elif c.score == "softmax":
        size += abs(c.scale) * log_scores(c, l.detach()).exp() * part
    return grad, size


@pytest.mark.parametrize("form", [f for f in FORMS if not f.get("shared")],
                         ids=lambda f: "-".join(f"{k}{v}" for k, v in f.items()))
@pytest.mark.parametrize("T", [1, 130, 4999])
def test_gradient_matches_the_formula(form, T):
    c = Case(T, **form)
    logits, bias = c.logits(7), c.make_bias()
    idx, _ = c.run(logits, bias)
    gw = torch.randn(T, c.k, generator=torch.Generator().manual_seed(2)).cuda()
    got = c.back(logits, idx, gw).double().cpu()
    want, size = _grad_formula(c, logits, idx, gw)
    bound = 2 * tol(logits.double()) * size + (2.0 ** -8 * want.abs() if c.dtype == W.BF16 else 0) + 2.0 ** -126
    off = float(((got - want).abs() / size.clamp_min(1e-30)).max())
    assert bool(((got - want).abs() <= bound).all()), off


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gradient_matches_differences(score, renorm):
    """Central differences of the weights in 64 bits, step h: off by h^2 times a
    third derivative (at most scale) and 2^-52 / h."""
    c = Case(2, E=12, k=3, score=score, renorm=renorm, scale=1.5)
    logits = c.logits(9)
    idx, _ = c.run(logits)
    gw = torch.tensor([[1.0, -2.0, 0.5], [0.25, 3.0, -1.0]], device="cuda")
    got = c.back(logits, idx, gw).double().cpu()
    l, h = logits.double().cpu(), 2.0 ** -14
    for e in range(12):
        d = torch.zeros_like(l)
        d[:, e] = h
        diff = ((weights(c, l + d, idx.cpu()) - weights(c, l - d, idx.cpu())) * gw.double().cpu()).sum(1) / (2 * h)
        assert torch.allclose(got[:, e], diff, rtol=0, atol=6 * 1.5 * h * h * 4 + 2 * tol(l) * 12)


@pytest.mark.parametrize("rep", [1, 1000])
@pytest.mark.parametrize("score,renorm", [("softmax", 0), ("softmax", 1), ("sigmoid", 0), ("sigmoid", 1)])
def test_gradient_of_absent_and_repeated_slots(score, renorm, rep):
    c = Case(5 * rep, E=16, k=4, score=score, renorm=renorm)
    logits = c.logits(11)[:5].repeat(rep, 1)
    idx = torch.tensor([[3, -1, 16, 5], [2, 2, 7, 2], [-1, -1, -1, -1], [1 << 30, 0, -(1 << 31), 15], [9, 9, 9, 9]],
                       dtype=torch.int32, device="cuda")
    gw = torch.randn(5, 4, generator=torch.Generator().manual_seed(4)).cuda()
    got = c.back(logits, idx.repeat(rep, 1), gw.repeat(rep, 1)).double().cpu()
    assert torch.equal(got, got[:5].repeat(rep, 1))
    for t in range(5):
        keep = [j for j in range(4) if 0 <= int(idx[t, j]) < 16]
        if not keep:
            assert bool((got[t] == 0).all())
            continue
        want, size = _grad_formula(c, logits[t:t + 1], idx[t:t + 1, keep], gw[t:t + 1, keep])
        # repeated slots add their sizes, and an exactly cancelling sum leaves only roundings
        assert bool(((got[t] - want[0]).abs() <= 2 * tol(logits.double()) * size[0] + 2.0 ** -126).all())


def test_gradient_with_a_shared_expert_ignores_its_slot():
    a, b = Case(9, E=64, k=6, score="sigmoid", shared=1), Case(9, E=64, k=6, score="sigmoid")
    logits = a.logits(1)
    idx, w = a.run(logits)
    gw = torch.randn(9, 7, generator=torch.Generator().manual_seed(6)).cuda()
    assert torch.equal(a.back(logits, idx, gw), b.back(logits, idx[:, :6].contiguous(), gw[:, :6].contiguous()))


def test_gradient_far_out():
    """Saturated scores: 1 - s is kept where s rounds to 1, and 0 gradient
    where a share is 1."""
    c = Case(2, E=8, k=2, score="sigmoid", renorm=0)
    logits = torch.full((2, 8), -30.0, device="cuda")
    logits[0, 3], logits[0, 4], logits[1, 0], logits[1, 1] = 25.0, 40.0, -60.0, 60.0
    idx = torch.tensor([[3, 4], [0, 1]], dtype=torch.int32, device="cuda")
    gw = torch.ones(2, 2, device="cuda")
    want, size = _grad_formula(c, logits, idx, gw)
    got = c.back(logits, idx, gw).double().cpu()
    assert torch.allclose(got, want, rtol=2 * (4 * 60 + 96) * U, atol=0)


def test_graph_capture_streams_and_repeats():
    """Captured and replayed on new inputs; on another stream; twice at once on
    one workspace; the same bits every time."""
    c = Case(300, **FORMS[0])
    logits, bias = c.logits(1), c.make_bias()
    idx, w = c.run(logits, bias)
    gw = torch.randn(300, 8, device="cuda")
    grad = c.back(logits, idx, gw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        idx2, w2 = c.run(logits, bias)
        g2 = c.back(logits, idx2, gw)
    idx3, w3 = c.run(logits, bias)
    torch.cuda.synchronize()
    assert torch.equal(idx, idx2) and torch.equal(w, w2) and torch.equal(grad, g2)
    assert torch.equal(idx, idx3) and torch.equal(w, w3)
    sl, si, sw, sg = logits.clone(), torch.empty_like(idx), torch.empty_like(w), torch.empty_like(logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_gate(c.shape, c.gate, sl, bias, si, sw, c.ws)
        moe.moe_gate_backward(c.shape, c.gate, sl, si, gw, sg)
    for seed in (2, 3):
        new = c.logits(seed)
        sl.copy_(new)
        graph.replay()
        i, ww = c.run(new, bias)
        torch.cuda.synchronize()
        assert torch.equal(si, i) and torch.equal(sw, ww) and torch.equal(sg, c.back(new, i, gw))


def test_gate_agrees_with_route_where_both_apply():
    """Plain softmax, no bias, no groups: moe_route's choice."""
    c = Case(500, E=256, k=8)
    logits = c.logits(3)
    idx, w = c.run(logits)
    ri, rw = torch.empty_like(idx), torch.empty_like(w)
    moe.moe_route(c.shape, logits, ri, rw, c.ws)
    torch.cuda.synchronize()
    assert torch.equal(idx, ri)
    assert torch.allclose(w, rw, rtol=2 * tol(logits), atol=0)


@pytest.mark.parametrize("E", [64, 256, 516, 1024, 66, 1001])
def test_softmax_gradient_of_far_experts_is_binary32s(E):
    """Logits 20 to 84 below the only chosen one, in steps that subtract exactly,
    so that the probability is one exp, off by 2 * 2^-23 = 4 U (U = 2^-24), times
    1 / z. z is 1 but for the others (1024 / 64 e^-20 / (1 - e^-(1/16)) < 0.6 U),
    one rounding as they are added, one of the reciprocal: 2.6 U, in p_e and in
    the sum over the chosen. With three products: 4 + 5.2 + 3 < 13 U."""
    c = Case(70, E=E, k=1, renorm=0)
    far = -(20 + 64 * torch.arange(E, dtype=torch.float64) / E)
    l = (far * 1024).round() / 1024
    l = l.repeat(70, 1)
    idx = torch.arange(70)[:, None] * 7 % E
    l.scatter_(1, idx, 0.0)
    l += torch.arange(70)[:, None].double() % 5          # every logit a multiple of 2^-10 below 2^7
    got = c.back(l.float().cuda(), idx.int().cuda(), torch.full((70, 1), 3.0, device="cuda")).double().cpu()
    p = torch.softmax(l, 1)
    want = 3 * p.gather(1, idx) * -p
    other = torch.ones_like(l, dtype=torch.bool).scatter_(1, idx, False)
    off = ((got - want).abs() / want.abs())[other]
    assert float(off.max()) <= 13 * U, float(off.max()) / U


def _gradient_by_case(c, l, idx, g):
    """(gradient, what its differences are made of) of finite and other logits, 64
    bits: an infinity counts as its limit where there is one."""
    s = torch.sigmoid(l).gather(1, idx)
    if c.score == "softmax":
        p = torch.softmax(l if not c.renorm else l.gather(1, idx), 1)      # +inf and NaN: a row of NaN
        q = p if c.renorm else p.gather(1, idx)
    else:
        # s / sum s by a factor common to all, so that no share underflows
        ls = -torch.logaddexp(torch.zeros_like(l), -l).gather(1, idx)
        q = torch.softmax(ls, 1) if c.renorm else s
    part, size = (q * g).sum(1, keepdim=True), (q * g).abs().sum(1, keepdim=True)
    grad, made = torch.zeros_like(l), torch.zeros_like(l)
    if c.score == "softmax" and not c.renorm:
        grad, made = -p * part, p * size
    rest = 1 - s if c.score == "sigmoid" else torch.ones_like(s)           # of +inf 0, of -inf 1
    d = q * (g - part) if c.renorm else q * g
    grad.scatter_add_(1, idx, c.scale * d * rest)
    # a plain sigmoid's gradient of one expert is made of nothing of the others
    alone = c.score == "sigmoid" and not c.renorm
    made.scatter_add_(1, idx, abs(c.scale) * q * (g.abs() if alone else g.abs() + size))
    return grad, made


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("score,renorm", [("softmax", 0), ("softmax", 1), ("sigmoid", 0), ("sigmoid", 1)])
@pytest.mark.parametrize("E,k", [(128, 6), (256, 8), (512, 9), (1000, 6), (63, 5), (1002, 12)])
def test_gradient_of_logits_that_are_not_finite(E, k, score, renorm, dtype):
    """NaN and the infinities at chosen experts and at others: what depends on
    them as include/moe.h says, and nothing else."""
    values = [float("nan"), float("inf"), float("-inf")]
    c = Case(40, E=E, k=k, score=score, renorm=renorm, dtype=dtype)
    logits = c.logits(3)
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(40)])
    for t in range(36):                       # rows 36 .. 39 stay finite
        row = idx[t].tolist()
        other = next(e for e in range(E) if e not in row)
        at = [row[0], other, row[k - 1]][t % 3]
        logits[t, at] = values[t // 3 % 3]
        if t >= 18:                           # two values in a row, one chosen and one not
            logits[t, row[1]] = values[t // 9 % 3]
            logits[t, E - 1 if E - 1 not in row else other] = values[t // 2 % 3]
        if t >= 33:                           # every chosen expert
            logits[t, idx[t]] = values[t % 3]
    gw = torch.randn(40, k, generator=torch.Generator().manual_seed(5)).cuda()
    got = c.back(logits, idx.int().cuda(), gw).double().cpu()
    want, made = _gradient_by_case(c, logits.double().cpu(), idx, gw.double().cpu())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    finite = logits.double().cpu()
    bound = 2 * tol(finite[torch.isfinite(finite)]) * made + (2.0 ** -8 * want.abs() if dtype == W.BF16 else 0) + 2.0 ** -126
    assert bool(((got - want).abs() <= bound)[ok].all())


@pytest.mark.parametrize("T", [4095, 4096, 5999, 6000, 8191, 10239, 10240, 12288, 16383, 16385])
@pytest.mark.parametrize("form", [
    dict(E=64, k=7, renorm=0), dict(E=60, k=6, score="sigmoid", bias=True), dict(E=64, k=6, groups=8, topk_groups=4, best=2),
    dict(E=128, k=8, dtype=W.BF16), dict(E=100, k=6, bias=True, dtype=W.BF16), dict(E=128, k=12, bias=True, score="sigmoid"),
    dict(E=160, k=6, score="sigmoid", bias=True, groups=8, topk_groups=3, best=2), dict(E=250, k=15, dtype=W.BF16),
    dict(E=192, k=8, bias=True, renorm=0), dict(E=196, k=8, bias=True),
], ids=lambda f: "-".join(f"{k}{v}" for k, v in f.items()))
def test_gate_around_the_sizes_where_lanes_change(form, T):
    """Fewer lanes take a token from some of these sizes on."""
    c = Case(T, **form)
    check(c, c.logits(T), c.make_bias())
