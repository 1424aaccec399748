"""moe_quant_i8 (to the bit) and moe_gemm_i8 against their formulas in 64 bits,
and an int8 layer built of the stages.

Tolerances. The sums are exact integers below 2^31. Rounding one to binary32
and the two products with the scales cost 2^-24 each: 3 * 2^-24 relative, and
rounding to bf16 2^-8 more. silu(g) u = g u / (1 + exp(-g)): g and u carry
3 * 2^-24 each, which silu amplifies by at most 1 + |g|; exp, the sum, the
quotient and the product add 2 * 2^-23 + 3 * 2^-24: (3 (1 + |g|) + 10) 2^-24.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from combine_softmax_top_b200 import moe
from combine_softmax_top_b200 import workloads as W

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.fixture(scope="module")
def ws():
    sh = moe.make_shape(W.spec("tiny"))
    t = torch.empty(moe.moe_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(sh, t)
    return t


def quant_ref(x):
    """(q, scale) by the definition: binary32 division is binary64 division
    rounded once more (53 >= 2 * 24 + 2 bits: the same value)."""
    x = x.float().cpu().numpy().astype(np.float64)
    amax = np.abs(x).max(1) if x.shape[1] else np.zeros(x.shape[0])
    bad = ~np.isfinite(x).all(1)
    with np.errstate(all="ignore"):
        s = np.maximum(amax.astype(np.float32) * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126))
        s = np.where(amax == 0, np.float32(1), s)
        q = np.rint((x / s.astype(np.float64)[:, None]).astype(np.float32))
    q[bad] = 0
    s[bad] = np.nan
    return q.astype(np.int8), s


def run_quant(x, **kw):
    q = torch.full(x.shape, 99, dtype=torch.int8, device="cuda")
    s = torch.full(x.shape[:1], -5.0, device="cuda")
    moe.moe_quant_i8(x, q, s, **kw)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 7168), (3, 48), (129, 2048), (700, 1040), (5, 40000), (2, 131056),
                                       (64, 528), (2000, 16)])
def test_quant_is_the_definition(dtype, rows, cols):
    x = (torch.randn(rows, cols, generator=gen(rows)) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=gen(1))))
    x = x.to(DT[dtype]).cuda()
    q, s = run_quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s, rs) and np.array_equal(q, rq)


def test_quant_ties_zeros_and_far_values():
    """Halves go to even; rows of zeros, subnormals, one large value, the
    lowest value of the type, NaN and infinities."""
    x = torch.zeros(12, 256)
    x[0] = torch.arange(256) - 127.5                       # scale 127.5/127
    x[1, :254] = torch.arange(254) / 2 - 63.5              # scale 0.5: halves never, quarters below
    x[1, 255] = 63.5
    x[2, :250] = torch.arange(250) * 0.5 - 62.25           # quotients n + 1/2 with scale 0.5
    x[2, 255] = -63.5
    x[4] = 1e-45 * torch.arange(256)                       # subnormals: scale 2^-126
    x[5, 3] = 1e-45
    x[6, 9] = -3.4028234663852886e38
    x[6, 10] = 1e38
    x[7, 200] = float("nan")
    x[8, 0] = float("inf")
    x[9, 255] = float("-inf")
    x[10] = -0.0
    x[11] = 2.0 ** -120 * torch.arange(256)
    q, s = run_quant(x.cuda())
    rq, rs = quant_ref(x)
    assert np.array_equal(s, rs, equal_nan=True) and np.array_equal(q, rq)
    assert np.isnan(s[7:10]).all() and not np.isnan(s[[0, 1, 2, 3, 4, 5, 6, 10, 11]]).any()
    assert s[3] == 1 and s[10] == 1 and (q[3] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quant_rounds_next_to_ties(dtype):
    """Elements at, and a unit beside, x = (n + 1/2) scale, of rows with scales
    over the whole exponent range."""
    g = gen(7)
    rows, cols = 3000, 1024
    amax = (torch.rand(rows, 1, generator=g) + 1) * torch.exp2(torch.randint(-149, 127, (rows, 1), generator=g).double())
    amax = amax.float().to(DT[dtype]).float()
    scale = torch.maximum(amax * (torch.tensor(1.0) / torch.tensor(127.0)), torch.tensor(2.0 ** -126))
    n = torch.randint(-127, 127, (rows, cols), generator=g)
    x = ((n + 0.5).double() * scale.double()).float()
    step = torch.randint(-2, 3, (rows, cols), generator=g, dtype=torch.int32)
    x = (x.view(torch.int32) + step).view(torch.float32)     # neighbouring numbers
    x = x.to(DT[dtype]).float()
    x = torch.where(torch.isfinite(x) & (x.abs() <= amax), x, torch.zeros(()))
    x[:, 77] = amax[:, 0]
    x = x.to(DT[dtype]).cuda()
    q, s = run_quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s, rs) and np.array_equal(q, rq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(9, 16), (9, 528), (2000, 64), (2000, 2048), (700, 8192), (5, 40000)])
def test_quant_of_rows_that_are_not_finite(dtype, rows, cols):
    x = torch.randn(rows, cols, generator=gen(3))
    x[::4, -1], x[1::4, 0], x[2::4, cols // 2] = float("nan"), float("inf"), float("-inf")
    x = x.to(DT[dtype]).cuda()
    q, s = run_quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s, rs, equal_nan=True) and np.array_equal(q, rq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quant_of_windows_leaves_other_rows(dtype):
    M, K = 900, 272
    x = torch.randn(M, K, generator=gen(5)).to(DT[dtype]).cuda()
    off = [640, 0, 128, 300, 877, 899, 900, -5, 2 ** 31 - 1, 500]
    cnt = [130, 1, 129, 0, 21, 50, 3, 9, 2 ** 31 - 1, -4]
    o, c = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (off, cnt))
    c[5] = 0                                               # 899 is the end of window 4's rows
    q, s = run_quant(x, offsets=o, counts=c)
    rq, rs = quant_ref(x)
    filled = np.zeros(M, bool)
    for a, n in zip(off, c.tolist()):
        if 0 <= a < M and n > 0:
            filled[a:min(M, a + n)] = True
    assert np.array_equal(q[filled], rq[filled]) and np.array_equal(s[filled], rs[filled])
    assert (q[~filled] == 99).all() and (s[~filled] == -5).all()
    c[4] = 1000                                            # a window past the last row is cut
    q, s = run_quant(x, offsets=o, counts=c)
    assert np.array_equal(q[877:], rq[877:])


def test_quant_nothing_to_do():
    run_quant(torch.empty(0, 128, device="cuda"))
    q, s = run_quant(torch.empty(3, 0, device="cuda"))
    assert (s == -5).all()


def test_no_windows_are_not_all_rows(ws):
    """Empty offsets and counts have no address; they are refused, not read as
    a call without windows."""
    x = torch.ones(4, 128, device="cuda")
    q, s = torch.full((4, 128), 99, dtype=torch.int8, device="cuda"), torch.full((4,), -5.0, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((4, 128), -5.0, device="cuda")
    for o, c in ((none, none), (none, one), (one, none), (None, one), (one, None)):
        with pytest.raises(ValueError, match="offsets|counts"):
            moe.moe_quant_i8(x, q, s, offsets=o, counts=c)
        with pytest.raises(ValueError, match="offsets|counts|windows"):
            moe.moe_gemm_i8(q, s, q, s, y, ws, offsets=o, counts=c)
    assert (q == 99).all() and (s == -5).all() and (y == -5).all()


# ---------------------------------------------------------------- products --

def ints(shape, seed, full=False):
    return torch.randint(-127, 128, shape, generator=gen(seed), dtype=torch.int8) if not full else \
        torch.full(shape, -128 if seed % 2 else 127, dtype=torch.int8)


def gemm_ref(x, xs, w, ws_, wu=None, us=None):
    """(values, |g|) in 64 bits; x [M, K], w [N, K]."""
    xd, xs = x.double(), xs.double()[:, None]
    g = (xd @ w.double().t()) * ws_.double()[None] * xs
    if wu is None:
        return g, torch.zeros_like(g)
    u = (xd @ wu.double().t()) * us.double()[None] * xs
    return g * torch.sigmoid(g) * u, g.abs()


def close(y, ref, g, out, swiglu):
    rel = ((3 * (1 + g) + 10) * U) if swiglu else torch.full_like(ref, 3 * U)
    rel = rel + (2.0 ** -8 if out == "bf16" else 0)
    err = (y.double().cpu() - ref).abs()
    assert bool((err <= rel * ref.abs() * (1 + 2.0 ** -7) + 2.0 ** -126).all()), float((err / ref.abs().clamp_min(1e-30)).max())


def scales(n, seed, base):
    return base * (0.5 + torch.rand(n, generator=gen(seed)))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 128, 128), (1, 7168, 2048), (2, 64, 144), (16, 256, 1040),
                                   (17, 129, 4096), (64, 65, 272), (65, 1000, 528), (128, 128, 64), (129, 320, 2064),
                                   (300, 1001, 1552), (1000, 136, 96), (33, 2048, 7168), (257, 511, 400),
                                   (1, 100, 1040), (5, 40, 8192), (64, 130, 2064), (65, 300, 4112), (130, 64, 16384),
                                   (2000, 4100, 160), (200, 4096, 1024),
                                   (2, 5000, 528), (3, 2371, 1040), (4, 4099, 2064), (4, 70, 12288), (3, 16, 16400),
                                   (5, 4099, 2064), (8, 2400, 7168), (7, 300, 1040), (6, 2500, 16384), (1, 40, 98304),
                                   (9, 2400, 1040)])
def test_dense_product(M, N, K, up, out, ws):
    x, w = ints((M, K), M), ints((N, K), N)
    xs, wsc = scales(M, 1, 1 / 64), scales(N, 2, 0.05 / K ** 0.5)
    wu, us = (ints((N, K), N + 2), scales(N, 3, 0.05 / K ** 0.5)) if up else (None, None)
    y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
    dev = [None if t is None else t.cuda() for t in (x, xs, w, wsc, wu, us)]
    moe.moe_gemm_i8(*dev[:4], y, ws, w_up=dev[4], up_scale=dev[5])
    assert moe.moe_poll_status(ws) == 0
    close(y, *gemm_ref(x, xs, w, wsc, wu, us), out, up)


@pytest.mark.parametrize("K", [16, 131056])
def test_largest_sums_stay_exact(K, ws):
    """-128 * -128 * K, the largest sum: below 2^31 for every K accepted."""
    M, N = 3, 130
    x, w = ints((M, K), 1, True), ints((N, K), 1, True)
    x[1] = 127
    w[7] = 127
    one = torch.ones(max(M, N))
    y = torch.empty(M, N, device="cuda")
    moe.moe_gemm_i8(x.cuda(), one[:M].cuda(), w.cuda(), one[:N].cuda(), y, ws)
    assert moe.moe_poll_status(ws) == 0
    close(y, *gemm_ref(x, one[:M], w, one[:N]), "f32", False)


def windows(counts, gap, M=None):
    """Windows in order with `gap` rows between them."""
    off, at = [], gap
    for c in counts:
        off.append(at)
        at += c + gap
    return off, M or at


GROUPS = [
    dict(counts=[0, 1, 127, 128, 129, 0, 300, 16], gap=0, N=256, K=256),
    dict(counts=[5, 0, 3, 64, 65], gap=7, N=129, K=400),
    dict(counts=[0, 0, 0], gap=16, N=64, K=128),
    dict(counts=[4] * 40, gap=124, N=192, K=1024),
    dict(counts=[700], gap=1, N=320, K=528),
    dict(counts=[1] * 200 + [400], gap=0, N=48, K=96),
    dict(counts=[256, 257, 511, 33], gap=0, N=512, K=640),
    dict(counts=[90, 100, 128, 129, 65, 3, 200, 70], gap=1, N=1500, K=272),
    # many units: chunks of up to 288 rows, which go around tensor memory in every way
    dict(counts=[270, 257, 288, 289, 300, 550, 560, 31, 0, 700, 230, 576], gap=3, N=2600, K=320),
]


@pytest.mark.parametrize("fill", [0, 1, 1 << 40], ids=["fill0", "few", "many"])
@pytest.mark.parametrize("up,out", [(False, "bf16"), (True, "bf16"), (False, "f32"), (True, "f32")])
@pytest.mark.parametrize("g", GROUPS, ids=lambda g: f"E{len(g['counts'])}gap{g['gap']}N{g['N']}K{g['K']}")
def test_grouped_product(g, up, out, fill, ws):
    """Every window's rows, none of the others, whatever number of rows the
    caller expects."""
    E, N, K = len(g["counts"]), g["N"], g["K"]
    off, M = windows(g["counts"], g["gap"], M=20 if not sum(g["counts"]) else None)
    x, xs = ints((M, K), 3), scales(M, 4, 1 / 64)
    w, wsc = ints((E, N, K), 5), scales(E * N, 6, 0.05 / K ** 0.5).view(E, N)
    wu, us = (ints((E, N, K), 7), scales(E * N, 8, 0.05 / K ** 0.5).view(E, N)) if up else (None, None)
    y = torch.full((M, N), 77.0, dtype=DT[out], device="cuda")
    dev = [None if t is None else t.cuda() for t in (x, xs, w, wsc, wu, us)]
    o, c = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (off, g["counts"]))
    moe.moe_gemm_i8(*dev[:4], y, ws, w_up=dev[4], up_scale=dev[5], offsets=o, counts=c, fill=fill)
    assert moe.moe_poll_status(ws) == 0
    ref, gg = torch.full((M, N), 77.0, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    for e, (a, n) in enumerate(zip(off, g["counts"])):
        if n:
            ref[a:a + n], gg[a:a + n] = gemm_ref(x[a:a + n], xs[a:a + n], w[e], wsc[e], *(
                (wu[e], us[e]) if up else ()))
    filled = torch.zeros(M, dtype=torch.bool)
    for a, n in zip(off, g["counts"]):
        filled[a:a + n] = True
    close(y[filled.cuda()], ref[filled], gg[filled], out, up)
    assert bool((y[~filled.cuda()] == 77.0).all())


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_a_row_has_the_same_bits_in_any_company(up, out, ws):
    """Alone, among few or many rows, dense or in a window: whichever kernel and
    tiles that takes, the sums are exact and the arithmetic after them the same."""
    M, N, K = 1200, 3000, 3200
    x, xs = ints((M, K), 1).cuda(), scales(M, 2, 1 / 64).cuda()
    w, wsc = ints((N, K), 3).cuda(), scales(N, 4, 0.05 / K ** 0.5).cuda()
    wu, us = (ints((N, K), 5).cuda(), scales(N, 6, 0.05 / K ** 0.5).cuda()) if up else (None, None)
    full = torch.empty(M, N, dtype=DT[out], device="cuda")
    moe.moe_gemm_i8(x, xs, w, wsc, full, ws, w_up=wu, up_scale=us)
    for m in (1, 2, 4, 8, 9, 33, 64, 65, 200, 300, 700):
        a = (7 * m) % (M - m)
        y = torch.empty(m, N, dtype=DT[out], device="cuda")
        moe.moe_gemm_i8(x[a:a + m].clone(), xs[a:a + m].clone(), w, wsc, y, ws, w_up=wu, up_scale=us)
        assert torch.equal(y, full[a:a + m]), m
    three = dict(w_up=None if wu is None else wu.view(3, 1000, K), up_scale=None if us is None else us.view(3, 1000))
    off = torch.tensor([3, 700, 1000], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([290, 1, 150], dtype=torch.int32, device="cuda")
    for fill in (0, 3, 441):
        y = torch.empty(M, 1000, dtype=DT[out], device="cuda")
        moe.moe_gemm_i8(x, xs, w.view(3, 1000, K), wsc.view(3, 1000), y, ws, offsets=off, counts=cnt, fill=fill, **three)
        for e, (o, c) in enumerate(zip(off.tolist(), cnt.tolist())):
            assert torch.equal(y[o:o + c], full[o:o + c, 1000 * e:1000 * (e + 1)]), (fill, e)
    assert moe.moe_poll_status(ws) == 0


def test_windows_out_of_range_are_cut(ws):
    M, N, K = 200, 64, 128
    x, xs, w = ints((M, K), 1), scales(M, 2, 1.0), ints((5, N, K), 3)
    wsc = scales(5 * N, 4, 1.0).view(5, N)
    o = torch.tensor([-3, 150, 200, 2 ** 31 - 1, 10], dtype=torch.int32, device="cuda")
    c = torch.tensor([50, 2 ** 31 - 1, 4, 7, -2 ** 31], dtype=torch.int32, device="cuda")
    y = torch.full((M, N), 77.0, device="cuda")
    moe.moe_gemm_i8(x.cuda(), xs.cuda(), w.cuda(), wsc.cuda(), y, ws, offsets=o, counts=c)
    assert moe.moe_poll_status(ws) == 0
    assert bool((y[:150] == 77).all())
    close(y[150:], *gemm_ref(x[150:], xs[150:], w[1], wsc[1]), "f32", False)


def test_overlapping_windows_stay_in_bounds(ws):
    """Windows that overlap have unspecified rows, and nothing else changes:
    1024 windows over the same rows have more units than any that do not."""
    M, N, K, E = 3000, 8, 32, 1024
    x, xs = ints((M, K), 1).cuda(), torch.ones(M, device="cuda")
    w, wsc = ints((E, N, K), 3).cuda(), torch.ones(E, N, device="cuda")
    o = torch.full((E,), 100, dtype=torch.int32, device="cuda")
    c = torch.full((E,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    for fill in (0, 1):
        y = torch.full((M, N), 77.0, device="cuda")
        moe.moe_gemm_i8(x, xs, w, wsc, y, ws, offsets=o, counts=c, fill=fill)
        assert moe.moe_poll_status(ws) == 0
        assert bool((y[:100] == 77).all())
    q, s = run_quant(torch.randn(M, 64, device="cuda"), offsets=o, counts=c)
    assert (q[:100] == 99).all() and (s[:100] == -5).all()
    # a second window repeats the first: the same weights give the same rows twice
    o = torch.tensor([100, 100], dtype=torch.int32, device="cuda")
    c = torch.tensor([1000, 1000], dtype=torch.int32, device="cuda")
    y = torch.full((M, N), 77.0, device="cuda")
    moe.moe_gemm_i8(x, xs, w[:1].expand(2, N, K).contiguous(), wsc[:2], y, ws, offsets=o, counts=c)
    close(y[100:1100], *gemm_ref(x[100:1100].cpu(), torch.ones(1000), w[0].cpu(), torch.ones(N)), "f32", False)
    assert bool((y[1100:] == 77).all())


def test_nan_scale_reaches_its_row_only(ws):
    x, w = ints((5, 64), 1).cuda(), ints((9, 64), 2).cuda()
    xs, wsc = torch.ones(5, device="cuda"), torch.ones(9, device="cuda")
    xs[2] = float("nan")
    y = torch.empty(5, 9, device="cuda")
    moe.moe_gemm_i8(x, xs, w, wsc, y, ws)
    assert bool(torch.isnan(y[2]).all()) and not bool(torch.isnan(y[[0, 1, 3, 4]]).any())


@pytest.mark.slow
def test_offsets_past_32_bits(ws):
    """Elements of x and y past 2^31."""
    M, N, K = 1_100_000, 2048, 2048
    x = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    xs, wsc = torch.ones(M, device="cuda"), torch.ones(1, N, device="cuda")
    w = ints((1, N, K), 5).cuda()
    tail = ints((300, K), 6)
    x[-300:] = tail.cuda()
    o = torch.tensor([M - 300], dtype=torch.int32, device="cuda")
    c = torch.tensor([300], dtype=torch.int32, device="cuda")
    moe.moe_gemm_i8(x, xs, w, wsc, y, ws, offsets=o, counts=c, fill=300)
    assert moe.moe_poll_status(ws) == 0
    close(y[-300:], *gemm_ref(tail, torch.ones(300), w[0].cpu(), torch.ones(N)), "bf16", False)
    assert bool((y[-301] == 0).all())
    q, s = torch.empty_like(x), torch.empty(M, device="cuda")
    moe.moe_quant_i8(y, q, s)
    rq, rs = quant_ref(y[-300:])
    assert np.array_equal(q[-300:].cpu().numpy(), rq) and np.array_equal(s[-300:].cpu().numpy(), rs)


def test_streams_graphs_and_two_calls_at_once(ws):
    M, N, K = 200, 640, 1024
    x = torch.randn(M, K, generator=gen(1)).bfloat16().cuda()
    w, wsc = ints((N, K), 2).cuda(), scales(N, 3, 0.01).cuda()

    def linear(x, q, s, y):
        moe.moe_quant_i8(x, q, s)
        moe.moe_gemm_i8(q, s, w, wsc, y, ws)

    def bufs():
        return (torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
                torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))

    a, b = bufs(), bufs()
    linear(x, *a)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):                                     # side by side, one workspace
        with torch.cuda.stream(st):
            linear(x, *b)
        linear(x, *a)
    torch.cuda.synchronize()
    assert torch.equal(a[2], b[2])
    b[2].zero_()                                            # a stream given by argument
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_quant_i8(x, b[0], b[1], stream=st)
    moe.moe_gemm_i8(b[0], b[1], w, wsc, b[2], ws, stream=st)
    st.synchronize()
    assert torch.equal(a[2], b[2])
    sx, c = x.clone(), bufs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linear(sx, *c)
    for seed in (5, 6):
        new = torch.randn(M, K, generator=gen(seed)).bfloat16().cuda()
        sx.copy_(new)
        graph.replay()
        linear(new, *a)
        torch.cuda.synchronize()
        assert torch.equal(a[2], c[2])
    assert moe.moe_poll_status(ws) == 0


def test_first_calls_may_be_captured():
    """A process whose first calls are captured into a graph."""
    code = """
import torch
from combine_softmax_top_b200 import moe, workloads as W
s = W.spec("decode", T=40, E=64, k=4, H=128, I=128, compact=1)
sh, g = moe.make_shape(s), moe.make_gate("sigmoid", 8, 4, 2)
ws = torch.empty(moe.moe_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
moe.moe_workspace_init(sh, ws)
l, b = torch.randn(40, 64, device="cuda"), torch.zeros(64, device="cuda")
i, w = torch.empty(40, 4, dtype=torch.int32, device="cuda"), torch.empty(40, 4, device="cuda")
x = torch.randn(40, 256, device="cuda")
q, xs = torch.empty(40, 256, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
wt, wsc = torch.ones(2048, 256, dtype=torch.int8, device="cuda"), torch.ones(2048, device="cuda")
y, gl = torch.empty(40, 2048, device="cuda"), torch.empty_like(l)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.moe_gate(sh, g, l, b, i, w, ws)
    moe.moe_gate_backward(sh, g, l, i, w, gl)
    moe.moe_quant_i8(x, q, xs)
    moe.moe_gemm_i8(q, xs, wt, wsc, y, ws)
graph.replay()
torch.cuda.synchronize()
assert moe.moe_poll_status(ws) == 0
ref = (q.double().sum(1) * xs.double())[:, None].expand_as(y)
assert torch.allclose(y.double(), ref, rtol=1e-6, atol=1e-6), (y, ref)
assert abs(float(w.sum()) - 40) < 1e-3
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("compact", [0, 1])
@pytest.mark.parametrize("T", [1, 40, 700])
def test_int8_layer_of_the_stages(T, compact):
    """moe_gate, moe_dispatch (bf16 windows), int8 gate/up and down products
    with their quantisations, moe_combine, and back from the output to the
    logits, against the same layer in 64 bits on the same choice.

    Quantising h may step where its bf16 rounding does: a step of one part in
    127 of a row's largest value for a few elements. Rounding q itself is off by
    half a step: both sides do that alike, so only flips differ. The bound
    allows every element of h a bf16 rounding (2^-8) and one flip in eight."""
    s = W.spec("skew", T=T, H=256, E=16, k=4, I=384, zipf_s=0.0, compact=compact)
    b = moe.alloc_buffers(s)
    gate = moe.make_gate("sigmoid", groups=4, topk_groups=2, group_best=2, scale=2.0)
    x = torch.randn(T, s.H, generator=gen(1)).bfloat16().cuda()
    logits, bias = torch.randn(T, s.E, generator=gen(2)).cuda(), (torch.randn(s.E, generator=gen(3)) * 0.1).cuda()
    wg, wu, wd = (ints(sh, i) for i, sh in enumerate([(16, 384, 256), (16, 384, 256), (16, 256, 384)]))
    sg, su, sd = (scales(16 * n, 9 + i, 0.02 / 73).view(16, n) for i, n in enumerate([384, 384, 256]))
    rows = b.xq.shape[0]
    xq, xs = torch.empty(rows, s.H, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    hq, hs = torch.empty(rows, s.I, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    dev = lambda *ts: [t.cuda() for t in ts]  # noqa: E731
    dwg, dsg, dwu, dsu, dwd, dsd = dev(wg, sg, wu, su, wd, sd)
    win = dict(offsets=b.offsets, counts=b.counts)

    moe.moe_gate(b.shape, gate, logits, bias, b.topk_idx, b.topk_w, b.ws)
    bufs = b.dispatch_bufs()
    moe.moe_dispatch(b.shape, x, b.topk_idx, b.ws, bufs)
    moe.moe_quant_i8(b.xq, xq, xs, **win)
    moe.moe_gemm_i8(xq, xs, dwg, dsg, b.hq, b.ws, w_up=dwu, up_scale=dsu, fill=T * s.k, **win)
    moe.moe_quant_i8(b.hq, hq, hs, **win)
    moe.moe_gemm_i8(hq, hs, dwd, dsd, b.y, b.ws, fill=T * s.k, **win)
    moe.moe_combine(b.shape, bufs, b.y, b.topk_w, b.ws, b.out)
    assert moe.moe_poll_status(b.ws) == 0

    q, sc = quant_ref(x)
    xd = torch.from_numpy(q).double() * torch.from_numpy(sc).double()[:, None]
    idx, w = b.topk_idx.cpu().long(), b.topk_w.double().cpu()
    want, slack = torch.zeros(T, s.H, dtype=torch.float64), torch.zeros(T, s.H, dtype=torch.float64)
    y_pair = torch.zeros(T, s.k, s.H, dtype=torch.float64)
    for t in range(T):
        for j in range(s.k):
            e = int(idx[t, j])
            g = (wg[e].double() * sg[e].double()[:, None]) @ xd[t]
            u = (wu[e].double() * su[e].double()[:, None]) @ xd[t]
            h = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
            qh, sh_ = quant_ref(h[None])
            hd = torch.from_numpy(qh[0]).double() * float(sh_[0])
            wdd = wd[e].double() * sd[e].double()[:, None]
            y_pair[t, j] = wdd @ hd
            want[t] += w[t, j] * y_pair[t, j]
            flip = 2.0 ** -8 * hd.abs() + float(sh_[0]) / 8
            slack[t] += w[t, j] * (wdd.abs() @ flip + 2.0 ** -8 * y_pair[t, j].abs())
    err = (b.out.double().cpu() - want).abs()
    assert bool((err <= slack + 2.0 ** -8 * want.abs()).all())
    assert float(err.norm() / want.norm()) < 0.02       # h, y and out rounded to bf16: 3 * 2^-8 at most, and flips

    # training: d out -> d topk_w = <d out, y of the pair> -> d logits
    gout = torch.randn(T, s.H, generator=gen(4)).double()
    gw = torch.einsum("th,tjh->tj", gout, y_pair).float().cuda()
    gl = torch.empty_like(logits)
    moe.moe_gate_backward(b.shape, gate, logits, b.topk_idx, gw, gl)
    l = logits.double().cpu().requires_grad_(True)
    sel = torch.sigmoid(l).gather(1, idx)
    (gr,) = torch.autograd.grad((2.0 * sel / sel.sum(1, keepdim=True) * gw.double().cpu()).sum(), l)
    bound = 2 * (4 * 6 + 96) * U * 2 * 2 * gw.double().cpu().abs().sum(1, keepdim=True)
    assert bool(((gl.double().cpu() - gr).abs() <= bound).all())


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 16), (8, 2400, 32), (40, 200, 144), (64, 130, 8192), (300, 520, 272),
                                   (1200, 1040, 160)])
def test_swiglu_of_gates_far_below_zero(M, N, K, out, ws):
    """Gates of -127 .. 20, exact, against ups large enough that silu(g) u is a
    normal number where exp(-g) is beyond binary32."""
    x, w, wu = (torch.zeros(s, dtype=torch.int8) for s in ((M, K), (N, K), (N, K)))
    x[:, 3] = 1
    w[:, 3] = (torch.arange(N) % 148 - 127).to(torch.int8)
    wu[:, 3] = (torch.arange(N) % 251 - 125).to(torch.int8)
    one, us = torch.ones(max(M, N)), torch.full((N,), 2.0 ** 60)
    y = torch.empty(M, N, dtype=DT[out], device="cuda")
    dev = [t.cuda() for t in (x, one[:M], w, one[:N], wu, us)]
    moe.moe_gemm_i8(*dev[:4], y, ws, w_up=dev[4], up_scale=dev[5])
    assert moe.moe_poll_status(ws) == 0
    close(y, *gemm_ref(x, one[:M], w, one[:N], wu, us), out, True)


def test_first_call_on_few_sms_leaves_later_ones_the_device():
    """A process whose first product runs on a green context of a few SMs: the
    next ones, on the whole device, are spread over all of it (an eighth of the
    SMs at most against all: 8 times the rate; 3 times is asked for)."""
    code = """
import torch
from combine_softmax_top_b200 import moe, workloads as W
sh = moe.make_shape(W.spec("tiny"))
ws = torch.empty(moe.moe_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
moe.moe_workspace_init(sh, ws)
x, xs = torch.ones(4096, 4096, dtype=torch.int8, device="cuda"), torch.ones(4096, device="cuda")
w, wsc = torch.ones(4096, 4096, dtype=torch.int8, device="cuda"), torch.ones(4096, device="cuda")
y = torch.empty(4096, 4096, dtype=torch.bfloat16, device="cuda")
x1, w1, y1 = x[:128], w[:, :512].contiguous(), torch.empty(128, 4096, dtype=torch.bfloat16, device="cuda")
x1 = x1[:, :512].contiguous()
part = moe.GreenPartition(16, 0)
assert part.dispatch_sms * 8 <= part.dispatch_sms + part.main_sms
few = torch.cuda.ExternalStream(part.dispatch_stream)
forms = [lambda s: moe.moe_gemm_i8(x, xs, w, wsc, y, ws, stream=s),                  # a CTA pair a unit
         lambda s: moe.moe_gemm_i8(x1, xs[:128], w1, wsc, y1, ws, stream=s)]         # one CTA a unit

def us(f, s, n):
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = 1e30
    for _ in range(n):
        a.record(s); f(s); b.record(s); b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best

torch.cuda.synchronize()
times = [(us(f, few, 3), us(f, torch.cuda.current_stream(), 5)) for f in forms]
assert moe.moe_poll_status(ws) == 0
part.close()
print("times", times)
assert times[0][1] * 3 < times[0][0], times
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-2000:]


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("M,N,K,windows_of", [(2000, 4100, 160, 0), (1500, 1100, 272, 40), (700, 600, 2064, 150)])
def test_many_units_captured_and_on_few_sms(M, N, K, windows_of, up, ws):
    """More units than workers, so that the grid is asked for in the call: in a
    capture, and on a green context's stream; the same bits as on this one."""
    E = max(1, M // windows_of) if windows_of else 1
    x, xs = ints((M, K), 1).cuda(), scales(M, 2, 1 / 64).cuda()
    w, wsc = ints((E, N, K), 3).cuda(), scales(E * N, 4, 0.05 / K ** 0.5).view(E, N).cuda()
    kw = dict(w_up=ints((E, N, K), 5).cuda(), up_scale=scales(E * N, 6, 0.05 / K ** 0.5).view(E, N).cuda()) if up else {}
    if windows_of:
        off = torch.arange(E, dtype=torch.int32, device="cuda") * windows_of
        kw.update(offsets=off, counts=torch.full_like(off, windows_of))
    else:
        w, wsc = w[0], wsc[0]
        kw = {n: t[0] for n, t in kw.items()}
    ys = [torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    moe.moe_gemm_i8(x, xs, w, wsc, ys[0], ws, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_gemm_i8(x, xs, w, wsc, ys[1], ws, **kw)
    graph.replay()
    torch.cuda.synchronize()
    part = moe.GreenPartition(16, torch.cuda.current_device())
    try:
        moe.moe_gemm_i8(x, xs, w, wsc, ys[2], ws, stream=torch.cuda.ExternalStream(part.dispatch_stream), **kw)
        torch.cuda.synchronize()
    finally:
        part.close()
    assert moe.moe_poll_status(ws) == 0
    assert bool(ys[0].any()) and torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
