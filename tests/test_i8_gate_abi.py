"""What the gate and the int8 products refuse, on the host and before any CUDA
call (no GPU needed), and what they accept as nothing to do."""
import ctypes

import pytest
import torch

from combine_softmax_top_b200 import moe
from combine_softmax_top_b200 import workloads as W

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = ctypes.c_void_p(1 << 20)          # an aligned address that nothing reads
ODD = ctypes.c_void_p((1 << 20) + 8)


def _shape(**over):
    sh = moe.make_shape(W.spec("sweep", T=4, H=128, E=64, k=4, xq=W.BF16))
    for f, v in over.items():
        setattr(sh, f, v)
    return sh


def _gate(**over):
    g = moe.make_gate("sigmoid", groups=8, topk_groups=4, group_best=2, scale=2.5)
    for f, v in over.items():
        setattr(g, f, v)
    return g


def _call_gate(sh, g, logits=P, bias=P, idx=P, w=P, ws=P):
    return moe.lib().moe_gate(ctypes.byref(sh), None if g is None else ctypes.byref(g), logits, bias, idx, w, ws, None)


def _call_back(sh, g, logits=P, idx=P, gw=P, gl=P):
    return moe.lib().moe_gate_backward(ctypes.byref(sh), None if g is None else ctypes.byref(g), logits, idx, gw, gl,
                                       None)


@pytest.mark.parametrize("over,code", [
    (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(logits_dtype=7), INVALID),
    (dict(logits_dtype=moe.MOE_E4M3), UNSUPPORTED), (dict(logits_dtype=moe.MOE_E2M1), INVALID),
    (dict(groups=0), INVALID), (dict(groups=64), INVALID), (dict(groups=7), INVALID),
    (dict(topk_groups=0), INVALID), (dict(topk_groups=9), INVALID), (dict(group_best=0), INVALID),
    (dict(group_best=3), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
])
def test_gate_refuses_descriptions(over, code):
    assert _call_gate(_shape(), _gate(**over)) == code
    assert _call_back(_shape(), _gate(**over)) == code


def test_gate_refuses_shapes_and_pointers():
    assert _call_gate(_shape(), None) == INVALID
    assert _call_gate(_shape(topk=0), _gate()) == INVALID
    most = moe.make_shape(W.spec("sweep", T=(1 << 31) - 60, H=128, E=1, k=1, xq=W.BF16, compact=0))
    most.cap_rows = 128
    one = _gate(groups=1, topk_groups=1, group_best=1)
    assert _call_gate(most, one) == INVALID and _call_back(most, one) == INVALID
    # 4 open groups of 8 experts hold 32, one open group 8
    assert _call_gate(_shape(topk=9), _gate(topk_groups=1)) == INVALID
    assert _call_back(_shape(topk=9), _gate(topk_groups=1)) == INVALID
    # groups of one expert have no second best
    assert _call_gate(_shape(E=32), _gate(groups=32, topk_groups=32)) == INVALID
    for bad in (dict(logits=None), dict(idx=None), dict(w=None), dict(logits=ODD), dict(bias=ODD), dict(idx=ODD),
                dict(w=ODD), dict(ws=None), dict(ws=ODD)):
        assert _call_gate(_shape(), _gate(), **bad) == INVALID, bad
    for bad in (dict(logits=None), dict(idx=None), dict(gw=None), dict(gl=None), dict(logits=ODD), dict(idx=ODD),
                dict(gw=ODD), dict(gl=ODD)):
        assert _call_back(_shape(), _gate(), **bad) == INVALID, bad
    assert _call_back(_shape(T=0), _gate(), None, None, None, None) == OK


def _quant(rows=4, cols=128, dt=moe.MOE_BF16, x=P, experts=0, offsets=None, counts=None, q=P, scale=P):
    return moe.lib().moe_quant_i8(rows, cols, dt, x, experts, offsets, counts, q, scale, None)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(cols=-16), INVALID), (dict(cols=8), INVALID),
    (dict(cols=130), INVALID), (dict(cols=(1 << 24) + 16), INVALID), (dict(dt=9), INVALID),
    (dict(dt=moe.MOE_E4M3), UNSUPPORTED), (dict(x=None), INVALID), (dict(q=None), INVALID),
    (dict(scale=None), INVALID), (dict(x=ODD), INVALID), (dict(q=ODD), INVALID), (dict(scale=ODD), INVALID),
    (dict(experts=4), INVALID), (dict(experts=4, offsets=P), INVALID), (dict(experts=4, counts=P), INVALID),
    (dict(experts=0, offsets=P, counts=P), INVALID), (dict(experts=1025, offsets=P, counts=P), INVALID),
    (dict(experts=-1, offsets=P, counts=P), INVALID),
    (dict(rows=0, x=None, q=None, scale=None), OK), (dict(cols=0, x=None, q=None, scale=None), OK),
])
def test_quant_refusals(over, code):
    assert _quant(**over) == code


def _gemm(M=4, N=128, K=128, experts=1, fill=0, out=moe.MOE_BF16, reserved=0, x=P, xs=P, w=P, ws_=P, wu=None, us=None,
          off=None, cnt=None, y=P, ws=P):
    d = moe.moe_gemm_i8_desc(M, N, K, experts, fill, out, reserved)
    return moe.lib().moe_gemm_i8(ctypes.byref(d), x, xs, w, ws_, wu, us, off, cnt, y, ws, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=(1 << 31) - 1, N=1 << 12), INVALID), (dict(M=(1 << 31) - 511, N=1), INVALID),
    (dict(M=-1), INVALID), (dict(M=1 << 31), INVALID), (dict(N=0), INVALID), (dict(N=1 << 31), INVALID),
    (dict(K=0), INVALID), (dict(K=24), INVALID), (dict(K=131072), INVALID), (dict(fill=-1), INVALID),
    (dict(reserved=1), INVALID), (dict(out=moe.MOE_E4M3), UNSUPPORTED), (dict(out=11), INVALID),
    (dict(experts=0), INVALID), (dict(experts=2), INVALID), (dict(experts=2, off=P), INVALID),
    (dict(experts=2, cnt=P), INVALID), (dict(experts=1, off=P), INVALID),
    (dict(experts=1025, off=P, cnt=P), INVALID), (dict(experts=1024, N=1 << 21, off=P, cnt=P), INVALID),
    (dict(wu=P), INVALID), (dict(us=P), INVALID), (dict(ws=None), INVALID), (dict(ws=ODD), INVALID),
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(w=None), INVALID), (dict(ws_=None), INVALID),
    (dict(y=None), INVALID), (dict(x=ODD), INVALID), (dict(xs=ODD), INVALID), (dict(w=ODD), INVALID),
    (dict(ws_=ODD), INVALID), (dict(y=ODD), INVALID), (dict(wu=ODD, us=P), INVALID), (dict(wu=P, us=ODD), INVALID),
    (dict(M=0, x=None, xs=None, w=None, ws_=None, y=None), OK),
])
def test_gemm_refusals(over, code):
    assert _gemm(**over) == code
    if code == INVALID and "ws" not in over:
        assert moe.lib().moe_gemm_i8(None, P, P, P, P, None, None, None, None, P, P, None) == INVALID


def test_python_binding_refuses_what_the_library_cannot_see():
    """Tensors off the device, strided, or of another type or shape."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="moe_quant_i8: x must be on the current CUDA device"):
        moe.moe_quant_i8(x, torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="moe_gemm_i8: x must be on the current CUDA device"):
        moe.moe_gemm_i8(x, None, torch.zeros(2, 8, 128, dtype=torch.int8), None, x, None,
                        offsets=torch.zeros(3, dtype=torch.int32), counts=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="x must be"):
        moe.moe_gemm_i8(x[0], None, x, None, x, None)
    with pytest.raises(ValueError, match="logits"):
        moe.moe_gate(_shape(), _gate(), torch.zeros(4, 64), None, None, None, None)
    with pytest.raises(KeyError):
        moe.make_gate("softmin")


class _FakeLibrary:
    """Takes every call and notes the workspace's address."""

    def __init__(self):
        self.seen = []

    def moe_gate(self, *args):
        self.seen.append(args[-2])
        return OK

    moe_gemm_i8 = moe_gate


@pytest.mark.parametrize("call", ["moe_gate", "moe_gemm_i8"])
def test_python_binding_refuses_workspaces_it_cannot_write_to(call, monkeypatch):
    """The library latches errors into a workspace's first 256 bytes: host memory, a
    shorter tensor or a strided one never get that far. Host tensors stand for
    the current device's here (device -1), and a fake for the library."""
    fake = _FakeLibrary()
    monkeypatch.setattr(moe, "lib", lambda: fake)
    monkeypatch.setattr(moe, "_begin", lambda fn, name, t, stream: (-1, 0))

    def run(ws):
        if call == "moe_gate":
            moe.moe_gate(_shape(), _gate(), torch.zeros(4, 64), None, torch.zeros(4, 4, dtype=torch.int32),
                         torch.zeros(4, 4), ws)
        else:
            moe.moe_gemm_i8(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4), torch.zeros(8, 128, dtype=torch.int8),
                            torch.zeros(8), torch.zeros(4, 8), ws)

    good = torch.zeros(256, dtype=torch.uint8)
    run(good)
    run(torch.zeros(64, dtype=torch.int32))
    assert fake.seen[0] == good.data_ptr() and len(fake.seen) == 2
    for bad in (None, torch.zeros(255, dtype=torch.uint8), torch.zeros(0, dtype=torch.uint8),
                torch.zeros(1024, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match=f"{call}: ws must be"):
            run(bad)
    monkeypatch.setattr(moe, "_dense", lambda fn, name, t, shape, dtypes, dev: t.data_ptr())
    monkeypatch.setattr(moe, "_begin", lambda fn, name, t, stream: (0, 0))   # device 0 is current, ws is the host's
    with pytest.raises(ValueError, match=f"{call}: ws must be"):
        run(good)
    assert len(fake.seen) == 2


@pytest.mark.parametrize("over", [
    # units (chunks of 64 rows, one more an expert, times tiles of 64 channels) that
    # 32 bits do not count: by the channels, and by the experts alone
    dict(M=(1 << 31) - 512, N=4097, K=16),
    dict(M=(1 << 31) - 512, N=4096, K=16, experts=9, off=P, cnt=P),
])
def test_gemm_refuses_more_units_than_32_bits(over):
    assert _gemm(**over) == INVALID


def test_gate_refuses_more_than_32_groups():
    """Where nothing else about 64 groups of one expert is wrong."""
    g = _gate(groups=64, topk_groups=64, group_best=1)
    assert _call_gate(_shape(), g) == INVALID and _call_back(_shape(), g) == INVALID
