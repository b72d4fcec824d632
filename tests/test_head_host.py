"""Refusals of the head's operators (CPU only: no call here reaches a CUDA API), in the
library and in the binding."""
import pytest
import torch

import sparsity_step_b200 as B
from sparsity_step_b200 import _lib, head
from sparsity_step_b200.build import build

BAD = 0x1001          # a misaligned fake device address (never dereferenced)
GOOD = 0x10000        # an aligned fake device address (never dereferenced)
INVALID, SHAPE, ALIGN, SPACE = -1, -2, -3, -7


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


def err(L):
    return L.bitlinear_last_error().decode()


def quant(L, fn="bitlinear_fp8_quant", x=GOOD, t=16, c=64, fmt=0, q=GOOD, s=GOOD, qt=None, st=None):
    return getattr(L, fn)(x, t, c, fmt, q, s, qt, st, None)


@pytest.mark.parametrize("fn", ["bitlinear_fp8_quant", "bitlinear_fp8_quant_weight"])
def test_quant_refusals(L, fn):
    assert quant(L, fn, fmt=2) == INVALID and "format" in err(L)
    assert quant(L, fn, fmt=-1) == INVALID
    assert quant(L, fn, qt=GOOD) == INVALID and "both" in err(L)
    assert quant(L, fn, st=GOOD) == INVALID
    for missing in ("x", "q", "s"):
        assert quant(L, fn, **{missing: None}) == INVALID
    for crooked in ("x", "q", "s"):
        assert quant(L, fn, **{crooked: BAD}) == ALIGN
    assert quant(L, fn, qt=BAD, st=GOOD) == ALIGN and quant(L, fn, qt=GOOD, st=BAD) == ALIGN
    for c in (0, 8, 72, -16, 1 << 31):
        assert quant(L, fn, c=c) == SHAPE, c
    assert quant(L, fn, t=-1) == SHAPE


def test_quant_of_nothing(L):
    assert quant(L, t=0, x=None, q=None, s=None) == 0
    assert quant(L, t=(1 << 30) + 1) == SHAPE
    # weights follow the layer's shapes: n_out % 16, k_in % 64
    assert quant(L, "bitlinear_fp8_quant_weight", t=24) == SHAPE
    assert quant(L, "bitlinear_fp8_quant_weight", c=80) == SHAPE
    # more tiles than one launch counts
    assert quant(L, t=1 << 30, c=1 << 30) == SHAPE


def fwd(L, x=GOOD, xt=0, xs=GOOD, w=GOOD, wf=0, ws=GOOD, t=64, k=64, n=16, y=GOOD, yd=0, sp=None, nb=0):
    return L.bitlinear_fp8_fwd(x, xt, xs, w, wf, ws, t, k, n, y, yd, sp, nb, None)


def test_fwd_refusals(L):
    assert fwd(L, xt=3) == INVALID and fwd(L, wf=2) == INVALID and fwd(L, yd=2) == INVALID
    for missing in ("x", "xs", "w", "ws", "y"):
        assert fwd(L, **{missing: None}) == INVALID, missing
        assert fwd(L, **{missing: BAD}) == ALIGN, missing
    for k, n in ((32, 16), (100, 16), (131136, 16), (64, 8), (64, 24)):
        assert fwd(L, k=k, n=n) == SHAPE
    assert fwd(L, t=-1) == SHAPE and fwd(L, t=1 << 31) == SHAPE
    # bf16 activations of more than a few tokens need room for their codes
    need = L.bitlinear_fp8_fwd_workspace_size(64, 64, 2)
    assert need >= 64 * 64 + 64 * 4
    assert fwd(L, xt=2, xs=None) == SPACE and fwd(L, xt=2, xs=None, sp=GOOD, nb=need - 1) == SPACE
    assert fwd(L, xt=2, xs=None, sp=BAD, nb=need) == ALIGN
    assert L.bitlinear_fp8_fwd_workspace_size(64, 64, 0) == 0 and L.bitlinear_fp8_fwd_workspace_size(1, 64, 2) == 0
    assert fwd(L, t=0, x=None, xs=None, y=None) == 0


def bwd(L, dq=GOOD, ds=GOOD, dt=GOOD, dts=GOOD, df=0, xt=GOOD, xts=GOOD, xf=0, wt=GOOD, wts=GOOD, wf=0, t=16, k=64, n=16,
        gx=GOOD, gw=GOOD, gd=0):
    return L.bitlinear_fp8_bwd(dq, ds, dt, dts, df, xt, xts, xf, wt, wts, wf, t, k, n, gx, gw, gd, None)


def test_bwd_refusals(L):
    assert bwd(L, gx=None, gw=None) == INVALID and "request" in err(L)
    assert bwd(L, df=2) == INVALID and bwd(L, xf=2) == INVALID and bwd(L, wf=2) == INVALID and bwd(L, gd=2) == INVALID
    for part in ("dq", "ds", "wt", "wts"):
        assert bwd(L, gw=None, **{part: None}) == INVALID, part
    for part in ("dt", "dts", "xt", "xts"):
        assert bwd(L, gx=None, **{part: None}) == INVALID, part
    for part in ("dq", "ds", "dt", "dts", "xt", "xts", "wt", "wts", "gx", "gw"):
        assert bwd(L, **{part: BAD}) == ALIGN, part
    assert bwd(L, k=65) == SHAPE and bwd(L, n=17) == SHAPE and bwd(L, t=-1) == SHAPE
    assert bwd(L, t=0, gw=None, dq=None, ds=None) == 0


def ce_fwd(L, x=GOOD, w=GOOD, y=GOOD, t=4, k=64, v=100, loss=GOOD, lse=GOOD, sp=GOOD, nb=1 << 40):
    return L.bitlinear_linear_ce_fwd(x, w, y, t, k, v, loss, lse, sp, nb, None)


def ce_bwd(L, x=GOOD, w=GOOD, y=GOOD, lse=GOOD, g=GOOD, t=4, k=64, v=100, gx=GOOD, gw=GOOD, gd=0, sp=GOOD, nb=1 << 40):
    return L.bitlinear_linear_ce_bwd(x, w, y, lse, g, t, k, v, gx, gw, gd, sp, nb, None)


def test_linear_ce_refusals(L):
    for part in ("x", "w", "y", "loss", "lse"):
        assert ce_fwd(L, **{part: None}) == INVALID, part
        assert ce_fwd(L, **{part: BAD}) == ALIGN, part
    for part in ("x", "w", "y", "lse", "g"):
        assert ce_bwd(L, **{part: None}) == INVALID, part
        assert ce_bwd(L, **{part: BAD}) == ALIGN, part
    for f in (ce_fwd, ce_bwd):
        assert f(L, k=32) == SHAPE and f(L, k=65) == SHAPE and f(L, v=0) == SHAPE and f(L, v=(1 << 30) + 1) == SHAPE
        assert f(L, t=-1) == SHAPE and f(L, t=(1 << 30) + 1) == SHAPE
        assert f(L, sp=None) == SPACE and f(L, nb=16) == SPACE and f(L, sp=BAD) == ALIGN
    assert ce_bwd(L, gx=None, gw=None) == INVALID and ce_bwd(L, gd=2) == INVALID
    assert ce_bwd(L, gx=BAD) == ALIGN and ce_bwd(L, gw=BAD) == ALIGN
    assert ce_fwd(L, t=0, x=None, y=None, loss=None, lse=None, sp=None, nb=0) == 0
    assert ce_bwd(L, t=0, x=None, y=None, lse=None, g=None, gw=None, sp=None, nb=0) == 0


def test_linear_ce_workspace_is_far_from_the_logits(L):
    t, k, v = 8192, 2048, 65536
    assert L.bitlinear_linear_ce_fwd_workspace_size(t, v) < 2 * t * v // 16
    assert L.bitlinear_linear_ce_bwd_workspace_size(t, k, v, 1) < 2 * t * v // 3
    assert L.bitlinear_linear_ce_fwd_workspace_size(0, v) == 0 and L.bitlinear_linear_ce_bwd_workspace_size(0, k, v, 1) == 0


@pytest.mark.parametrize("v", [1, 1000, 1024, 1025, 2000, 4000, 32003, 65536])
@pytest.mark.parametrize("t", [1, 33, 8192, 16384, 57344, 65536, 1 << 20])
def test_linear_ce_workspace_is_what_the_header_states(L, t, v):
    # besides dl: a copy of x, six words a token and, with grad_x, its fp32 sum
    k, rows = 64, (t + 255) // 256 * 256
    dl = L.bitlinear_linear_ce_bwd_workspace_size(t, k, v, 0) - rows * (2 * k + 24) - 256
    mib, padded = 1 << 20, (v + 255) // 256 * 256
    whole = 2 * max(t, 64) * padded
    assert dl <= (whole if whole <= 64 * mib or v <= 1024 else 2 * max(112 * mib, 2048 * t)) + 1024
    sums = L.bitlinear_linear_ce_bwd_workspace_size(t, k, v, 1) - L.bitlinear_linear_ce_bwd_workspace_size(t, k, v, 0)
    assert sums % (rows * k * 4) == 0 and sums > 0 and (t < 74 * 256 or sums == rows * k * 4)


# ------------------------------------------------------------------ the binding

def test_binding_refuses_host_and_mistyped_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.bitlinear_fp8_quant(x)
    with pytest.raises(TypeError, match="bfloat16"):
        B.bitlinear_fp8_quant(x.float())
    with pytest.raises(TypeError, match="float32"):
        B.bitlinear_fp8_quant_weight(x)
    with pytest.raises(ValueError, match="two dimensions"):
        B.bitlinear_fp8_quant(x[0])
    with pytest.raises(TypeError, match="Tensor"):
        B.bitlinear_fp8_quant([1.0])
    wq, ws = torch.zeros(16, 64, dtype=torch.float8_e4m3fn), torch.zeros(1, 16, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        B.bitlinear_fp8_fwd(x, wq, ws)
    with pytest.raises(ValueError, match="x_scales"):
        B.bitlinear_fp8_fwd(x, wq, ws, x_scales=ws)
    with pytest.raises(ValueError, match="x_scales"):
        B.bitlinear_fp8_fwd(x.to(torch.float8_e4m3fn), wq, ws)
    with pytest.raises(TypeError, match="float8"):
        B.bitlinear_fp8_fwd(x.float(), wq, ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.bitlinear_linear_ce_fwd(x, x, torch.zeros(4, dtype=torch.int64))


def test_binding_wants_the_transposed_copies():
    q = {"q": torch.zeros(4, 64, dtype=torch.float8_e4m3fn), "scales": torch.zeros(1, 4, 4, dtype=torch.uint8)}
    with pytest.raises(ValueError, match="want_t"):
        B.bitlinear_fp8_bwd(q, q, q)
    with pytest.raises(ValueError, match="needs w"):
        B.bitlinear_fp8_bwd(q, q, None)
    with pytest.raises(ValueError, match="needs x"):
        B.bitlinear_fp8_bwd(q, None, q, want_grad_x=False)
    with pytest.raises(ValueError, match="request"):
        B.bitlinear_fp8_bwd(q, q, q, want_grad_x=False, want_grad_w=False)


def test_scales_shape():
    assert B.fp8_scales_shape(7, 64) == (1, 7, 4) and B.fp8_scales_shape(1, 513) == (2, 1, 4)
    assert B.fp8_scales_shape(5, 0) == (0, 5, 4)
    assert set(head.__all__) <= set(dir(head))


def test_own_workspace_is_recorded_on_a_given_stream():
    class Memory:
        stream = None

        def record_stream(self, stream):
            self.stream = stream

    class X:
        device = torch.device("cpu")

        def new_empty(self, shape, dtype):
            assert shape == (64,) and dtype == torch.uint8
            return Memory()

    side = object()
    assert head._workspace(None, 64, X(), side).stream is side
    assert head._workspace(None, 64, X(), None).stream is None
    assert head._workspace(None, 0, X(), side) is None


def test_memory_of_a_call_comes_from_its_stream(monkeypatch):
    current = ["current"]

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *exc):
            current.pop()

    class Memory:
        def __init__(self):
            self.pool, self.used_on = current[-1], []

        def record_stream(self, stream):
            self.used_on.append(stream)

    class X:
        device = torch.device("cuda", 0)

        def new_empty(self, shape, dtype):
            return Memory()

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: current[-1])
    for make in (head._empty, head._result):
        assert make(X(), (4,), torch.uint8, None).pool == "current" and make(X(), (4,), torch.uint8, "side").pool == "side"
    assert head._workspace(None, 64, X(), "side").pool == "side" and head._workspace(None, 64, X(), None).pool == "current"
    # results go on to the current stream
    assert head._result(X(), (4,), torch.uint8, "side").used_on == ["current"] and current == ["current"]
    assert head._result(X(), (4,), torch.uint8, None).used_on == []
