"""Python binding of the head's operators (include/bitlinear.h): the block-scaled 8-bit
float linear and the linear cross entropy. Argument checks and marshalling only, as in
``bitlinear.py``."""
from __future__ import annotations

import functools

import torch

from ._lib import BL_OUT_BF16, BL_OUT_F32, check, lib
from .bitlinear import _call, _empty, _need, _need_bytes, _ptr, _result

BL_FP8_E4M3 = 0
BL_FP8_E5M2 = 1
BL_X_BF16 = 2
_FP8 = {torch.float8_e4m3fn: BL_FP8_E4M3, torch.float8_e5m2: BL_FP8_E5M2}


def _fmt(dtype, name: str) -> int:
    if dtype not in _FP8:
        raise TypeError(f"{name}: expected torch.float8_e4m3fn or torch.float8_e5m2, got {dtype}")
    return _FP8[dtype]


def _check(t, dtype, shape, name: str, dev) -> None:
    """``_need`` with its passing case first: a single-token call is short enough for its
    checks to count."""
    if (getattr(t, "dtype", None) == dtype and t.shape == shape and t.device == dev and dev.type == "cuda"
            and t.is_contiguous()):
        return
    _need(t, dtype, shape, name, dev)


def _launch(fn, dev: torch.device, stream, *args) -> int:
    """``_call``, without the stream object where the tensors' device is current and the
    call goes to its current stream."""
    if stream is None and torch.cuda.current_device() == dev.index:
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    return _call(fn, dev, stream, *args)


def _matrix(t, name: str) -> tuple[int, int]:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected two dimensions, got shape {tuple(shape)}")
    return shape[0], shape[1]


@functools.lru_cache(maxsize=4096)
def _size(fn: str, *args) -> int:
    """A workspace size (a function of the arguments alone)."""
    return int(getattr(lib(), fn)(*args))


def _workspace(given, need: int, x: torch.Tensor, stream):
    """The caller's workspace, or one of this call. The latter goes back to the allocator as
    soon as the call returns: work on a stream other than the current one has to be over
    before its memory is handed out again."""
    if given is not None:
        _need_bytes(given, need, "workspace", x.device)
        return given
    if not need:
        return None
    own = _empty(x, (need,), torch.uint8, stream)
    if stream is not None:
        own.record_stream(stream)
    return own


def fp8_scales_shape(rows: int, cols: int) -> tuple[int, int, int]:
    """Shape of the scales of [rows, cols] codes: block b of row r at [b // 4, r, b % 4]."""
    return (cols + 511) // 512, rows, 4


def _rows16(rows: int) -> int:
    return (rows + 15) // 16 * 16


def _quant(fn, name: str, src, dtype, want_t: bool, fmt, out: dict | None, stream) -> dict:
    rows, cols = _matrix(src, name)
    code, dev = _fmt(fmt, "fmt"), src.device
    _check(src, dtype, (rows, cols), name, dev)
    o = dict(out or {})
    shapes = {"q": ((rows, cols), fmt), "scales": (fp8_scales_shape(rows, cols), torch.uint8)}
    if want_t:
        shapes["qt"] = ((cols, _rows16(rows)), fmt)
        shapes["scales_t"] = (fp8_scales_shape(cols, rows), torch.uint8)
    for key, (shape, dt) in shapes.items():
        if key in o:
            _check(o[key], dt, shape, key, dev)
        else:
            o[key] = _result(src, shape, dt, stream)
    st = _launch(getattr(lib(), fn), dev, stream, _ptr(src), rows, cols, code, _ptr(o["q"]), _ptr(o["scales"]),
               _ptr(o["qt"]) if want_t else None, _ptr(o["scales_t"]) if want_t else None)
    check(st, fn)
    return o


def bitlinear_fp8_quant(x: torch.Tensor, *, want_t: bool = False, fmt=torch.float8_e4m3fn, out: dict | None = None,
                        stream=None) -> dict:
    """8-bit float codes of activations or output gradients x [t, cols] (bf16), one
    power-of-two scale per token and 128 columns.

    Returns a dict with ``q`` (``fmt`` [t, cols]) and ``scales`` (uint8,
    ``fp8_scales_shape(t, cols)``) and, with ``want_t``, the transposed copy for the
    backward products: ``qt`` (``fmt`` [cols, t rounded up to 16]) and ``scales_t``, one
    scale per column and 128 tokens. Buffers given in ``out`` are filled in place."""
    return _quant("bitlinear_fp8_quant", "x", x, torch.bfloat16, want_t, fmt, out, stream)


def bitlinear_fp8_quant_weight(w: torch.Tensor, *, want_t: bool = False, fmt=torch.float8_e4m3fn,
                               out: dict | None = None, stream=None) -> dict:
    """8-bit float codes of weights w [n_out, k_in] (fp32) with one power-of-two scale per
    128 x 128 block; the dict of ``bitlinear_fp8_quant`` (``qt`` is [k_in, n_out])."""
    return _quant("bitlinear_fp8_quant_weight", "w", w, torch.float32, want_t, fmt, out, stream)


def bitlinear_fp8_fwd_workspace_size(t: int, k_in: int, x_dtype=torch.bfloat16) -> int:
    x_type = BL_X_BF16 if x_dtype == torch.bfloat16 else _fmt(x_dtype, "x_dtype")
    return _size("bitlinear_fp8_fwd_workspace_size", t, k_in, x_type)


def bitlinear_fp8_fwd(x: torch.Tensor, w_q: torch.Tensor, w_scales: torch.Tensor, *,
                      x_scales: torch.Tensor | None = None, y_dtype=torch.bfloat16, y: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [t, n_out] = x . w^T from block-scaled codes. ``x`` is bf16 (quantised to e4m3 by
    the call) or 8-bit codes with their ``x_scales``; ``w_q`` and ``w_scales`` come from
    ``bitlinear_fp8_quant_weight``."""
    t, k_in = _matrix(x, "x")
    n_out = _matrix(w_q, "w_q")[0]
    dev = x.device
    if x.dtype == torch.bfloat16:
        x_type = BL_X_BF16
        if x_scales is not None:
            raise ValueError("x_scales belongs to 8-bit x")
    else:
        x_type = _fmt(x.dtype, "x")
        if x_scales is None:
            raise ValueError("8-bit x needs x_scales")
        _check(x_scales, torch.uint8, fp8_scales_shape(t, k_in), "x_scales", dev)
    _check(x, x.dtype, (t, k_in), "x", dev)
    w_fmt = _fmt(w_q.dtype, "w_q")
    _check(w_q, w_q.dtype, (n_out, k_in), "w_q", dev)
    _check(w_scales, torch.uint8, fp8_scales_shape(n_out, k_in), "w_scales", dev)
    if y is None:
        y = _result(x, (t, n_out), y_dtype, stream)
    else:
        _check(y, y.dtype, (t, n_out), "y", dev)
    if y.dtype != torch.bfloat16 and y.dtype != torch.float32:
        raise TypeError(f"y: expected bfloat16 or float32, got {y.dtype}")
    need = _size("bitlinear_fp8_fwd_workspace_size", t, k_in, x_type) if x_type == BL_X_BF16 else 0
    workspace = _workspace(workspace, need, x, stream)
    st = _launch(lib().bitlinear_fp8_fwd, dev, stream, _ptr(x), x_type, _ptr(x_scales), _ptr(w_q), w_fmt, _ptr(w_scales),
               t, k_in, n_out, _ptr(y), BL_OUT_F32 if y.dtype == torch.float32 else BL_OUT_BF16, _ptr(workspace),
               0 if workspace is None else workspace.numel())
    check(st, "bitlinear_fp8_fwd")
    return y


def bitlinear_fp8_bwd(dy: dict, x: dict | None, w: dict | None, *, want_grad_x: bool = True, want_grad_w: bool = True,
                      grad_w_dtype=torch.bfloat16, grad_x: torch.Tensor | None = None,
                      grad_w: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """Gradients of ``bitlinear_fp8_fwd``; returns (grad_x or None, grad_w or None).

    ``dy``, ``x`` and ``w`` are the dicts of ``bitlinear_fp8_quant`` (dy, x) and
    ``bitlinear_fp8_quant_weight`` (w), all made with ``want_t``. grad_x needs dy and w,
    grad_w needs dy and x."""
    t, n_out = _matrix(dy["q"], "dy q")
    dev = dy["q"].device
    want_grad_x, want_grad_w = want_grad_x or grad_x is not None, want_grad_w or grad_w is not None
    if want_grad_x and w is None:
        raise ValueError("grad_x needs w")
    if want_grad_w and x is None:
        raise ValueError("grad_w needs x")
    if not want_grad_x and not want_grad_w:
        raise ValueError("request grad_x, grad_w or both")
    for part, name, on in ((x, "x", want_grad_w), (w, "w", want_grad_x), (dy, "dy", want_grad_w)):
        if on and ("qt" not in part or "scales_t" not in part):
            raise ValueError(f"{name}: needs its transposed copy (want_t=True)")
    k_in = _matrix(w["qt"] if want_grad_x else x["qt"], "qt")[0]
    t16 = _rows16(t)
    dy_fmt = _fmt(dy["q"].dtype, "dy")
    x_fmt = w_fmt = BL_FP8_E4M3
    if want_grad_x:
        _check(dy["q"], dy["q"].dtype, (t, n_out), "dy q", dev)
        _check(dy["scales"], torch.uint8, fp8_scales_shape(t, n_out), "dy scales", dev)
        w_fmt = _fmt(w["qt"].dtype, "w")
        _check(w["qt"], w["qt"].dtype, (k_in, n_out), "w qt", dev)
        _check(w["scales_t"], torch.uint8, fp8_scales_shape(k_in, n_out), "w scales_t", dev)
        if grad_x is None:
            grad_x = _result(dy["q"], (t, k_in), torch.bfloat16, stream)
        _check(grad_x, torch.bfloat16, (t, k_in), "grad_x", dev)
    if want_grad_w:
        _check(dy["qt"], dy["q"].dtype, (n_out, t16), "dy qt", dev)
        _check(dy["scales_t"], torch.uint8, fp8_scales_shape(n_out, t), "dy scales_t", dev)
        x_fmt = _fmt(x["qt"].dtype, "x")
        _check(x["qt"], x["qt"].dtype, (k_in, t16), "x qt", dev)
        _check(x["scales_t"], torch.uint8, fp8_scales_shape(k_in, t), "x scales_t", dev)
        if grad_w is None:
            grad_w = _result(dy["q"], (n_out, k_in), grad_w_dtype, stream)
        if grad_w.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"grad_w: expected bfloat16 or float32, got {grad_w.dtype}")
        _check(grad_w, grad_w.dtype, (n_out, k_in), "grad_w", dev)
    gwdt = BL_OUT_F32 if grad_w is not None and grad_w.dtype == torch.float32 else BL_OUT_BF16
    xp, wp = x if want_grad_w else {}, w if want_grad_x else {}
    dyt = dy if want_grad_w else {}
    st = _launch(lib().bitlinear_fp8_bwd, dev, stream, _ptr(dy["q"]), _ptr(dy.get("scales")), _ptr(dyt.get("qt")),
               _ptr(dyt.get("scales_t")), dy_fmt, _ptr(xp.get("qt")), _ptr(xp.get("scales_t")), x_fmt, _ptr(wp.get("qt")),
               _ptr(wp.get("scales_t")), w_fmt, t, k_in, n_out, _ptr(grad_x), _ptr(grad_w), gwdt)
    check(st, "bitlinear_fp8_bwd")
    return grad_x, grad_w


def _check_ce(x, w, targets) -> tuple[int, int, int]:
    t, k_in = _matrix(x, "x")
    v = _matrix(w, "w")[0]
    _check(x, torch.bfloat16, (t, k_in), "x", x.device)
    _check(w, torch.bfloat16, (v, k_in), "w", x.device)
    _check(targets, torch.int64, (t,), "targets", x.device)
    return t, k_in, v


def bitlinear_linear_ce_fwd_workspace_size(t: int, v: int) -> int:
    return _size("bitlinear_linear_ce_fwd_workspace_size", t, v)


def bitlinear_linear_ce_fwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, *,
                            loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Per-token softmax cross entropy of the logits x . w^T (x bf16 [t, k_in], w bf16
    [v, k_in], targets int64 [t]) without storing them; returns (loss, lse), fp32 [t].
    A token whose target is outside [0, v) has loss 0 and no gradient."""
    t, k_in, v = _check_ce(x, w, targets)
    dev = x.device
    if loss is None:
        loss = _result(x, (t,), torch.float32, stream)
    else:
        _check(loss, torch.float32, (t,), "loss", dev)
    if lse is None:
        lse = _result(x, (t,), torch.float32, stream)
    else:
        _check(lse, torch.float32, (t,), "lse", dev)
    need = bitlinear_linear_ce_fwd_workspace_size(t, v)
    workspace = _workspace(workspace, need, x, stream)
    st = _launch(lib().bitlinear_linear_ce_fwd, dev, stream, _ptr(x), _ptr(w), _ptr(targets), t, k_in, v, _ptr(loss),
               _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.numel())
    check(st, "bitlinear_linear_ce_fwd")
    return loss, lse


def bitlinear_linear_ce_bwd_workspace_size(t: int, k_in: int, v: int, want_grad_x: bool = True) -> int:
    return _size("bitlinear_linear_ce_bwd_workspace_size", t, k_in, v, int(want_grad_x))


def bitlinear_linear_ce_bwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                            grad_loss: torch.Tensor, *, want_grad_x: bool = True, want_grad_w: bool = True,
                            grad_w_dtype=torch.bfloat16, grad_x: torch.Tensor | None = None,
                            grad_w: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                            stream=None) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """Gradients of ``bitlinear_linear_ce_fwd`` with respect to x (bf16) and w
    (``grad_w_dtype``), given its ``lse`` and ``grad_loss`` [t] (fp32), the derivative of
    the total with respect to each token's loss; returns (grad_x or None, grad_w or None)."""
    t, k_in, v = _check_ce(x, w, targets)
    dev = x.device
    _check(lse, torch.float32, (t,), "lse", dev)
    _check(grad_loss, torch.float32, (t,), "grad_loss", dev)
    if want_grad_x and grad_x is None:
        grad_x = _result(x, (t, k_in), torch.bfloat16, stream)
    if want_grad_w and grad_w is None:
        grad_w = _result(x, (v, k_in), grad_w_dtype, stream)
    if grad_x is not None:
        _check(grad_x, torch.bfloat16, (t, k_in), "grad_x", dev)
    if grad_w is not None:
        if grad_w.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"grad_w: expected bfloat16 or float32, got {grad_w.dtype}")
        _check(grad_w, grad_w.dtype, (v, k_in), "grad_w", dev)
    gwdt = BL_OUT_F32 if grad_w is not None and grad_w.dtype == torch.float32 else BL_OUT_BF16
    need = bitlinear_linear_ce_bwd_workspace_size(t, k_in, v, grad_x is not None)
    workspace = _workspace(workspace, need, x, stream)
    st = _launch(lib().bitlinear_linear_ce_bwd, dev, stream, _ptr(x), _ptr(w), _ptr(targets), _ptr(lse), _ptr(grad_loss), t,
               k_in, v, _ptr(grad_x), _ptr(grad_w), gwdt, _ptr(workspace), 0 if workspace is None else workspace.numel())
    check(st, "bitlinear_linear_ce_bwd")
    return grad_x, grad_w


__all__ = [
    "BL_FP8_E4M3", "BL_FP8_E5M2", "BL_X_BF16", "fp8_scales_shape", "bitlinear_fp8_quant", "bitlinear_fp8_quant_weight",
    "bitlinear_fp8_fwd_workspace_size", "bitlinear_fp8_fwd", "bitlinear_fp8_bwd", "bitlinear_linear_ce_fwd_workspace_size",
    "bitlinear_linear_ce_fwd", "bitlinear_linear_ce_bwd_workspace_size", "bitlinear_linear_ce_bwd",
]
