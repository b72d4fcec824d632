"""Python binding of the head's operators (include/bitlinear.h): the block-scaled 8-bit
float linear and the linear cross entropy. Argument checks and marshalling only, as in
``bitlinear.py``."""
from __future__ import annotations

import torch

from ._lib import BL_OUT_BF16, BL_OUT_F32, check, lib
from .bitlinear import _call, _need, _need_bytes, _need_vec, _ptr

BL_FP8_E4M3 = 0
BL_FP8_E5M2 = 1
BL_X_BF16 = 2
_FP8 = {torch.float8_e4m3fn: BL_FP8_E4M3, torch.float8_e5m2: BL_FP8_E5M2}


def _fmt(dtype, name: str) -> int:
    if dtype not in _FP8:
        raise TypeError(f"{name}: expected torch.float8_e4m3fn or torch.float8_e5m2, got {dtype}")
    return _FP8[dtype]


def _matrix(t, name: str) -> tuple[int, int]:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected two dimensions, got shape {tuple(t.shape)}")
    return int(t.shape[0]), int(t.shape[1])


def fp8_scales_shape(rows: int, cols: int) -> tuple[int, int, int]:
    """Shape of the scales of [rows, cols] codes: block b of row r at [b // 4, r, b % 4]."""
    return (cols + 511) // 512, rows, 4


def _rows16(rows: int) -> int:
    return (rows + 15) // 16 * 16


def _quant(fn, name: str, src, dtype, want_t: bool, fmt, out: dict | None, stream) -> dict:
    rows, cols = _matrix(src, name)
    _need(src, dtype, None, name)
    code, dev = _fmt(fmt, "fmt"), src.device
    o = dict(out or {})
    shapes = {"q": ((rows, cols), fmt), "scales": (fp8_scales_shape(rows, cols), torch.uint8)}
    if want_t:
        shapes["qt"] = ((cols, _rows16(rows)), fmt)
        shapes["scales_t"] = (fp8_scales_shape(cols, rows), torch.uint8)
    for key, (shape, dt) in shapes.items():
        if key not in o:
            o[key] = torch.empty(shape, dtype=dt, device=dev)
        _need(o[key], dt, shape, key, dev)
    st = _call(getattr(lib(), fn), dev, stream, _ptr(src), rows, cols, code, _ptr(o["q"]), _ptr(o["scales"]),
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
    return int(lib().bitlinear_fp8_fwd_workspace_size(t, k_in, x_type))


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
        _need(x_scales, torch.uint8, fp8_scales_shape(t, k_in), "x_scales", dev)
    _need(x, x.dtype, None, "x")
    w_fmt = _fmt(w_q.dtype, "w_q")
    _need(w_q, w_q.dtype, (n_out, k_in), "w_q", dev)
    _need(w_scales, torch.uint8, fp8_scales_shape(n_out, k_in), "w_scales", dev)
    if y is None:
        y = torch.empty((t, n_out), dtype=y_dtype, device=dev)
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"y: expected bfloat16 or float32, got {y.dtype}")
    _need(y, y.dtype, (t, n_out), "y", dev)
    need = int(lib().bitlinear_fp8_fwd_workspace_size(t, k_in, x_type))
    if need and workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need_bytes(workspace, need, "workspace", dev)
    st = _call(lib().bitlinear_fp8_fwd, dev, stream, _ptr(x), x_type, _ptr(x_scales), _ptr(w_q), w_fmt, _ptr(w_scales),
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
        _need(dy["q"], dy["q"].dtype, (t, n_out), "dy q", dev)
        _need(dy["scales"], torch.uint8, fp8_scales_shape(t, n_out), "dy scales", dev)
        w_fmt = _fmt(w["qt"].dtype, "w")
        _need(w["qt"], w["qt"].dtype, (k_in, n_out), "w qt", dev)
        _need(w["scales_t"], torch.uint8, fp8_scales_shape(k_in, n_out), "w scales_t", dev)
        if grad_x is None:
            grad_x = torch.empty((t, k_in), dtype=torch.bfloat16, device=dev)
        _need(grad_x, torch.bfloat16, (t, k_in), "grad_x", dev)
    if want_grad_w:
        _need(dy["qt"], dy["q"].dtype, (n_out, t16), "dy qt", dev)
        _need(dy["scales_t"], torch.uint8, fp8_scales_shape(n_out, t), "dy scales_t", dev)
        x_fmt = _fmt(x["qt"].dtype, "x")
        _need(x["qt"], x["qt"].dtype, (k_in, t16), "x qt", dev)
        _need(x["scales_t"], torch.uint8, fp8_scales_shape(k_in, t), "x scales_t", dev)
        if grad_w is None:
            grad_w = torch.empty((n_out, k_in), dtype=grad_w_dtype, device=dev)
        if grad_w.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"grad_w: expected bfloat16 or float32, got {grad_w.dtype}")
        _need(grad_w, grad_w.dtype, (n_out, k_in), "grad_w", dev)
    gwdt = BL_OUT_F32 if grad_w is not None and grad_w.dtype == torch.float32 else BL_OUT_BF16
    xp, wp = x if want_grad_w else {}, w if want_grad_x else {}
    dyt = dy if want_grad_w else {}
    st = _call(lib().bitlinear_fp8_bwd, dev, stream, _ptr(dy["q"]), _ptr(dy.get("scales")), _ptr(dyt.get("qt")),
               _ptr(dyt.get("scales_t")), dy_fmt, _ptr(xp.get("qt")), _ptr(xp.get("scales_t")), x_fmt, _ptr(wp.get("qt")),
               _ptr(wp.get("scales_t")), w_fmt, t, k_in, n_out, _ptr(grad_x), _ptr(grad_w), gwdt)
    check(st, "bitlinear_fp8_bwd")
    return grad_x, grad_w


def _check_ce(x, w, targets) -> tuple[int, int, int]:
    t, k_in = _matrix(x, "x")
    v = _matrix(w, "w")[0]
    _need(x, torch.bfloat16, None, "x")
    _need(w, torch.bfloat16, (v, k_in), "w", x.device)
    _need(targets, torch.int64, (t,), "targets", x.device)
    return t, k_in, v


def bitlinear_linear_ce_fwd_workspace_size(t: int, v: int) -> int:
    return int(lib().bitlinear_linear_ce_fwd_workspace_size(t, v))


def bitlinear_linear_ce_fwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, *,
                            loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Per-token softmax cross entropy of the logits x . w^T (x bf16 [t, k_in], w bf16
    [v, k_in], targets int64 [t]) without storing them; returns (loss, lse), fp32 [t].
    A token whose target is outside [0, v) has loss 0 and no gradient."""
    t, k_in, v = _check_ce(x, w, targets)
    dev = x.device
    if loss is None:
        loss = torch.empty((t,), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((t,), dtype=torch.float32, device=dev)
    _need(loss, torch.float32, (t,), "loss", dev)
    _need(lse, torch.float32, (t,), "lse", dev)
    need = bitlinear_linear_ce_fwd_workspace_size(t, v)
    if need and workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need_bytes(workspace, need, "workspace", dev)
    st = _call(lib().bitlinear_linear_ce_fwd, dev, stream, _ptr(x), _ptr(w), _ptr(targets), t, k_in, v, _ptr(loss),
               _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.numel())
    check(st, "bitlinear_linear_ce_fwd")
    return loss, lse


def bitlinear_linear_ce_bwd_workspace_size(t: int, k_in: int, v: int, want_grad_x: bool = True) -> int:
    return int(lib().bitlinear_linear_ce_bwd_workspace_size(t, k_in, v, int(want_grad_x)))


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
    _need_vec(lse, torch.float32, t, "lse", dev)
    _need_vec(grad_loss, torch.float32, t, "grad_loss", dev)
    if want_grad_x and grad_x is None:
        grad_x = torch.empty((t, k_in), dtype=torch.bfloat16, device=dev)
    if want_grad_w and grad_w is None:
        grad_w = torch.empty((v, k_in), dtype=grad_w_dtype, device=dev)
    if grad_x is not None:
        _need(grad_x, torch.bfloat16, (t, k_in), "grad_x", dev)
    if grad_w is not None:
        if grad_w.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"grad_w: expected bfloat16 or float32, got {grad_w.dtype}")
        _need(grad_w, grad_w.dtype, (v, k_in), "grad_w", dev)
    gwdt = BL_OUT_F32 if grad_w is not None and grad_w.dtype == torch.float32 else BL_OUT_BF16
    need = bitlinear_linear_ce_bwd_workspace_size(t, k_in, v, grad_x is not None)
    if need and workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need_bytes(workspace, need, "workspace", dev)
    st = _call(lib().bitlinear_linear_ce_bwd, dev, stream, _ptr(x), _ptr(w), _ptr(targets), _ptr(lse), _ptr(grad_loss), t,
               k_in, v, _ptr(grad_x), _ptr(grad_w), gwdt, _ptr(workspace), 0 if workspace is None else workspace.numel())
    check(st, "bitlinear_linear_ce_bwd")
    return grad_x, grad_w


__all__ = [
    "BL_FP8_E4M3", "BL_FP8_E5M2", "BL_X_BF16", "fp8_scales_shape", "bitlinear_fp8_quant", "bitlinear_fp8_quant_weight",
    "bitlinear_fp8_fwd_workspace_size", "bitlinear_fp8_fwd", "bitlinear_fp8_bwd", "bitlinear_linear_ce_fwd_workspace_size",
    "bitlinear_linear_ce_fwd", "bitlinear_linear_ce_bwd_workspace_size", "bitlinear_linear_ce_bwd",
]
