"""Plain CPU oracle of the head's operators: block-scaled 8-bit float linears and the
linear cross entropy, in numpy and 64 bits, straight from their definitions
(include/bitlinear.h). Shares no code with the product; tests only.
"""
from __future__ import annotations

import numpy as np

MANTISSA = {"e4m3": 3, "e5m2": 2}
BIAS = {"e4m3": 7, "e5m2": 15}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
NAN_CODE = 0x7F


def code_value(code: int, fmt: str) -> float:
    """Value of one 8-bit code, read off its sign, exponent and mantissa fields."""
    mb = MANTISSA[fmt]
    sign = -1.0 if code & 0x80 else 1.0
    exp, man = (code & 0x7F) >> mb, code & ((1 << mb) - 1)
    if fmt == "e4m3" and (code & 0x7F) == 0x7F:
        return float("nan")
    if fmt == "e5m2" and exp == 31:
        return sign * float("inf") if man == 0 else float("nan")
    if exp == 0:
        return sign * man * 2.0 ** (1 - BIAS[fmt] - mb)
    return sign * (1.0 + man / 2.0 ** mb) * 2.0 ** (exp - BIAS[fmt])


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    return np.array([code_value(c, fmt) for c in range(256)])[codes]


def encode(values: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest code of values within the format's range, ties to the even code."""
    v = np.array([code_value(c, fmt) for c in range(128)])
    v = v[np.isfinite(v)]                       # ascending, code = index
    mag = np.abs(values)
    hi = np.clip(np.searchsorted(v, mag), 1, len(v) - 1)
    lo = hi - 1
    up, down = v[hi] - mag, mag - v[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (pick | np.where(np.signbit(values), 0x80, 0)).astype(np.uint8)


def block_exponent(amax: float, fmt: str) -> int:
    """Smallest e >= -127 with amax <= top * 2^e, by trial."""
    if amax == 0.0:
        return -127
    e = int(np.floor(np.log2(amax / TOP[fmt]))) - 2
    while TOP[fmt] * 2.0 ** e < amax:
        e += 1
    return max(e, -127)


def fp8_quant(x: np.ndarray, fmt: str, block_rows: int = 1):
    """(codes uint8 [r, c], scale bytes uint8 [ceil(c / 512), r, 4], values fp64 [r, c])."""
    x = x.astype(np.float64)
    r, c = x.shape
    codes = np.zeros((r, c), np.uint8)
    scales = np.zeros(((c + 511) // 512, r, 4), np.uint8)
    values = np.zeros((r, c))
    for r0 in range(0, r, block_rows):
        for b in range((c + 127) // 128):
            rows, cols = slice(r0, min(r0 + block_rows, r)), slice(128 * b, min(128 * b + 128, c))
            blk = x[rows, cols]
            if not np.all(np.isfinite(blk)):
                codes[rows, cols], scales[b // 4, rows, b % 4], values[rows, cols] = NAN_CODE, 255, np.nan
                continue
            e = block_exponent(float(np.max(np.abs(blk))), fmt)
            q = encode(blk * 2.0 ** -e, fmt)
            codes[rows, cols], scales[b // 4, rows, b % 4] = q, e + 127
            values[rows, cols] = decode(q, fmt) * 2.0 ** e
    return codes, scales, values


def fp8_quant_both(x: np.ndarray, fmt: str, block_rows: int = 1) -> dict:
    """Codes and scales along the rows and of the transposed copy padded to 16 rows."""
    q, s, v = fp8_quant(x, fmt, block_rows)
    xt = np.zeros((x.shape[1], (x.shape[0] + 15) // 16 * 16))
    xt[:, : x.shape[0]] = x.T
    qt, st, vt = fp8_quant(xt, fmt, block_rows)
    return {"q": q, "scales": s, "values": v, "qt": qt, "scales_t": st, "values_t": vt}


def linear_ce(x: np.ndarray, w: np.ndarray, targets: np.ndarray, grad_loss: np.ndarray | None = None) -> dict:
    """Loss, log-sum-exp and, with grad_loss, dl and both gradients."""
    x, w = x.astype(np.float64), w.astype(np.float64)
    logits = x @ w.T
    top = logits.max(axis=1, keepdims=True)
    lse = (top + np.log(np.exp(logits - top).sum(axis=1, keepdims=True)))[:, 0]
    live = (targets >= 0) & (targets < w.shape[0])
    rows = np.arange(x.shape[0])
    loss = np.zeros(x.shape[0])
    loss[live] = lse[live] - logits[rows[live], targets[live]]
    out = {"logits": logits, "lse": lse, "loss": loss, "live": live}
    if grad_loss is not None:
        p = np.exp(logits - lse[:, None])
        dl = p.copy()
        dl[rows[live], targets[live]] -= 1.0
        g = np.where(live, grad_loss.astype(np.float64), 0.0)[:, None]
        dl = np.where(g == 0.0, 0.0, dl * g)
        out.update(p=np.where(g == 0.0, 0.0, p * np.abs(g)), dl=dl, grad_x=dl @ w, grad_w=dl.T @ x)
    return out
