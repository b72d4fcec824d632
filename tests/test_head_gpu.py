"""GPU parity of the head's operators against the oracle in 64 bits.

Tolerances. Codes and scales are exact. A product of codes is exact in fp32 and each
addition of the accumulation is off by at most 2^-23 of the magnitudes summed so far (a
truncating adder; a rounding one is twice as good): with S = sum |a b| and one addition
per MMA of depth d plus the adds inside it (log2 d levels), |error| <= (K / d + log2 d) 2^-23 S.
bf16 outputs add half a step, 2^-8 relative. dl is rounded to bf16 once, half a step again.
"""
import numpy as np
import pytest
import torch

import sparsity_step_b200 as B
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu
FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BF16 = 2.0 ** -8
U = 2.0 ** -23
INF = float("inf")


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def bf16(rng, *shape, scale=1.0, outliers=True):
    """bf16-valued fp32 array: N(0, scale) with 1% of entries 20 times as large."""
    x = rng.normal(size=shape).astype(np.float32) * scale
    if outliers:
        x = np.where(rng.random(shape) < 0.01, x * 20, x)
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy()


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def acc_bound(k, depth, s):
    return (k / depth + np.log2(depth) + 1) * U * s


def check_quant(got, want, with_t):
    assert np.array_equal(u8(got["scales"]), want["scales"])
    assert np.array_equal(u8(got["q"]), want["q"])
    if with_t:
        assert np.array_equal(u8(got["scales_t"]), want["scales_t"])
        assert np.array_equal(u8(got["qt"]), want["qt"])


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("t,c", [(1, 16), (1, 64), (3, 2048), (16, 128), (17, 144), (100, 208), (128, 512), (129, 528),
                                 (300, 1088), (513, 64)])
def test_quant(t, c, fmt):
    rng = np.random.default_rng(t * 1000 + c)
    x = bf16(rng, t, c) * np.exp2(rng.integers(-6, 6, (t, 1))).astype(np.float32)
    x[t // 2, c // 2:] = 0.0
    want = H.fp8_quant_both(x, fmt)
    xd = dev(x, torch.bfloat16)
    check_quant(B.bitlinear_fp8_quant(xd, want_t=True, fmt=FMT[fmt]), want, True)
    check_quant(B.bitlinear_fp8_quant(xd, fmt=FMT[fmt]), want, False)


def test_quant_extremes():
    # borders of the scale, denormals, the largest values, an all-zero block, infinities and NaN
    x = np.zeros((9, 256), np.float32)
    x[0, :2] = [448.0, -448.0]
    x[1, :2] = [450.0, 1.0]
    x[2, 0] = 1.75
    x[3, 0] = 1.7578125
    x[4, 0] = 2.0 ** -133
    x[5, :128] = 3.3895314e38
    x[6, 7] = np.inf
    x[7, 200] = np.nan
    x[8, 130:140] = 2.0 ** -126
    x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    got = B.bitlinear_fp8_quant(dev(x, torch.bfloat16), want_t=True)
    check_quant(got, H.fp8_quant(x, "e4m3") and dict(zip(("q", "scales"), H.fp8_quant(x, "e4m3")[:2])), False)
    want = H.fp8_quant_both(x, "e4m3")
    assert np.array_equal(u8(got["scales_t"]), want["scales_t"])
    fine = want["scales_t"][0, :, 0] != 255
    assert np.array_equal(u8(got["qt"])[fine], want["qt"][fine])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("n,k", [(16, 64), (48, 128), (128, 192), (144, 576), (272, 1088)])
def test_quant_weight(n, k, fmt):
    rng = np.random.default_rng(n + k)
    w = (rng.normal(size=(n, k)) * 0.02).astype(np.float32)
    w[:, :64] *= 1e-3
    want = H.fp8_quant_both(w, fmt, 128)
    check_quant(B.bitlinear_fp8_quant_weight(dev(w), want_t=True, fmt=FMT[fmt]), want, True)
    check_quant(B.bitlinear_fp8_quant_weight(dev(w), fmt=FMT[fmt]), want, False)


# ------------------------------------------------------------------ 8-bit products

def product_close(y, a, b, k):
    """y against a . b^T of code values."""
    want, s = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = acc_bound(k, 32, s) + (BF16 * np.abs(want) if y.dtype == torch.bfloat16 else 0.0)
    err = np.abs(f64(y) - want)
    worst = np.max(err / np.maximum(tol, 1e-300))
    assert worst <= 1.0, f"worst error {worst:.3f} of its bound"


SHAPES = [(1, 64, 16), (1, 2048, 48), (2, 192, 16), (7, 1088, 32), (8, 576, 64), (9, 128, 16), (16, 640, 80), (17, 64, 48),
          (32, 1024, 240), (33, 64, 16), (33, 1088, 256), (100, 576, 224), (128, 192, 512), (255, 128, 240), (257, 704, 272),
          (600, 2112, 1040)]


@pytest.mark.parametrize("t,k,n", SHAPES)
def test_fwd(t, k, n):
    rng = np.random.default_rng(t + k + n)
    x, w = bf16(rng, t, k), (rng.normal(size=(n, k)) * 0.02).astype(np.float32)
    w[: n // 2] *= 30.0   # blocks and rows with scales of their own
    xo, wo = H.fp8_quant(x, "e4m3")[2], H.fp8_quant(w, "e4m3", 128)[2]
    xd, wq = dev(x, torch.bfloat16), B.bitlinear_fp8_quant_weight(dev(w))
    y = B.bitlinear_fp8_fwd(xd, wq["q"], wq["scales"])
    product_close(y, xo, wo, k)
    xq = B.bitlinear_fp8_quant(xd)
    y32 = B.bitlinear_fp8_fwd(xq["q"], wq["q"], wq["scales"], x_scales=xq["scales"], y_dtype=torch.float32)
    product_close(y32, xo, wo, k)
    assert B.bitlinear_device_status()[0] == 0


# few tokens: row blocks that one CTA walks over, K split by 2, 4 and 8, a ragged last row
# block, the widest K that still fits beside the weights and ones that do not
FEW_SHAPES = [(1, 192, 40016), (3, 64, 19008), (16, 2048, 11008), (32, 2048, 4112), (17, 1088, 2064), (8, 11008, 2064),
              (1, 320, 16), (20, 24640, 48), (20, 39936, 32), (8, 131072, 16), (129, 1088, 48), (300, 4096, 144), (512, 576, 272)]


@pytest.mark.parametrize("t,k,n", FEW_SHAPES)
def test_fwd_few_tokens(t, k, n):
    rng = np.random.default_rng(t + k + n)
    x, w = bf16(rng, t, k), (rng.normal(size=(n, k)) * 0.02).astype(np.float32)
    w[n // 3:] *= 5.0
    xd, wq = dev(x, torch.bfloat16), B.bitlinear_fp8_quant_weight(dev(w))
    xo = H.fp8_quant(x, "e4m3")[2]
    wo = H.decode(u8(wq["q"]), "e4m3") * np.exp2(u8(wq["scales"]).transpose(1, 0, 2).reshape(n, -1).astype(np.float64) - 127.0
                                                 ).repeat(128, 1)[:, :k]
    y = B.bitlinear_fp8_fwd(xd, wq["q"], wq["scales"], y_dtype=torch.float32)
    product_close(y, xo, wo, k)
    xq = B.bitlinear_fp8_quant(xd)
    assert torch.equal(B.bitlinear_fp8_fwd(xq["q"], wq["q"], wq["scales"], x_scales=xq["scales"], y_dtype=torch.float32), y)
    assert B.bitlinear_device_status()[0] == 0


@pytest.mark.parametrize("xf,wf", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("t", [3, 12, 20, 150])
def test_fwd_formats(t, xf, wf):
    k, n = 704, 144
    rng = np.random.default_rng(t)
    x, w = bf16(rng, t, k), (rng.normal(size=(n, k)) * 0.02).astype(np.float32)
    xo, wo = H.fp8_quant(x, xf)[2], H.fp8_quant(w, wf, 128)[2]
    xd, wq = dev(x, torch.bfloat16), B.bitlinear_fp8_quant_weight(dev(w), fmt=FMT[wf])
    xq = B.bitlinear_fp8_quant(xd, fmt=FMT[xf])
    product_close(B.bitlinear_fp8_fwd(xq["q"], wq["q"], wq["scales"], x_scales=xq["scales"], y_dtype=torch.float32), xo, wo, k)
    if xf == "e5m2":
        product_close(B.bitlinear_fp8_fwd(xd, wq["q"], wq["scales"]), H.fp8_quant(x, "e4m3")[2], wo, k)


@pytest.mark.parametrize("t", [2, 20, 64])
def test_fwd_row_scales_and_not_finite_rows(t):
    # every row and block of both operands with a scale of its own, one row with an infinity:
    # that token's outputs are NaN, the others are what they would be without it
    k, n = 1088, 272
    rng = np.random.default_rng(9)
    x = bf16(rng, t, k, outliers=False) * np.exp2(rng.integers(-20, 20, (t, 1))).astype(np.float32)
    x[:, 128:256] *= 2.0 ** 9
    w = (rng.normal(size=(n, k))).astype(np.float32) * np.exp2(np.repeat(rng.integers(-9, 9, (n + 127) // 128), 128)[:n, None]).astype(np.float32)
    wq = B.bitlinear_fp8_quant_weight(dev(w))
    clean = B.bitlinear_fp8_fwd(dev(x, torch.bfloat16), wq["q"], wq["scales"], y_dtype=torch.float32)
    product_close(clean, H.fp8_quant(x, "e4m3")[2], H.fp8_quant(w, "e4m3", 128)[2], k)
    x[1, 700] = np.inf
    y = B.bitlinear_fp8_fwd(dev(x, torch.bfloat16), wq["q"], wq["scales"], y_dtype=torch.float32)
    assert torch.isnan(y[1]).all()
    keep = torch.arange(t, device="cuda") != 1
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("t", [3, 40, 300])
def test_fwd_extreme_scales(t):
    # scales near both ends that cancel in the product, blocks and rows of zeros
    k, n = 640, 272
    rng = np.random.default_rng(t)
    x = bf16(rng, t, k, outliers=False) * 2.0 ** 90
    w = (rng.normal(size=(n, k)) * 2.0 ** -95).astype(np.float32)
    x[0], x[:, 256:384], w[128:256, 384:512] = 0.0, 0.0, 0.0
    x[1] *= np.float32(2.0 ** -150)   # zeros too: half of the least fp32 number rounds to even
    x[2] *= np.float32(2.0 ** -100)
    xd, wq = dev(x, torch.bfloat16), B.bitlinear_fp8_quant_weight(dev(w))
    x = f64(xd)
    y = B.bitlinear_fp8_fwd(xd, wq["q"], wq["scales"], y_dtype=torch.float32)
    product_close(y, H.fp8_quant(x, "e4m3")[2], H.fp8_quant(w, "e4m3", 128)[2], k)
    assert not y[:2].any() and y[2].any()


@pytest.mark.parametrize("t,k,n,df", [(1, 64, 16, "e4m3"), (5, 128, 48, "e5m2"), (16, 576, 224, "e4m3"), (37, 192, 1040, "e5m2"),
                                      (130, 1088, 256, "e4m3"), (600, 704, 272, "e5m2"), (1025, 320, 528, "e4m3")])
def test_bwd(t, k, n, df):
    rng = np.random.default_rng(t + n)
    x, dy = bf16(rng, t, k), bf16(rng, t, n, scale=1e-2, outliers=False)
    w = (rng.normal(size=(n, k)) * 0.02).astype(np.float32)
    dyo, xo, wo = H.fp8_quant_both(dy, df), H.fp8_quant_both(x, "e4m3"), H.fp8_quant_both(w, "e4m3", 128)
    dyq = B.bitlinear_fp8_quant(dev(dy, torch.bfloat16), want_t=True, fmt=FMT[df])
    xq = B.bitlinear_fp8_quant(dev(x, torch.bfloat16), want_t=True)
    wq = B.bitlinear_fp8_quant_weight(dev(w), want_t=True)
    gx, gw = B.bitlinear_fp8_bwd(dyq, xq, wq, grad_w_dtype=torch.float32)
    product_close(gx, dyo["values"], wo["values_t"], n)
    product_close(gw, dyo["values_t"], xo["values_t"], t + 32)
    gx2, none = B.bitlinear_fp8_bwd(dyq, None, wq, want_grad_w=False)
    assert none is None and torch.equal(gx2, gx)
    none, gw2 = B.bitlinear_fp8_bwd(dyq, xq, None, want_grad_x=False)
    assert none is None and torch.equal(gw2, gw.to(torch.bfloat16))
    assert B.bitlinear_device_status()[0] == 0


@pytest.mark.parametrize("t,k,n", [(48, 128, 16), (300, 4864, 896), (700, 2048, 4096), (2100, 1088, 2064), (4095, 512, 4864)])
@pytest.mark.parametrize("dw", [torch.bfloat16, torch.float32])
def test_bwd_together_and_apart(t, k, n, dw):
    # both gradients from one call (one launch where both take the pair product) are those of two
    gen = torch.Generator(device="cuda").manual_seed(t)
    x = B.bitlinear_fp8_quant(torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16), want_t=True)
    dy = B.bitlinear_fp8_quant(torch.randn(t, n, generator=gen, device="cuda").to(torch.bfloat16), want_t=True,
                               fmt=torch.float8_e5m2)
    w = B.bitlinear_fp8_quant_weight(torch.randn(n, k, generator=gen, device="cuda"), want_t=True)
    gx, gw = B.bitlinear_fp8_bwd(dy, x, w, grad_w_dtype=dw)
    gx1, none = B.bitlinear_fp8_bwd(dy, x, w, want_grad_w=False)
    assert none is None and torch.equal(gx, gx1)
    none, gw1 = B.bitlinear_fp8_bwd(dy, x, w, want_grad_x=False, grad_w_dtype=dw)
    assert none is None and torch.equal(gw, gw1) and gw.any()
    rows = torch.arange(0, n, max(1, n // 16), device="cuda")   # some rows against 64 bits
    codes = lambda d, r: d["qt"][:, :t].double() * torch.exp2(   # values of a transposed copy
        d["scales_t"].permute(1, 0, 2).reshape(r, -1)[:, :(t + 127) // 128].double() - 127.0).repeat_interleave(128, 1)[:, :t]
    product_close(gw[rows], f64(codes(dy, n)[rows]), f64(codes(x, k)), (t + 15) // 16 * 16)
    assert B.bitlinear_device_status()[0] == 0


def test_fp8_empty_batch():
    w = B.bitlinear_fp8_quant_weight(torch.randn(32, 128, device="cuda"), want_t=True)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    xq = B.bitlinear_fp8_quant(x, want_t=True)
    assert B.bitlinear_fp8_fwd(x, w["q"], w["scales"]).shape == (0, 32)
    dyq = B.bitlinear_fp8_quant(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), want_t=True)
    gw = torch.ones(32, 128, dtype=torch.float32, device="cuda")
    gx, gw = B.bitlinear_fp8_bwd(dyq, xq, w, grad_w=gw)
    assert gx.shape == (0, 128) and not gw.any()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quant_extremes_of_both_formats(fmt):
    # as above, against each format's own ends: its largest values and the next above, the
    # scale's least byte and the fp32 values below it, an infinity, a NaN of either sign
    top = H.TOP[fmt]
    x = np.zeros((12, 272), np.float32)
    x[0, :2], x[1, :2] = [top, -top], [top * (1 + 2.0 ** -7), 1.0]
    x[2, 0], x[3, 0] = 1.75, 1.7578125
    x[4, 0], x[5, 3], x[6, 0] = 2.0 ** -133, 2.0 ** -126, top * 2.0 ** -127
    x[7, :128] = 3.3895314e38
    x[8, 7], x[9, 200], x[10, 260], x[11, 130] = np.inf, np.nan, -np.inf, -np.nan
    x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    got = B.bitlinear_fp8_quant(dev(x, torch.bfloat16), want_t=True, fmt=FMT[fmt])
    want = H.fp8_quant_both(x, fmt)
    check_quant(got, want, False)
    assert np.array_equal(u8(got["scales_t"]), want["scales_t"])
    fine = want["scales_t"][0, :, 0] != 255
    assert np.array_equal(u8(got["qt"])[fine], want["qt"][fine]) and np.all(u8(got["qt"])[~fine][:, :12] == H.NAN_CODE)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quant_weight_extremes(fmt):
    # one block of weights each: an infinity, a NaN, zeros, the largest fp32 values, values
    # around the least scale and below fp32's normal ones, the format's own ends
    top = H.TOP[fmt]
    w = np.zeros((144, 1088), np.float32)
    w[3, 5], w[140, 130] = np.inf, np.nan
    w[:, 256:384] = 3.4028235e38 * np.linspace(-1, 1, 144, dtype=np.float32)[:, None]
    w[7, 384:387] = [top * 2.0 ** -127, 2.0 ** -130, -2.0 ** -149]
    w[9, 512:514] = [2.0 ** -140, 2.0 ** -149]
    w[130, 640:642], w[5, 640:642] = [top, -top], [np.nextafter(np.float32(top), np.float32(np.inf)), 1.0]
    w[:, 768:896] = -np.nan
    w[143, 1087] = -np.inf
    got, want = B.bitlinear_fp8_quant_weight(dev(w), want_t=True, fmt=FMT[fmt]), H.fp8_quant_both(w, fmt, 128)
    check_quant(got, want, True)


@pytest.mark.parametrize("xf,wf", [("e4m3", "e4m3"), ("e5m2", "e5m2"), ("e4m3", "e5m2")])
@pytest.mark.parametrize("t", [2, 20, 64, 300])
def test_products_of_not_finite_blocks(t, xf, wf):
    # forward and both gradients: what a block with an infinity or NaN enters is NaN, in either
    # operand and format, and the rest is what it is without it
    k, n = 640, 272
    rng = np.random.default_rng(21)
    x, dy = bf16(rng, t, k), bf16(rng, t, n, outliers=False)
    w = rng.normal(size=(n, k)).astype(np.float32)

    def run(x, w, dy):
        xq = B.bitlinear_fp8_quant(dev(x, torch.bfloat16), want_t=True, fmt=FMT[xf])
        wq = B.bitlinear_fp8_quant_weight(dev(w), want_t=True, fmt=FMT[wf])
        dq = B.bitlinear_fp8_quant(dev(dy, torch.bfloat16), want_t=True, fmt=FMT[xf])
        y = B.bitlinear_fp8_fwd(xq["q"], wq["q"], wq["scales"], x_scales=xq["scales"], y_dtype=torch.float32)
        return [f64(a) for a in (y, *B.bitlinear_fp8_bwd(dq, xq, wq, grad_w_dtype=torch.float32))]

    clean = run(x, w, dy)
    x[1, 300], dy[0, 17], w[130, 5] = np.inf, np.nan, -np.inf
    got = run(x, w, dy)
    y, gx, gw = (np.isnan(a) for a in got)
    rows, cols = np.arange(t), np.arange(n)
    assert np.array_equal(y, (rows == 1)[:, None] | ((cols >= 128) & (cols < 256))[None, :])
    # w's block (rows 128 to 255, columns 0 to 127) enters grad_x's columns 0 to 127
    assert np.array_equal(gx, (rows == 0)[:, None] | (np.arange(k) < 128)[None, :])
    assert np.array_equal(gw, (cols == 17)[:, None] | (np.arange(k) == 300)[None, :])
    for a, b in zip(got, clean):
        assert np.array_equal(a[~np.isnan(a)], b[~np.isnan(a)])


# ------------------------------------------------------------------ linear cross entropy

def ce_inputs(t, k, v, seed, logit_std=2.0):
    rng = np.random.default_rng(seed)
    x, w = bf16(rng, t, k, outliers=False), bf16(rng, v, k, scale=logit_std / np.sqrt(k), outliers=False)
    y = rng.integers(0, v, t)
    y[rng.random(t) < 0.2] = -100
    if t > 4:
        y[1], y[2], y[3] = v, v - 1, 0     # just outside, the last and the first
    g = rng.normal(size=t).astype(np.float32)
    return x, w, y.astype(np.int64), g


def logit_errors(x, w, k):
    """Bound on each token's largest logit error."""
    return acc_bound(k, 16, np.abs(x).astype(np.float64) @ np.abs(w).astype(np.float64).T).max(axis=1)


def check_loss(loss, lse, o, d):
    # lse moves by at most the largest logit error; its exponentials and sums add a few
    # units, its fp32 value and the base-2 scaling two units of its magnitude
    tol = d + 2.0 ** -20 + 4 * U * np.maximum(np.abs(o["lse"]), np.abs(o["logits"]).max(axis=1))
    assert np.all(np.abs(f64(lse) - o["lse"]) <= tol)
    assert np.all(np.abs(f64(loss) - o["loss"]) <= 2 * tol)
    assert np.all(f64(loss)[~o["live"]] == 0.0)


CE_SHAPES = [(1, 64, 1), (1, 2048, 1000), (2, 128, 2), (3, 64, 255), (8, 192, 256), (9, 64, 257), (32, 576, 31), (33, 64, 33),
             (100, 128, 5003), (255, 320, 640), (257, 1088, 1031), (300, 64, 12289),
             (1, 2048, 40001), (32, 64, 50001), (17, 1088, 5003), (5, 11008, 300), (32, 8192, 1000), (20, 2112, 19)]


@pytest.mark.parametrize("t,k,v", CE_SHAPES)
def test_linear_ce(t, k, v):
    x, w, y, g = ce_inputs(t, k, v, t + v)
    o = H.linear_ce(x, w, y, g)
    xd, wd, yd, gd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y), dev(g)
    loss, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    d = logit_errors(x, w, k)
    check_loss(loss, lse, o, d)
    gx, gw = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd)
    check_ce_grads(gx, gw, x, w, o, d, k, v, t)
    gx2, none = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd, want_grad_w=False)
    assert none is None and torch.equal(gx2, gx)
    none, gw32 = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd, want_grad_x=False, grad_w_dtype=torch.float32)
    assert none is None and torch.equal(gw32.to(torch.bfloat16), gw)
    assert B.bitlinear_device_status()[0] == 0


def check_ce_grads(gx, gw, x, w, o, d, k, v, t):
    """dl: half a bf16 step, plus p times what the exponent is off by (logit and lse errors
    and their base-2 scaling); then the products' accumulation and the outputs' rounding."""
    spread = 2 * d + 2.0 ** -20 + 8 * U * np.abs(o["logits"]).max(axis=1) + 4 * U * np.abs(o["lse"])
    ddl = BF16 * np.abs(o["dl"]) + (1 + BF16) * o["p"] * np.expm1(spread)[:, None]
    for got, want, err, s, depth in ((gx, o["grad_x"], ddl @ np.abs(w), np.abs(o["dl"]) @ np.abs(w), v),
                                     (gw, o["grad_w"], ddl.T @ np.abs(x), np.abs(o["dl"]).T @ np.abs(x), t)):
        tol = err + acc_bound(depth + 256, 16, s) + BF16 * (np.abs(want) + err) + 1e-37
        worst = np.max(np.abs(f64(got) - want) / tol)
        assert worst <= 1.0, f"worst error {worst:.3f} of its bound"


@pytest.mark.parametrize("t,k,v", [(2, 64, 70001), (300, 64, 40000), (3000, 64, 30011)])
def test_linear_ce_few_tiles(t, k, v):
    # grad_x has so few tiles that its sum over the vocabulary is split, with and without
    # several pieces, the last one short
    x, w, y, g = ce_inputs(t, k, v, 6)
    o = H.linear_ce(x, w, y, g)
    xd, wd, yd, gd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y), dev(g)
    loss, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    d = logit_errors(x, w, k)
    check_loss(loss, lse, o, d)
    gx, gw = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd)
    check_ce_grads(gx, gw, x, w, o, d, k, v, t)
    again = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


def test_linear_ce_pieces():
    # more than one piece of the vocabulary, the last one ragged
    t, k, v = 4500, 64, 9001
    x, w, y, g = ce_inputs(t, k, v, 5)
    o = H.linear_ce(x, w, y, g)
    xd, wd, yd, gd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y), dev(g)
    assert B.bitlinear_linear_ce_bwd_workspace_size(t, k, v) < 2 * t * v
    loss, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    d = logit_errors(x, w, k)
    check_loss(loss, lse, o, d)
    check_ce_grads(*B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd), x, w, o, d, k, v, t)


@pytest.mark.parametrize("std", [0.0, 40.0])
def test_linear_ce_flat_and_peaked(std):
    # all logits equal (loss log v) and logits of some hundred (one column has all the mass)
    t, k, v = 40, 128, 700
    x, w, y, g = ce_inputs(t, k, v, 3, std)
    o = H.linear_ce(x, w, y, g)
    xd, wd, yd, gd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y), dev(g)
    loss, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    check_loss(loss, lse, o, logit_errors(x, w, k))
    check_ce_grads(*B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd), x, w, o, logit_errors(x, w, k), k, v, t)


def test_linear_ce_nothing_counts():
    t, k, v = 70, 64, 300
    x, w, _, g = ce_inputs(t, k, v, 4)
    y = np.full(t, -100, np.int64)
    xd, wd, yd, gd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y), dev(g)
    loss, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    gx, gw = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd)
    assert not loss.any() and not gx.any() and not gw.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("t", [20, 200])
def test_linear_ce_padding_may_hold_anything(t):
    # infinities and NaN in the rows, lse and grad_loss of tokens without a loss
    k, v = 128, 700
    x, w, y, g = ce_inputs(t, k, v, 8)
    xd, wd, yd, gd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y), dev(g)
    dead = (yd < 0) | (yd >= v)
    xd[dead] = float("nan")
    xd[3 if y[3] < 0 else int(dead.nonzero()[0]), :5] = float("inf")
    x0 = np.where((y < 0)[:, None] | (y >= v)[:, None], 0.0, x)
    o = H.linear_ce(x0, w, y, g)
    loss, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    d = logit_errors(x0, w, k)
    live = o["live"]
    tol = d + 2.0 ** -20 + 4 * U * np.maximum(np.abs(o["lse"]), np.abs(o["logits"]).max(axis=1))
    assert np.all(np.abs(f64(loss) - o["loss"])[live] <= 2 * tol[live]) and not loss[dead].any()
    gd[dead] = float("nan")
    gx, gw = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd)
    check_ce_grads(gx, gw, x0, w, o, d, k, v, t)
    assert not gx[dead].any()


@pytest.mark.parametrize("t,v", [(1, 40), (3, 700), (20, 20001), (200, 700)])
def test_linear_ce_infinite_logits(t, v):
    # a vocabulary closed by weights of -infinity behind its first rows (and a token that
    # turns them into +infinity): the others' loss is that of the first rows alone
    k, first = 128, 24
    x, w, y, _ = ce_inputs(t, k, v, 11)
    x[:, 0], y[:] = 1.0, np.arange(t) % first
    if t > 1:
        x[1, 0] = -1.0
    xd, wd, yd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y)
    wd[first:], wd[first:, 0] = 0.0, float("-inf")
    loss, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    o = H.linear_ce(x, w[:first], y)
    d = logit_errors(x, w[:first], k)
    keep = np.arange(t) != 1
    check_loss(loss[dev(keep)], lse[dev(keep)], {n: a[keep] for n, a in o.items()}, d[keep])
    assert t == 1 or (loss[1] == float("inf") and lse[1] == float("inf"))


@pytest.mark.parametrize("t,v", [(1, 40), (5, 700), (20, 20001), (32, 50001), (33, 700), (300, 513)])
def test_linear_ce_infinite_target_logit(t, v):
    # row 5 of the head gives +infinity, for the second token -infinity: lse - l_y is infinity
    # minus infinity where it is the target, whatever the others are
    k = 128
    x, w, _, _ = ce_inputs(t, k, v, 15)
    x[:, 0] = 1.0
    y = np.full(t, 5)
    y[2:] = np.resize([5, 7, -100, 5, v], max(0, t - 2))
    if t > 1:
        x[1, 0] = -1.0
    xd, wd, yd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y)
    wd[5], wd[5, 0] = 0.0, INF
    loss, lse = (f64(a) for a in B.bitlinear_linear_ce_fwd(xd, wd, yd))
    first = np.arange(t) != 1
    assert np.all(lse[first] == INF)
    assert np.all(np.isnan(loss[first & (y == 5)])) and np.all(loss[first & (y == 7)] == INF)
    assert np.all(loss[(y < 0) | (y >= v)] == 0.0)
    if t > 1:   # l_y is -infinity: the others' lse, and an infinite loss
        o = H.linear_ce(x[1:2], np.delete(w, 5, 0), np.array([-1]))
        assert loss[1] == INF and abs(lse[1] - o["lse"][0]) <= logit_errors(x, w, k)[1] + 2.0 ** -20 + 4 * U * abs(o["lse"][0])
    wd[9 % v, 0] = INF   # another one beside it
    loss, lse = (f64(a) for a in B.bitlinear_linear_ce_fwd(xd, wd, yd))
    assert np.all(lse[first] == INF) and np.all(np.isnan(loss[first & (y == 5)]))


@pytest.mark.parametrize("low", [-INF, -3.3895313892515355e38])
@pytest.mark.parametrize("t,v", [(1, 1), (4, 1), (4, 700), (20, 20001), (40, 1), (200, 700)])
def test_linear_ce_no_finite_logit(t, v, low):
    # every logit -infinity, or the type's lowest value (2.36e38 and beyond count as infinite):
    # the logarithm of an empty sum is -infinity, and the loss of a target there is no number
    x, w, _, _ = ce_inputs(t, 64, v, 16)
    x[:, 0] = 1.0
    y = np.where(np.arange(t) % 2 == 0, v // 2, -100)
    xd, wd, yd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y)
    wd[:], wd[:, 0] = 0.0, low
    loss, lse = (f64(a) for a in B.bitlinear_linear_ce_fwd(xd, wd, yd))
    assert np.all(lse == -INF) and np.all(np.isnan(loss[::2])) and np.all(loss[1::2] == 0.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("t", [1, 20, 300])
def test_linear_ce_not_finite_grad_loss(t, bad):
    # it stays with its token: the other rows of grad_x are what they are with 0 in its place
    k, v = 128, 700
    x, w, y, g = ce_inputs(t, k, v, 12)
    y[t // 2] = 5
    g[t // 2] = 0.0
    xd, wd, yd, gd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y), dev(g)
    _, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    want, _ = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd)
    gd[t // 2] = bad
    gx, gw = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, gd)
    keep = torch.arange(t, device="cuda") != t // 2
    assert torch.equal(gx[keep], want[keep]) and not want[t // 2].any()
    assert not torch.isfinite(gx[t // 2]).any() and not torch.isfinite(gw[5]).any()


@pytest.mark.parametrize("t,k,v,live", [(1, 64, 500, 1), (1, 1088, 5003, 1), (2, 128, 700, 2), (5, 2048, 1003, 4), (32, 64, 40001, 32),
                                        (33, 320, 2500, 32), (64, 192, 600, 17), (200, 64, 513, 7), (300, 256, 1031, 32)])
def test_linear_ce_few_tokens_keep_dl(t, k, v, live):
    # up to 32 tokens with a loss: dl as two bf16 numbers, so that it is off by a half step
    # (2^-8) of what a half step leaves (2^-8 of dl), where one number would be off by 2^-8
    x, w, _, _ = ce_inputs(t, k, v, 14)
    rng = np.random.default_rng(t + v)
    y = np.full(t, -1)
    y[rng.permutation(t)[:live]] = rng.integers(0, v, live)
    g = np.where(rng.random(t) < 0.5, 1.0 / t, rng.normal(size=t)).astype(np.float32)
    o, d = H.linear_ce(x, w, y, g), logit_errors(x, w, k)
    xd, wd, yd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y)
    _, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    gx, gw = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, dev(g), grad_w_dtype=torch.float32)
    spread = 2 * d + 2.0 ** -20 + 8 * U * np.abs(o["logits"]).max(axis=1) + 4 * U * np.abs(o["lse"])   # as in check_ce_grads
    ddl = (BF16 ** 2 + 4 * U) * np.abs(o["dl"]) + (1 + BF16) * o["p"] * np.expm1(spread)[:, None]
    for got, want, err, s, depth in ((gx, o["grad_x"], ddl @ np.abs(w), np.abs(o["dl"]) @ np.abs(w), v),
                                     (gw, o["grad_w"], ddl.T @ np.abs(x), np.abs(o["dl"]).T @ np.abs(x), t)):
        tol = err + acc_bound(2 * depth + 256, 16, s) + (BF16 if got.dtype == torch.bfloat16 else U) * (np.abs(want) + err) + 1e-37
        worst = np.max(np.abs(f64(got) - want) / tol)
        assert worst <= 1.0, f"worst error {worst:.3f} of its bound"


def sure_inputs(t, k, v, seed, top=18.0):
    """Hidden states whose targets' logits run from about 0 to `top` (others: N(0, 0.02^2 k))."""
    rng = np.random.default_rng(seed)
    w, y = bf16(rng, v, k, scale=0.02, outliers=False), rng.permutation(v)[:t]
    push = np.linspace(top / t, top, t)[:, None]
    x = rng.normal(size=(t, k)) + push * w[y] / (w[y] ** 2).sum(1, keepdims=True)
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).float().numpy(), w, y.astype(np.int64)


@pytest.mark.parametrize("t,k,v", [(1, 2048, 1000), (32, 2048, 1000), (33, 2048, 1000), (200, 2048, 1000), (20, 8192, 1000),
                                   (100, 8192, 700), (40, 512, 5003), (64, 2048, 9001), (20, 16448, 700)])
def test_linear_ce_gradient_of_sure_tokens(t, k, v):
    """dl of tokens that are nearly sure of their target, one at a time (g is 0 elsewhere, so
    that grad_w of row u is dl_u x): with 1 - p down to 1e-5 it has to come from l_y - lse as
    the forward pass had them. The errors of the logits count by what they move the others'
    sum, 1 - p of them; the rest is the rounding of l_y and lse, and of dl itself."""
    x, w, y = sure_inputs(t, k, v, 20)
    o, d = H.linear_ce(x, w, y, np.ones(t)), logit_errors(x, w, k)
    xd, wd, yd = dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y)
    _, lse = B.bitlinear_linear_ce_fwd(xd, wd, yd)
    for i in sorted({t - 1, t - 1 - t // 20, t - 1 - t // 10, t // 2}):
        g = torch.zeros(t, device="cuda")
        g[i] = 1.0
        _, gw = B.bitlinear_linear_ce_bwd(xd, wd, yd, lse, g, want_grad_x=False, grad_w_dtype=torch.float32)
        j = np.argmax(np.abs(x[i]))
        dl, got = o["dl"][i], f64(gw[:, j]) / x[i, j]
        l, rest = o["logits"][i], -o["dl"][i, y[i]]
        spread = 2 * d[i] + 2.0 ** -18 + U * (8 * np.abs(l).max() + 4 * np.abs(o["lse"][i]))
        err = np.where(np.arange(v) == y[i], rest * np.expm1(spread) + U * (abs(o["lse"][i]) + abs(l[y[i]])),
                       o["p"][i] * np.expm1(spread))
        half = BF16 ** 2 if t <= 32 else BF16
        tol = err + (half + 8 * U) * (np.abs(dl) + err)
        worst = np.max(np.abs(got - dl) / tol)
        assert worst <= 1.0, f"token {i}: 1 - p {rest:.2e}, worst error {worst:.3f} of its bound"


@pytest.mark.parametrize("t,k,v", [(1, 2048, 1000), (32, 2048, 1000), (33, 2048, 1000), (512, 2048, 700), (32, 8192, 1000),
                                   (300, 8192, 1000), (1000, 896, 5003), (300, 2048, 8192)])
def test_linear_ce_loss_to_its_stated_error(t, k, v):
    """At the size the errors have, where the bounds above count every one at its largest and
    of one sign. A tensor core's accumulation loses half a unit of its running sum per MMA (16
    of K) on average, towards zero: over 512 of K the target's logit, which grows evenly, comes
    out 32 / 2 * 2^-24 = 2^-20 of itself too small (twice that is allowed); as a dot product
    (few tokens, large vocabularies) it is rounded to nearest, half a unit for each of the last
    five halvings. The others' are off by 2^-20 of themselves, of sizes about 1 here. The loss
    takes 1 - p of both, and three roundings of half a unit. lse has the target's error in full
    where the token is sure."""
    x, w, y = sure_inputs(t, k, v, 19)
    o = H.linear_ce(x, w, y)
    loss, lse = B.bitlinear_linear_ce_fwd(dev(x, torch.bfloat16), dev(w, torch.bfloat16), dev(y))
    l = np.abs(o["logits"][np.arange(t), y])
    own = l * (5 * 2.0 ** -24 if t <= 32 or v >= 8192 else 2.0 ** -19)
    rest = -np.expm1(-o["loss"])
    err = np.abs(f64(loss) - o["loss"])
    assert np.all(err <= rest * (own + 1e-6) + 3 * 2.0 ** -24 * np.exp2(np.ceil(np.log2(np.maximum(o["loss"], 1e-30)))))
    assert np.all(np.abs(f64(lse) - o["lse"]) <= own + 1e-6 + 3 * U * np.maximum(np.abs(o["lse"]), l))
    assert err.mean() <= (3.5e-7 if t <= 32 else 1e-6)


def test_linear_ce_empty_batch():
    w = torch.randn(50, 64, device="cuda").to(torch.bfloat16)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = B.bitlinear_linear_ce_fwd(x, w, y)
    gw = torch.ones(50, 64, dtype=torch.bfloat16, device="cuda")
    gx, gw = B.bitlinear_linear_ce_bwd(x, w, y, lse, torch.empty(0, device="cuda"), grad_w=gw)
    assert loss.shape == (0,) and gx.shape == (0, 64) and not gw.any()


# ------------------------------------------------------------------ as they are used

def test_head_training_step_runs_together():
    """A ternary layer, an 8-bit float projection and the head's loss, forward and back, on
    a stream of their own, twice into the same buffers and once as a replayed graph: the
    three runs agree bit for bit."""
    t, k, n, v = 200, 256, 512, 1003
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16)
    w1 = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    w2 = torch.randn(k, n, generator=gen, device="cuda") * 0.02
    head = (torch.randn(v, k, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    g = torch.full((t,), 1.0 / t, device="cuda")

    def step():
        qm = B.bitlinear_quant_mask(w1, 6, 8)
        xq, a = B.bitlinear_act_quant(x)
        h, _ = B.bitlinear_fwd(xq, a, qm["w_scale"], w_i8=qm["w_i8"])
        wq = B.bitlinear_fp8_quant_weight(w2, want_t=True)
        hq = B.bitlinear_fp8_quant(h, want_t=True)
        z = B.bitlinear_fp8_fwd(hq["q"], wq["q"], wq["scales"], x_scales=hq["scales"])
        loss, lse = B.bitlinear_linear_ce_fwd(z, head, y)
        dz, dhead = B.bitlinear_linear_ce_bwd(z, head, y, lse, g)
        dzq = B.bitlinear_fp8_quant(dz, want_t=True, fmt=torch.float8_e5m2)
        dh, dw2 = B.bitlinear_fp8_bwd(dzq, hq, wq)
        dx, dw1 = B.bitlinear_bwd(dh, x, qm["codes"], qm["w_scale"])
        return loss, dhead, dw2, dx, dw1

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = step()
        again = step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = step()
        graph.replay()
        s.synchronize()
    for a, b, c in zip(first, again, captured):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.isfinite(a.float()).all()
    assert float(first[0].mean()) > 1.0


def test_two_streams_at_once():
    """The same calls on two streams side by side, each with its own data, many times over:
    every result is what the call alone gives."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    sets = []
    for t, k, n, v in ((16, 1024, 2048, 3001), (300, 512, 1040, 2500)):
        x = torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16)
        w = B.bitlinear_fp8_quant_weight(torch.randn(n, k, generator=gen, device="cuda"))
        head = torch.randn(v, k, generator=gen, device="cuda").to(torch.bfloat16) * 0.1
        y = torch.randint(-1, v, (t,), generator=gen, device="cuda")
        sets.append((x, w, head, y, torch.randn(t, generator=gen, device="cuda")))

    def run(x, w, head, y, g):
        a = B.bitlinear_fp8_fwd(x, w["q"], w["scales"])
        q = B.bitlinear_fp8_quant(x, want_t=True)
        loss, lse = B.bitlinear_linear_ce_fwd(x, head, y)
        return [a, q["qt"].view(torch.uint8), loss, *B.bitlinear_linear_ce_bwd(x, head, y, lse, g)]

    alone = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, alone[i]))
    assert B.bitlinear_device_status()[0] == 0


def test_chain_reads_what_the_call_before_wrote():
    """Each call's input is the previous call's output in the same buffers, for many steps:
    a kernel set up behind its predecessor must not read an earlier step's values."""
    t, k = 64, 1024
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = B.bitlinear_fp8_quant_weight(torch.randn(k, k, generator=gen, device="cuda") / k ** 0.5)
    x0 = torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16)

    def chain(sync):
        a, b = x0.clone(), torch.empty_like(x0)
        q = B.bitlinear_fp8_quant(a)
        out = []
        for _ in range(30):
            B.bitlinear_fp8_quant(a, out=q)
            B.bitlinear_fp8_fwd(q["q"], w["q"], w["scales"], x_scales=q["scales"], y=b)
            if sync:
                torch.cuda.synchronize()
            a, b = b, a
            out.append(a.clone())
        return torch.stack(out)

    assert torch.equal(chain(True), chain(False))


def test_streams_other_than_the_current_one():
    s = torch.cuda.Stream()
    x = torch.randn(5, 256, device="cuda").to(torch.bfloat16)
    w = B.bitlinear_fp8_quant_weight(torch.randn(64, 256, device="cuda"))
    want = B.bitlinear_fp8_fwd(x, w["q"], w["scales"])
    s.wait_stream(torch.cuda.current_stream())
    got = B.bitlinear_fp8_fwd(x, w["q"], w["scales"], stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_own_workspace_on_another_stream():
    # the call's own workspace is not handed out again while its stream still has the work
    # before it: an allocation of the same size right after the call must not be that memory
    t, k, n = 300, 512, 64
    x = torch.randn(t, k, device="cuda").to(torch.bfloat16)
    w = B.bitlinear_fp8_quant_weight(torch.randn(n, k, device="cuda"))
    need = B.bitlinear_fp8_fwd_workspace_size(t, k)
    assert need > 0
    want, y = B.bitlinear_fp8_fwd(x, w["q"], w["scales"]), torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    B.bitlinear_fp8_fwd(x, w["q"], w["scales"], y=y, stream=s)
    ran = s.query()
    junk = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert not ran and torch.equal(y, want) and junk.numel() == need


def test_results_are_not_written_by_an_earlier_call_on_the_current_stream():
    # a call on the current stream whose results are dropped has yet to write them; a call on
    # another stream must not be handed their memory, which the first would then write over
    t, k, n, v = 300, 512, 64, 700
    gen = torch.Generator(device="cuda").manual_seed(17)
    a, b = (torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = B.bitlinear_fp8_quant_weight(torch.randn(n, k, generator=gen, device="cuda"), want_t=True)
    ws = {id(x): torch.randn(n, k, generator=gen, device="cuda") for x in (a, b)}
    head = (torch.randn(v, k, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    y, g = torch.randint(0, v, (t,), generator=gen, device="cuda"), torch.randn(t, generator=gen, device="cuda")
    lses = {id(x): B.bitlinear_linear_ce_fwd(x, head, y)[1] for x in (a, b)}
    quants = {id(x): B.bitlinear_fp8_quant(x, want_t=True) for x in (a, b)}
    dy = B.bitlinear_fp8_quant(torch.randn(t, n, generator=gen, device="cuda").to(torch.bfloat16), want_t=True)
    s = torch.cuda.Stream()
    calls = {"quant": lambda x, **o: list(B.bitlinear_fp8_quant(x, want_t=True, **o).values()),
             "quant_weight": lambda x, **o: list(B.bitlinear_fp8_quant_weight(ws[id(x)], want_t=True, **o).values()),
             "fwd": lambda x, **o: [B.bitlinear_fp8_fwd(x, w["q"], w["scales"], **o)],
             "bwd": lambda x, **o: list(B.bitlinear_fp8_bwd(dy, quants[id(x)], w, **o)),
             "ce_fwd": lambda x, **o: list(B.bitlinear_linear_ce_fwd(x, head, y, **o)),
             "ce_bwd": lambda x, **o: list(B.bitlinear_linear_ce_bwd(x, head, y, lses[id(x)], g, **o))}
    for name, call in calls.items():
        want = [r.clone() for r in call(b)]
        torch.cuda.synchronize()
        torch.cuda._sleep(400_000_000)   # 0.2 s: new memory for the other stream may take tens of ms
        call(a)
        got = call(b, stream=s)
        s.synchronize()
        waiting = not torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        assert waiting, name
        for i, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), (name, i)


def test_dropped_results_of_a_given_stream():
    # the other way round: a result dropped at once, before the given stream has written it,
    # must not become memory of the current stream
    t, k, v = 300, 512, 700
    gen = torch.Generator(device="cuda").manual_seed(18)
    x = torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16)
    head = (torch.randn(v, k, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    want = B.bitlinear_linear_ce_fwd(x, head, y)[0]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    loss, _ = B.bitlinear_linear_ce_fwd(x, head, y, stream=s)
    waiting = not s.query()
    _ = None
    junk = [torch.full((t,), 7.0, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    assert waiting and torch.equal(loss, want) and all(bool((j == 7.0).all()) for j in junk)


def test_given_stream_in_a_captured_graph():
    # a call on a stream that joined the capture, its results and workspace its own
    t, k, v = 300, 512, 700
    gen = torch.Generator(device="cuda").manual_seed(24)
    x = torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16)
    head = (torch.randn(v, k, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    y, g = torch.randint(0, v, (t,), generator=gen, device="cuda"), torch.randn(t, generator=gen, device="cuda")
    loss, lse = B.bitlinear_linear_ce_fwd(x, head, y)
    want = [loss, *B.bitlinear_linear_ce_bwd(x, head, y, lse, g)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        loss, lse = B.bitlinear_linear_ce_fwd(x, head, y, stream=side)
        got = [loss, *B.bitlinear_linear_ce_bwd(x, head, y, lse, g, stream=side)]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for a in got:
            a.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_more_than_2_to_31_elements():
    # 384 rows over and over: the last copy, whose offsets pass 32 bits, comes out as the first
    reps, rows, k, n = 2732, 384, 2048, 16
    rng = np.random.default_rng(13)
    base = bf16(rng, rows, k, scale=2.0 / np.sqrt(k), outliers=False)
    small = dev(base, torch.bfloat16)
    big = small.repeat(reps, 1)
    assert big.numel() > 2 ** 31
    q, first = B.bitlinear_fp8_quant(big, want_t=True), B.bitlinear_fp8_quant(small, want_t=True)
    last = slice((reps - 1) * rows, reps * rows)
    for at in (slice(0, rows), last):
        assert np.array_equal(u8(q["q"][at]), u8(first["q"])) and np.array_equal(u8(q["qt"][:, at]), u8(first["qt"]))
        assert torch.equal(q["scales"][:, at], first["scales"])
    w = B.bitlinear_fp8_quant_weight(dev(rng.normal(size=(n, k)).astype(np.float32)))
    y = B.bitlinear_fp8_fwd(q["q"], w["q"], w["scales"], x_scales=q["scales"])
    assert torch.equal(y[last], y[:rows]) and y[last].any()
    del q, y

    for t in (3, 40):   # `big` as the vocabulary, targets in its last copy
        x, g = bf16(rng, t, k, outliers=False), rng.normal(size=t).astype(np.float32)
        y = rng.integers(0, rows, t)
        xd, yd = dev(x, torch.bfloat16), dev(y) + (reps - 1) * rows
        loss, lse = B.bitlinear_linear_ce_fwd(xd, big, yd)
        o, d = H.linear_ce(x, base, y, g), logit_errors(x, base, k)
        p, onehot = o["p"] / reps, np.zeros((t, rows))
        onehot[np.arange(t), y] = 1.0
        o.update(lse=o["lse"] + np.log(reps), loss=o["loss"] + np.log(reps))
        check_loss(loss, lse, o, d)
        gw = B.bitlinear_linear_ce_bwd(xd, big, yd, lse, dev(g), want_grad_x=False)[1][last]
        dl = p * np.sign(g)[:, None] - onehot * g[:, None]
        spread = 2 * d + 2.0 ** -20 + 8 * U * np.abs(o["logits"]).max(axis=1) + 4 * U * np.abs(o["lse"])   # as in check_ce_grads
        err = (BF16 * np.abs(dl) + (1 + BF16) * p * np.expm1(spread)[:, None]).T @ np.abs(x)
        want = dl.T @ x
        tol = err + acc_bound(t + 256, 16, np.abs(dl).T @ np.abs(x)) + BF16 * (np.abs(want) + err) + 1e-37
        assert np.all(np.abs(f64(gw) - want) <= tol)
