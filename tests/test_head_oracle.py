"""Pins of the head's oracle (CPU): 8-bit float codes by hand, scales at their borders,
the cross entropy's gradients against differences."""
import math

import numpy as np
import pytest
import torch

from oracle import head_oracle as H


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_codes_are_the_format(fmt, dtype):
    # every code's value, and the rounding of a dense sweep, against torch's own casts
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(dtype).double().numpy()
    assert np.array_equal(H.decode(codes, fmt), want, equal_nan=True)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-1, 1, 20000) * H.TOP[fmt] * 2.0 ** rng.integers(-25, 1, 20000),
                        [0.0, H.TOP[fmt], -H.TOP[fmt]]]).astype(np.float32)
    got = H.encode(v.astype(np.float64), fmt)
    assert np.array_equal(got, torch.from_numpy(v).to(dtype).view(torch.uint8).numpy())


def test_hand_worked_codes():
    # e4m3: 1.0 = 0x38, 448 = 0x7E, the smallest subnormal 2^-9 = 0x01
    assert [H.code_value(c, "e4m3") for c in (0x38, 0x7E, 0x01, 0xB8)] == [1.0, 448.0, 2.0 ** -9, -1.0]
    assert [H.code_value(c, "e5m2") for c in (0x3C, 0x7B, 0x01)] == [1.0, 57344.0, 2.0 ** -16]
    # 17 lies between 16 (0x58) and 18 (0x59): the tie goes to the even code
    assert H.encode(np.array([17.0, 19.0, -17.0]), "e4m3").tolist() == [0x58, 0x5A, 0xD8]


@pytest.mark.parametrize("amax,fmt,e", [(448.0, "e4m3", 0), (449.0, "e4m3", 1), (1.75, "e4m3", -8),
                                        (1.7500001, "e4m3", -7), (1.0, "e4m3", -8), (2.0 ** -140, "e4m3", -127),
                                        (0.0, "e4m3", -127), (57344.0, "e5m2", 0), (57345.0, "e5m2", 1)])
def test_scale_at_its_borders(amax, fmt, e):
    assert H.block_exponent(amax, fmt) == e
    x = np.zeros((1, 200))
    x[0, 3] = -amax
    q, s, v = H.fp8_quant(x, fmt)
    assert s[0, 0].tolist() == [e + 127, 0, 0, 0]     # one block of 128, one of 72, none after
    if 0 < amax < 1e30 and e > -127:
        assert v[0, 3] == pytest.approx(-amax, rel=2.0 ** -4)


def test_blocks_of_weights_share_their_scale():
    rng = np.random.default_rng(1)
    w = rng.normal(size=(144, 192)) * 0.02
    w[130, 5] = 1000.0
    _, s, _ = H.fp8_quant(w, "e4m3", 128)
    assert len(set(s[0, :128, 0])) == 1 and len(set(s[0, 128:, 0])) == 1 and s[0, 0, 0] != s[0, 128, 0]
    assert H.fp8_quant(w.T, "e4m3", 128)[1][0, 5, 1] == s[0, 130, 0]   # the same block from the other side


def test_not_finite_blocks():
    x = np.ones((2, 256))
    x[0, 130] = np.inf
    q, s, v = H.fp8_quant(x, "e4m3")
    assert s[0, 0].tolist()[1] == 255 and set(q[0, 128:]) == {0x7F} and np.all(np.isfinite(v[0, :128])) and np.all(np.isfinite(v[1]))


def test_linear_ce_by_hand():
    # two columns with logits 0 and log 3: probabilities 1/4 and 3/4
    x, w = np.array([[1.0, 0.0]]), np.array([[0.0, 0.0], [math.log(3.0), 0.0]])
    o = H.linear_ce(x, w, np.array([1]), np.array([2.0]))
    assert o["loss"][0] == pytest.approx(math.log(4 / 3)) and o["lse"][0] == pytest.approx(math.log(4.0))
    assert o["dl"][0] == pytest.approx([0.5, -0.5])
    assert H.linear_ce(x, w, np.array([-100]), np.array([2.0]))["loss"][0] == 0.0
    assert not H.linear_ce(x, w, np.array([2]), np.array([2.0]))["grad_w"].any()


def test_linear_ce_gradients_against_differences():
    rng = np.random.default_rng(2)
    x, w = rng.normal(size=(4, 6)), rng.normal(size=(9, 6))
    y, g = np.array([3, -100, 8, 0]), rng.normal(size=4)
    o = H.linear_ce(x, w, y, g)
    f = lambda x, w: float((H.linear_ce(x, w, y)["loss"] * g).sum())   # noqa: E731
    h = 1e-6
    for a, grad, other in ((x, o["grad_x"], "x"), (w, o["grad_w"], "w")):
        for i in np.ndindex(a.shape):
            up, down = a.copy(), a.copy()
            up[i] += h
            down[i] -= h
            d = (f(up, w) - f(down, w)) if other == "x" else (f(x, up) - f(x, down))
            assert d / (2 * h) == pytest.approx(grad[i], abs=1e-7)
