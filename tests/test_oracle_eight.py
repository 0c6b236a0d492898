"""CPU pins of the 8-bit oracle: E4M3 against its bit layout and another implementation of its
rounding, the scale rule against exact rationals, the activation and the router against differences."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O


def test_e4m3_values():
    assert O.E4M3[0x7E] == 448 and O.E4M3[0x01] == 2.0 ** -9 and O.E4M3[0x08] == 2.0 ** -6 and O.E4M3[0x38] == 1.0
    assert math.isnan(O.E4M3[0x7F]) and math.isnan(O.E4M3[0xFF]) and O.E4M3[0xB8] == -1.0
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, O.E4M3, equal_nan=True)


def test_rounding_equals_another_implementation_on_ties_and_all_bf16_steps():
    ties = (O.E4M3[:126] + O.E4M3[1:127]) / 2
    a = np.unique(np.concatenate([O.E4M3[:127], ties, np.nextafter(ties, 0), np.nextafter(ties, 1e9),
                                  np.linspace(0, 448, 5001)])).astype(np.float32)
    x = np.zeros((len(a), 128), np.float32)
    x[:, 0], x[:, 1], x[:, 2] = 448.0, a, -a     # scale 1
    codes, scales = O.quantize8(x)
    assert np.all(scales == 127)
    want = torch.from_numpy(x[:, 1:3].copy()).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes[:, 1:3], want)


def test_scale_is_the_smallest_that_holds_the_block():
    rng = np.random.default_rng(0)
    amax = np.concatenate([np.float32(2.0) ** np.arange(-149, 128), [448, 449, 447.99997, 1.75, 1.7500001, 3.4e38],
                           np.abs(rng.standard_normal(200) * 10.0 ** rng.integers(-30, 30, 200))]).astype(np.float32)
    amax = np.concatenate([amax, np.nextafter(amax, np.float32(0)), np.float32(1.75) * np.float32(2.0) ** np.arange(-120, 120)])
    for a in amax[amax > 0].astype(np.float32):
        _, s = O.quantize8(np.array([[a, -a / 3]]))
        e = int(s[0, 0]) - 127
        assert Fraction(float(a)) <= 448 * Fraction(2) ** e
        assert e == -127 or Fraction(float(a)) > 448 * Fraction(2) ** (e - 1)


@pytest.mark.parametrize("shape", [(1, 1), (5, 300), (130, 128), (257, 129)])
def test_quantized_values_are_within_half_a_step(shape):
    x = np.random.default_rng(1).standard_normal(shape) * 3
    for h, w in ((1, 128), (128, 128)):
        q = O.quantize8(x, h, w)
        v = O.dequantize8(*q)
        step = np.exp2(np.repeat(q[1].astype(float), 128, axis=1)[:, :shape[1]] - 127 - 9)
        assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step / 2))
        again = O.quantize8(v, h, w)           # the values are representable: a second time changes none
        assert np.array_equal(O.dequantize8(*again), v)


def test_zero_negative_zero_and_non_finite_blocks():
    x = np.zeros((3, 256))
    x[0, 0] = -0.0
    x[1, 130], x[2, 3] = np.nan, -np.inf
    codes, scales = O.quantize8(x)
    assert codes[0, 0] == 0x80 and codes[0, 1] == 0 and scales[0].tolist() == [0, 0]
    assert scales[1].tolist() == [0, 255] and scales[2].tolist() == [255, 0] and not codes[1:].any()


def test_layer_is_the_textbook_layer_on_exact_values():
    rng = np.random.default_rng(2)
    x, w, dy = (rng.integers(-8, 9, s).astype(float) for s in ((70, 200), (150, 200), (70, 150)))
    (y, _), xq, wq = O.linear8_fwd(x, w)
    (dx, _), (dw, _) = O.linear8_bwd(dy, xq, wq)
    assert np.array_equal(y, x @ w.T) and np.array_equal(dx, dy @ w) and np.array_equal(dw, dy.T @ x)


@pytest.mark.parametrize("act", [O.SILU, O.GELU])
def test_activation_gradient_against_differences(act):
    z = np.random.default_rng(3).standard_normal((6, 20)) * 3
    dh = np.random.default_rng(4).standard_normal((6, 10))
    d = O.glu_bwd(dh, z[:, :10], z[:, 10:], act)
    for i, j in np.ndindex(*z.shape):
        up, down = z.copy(), z.copy()
        up[i, j] += 1e-6
        down[i, j] -= 1e-6
        diff = ((O.glu(up, act) - O.glu(down, act)) * dh).sum() / 2e-6
        assert abs(diff - d[i, j]) < 1e-8 * (1 + np.abs(dh).max() * 50)


def test_router_worked_example():
    logits = np.log([[4.0, 1.0, 3.0, 2.0], [1.0, 1.0, 1.0, 1.0]])
    ids, p, counts, sums, loss = O.route(logits, 2, False)
    assert ids.tolist() == [[0, 2], [0, 1]] and counts.tolist() == [2, 1, 1, 0, 2]
    assert np.allclose(p, [[0.4, 0.3], [0.25, 0.25]]) and np.allclose(sums, [0.65, 0.35, 0.55, 0.45])
    assert math.isclose(loss, 4 * (0.5 * 0.325 + 0.25 * 0.175 + 0.25 * 0.275))
    assert np.allclose(O.route(logits, 2, True)[1], [[4 / 7, 3 / 7], [0.5, 0.5]])
    logits[0, 1:] = -np.inf
    ids, p, counts, _, _ = O.route(logits, 2, True, mask=[True, False])
    assert ids.tolist() == [[0, -1], [-1, -1]] and p.tolist() == [[1, 0], [0, 0]] and counts.tolist() == [1, 0, 0, 0, 1]


@pytest.mark.parametrize("renormalize", [False, True])
def test_router_gradient_against_differences(renormalize):
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((7, 6)) * 2
    logits[2, 1], logits[3] = -np.inf, -np.inf
    mask = np.array([1, 1, 1, 1, 0, 1, 1], bool)
    dp = rng.standard_normal((7, 3))
    ids, _, counts, _, _ = O.route(logits, 3, renormalize, mask)
    d, _ = O.route_bwd(logits, ids, counts, dp, 0.7, renormalize, mask)

    def value(l):
        i, p, c, _, loss = O.route(l, 3, renormalize, mask)
        assert np.array_equal(i, ids)
        return (p * dp).sum() + 0.7 * loss

    for t, e in np.ndindex(*logits.shape):
        if logits[t, e] == -np.inf:
            assert d[t, e] == 0
            continue
        up, down = logits.copy(), logits.copy()
        up[t, e] += 1e-6
        down[t, e] -= 1e-6
        assert abs((value(up) - value(down)) / 2e-6 - d[t, e]) < 1e-8
