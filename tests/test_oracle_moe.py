"""CPU pins of the expert routing oracle: a worked example, the transposes' inner-product
identity, gradients against differences, and the few-row product against a textbook matmul."""
import numpy as np

import oracle as O

IDS = np.array([[2, 0], [0, -1], [2, 2], [5, 1]])   # 3 experts: -1 and 5 take part in nothing


def test_plan_worked_example():
    offs, src, pos = O.moe_plan(IDS, 3)
    assert offs.tolist() == [0, 2, 3, 6]
    assert src.tolist() == [1, 2, 7, 0, 4, 5, -1, -1]
    assert pos.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]]


def test_plan_is_a_stable_sort():
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 9, (50, 3))
    offs, src, pos = O.moe_plan(ids, 8)
    flat = ids.reshape(-1)
    kept = np.nonzero((flat >= 0) & (flat < 8))[0]
    order = kept[np.argsort(flat[kept], kind="stable")]
    assert np.array_equal(src[:offs[-1]], order) and np.all(src[offs[-1]:] == -1)
    assert np.array_equal(np.diff(offs), np.bincount(flat[kept], minlength=8))
    assert np.all(pos.reshape(-1)[order] == np.arange(offs[-1]))


def test_dispatch_and_combine_are_transposes():
    rng = np.random.default_rng(1)
    _, _, pos = O.moe_plan(IDS, 3)
    w = rng.standard_normal(pos.shape)
    x, z = rng.standard_normal((4, 5)), rng.standard_normal((8, 5))
    for weights in (w, None):
        left = np.sum(O.moe_dispatch(x, pos, weights, np.zeros((8, 5))) * z)
        right = np.sum(x * O.moe_combine(z, pos, weights)[0])
        assert np.isclose(left, right, rtol=1e-13)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(2)
    _, _, pos = O.moe_plan(IDS, 3)
    w, z, dy = rng.standard_normal(pos.shape), rng.standard_normal((8, 5)), rng.standard_normal((4, 5))
    dz, dw, _ = O.moe_combine_bwd(dy, z, pos, w, np.zeros((8, 5)))
    loss = lambda z, w: np.sum(dy * O.moe_combine(z, pos, w)[0])  # noqa: E731
    # the loss is linear in z and in w: a central difference is exact up to rounding
    for a, g, f in ((z, dz, lambda a: loss(a, w)), (w, dw, lambda a: loss(z, a))):
        for i in np.ndindex(*a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += 0.5
            dn[i] -= 0.5
            assert abs((f(up) - f(dn)) - g[i]) < 1e-12


def test_slots_left_out_do_not_count():
    _, _, pos = O.moe_plan(IDS, 3)
    w = np.ones(pos.shape)
    w[pos < 0] = np.nan
    z = np.ones((8, 2))
    z[6:] = np.nan                      # rows no slot maps to
    y, _ = O.moe_combine(z, pos, w)
    assert y[:, 0].tolist() == [2, 1, 2, 1]


def test_gemv_is_the_textbook_product():
    rng = np.random.default_rng(3)
    w = rng.choice([-6, -1.5, 0, 0.5, 3, 4], (7, 64)) * 4.0
    codes, scales = O.quantize(w.astype(np.float32), O.ROW, O.RNE)
    assert np.array_equal(O.dequantize(codes, scales, 7, 64), w)
    x = rng.standard_normal((3, 64))
    y, mag = O.gemv(x, codes, np.pad(scales, ((0, 0), (0, 3)), constant_values=9), 0.5)
    assert np.allclose(y, 0.5 * x @ w.T, rtol=1e-13) and np.all(mag >= np.abs(y) - 1e-12)
    y, _ = O.gemv_grouped(x, np.stack([codes, codes]), np.stack([scales, scales]), [0, 2, 3],
                          np.array([4, 1, 3, -1]), 2, 4)
    assert np.allclose(y[:3], (x @ w.T)[[2, 0, 1]], rtol=1e-13) and np.all(np.isnan(y[3]))
