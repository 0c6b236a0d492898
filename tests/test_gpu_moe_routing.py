"""GPU checks of the expert routing operators (plan, dispatch, combine and their gradients)
against the float64 oracle, at the sizes, strides and masks where they can go wrong.

Tolerances: a plain copy, the plan and packed outputs are exact.  A product rounded to float32
is off by at most 2^-24 of it, a sum of n float32 terms by at most (n + 1) 2^-24 of the terms'
magnitudes (first order; the products' rounding included), and the rounding to bf16 adds 2^-8 of
the value (2^-24 for float32).  2^-140 covers results below the normal range."""
import numpy as np
import pytest
import torch

import oracle as O
from mxfp4_microscaling_quantization_amd import mx, synth
from tests.gpu_util import DEV, assert_bytes_equal, host, oracle_input, upload

pytestmark = pytest.mark.gpu

STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 2.0 ** -140


def stored(x, dtype):
    """float32 values as an array of the storage type (bf16: bit patterns)."""
    x = np.asarray(x, np.float32)
    return synth.f32_to_bf16_bits(x) if dtype == "bf16" else x


def torch_type(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def values(t):
    """float64 values of a device tensor."""
    return t.detach().to(torch.float64).cpu().numpy()


def strided(a, dtype, ld):
    """The matrix a on the device with rows ld elements apart, NaN between them."""
    full = torch.full((a.shape[0], ld), float("nan"), dtype=torch_type(dtype), device=DEV)
    full[:, :a.shape[1]] = upload(a, dtype)
    return full[:, :a.shape[1]]


def routing(rng, tokens, top_k, experts, left_out=0.2, same=False):
    ids = rng.integers(0, experts, (tokens, top_k))
    if same:
        ids[:] = experts // 2
    out = rng.random(ids.shape) < left_out
    ids[out] = rng.choice([-1, experts, -7, 1 << 20], out.sum())
    if tokens > 2:
        ids[1] = -1                                  # a token without any expert
    return ids


def dev_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def dev_f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,top_k,experts", [
    (0, 1, 4), (1, 1, 1), (1, 8, 128), (63, 1, 2), (64, 1, 7), (65, 3, 128), (341, 3, 33),
    (1024, 1, 8), (1025, 1, 8), (700, 3, 5), (5000, 4, 32), (16384, 4, 32), (65537, 5, 128)])
def test_plan(tokens, top_k, experts, id_type):
    rng = np.random.default_rng(tokens + experts)
    for same in (False, True):
        ids = routing(rng, tokens, top_k, experts, same=same)
        offs, src, pos = mx.moe_plan(torch.from_numpy(ids).to(DEV).to(id_type), experts)
        if id_type == torch.int32:
            ids = ids.astype(np.int32)
        want = O.moe_plan(ids, experts)
        for got, w, name in zip((offs, src, pos), want, ("offs", "src", "pos")):
            assert_bytes_equal(host(got), w, f"{name} T={tokens} k={top_k} E={experts} same={same}")


def test_plan_takes_ids_of_the_types_limits():
    big = np.array([[2 ** 31, -2 ** 31], [2 ** 62, -2 ** 62], [2 ** 32, 2 ** 32 + 1], [0, 1]])
    offs, src, pos = mx.moe_plan(torch.from_numpy(big).to(DEV), 2)
    assert host(offs).tolist() == [0, 1, 2] and host(src)[:2].tolist() == [6, 7]
    assert np.all(host(src)[2:] == -1) and np.all(host(pos)[:3] == -1)


# ------------------------------------------------------------------ dispatch
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,cols,pad", [
    (1, 1, 1, 0), (1, 4, 8, 0), (5, 2, 33, 0), (7, 3, 33, 7), (3, 9, 40, 0), (64, 4, 264, 8),
    (33, 2, 2880, 0), (19, 1, 385, 3), (300, 6, 96, 4), (40, 17, 24, 0)])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch(dtype, tokens, top_k, cols, pad, weighted):
    rng = np.random.default_rng(cols)
    _, _, pos = O.moe_plan(routing(rng, tokens, top_k, 6), 6)
    rows = tokens * top_k + 2
    a = stored(rng.standard_normal((tokens, cols)), dtype)
    w = rng.standard_normal(pos.shape).astype(np.float32)
    w[pos < 0] = np.nan
    out = torch.full((rows, cols + pad), -7.0, dtype=torch_type(dtype), device=DEV)
    x = strided(a, dtype, cols + pad)
    got = mx.moe_dispatch(x, dev_i32(pos), dev_f32(w) if weighted else None, out=out[:, :cols])
    want = O.moe_dispatch(oracle_input(a, dtype), pos, w if weighted else None, np.full((rows, cols), -7.0))
    err = np.abs(values(got) - want)
    tol = (2.0 ** -24 + STEP[dtype]) * np.abs(want) + TINY if weighted else 0.0
    assert np.all(err <= tol), err.max()
    assert np.all(values(out)[:, cols:] == -7.0)


def test_dispatch_copies_nan_and_infinity_bits():
    a = np.array([[0x7FC1, 0xFFC0, 0x7F80, 0xFF80, 0x8000, 0x0001, 0x7F81, 0x3F80]], np.uint16)
    for cols in (8, 7):
        got = mx.moe_dispatch(upload(a[:, :cols], "bf16"), dev_i32([[1, 0]]))
        assert np.array_equal(host(got), np.repeat(a[:, :cols], 2, 0))
    f = a.astype(np.uint32) << 16 | 0x1234
    got = mx.moe_dispatch(torch.from_numpy(f.view(np.float32)).to(DEV), dev_i32([[1, 0]]))
    assert np.array_equal(host(got).view(np.uint32), np.repeat(f, 2, 0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,cols,pad,pitch", [
    (1, 1, 32, 0, 1), (5, 3, 96, 0, 3), (9, 2, 160, 8, 16), (31, 4, 2880, 0, 96), (6, 2, 64, 5, 7),
    (130, 8, 384, 0, 12), (3, 4, 1056, 1, 33), (17, 19, 128, 0, 4)])
def test_dispatch_quantize_equals_quantizing_the_gathered_rows(dtype, tokens, top_k, cols, pad, pitch):
    rng = np.random.default_rng(cols + tokens)
    _, _, pos = O.moe_plan(routing(rng, tokens, top_k, 5), 5)
    rows = tokens * top_k + 1
    v = rng.standard_t(3, (tokens, cols)).astype(np.float32)
    v[0, :32] = 0.0
    v[tokens // 2, 32 % cols] = np.inf
    v[tokens - 1, cols - 1] = np.nan
    v[0, 5] = -0.0
    a = stored(v, dtype)
    codes = torch.full((rows, cols // 2), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, pitch), 0xCD, dtype=torch.uint8, device=DEV)
    mx.moe_dispatch_quantize(strided(a, dtype, cols + pad), dev_i32(pos), out=(codes, scales))
    want_c, want_s = np.full(codes.shape, 0xAB, np.uint8), np.full(scales.shape, 0xCD, np.uint8)
    with np.errstate(invalid="ignore"):
        qc, qs = O.quantize(oracle_input(a, dtype), O.ROW, O.RNE)
    for t, j in np.argwhere(pos >= 0):
        want_c[pos[t, j]], want_s[pos[t, j], :cols // 32] = qc[t], qs[t]
    assert_bytes_equal(host(codes), want_c, "codes")
    assert_bytes_equal(host(scales), want_s, "scales")


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("z_type", ["f32", "bf16"])
@pytest.mark.parametrize("y_type", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,cols,pad", [
    (1, 1, 1, 0), (1, 8, 16, 0), (5, 2, 33, 0), (7, 3, 33, 7), (3, 9, 40, 0), (64, 4, 264, 8),
    (33, 2, 2880, 0), (19, 1, 385, 3), (300, 6, 96, 4), (40, 17, 24, 0)])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(z_type, y_type, tokens, top_k, cols, pad, weighted):
    rng = np.random.default_rng(cols)
    _, _, pos = O.moe_plan(routing(rng, tokens, top_k, 6), 6)
    rows = tokens * top_k + 2
    v = rng.standard_normal((rows, cols))
    v[np.setdiff1d(np.arange(rows), pos)] = np.nan           # rows no slot maps to
    a = stored(v, z_type)
    w = rng.standard_normal(pos.shape).astype(np.float32)
    w[pos < 0] = np.nan
    out = torch.full((tokens, cols + pad), -7.0, dtype=torch_type(y_type), device=DEV)
    got = mx.moe_combine(strided(a, z_type, cols + pad), dev_i32(pos), dev_f32(w) if weighted else None,
                         out=out[:, :cols])
    want, mag = O.moe_combine(oracle_input(a, z_type), pos, w if weighted else None)
    err = np.abs(values(got) - want)
    assert np.all(err <= (top_k + 1) * 2.0 ** -24 * mag + STEP[y_type] * np.abs(want) + TINY), err.max()
    assert np.all(values(out)[:, cols:] == -7.0)
    if tokens > 2:
        assert np.all(values(got)[1] == 0.0)                 # the token without any expert


def test_combine_passes_nan_and_infinity_of_mapped_rows_only():
    z = torch.tensor([[1.0, 2.0], [float("inf"), 3.0], [float("nan"), 4.0]], device=DEV)
    pos = dev_i32([[0, 1], [0, -1], [2, 0], [-1, -1], [99, -5]])
    w = dev_f32([[1, 1], [1, np.nan], [1, 1], [np.inf, np.nan], [1, 1]])
    y = host(mx.moe_combine(z, pos, w))
    assert np.isposinf(y[0, 0]) and y[0, 1] == 5 and y[1].tolist() == [1, 2]
    assert np.isnan(y[2, 0]) and y[2, 1] == 6 and np.all(y[3:] == 0)
    dz, dw = mx.moe_combine_bwd(torch.ones(5, 2, device=DEV), z, pos, w,
                                out=torch.full((3, 2), 9.0, device=DEV))
    dw = host(dw)
    assert dw[0].tolist() == [3, np.inf] and dw[1].tolist() == [3, 0] and np.isnan(dw[2, 0])
    assert np.all(dw[3:] == 0)


def test_combine_without_rows_is_zero():
    y = mx.moe_combine(torch.empty((0, 24), device=DEV), dev_i32([[0, -1]] * 3))
    assert y.shape == (3, 24) and np.all(host(y) == 0)


@pytest.mark.parametrize("g_type", ["f32", "bf16"])
@pytest.mark.parametrize("z_type", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,cols,pad", [
    (1, 1, 1, 0), (1, 8, 16, 0), (5, 2, 33, 0), (7, 3, 33, 7), (3, 9, 40, 0), (64, 4, 264, 8),
    (33, 2, 2880, 0), (19, 1, 385, 3), (300, 6, 96, 4), (40, 17, 24, 0), (2, 2, 14336, 0)])
def test_combine_gradient(g_type, z_type, tokens, top_k, cols, pad):
    rng = np.random.default_rng(cols)
    _, _, pos = O.moe_plan(routing(rng, tokens, top_k, 6), 6)
    rows = tokens * top_k + 2
    v = rng.standard_normal((rows, cols))
    v[np.setdiff1d(np.arange(rows), pos)] = np.nan
    a, g = stored(v, z_type), stored(rng.standard_normal((tokens, cols)) * 1e-3, g_type)
    w = rng.standard_normal(pos.shape).astype(np.float32)
    w[pos < 0] = np.nan
    for weights in (w, None):
        out = torch.full((rows, cols + pad), -7.0, dtype=torch_type(g_type), device=DEV)
        dz, dw = mx.moe_combine_bwd(strided(g, g_type, cols + pad), strided(a, z_type, cols + pad), dev_i32(pos),
                                    None if weights is None else dev_f32(weights), out=out[:, :cols])
        want, want_w, mag = O.moe_combine_bwd(oracle_input(g, g_type), oracle_input(a, z_type), pos, weights,
                                              np.full((rows, cols), -7.0))
        err = np.abs(values(dz) - want)
        tol = 0.0 if weights is None else (2.0 ** -24 + STEP[g_type]) * np.abs(want) + TINY
        assert np.all(err <= tol), err.max()
        assert np.all(values(out)[:, cols:] == -7.0)
        # any order of cols float32 additions stays within cols + 1 roundings of the magnitudes
        err = np.abs(values(dw) - want_w)
        assert np.all(err <= (cols + 1) * 2.0 ** -24 * mag + TINY), err.max()


def test_combine_gradient_against_differences():
    """The loss sum(dy * combine(z, w)) is linear in z and in w, so the difference over a step of
    any size is the gradient; powers of two keep every value exact in float32."""
    rng = np.random.default_rng(5)
    ids = torch.from_numpy(rng.integers(-1, 3, (4, 2))).to(DEV)
    _, _, pos = mx.moe_plan(ids, 3)
    pick = lambda *s: torch.from_numpy(rng.choice([-2.0, -1.0, -0.5, 0.5, 1.0, 2.0], s).astype(np.float32)).to(DEV)
    z, w, dy = pick(8, 8), pick(4, 2), pick(4, 8)
    dz, dw = mx.moe_combine_bwd(dy, z, pos, w, out=torch.zeros_like(z))
    loss = lambda: float((dy * mx.moe_combine(z, pos, w)).double().sum())  # noqa: E731
    base = loss()
    for a, grad in ((z, dz), (w, dw)):
        for i in np.ndindex(*a.shape):
            a[i] += 4.0
            assert loss() - base == 4.0 * float(grad[i])
            a[i] -= 4.0


def test_results_are_the_same_in_every_run():
    rng = np.random.default_rng(6)
    _, _, pos = mx.moe_plan(torch.from_numpy(rng.integers(0, 8, (3000, 4))).to(DEV), 8)
    z, dy = torch.randn(12000, 320, device=DEV), torch.randn(3000, 320, device=DEV)
    w = torch.rand(3000, 4, device=DEV)
    first = [mx.moe_combine(z, pos, w), *mx.moe_combine_bwd(dy, z, pos, w)]
    for _ in range(4):
        for a, b in zip(first, [mx.moe_combine(z, pos, w), *mx.moe_combine_bwd(dy, z, pos, w)]):
            assert torch.equal(a, b)


def test_rows_past_two_to_the_31_elements():
    """Offsets past 2^31 elements in the expert-ordered matrices: 500000 rows of 4608."""
    rows, cols = 500_000, 4608
    z = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    pos = dev_i32([[rows - 1, 3], [7, rows - 2], [480_001, -1]])
    x = torch.randn(3, cols, device=DEV).to(torch.bfloat16)
    mx.moe_dispatch(x, pos, out=z)
    assert torch.equal(z[pos[:2].long()], x[:2, None].expand(2, 2, cols)) and torch.equal(z[480_001], x[2])
    assert int((z != 0).any(dim=1).sum()) == 5
    y = mx.moe_combine(z, pos, out_dtype=torch.bfloat16)
    assert torch.equal(y[:2], (x[:2].float() * 2).to(torch.bfloat16)) and torch.equal(y[2], x[2])
    dz, dw = mx.moe_combine_bwd(x, z, pos, out=torch.zeros_like(z))
    assert torch.equal(dz[480_001], x[2]) and torch.equal(dz[rows - 1], x[0])
    want = (x.double() ** 2).sum(dim=1, keepdim=True) * (pos >= 0)
    assert torch.all((dw - want).abs() <= (cols + 1) * 2.0 ** -24 * want)
