"""GPU checks of the few-row products with packed weights (mx_gemv, mx_gemv_grouped) against the
float64 oracle.

Tolerance: every product of x and an E2M1 value times a power of two is exact in float32 or is a
sum of at most three such terms, so only the additions round.  With 3 terms per value the longest
chain of additions over K values is below 3 K / 32 + 64 (32 values meet inside a matrix instruction,
the rest are instructions, lanes and waves in a row); each is counted as a full step 2^-23 of the
magnitudes' sum, since the matrix unit's inner additions may truncate.  Times alpha and the rounding
to the output type: 2^-24 and 2^-24 or 2^-8 of the value.  2^-120 covers products below the normal
range under extreme scales."""
import numpy as np
import pytest
import torch

import oracle as O
from mxfp4_microscaling_quantization_amd import mx
from tests.gpu_util import DEV, host, oracle_input, to_dev_u8
from tests.test_gpu_moe_routing import STEP, dev_i32, routing, stored, strided, torch_type, values

pytestmark = pytest.mark.gpu


def weights(rng, shape, K, pitch=None, low=110, high=140):
    codes = rng.integers(0, 256, (*shape, K // 2), dtype=np.uint8)
    scales = rng.integers(low, high, (*shape, pitch or K // 32), dtype=np.uint8)
    scales[..., K // 32:] = 0xFF                    # padding bytes are never used
    return codes, scales


def check(got, want, mag, K, y_type, what=""):
    got, real = values(got), np.isfinite(want)
    assert np.array_equal(np.isfinite(got), real), what
    tol = (3 * K / 32 + 64) * 2.0 ** -23 * mag + (2.0 ** -24 + STEP[y_type]) * np.abs(want) + 2.0 ** -120
    err = np.abs(got - want)
    bad = real & (err > tol)
    assert not bad.any(), (what, np.argwhere(bad)[:4], float((err / tol)[real].max()))


def few_rows(rng, M, K, x_type):
    x = rng.standard_normal((M, K))
    x[:, rng.integers(0, K, max(1, K // 100))] *= 30.0
    return stored(x, x_type)


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 5, 64), (1, 64, 96), (1, 17, 128), (2, 63, 160), (15, 65, 256), (16, 130, 288),
    (17, 31, 1056), (31, 200, 544), (33, 129, 416), (64, 64, 1024), (65, 48, 224), (130, 33, 512),
    (1, 1536, 384), (1, 2880, 2880), (5, 333, 14336), (48, 77, 4096), (1, 3, 20480)])
def test_gemv(x_type, M, N, K):
    rng = np.random.default_rng(M + N + K)
    a = few_rows(rng, M, K, x_type)
    codes, scales = weights(rng, (N,), K)
    want, mag = O.gemv(oracle_input(a, x_type), codes, scales)
    w = to_dev_u8(codes), to_dev_u8(scales)
    x = strided(a, x_type, K)
    for y_type in ("f32", "bf16"):
        check(mx.gemv(x, w, out_dtype=torch_type(y_type)), want, mag, K, y_type, (M, N, K))


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("y_type", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,x_pad,y_pad,pitch", [
    (1, 9, 64, 3, 0, 2), (3, 65, 160, 1, 5, 7), (20, 130, 224, 8, 2, 16), (5, 16, 2880, 0, 16, 96),
    (40, 34, 96, 2, 1, 3), (66, 20, 128, 4, 3, 5)])
def test_gemv_strides_and_alpha(x_type, y_type, M, N, K, x_pad, y_pad, pitch):
    rng = np.random.default_rng(N)
    a = few_rows(rng, M, K, x_type)
    codes, scales = weights(rng, (N,), K, pitch)
    want, mag = O.gemv(oracle_input(a, x_type), codes, scales, -0.3)
    out = torch.full((M, N + y_pad), 77.0, dtype=torch_type(y_type), device=DEV)
    got = mx.gemv(strided(a, x_type, K + x_pad), (to_dev_u8(codes), to_dev_u8(scales)), alpha=-0.3, out=out[:, :N])
    check(got, want, mag, K, y_type)    # alpha's own rounding is inside the chain's count
    assert np.all(values(out)[:, N:] == 77.0)


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
def test_gemv_takes_x_at_full_precision(x_type):
    """One non-zero per row: y is that value times an E2M1 value, exactly."""
    rng = np.random.default_rng(1)
    K, N = 256, 16
    a = stored(np.diag(np.ldexp(rng.uniform(1, 2, K), rng.integers(-100, 100, K))), x_type)
    codes, scales = weights(rng, (N,), K, low=127, high=128)
    got = mx.gemv(strided(a, x_type, K), (to_dev_u8(codes), to_dev_u8(scales)))
    want = oracle_input(a, x_type).diagonal().astype(np.float64)[:, None] * O.dequantize(codes, scales, N, K).T
    assert np.array_equal(host(got), want.astype(np.float32))


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("byte,power", [(0, 120), (1, 120), (2, 110), (60, 60), (200, -70), (252, -120), (254, -124)])
def test_gemv_extreme_scales(x_type, byte, power):
    """Block scales at both ends, with rows of the opposite magnitude: results stay ordinary."""
    rng = np.random.default_rng(byte)
    M, N, K = 3, 20, 96
    a = stored(np.ldexp(rng.uniform(1, 2, (M, K)) * rng.choice([-1, 1], (M, K)), power), x_type)
    codes, scales = weights(rng, (N,), K, low=byte, high=byte + 1)
    if byte > 252:                      # no quantizer writes these: codes above 1.5 pass the float32 range
        codes &= 0xBB
    want, mag = O.gemv(oracle_input(a, x_type), codes, scales)
    if x_type == "f32":
        # The three bf16 terms of a float32 value hold its bits down to bf16's smallest subnormal:
        # truncation leaves x - hi - mid - lo in [0, 2^-133), so a sum misses below 2^-133 sum |w|.
        # Written as magnitudes for check(), which multiplies them by 2^-23 and a count above 64.
        dropped = 2.0 ** -133 * np.abs(O.dequantize(codes, scales, N, K)).sum(axis=1)
        mag = mag + dropped / (64 * 2.0 ** -23)
    check(mx.gemv(strided(a, x_type, K), (to_dev_u8(codes), to_dev_u8(scales))), want, mag, K, "f32", byte)


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 96), (3, 4096), (20, 160)])
def test_gemv_nan_and_infinity(x_type, M, K):
    """NaN and Inf reach their own row or column only, whatever lies in the tails beside them."""
    rng = np.random.default_rng(2)
    N = 37
    a = few_rows(rng, M, K, x_type)
    codes, scales = weights(rng, (N,), K)
    codes = np.where(codes & 0x0F == 0, codes | 1, codes)
    codes = np.where(codes & 0x70 == 0, codes | 0x10, codes)   # no zero codes: Inf stays Inf
    codes = np.where(codes & 0x07 == 0, codes | 1, codes).astype(np.uint8)
    scales[5, K // 32 - 1] = 0xFF
    f = oracle_input(a, x_type).copy()
    f[M - 1, K - 1] = np.inf
    if M > 1:
        f[0, 0] = np.nan
    a = stored(f, x_type)
    if M > 1 and x_type == "f32":
        a.view(np.uint32)[0, 0] = 0x7F800001                   # a NaN with only low bits
    want, mag = O.gemv(oracle_input(a, x_type), codes, scales)
    got = host(mx.gemv(strided(a, x_type, K), (to_dev_u8(codes), to_dev_u8(scales))))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert np.all(np.isfinite(got) == np.isfinite(want))


def test_gemv_empty_contraction_and_no_rows():
    for K, M in ((0, 3), (64, 0)):
        w = torch.zeros((5, K // 2), dtype=torch.uint8, device=DEV), torch.zeros((5, K // 32), dtype=torch.uint8, device=DEV)
        y = mx.gemv(torch.ones((M, K), device=DEV), w)
        assert y.shape == (M, 5) and np.all(host(y) == 0)


def test_gemv_matches_the_library_s_own_product_of_quantized_rows():
    """Rows that are exact in MXFP4: mx_gemm on the packed rows and mx_gemv on the rows agree."""
    rng = np.random.default_rng(3)
    M, N, K = 24, 96, 512
    x = mx.dequantize(*mx.quantize(torch.randn(M, K, device=DEV)), M, K)
    codes, scales = weights(rng, (N,), K, low=120, high=130)
    w = to_dev_u8(codes), to_dev_u8(scales)
    want, mag = O.gemv(host(x), codes, scales)
    check(mx.gemm(mx.quantize(x), w, M, N, K), want, mag, K, "f32")
    check(mx.gemv(x, w), want, mag, K, "f32")
    check(mx.gemv(x.to(torch.bfloat16), w), want, mag, K, "f32")


def test_gemv_weights_past_two_to_the_31_bytes():
    N, K = 700_000, 6400                                # 2.24e9 bytes of codes
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    codes[N - 3] = 0x22
    codes[671_100] = 0x44
    x = torch.ones((2, K), dtype=torch.bfloat16, device=DEV)
    y = mx.gemv(x, (codes, scales))
    assert host(y[:, [N - 3, 671_100]]).tolist() == [[K, 2 * K]] * 2
    assert int((y != 0).sum()) == 4


def test_gemv_of_the_most_rows():
    """2^31 - 1 rows, dense and of one expert, with nothing to sum: y is 0 in every row."""
    M = 2**31 - 1
    x = torch.empty((M, 0), dtype=torch.bfloat16, device=DEV)
    codes = torch.empty((1, 1, 0), dtype=torch.uint8, device=DEV)
    y = torch.ones((M, 1), dtype=torch.bfloat16, device=DEV)
    mx.gemv(x, (codes[0], codes[0]), out=y)
    assert torch.equal(y.amax(), y.amin()) and float(y[0]) == 0
    y.fill_(1)
    offs = torch.tensor([0, M], device=DEV)
    mx.gemv_grouped(x, (codes, codes), offs, out=y)
    assert torch.equal(y.amax(), y.amin()) and float(y[0]) == 0


# ------------------------------------------------------------------ grouped
@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,experts,N,K,left_out", [
    (1, 1, 1, 1, 32, 0.0), (1, 4, 32, 70, 96, 0.0), (3, 2, 128, 64, 160, 0.3), (16, 4, 8, 33, 288, 0.2),
    (61, 4, 32, 100, 416, 0.0), (40, 3, 2, 65, 128, 0.1), (64, 8, 4, 48, 544, 0.5), (9, 6, 60, 130, 2880, 0.0)])
def test_gemv_grouped(x_type, tokens, top_k, experts, N, K, left_out):
    rng = np.random.default_rng(tokens + N)
    a = few_rows(rng, tokens, K, x_type)
    codes, scales = weights(rng, (experts, N), K, K // 32 + 2)
    w = to_dev_u8(codes), to_dev_u8(scales)
    ids = routing(rng, tokens, top_k, experts, left_out)
    offs, src, pos = mx.moe_plan(torch.from_numpy(ids).to(DEV), experts)
    want, mag = O.gemv_grouped(oracle_input(a, x_type), codes, scales, host(offs), host(src), top_k, tokens * top_k)
    held = int(host(offs)[-1])
    for y_type in ("f32", "bf16"):
        out = torch.full((tokens * top_k, N), 5.0, dtype=torch_type(y_type), device=DEV)
        got = mx.gemv_grouped(strided(a, x_type, K), w, offs, src, top_k, out=out)
        check(got[:held], want[:held], mag[:held], K, y_type, (tokens, top_k, experts))
        assert np.all(values(got[held:]) == 5.0)        # rows behind the last expert's stay


def test_gemv_grouped_rows_of_their_own_and_one_expert_that_takes_all():
    rng = np.random.default_rng(4)
    N, K, rows = 40, 192, 90
    codes, scales = weights(rng, (5, N), K)
    w = to_dev_u8(codes), to_dev_u8(scales)
    a = few_rows(rng, rows, K, "bf16")
    x = strided(a, "bf16", K + 8)
    for ends in ([0, 0, 90, 90, 90, 90], [0, 1, 2, 2, 60, 90], [0, 0, 0, 0, 0, 90], [0] * 6):
        offs = torch.tensor(ends, device=DEV)
        out = torch.full((rows, N), 5.0, device=DEV)
        mx.gemv_grouped(x, w, offs, alpha=2.0, out=out)
        want, mag = O.gemv_grouped(oracle_input(a, "bf16"), codes, scales, ends, None, 1, rows, 2.0)
        check(out[:ends[-1]], want[:ends[-1]], mag[:ends[-1]], K, "f32", ends)
        assert np.all(host(out[ends[-1]:]) == 5.0)


def test_gemv_grouped_leaves_rows_whose_source_is_outside_x():
    rng = np.random.default_rng(5)
    codes, scales = weights(rng, (2, 20), 64)
    a = few_rows(rng, 3, 64, "f32")
    src = dev_i32([0, 5, 6, -1, 100, 3])
    out = torch.full((6, 20), 5.0, device=DEV)
    mx.gemv_grouped(strided(a, "f32", 64), (to_dev_u8(codes), to_dev_u8(scales)),
                    torch.tensor([0, 4, 6], device=DEV), src, 2, out=out)
    want, mag = O.gemv_grouped(oracle_input(a, "f32"), codes, scales, [0, 4, 6], host(src), 2, 6)
    real = np.array([0, 1, 5])
    check(out[real], want[real], mag[real], 64, "f32")
    assert np.all(host(out)[[2, 3, 4]] == 5.0)


def test_results_are_the_same_in_every_run():
    rng = np.random.default_rng(7)
    codes, scales = weights(rng, (300,), 2880)
    w = to_dev_u8(codes), to_dev_u8(scales)
    x = torch.randn(16, 2880, device=DEV)
    first = mx.gemv(x, w)
    for _ in range(4):
        assert torch.equal(mx.gemv(x, w), first)
