"""GPU checks of the few-row products whose contraction is longer than a workgroup's windows and
goes in rounds of them, and of those whose contraction is empty.  References are float64 products
of the decoded weights on the device.  Tolerances are those of
test_gpu_gemv: a round adds its waves' sums to the rounds' before, which its count of additions
covers (a round is at least 128 values, counted as 12 additions, and adds one)."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mx
from tests.gpu_util import DEV, host, oracle_input, to_dev_u8
from tests.test_gpu_gemv import check, few_rows, weights
from tests.test_gpu_moe_routing import STEP, dev_i32, routing, strided, torch_type, values

pytestmark = pytest.mark.gpu


def decoded(codes, scales, K):
    """float64 values [..., K] of packed device matrices, by a table and a power of two."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    table = torch.cat([table, -table])
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], dim=-1).flatten(-2)
    byte = scales[..., :K // 32].long()
    power = (byte - 127 + 1023 << 52).view(torch.float64)       # 2^(byte - 127) from its bits
    power = torch.where(byte == 255, torch.full_like(power, float("nan")), power)
    return v * power.repeat_interleave(32, dim=-1)


def product(x64, w64):
    """(x w^T, sum of magnitudes) in float64."""
    return x64 @ w64.t().contiguous(), x64.abs() @ w64.abs().t().contiguous()


# the rows up to which a contraction of two windows stays in rounds, by the type of x
ROUNDS_ROWS = {"bf16": 8, "f32": 2}


@pytest.mark.parametrize("x_type,M,N,K", [
    (t, M, N, K) for t in ("f32", "bf16") for M, N, K in (
        (1, 300, 8192),                # two rounds, whole windows
        (ROUNDS_ROWS[t], 300, 8192),
        (ROUNDS_ROWS[t], 77, 4128),    # two rounds, most windows short, some empty
        (1, 4161, 14336),              # four rounds
        (ROUNDS_ROWS[t], 4161, 12320),
        (ROUNDS_ROWS[t], 17001, 4128))])   # several tiles a workgroup
def test_gemv_in_rounds(x_type, M, N, K):
    assert mx.mx_gemv_workspace_size(mx.MX_BF16 if x_type == "bf16" else mx.MX_F32, M, N, K) == 0
    rng = np.random.default_rng(M + N + K)
    a = few_rows(rng, M, K, x_type)
    codes, scales = weights(rng, (N,), K, K // 32 + 3)
    w = to_dev_u8(codes), to_dev_u8(scales)
    x = strided(a, x_type, K + 5)
    want, mag = product(x.double(), decoded(*w, K))
    for y_type in ("f32", "bf16"):
        got = mx.gemv(x, w, alpha=0.5, out_dtype=torch_type(y_type))
        check(got, values(0.5 * want), values(0.5 * mag), K, y_type, (M, N, K))


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,experts,N,K,left_out", [
    (1, 2, 8, 200, 14336, 0.0),        # a decode step's single token, four rounds
    (19, 3, 5, 130, 4128, 0.2),        # ragged groups, two rounds
    (60, 2, 3, 70, 5760, 0.1),         # some 40 rows a group: several row tiles of both types
    (24, 4, 24, 1100, 4128, 0.1)])     # more tiles than workgroups
def test_gemv_grouped_in_rounds(x_type, tokens, top_k, experts, N, K, left_out):
    rng = np.random.default_rng(tokens + N)
    a = few_rows(rng, tokens, K, x_type)
    codes, scales = weights(rng, (experts, N), K, K // 32 + 1)
    w = to_dev_u8(codes), to_dev_u8(scales)
    ids = routing(rng, tokens, top_k, experts, left_out)
    if tokens == 1:
        ids[:] = [[6, 1]]
    offs, src, _ = mx.moe_plan(torch.from_numpy(ids).to(DEV), experts)
    slots, ends = host(src).copy(), host(offs)
    held, rows = int(ends[-1]), tokens * top_k
    if held > 8:                       # rows without a source: in front, inside and at the end
        slots[[0, held // 2, held - 1]] = [-1, tokens * top_k, 1 << 30]
    x = strided(a, x_type, K)
    want = torch.full((rows, N), float("nan"), dtype=torch.float64, device=DEV)
    mag = torch.full_like(want, float("nan"))
    for e in range(experts):
        mine = [r for r in range(int(ends[e]), int(ends[e + 1])) if 0 <= slots[r] < tokens * top_k]
        if mine:
            token = torch.from_numpy(slots[mine] // top_k).long().to(DEV)
            want[mine], mag[mine] = product(x[token].double(), decoded(w[0][e], w[1][e], K))
    real = ~np.isnan(values(want[:, 0]))
    assert real.sum() == held - (3 if held > 8 else 0)
    for y_type in ("f32", "bf16"):
        out = torch.full((rows, N + 3), 5.0, dtype=torch_type(y_type), device=DEV)
        mx.gemv_grouped(x, w, offs, dev_i32(slots), top_k, out=out[:, :N])
        got = out[torch.from_numpy(real).to(DEV)]
        check(got[:, :N], values(want)[real], values(mag)[real], K, y_type, (tokens, top_k, experts))
        assert np.all(values(got)[:, N:] == 5.0)
        assert np.all(values(out)[~real] == 5.0)      # rows without a source or behind the last


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
def test_nan_and_infinity_in_any_round_reach_their_own_row_or_column_only(x_type):
    rng = np.random.default_rng(2)
    M, N, K = 2, 4100, 14336 - 32      # four rounds: more than 64 column tiles are not sliced
    assert mx.mx_gemv_workspace_size(mx.MX_BF16 if x_type == "bf16" else mx.MX_F32, M, N, K) == 0
    codes, scales = weights(rng, (N,), K)
    codes |= 0x11                      # no zero codes: Inf stays Inf
    for at in (0, 5000, 9000, K - 1):
        s = scales.copy()
        s[5, at // 32] = 0xFF
        x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DEV).to(torch_type(x_type))
        x[1, at] = float("inf")
        w = to_dev_u8(codes), to_dev_u8(s)
        got = host(mx.gemv(x, w))
        column = codes[:, at // 2] >> (4 * (at % 2)) & 15
        assert np.all(np.isnan(got[:, 5])) and np.all(np.isfinite(np.delete(got[0], 5)))
        inf = np.where(column & 8, -np.inf, np.inf)
        assert np.array_equal(np.delete(got[1], 5), np.delete(inf, 5)), at


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(70, 65, 2304), (70, 40, 4128), (21, 300, 96), (40, 70, 14336)])
def test_each_of_many_rows_agrees_with_its_one_row_call(x_type, M, N, K):
    """The same sum in two orders: each is within the bound of the exact one."""
    rng = np.random.default_rng(M + K)
    codes, scales = weights(rng, (N,), K)
    w = to_dev_u8(codes), to_dev_u8(scales)
    x = strided(few_rows(rng, M, K, x_type), x_type, K)
    y = mx.gemv(x, w)
    one = torch.cat([mx.gemv(x[m:m + 1].clone(), w) for m in range(M)])
    _, mag = product(x.double(), decoded(*w, K))
    assert torch.all((y.double() - one.double()).abs() <= 2 * (3 * K / 32 + 64) * 2.0 ** -23 * mag)


@pytest.mark.parametrize("alpha", [-0.3, float("inf"), float("nan")])
def test_empty_contraction_is_zero_under_any_alpha(alpha):
    """As in the other products, K = 0 gives y = 0 without a look at alpha."""
    w = torch.empty((2, 5, 0), dtype=torch.uint8, device=DEV)
    y = torch.full((3, 5), 7.0, device=DEV)
    mx.gemv(torch.empty((3, 0), device=DEV), (w[0], w[0]), alpha=alpha, out=y)
    assert np.all(host(y) == 0)
    y.fill_(7.0)
    mx.gemv_grouped(torch.empty((3, 0), device=DEV), (w, w), torch.tensor([0, 1, 2], device=DEV), alpha=alpha, out=y)
    assert np.all(host(y[:2]) == 0) and np.all(host(y[2]) == 7)
