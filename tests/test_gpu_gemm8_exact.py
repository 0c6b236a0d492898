"""GPU checks of each kernel of the 8-bit products on operands whose products and sums are exact: every output, bit
for bit.

Codes are the whole numbers -3 .. 3 and scales 2^-1, 1 or 2, so a product is a multiple of 2^-2 of at most 36, and a
sum of K of them a multiple of 2^-2 below 2^22 as long as K <= 2^24 / 144: float32 holds every partial sum in any
order, also over slices.  The 8-bit instructions keep 13 bits below the largest of eight neighbouring products, which
share their scales: from 9 down to 1 are 4 bits.  alpha = -3 / 8 multiplies by three once more.  So a float32 C is
the float64 sum itself, and a bf16 C that rounded once.  Missing, doubled or misplaced values of the last steps, rows
or columns show whatever their share.

Which kernel a shape takes is a matter of measured costs; a CPU test holds these lists to their names."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mx
from tests.gpu_util import DEV
from tests.test_gpu_moe_routing import torch_type

pytestmark = pytest.mark.gpu

ROWS = [(1, 77, 1300), (5, 8300, 130), (16, 33, 2047), (33, 100, 4100), (48, 8191, 640), (64, 257, 14336)]
TILES = [(65, 40, 700), (197, 1536, 384), (300, 300, 320), (1001, 260, 33), (6000, 1100, 96), (3841, 4097, 1344)]
SLICED = [(65, 1000, 4176), (128, 4096, 2048), (260, 130, 30000), (129, 127, 14000)]     # every tile in slices
TAIL = [(3400, 2400, 4112), (3330, 2433, 4100), (2300, 3700, 5000)]                       # those behind full rounds
# tiles of 256: whole last steps and partial ones of 16 to 112 values, odd and even numbers of steps, rows and columns
# that end inside a tile by one, by half and more
BIG = [(3900, 3850, 1300), (4096, 3500, 4176), (3800, 3584, 2880), (4000, 3900, 1280), (3700, 3700, 1408), (7700, 1950, 2000),
       (1950, 7700, 1250), (12500, 1250, 1700), (4093, 4001, 1409), (3841, 4096, 3713)]


def operand(rows, K, g):
    """An 8-bit matrix, 0xFF where scale rows are padded, and its values in float64."""
    v = torch.randint(-3, 4, (rows, K), generator=g, device=DEV)
    table = torch.tensor([0xC4, 0xC0, 0xB8, 0, 0x38, 0x40, 0x44], dtype=torch.uint8, device=DEV)
    codes = torch.zeros((rows, -(-K // 16) * 16), dtype=torch.uint8, device=DEV)
    codes[:, :K] = table[v + 3]
    blocks = -(-K // 128)
    s = torch.randint(126, 129, (rows, blocks), generator=g, device=DEV)
    scales = torch.full((rows, -(-K // 512) * 4), 0xFF, dtype=torch.uint8, device=DEV)
    scales[:, :blocks] = s.to(torch.uint8)
    power = torch.exp2((s - 127).double()).repeat_interleave(128, dim=1)[:, :K]
    return (codes, scales), v.double() * power


@pytest.mark.parametrize("M,N,K", ROWS + TILES + SLICED + TAIL + BIG)
def test_every_output_is_exact(M, N, K):
    assert K <= 2 ** 24 // (3 * 144)
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    (a, va), (b, vb) = operand(M, K, g), operand(N, K, g)
    want = torch.mm(va, vb.t().contiguous())
    for y_type in ("f32", "bf16"):
        t = torch_type(y_type)
        got = mx.gemm8(a, b, out_dtype=t)
        bad = got != want.float().to(t)
        assert not bad.any(), (y_type, int(bad.sum()), bad.nonzero()[:4].tolist(), bad.nonzero()[-4:].tolist())
        out = torch.full((M + 1, N + 7), 7.0, dtype=t, device=DEV)     # rows at odd places, a factor
        mx.gemm8(a, b, alpha=-0.375, out=out[:M, :N])
        bad = out[:M, :N] != (want * -0.375).float().to(t)
        assert not bad.any(), (y_type, int(bad.sum()), bad.nonzero()[:4].tolist(), bad.nonzero()[-4:].tolist())
        assert torch.all(out[M:] == 7.0) and torch.all(out[:, N:] == 7.0)


@pytest.mark.parametrize("M,N,K", [(2048, 2050, 2100), (4200, 1300, 1290), (3900, 3850, 1300), (130, 4200, 300)])
def test_both_gradients_are_exact(M, N, K):
    """The layer's backward, both products in a launch or one after the other: dY and X are what their second
    quantization keeps (whole numbers up to 3)."""
    g = torch.Generator(device=DEV).manual_seed(M)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device=DEV).float()  # noqa: E731
    x, w, dy = whole(M, K), whole(N, K), whole(M, N)
    y, xq, wq = mx.linear8_fwd(x, w)
    assert torch.equal(y, torch.mm(x.double(), w.double().t().contiguous()).float())
    for t in (torch.float32, torch.bfloat16):
        dx, dw = mx.linear8_bwd(dy, xq, wq, M, N, K, dx_dtype=t)
        assert torch.equal(dx, torch.mm(dy.double(), w.double()).float().to(t))
        assert torch.equal(dw, torch.mm(dy.double().t().contiguous(), x.double()).float())
