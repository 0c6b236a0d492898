"""CPU checks of the rule that gives a product of 8-bit matrices its kernel (csrc/gemm8_plan.h, compiled here on its
own): the shapes of the GPU tests reach the kernels that these tests are written for, also after costs are
measured anew, and slices cover the contraction."""
import ctypes
import os
import random
import subprocess

import pytest

from tests import test_gpu_gemm8 as G
from tests import test_gpu_gemm8_exact as X

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp4_microscaling_quantization_amd", "csrc")
SOURCE = """
#include "gemm8_plan.h"
extern "C" void plan(int64_t M, int64_t N, int64_t K, int wide, int64_t* out) {
  const mx::Plan8 p = mx::gemm8_plan(M, N, (K + 15) / 16 * 16, wide != 0);
  out[0] = p.rows, out[1] = p.big, out[2] = p.whole, out[3] = p.slices, out[4] = p.slice;
  out[5] = (int64_t)mx::plan8_bytes(p, M, N);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    path = tmp_path_factory.mktemp("plan")
    (path / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(path / "plan.cpp"),
                    "-o", str(path / "plan.so")], check=True)
    call = ctypes.CDLL(str(path / "plan.so")).plan
    call.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]
    call.restype = None

    def ask(M, N, K, wide):
        out = (ctypes.c_int64 * 6)()
        call(M, N, K, wide, out)
        return dict(zip(("rows", "big", "whole", "slices", "slice", "bytes"), out))

    return ask


def kind(p):
    if p["rows"]:
        return "rows"
    if p["big"]:
        return "tiles of 256"
    if p["slices"] == 1:
        return "tiles of 128"
    return "last tiles in slices" if p["whole"] else "slices"


@pytest.mark.parametrize("wide", [0, 1])
@pytest.mark.parametrize("name,shapes", [
    ("rows", X.ROWS), ("tiles of 128", X.TILES), ("slices", X.SLICED), ("last tiles in slices", X.TAIL),
    ("tiles of 256", X.BIG), ("tiles of 256", G.NAN_SCALES_BIG), ("slices", G.NAN_SCALES_SLICED)])
def test_shapes_reach_the_kernels_they_are_listed_for(plan, name, shapes, wide):
    assert shapes and {s: kind(plan(*s, wide)) for s in shapes} == {s: name for s in shapes}


def test_the_large_shapes_end_in_every_way():
    """Whole and partial last steps, odd and even numbers of steps of 128, ragged rows and columns of tiles of 256."""
    steps = {(-(-k // 128) % 2, -(-k // 16) * 16 % 128 == 0) for _, _, k in X.BIG}
    assert steps == {(0, True), (0, False), (1, True), (1, False)}
    assert {-(-k // 16) * 16 % 128 > 64 for _, _, k in X.BIG} == {True, False}
    for axis in (0, 1):
        ends = [s[axis] % 256 for s in X.BIG]
        assert any(0 < e <= 64 for e in ends) and any(e > 128 for e in ends)
    assert any(m % 256 == 1 for m, _, _ in X.BIG) and any(n % 256 == 0 or n % 256 == 128 for _, n, _ in X.BIG)


def test_slices_cover_the_contraction(plan):
    rng = random.Random(0)
    size = lambda high: int(2 ** rng.uniform(0, high))  # noqa: E731
    seen = set()
    for _ in range(4000):
        M, N, K, wide = size(15), size(15), size(17), rng.randrange(2)
        p, tiles, k = plan(M, N, K, wide), -(-M // 128) * -(-N // 128), -(-K // 16) * 16
        seen.add(kind(p))
        if p["slices"] == 1:
            assert p["bytes"] == 0
            continue
        assert not p["rows"] and not p["big"] and p["slice"] % 512 == 0 and 0 <= p["whole"] < tiles
        assert p["whole"] % 512 == 0 and tiles - p["whole"] < 256 and (tiles - p["whole"]) * p["slices"] <= 512
        assert (p["slices"] - 1) * p["slice"] < k <= p["slices"] * p["slice"]
        assert p["bytes"] == (tiles - p["whole"]) * p["slices"] * 128 * 128 * 4
    assert len(seen) == 5
