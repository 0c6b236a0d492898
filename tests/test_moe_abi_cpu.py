"""CPU checks of the routing and few-row entry points: arguments are refused before anything
is launched (no compute calls here), by the library and by the tensor conveniences."""
import os
import subprocess
import sys

import pytest
import torch

from mxfp4_microscaling_quantization_amd import build, mx
from tests.test_abi_sanitized import ROOT, sanitized_library

BAD = 0x1001       # non-null, misaligned
GOOD = 0x10000     # non-null, aligned: only reached by calls that fail validation
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    return mx.lib()


def test_gemv_validation(L):
    def call(x=GOOD, xt=1, ldx=64, c=GOOD, s=GOOD, pitch=2, M=1, N=5, K=64, y=GOOD, yt=0, ldy=5,
             ws=None, n=0):
        return L.mx_gemv(x, xt, ldx, c, s, pitch, M, N, K, 1.0, y, yt, ldy, ws, n, None)

    assert call(xt=2) == mx.MX_ERR_ENUM
    assert call(yt=-1) == mx.MX_ERR_ENUM
    for bad in ({"K": 48}, {"K": -32}, {"ldx": 63}, {"pitch": 1}, {"ldy": 4}, {"M": -1}, {"N": -1},
                {"M": BIG}, {"N": BIG, "ldy": BIG}, {"K": 1 << 26, "ldx": 1 << 26, "pitch": 1 << 21}, {"pitch": 1 << 26}):
        assert call(**bad) == mx.MX_ERR_SHAPE, bad
    for name in ("x", "c", "s", "y"):
        assert call(**{name: None}) == mx.MX_ERR_NULL, name
        assert call(**{name: BAD}) == mx.MX_ERR_ALIGN, name
    assert call(x=None, c=None, s=None, y=None, M=0) == mx.MX_OK
    assert call(x=None, c=None, s=None, y=None, N=0) == mx.MX_OK
    assert call(y=None, K=0) == mx.MX_ERR_NULL
    size = L.mx_gemv_workspace_size
    assert size(1, 1, 64, 64) == size(7, 1, 64, 64) == size(1, -1, 64, 64) == size(1, 1, 64, 1 << 26) == 0
    need = size(1, 40, 4096, 14336)
    assert need >= 2 * 40 * 4096 * 4
    long = {"M": 40, "N": 4096, "K": 14336, "ldx": 14336, "pitch": 448, "ldy": 4096}
    assert call(**long) == mx.MX_ERR_WORKSPACE
    assert call(**long, ws=GOOD, n=need - 1) == mx.MX_ERR_WORKSPACE
    assert call(**long, ws=BAD, n=need) == mx.MX_ERR_ALIGN


def test_gemv_grouped_validation(L):
    def call(x=GOOD, xt=1, ldx=64, xr=3, src=GOOD, top_k=2, c=GOOD, s=GOOD, pitch=2, offs=GOOD, groups=4,
             rows=6, N=5, K=64, y=GOOD, yt=0, ldy=5):
        return L.mx_gemv_grouped(x, xt, ldx, xr, src, top_k, c, s, pitch, offs, groups, rows, N, K, 1.0, y,
                                 yt, ldy, None)

    for bad in ({"K": 33}, {"ldx": 63}, {"pitch": 1}, {"ldy": 4}, {"rows": -1}, {"groups": 0},
                {"groups": mx.MX_MAX_GROUPS + 1}, {"top_k": 0}, {"xr": -1}, {"xr": BIG}, {"top_k": BIG}):
        assert call(**bad) == mx.MX_ERR_SHAPE, bad
    assert call(xt=9) == mx.MX_ERR_ENUM
    for name in ("x", "c", "s", "y", "offs"):
        assert call(**{name: None}) == mx.MX_ERR_NULL, name
        assert call(**{name: BAD}) == mx.MX_ERR_ALIGN, name
    assert call(src=BAD) == mx.MX_ERR_ALIGN
    assert call(rows=0, x=None, y=None, offs=None) == mx.MX_OK


def test_plan_validation(L):
    size = L.mx_moe_plan_workspace_size
    assert size(1, 1, 1) == 0 and size(0, 4, 8) == 0
    assert size(1 << 20, 4, 32) > 0
    assert size(-1, 1, 1) == size(1, 0, 1) == size(1, 1, 0) == size(1, 1, mx.MX_MAX_GROUPS + 1) == 0

    def call(ids=GOOD, it=1, T=4, k=2, E=8, offs=GOOD, src=GOOD, pos=GOOD, ws=None, n=0):
        return L.mx_moe_plan(ids, it, T, k, E, offs, src, pos, ws, n, None)

    for bad in ({"T": -1}, {"k": 0}, {"E": 0}, {"E": mx.MX_MAX_GROUPS + 1}, {"T": 1 << 30, "k": 2}):
        assert call(**bad) == mx.MX_ERR_SHAPE, bad
    assert call(it=2) == mx.MX_ERR_ENUM
    for name in ("ids", "offs", "src", "pos"):
        assert call(**{name: None}) == mx.MX_ERR_NULL, name
        assert call(**{name: BAD}) == mx.MX_ERR_ALIGN, name
    need = size(1 << 20, 4, 8)
    big = {"T": 1 << 20, "k": 4}
    assert call(**big) == mx.MX_ERR_WORKSPACE
    assert call(**big, ws=GOOD, n=need - 1) == mx.MX_ERR_WORKSPACE
    assert call(**big, ws=BAD, n=need) == mx.MX_ERR_ALIGN


def test_row_call_validation(L):
    def dispatch(x=GOOD, dt=1, ldx=40, pos=GOOD, w=GOOD, T=4, k=2, rows=8, cols=40, out=GOOD, ldo=40):
        return L.mx_moe_dispatch(x, dt, ldx, pos, w, T, k, rows, cols, out, ldo, None)

    def quantize(x=GOOD, dt=1, ldx=64, pos=GOOD, T=4, k=2, rows=8, cols=64, c=GOOD, s=GOOD, pitch=2):
        return L.mx_moe_dispatch_quantize(x, dt, ldx, pos, T, k, rows, cols, c, s, pitch, None)

    def combine(z=GOOD, zt=0, ldz=40, rows=8, pos=GOOD, w=GOOD, T=4, k=2, cols=40, y=GOOD, yt=1, ldy=40):
        return L.mx_moe_combine(z, zt, ldz, rows, pos, w, T, k, cols, y, yt, ldy, None)

    def bwd(dy=GOOD, dt=1, lddy=40, z=GOOD, zt=0, ldz=40, rows=8, pos=GOOD, w=GOOD, T=4, k=2, cols=40,
            dz=GOOD, lddz=40, dw=GOOD):
        return L.mx_moe_combine_bwd(dy, dt, lddy, z, zt, ldz, rows, pos, w, T, k, cols, dz, lddz, dw, None)

    shapes = ({"T": -1}, {"k": 0}, {"cols": -32}, {"rows": -1}, {"rows": BIG}, {"T": 1 << 30, "k": 2})
    for call, lds, ptrs, enums in ((dispatch, ("ldx", "ldo"), ("x", "pos", "out"), ("dt",)),
                                   (quantize, ("ldx", "pitch"), ("x", "pos", "c", "s"), ("dt",)),
                                   (combine, ("ldz", "ldy"), ("z", "pos", "y"), ("zt", "yt")),
                                   (bwd, ("lddy", "ldz", "lddz"), ("dy", "z", "pos", "dz", "dw"), ("dt", "zt"))):
        for bad in shapes:
            assert call(**bad) == mx.MX_ERR_SHAPE, (call, bad)
        for name in lds:
            assert call(**{name: 1}) == mx.MX_ERR_SHAPE, (call, name)
        for name in ptrs:
            assert call(**{name: None}) == mx.MX_ERR_NULL, (call, name)
            assert call(**{name: BAD}) == mx.MX_ERR_ALIGN, (call, name)
        for name in enums:
            assert call(**{name: 7}) == mx.MX_ERR_ENUM, (call, name)
        assert call(T=0) == mx.MX_OK, call
    assert quantize(cols=40) == mx.MX_ERR_SHAPE
    for call in (dispatch, combine, bwd):
        assert call(w=BAD) == mx.MX_ERR_ALIGN, call
    assert dispatch(rows=0, x=None) == dispatch(cols=0, ldx=0, ldo=0, x=None) == mx.MX_OK
    assert combine(rows=0, z=None, y=None) == mx.MX_ERR_NULL
    assert combine(cols=0, y=None) == mx.MX_OK
    assert bwd(rows=0, z=None, dz=None, dy=None, dw=None) == mx.MX_ERR_NULL


def test_conveniences_refuse_what_the_library_cannot_see():
    """CPU tensors, wrong types and shapes raise before the library is called."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x, w = torch.zeros(2, 64), (u8(5, 32), u8(5, 2))
    with pytest.raises(ValueError, match="columns"):
        mx.gemv(torch.zeros(2, 32), w)
    with pytest.raises(ValueError, match="uint8"):
        mx.gemv(x, (w[0].int(), w[1]))
    with pytest.raises(ValueError, match="same rows"):
        mx.gemv(x, (w[0], u8(4, 2)))
    with pytest.raises(ValueError, match="contiguous"):
        mx.gemv(x, (w[0], u8(2, 5).t()))
    with pytest.raises(ValueError, match="one packed weight"):
        mx.gemv(x, (u8(3, 5, 32), u8(3, 5, 2)))
    offs = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="offs must be int64"):
        mx.gemv_grouped(x, (w[0][None], w[1][None]), offs)
    with pytest.raises(ValueError, match="same rows"):
        mx.gemv_grouped(x, (u8(3, 5, 32), u8(3, 5, 2)), offs.long())
    with pytest.raises(ValueError, match="int32 or int64"):
        mx.moe_plan(torch.zeros(4, 2), 8)
    pos = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="pos is for 2 tokens"):
        mx.moe_dispatch(torch.zeros(3, 8), pos)
    with pytest.raises(ValueError, match="pos must be int32"):
        mx.moe_combine(x, pos.long())
    with pytest.raises(ValueError, match="weights must be float32"):
        mx.moe_combine(x, pos, torch.zeros(2, 2, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="same columns"):
        mx.moe_combine_bwd(x, torch.zeros(4, 32), pos)
    with pytest.raises(ValueError, match="packed uint8"):
        mx.moe_dispatch_quantize(x, pos, out=(u8(4, 32), u8(3, 2)))


RUNNER = """
import sys
from mxfp4_microscaling_quantization_amd import build, mx
mx.LIB_PATH = build.SAN_LIB
import pytest
sys.exit(pytest.main(["-q", "-p", "no:cacheprovider", "tests/test_moe_abi_cpu.py",
                      "-k", "validation"]))
"""


@pytest.mark.slow
def test_entry_points_under_address_and_undefined_behaviour_sanitizers():
    sanitized_library()
    env = dict(os.environ, PYTHONPATH=ROOT, LD_PRELOAD=str(build.sanitizer_runtime()),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-c", RUNNER], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=600)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-3000:]
    assert "4 passed" in res.stdout and "failed" not in res.stdout
