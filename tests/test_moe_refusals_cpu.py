"""CPU checks of what the routing and few-row conveniences refuse before the library is called:
workspaces that are not one run of memory, streams of another device,
a number of rows that is not out's."""
from types import SimpleNamespace

import pytest
import torch

from mxfp4_microscaling_quantization_amd import mx


def packed(*shape):
    """Packed weights [..., N, K] of zeros."""
    *rows, K = shape
    return (torch.zeros((*rows, K // 2), dtype=torch.uint8), torch.zeros((*rows, K // 32), dtype=torch.uint8))


@pytest.mark.parametrize("workspace", [
    torch.zeros(1, dtype=torch.uint8).expand(1 << 20),       # a byte seen as a million
    torch.zeros((64, 4096), dtype=torch.uint8)[:, :2048],    # other data between its rows
    torch.zeros(1 << 16, dtype=torch.int32)[::2]])
def test_workspaces_that_are_not_contiguous_are_refused(workspace):
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        mx.gemv(torch.zeros(40, 14336), packed(64, 14336), workspace=workspace)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        mx.moe_plan(torch.zeros((4096, 4), dtype=torch.int64), 8, workspace=workspace)


def calls(stream):
    """Every convenience that takes a stream, on tensors of the device that torch names -1."""
    x, pos, ids = torch.zeros(2, 64), torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int64)
    offs, src = torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)
    z = torch.zeros(4, 64)
    return {"gemv": lambda: mx.gemv(x, packed(5, 64), out=torch.zeros(2, 5), stream=stream),
            "gemv_grouped": lambda: mx.gemv_grouped(x, packed(3, 5, 64), offs, src, 2, out=torch.zeros(4, 5), stream=stream),
            "moe_plan": lambda: mx.moe_plan(ids, 3, stream=stream),
            "moe_dispatch": lambda: mx.moe_dispatch(x, pos, out=z, stream=stream),
            "moe_dispatch_quantize": lambda: mx.moe_dispatch_quantize(x, pos, out=packed(4, 64), stream=stream),
            "moe_combine": lambda: mx.moe_combine(z, pos, out=torch.zeros(2, 64), stream=stream),
            "moe_combine_bwd": lambda: mx.moe_combine_bwd(x, z, pos, out=torch.zeros(4, 64), stream=stream)}


@pytest.mark.parametrize("name", list(calls(None)))
def test_streams_of_another_device_are_refused(name, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    other = SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0x1000)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        calls(other)[name]()


def test_rows_that_are_not_out_s_are_refused():
    x, pos = torch.zeros(2, 64), torch.zeros((2, 2), dtype=torch.int32)
    for rows in (2, 8):
        with pytest.raises(ValueError, match=f"out has 4 rows, not {rows}"):
            mx.moe_dispatch(x, pos, rows=rows, out=torch.zeros(4, 64))
        with pytest.raises(ValueError, match=f"out has 4 rows, not {rows}"):
            mx.moe_dispatch_quantize(x, pos, rows=rows, out=packed(4, 64))
