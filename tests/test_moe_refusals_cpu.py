"""CPU checks of what the routing and few-row conveniences refuse before the library is called:
workspaces that are not one run of memory."""
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
