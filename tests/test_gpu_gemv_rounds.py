"""GPU checks of the few-row products where the contraction is empty, against the definition."""
import numpy as np
import pytest
import torch

from mxfp4_microscaling_quantization_amd import mx
from tests.gpu_util import DEV, host

pytestmark = pytest.mark.gpu


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
