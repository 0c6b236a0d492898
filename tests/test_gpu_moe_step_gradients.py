"""The expert layer's way back as a training step runs it: the routed gradient through the grouped
backward and the dispatch's gradient, every part against the float64 oracle on the operands that
the step itself made."""
import numpy as np
import pytest
import torch

import oracle as O
from mxfp4_microscaling_quantization_amd import mx
from tests.gpu_util import DEV, host
from tests.test_gpu_grouped_bwd import check_grouped_bwd
from tests.test_gpu_moe_layer import E, F, H, T, TOP_K, batch, packed_experts

pytestmark = pytest.mark.gpu


def test_gradients_of_the_experts_weights_and_inputs():
    x, ids, p = batch(1)
    (wc, ws), _ = packed_experts(2, F, H)
    wq = wc.reshape(E * F, -1), ws.reshape(E * F, -1)
    offs, src, pos = mx.moe_plan(ids, E)
    ends = offs.tolist()
    R = ends[-1]
    xq = tuple(a[:R].contiguous() for a in mx.moe_dispatch_quantize(x, pos))
    g = torch.Generator(device=DEV).manual_seed(3)
    dy = (torch.randn((T, F), generator=g, device=DEV) * 1e-2).to(torch.bfloat16)
    z = torch.randn((pos.numel(), F), generator=g, device=DEV)
    dz, _ = mx.moe_combine_bwd(dy, z, pos, p)
    dz = dz[:R].contiguous()

    # the rows' and the weights' gradients, within the products' bound of the oracle's
    check_grouped_bwd(host(dz), "bf16", tuple(map(host, xq)), tuple(map(host, wq)), ends, F, H, seed=7)

    # the tokens' gradients: top_k float32 additions of rows of the first
    dxr, _ = mx.grouped_linear_bwd(dz, xq, wq, ends, F, H, 7)
    dx = host(mx.moe_combine(dxr, pos))
    want, mag = O.moe_combine(host(dxr), host(pos), None)
    assert np.all(np.abs(dx - want) <= (TOP_K + 1) * 2.0 ** -24 * mag + 2.0 ** -140)
