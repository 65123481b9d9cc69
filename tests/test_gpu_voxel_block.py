"""The example block's first layer: the convolution's weight gradient that comes
out of the whole block's backward pass, against the formula in 64 bits."""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


def test_convolution_weight_gradient_through_the_block():
    import voxel_attention as va
    from test_gpu_voxel_attention import reference
    coords, off, dims = va.packed_scans(2, 300, seed=8)
    block = va.Block(coords, off, dims, seed=4)
    g = torch.Generator().manual_seed(7)
    n = coords.shape[0]
    feats = torch.randn((n, 32), generator=g).half().cuda()
    gy = torch.randn((n, 32), generator=g).half().cuda()
    block.forward(feats)
    g_conv = block.backward(gy)[0]
    # the gradient of the convolution's output, by autograd through the rest of the block
    x = block.saved[1].double().cpu().requires_grad_(True)
    reference(block, x, gy)
    gx = x.grad
    # dW[k, ci, co] = sum over the pairs (i, j) whose coordinates differ by offset k of f_j,ci gx_i,co
    c = coords.cpu()
    at = {tuple(r): i for i, r in enumerate(c.tolist())}
    offsets = [(a, b, e) for a in (-1, 0, 1) for b in (-1, 0, 1) for e in (-1, 0, 1)]
    f = feats.double().cpu()
    want = torch.zeros((27, 32, 32), dtype=torch.float64)
    for k, (a, b, e) in enumerate(offsets):
        pairs = [(i, at[s, p + a, q + b, r + e]) for i, (s, p, q, r) in enumerate(c.tolist())
                 if (s, p + a, q + b, r + e) in at]
        if pairs:
            i, j = torch.tensor(pairs).T
            want[k] = f[j].T @ gx[i]
    # gx lies about ten roundings to half precision behind gy, and the sums' result one more
    err = float((g_conv.double().cpu() - want).norm() / want.norm())
    assert err <= 20 * 2.0 ** -11, err
