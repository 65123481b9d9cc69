"""The example block (convolution, per-head norm and rotation, attention over
packed scenes) end to end: its gradients against torch autograd in 64 bits, and
its loss."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from submanifold_sparse_convolution_hash_gb300 import binding as sc

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


def reference(block, x, gy):
    """y and the gradients of (x, qkv, proj, wq, wk) from the convolution's output on, in 64 bits."""
    import voxel_attention as va
    x, qkv, proj, wq, wk = (t.double().cpu().requires_grad_(True)
                            for t in (x, block.qkv, block.proj, block.wq, block.wk))
    rows = (x @ qkv).view(-1, va.HEADS, va.HEAD_DIM)
    q, k, v = rows.split([va.HEADS_Q, va.HEADS_KV, va.HEADS_KV], 1)
    per = va.ROT // 6
    pos = block.coords[:, 1:].cpu().double()
    phi = torch.cat([pos[:, a:a + 1] * block.freq[a * per:(a + 1) * per].cpu().double() for a in range(3)], 1)[:, None]

    def turn(z, w):
        z = z / torch.sqrt(z.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b, rest = z.split([va.ROT // 2, va.ROT // 2, va.HEAD_DIM - va.ROT], -1)
        return torch.cat([a * phi.cos() - b * phi.sin(), b * phi.cos() + a * phi.sin(), rest], -1)

    q, k = turn(q, wq), turn(k, wk)
    off = block.off.tolist()
    out = []
    for a, b in zip(off[:-1], off[1:]):
        heads = []
        for h in range(va.HEADS_Q):
            j = h // (va.HEADS_Q // va.HEADS_KV)
            p = torch.softmax(q[a:b, h] @ k[a:b, j].T * va.HEAD_DIM ** -0.5, -1)
            heads.append(p @ v[a:b, j])
        out.append(torch.stack(heads, 1))
    y = x + torch.cat(out).flatten(1) @ proj
    y.backward(gy.double().cpu())
    return y.detach(), [t.grad for t in (qkv, proj, wq, wk)]


def test_gradients_match_autograd():
    import voxel_attention as va
    coords, off, dims = va.packed_scans(3, 400, seed=5)
    block = va.Block(coords, off, dims, seed=2)
    g = torch.Generator().manual_seed(3)
    feats = torch.randn((coords.shape[0], 32), generator=g).half().cuda()
    gy = torch.randn((coords.shape[0], 32), generator=g).half().cuda()
    y = block.forward(feats)
    g_conv, *grads = block.backward(gy)
    sc.sc_attn_check()
    ref, want = reference(block, block.saved[1], gy)
    # about ten roundings to half precision (2^-11 each) lie between inputs and results
    assert float((y.double().cpu() - ref).norm() / ref.norm()) <= 10 * 2.0 ** -11
    for got, w in zip(grads, want):
        assert float((got.double().cpu() - w).norm() / w.norm()) <= 20 * 2.0 ** -11
    assert torch.isfinite(g_conv).all()


def test_loss_falls():
    import voxel_attention as va
    losses = va.train(scans=2, voxels=500, steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
