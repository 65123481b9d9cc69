"""The example's transformer block (convolution, norms, linear layers, attention, clipping) run
together as it is used: gradients against torch autograd in 64 bits, a whole step captured and
replayed, the 8-bit forward pass, and the example itself."""
import math
import os
import sys

import pytest
import torch

from conftest import ROOT
from submanifold_sparse_convolution_hash_gb300 import binding as sc

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu

H = 2.0 ** -11  # a rounding to half precision


def small(seed, scans=3, voxels=300):
    import voxel_transformer as vt
    coords, off, dims = vt.packed_scans(scans, voxels, seed=seed)
    block = vt.Transformer(coords, off, dims, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    feats, gy = (torch.randn((coords.shape[0], 32), generator=g).half().cuda() for _ in range(2))
    return vt, block, feats, gy


def reference(vt, block, h0, gy):
    """y and the gradients of every parameter behind the convolution, in 64 bits."""
    names = vt.NAMES[1:]
    p = {n: getattr(block, n).double().cpu().requires_grad_(True) for n in names}
    h0 = h0.double().cpu()

    def norm(x, w):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w

    rows = (norm(h0, p["n1"]) @ p["qkv"]).view(-1, vt.HEADS, vt.HEAD_DIM)
    q, k, v = rows.split([vt.HEADS_Q, vt.HEADS_KV, vt.HEADS_KV], 1)
    per = vt.ROT // 6
    pos = block.coords[:, 1:].cpu().double()
    phi = torch.cat([pos[:, a:a + 1] * block.freq[a * per:(a + 1) * per].cpu().double() for a in range(3)], 1)[:, None]

    def turn(z, w):
        a, b, rest = norm(z, w).split([vt.ROT // 2, vt.ROT // 2, vt.HEAD_DIM - vt.ROT], -1)
        return torch.cat([a * phi.cos() - b * phi.sin(), b * phi.cos() + a * phi.sin(), rest], -1)

    q, k = turn(q, p["wq"]), turn(k, p["wk"])
    off, out = block.off.tolist(), []
    for a, b in zip(off[:-1], off[1:]):
        heads = []
        for h in range(vt.HEADS_Q):
            j = h // (vt.HEADS_Q // vt.HEADS_KV)
            w = torch.softmax(q[a:b, h] @ k[a:b, j].T * vt.HEAD_DIM ** -0.5, -1)
            heads.append(w @ v[a:b, j])
        out.append(torch.stack(heads, 1))
    h1 = h0 + torch.cat(out).flatten(1) @ p["proj"]
    z = norm(h1, p["n2"]) @ p["up"] + p["b_up"]
    y = h1 + (z * torch.special.ndtr(z)) @ p["down"] + p["b_down"]
    y.backward(gy.double().cpu())
    return y.detach(), {n: p[n].grad for n in names}


def test_gradients_match_autograd():
    vt, block, feats, gy = small(5)
    y = block.forward(feats)
    grads = dict(zip(vt.NAMES, block.backward(gy)))
    sc.sc_attn_check()
    sc.sc_rows_check()
    ref, want = reference(vt, block, block.saved[1], gy)
    # about twelve roundings to half precision lie between inputs and results, each entering with a
    # factor near one; gradients pass them forward and back
    assert float((y.double().cpu() - ref).norm() / ref.norm()) <= 12 * H
    for n, w in want.items():
        assert float((grads[n].double().cpu() - w).norm() / w.norm()) <= 30 * H, n
    assert torch.isfinite(grads["conv"]).all()


def test_clipped_gradients_of_the_block():
    vt, block, feats, gy = small(6)
    block.forward(feats)
    grads = block.backward(gy)
    kept = [t.clone() for t in grads]
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in kept))
    got = sc.sc_grad_clip(grads, norm / 3)
    assert abs(float(got) - norm) <= 1e-6 * norm
    for t, k in zip(grads, kept):
        u = H if t.dtype is torch.float16 else 2.0 ** -24
        assert bool(((t.double() - k.double() / 3).abs() <= (u + 2.0 ** -20) * k.double().abs() / 3 + 2.0 ** -25).all())


def test_a_captured_step_gives_the_same_bits():
    _, block, feats, gy = small(7)
    y = block.forward(feats)
    grads = block.backward(gy)
    norm = sc.sc_grad_clip(grads, 1.0)
    want = [y.clone(), norm.clone()] + [t.clone() for t in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = block.forward(feats)
        grads2 = block.backward(gy)
        norm2 = sc.sc_grad_clip(grads2, 1.0)
    held = [y2, norm2] + list(grads2)
    # the convolution's weight gradient adds with atomics: its order is not fixed, and the norm has it in it
    loose = {1, 2}
    for _ in range(2):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(held, want)):
            if i in loose:
                assert float((a.double() - b.double()).norm()) <= 2 * H * float(b.double().norm())
            else:  # scaled by a norm that may differ in its last bits
                assert float((a.double() - b.double()).norm()) <= H * float(b.double().norm())
    assert torch.equal(y2, want[0])


def test_8_bit_forward():
    _, block, feats, _ = small(8)
    block.quantise()
    y, y8 = block.forward(feats).double(), block.forward_e4m3(feats).double()
    sc.sc_rows_check()
    # four products, each of two operands off by at most 2^-4 of themselves: no more than
    # half of what the branches add, were all errors of one sign
    assert float((y8 - y).norm() / y.norm()) <= 0.5


def test_the_example_runs():
    import voxel_transformer as vt
    said, off8 = vt.train(scans=2, voxels=400, steps=3)
    assert len(said) == 3 and all(math.isfinite(a) and math.isfinite(b) and b > 0 for a, b in said)
    assert 0 < off8 < 0.5
