"""A block that mixes voxels near and far, and its training step.

A submanifold convolution mixes neighbours; attention over each scene of the
packed batch then mixes voxels at any distance, its queries and keys normed per
head and rotated by the voxels' x, y, z.  The step runs forward and backward on
the library's kernels (the projections are torch matrix products), takes a
gradient step and prints the loss:

    python examples/voxel_attention.py [--scans 4] [--voxels 3000] [--steps 5]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from submanifold_sparse_convolution_hash_gb300 import binding as sc  # noqa: E402
from submanifold_sparse_convolution_hash_gb300 import scenes  # noqa: E402

HEADS_Q, HEADS_KV, HEAD_DIM, ROT = 4, 2, 32, 24  # 8 values of a head turn with each axis, 8 stay
HEADS = HEADS_Q + 2 * HEADS_KV


def packed_scans(scans: int, voxels: int, seed: int = 1, device="cuda"):
    """(coords int32 [N, 4] with each scan's rows together, offsets int32 [scans + 1], dims)."""
    s = scenes.batch_of_scans(seed, scans, voxels, (160, 160, 41))
    coords = s.coords[np.argsort(s.coords[:, 0], kind="stable")]
    off = np.concatenate([[0], np.cumsum(np.bincount(coords[:, 0], minlength=scans))])
    return (torch.from_numpy(np.ascontiguousarray(coords)).to(device),
            torch.from_numpy(off.astype(np.int32)).to(device), s.dims)


class Block:
    """Convolution, then attention with a residual; weights and their gradients in half precision."""

    def __init__(self, coords, offsets, dims, channels=32, seed=0):
        self.coords, self.off = coords, offsets
        self.kmap = sc.sc_kmap_build(sc.sc_hash_build(coords), 3, 3, dims)
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g) / fan ** 0.5).half().to(coords.device)

        self.conv = weight(27, channels, channels, fan=27 * channels / 4)
        self.qkv = weight(channels, HEADS * HEAD_DIM, fan=channels)
        self.proj = weight(HEADS_Q * HEAD_DIM, channels, fan=HEADS_Q * HEAD_DIM)
        self.wq = torch.ones(HEAD_DIM, device=coords.device)
        self.wk = torch.ones(HEAD_DIM, device=coords.device)
        self.freq, self.amp = sc.rope_frequencies(ROT, axes=3, base=100.0, device=coords.device)

    def rope(self):
        return dict(pos=self.coords[:, 1:], freq=self.freq, wq=self.wq, wk=self.wk, amp=self.amp)

    def forward(self, feats):
        x = sc.sc_subm_conv_fwd(self.kmap, feats, self.conv)
        rows = (x @ self.qkv).view(-1, HEADS, HEAD_DIM)  # q, k and v heads side by side
        q, k, v = rows.split([HEADS_Q, HEADS_KV, HEADS_KV], 1)
        qr, kr = sc.sc_qk_norm_rope_fwd(q, k, **self.rope())
        out, lse = sc.sc_attn_fwd(qr, kr, v, self.off, return_lse=True)
        self.saved = feats, x, q, k, v, qr, kr, out, lse
        return x + out.flatten(1) @ self.proj

    def backward(self, gy):
        """Gradients of (conv, qkv, proj, wq, wk)."""
        feats, x, q, k, v, qr, kr, out, lse = self.saved
        g_proj = out.flatten(1).t() @ gy
        gout = (gy @ self.proj.t()).view(-1, HEADS_Q, HEAD_DIM)
        grows = torch.empty((x.shape[0], HEADS, HEAD_DIM), dtype=x.dtype, device=x.device)
        gq, gk, gv = grows.split([HEADS_Q, HEADS_KV, HEADS_KV], 1)
        # written where the projection's gradient reads them
        sc.sc_attn_bwd(gout, qr, kr, v, out, lse, self.off, gq=gq, gk=gk, gv=gv)
        _, _, g_wq, g_wk = sc.sc_qk_norm_rope_bwd(gq, gk, q, k, gin_q=gq, gin_k=gk, **self.rope())
        g_qkv = x.t() @ grows.flatten(1)
        gx = gy + grows.flatten(1) @ self.qkv.t()
        g_conv = sc.sc_subm_conv_bwd_weight(self.kmap, feats, gx.contiguous())
        return g_conv, g_qkv, g_proj, g_wq, g_wk

    def params(self):
        return self.conv, self.qkv, self.proj, self.wq, self.wk


def train(scans=4, voxels=3000, steps=5, rate=0.5, seed=1):
    """The losses of `steps` gradient steps towards a smooth function of the coordinates."""
    coords, off, dims = packed_scans(scans, voxels, seed)
    n, channels = coords.shape[0], 32
    g = torch.Generator(device="cuda").manual_seed(seed)
    feats = torch.randn((n, channels), generator=g, device="cuda").half()
    mix = torch.randn((3, channels), generator=g, device="cuda") * 0.05
    target = torch.sin(coords[:, 1:].float() @ mix)
    block = Block(coords, off, dims, channels, seed)
    losses = []
    for _ in range(steps):
        y = block.forward(feats)
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        # the loss gradient times n stays in half precision's range
        grads = block.backward((diff * (2.0 / channels)).half())
        for w, gw in zip(block.params(), grads):
            w -= (gw.float() * (rate / n)).to(w.dtype)
    sc.sc_attn_check()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--scans", type=int, default=4)
    ap.add_argument("--voxels", type=int, default=3000)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.scans, a.voxels, a.steps)):
        print(f"step {i}: loss {loss:.5f}")
