"""A transformer block on the voxels of packed scans, its training step and its 8-bit inference.

A submanifold convolution mixes neighbours; attention over each scan and a two-layer MLP follow,
each behind a norm, with the residual's addition folded into the next norm or product.  Every step
runs on the library's kernels, forward and backward; the gradients are clipped to a norm together
before the step:

    python examples/voxel_transformer.py [--scans 4] [--voxels 3000] [--steps 5]

It prints each step's loss and gradient norm, and how far the 8-bit forward pass is from the
16-bit one.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from submanifold_sparse_convolution_hash_gb300 import binding as sc  # noqa: E402
from voxel_attention import HEAD_DIM, HEADS, HEADS_KV, HEADS_Q, ROT, packed_scans  # noqa: E402

MATRICES = ("qkv", "proj", "up", "down")
NAMES = ("conv", "n1", "qkv", "wq", "wk", "proj", "n2", "up", "b_up", "down", "b_down")


class Transformer:
    """Convolution, then attention and MLP with their norms; matrices in half precision, the rest in float32."""

    def __init__(self, coords, offsets, dims, channels=32, hidden=128, seed=0):
        self.coords, self.off = coords, offsets
        self.kmap = sc.sc_kmap_build(sc.sc_hash_build(coords), 3, 3, dims)
        g = torch.Generator().manual_seed(seed)
        dev = coords.device

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g) / fan ** 0.5).half().to(dev)

        def vector(n, at):
            return (at + 0.1 * torch.randn(n, generator=g)).to(dev)

        self.conv = weight(27, channels, channels, fan=27 * channels / 4)
        self.n1, self.n2 = vector(channels, 1.0), vector(channels, 1.0)
        self.qkv = weight(channels, HEADS * HEAD_DIM, fan=channels)
        self.wq, self.wk = vector(HEAD_DIM, 1.0), vector(HEAD_DIM, 1.0)
        self.proj = weight(HEADS_Q * HEAD_DIM, channels, fan=HEADS_Q * HEAD_DIM)
        self.up, self.b_up = weight(channels, hidden, fan=channels), vector(hidden, 0.0)
        self.down, self.b_down = weight(hidden, channels, fan=hidden), vector(channels, 0.0)
        self.freq, self.amp = sc.rope_frequencies(ROT, axes=3, base=100.0, device=dev)

    def params(self):
        return [getattr(self, n) for n in NAMES]

    def rope(self):
        return dict(pos=self.coords[:, 1:], freq=self.freq, wq=self.wq, wk=self.wk, amp=self.amp)

    def attend(self, rows):
        q, k, v = rows.view(-1, HEADS, HEAD_DIM).split([HEADS_Q, HEADS_KV, HEADS_KV], 1)
        qr, kr = sc.sc_qk_norm_rope_fwd(q, k, **self.rope())
        out, lse = sc.sc_attn_fwd(qr, kr, v, self.off, return_lse=True)
        return out, (q, k, v, qr, kr, out, lse)

    def forward(self, feats):
        h0 = sc.sc_subm_conv_fwd(self.kmap, feats, self.conv)
        y1 = sc.sc_add_norm_fwd(h0, self.n1)
        out, heads = self.attend(sc.sc_linear_fwd(y1, self.qkv))
        a = sc.sc_linear_fwd(out.flatten(1), self.proj)
        y2, h1 = sc.sc_add_norm_fwd(a, self.n2, res=h0)
        z, pre = sc.sc_linear_fwd(y2, self.up, bias=self.b_up, act="gelu", return_pre=True)
        self.saved = feats, h0, y1, heads, y2, h1, z, pre
        return sc.sc_linear_fwd(z, self.down, bias=self.b_down, res=h1)

    def backward(self, gy):
        """The gradients of params(), in their order."""
        feats, h0, y1, (q, k, v, qr, kr, out, lse), y2, h1, z, pre = self.saved
        gz, g_down, g_b_down = sc.sc_linear_bwd(gy, z, self.down, bias=True)
        gy2, g_up, g_b_up = sc.sc_linear_bwd(gz, y2, self.up, pre=pre, act="gelu", bias=True)
        gh1, g_n2 = sc.sc_add_norm_bwd(gy2, h1, self.n2, gsum=gy)
        gout, g_proj, _ = sc.sc_linear_bwd(gh1, out.flatten(1), self.proj)
        grows = torch.empty((h0.shape[0], HEADS, HEAD_DIM), dtype=h0.dtype, device=h0.device)
        gq, gk, gv = grows.split([HEADS_Q, HEADS_KV, HEADS_KV], 1)
        sc.sc_attn_bwd(gout.view(-1, HEADS_Q, HEAD_DIM), qr, kr, v, out, lse, self.off, gq=gq, gk=gk, gv=gv)
        _, _, g_wq, g_wk = sc.sc_qk_norm_rope_bwd(gq, gk, q, k, gin_q=gq, gin_k=gk, **self.rope())
        gy1, g_qkv, _ = sc.sc_linear_bwd(grows.flatten(1), y1, self.qkv)
        gh0, g_n1 = sc.sc_add_norm_bwd(gy1, h0, self.n1, gsum=gh1)
        g_conv = sc.sc_subm_conv_bwd_weight(self.kmap, feats, gh0)
        return [g_conv, g_n1, g_qkv, g_wq, g_wk, g_proj, g_n2, g_up, g_b_up, g_down, g_b_down]

    def quantise(self):
        """The matrices in 8 bits, [out, in], with a scale for each output: once, before inference."""
        self.e4m3 = {n: sc.sc_add_norm_fwd(getattr(self, n).t().contiguous(), e4m3=True) for n in MATRICES}

    def forward_e4m3(self, feats):
        """forward with 8-bit products: the rows are quantised where they are normed, or as they are."""
        def product(name, rows, scale, **kw):
            w, sw = self.e4m3[name]
            return sc.sc_linear_fwd(rows, w, scale_x=scale, scale_w=sw, dtype=torch.float16, **kw)

        h0 = sc.sc_subm_conv_fwd(self.kmap, feats, self.conv)
        out, _ = self.attend(product("qkv", *sc.sc_add_norm_fwd(h0, self.n1, e4m3=True)))
        a = product("proj", *sc.sc_add_norm_fwd(out.flatten(1), e4m3=True))
        y2, s2, h1 = sc.sc_add_norm_fwd(a, self.n2, res=h0, e4m3=True)
        z = product("up", y2, s2, bias=self.b_up, act="gelu")
        return product("down", *sc.sc_add_norm_fwd(z, e4m3=True), bias=self.b_down, res=h1)


def train(scans=4, voxels=3000, steps=5, rate=0.05, max_norm=1.0, seed=1):
    """[(loss, gradient norm)] of `steps` clipped gradient steps, and the 8-bit forward pass's relative distance."""
    coords, off, dims = packed_scans(scans, voxels, seed)
    n, channels = coords.shape[0], 32
    g = torch.Generator(device="cuda").manual_seed(seed)
    feats = torch.randn((n, channels), generator=g, device="cuda").half()
    mix = torch.randn((3, channels), generator=g, device="cuda") * 0.05
    target = torch.sin(coords[:, 1:].float() @ mix)
    block = Transformer(coords, off, dims, channels, seed=seed)
    said = []
    for _ in range(steps):
        diff = block.forward(feats).float() - target
        # the loss gradient times n stays in half precision's range; the norm is that of the sums
        grads = block.backward((diff * (2.0 / channels)).half())
        norm = sc.sc_grad_clip(grads, max_norm * n)
        for w, gw in zip(block.params(), grads):
            w -= (gw.float() * (rate / n)).to(w.dtype)
        said.append((float(diff.square().mean()), float(norm) / n))
    block.quantise()
    y, y8 = block.forward(feats).float(), block.forward_e4m3(feats).float()
    sc.sc_attn_check()
    sc.sc_rows_check()
    return said, float((y8 - y).norm() / y.norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--scans", type=int, default=4)
    ap.add_argument("--voxels", type=int, default=3000)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    said, off8 = train(a.scans, a.voxels, a.steps)
    for i, (loss, norm) in enumerate(said):
        print(f"step {i}: loss {loss:.5f}, gradient norm {norm:.4f}")
    print(f"8-bit forward: {off8:.4f} off")
