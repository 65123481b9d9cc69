"""The example block's 8-bit forward pass, step by step: its matrices, each quantising norm and each
product against 64 bits on the step's own inputs, and what feeds what.  Tolerances as in test_gpu_rows.py."""
import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding as sc
from test_gpu_rows import E, linear_check, within
from test_gpu_voxel_transformer import small

pytestmark = pytest.mark.gpu


def quantised(q, s, y, what):
    ref = y.abs().amax(-1) / 448
    within(s, ref, 128 * E * ref, what)
    bound = (2.0 ** -4 + 512 * E) * y.abs() + 2.0 ** -10 * 1.001 * ref[:, None]
    within(q.double() * s.double()[:, None], y, bound, what)


def test_every_step_of_the_8_bit_forward(monkeypatch):
    vt, block, feats, _ = small(9)
    block.quantise()
    for n in vt.MATRICES:
        quantised(*block.e4m3[n], getattr(block, n).double().t(), n)
    norms, products = [], []
    norm, product = sc.sc_add_norm_fwd, sc.sc_linear_fwd

    def kept_norm(x, w=None, res=None, **kw):
        got = norm(x, w, res=res, **kw)
        norms.append((x, w, res, kw, got))
        return got

    def kept_product(x, W, **kw):
        got = product(x, W, **kw)
        products.append((x, W, kw, got))
        return got

    monkeypatch.setattr(sc, "sc_add_norm_fwd", kept_norm)
    monkeypatch.setattr(sc, "sc_linear_fwd", kept_product)
    y8 = block.forward_e4m3(feats)
    sc.sc_rows_check()
    sc.sc_attn_check()
    assert len(norms) == 4 and len(products) == 4
    for (x, w, res, kw, got), weights in zip(norms, (block.n1, None, block.n2, None)):
        assert kw == {"e4m3": True} and w is weights
        h = x.double() if res is None else x.double() + res.double()
        y = h if w is None else h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        quantised(got[0], got[1], y, "norm")
    for (x, W, kw, got), n, fed in zip(products, vt.MATRICES, norms):
        q, s = block.e4m3[n]
        assert W is q and kw["scale_w"] is s and x is fed[4][0] and kw["scale_x"] is fed[4][1]
        xd, wd = x.double() * kw["scale_x"].double()[:, None], (W.double() * s.double()[:, None]).t()
        linear_check(got, None, xd, wd, kw.get("bias"), kw.get("res"), kw.get("act", "none"), "f16", x.shape[1] + 64)
    # the residual stream, and the biases and the activation where they belong
    h0, h1 = norms[0][0], norms[2][4][2]
    assert norms[2][0] is products[1][3] and norms[2][2] is h0 and norms[3][0] is products[2][3]
    assert products[2][2]["bias"] is block.b_up and products[2][2]["act"] == "gelu"
    assert products[3][2]["bias"] is block.b_down and products[3][2]["res"] is h1 and y8 is products[3][3]
    assert torch.equal(h0, sc.sc_subm_conv_fwd(block.kmap, feats, block.conv))
