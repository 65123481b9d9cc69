"""GPU tests of the token-row operators where values, sizes or layouts are at
their limits.  Tolerances are fixed from the formats as in test_gpu_tokens.py;
what differs is stated at each test."""
import ctypes

import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding as sc
from test_gpu_tokens import U

pytestmark = pytest.mark.gpu


def _grads64(q, k, v, gout, scale):
    """Gradients of one sequence and one head in 64 bits, on the device."""
    q, k, v, g = (x[:, 0].double() for x in (q, k, v, gout))
    p = torch.softmax(q @ k.T * scale, 1)
    gv = p.T @ g
    ds = g @ v.T
    ds -= (g * (p @ v)).sum(1, keepdim=True)
    ds *= p
    return ds @ k * scale, ds.T @ q * scale, gv


def test_attention_gradient_of_a_list_that_one_block_walks():
    """The keys of gq's rows are not cut: one query on a million keys is 7,813 steps of one block, far past
    what any one wait may take if it covered them all."""
    n, d = 1_000_000, 32
    g = torch.Generator(device="cuda").manual_seed(9)
    q, gout = (torch.randn((1, 1, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((n, 1, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    off, koff = (torch.tensor([0, m], dtype=torch.int32).cuda() for m in (1, n))
    o, l = sc.sc_attn_fwd(q, k, v, off, k_off=koff, return_lse=True)
    gq, gk, gv = sc.sc_attn_bwd(gout, q, k, v, o, l, off, k_off=koff)
    sc.sc_attn_check()
    wq, wk, wv = _grads64(q, k, v, gout, d ** -0.5)
    for got, want in ((gk, wk), (gv, wv), (gq, wq)):
        assert float((got[:, 0].double() - want).norm() / want.norm()) <= 3 * U["bf16"]


# ---------------------------------------------------------------- refusals --
def test_weight_gradients_of_a_side_without_heads_are_looked_at():
    """They are written (with zeros), so a host address is refused although the side has no rows."""
    x = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    y, w = torch.zeros_like(x), torch.ones(64, device="cuda")
    gwk = torch.full((64,), 7.0, device="cuda")
    view = [ctypes.byref(sc._Heads(t.data_ptr(), 128, 64)) for t in (x, y)]
    host = (ctypes.c_float * 64)()

    def call(gwq):
        return sc.lib().sc_qk_norm_rope_bwd(None, view[0], None, view[0], None, view[1], gwq, gwk.data_ptr(),
                                            w.data_ptr(), w.data_ptr(), None, 0, 1, None, 4, 0, 2, 64, 0, 1e-6, 1.0, 1,
                                            0, torch.cuda.current_stream().cuda_stream)

    assert call(ctypes.addressof(host)) == 1
    assert b"weight gradients" in sc.lib().sc_last_error()
    gwq = torch.full((64,), 7.0, device="cuda")
    assert call(gwq.data_ptr()) == 0
    assert not gwq.any() and not gwk.any()


def test_views_past_the_address_space_are_refused():
    """Strides and counts that are legal each and together pass 64 bits: refused by the host, nothing runs."""
    x = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    y = torch.zeros_like(x)
    far = ctypes.byref(sc._Heads(x.data_ptr(), 1 << 36, 64))
    out = ctypes.byref(sc._Heads(y.data_ptr(), 128, 64))
    st = sc.lib().sc_qk_norm_rope_fwd(far, None, out, None, None, None, None, 0, 1, None, (1 << 31) - 1, 2, 0, 64, 0,
                                      1e-6, 1.0, 1, 0, None)
    assert st == 1 and b"address space" in sc.lib().sc_last_error()
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    near = ctypes.byref(sc._Heads(x.data_ptr(), 128, 64))
    st = sc.lib().sc_attn_fwd(near, far, near, out, None, off.data_ptr(), off.data_ptr(), None, 1, 4, 1 << 30, 2, 2, 64,
                              0.1, 1, 0, None)
    assert st == 1 and b"address space" in sc.lib().sc_last_error()
