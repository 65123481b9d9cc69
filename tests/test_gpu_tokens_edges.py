"""GPU tests of the token-row operators where values, sizes or layouts are at
their limits.  Tolerances are fixed from the formats as in test_gpu_tokens.py;
what differs is stated at each test."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding as sc
from test_gpu_tokens import DT, U, attn_inputs, attn_ref, close

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


def same(a, b):
    """Equal bits, where NaN equals NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a.float(), nan=7.0),
                                                                       torch.nan_to_num(b.float(), nan=7.0))


# ---------------------------------------------------------------- rotation --
# Pairings: (2i, 2i + 1); halves on the eight-value grid, of an even, of an odd number of pairs; no rotation.
PARTS = [(64, 32, True), (96, 50, True), (64, 48, False), (64, 44, False), (64, 42, False), (64, 0, True),
         (64, 0, False), (128, 64, False)]


def _part(d, rot, dtype):
    g = torch.Generator().manual_seed(d + rot)
    clean = torch.randn((6, 2, d), generator=g).to(DT[dtype])
    x = clean.clone()
    x[1, 0, rot] = math.inf
    x[2, 1, rot + 1] = math.nan
    x[3, 0, d - 1] = -math.inf
    x[4, 1, d - 2] = math.nan
    kw = {}
    if rot:
        f, _ = sc.rope_frequencies(rot, device="cuda")
        kw = dict(pos=torch.arange(6, dtype=torch.int32).cuda() * 1000 - 2500, freq=f, amp=1.25)
    return clean.cuda(), x.cuda(), kw


@pytest.mark.parametrize("d,rot,ilv", PARTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rope_values_that_do_not_turn_stay_themselves(d, rot, ilv, dtype):
    """Without a norm they come out as they went in, whatever they and their neighbours are, and the
    turned ones do not see them; the gradient, being a rotation back, likewise."""
    clean, x, kw = _part(d, rot, dtype)
    kw["interleaved"] = ilv
    for call in (lambda a: sc.sc_qk_norm_rope_fwd(a, None, **kw)[0],
                 lambda a: sc.sc_qk_norm_rope_bwd(a, None, **kw)[0]):
        y, want = call(x), call(clean)
        assert same(y[..., rot:], x[..., rot:])
        assert same(y[..., :rot], want[..., :rot])


@pytest.mark.parametrize("d,rot,ilv", PARTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rope_norm_beside_values_that_do_not_turn(d, rot, ilv, dtype):
    """With the norm an infinite value makes its row's 1/sqrt(mean) 0: it becomes NaN and the others 0.  In the
    gradient an infinite or NaN gout reaches its row, and the weight's gradient at its own place alone."""
    clean, x, kw = _part(d, rot, dtype)
    kw["interleaved"] = ilv
    w = torch.linspace(0.5, 1.5, d).cuda()
    y, _ = sc.sc_qk_norm_rope_fwd(x, None, wq=w, **kw)
    want = torch.zeros((d,), dtype=torch.bool)
    want[rot] = True
    assert torch.equal(torch.isnan(y[1, 0]).cpu(), want) and not y[1, 0].cpu()[~want].any()
    want = torch.zeros((d,), dtype=torch.bool)
    want[d - 1] = True
    assert torch.equal(torch.isnan(y[3, 0]).cpu(), want) and not y[3, 0].cpu()[~want].any()
    assert torch.isnan(y[2, 1]).all() and torch.isnan(y[4, 1]).all()
    _, _, gw, _ = sc.sc_qk_norm_rope_bwd(x, None, clean, None, wq=w, **kw)
    want = torch.zeros((d,), dtype=torch.bool)
    want[[rot, rot + 1, d - 1, d - 2]] = True
    assert torch.equal(~torch.isfinite(gw).cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("ilv", [False, True])
def test_rope_any_position(dtype, ilv):
    """Positions to the ends of int32, frequencies above and below half a turn a position.  The reference's
    angles: the position in two parts whose products with a frequency are exact in 64 bits, and the sum's
    formula.  The bound is that of the rotation at small positions."""
    pos = [0, 1, -1, 40000, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, -2 ** 24, -2 ** 24 - 1, 2 ** 31 - 1, -2 ** 31, 123456789,
           -987654321, 2 ** 30 + 4095, -2 ** 30 - 1, 1999999999]
    f = torch.cat([sc.rope_frequencies(48)[0], torch.tensor([3.0, -2.5, 7.0, 100.25, 6.2831855, 1e-9, 5000.0, 0.0])])
    p = torch.tensor(pos, dtype=torch.int64)
    hi = p // 65536 * 65536
    a, b = hi.double()[:, None] * f.double(), (p - hi).double()[:, None] * f.double()
    c = (a.cos() * b.cos() - a.sin() * b.sin())[:, None]
    s = (a.sin() * b.cos() + a.cos() * b.sin())[:, None]
    x = torch.randn((len(pos), 2, 64), generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    y, _ = sc.sc_qk_norm_rope_fwd(x.cuda(), None, p.int().cuda(), f.cuda(), interleaved=ilv)
    z = x.double()
    want = torch.empty_like(z)
    ia, ib = (slice(0, 64, 2), slice(1, 64, 2)) if ilv else (slice(0, 32), slice(32, 64))
    want[..., ia] = z[..., ia] * c - z[..., ib] * s
    want[..., ib] = z[..., ib] * c + z[..., ia] * s
    big = want.abs().amax(-1, keepdim=True)
    err = (y.double().cpu() - want).abs()
    bound = U[dtype] * want.abs() + 64 * 2.0 ** -24 * big + 2.0 ** -25 * (dtype == "f16")
    assert bool((err <= bound).all()), float((err / bound).max())


def test_rope_a_frequency_that_is_not_finite_spoils_its_own_pair():
    f, _ = sc.rope_frequencies(64)
    x = torch.randn((5, 2, 64), generator=torch.Generator().manual_seed(1)).half().cuda()
    pos = torch.arange(5, dtype=torch.int32).cuda()
    want, _ = sc.sc_qk_norm_rope_fwd(x, None, pos, f.cuda())
    f[3], f[20] = math.nan, math.inf
    y, _ = sc.sc_qk_norm_rope_fwd(x, None, pos, f.cuda())
    bad = [3, 35, 20, 52]
    keep = [i for i in range(64) if i not in bad]
    assert torch.isnan(y[1:, :, bad]).all() and torch.equal(y[..., keep], want[..., keep])


# --------------------------------------------------------------- attention --
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[50, 130, 64], [1, 3, 40], [300, 200, 290]])
def test_attention_huge_values_stay_in_their_sequence(lens, dtype):
    """Finite values of the largest sizes in one sequence change no bit of the others."""
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lens, None, 4, 2, 64, dtype, sharp=0.05)
    a, b = lens[0], lens[0] + lens[1]
    qh, kvh, gh = q.clone(), kvd.clone(), gout.clone()
    for x in (qh, kvh, gh):
        x[a:b] = torch.sign(x[a:b].float()).to(x.dtype) * 60000.0
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[a:b] = False
    got = []
    for qq, kv, gg in ((q, kvd, gout), (qh, kvh, gh)):
        o, l = sc.sc_attn_fwd(qq.cuda(), kv[:, :2], kv[:, 2:4], qo.cuda(), scale=60.0, return_lse=True)
        got.append((o, l) + sc.sc_attn_bwd(gg.cuda(), qq.cuda(), kv[:, :2], kv[:, 2:4], o, l, qo.cuda(), scale=60.0))
    for x, y in zip(*got):
        assert torch.equal(x.cpu()[keep], y.cpu()[keep])


@pytest.mark.parametrize("g", [3, 7])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_bits_do_not_depend_on_what_ran_before(g, d):
    """Three (seven) heads a key head leave rows of a tile that no copy writes; what an earlier call left
    there changes no bit."""
    lq = [200, 30]
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lq, None, 2 * g, 2, d, "f16", sharp=0.05)
    qo = qo.cuda()
    got = []
    for fill in (0.0, 60000.0):
        before = torch.full((4096, 4, d), fill, dtype=torch.float16, device="cuda")
        small = torch.full_like(before, 1.0 if fill else 0.0)
        off = torch.arange(33, dtype=torch.int32, device="cuda") * 128
        sc.sc_attn_fwd(before, small, small, off, scale=60.0)
        o, l = sc.sc_attn_fwd(q.cuda(), kvd[:, :2], kvd[:, 2:4], qo, scale=60.0, return_lse=True)
        got.append((o, l) + sc.sc_attn_bwd(gout.cuda(), q.cuda(), kvd[:, :2], kvd[:, 2:4], o, l, qo, scale=60.0))
    for x, y in zip(*got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("lq", [1, 200])
@pytest.mark.parametrize("at", [1, 2])
@pytest.mark.parametrize("first,then", [(1635, 1639), (1637, 1642), (-1639, -1635), (-1642, -1637)])
def test_attention_scores_that_cross_2_to_the_24(lq, at, first, then):
    """A row whose largest score (in powers of two) grows past 2^24, where fp32 holds no fraction, or comes up
    from under -2^24: the weights of the 128 keys before and of the one after agree.  The scores, 4096 * 3276 + 2 e
    or their negatives, are whole numbers that fp32 holds, and with 1.25 powers of two each the first base's fraction
    is a half.  A weight is off by its exponent's own rounding and by that of scale log2 e over a difference of at
    most 13 (together under 2^-19), and by its rounding to 16 bits."""
    d, scale = 16, float(np.float32(1.25 * math.log(2.0)))
    up = 1 if first > 0 else -1
    q = torch.zeros((lq, 1, d), dtype=torch.float16)
    q[:, 0, 0], q[:, 0, 1] = 4096.0 * up, 2.0
    k = torch.zeros((384, 1, d), dtype=torch.float16)
    k[:, 0, 0] = 3276.0
    k[:128, 0, 1] = first
    k[128:, 0, 1] = first - 400  # 1000 powers of two less
    k[at * 128 + 17, 0, 1] = then
    v = torch.randn((384, 1, d), generator=torch.Generator().manual_seed(2)).half()
    out, _, mag, _, _, _ = attn_ref(q.double(), k.double(), v.double(), [lq], [384], [0, 384], False, scale)
    off = [torch.tensor([0, n], dtype=torch.int32).cuda() for n in (lq, 384)]
    o = sc.sc_attn_fwd(q.cuda(), k.cuda(), v.cuda(), off[0], k_off=off[1], scale=scale)
    close(o, out, mag, U["f16"], 2.0 ** -19, "out")


@pytest.mark.parametrize("lq,hq,hk", [(1, 1, 1), (1, 8, 2), (130, 2, 2), (78000, 1, 1)])
@pytest.mark.parametrize("below", [15.5, 17.0, 18.2])
@pytest.mark.parametrize("value", [0.0, 0.25])
def test_attention_one_key_and_a_long_tail(lq, hq, hk, below, value):
    """f16: one key far above 120,000 nearly alike, whose own value is zero (all that comes out is the tail) or not.
    Besides its relative rounding a weight is off by half the format's smallest step, which the kernel's power of
    two brings to 2^-32 of the largest weight.  The last shape's lists are not cut, so one fp32 sum takes all
    120,000 products; the tensor cores cut a product off at 2^-25 of the sum that it is added to."""
    n, d = 120000, 64
    g = torch.Generator().manual_seed(6)
    q = torch.zeros((lq, hq, d))
    q[..., 0], q[..., 1] = 8.0, 1.0
    k = torch.zeros((n, hk, d))
    k[..., 1] = torch.randn((n, hk), generator=g) * 0.1
    k[77, :, 0] = below / 8.0
    v = torch.ones((n, hk, d))
    v[77] = value
    q, k, v = q.half(), k.half(), v.half()
    x = torch.einsum("hd,nhd->hn", q[0].double(), k.double().repeat_interleave(hq // hk, 1))
    p = torch.softmax(x, 1)
    want = ((1.0 - p[:, 77]) + value * p[:, 77])[:, None]
    off = [torch.tensor([0, m], dtype=torch.int32).cuda() for m in (lq, n)]
    o, l = sc.sc_attn_fwd(q.cuda(), k.cuda(), v.cuda(), off[0], k_off=off[1], scale=1.0, return_lse=True)
    u, rel = U["f16"], 2.0 ** -22 * 19 + 2.0 ** -20
    bound = 1.5 * ((2 * u + rel + 2.0 ** -25 * n) * want + 2.0 ** -32 * n) + 2.0 ** -24
    err = (o.double().cpu() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    # 938 tiles' sums are added one after the other in fp32, each to half a unit
    assert bool(((l.double().cpu() - torch.logsumexp(x, 1)).abs() <= 938 * 2.0 ** -24 + rel).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_extremes_gradients(dtype):
    """Scores of the format's largest sizes: lse no longer holds a weight's exponent, but a weight is never
    above 1, so the gradients are finite and gv is at most the sum of |gout|."""
    d, n = 64, 17
    q = torch.zeros((n, 1, d), dtype=DT[dtype])
    k = torch.zeros((200, 1, d), dtype=DT[dtype])
    q[:8, 0, 0], q[8:16, 0, 0] = torch.linspace(30000, 60000, 8), -torch.linspace(31000, 59000, 8)
    k[:, 0, 0] = torch.linspace(-60000, 60000, 200)
    g = torch.Generator().manual_seed(1)
    v, gout = (torch.randn((m, 1, d), generator=g).to(DT[dtype]).cuda() for m in (200, n))
    off, koff = (torch.tensor([0, m], dtype=torch.int32).cuda() for m in (n, 200))
    kw = dict(k_off=koff, scale=1.0)
    o, l = sc.sc_attn_fwd(q.cuda(), k.cuda(), v, off, return_lse=True, **kw)
    gq, gk, gv = sc.sc_attn_bwd(gout, q.cuda(), k.cuda(), v, o, l, off, **kw)
    assert all(bool(torch.isfinite(x).all()) for x in (gk, gv)), "gk, gv"
    assert bool(torch.isfinite(gq).all()), "gq"
    assert bool((gv.double().abs() <= gout.double().abs().sum(0) * (1 + 2 * U[dtype])).all())
    # the last row's scores are equal and its lse is small: all that the keys in the middle get
    want = gout[n - 1, 0].double() / 200
    err = gv.double()[95:105, 0] - want
    assert bool((err.abs() <= 1.5 * 2 * U[dtype] * want.abs() + 2.0 ** -24).all())


def test_attention_scores_of_thousands():
    """Gradients where |lse| is in the thousands: a weight taken from the fp32 lse is off by 2^-22 |lse|."""
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs([70, 200], None, 4, 2, 64, "bf16", sharp=64.0)
    out, lse, mag, grads, gmag, smax = attn_ref(q.double(), k.double(), v.double(), [70, 200], lk, ko.tolist(), True,
                                                1.0, gout.double())
    kw = dict(causal=True, scale=1.0)
    args = (q.cuda(), kvd[:, :2], kvd[:, 2:4])
    o, l = sc.sc_attn_fwd(*args, qo.cuda(), return_lse=True, **kw)
    gs = sc.sc_attn_bwd(gout.cuda(), *args, o, l, qo.cuda(), **kw)
    rel = 2.0 ** -22 * smax + 2.0 ** -20
    close(o, out, mag, U["bf16"], rel, "out")
    for got, want, m, name in zip(gs, grads, gmag, ("gq", "gk", "gv")):
        close(got, want, m, U["bf16"], 4 * rel, name)


@pytest.mark.parametrize("lq,lk,sq,sk,which", [(64, 16384, 2.0 ** -6, 16.0, 0), (4096, 16384, 16.0, 2.0 ** -6, 1)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -8])
def test_attention_small_gradients_over_long_lists(lq, lk, sq, sk, which, size):
    """f16: dS of nearly even weights over 16384 keys lies below 2^-18.  gq (and gk) are sums of thousands of
    terms of either sign, each off by the roundings of P and dS; with the result's own that is at most three
    times u in the 2-norm."""
    d, scale = 128, 128 ** -0.5
    g = torch.Generator(device="cuda").manual_seed(8)

    def rows(n, s):
        return (torch.randn((n, 1, d), generator=g, device="cuda") * s).half()

    q, k, v, gout = rows(lq, sq), rows(lk, sk), rows(lk, 1.0), rows(lq, size)
    off = [torch.tensor([0, n], dtype=torch.int32).cuda() for n in (lq, lk)]
    kw = dict(k_off=off[1], scale=scale)
    o, l = sc.sc_attn_fwd(q, k, v, off[0], return_lse=True, **kw)
    got = sc.sc_attn_bwd(gout, q, k, v, o, l, off[0], **kw)[which][:, 0].double()
    want = _grads64(q, k, v, gout, scale)[which]
    err = float((got - want).norm() / want.norm())
    assert err <= 3 * U["f16"], err


def test_attention_large_gradients_that_fit():
    """f16: gout and v whose products pass 65504 while every gradient is below it."""
    d, lq, lk = 128, [2, 3], [2, 5]
    g = torch.Generator().manual_seed(11)

    def rows(n, s):
        return (torch.randn((n, 1, d), generator=g) * s).half()

    q, k, v, gout = rows(5, 0.1), rows(7, 0.1), rows(7, 8.0), rows(5, 2048.0)
    off = [torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32) for x in (lq, lk)]
    ref = attn_ref(q.double(), k.double(), v.double(), lq, lk, off[1].tolist(), False, 0.1, gout.double())
    out, lse, mag, grads, gmag, smax = ref
    assert max(float(x.abs().max()) for x in grads) < 60000
    args = [x.cuda() for x in (q, k, v)]
    kw = dict(k_off=off[1].cuda(), scale=0.1)
    o, l = sc.sc_attn_fwd(*args, off[0].cuda(), return_lse=True, **kw)
    gs = sc.sc_attn_bwd(gout.cuda(), *args, o, l, off[0].cuda(), **kw)
    rel = 2.0 ** -22 + 2.0 ** -20
    for got, want, m, name in zip(gs, grads, gmag, ("gq", "gk", "gv")):
        close(got, want, m, U["f16"], 4 * rel, name)


def test_attention_sharp_scores_half_precision():
    """f16 gradients at sharp scores, most of whose weights are far below the format's range.  Besides the
    roundings a weight is off by 2^-25 2^-8 (P is held times 2^8) and a dS by 2^-25 where its bound, 2 head_dim
    times the sequence's largest values of gout and v, is brought to between 2^14 and 2^15."""
    lens = [70, 200]
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lens, None, 4, 2, 64, "f16", sharp=64.0)
    out, lse, mag, grads, gmag, smax = attn_ref(q.double(), k.double(), v.double(), lens, lk, ko.tolist(), True, 1.0,
                                                gout.double())
    a = 0
    for n in lens:
        step = 2.0 ** -25 * 2.0 ** -14 * 2 * 64 * float(gout[a:a + n].abs().max()) * float(v[a:a + n].abs().max())
        for h in range(4):
            j = h // 2
            gmag[0][a:a + n, h] += step / U["f16"] * k[a:a + n, j].double().abs().cumsum(0)
            gmag[1][a:a + n, j] += step / U["f16"] * q[a:a + n, h].double().abs().flip(0).cumsum(0).flip(0)
            gmag[2][a:a + n, j] += 2.0 ** -33 / U["f16"] * gout[a:a + n, h].double().abs().flip(0).cumsum(0).flip(0)
        a += n
    kw = dict(causal=True, scale=1.0)
    args = (q.cuda(), kvd[:, :2], kvd[:, 2:4])
    o, l = sc.sc_attn_fwd(*args, qo.cuda(), return_lse=True, **kw)
    gs = sc.sc_attn_bwd(gout.cuda(), *args, o, l, qo.cuda(), **kw)
    rel = 2.0 ** -22 * smax + 2.0 ** -20
    for got, want, m, name in zip(gs, grads, gmag, ("gq", "gk", "gv")):
        close(got, want, m, U["f16"], 4 * rel, name)


def test_attention_errors_reach_the_one_who_checks():
    """A thread whose calls fail, one after another, and a thread that checks on a stream of its own: every
    error is seen, those too that come while a check is under way."""
    sc.sc_attn_check()
    x, y, out = (torch.zeros((16, 2, 32), dtype=torch.float16, device="cuda") for _ in range(3))
    off = torch.tensor([0, 40, 16], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    seen, stop, failed = threading.Semaphore(0), threading.Event(), []

    def check():
        s = torch.cuda.Stream()
        while not stop.is_set():
            try:
                sc.sc_attn_check(stream=s)
            except sc.ScError:
                seen.release()

    t = threading.Thread(target=check)
    t.start()
    try:
        for i in range(200):
            sc.sc_attn_fwd(x, y, y, off, out=out)
            torch.cuda.current_stream().synchronize()
            if not seen.acquire(timeout=5):
                failed.append(i)
                break
    finally:
        stop.set()
        t.join()
    assert not failed, failed


# ------------------------------------------------------------------- views --
def test_views_that_interleave_by_head():
    """q, k and v of each head side by side ([tokens, heads, 3, head_dim] storage): rotated in place, and
    gradients written into a buffer laid out alike."""
    t, h, d = 70, 4, 32
    g = torch.Generator().manual_seed(5)
    rows = torch.randn((t, h, 3, d), generator=g).half().cuda()
    q, k, v = rows.unbind(2)
    f, _ = sc.rope_frequencies(d, device="cuda")
    pos = torch.arange(t, dtype=torch.int32).cuda()
    off = torch.tensor([0, 50, 70], dtype=torch.int32).cuda()
    want = sc.sc_qk_norm_rope_fwd(q.contiguous(), k.contiguous(), pos, f)
    keep = v.clone()
    sc.sc_qk_norm_rope_fwd(q, k, pos, f, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep)
    gout = torch.randn((t, h, d), generator=g).half().cuda()
    o, l = sc.sc_attn_fwd(q, k, v, off, return_lse=True)
    want = sc.sc_attn_bwd(gout, q, k, v, o, l, off)
    grads = torch.full_like(rows, math.nan)
    sc.sc_attn_bwd(gout, q, k, v, o, l, off, gq=grads[:, :, 0], gk=grads[:, :, 1], gv=grads[:, :, 2])
    assert torch.equal(grads, torch.stack(want, 2))
    # [heads, 2, tokens, head_dim] storage: heads lie farther apart than tokens
    kv = torch.full((h, 2, t, d), math.nan, dtype=torch.float16, device="cuda")
    gk, gv = kv[:, 0].transpose(0, 1), kv[:, 1].transpose(0, 1)
    sc.sc_attn_bwd(gout, q, k, v, o, l, off, gk=gk, gv=gv)
    assert torch.equal(gk, want[1]) and torch.equal(gv, want[2])


def test_views_that_share_rows_are_refused():
    """Interleaved views of which some rows do fall on one another."""
    rows = torch.zeros((70, 9, 32), dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    q, k, v = rows[:, 0:6:3], rows[:, 1:6:3], rows[:, 2:6:3]
    o, l = sc.sc_attn_fwd(q, k, v, off, return_lse=True)
    g = torch.zeros_like(rows)
    for gk in (g[:, 3:9:3], g[:, 0:4:2], g[:, 2:4]):  # one head of gq's 0 and 3, of gv's 2 and 5
        with pytest.raises(sc.ScError, match="overlap"):
            sc.sc_attn_bwd(o, q, k, v, o.clone(), l, off, gq=g[:, 0:6:3], gk=gk, gv=g[:, 2:6:3])
    with pytest.raises(sc.ScError, match="overlap"):
        sc.sc_attn_fwd(q, k, v, off, out=rows[:, 3:9:3])
    with pytest.raises(sc.ScError, match="overlap"):  # the same columns a row further on
        sc.sc_attn_fwd(q[:-1], k[:-1], v[:-1], off - (off > 0).int(), out=rows[1:, 0:6:3])


# ------------------------------------------------------- plans, long lists --
def test_attention_parts_that_do_not_fit_are_whole_again():
    """Many single queries, some on long key lists, and one long sequence of queries: by the average there is
    room for parts of a few rows each, by the longest there is not, and no list is cut."""
    g = torch.Generator().manual_seed(3)
    lq = [1] * 1400
    lq[700] = 300
    lk = [1] * 1400
    for i in range(0, 1400, 35):
        lk[i] = 5000 + i
    lk[700] = 400
    test = attn_inputs(lq, lk, 1, 1, 32, "f16")
    q, k, v, gout, qo, ko, lk, kvd = test
    scale = 32 ** -0.5
    out, lse, mag, grads, gmag, smax = attn_ref(q.double(), k.double(), v.double(), lq, lk, ko.tolist(), False, scale,
                                                gout.double())
    args = (q.cuda(), kvd[:, :1], kvd[:, 1:2])
    kw = dict(k_off=ko.cuda(), scale=scale)
    o, l = sc.sc_attn_fwd(*args, qo.cuda(), return_lse=True, **kw)
    gs = sc.sc_attn_bwd(gout.cuda(), *args, o, l, qo.cuda(), **kw)
    sc.sc_attn_check()
    rel = 2.0 ** -22 * max(1.0, smax) + 2.0 ** -20
    close(o, out, mag, U["f16"], rel, "out")
    assert bool(((l.double().cpu() - lse).abs() <= rel + 2.0 ** -22 * lse.abs()).all())
    for got, want, m, name in zip(gs, grads, gmag, ("gq", "gk", "gv")):
        close(got, want, m, U["f16"], 4 * rel, name)


def test_views_that_broadcast():
    """Steps of zero: one key head's rows seen as four heads', one row of gout as every token's."""
    lq, hq, d = [150, 9, 300], 4, 64
    g = torch.Generator().manual_seed(5)
    q = torch.randn((459, hq, d), generator=g).half().cuda()
    k, v = (torch.randn((459, 1, d), generator=g).half().cuda().expand(459, hq, d) for _ in range(2))
    gout = torch.randn((1, 1, d), generator=g).half().cuda().expand(459, hq, d)
    row = torch.randn((1, hq, d), generator=g).half().cuda().expand(459, hq, d)
    off = torch.tensor([0, 150, 159, 459], dtype=torch.int32).cuda()
    for qq in (q, row):
        o, l = sc.sc_attn_fwd(qq, k, v, off, causal=True, return_lse=True)
        got = (o, l) + sc.sc_attn_bwd(gout, qq, k, v, o, l, off, causal=True)
        c = [x.contiguous() for x in (gout, qq, k, v)]
        o, l = sc.sc_attn_fwd(*c[1:], off, causal=True, return_lse=True)
        want = (o, l) + sc.sc_attn_bwd(*c, o, l, off, causal=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    f, _ = sc.rope_frequencies(d, device="cuda")
    pos = torch.arange(459, dtype=torch.int32).cuda()
    w = torch.linspace(0.5, 1.5, d).cuda()
    got = sc.sc_qk_norm_rope_fwd(row, k, pos, f, w, w) + sc.sc_qk_norm_rope_bwd(gout, gout, row, k, pos, f, w, w)
    row, k, gout = (x.contiguous() for x in (row, k, gout))
    want = sc.sc_qk_norm_rope_fwd(row, k, pos, f, w, w) + sc.sc_qk_norm_rope_bwd(gout, gout, row, k, pos, f, w, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_arguments_of_the_wrong_kind():
    """Refused with the errors that the wrappers name, not with those of what they do inside."""
    x = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for freq in (1.0, [1.0] * 32, torch.tensor(1.0, device="cuda"), torch.ones((32, 1), device="cuda")):
        with pytest.raises(ValueError, match="freq"):
            sc.sc_qk_norm_rope_fwd(x, None, pos, freq)
    z = torch.zeros((4, 2, 0), dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(sc.ScError, match="head_dim"):
        sc.sc_attn_fwd(z, z, z, off)
