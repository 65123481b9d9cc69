"""GPU tests of the operators on token rows (per-head norm with the position
rotation, attention over packed sequences) against plain forms in 64 bits.

Tolerances, fixed from the formats.  u is the unit roundoff, the largest
relative error of one rounding: 2^-8 for bf16 (8 bits), 2^-11 for f16, 2^-24 for f32.  A result that is computed in fp32 and
rounded once is off by at most u |y| + 64 * 2^-24 * (the row's largest value).
In attention the weights exp(S - max) (and the gradients' P and dS) are rounded
once before a product, so a row is off by at most u * sum_j P_ij |v_jd| more,
plus the output's own rounding; the fp32 exponent of S adds a relative 2^-22 *
max|S| + 2^-20 to each weight.  The bounds below are these with a factor of
1.5 (the backward reads out rounded to the format: delta is off by u |gout|.|out|)."""
import math

import numpy as np
import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding as sc

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


# ---------------------------------------------------------------- rotation --
def rope_ref(x, w, pos, freq, eps, interleaved, amp):
    """64-bit forward on the host."""
    z = x
    if w is not None:
        z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if freq is None:
        return z
    h = freq.shape[0]
    axes = pos.shape[1]
    per = h // axes
    phi = torch.stack([pos[:, i // per].double() * freq[i].double() for i in range(h)], -1)[:, None]
    c, s = torch.cos(phi) * amp, torch.sin(phi) * amp
    y = z.clone()
    ia, ib = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    a, b = z[..., ia], z[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


ROPE = [
    # tokens, heads_q, heads_k, head_dim, rot_dim, axes, interleaved, norm, dtype
    (1, 1, 1, 16, 16, 1, False, True, "bf16"),
    (1, 32, 8, 128, 128, 1, False, True, "bf16"),
    (7, 3, 1, 64, 64, 1, False, True, "f16"),
    (33, 8, 8, 32, 32, 1, True, True, "bf16"),
    (33, 4, 4, 64, 60, 3, False, True, "f16"),     # pairs off the eight-value grid
    (19, 2, 2, 64, 42, 3, False, True, "f16"),     # an odd number of pairs
    (19, 2, 2, 64, 42, 3, True, False, "f32"),
    (65, 6, 2, 96, 48, 1, True, True, "bf16"),
    (65, 6, 2, 96, 48, 1, False, True, "f32"),
    (130, 5, 1, 80, 80, 2, False, False, "bf16"),
    (40, 3, 3, 256, 128, 4, False, True, "bf16"),
    (40, 3, 0, 24, 24, 3, False, True, "f16"),     # queries alone
    (40, 0, 2, 128, 64, 1, False, True, "f16"),    # keys alone
    (50, 4, 2, 128, 0, 1, False, True, "bf16"),    # the norm alone
    (2500, 12, 4, 64, 60, 3, False, True, "bf16"),
    (3001, 8, 8, 32, 32, 1, False, True, "f16"),
]


def rope_inputs(t, hq, hk, d, rot, axes, norm, dtype, strided=True):
    g = torch.Generator().manual_seed(t * 7 + d + rot)
    n = hq + hk
    buf = torch.randn((t, n + 1, d), generator=g).to(DT[dtype])
    dev = buf.cuda() if strided else None
    q, k = buf[:, :hq], buf[:, hq:n]
    qd, kd = dev[:, :hq], dev[:, hq:n]
    coords = torch.randint(-40000, 40000, (t, 4), generator=g, dtype=torch.int32)
    pos = coords[:, :axes]
    posd = coords.cuda()[:, :axes]
    freq = None
    if rot:
        freq, _ = sc.rope_frequencies(rot, axes=axes)
    w = [1 + 0.3 * torch.randn(d, generator=g) if norm else None for _ in range(2)]
    return q, k, qd, kd, pos, posd, freq, w, g


@pytest.mark.parametrize("t,hq,hk,d,rot,axes,ilv,norm,dtype", ROPE)
def test_qk_norm_rope_forward_and_gradients(t, hq, hk, d, rot, axes, ilv, norm, dtype):
    q, k, qd, kd, pos, posd, freq, w, g = rope_inputs(t, hq, hk, d, rot, axes, norm, dtype)
    eps, amp = 1e-5, 1.25
    gy = [torch.randn((t, h, d), generator=g).to(DT[dtype]) for h in (hq, hk)]
    fd = freq.cuda() if freq is not None else None
    wd = [x.cuda() if x is not None else None for x in w]
    kw = dict(pos=posd, freq=fd, wq=wd[0] if hq else None, wk=wd[1] if hk else None, eps=eps, interleaved=ilv, amp=amp)
    ys = sc.sc_qk_norm_rope_fwd(qd if hq else None, kd if hk else None, **kw)
    gs = sc.sc_qk_norm_rope_bwd(*(x.cuda() if h else None for x, h in zip(gy, (hq, hk))), qd if hq else None,
                                kd if hk else None, **kw)
    u = U[dtype]
    for s, (x, h) in enumerate(((q, hq), (k, hk))):
        if not h:
            assert ys[s] is None and gs[s] is None
            continue
        xr = x.double().clone().requires_grad_(True)
        wr = w[s].double().requires_grad_(True) if norm else None
        ref = rope_ref(xr, wr, pos, freq, eps, ilv, amp)
        ref.backward(gy[s].double())
        for got, want in ((ys[s], ref.detach()), (gs[s], xr.grad)):
            big = want.abs().amax(-1, keepdim=True)
            bound = u * want.abs() + 64 * 2.0 ** -24 * big + 1e-30
            if dtype == "f16":
                bound = bound + 2.0 ** -25  # below the smallest normal number
            err = (got.double().cpu() - want).abs()
            assert bool((err <= bound).all()), float((err / bound).max())
        if norm:
            gw, want = gs[2 + s].double().cpu(), wr.grad
            # sums of t * h products g x r; g, turned back, is off by 2^-21 of its pair's length
            mag = (rope_grad_terms(x.double(), gy[s].double(), pos, freq, eps, ilv, amp)).abs().sum((0, 1))
            assert bool(((gw - want).abs() <= 2.0 ** -20 * mag + 1e-30).all())
        else:
            assert gs[2 + s] is None


def rope_grad_terms(x, gy, pos, freq, eps, ilv, amp):
    back = gy.clone()
    if freq is not None:
        h = freq.shape[0]
        ia, ib = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if ilv else (slice(0, h), slice(h, 2 * h))
        back[..., ia] = back[..., ib] = amp * torch.hypot(gy[..., ia], gy[..., ib])
    return back * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def test_rope_in_place_and_same_bits_again():
    q, k, qd, kd, pos, posd, freq, w, g = rope_inputs(301, 4, 4, 64, 60, 3, True, "bf16")
    kw = dict(pos=posd, freq=freq.cuda(), wq=w[0].cuda(), wk=w[1].cuda())
    a = sc.sc_qk_norm_rope_fwd(qd, kd, **kw)
    gy = [torch.randn_like(x) for x in a]
    first = sc.sc_qk_norm_rope_bwd(gy[0], gy[1], qd, kd, **kw)
    again = sc.sc_qk_norm_rope_bwd(gy[0], gy[1], qd, kd, **kw)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    sc.sc_qk_norm_rope_fwd(qd, kd, out_q=qd, out_k=kd, **kw)
    assert torch.equal(qd, a[0]) and torch.equal(kd, a[1])
    sc.sc_qk_norm_rope_bwd(gy[0], gy[1], q.cuda(), k.cuda(), gin_q=gy[0], gin_k=gy[1], **kw)
    assert torch.equal(gy[0], first[0]) and torch.equal(gy[1], first[1])


def test_rope_gradient_against_differences():
    """f32: central differences of sum(y * gy) along random directions."""
    q, k, qd, kd, pos, posd, freq, w, g = rope_inputs(5, 2, 1, 32, 24, 3, True, "f32")
    kw = dict(pos=posd, freq=freq.cuda(), wk=w[1].cuda(), eps=1e-5, amp=1.1)
    wq = w[0].cuda()
    gy = [torch.randn((5, h, 32), generator=g).cuda() for h in (2, 1)]
    gq, gk, gwq, gwk = sc.sc_qk_norm_rope_bwd(gy[0], gy[1], qd, kd, wq=wq, **kw)

    def loss(a, ww):
        y, _ = sc.sc_qk_norm_rope_fwd(a, kd, wq=ww, **kw)
        return float((y.double() * gy[0].double()).sum())

    h = 2.0 ** -7  # the third-order term: h^2 / 6 of a direction's third derivative, below 1e-3 here
    dx = torch.randn((5, 2, 32), generator=g).cuda()
    dw = torch.randn(32, generator=g).cuda()
    base = qd.contiguous()
    num = (loss(base + h * dx, wq) - loss(base - h * dx, wq)) / (2 * h)
    assert abs(num - float((gq.double() * dx.double()).sum())) <= 5e-3 * max(1.0, abs(num))
    num = (loss(base, wq + h * dw) - loss(base, wq - h * dw)) / (2 * h)
    assert abs(num - float((gwq.double() * dw.double()).sum())) <= 1e-3 * max(1.0, abs(num))


def test_rope_no_tokens():
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    w = torch.ones(64, device="cuda")
    f = torch.ones(16, device="cuda")
    p = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    a, b = sc.sc_qk_norm_rope_fwd(q, q.clone(), p, f, w, w)
    assert a.shape == b.shape == (0, 4, 64)
    *_, gwq, gwk = sc.sc_qk_norm_rope_bwd(q, q.clone(), q, q, p, f, w, w)
    assert not gwq.any() and not gwk.any()


def test_rope_nan_stays_in_its_row():
    x = torch.randn((9, 4, 64), device="cuda").half()
    x[3, 2, 17] = math.nan
    x[5, 1, 0] = math.inf
    f, _ = sc.rope_frequencies(64, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    y, _ = sc.sc_qk_norm_rope_fwd(x, None, pos, f, wq=w)
    bad = ~torch.isfinite(y).all(-1)
    want = torch.zeros((9, 4), dtype=torch.bool)
    want[3, 2] = want[5, 1] = True
    assert torch.equal(bad.cpu(), want)


# --------------------------------------------------------------- attention --
def attn_ref(q, k, v, lq, lk, koff, causal, scale, gout=None):
    """64 bits, one sequence and head at a time, on the host: out, lse, the
    sum of P |v|, and with gout the gradients and their bounds' terms."""
    t, hq, d = q.shape
    hk = k.shape[1]
    out = torch.zeros_like(q)
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64)
    mag = torch.zeros_like(q)
    grads = [torch.zeros_like(x) for x in (q, k, v)] if gout is not None else None
    gmag = [torch.zeros_like(x) for x in (q, k, v)] if gout is not None else None
    a = 0
    smax = 0.0
    for s, n in enumerate(lq):
        b, m = koff[s], lk[s]
        for h in range(hq if n else 0):
            j = h // (hq // hk)
            if not m:
                continue
            qs, ks, vs = q[a:a + n, h], k[b:b + m, j], v[b:b + m, j]
            x = qs @ ks.T * scale
            if causal:
                keep = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)
                x = torch.where(keep, x, -math.inf)
            fin = x[torch.isfinite(x)]
            if fin.numel():
                smax = max(smax, float(fin.abs().max()))
            ls = torch.logsumexp(x, 1)
            p = torch.where(ls[:, None] == -math.inf, 0.0, torch.exp(x - ls[:, None]))
            out[a:a + n, h], lse[a:a + n, h], mag[a:a + n, h] = p @ vs, ls, p @ vs.abs()
            if gout is not None:
                g = gout[a:a + n, h]
                dp = g @ vs.T
                delta = (g * out[a:a + n, h]).sum(1, keepdim=True)
                # what rounding out does to delta, and the sizes of the products' terms
                dmag = (g.abs() * out[a:a + n, h].abs()).sum(1, keepdim=True)
                ds = p * (dp - delta) * scale
                dsm = ds.abs() + p * dmag * scale
                grads[0][a:a + n, h] = ds @ ks
                grads[1][b:b + m, j] += ds.T @ qs
                grads[2][b:b + m, j] += p.T @ g
                gmag[0][a:a + n, h] = dsm @ ks.abs()
                gmag[1][b:b + m, j] += dsm.T @ qs.abs()
                gmag[2][b:b + m, j] += p.T @ g.abs()
        a += n
    return out, lse, mag, grads, gmag, smax


def close(got, want, mag, u, rel, what):
    """|got - want| <= 1.5 (u |want| + (u + rel) * mag), mag the sum of the absolute terms."""
    g = got.double().cpu()
    assert bool(torch.isfinite(g).all()), what
    bound = 1.5 * (u * want.abs() + (u + rel) * mag) + (2.0 ** -24 if u == 2.0 ** -11 else 1e-30)
    err = (g - want).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


ATTN = [
    # query lengths, key lengths (None: the same), heads_q, heads_kv, head_dim, causal, dtype
    ([1], None, 1, 1, 16, False, "bf16"),
    ([1, 0, 5], None, 4, 2, 64, True, "f16"),
    ([130], None, 2, 2, 64, True, "bf16"),
    ([257, 128, 1, 300], None, 4, 1, 128, True, "bf16"),
    ([257, 128, 1, 300], None, 4, 4, 32, False, "f16"),
    ([40, 513], None, 6, 2, 96, True, "f16"),            # three heads a key head
    ([100, 7], [100, 300], 7, 1, 80, True, "bf16"),      # seven
    ([5, 3, 0, 9], [0, 200, 31, 2], 4, 2, 64, False, "bf16"),   # no keys, no queries
    ([5, 30, 9], [0, 10, 2], 4, 2, 64, True, "f16"),     # more queries than keys: rows that see nothing
    ([1, 1, 1, 1], [1, 700, 128, 129], 8, 2, 128, True, "bf16"),
    ([1, 1, 1], [5000, 3, 1400], 32, 8, 64, False, "f16"),
    ([4, 2], [1030, 900], 16, 2, 128, True, "f16"),
    ([60], [4100], 8, 8, 64, False, "bf16"),
    ([33], [64], 128, 1, 24, True, "bf16"),              # one key head for 128
    ([700], None, 3, 3, 40, True, "bf16"),
]


def attn_inputs(lq, lk, hq, hk, d, dtype, seed=3, sharp=1.5):
    g = torch.Generator().manual_seed(seed + sum(lq) * 3 + d)
    lk = list(lq) if lk is None else lk
    tq, tk = sum(lq), sum(lk)
    q = (torch.randn((tq, hq, d), generator=g) * sharp).to(DT[dtype])
    kv = torch.randn((tk, 2 * hk + 1, d), generator=g).to(DT[dtype])
    gout = torch.randn((tq, hq, d), generator=g).to(DT[dtype])
    off = [torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32) for x in (lq, lk)]
    return q, kv[:, :hk], kv[:, hk:2 * hk], gout, off[0], off[1], lk, kv.cuda()


@pytest.mark.parametrize("lq,lk,hq,hk,d,causal,dtype", ATTN)
def test_attention_forward_and_gradients(lq, lk, hq, hk, d, causal, dtype):
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lq, lk, hq, hk, d, dtype)
    scale = 1.1 / math.sqrt(d)
    ref = attn_ref(q.double(), k.double(), v.double(), lq, lk, ko.tolist(), causal, scale, gout.double())
    out, lse, mag, grads, gmag, smax = ref
    qd, kd, vd = q.cuda(), kvd[:, :hk], kvd[:, hk:2 * hk]
    kw = dict(k_off=ko.cuda(), causal=causal, scale=scale)
    o, l = sc.sc_attn_fwd(qd, kd, vd, qo.cuda(), return_lse=True, **kw)
    gs = sc.sc_attn_bwd(gout.cuda(), qd, kd, vd, o, l, qo.cuda(), **kw)
    sc.sc_attn_check()
    rel = 2.0 ** -22 * max(1.0, smax) + 2.0 ** -20
    close(o, out, mag, U[dtype], rel, "out")
    lc = l.double().cpu()
    empty = lse == -math.inf
    assert torch.equal(lc == -math.inf, empty)
    assert bool(((lc - lse)[~empty].abs() <= rel + 2.0 ** -22 * lse[~empty].abs()).all())
    assert not o.cpu()[empty].any()
    for got, want, m, name in zip(gs, grads, gmag, ("gq", "gk", "gv")):
        close(got, want, m, U[dtype], 4 * rel, name)


def test_attention_same_bits_again_and_on_another_stream():
    lq = [300, 1, 77]
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lq, None, 8, 2, 64, "bf16")
    args = (q.cuda(), kvd[:, :2], kvd[:, 2:4])
    qo = qo.cuda()
    o, l = sc.sc_attn_fwd(*args, qo, causal=True, return_lse=True)
    g = sc.sc_attn_bwd(gout.cuda(), *args, o, l, qo, causal=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            o2, l2 = sc.sc_attn_fwd(*args, qo, causal=True, return_lse=True)
            g2 = sc.sc_attn_bwd(gout.cuda(), *args, o2, l2, qo, causal=True)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(l, l2)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lq", [1, 200])
def test_attention_key_lists_with_room_between(causal, lq):
    """Key lists that grow in place: rows past a list's length hold NaN and are not seen."""
    cap, lens, hq, hk, d = 700, [1, 700, 0, 333], 8, 2, 64
    g = torch.Generator().manual_seed(9)
    q = torch.randn((4 * lq, hq, d), generator=g).bfloat16()
    k, v = (torch.randn((4 * cap, hk, d), generator=g).bfloat16() for _ in range(2))
    for s, n in enumerate(lens):
        k[s * cap + n:(s + 1) * cap] = math.nan
        v[s * cap + n:(s + 1) * cap] = math.nan
    qo = torch.arange(5, dtype=torch.int32) * lq
    ko = torch.arange(5, dtype=torch.int32) * cap
    out = sc.sc_attn_fwd(q.cuda(), k.cuda(), v.cuda(), qo.cuda(), k_off=ko.cuda(),
                         k_len=torch.tensor(lens, dtype=torch.int32).cuda(), causal=causal)
    sc.sc_attn_check()
    ref, _, mag, _, _, smax = attn_ref(q.double(), k.double(), v.double(), [lq] * 4, lens, ko.tolist(), causal,
                                       d ** -0.5)
    close(out, ref, mag, U["bf16"], 2.0 ** -22 * max(1.0, smax) + 2.0 ** -20, "out")


def test_attention_nan_stays_in_its_sequence():
    lq = [50, 130, 64]
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lq, None, 4, 2, 64, "f16")
    good = sc.sc_attn_fwd(q.cuda(), kvd[:, :2], kvd[:, 2:4], qo.cuda(), return_lse=True)
    ggood = sc.sc_attn_bwd(gout.cuda(), q.cuda(), kvd[:, :2], kvd[:, 2:4], *good, qo.cuda())
    qn, kvn, gn = q.clone(), kvd.clone(), gout.clone()
    for x in (qn, kvn, gn):
        x[50:180] = math.nan
    o, l = sc.sc_attn_fwd(qn.cuda(), kvn[:, :2], kvn[:, 2:4], qo.cuda(), return_lse=True)
    gs = sc.sc_attn_bwd(gn.cuda(), qn.cuda(), kvn[:, :2], kvn[:, 2:4], o, l, qo.cuda())
    keep = torch.ones(244, dtype=torch.bool)
    keep[50:180] = False
    assert torch.equal(o.cpu()[keep], good[0].cpu()[keep])
    for a, b in zip(gs, ggood):
        assert torch.equal(a.cpu()[keep], b.cpu()[keep])
    assert torch.isnan(o[60]).all()


def test_attention_extremes():
    """Scores of the format's largest sizes: the softmax stays finite and exact."""
    d = 64
    q = torch.zeros((3, 1, d), dtype=torch.float16)
    k = torch.zeros((200, 1, d), dtype=torch.float16)
    q[:, 0, 0] = torch.tensor([60000.0, -60000.0, 0.0])
    k[:, 0, 0] = torch.linspace(-60000, 60000, 200).half()
    v = torch.randn((200, 1, d), generator=torch.Generator().manual_seed(1)).half()
    off = torch.tensor([0, 3], dtype=torch.int32).cuda()
    koff = torch.tensor([0, 200], dtype=torch.int32).cuda()
    out = sc.sc_attn_fwd(q.cuda(), k.cuda(), v.cuda(), off, k_off=koff, scale=1.0).cpu()
    assert torch.equal(out[0, 0], v[199, 0]) and torch.equal(out[1, 0], v[0, 0])
    want = v.double().mean(0)[0]
    assert bool(((out[2, 0].double() - want).abs() <= 2.0 ** -11).all())


def test_attention_gradient_against_differences():
    """f16: a central difference of sum(out * gout) along random directions.  The step is a
    power of two that f16 holds; out is off by 1e-3 of its size at random, so the difference
    of sums over n values of size 1 by about 1e-3 sqrt(n) / h."""
    lq = [37, 64]
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lq, None, 4, 2, 32, "f16", sharp=1.0)
    qd, kd, vd, gd, qo = q.cuda(), k.cuda(), v.cuda(), gout.cuda(), qo.cuda()
    o, l = sc.sc_attn_fwd(qd, kd, vd, qo, causal=True, return_lse=True)
    grads = sc.sc_attn_bwd(gd, qd, kd, vd, o, l, qo, causal=True)
    g = torch.Generator().manual_seed(4)
    h = 0.25

    def loss(*x):
        return float((sc.sc_attn_fwd(*x, qo, causal=True).double() * gd.double()).sum())

    for i in range(3):
        x = [qd, kd, vd]
        step = torch.sign(torch.randn(x[i].shape, generator=g)).half().cuda() * (h / 8)
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + step, x[i] - step
        moved = (hi[i].double() - lo[i].double())  # what f16 made of the step
        num = loss(*hi) - loss(*lo)
        want = float((grads[i].double() * moved).sum())
        noise = 2.0 ** -11 * math.sqrt(2 * o.numel()) * float(gd.double().abs().mean()) * 4
        assert abs(num - want) <= noise + 0.02 * abs(want), (i, num, want)


def test_attention_bad_offsets_are_latched_and_write_nothing():
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs([8, 8], None, 2, 2, 32, "f16")
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    for bad in ([0, 9, 8], [0, 8, 17], [-1, 8, 16], [0, 40, 16]):
        off = torch.tensor(bad, dtype=torch.int32).cuda()
        out = torch.full_like(qd, 7.0)
        sc.sc_attn_fwd(qd, kd, vd, off, out=out)
        with pytest.raises(sc.ScError) as e:
            sc.sc_attn_check()
        assert e.value.code == 2
        assert bool((out == 7.0).all())
    sc.sc_attn_check()
    assert torch.isfinite(sc.sc_attn_fwd(qd, kd, vd, qo.cuda())).all()


def test_attention_empty_calls():
    z = torch.zeros((0, 2, 32), dtype=torch.float16, device="cuda")
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert sc.sc_attn_fwd(z, z.clone(), z.clone(), off).shape == (0, 2, 32)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    o, l = sc.sc_attn_fwd(z, z.clone(), z.clone(), off, return_lse=True)
    assert all(x.shape == (0, 2, 32) for x in sc.sc_attn_bwd(z, z.clone(), z.clone(), z.clone(), o, l, off))
    # keys that nobody reads: their gradients are zero
    k = torch.randn((20, 2, 32), device="cuda").half()
    qo = torch.zeros(2, dtype=torch.int32, device="cuda")
    ko = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    gq, gk, gv = sc.sc_attn_bwd(z, z.clone(), k, k.clone(), o, l, qo, k_off=ko)
    assert not gk.any() and not gv.any()
    # queries without keys
    out, l = sc.sc_attn_fwd(k, z, z.clone(), ko, k_off=qo, return_lse=True)
    assert not out.any() and bool((l == -math.inf).all())


def test_refusals_that_need_a_device():
    x = torch.zeros((16, 2, 64), dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    y = x.clone()
    with pytest.raises(sc.ScError, match="overlaps"):
        sc.sc_attn_fwd(x, y, y, off, out=x)
    with pytest.raises(sc.ScError, match="16-byte"):
        big = torch.zeros(16 * 2 * 64 + 8, dtype=torch.float16, device="cuda")
        sc.sc_attn_fwd(big[1:1 + 2048].view(16, 2, 64), y, y, off)
    with pytest.raises(sc.ScError, match="strides"):
        odd = torch.zeros((16, 2, 67), dtype=torch.float16, device="cuda")[..., :64]
        sc.sc_attn_fwd(odd, y, y, off)
    with pytest.raises(sc.ScError, match="head_dim"):
        z = torch.zeros((16, 2, 136), dtype=torch.float16, device="cuda")
        sc.sc_attn_fwd(z, z, z, off)
    with pytest.raises(sc.ScError, match="f16 or bf16"):
        sc.sc_attn_fwd(x.float(), y.float(), y.float(), off)
    with pytest.raises(sc.ScError, match="multiple of heads_kv"):
        sc.sc_attn_fwd(torch.zeros((16, 3, 64), dtype=torch.float16, device="cuda"), y, y, off)
    with pytest.raises(sc.ScError, match="scale"):
        sc.sc_attn_fwd(x, y, y, off, scale=0.0)
    with pytest.raises(ValueError, match="q_off"):
        sc.sc_attn_fwd(x, y, y, off.long())
    f = torch.ones(32, device="cuda")
    p = torch.zeros((16, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(sc.ScError, match="axes"):
        sc.sc_qk_norm_rope_fwd(x, None, p, f)
    with pytest.raises(sc.ScError, match="overlap"):
        sc.sc_qk_norm_rope_fwd(x, y, p[:, 0], f, out_q=y, out_k=x)
    with pytest.raises(ValueError, match="both norm weights"):
        sc.sc_qk_norm_rope_fwd(x, y, p[:, 0], f, wq=torch.ones(64, device="cuda"))


@pytest.mark.parametrize("hk,d,dtype", [(8, 32, "f16"), (2, 64, "bf16"), (2, 128, "f16")])
def test_attention_copies_of_a_sequence_have_the_same_bits(hk, d, dtype):
    """Enough work for every block to run several tiles in a row, in which its warps drift apart:
    what one copy's outputs and gradients are, all copies' are."""
    n, copies = 400, 120
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs([n], None, 8, hk, d, dtype)
    qd, kd, vd, gd = (x.cuda().repeat(copies, 1, 1) for x in (q, k, v, gout))
    off = torch.arange(copies + 1, dtype=torch.int32).cuda() * n
    scale = d ** -0.5
    out, lse, mag, grads, gmag, smax = attn_ref(q.double(), k.double(), v.double(), [n], [n], [0, n], False, scale,
                                                gout.double())
    rel = 2.0 ** -22 * max(1.0, smax) + 2.0 ** -20
    for _ in range(3):
        o, l = sc.sc_attn_fwd(qd, kd, vd, off, return_lse=True)
        got = (o,) + sc.sc_attn_bwd(gd, qd, kd, vd, o, l, off)
        for x, want, m, f, name in zip(got, (out,) + tuple(grads), (mag,) + tuple(gmag), (1, 4, 4, 4),
                                       ("out", "gq", "gk", "gv")):
            c = x.view(copies, n, *x.shape[1:])
            same = (c == c[:1]).flatten(1).all(1)
            assert bool(same.all()), (name, (~same).nonzero().flatten().tolist())
            close(c[0], want, m, U[dtype], f * rel, name)


LONG = [
    # keys cut where row tiles are few but whole (two parts of rows a block, several of keys)
    ([300], [5000], 2, 1, 128, True, "bf16"),
    ([300, 20], [2600, 4000], 4, 4, 64, False, "f16"),
    # one row tile a sequence, keys cut in odd numbers of tiles
    ([9, 1, 30], [1153, 6000, 385], 4, 2, 32, False, "bf16"),
    ([2, 2], [129, 2500], 8, 1, 128, True, "f16"),
    # few keys, many rows: the rows of a key tile cut in the gradients
    ([3000], [130], 4, 2, 64, False, "f16"),
    ([2500, 40], [1, 260], 6, 2, 128, False, "bf16"),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,causal,dtype", LONG)
def test_attention_with_cut_keys_and_rows(lq, lk, hq, hk, d, causal, dtype):
    test_attention_forward_and_gradients(lq, lk, hq, hk, d, causal, dtype)


def test_attention_many_sequences():
    """More sequences than the plan looks at in one run, most of them tiny or empty."""
    g = torch.Generator().manual_seed(12)
    lq = torch.randint(0, 4, (2300,), generator=g).tolist()
    lq[5], lq[1500], lq[2299] = 140, 77, 0
    test_attention_forward_and_gradients(lq, None, 2, 1, 16, True, "f16")


def test_attention_in_a_graph():
    """The calls can be captured and replayed on new inputs in the same buffers."""
    lq = [200, 31]
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lq, None, 4, 2, 64, "bf16")
    qd, kd, vd, gd, qo = q.cuda(), k.cuda(), v.cuda(), gout.cuda(), qo.cuda()
    freq, _ = sc.rope_frequencies(64, device="cuda")
    pos = torch.arange(231, dtype=torch.int32, device="cuda")

    def step():
        qr, kr = sc.sc_qk_norm_rope_fwd(qd, kd, pos, freq)
        o, l = sc.sc_attn_fwd(qr, kr, vd, qo, causal=True, return_lse=True)
        return (o,) + sc.sc_attn_bwd(gd, qr, kr, vd, o, l, qo, causal=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for scale in (1.0, 0.5):
        qd.copy_((q * scale).cuda())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    sc.sc_attn_check()


def test_fused_buffers_side_by_side():
    """Inputs and gradients that lie side by side in the rows of one buffer."""
    lq = [150, 9]
    hq, hk, d = 4, 2, 32
    q, k, v, gout, qo, ko, lk, kvd = attn_inputs(lq, None, hq, hk, d, "f16")
    rows = torch.cat([q, k, v], 1).cuda()
    qd, kd, vd = rows.split([hq, hk, hk], 1)
    qo = qo.cuda()
    o, l = sc.sc_attn_fwd(qd, kd, vd, qo, return_lse=True)
    want = sc.sc_attn_bwd(gout.cuda(), qd, kd, vd, o, l, qo)
    grads = torch.full_like(rows, math.nan)
    gq, gk, gv = grads.split([hq, hk, hk], 1)
    sc.sc_attn_bwd(gout.cuda(), qd, kd, vd, o, l, qo, gq=gq, gk=gk, gv=gv)
    assert torch.equal(grads, torch.cat(want, 1))
    # [heads, tokens, head_dim] storage
    t = [x.contiguous().permute(1, 0, 2).contiguous().permute(1, 0, 2) for x in (qd, kd, vd)]
    assert torch.equal(sc.sc_attn_fwd(*t, qo), o)
