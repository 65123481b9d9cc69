"""GPU tests of the operators on rows (norm with the residual's addition, linear layers,
gradient clipping) against plain forms in 64 bits.

Tolerances, fixed from the formats.  u is the largest relative error of one rounding: 2^-8 for
bf16, 2^-11 for f16, 2^-24 for f32, 2^-4 for e4m3.  A value computed in fp32 and rounded once is
off by at most u |y| and fp32's own errors:

- Norm: a row's squares are summed in chains of at most 32 values, then across at most 512 lanes
  pairwise (ten additions) and 16 warps: 64 roundings bound them, 128 with the other operations.
  Below a format's normal range a rounding is off by half its smallest step (f16: 2^-25; bf16, whose
  smallest value is 2^-133: 2^-134; e4m3: 2^-10 of the row's scale).
- Its weight gradient: chains over a block's rows, then over the blocks: at most rows + 64 roundings
  of the sum of magnitudes.
- Products: the tensor cores add 16 (8 bits: 32) products at a time to a sum and cut what lies
  below 2^-24 of it, so k values are off by at most (k / 16 + 16) 2^-23 of the sum of magnitudes;
  cut sums add one rounding a part, of at most 160.
- Activations: none is steeper than 1.13; exp and erf are good to 2^-20 of the value they form.
- Linear gradients: gz is rounded once more to the format, so a product of it is off by u times the
  sum of magnitudes.  A slope is a sum of two terms that cancel where it crosses zero: silu' = p + z p (1 - p)
  with p in (0, 1) and |z| p (1 - p) < 0.23, gelu' = Phi + z phi with |z| phi < 0.25.  Each term is off by at
  most 2^-20 of itself, so the slope by 2^-20 * 1.25 < 2^-19 at any z, whatever it is itself."""
import math

import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding as sc

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 0.0}
E = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def wide(t, room):
    """The same rows as parts of wider ones."""
    if not room:
        return t
    buf = torch.full((t.shape[0], t.shape[1] + room), math.nan, device="cuda").to(t.dtype)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / bound.clamp(min=1e-300)).nan_to_num(1e9).max()))


# -------------------------------------------------------------------- norm --
NORM = [
    # rows, channels, dtype, residual, room
    (1, 8, "bf16", True, 0),
    (3, 8, "f32", False, 8),
    (5, 24, "f16", True, 8),
    (33, 40, "bf16", True, 0),
    (7, 64, "f32", True, 4),
    (1, 128, "f16", False, 0),
    (100, 136, "bf16", True, 24),
    (257, 256, "f16", True, 0),
    (9, 264, "f32", True, 0),
    (40, 512, "bf16", True, 0),
    (3000, 504, "bf16", True, 8),
    (2500, 1000, "f16", True, 0),
    (2100, 1024, "f32", True, 0),
    (31, 1032, "bf16", True, 0),
    (2, 2056, "f16", True, 24),
    (2053, 2056, "f32", True, 0),
    (64, 4096, "bf16", True, 0),
    (2500, 4096, "bf16", False, 0),
    (3, 8184, "f32", True, 0),
    (2, 16384, "bf16", True, 0),
    (2050, 16384, "f16", True, 0),
    (1, 16384, "f32", True, 0),
    (4801, 16, "f16", True, 0),
]


def norm_inputs(rows, channels, dtype, residual, room, seed=1):
    g = gen(seed)
    x = wide(normal(g, rows, channels, std=1.5, dtype=DT[dtype]), room)
    res = normal(g, rows, channels, std=0.7, dtype=DT[dtype]) if residual else None
    w = 1.0 + 0.2 * normal(g, channels)
    return g, x, res, w


@pytest.mark.parametrize("rows,channels,dtype,residual,room", NORM)
def test_norm_forward(rows, channels, dtype, residual, room):
    _, x, res, w = norm_inputs(rows, channels, dtype, residual, room)
    h = x.double() if res is None else x.double() + res.double()
    y = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    got = sc.sc_add_norm_fwd(x, w, res=res)
    out, total = got if residual else (got, None)
    bound = (U[dtype] + 128 * E) * y.abs() + TINY[dtype]
    within(out, y, bound, "y")
    if residual:
        within(total, h, (U[dtype] + E) * h.abs() + TINY[dtype], "sum")
    # 8 bits
    got = sc.sc_add_norm_fwd(x, w, res=res, e4m3=True)
    q, s = got[:2]
    assert q.dtype == torch.float8_e4m3fn
    ref = y.abs().amax(-1) / 448
    within(s, ref, 128 * E * ref, "scale")
    bound = (2.0 ** -4 + 512 * E) * y.abs() + 2.0 ** -10 * 1.001 * ref[:, None]
    within(q.double() * s.double()[:, None], y, bound, "y in 8 bits")
    if residual:
        assert torch.equal(got[2], total)


@pytest.mark.parametrize("rows,channels,dtype",
                         [(5, 8, "f32"), (70, 264, "bf16"), (3, 4096, "f16"), (2500, 96, "bf16")])
def test_rows_quantised_as_they_are(rows, channels, dtype):
    g = gen(3)
    x = normal(g, rows, channels, std=3.0, dtype=DT[dtype])
    x[0] = 0
    if rows > 2:
        x[1] *= 2.0 ** -10
        x[2, 1:] = 0  # one value: the others are exact zeros
    q, s = sc.sc_add_norm_fwd(x, e4m3=True)
    ref = x.double().abs().amax(-1) / 448
    within(s, ref, 4 * E * ref, "scale")
    assert s[0] == 0 and not q[0].float().any()
    within(q.double() * s.double()[:, None], x.double(),
           (2.0 ** -4 + 64 * E) * x.double().abs() + 2.0 ** -10 * 1.001 * ref[:, None], "values")


def test_norm_of_zeros_and_of_values_that_are_none():
    x = torch.zeros((4, 64), device="cuda", dtype=torch.bfloat16)
    x[1, 3] = math.nan
    x[2, 3] = math.inf
    x[3] = 2.0
    w = torch.ones(64, device="cuda")
    y = sc.sc_add_norm_fwd(x, w)
    assert not y[0].any() and y[1].isnan().all() and torch.equal(y[3].float(), torch.ones(64, device="cuda"))
    assert y[2, 3].isnan() and not y[2, :3].any()
    q, s = sc.sc_add_norm_fwd(x, e4m3=True)
    assert s[0] == 0 and not q[0].float().any()
    assert q[1, 3].float().isnan() and not q[1, :3].float().any()
    assert s[2].isinf() and (q[2].float() * s[2]).isnan().all()
    assert torch.equal(q[3].float() * s[3], x[3].float())


def norm_grad_ref(gout, h, gsum, w, eps=1e-6):
    h, g, w = h.double(), gout.double(), w.double()
    r = 1 / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    n, z = h * r, g * w
    m = (z * n).mean(-1, keepdim=True)
    gin = r * (z - n * m)
    size = r * (z.abs() + n.abs() * (z * n).abs().mean(-1, keepdim=True))
    if gsum is not None:
        gin = gin + gsum.double()
        size = size + gsum.double().abs()
    return gin, size, (g * n).sum(0), (g * n).abs().sum(0)


@pytest.mark.parametrize("rows,channels,dtype,residual,room", NORM)
def test_norm_gradients(rows, channels, dtype, residual, room):
    g, h, gsum, w = norm_inputs(rows, channels, dtype, residual, room, seed=5)
    gout = normal(g, rows, channels, std=0.3, dtype=DT[dtype])
    gin, gw = sc.sc_add_norm_bwd(gout, h, w, gsum=gsum)
    ref, size, gw_ref, gw_size = norm_grad_ref(gout, h, gsum, w)
    within(gin, ref, U[dtype] * ref.abs() + 256 * E * size + TINY[dtype], "gin")
    within(gw, gw_ref, (rows + 64 + 128) * E * gw_size, "gw")
    again, gw2 = sc.sc_add_norm_bwd(gout, h, w, gsum=gsum)
    assert torch.equal(gin, again) and torch.equal(gw, gw2)
    only, none = sc.sc_add_norm_bwd(gout, h, w, gsum=gsum, need_gw=False)
    assert torch.equal(only, gin) and none is None


def test_norm_gradients_against_differences():
    """f32, so that a difference over 2^-8 has bits left: its own error is about step^2 times the third
    derivative (4e-5 here) and 2^-24 / step of the sum (2e-5); 2e-3 of the gradient's size is far above both."""
    g, x, res, w = norm_inputs(6, 40, "f32", True, 0, seed=9)
    c = normal(g, 6, 40, dtype=torch.float64)
    y, h = sc.sc_add_norm_fwd(x, w, res=res)
    gin, gw = sc.sc_add_norm_bwd(c.float(), h, w, gsum=c.float())

    def loss(x_, w_):
        y_, h_ = sc.sc_add_norm_fwd(x_, w_, res=res)
        return ((y_.double() + h_.double()) * c).sum()

    step = 2.0 ** -8
    for _ in range(4):
        d = normal(g, 6, 40)
        num = (loss(x + step * d, w) - loss(x - step * d, w)) / (2 * step)
        assert abs(num - (gin.double() * d).sum()) < 2e-3 * (gin.double() * d).abs().sum()
        d = normal(g, 40)
        num = (loss(x, w + step * d) - loss(x, w - step * d)) / (2 * step)
        assert abs(num - (gw.double() * d).sum()) < 2e-3 * (gw.double() * d).abs().sum()


def test_norm_in_place():
    for rows, channels in [(300, 256), (300, 4096), (2600, 1000)]:
        g, x, res, w = norm_inputs(rows, channels, "bf16", True, 0, seed=11)
        y, h = sc.sc_add_norm_fwd(x, w, res=res)
        a, r = x.clone(), res.clone()
        y2, h2 = sc.sc_add_norm_fwd(a, w, res=r, out=a, sum=r)
        assert y2 is a and h2 is r and torch.equal(y, a) and torch.equal(h, r)
        gout = normal(g, rows, channels, dtype=torch.bfloat16)
        gin, gw = sc.sc_add_norm_bwd(gout, h, w, gsum=res)
        for which in range(3):
            t = [gout.clone(), h.clone(), res.clone()]
            gin2, gw2 = sc.sc_add_norm_bwd(t[0], t[1], w, gsum=t[2], gin=t[which])
            assert torch.equal(gin, gin2) and torch.equal(gw, gw2)


def test_norm_without_rows():
    x = torch.empty((0, 64), device="cuda", dtype=torch.float16)
    w = torch.ones(64, device="cuda")
    assert sc.sc_add_norm_fwd(x, w).shape == (0, 64)
    q, s = sc.sc_add_norm_fwd(x, w, e4m3=True)
    assert q.shape == (0, 64) and s.shape == (0,)
    gin, gw = sc.sc_add_norm_bwd(x, x, w)
    assert gin.shape == (0, 64) and not gw.any()


# ------------------------------------------------------------------ linear --
def act_ref(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * torch.special.ndtr(z),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def slope_ref(z, act):
    p = torch.sigmoid(z)
    return {"none": lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(),
            "gelu": lambda: torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
            "silu": lambda: p * (1 + z * (1 - p))}[act]()


def sums(k):
    return (k / 16 + 16) * 2.0 ** -23 + 160 * E


LINEAR = [
    # rows, c_in, c_out, dtype, act, bias, residual, pre, room
    (1, 8, 8, "bf16", "none", False, False, False, 0),
    (1, 4096, 1000, "bf16", "silu", True, True, True, 0),
    (7, 72, 200, "f16", "gelu", True, True, True, 8),
    (16, 1000, 72, "bf16", "relu", True, False, True, 0),
    (17, 264, 520, "f16", "none", False, True, False, 16),
    (100, 512, 136, "bf16", "gelu", True, True, False, 0),
    (128, 64, 2048, "f16", "silu", True, False, False, 0),
    (129, 64, 64, "f16", "silu", True, False, True, 0),
    (255, 576, 264, "bf16", "gelu", True, True, True, 0),
    (256, 4096, 1024, "f16", "none", False, True, False, 0),
    (257, 1024, 1024, "bf16", "silu", True, True, True, 0),
    (200, 8, 16, "bf16", "none", True, True, True, 0),
    (300, 1000, 8, "f16", "relu", True, True, False, 8),
    (1000, 256, 256, "bf16", "gelu", True, True, True, 0),
    (1500, 2048, 264, "bf16", "none", False, True, False, 0),
    (5000, 136, 520, "f16", "silu", True, True, True, 24),
    (3333, 1024, 1160, "bf16", "gelu", True, True, True, 0),
    (20011, 128, 256, "f16", "silu", True, False, True, 0),
    (4100, 512, 2056, "bf16", "none", True, True, False, 0),
    (9001, 72, 40, "f16", "relu", True, True, True, 0),
]


def linear_inputs(rows, c_in, c_out, dtype, bias, residual, room, seed=21):
    g = gen(seed)
    x = wide(normal(g, rows, c_in, dtype=DT[dtype]), room)
    W = normal(g, c_in, c_out, std=c_in ** -0.5, dtype=DT[dtype])
    b = normal(g, c_out, std=0.5) if bias else None
    res = wide(normal(g, rows, c_out, dtype=DT[dtype]), room) if residual else None
    return g, x, W, b, res


def linear_check(out, pre, x, W, b, res, act, dtype, k):
    z = x @ W
    size = x.abs() @ W.abs()
    off = sums(k) * size
    if b is not None:
        z = z + b.double()
        off = off + 2 * E * z.abs()
    if pre is not None:
        within(pre, z, U[dtype] * z.abs() + (1 + U[dtype]) * off + TINY[dtype], "pre")
    y = act_ref(z, act)
    off = 1.13 * off + 2.0 ** -20 * z.abs()
    if res is not None:
        y = y + res.double()
        off = off + E * y.abs()
    within(out, y, U[dtype] * y.abs() + (1 + U[dtype]) * off + TINY[dtype], "out")


@pytest.mark.parametrize("rows,c_in,c_out,dtype,act,bias,residual,pre,room", LINEAR)
def test_linear_forward(rows, c_in, c_out, dtype, act, bias, residual, pre, room):
    _, x, W, b, res = linear_inputs(rows, c_in, c_out, dtype, bias, residual, room)
    got = sc.sc_linear_fwd(x, W, bias=b, act=act, res=res, return_pre=pre)
    out, z = got if pre else (got, None)
    linear_check(out, z, x.double(), W.double(), b, res, act, dtype, c_in)
    again = sc.sc_linear_fwd(x, W, bias=b, act=act, res=res)
    assert torch.equal(out, again)
    sc.sc_rows_check()


@pytest.mark.parametrize("rows,c_in,c_out,dtype,act,bias,residual,pre,room",
                         [c for c in LINEAR if c[1] % 16 == 0] + [(33, 16, 24, "bf16", "none", False, False, False, 0),
                                                                  (777, 4112, 264, "f16", "none", True, True, True, 0)])
def test_linear_in_8_bits(rows, c_in, c_out, dtype, act, bias, residual, pre, room):
    _, x, W, b, res = linear_inputs(rows, c_in, c_out, dtype, bias, residual, room, seed=23)
    xq, sx = sc.sc_add_norm_fwd(x, e4m3=True)
    wq, sw = sc.sc_add_norm_fwd(W.t().contiguous(), e4m3=True) if c_in >= 8 else None
    if room:
        buf = torch.full((rows, c_in + 16), 127, device="cuda", dtype=torch.uint8)  # NaN beside the rows
        buf[:, :c_in] = xq.view(torch.uint8)
        xq = buf.view(torch.float8_e4m3fn)[:, :c_in]
    got = sc.sc_linear_fwd(xq, wq, bias=b, act=act, res=res, scale_x=sx, scale_w=sw, dtype=DT[dtype], return_pre=pre)
    out, z = got if pre else (got, None)
    xd = xq.double() * sx.double()[:, None]
    wd = (wq.double() * sw.double()[:, None]).t()
    # the scales' product adds two roundings
    linear_check(out, z, xd, wd, b, res, act, dtype, c_in + 64)
    sc.sc_rows_check()


LINEAR_GRAD = [c[:6] + (c[8],) for c in LINEAR] + [
    (50000, 64, 128, "f16", "silu", True, 0),
    (30001, 256, 264, "bf16", "gelu", True, 0),
    (129, 2048, 4096, "bf16", "none", False, 0),
]


@pytest.mark.parametrize("rows,c_in,c_out,dtype,act,bias,room", LINEAR_GRAD)
def test_linear_gradients(rows, c_in, c_out, dtype, act, bias, room):
    g, x, W, _, _ = linear_inputs(rows, c_in, c_out, dtype, False, False, room, seed=25)
    gout = wide(normal(g, rows, c_out, std=0.3, dtype=DT[dtype]), room)
    pre = wide(normal(g, rows, c_out, dtype=DT[dtype]), room) if act != "none" else None
    gin, gw, gb = sc.sc_linear_bwd(gout, x, W, pre=pre, act=act, bias=bias)
    gz = gout.double()
    if pre is not None:
        gz = gz * slope_ref(pre.double(), act)
    u = U[dtype] if act != "none" else 0.0  # gz's own rounding
    slope = 2.0 ** -19 * gout.double().abs() if act != "none" else 0.0 * gout.double()
    tiny = TINY[dtype] if act != "none" else 0.0
    xd, wd = x.double(), W.double()
    ref, size = gz @ wd.t(), gz.abs() @ wd.abs().t() + 1e-30
    bound = (U[dtype] * ref.abs() + 1.01 * ((u + sums(c_out)) * size + slope @ wd.abs().t())
             + tiny * wd.abs().sum(1) + TINY[dtype])
    within(gin, ref, bound, "gin")
    ref, size = xd.t() @ gz, xd.abs().t() @ gz.abs() + 1e-30
    bound = (U[dtype] * ref.abs() + 1.01 * ((u + sums(rows)) * size + xd.abs().t() @ slope)
             + tiny * xd.abs().sum(0)[:, None] + TINY[dtype])
    within(gw, ref, bound, "gW")
    if bias:
        size = gz.abs().sum(0)
        within(gb, gz.sum(0), (rows + 64) * E * size + slope.sum(0), "gbias")
    else:
        assert gb is None
    again = sc.sc_linear_bwd(gout, x, W, pre=pre, act=act, bias=bias)
    assert torch.equal(gin, again[0]) and torch.equal(gw, again[1])
    assert not bias or torch.equal(gb, again[2])
    part = sc.sc_linear_bwd(gout, x, W, pre=pre, act=act, need_gin=False, need_gW=True)
    assert part[0] is None and part[2] is None and torch.equal(part[1], gw)
    part = sc.sc_linear_bwd(gout, x, W, pre=pre, act=act, bias=True, need_gin=True, need_gW=False)
    assert part[1] is None and torch.equal(part[0], gin)
    sc.sc_rows_check()


def test_linear_without_rows():
    x = torch.empty((0, 64), device="cuda", dtype=torch.float16)
    W = torch.ones((64, 32), device="cuda", dtype=torch.float16)
    assert sc.sc_linear_fwd(x, W).shape == (0, 32)
    gin, gw, gb = sc.sc_linear_bwd(torch.empty((0, 32), device="cuda", dtype=torch.float16), x, W, bias=True)
    assert gin.shape == (0, 64) and not gw.any() and not gb.any()


def test_rows_beside_the_last_stay_as_they_are():
    """Outputs inside larger buffers: what lies around them is not written."""
    g, x, W, b, res = linear_inputs(333, 72, 200, "f16", True, True, 0, seed=29)
    for rows in (5, 333):
        buf = torch.full((rows + 8, 216), 7.0, device="cuda", dtype=torch.float16)
        out = buf[4:4 + rows, 8:208]
        sc.sc_linear_fwd(x[:rows], W, bias=b, res=res[:rows], out=out)
        assert torch.equal(out, sc.sc_linear_fwd(x[:rows], W, bias=b, res=res[:rows]))
        buf[4:4 + rows, 8:208] = 7.0
        assert (buf == 7.0).all()


# ---------------------------------------------------------------- clipping --
def grads_of(sizes, dtypes, seed=31, std=0.02, shift=0):
    """Gradients cut from one buffer a dtype, so that they are aligned to nothing."""
    g = gen(seed)
    out = []
    for dt in dict.fromkeys(dtypes):
        n = [s for s, d in zip(sizes, dtypes) if d == dt]
        flat = normal(g, sum(n) + shift, std=std, dtype=DT[dt])[shift:]
        out += list(flat.split(n))
    return out


def clip_ref(grads, max_norm):
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    by = min(1.0, max_norm / norm) if norm > 0 else 1.0
    return norm, [t.double() * by for t in grads]


CLIP = [
    ([1], ["f32"], 0.001),
    ([3, 0, 5], ["f16"] * 3, 0.01),
    ([16384, 16383, 16385, 1, 7], ["bf16"] * 5, 1.0),
    ([8192, 8193, 100001, 17], ["f32"] * 4, 1.0),
    ([5000, 70000, 3, 9999], ["bf16", "f32", "f16", "f32"], 0.25),
    ([37] * 70, ["f16", "f32"] * 35, 0.1),
    ([11] * 1000 + [5] * 1500, ["bf16"] * 2500, 0.1),
    ([3000001], ["bf16"], 1.0),
    ([1000, 2000], ["f32", "bf16"], 1e6),
]


@pytest.mark.parametrize("sizes,dtypes,max_norm", CLIP)
@pytest.mark.parametrize("shift", [0, 1])
def test_clip(sizes, dtypes, max_norm, shift):
    grads = grads_of(sizes, dtypes, shift=shift)
    norm, ref = clip_ref(grads, max_norm)
    out = [torch.full((t.numel() + 3,), 9.0, device="cuda", dtype=t.dtype) for t in grads]
    for i in range(0, len(out), 2):  # an address of another alignment than the gradient's
        out[i] = out[i][1:]
    out = [o[:t.numel()] for o, t in zip(out, grads)]
    before = [t.clone() for t in grads]
    got = sc.sc_grad_clip(sc.GradList(grads, out=out), max_norm)
    assert got.shape == (1,) and abs(float(got) - norm) <= 64 * E * norm
    for t, o, r, b in zip(grads, out, ref, before):
        name = {v: k for k, v in DT.items()}[t.dtype]
        assert torch.equal(t, b)
        within(o, r, (U[name] + 4 * E) * r.abs() + TINY[name], "scaled")
    inside = sc.sc_grad_clip(grads, max_norm)  # in place
    assert torch.equal(inside, got)
    for t, o in zip(grads, out):
        assert torch.equal(t, o)


def test_clip_values_whose_squares_leave_the_range():
    for scale in (1e30, 1e-30, 1e-40):
        grads = [t * scale for t in grads_of([1000, 33], ["f32", "f32"], std=1.0)]
        norm, ref = clip_ref(grads, scale)
        got = sc.sc_grad_clip(grads, scale)
        assert abs(float(got) - norm) <= max(64 * E * norm, 2.0 ** -149)
        for t, r in zip(grads, ref):
            within(t, r, 8 * E * r.abs() + 2.0 ** -148, "scaled")
    # a few tiny values beside large ones, and the other way round
    t = torch.full((70000,), 1e-25, device="cuda")
    t[12345] = 1e-15
    norm, _ = clip_ref([t], 1.0)
    assert abs(float(sc.sc_grad_clip([t], 1.0)) - norm) <= 64 * E * norm
    zero = torch.zeros(100, device="cuda")
    assert float(sc.sc_grad_clip([zero], 1.0)) == 0 and not zero.any()
    assert float(sc.sc_grad_clip([], 1.0)) == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_clip_leaves_gradients_of_no_finite_norm(bad):
    for at in (0, 999, 69999):
        grads = [torch.ones(70000, device="cuda"), torch.ones(5, device="cuda", dtype=torch.bfloat16)]
        grads[0][at] = bad
        out = [torch.empty_like(t) for t in grads]
        norm = sc.sc_grad_clip(sc.GradList(grads, out=out), 1.0)
        assert norm.isnan() if math.isnan(bad) else norm.isinf()
        assert torch.equal(out[1], grads[1]) and torch.equal(out[0].nan_to_num(3.0), grads[0].nan_to_num(3.0))


def test_clip_to_nothing_and_to_infinity():
    grads = [torch.ones(100, device="cuda")]
    assert float(sc.sc_grad_clip(grads, math.inf)) == 10 and (grads[0] == 1).all()
    assert float(sc.sc_grad_clip(grads, 0.0)) == 10 and not grads[0].any()


def test_clip_refuses():
    t = torch.ones(100, device="cuda")
    for bad in (-1.0, math.nan):
        with pytest.raises(sc.ScError):
            sc.sc_grad_clip([t], bad)
    with pytest.raises(ValueError, match="share memory"):
        sc.GradList([t, t])
    with pytest.raises(ValueError, match="share memory"):
        sc.GradList([t[:60], t[50:]])
    with pytest.raises(ValueError, match="share memory"):
        sc.GradList([t[:60], t[60:]], out=[t[40:100], torch.empty(40, device="cuda")])
    with pytest.raises(ValueError, match="share memory"):
        sc.GradList([t[:60], t[60:]], out=[torch.empty(60, device="cuda"), t[:40]])
    sc.GradList([t, t], out=[torch.empty(100, device="cuda"), torch.empty(100, device="cuda")])  # read twice
    with pytest.raises(ValueError, match="contiguous"):
        sc.GradList([t.view(10, 10).t()])
    with pytest.raises(ValueError, match="dtype and size"):
        sc.GradList([t], out=[t.half()])


# ------------------------------------------------------- refusals, streams --
def test_refusals():
    x = torch.ones((4, 64), device="cuda", dtype=torch.float16)
    w = torch.ones(64, device="cuda")
    W = torch.ones((64, 32), device="cuda", dtype=torch.float16)
    with pytest.raises(sc.ScError):  # overlaps without being the same view
        buf = torch.ones((5, 64), device="cuda", dtype=torch.float16)
        sc.sc_add_norm_fwd(buf[:4], w, out=buf[1:])
    with pytest.raises(sc.ScError):  # 8 bits over the rows that are read
        sc.sc_add_norm_fwd(x, w, e4m3=True, out=x.view(torch.float8_e4m3fn)[:, :64])
    with pytest.raises(sc.ScError):
        sc.sc_add_norm_fwd(x)  # no weights, 16 bits
    with pytest.raises(sc.ScError):
        sc.sc_add_norm_fwd(torch.ones((4, 12), device="cuda"), torch.ones(12, device="cuda"))
    with pytest.raises(sc.ScError):
        sc.sc_add_norm_fwd(x, w, eps=-1.0)
    with pytest.raises(ValueError):
        sc.sc_add_norm_fwd(x, w, res=x[:3])
    with pytest.raises(ValueError):
        sc.sc_add_norm_fwd(x, w.half())
    with pytest.raises(sc.ScError):  # rows that overlap one another
        sc.sc_linear_fwd(x[:1].expand(4, 64), W)
    with pytest.raises(sc.ScError):
        sc.sc_linear_fwd(x.float(), W.float())
    with pytest.raises(sc.ScError):
        sc.sc_linear_fwd(x[:, :12].contiguous(), W[:12].contiguous())
    with pytest.raises(sc.ScError):  # not 16-byte aligned
        sc.sc_linear_fwd(torch.ones((4, 72), device="cuda", dtype=torch.float16)[:, 1:65], W)
    with pytest.raises(ValueError):
        sc.sc_linear_fwd(x, W.t())
    with pytest.raises(ValueError):
        sc.sc_linear_fwd(x, W, act="tanh")
    with pytest.raises(ValueError):
        sc.sc_linear_bwd(torch.ones((4, 32), device="cuda", dtype=torch.float16), x, W, act="gelu")
    with pytest.raises(ValueError):
        sc.sc_linear_fwd(x, W, scale_x=torch.ones(4, device="cuda"))
    out = torch.empty((4, 32), device="cuda", dtype=torch.float16)
    with pytest.raises(sc.ScError):
        sc.sc_linear_fwd(x, W, out=x[:, :32])
    sc.sc_linear_fwd(x, W, res=out, out=out)  # the residual's own rows


def everything(x, w, W, b, c):
    """A norm, a layer and their gradients, then a norm over what they give."""
    y, h = sc.sc_add_norm_fwd(x, w, res=c)
    z, pre = sc.sc_linear_fwd(y, W, bias=b, act="silu", return_pre=True)
    gin, gW, gb = sc.sc_linear_bwd(z, y, W, pre=pre, act="silu", bias=True)
    gx, gw = sc.sc_add_norm_bwd(gin, h, w, gsum=h)
    grads = [gW, gb, gw]
    norm = sc.sc_grad_clip(grads, 1.0)
    return [y, h, z, pre, gin, gx, norm] + grads


def test_another_stream_and_a_captured_graph():
    g = gen(41)
    rows = 700
    x, c = (normal(g, rows, 128, dtype=torch.bfloat16) for _ in range(2))
    w, b = 1 + normal(g, 128, std=0.1), normal(g, 264)
    W = normal(g, 128, 264, std=0.1, dtype=torch.bfloat16)
    ref = everything(x, w, W, b, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = everything(x, w, W, b, c)
    s.synchronize()
    for a, r in zip(got, ref):
        assert torch.equal(a, r)
    graphs = []
    for _ in range(2):  # two graphs, replayed at once
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = everything(x, w, W, b, c)
        graphs.append((graph, held))
    new = normal(g, rows, 128, dtype=torch.bfloat16)
    x.copy_(new)
    ref = everything(x, w, W, b, c)
    for _, held in graphs:
        for t in held:
            t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(s):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, held in graphs:
        for a, r in zip(held, ref):
            assert torch.equal(a, r)
    sc.sc_rows_check()


def test_caller_allocator():
    g = gen(43)
    x, c = (normal(g, 300, 128, dtype=torch.float16) for _ in range(2))
    w, b = 1 + normal(g, 128, std=0.1), normal(g, 264)
    W = normal(g, 128, 264, std=0.1, dtype=torch.float16)
    ref = everything(x, w, W, b, c)
    sc.use_torch_allocator()
    try:
        got = everything(x, w, W, b, c)
    finally:
        sc.use_torch_allocator(False)
    for a, r in zip(got, ref):
        assert torch.equal(a, r)
