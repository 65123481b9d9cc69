"""GPU tests of the operators on rows at their limits: offsets past 32 bits, values that are none,
widths and cuts at their ends, outputs over their inputs, calls at once.

Tolerances as in test_gpu_rows.py, from the formats."""
import math

import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding as sc
from test_gpu_rows import DT, E, TINY, U, act_ref, gen, linear_check, normal, slope_ref, sums, within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------- far addresses --
def far_rows(rows, channels, dtype):
    """Rows 2^29 values apart: the ninth lies past 2^32."""
    step = 1 << 29
    buf = torch.empty((rows - 1) * step + channels, device="cuda", dtype=dtype)
    return buf.as_strided((rows, channels), (step, 1))


def test_rows_past_32_bits():
    g = gen(51)
    rows, c, co = 10, 64, 72
    x, s = far_rows(rows, c, torch.bfloat16), far_rows(rows, c, torch.bfloat16)
    near = normal(g, rows, c, dtype=torch.bfloat16)
    x.copy_(near)
    w = 1 + normal(g, c, std=0.1)
    y, h = sc.sc_add_norm_fwd(x, w, res=near, sum=s)
    y0, h0 = sc.sc_add_norm_fwd(near, w, res=near)
    assert h is s and torch.equal(y, y0) and torch.equal(h, h0)
    gin, gw = sc.sc_add_norm_bwd(near, x, w, gsum=s, gin=s)
    gin0, gw0 = sc.sc_add_norm_bwd(near, near, w, gsum=h0)
    assert torch.equal(gin, gin0) and torch.equal(gw, gw0)
    W = normal(g, c, co, std=0.1, dtype=torch.bfloat16)
    assert torch.equal(sc.sc_linear_fwd(x, W), sc.sc_linear_fwd(near, W))
    del s, h, gin
    out = far_rows(rows, co, torch.bfloat16)
    assert torch.equal(sc.sc_linear_fwd(near, W, out=out), sc.sc_linear_fwd(near, W))


def test_many_rows_past_32_bits():
    """300 rows, so that the form for many rows runs, 2^24 values apart."""
    g = gen(52)
    rows, c = 300, 64
    near = normal(g, rows, c, dtype=torch.float16)
    W = normal(g, c, c, std=0.1, dtype=torch.float16)
    buf = torch.empty((rows - 1) * (1 << 24) + c, device="cuda", dtype=torch.float16)
    x = buf.as_strided((rows, c), (1 << 24, 1))
    x.copy_(near)
    ref = sc.sc_linear_fwd(near, W, res=near)
    assert torch.equal(sc.sc_linear_fwd(x, W, res=near), ref)
    assert torch.equal(sc.sc_linear_bwd(near, x, W)[1], sc.sc_linear_bwd(near, near, W)[1])
    assert torch.equal(sc.sc_linear_fwd(near, W, res=x, out=x), ref)


def test_a_gradient_past_32_bits():
    n = (1 << 31) + 1001
    t = torch.full((n,), 0.5, device="cuda", dtype=torch.float16)
    t[-1] = 16384.0
    norm = sc.sc_grad_clip([t], 1000.0)
    want = math.sqrt(0.25 * (n - 1) + 16384.0 ** 2)
    assert abs(float(norm) - want) <= 1e-6 * want
    by = 1000.0 / want
    assert abs(float(t[-1]) - 16384.0 * by) <= 2.0 ** -10 * 16384.0 * by
    for i in (0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 2):
        assert abs(float(t[i]) - 0.5 * by) <= 2.0 ** -10 * 0.5 * by
    a, b = t[:-1].amin(), t[:-1].amax()
    assert torch.equal(a, b)


# -------------------------------------------------- values that are none --
@pytest.mark.parametrize("rows", [5, 700])
def test_values_that_are_none_stay_in_their_rows_and_columns(rows):
    g = gen(53)
    c, co = 200, 136  # k ends inside a block
    x = normal(g, rows, c, dtype=torch.bfloat16)
    W = normal(g, c, co, std=0.1, dtype=torch.bfloat16)
    gout = normal(g, rows, co, dtype=torch.bfloat16)
    clean, clean_gw = sc.sc_linear_fwd(x, W), sc.sc_linear_bwd(gout, x, W)[1]
    for bad in (math.nan, math.inf):
        xb = x.clone()
        xb[rows - 1, c - 1] = bad
        y, gw = sc.sc_linear_fwd(xb, W), sc.sc_linear_bwd(gout, xb, W)[1]
        assert torch.equal(y[:-1], clean[:-1]) and not torch.isfinite(y[-1]).any()
        assert torch.equal(gw[:-1], clean_gw[:-1]) and not torch.isfinite(gw[-1]).any()
        Wb = W.clone()
        Wb[c - 1, co - 1] = bad
        y = sc.sc_linear_fwd(x, Wb)
        assert torch.equal(y[:, :-1], clean[:, :-1]) and not torch.isfinite(y[:, -1]).any()
    z = torch.full((rows, co), math.nan, device="cuda", dtype=torch.bfloat16)
    for act in ("relu", "gelu", "silu"):
        assert sc.sc_linear_fwd(x, W, bias=torch.full((co,), math.nan, device="cuda"), act=act).isnan().all()
    assert sc.sc_linear_fwd(x, W, res=z).isnan().all()


def test_activations_far_from_zero():
    """z through a product with one: exact, so that the activation alone is seen, to the ends of f16 and bf16."""
    for dtype, ends in (("f16", [65504.0, 100.0, 12.0, 6e-8]), ("bf16", [3e38, 1e4, 20.0, 1e-38])):
        vals = torch.tensor([s * e for e in ends for s in (1, -1)] + [0.0, 1.0, -1.0, 5.0, -5.0, -8.0, -13.0, 3.0],
                            device="cuda").to(DT[dtype])
        x = torch.zeros((300, 16), device="cuda", dtype=DT[dtype])
        x[:] = vals
        eye = torch.eye(16, device="cuda", dtype=DT[dtype])
        for act in ("relu", "gelu", "silu"):
            for rows in (3, 300):
                y = sc.sc_linear_fwd(x[:rows], eye, act=act)
                ref = act_ref(x[:rows].double(), act)
                # the integral is off by 2^-22 (and by 2^-18 of itself): values past the last bits are 0
                bound = ((U[dtype] + 2.0 ** -18) * ref.abs() + 2.0 ** -22 * x[:rows].double().abs().clamp(max=16)
                         + TINY[dtype])
                within(y, ref, bound, act)
            pre = x
            gout = torch.ones_like(x)
            gin = sc.sc_linear_bwd(gout, x, eye, pre=pre, act=act, need_gW=False)[0]
            ref = slope_ref(pre.double(), act)
            within(gin, ref, 2 * U[dtype] * ref.abs() + 2.0 ** -19 + TINY[dtype], act + "'")


# ------------------------------------------------------- widths and cuts --
WIDTHS = [
    # rows, c_in, c_out
    (3, 65536, 8), (2, 8, 65536), (300, 65536, 8), (300, 8, 65536), (1, 576, 8), (5, 520, 128), (128, 4160, 136),
    (100, 16384, 264), (129, 8, 8), (1000, 4096, 64), (1000, 8, 8),
]


@pytest.mark.parametrize("rows,c_in,c_out", WIDTHS)
def test_widths_and_cuts_of_k(rows, c_in, c_out):
    g = gen(55)
    x = normal(g, rows, c_in, dtype=torch.bfloat16)
    W = normal(g, c_in, c_out, std=c_in ** -0.5, dtype=torch.bfloat16)
    gout = normal(g, rows, c_out, dtype=torch.bfloat16)
    b = normal(g, c_out)
    out, pre = sc.sc_linear_fwd(x, W, bias=b, act="silu", res=gout, return_pre=True)
    linear_check(out, pre, x.double(), W.double(), b, gout, "silu", "bf16", c_in)
    gin, gw, gb = sc.sc_linear_bwd(gout, x, W, bias=True)
    gd, xd, wd, u = gout.double(), x.double(), W.double(), U["bf16"]
    ref = gd @ wd.t()
    within(gin, ref, u * ref.abs() + 1.01 * sums(c_out) * (gd.abs() @ wd.abs().t()), "gin")
    ref = xd.t() @ gd
    within(gw, ref, u * ref.abs() + 1.01 * sums(rows) * (xd.abs().t() @ gd.abs()), "gW")
    within(gb, gd.sum(0), (rows + 64) * E * gd.abs().sum(0), "gbias")
    sc.sc_rows_check()


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 127, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_few_rows(rows, dtype):
    g = gen(57 + rows)
    x = normal(g, rows, 1032, dtype=DT[dtype])
    W = normal(g, 1032, 392, std=1032 ** -0.5, dtype=DT[dtype])
    b, res = normal(g, 392), normal(g, rows, 392, dtype=DT[dtype])
    out, pre = sc.sc_linear_fwd(x, W, bias=b, act="gelu", res=res, return_pre=True)
    linear_check(out, pre, x.double(), W.double(), b, res, "gelu", dtype, 1032)


# ------------------------------------------- over their inputs, at once --
@pytest.mark.parametrize("rows,c,co", [(9, 256, 512), (3333, 264, 520), (40000, 64, 128)])
def test_the_residual_is_overwritten_in_place(rows, c, co):
    g = gen(61)
    x, W = normal(g, rows, c, dtype=torch.float16), normal(g, c, co, std=0.1, dtype=torch.float16)
    res = normal(g, rows, co, dtype=torch.float16)
    b = normal(g, co)
    ref = sc.sc_linear_fwd(x, W, bias=b, act="relu", res=res)
    kept = res.clone()
    got = sc.sc_linear_fwd(x, W, bias=b, act="relu", res=res, out=res)
    assert got is res and torch.equal(got, ref)
    got, _ = sc.sc_linear_fwd(x, W, bias=b, act="relu", res=kept, out=kept, return_pre=True)
    assert torch.equal(got, ref)


def test_calls_at_once_on_two_streams():
    g = gen(63)
    shapes = [(16, 4096, 512), (2000, 256, 264), (700, 4096, 64)]
    work = []
    for rows, c, co in shapes:
        x, W = normal(g, rows, c, dtype=torch.bfloat16), normal(g, c, co, std=0.05, dtype=torch.bfloat16)
        gout = normal(g, rows, co, dtype=torch.bfloat16)
        w = 1 + normal(g, c, std=0.1)
        work.append((x, W, gout, w))

    def run(x, W, gout, w):
        y = sc.sc_add_norm_fwd(x, w)
        z = sc.sc_linear_fwd(y, W, act="gelu")
        gin, gW, gb = sc.sc_linear_bwd(gout, y, W, pre=z, act="gelu", bias=True)
        gx, gw = sc.sc_add_norm_bwd(gin, x, w)
        norm = sc.sc_grad_clip([gW, gb, gw], 0.5)
        return [y, z, gin, gW, gb, gx, gw, norm]

    ref = [run(*a) for a in work]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [[] for _ in work]
    for _ in range(5):
        for i, (s, a) in enumerate(zip(streams, work)):
            with torch.cuda.stream(s):
                got[i].append(run(*a))
    torch.cuda.synchronize()
    for r, many in zip(ref, got):
        for one in many:
            assert all(torch.equal(a, b) for a, b in zip(r, one))
    sc.sc_rows_check()


def test_broadcast_rows_may_be_read():
    """Rows of stride 0: one vector for every row of a norm."""
    g = gen(65)
    x = normal(g, 50, 128, dtype=torch.bfloat16)
    one = normal(g, 1, 128, dtype=torch.bfloat16)
    w = torch.ones(128, device="cuda")
    many = one.expand(50, 128)
    a = sc.sc_add_norm_fwd(x, w, res=many)
    b = sc.sc_add_norm_fwd(x, w, res=many.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = torch.ones(2056, device="cuda")
    y = sc.sc_add_norm_fwd(torch.ones((1, 2056), device="cuda").expand(9, 2056), wide)
    assert torch.equal(y, y[:1].expand(9, 2056).contiguous())
    with pytest.raises(sc.ScError):  # written rows lie apart
        sc.sc_add_norm_fwd(x, w, out=torch.empty((1, 128), device="cuda", dtype=torch.bfloat16).expand(50, 128))


def test_the_rows_launch_and_their_names():
    """The kernels that a block's layers run are the library's own."""
    x = torch.ones((400, 64), device="cuda", dtype=torch.float16)
    W = torch.ones((64, 64), device="cuda", dtype=torch.float16)
    sc.profile_enable(True)
    sc.profile_reset()
    try:
        sc.sc_linear_fwd(x, W)
        sc.sc_linear_fwd(x[:3], W)
        sc.sc_add_norm_fwd(x, torch.ones(64, device="cuda"))
        sc.sc_grad_clip([torch.ones(5, device="cuda")], 1.0)
        ran = {k for k, v in sc.profile_collect().items() if v[0]}
    finally:
        sc.profile_enable(False)
    assert {"linear_gemm", "linear_few", "add_norm_fwd", "grad_squares", "grad_scale"} <= ran
