"""GPU tests of the operators on rows where a block takes many turns, where sums are exact, and where
values leave a format's range.

Sums of whole numbers below 2^24 are exact in fp32 in any order, and a result of at most 2048 (f16) or
256 (bf16) is exact after its rounding, so the products' tests with whole numbers compare for equality: a row
or a run of k that is lost, or added twice, shows.  The other tolerances are test_gpu_rows.py's; where a
bound there grows with the number of rows, the longest chain of additions takes its place."""
import ctypes
import math
import threading

import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding as sc
from test_gpu_rows import DT, E, TINY, U, clip_ref, gen, norm_grad_ref, norm_inputs, normal, within
from test_gpu_voxel_transformer import small

pytestmark = pytest.mark.gpu


# ------------------------------------------- norms: many turns of a block --
# Rows for several turns of a grid of at most 8 blocks (of 64, 32, 16 or 8 rows) on 152 SMs, and a rest.
TURNS = [
    # rows, channels, dtype, residual, room
    (250007, 8, "bf16", True, 0),
    (200003, 24, "f16", False, 0),
    (170001, 32, "f32", True, 4),
    (90001, 64, "f32", True, 0),
    (120011, 56, "bf16", False, 8),
    (60007, 128, "bf16", True, 0),
    (61003, 120, "f32", False, 0),
    (40003, 256, "f16", True, 0),
    (30011, 256, "f32", True, 0),
    (33333, 200, "bf16", True, 16),
    (20011, 512, "bf16", True, 0),
    (20003, 440, "f32", False, 0),
    (15013, 1024, "f16", True, 0),
    (12007, 1000, "f32", True, 0),
    (9001, 1032, "bf16", True, 0),
    (5003, 4096, "f16", True, 0),
]


@pytest.mark.parametrize("rows,channels,dtype,residual,room", TURNS)
def test_norm_forward_in_many_turns(rows, channels, dtype, residual, room):
    _, x, res, w = norm_inputs(rows, channels, dtype, residual, room, seed=71)
    h = x.double() if res is None else x.double() + res.double()
    y = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    got = sc.sc_add_norm_fwd(x, w, res=res)
    out, total = got if residual else (got, None)
    within(out, y, (U[dtype] + 128 * E) * y.abs() + TINY[dtype], "y")
    if residual:
        within(total, h, (U[dtype] + E) * h.abs() + TINY[dtype], "sum")
    q, s = sc.sc_add_norm_fwd(x, w, res=res, e4m3=True)[:2]
    ref = y.abs().amax(-1) / 448
    within(s, ref, 128 * E * ref, "scale")
    bound = (2.0 ** -4 + 512 * E) * y.abs() + 2.0 ** -10 * 1.001 * ref[:, None]
    within(q.double() * s.double()[:, None], y, bound, "y in 8 bits")


@pytest.mark.parametrize("rows,channels,dtype,residual,room", TURNS)
def test_norm_gradients_in_many_turns(rows, channels, dtype, residual, room):
    g, h, gsum, w = norm_inputs(rows, channels, dtype, residual, room, seed=73)
    gout = normal(g, rows, channels, std=0.3, dtype=DT[dtype])
    gin, gw = sc.sc_add_norm_bwd(gout, h, w, gsum=gsum)
    ref, size, gw_ref, gw_size = norm_grad_ref(gout, h, gsum, w)
    within(gin, ref, U[dtype] * ref.abs() + 256 * E * size + TINY[dtype], "gin")
    # a lane's chain over the turns (a block for each SM at least, each of one row at least; of 8 rows up to
    # 1,024 channels), the block's 64 groups at most, 1,216 blocks at most by 32 ways, five levels
    chain = rows / (152 * (8 if channels <= 1024 else 1)) + 64 + 38 + 5
    within(gw, gw_ref, (chain + 128) * E * gw_size, "gw")


def test_norm_in_place_in_many_turns():
    for rows, channels in [(200003, 24), (40003, 256), (20011, 512)]:
        g, x, res, w = norm_inputs(rows, channels, "bf16", True, 0, seed=75)
        y, h = sc.sc_add_norm_fwd(x, w, res=res)
        gout = normal(g, rows, channels, dtype=torch.bfloat16)
        gin, gw = sc.sc_add_norm_bwd(gout, h, w, gsum=res)
        a, r = x.clone(), res.clone()
        sc.sc_add_norm_fwd(a, w, res=r, out=a, sum=r)
        assert torch.equal(y, a) and torch.equal(h, r)
        for which in range(3):
            t = [gout.clone(), h.clone(), res.clone()]
            gin2, gw2 = sc.sc_add_norm_bwd(t[0], t[1], w, gsum=t[2], gin=t[which])
            assert torch.equal(gin, gin2) and torch.equal(gw, gw2)


# --------------------------------------------- products of whole numbers --
def whole(g, *shape, dtype, one_in):
    """-1, 0 and 1, one value in `one_in` not 0."""
    t = torch.randint(0, 2 * one_in, shape, generator=g, device="cuda")
    return ((t == 0).to(torch.int8) - (t == 1).to(torch.int8)).to(dtype)


# rows, c_in, c_out, dtype, one_in: the sums' deviation is sqrt(n) / one_in, kept below a sixth of
# the largest whole number that the format holds
WHOLE = [
    (50000, 64, 128, "f16", 2), (100003, 256, 264, "f16", 2), (30001, 256, 264, "bf16", 8),
    (9973, 1992, 1048, "bf16", 4), (65537, 8, 8, "f16", 2), (20000003, 8, 8, "f16", 20), (129, 2048, 4096, "f16", 2),
    (777, 4104, 520, "f16", 2), (100, 8192, 1024, "f16", 2), (1, 16384, 1000, "f16", 2),
]


@pytest.mark.parametrize("rows,c_in,c_out,dtype,one_in", WHOLE)
def test_products_of_whole_numbers(rows, c_in, c_out, dtype, one_in):
    g = gen(77)
    x, W = (whole(g, *s, dtype=DT[dtype], one_in=one_in) for s in [(rows, c_in), (c_in, c_out)])
    gout = whole(g, rows, c_out, dtype=DT[dtype], one_in=one_in)
    ref = (x.double() @ W.double()).to(DT[dtype])
    assert torch.equal(sc.sc_linear_fwd(x, W), ref)
    gin, gW, gb = sc.sc_linear_bwd(gout, x, W, bias=True)
    assert torch.equal(gin, (gout.double() @ W.double().t()).to(DT[dtype]))
    assert torch.equal(gb, gout.double().sum(0).float())
    ref = x.double().t() @ gout.double()
    assert float(ref.abs().max()) <= (2048 if dtype == "f16" else 256)
    assert torch.equal(gW, ref.to(DT[dtype]))
    # relu passes or stops each value whole
    pre = whole(g, rows, c_out, dtype=DT[dtype], one_in=2)
    gin, gW, gb = sc.sc_linear_bwd(gout, x, W, pre=pre, act="relu", bias=True)
    gz = gout.double() * (pre > 0)
    assert torch.equal(gin, (gz @ W.double().t()).to(DT[dtype]))
    assert torch.equal(gW, (x.double().t() @ gz).to(DT[dtype])) and torch.equal(gb, gz.sum(0).float())
    sc.sc_rows_check()


@pytest.mark.parametrize("rows,c_in,c_out", [(3, 65536, 72), (128, 28672, 264), (300, 65536, 136), (2000, 16384, 520),
                                             (40001, 4112, 64), (1, 16, 65536), (20011, 48, 1160)])
def test_products_of_whole_numbers_in_8_bits(rows, c_in, c_out):
    """Scales of powers of two, so that they change no bit."""
    g = gen(79)
    x = whole(g, rows, c_in, dtype=torch.float32, one_in=2).to(torch.float8_e4m3fn)
    W = whole(g, c_out, c_in, dtype=torch.float32, one_in=2).to(torch.float8_e4m3fn)
    sx = 2.0 ** torch.randint(-2, 3, (rows,), generator=g, device="cuda").float()
    sw = 2.0 ** torch.randint(-2, 1, (c_out,), generator=g, device="cuda").float()
    ref = (x.double() @ W.double().t()) * sx.double()[:, None] * sw.double()
    got = sc.sc_linear_fwd(x, W, scale_x=sx, scale_w=sw, dtype=torch.float16)
    assert torch.equal(got, ref.to(torch.float16))
    sc.sc_rows_check()


def test_one_row_of_any_stride():
    """A single row's stride says nothing: a column read as a row."""
    g = gen(81)
    for c in (64, 2056):
        x = normal(g, c, 1, dtype=torch.float16).t()
        gout = normal(g, 72, 1, dtype=torch.float16).t()
        assert x.stride() == (1, 1)
        w, W = 1 + normal(g, c, std=0.1), normal(g, c, 72, std=0.1, dtype=torch.float16)
        near, gnear = x.clone(memory_format=torch.contiguous_format), gout.clone(memory_format=torch.contiguous_format)
        assert torch.equal(sc.sc_add_norm_fwd(x, w), sc.sc_add_norm_fwd(near.view(1, c), w))
        want = sc.sc_linear_fwd(near.view(1, c), W, res=gnear.view(1, 72))
        assert torch.equal(sc.sc_linear_fwd(x, W, res=gout), want)
        got = sc.sc_linear_bwd(gout, x, W, pre=gout, act="silu", bias=True)
        want = sc.sc_linear_bwd(gnear.view(1, 72), near.view(1, c), W, pre=gnear.view(1, 72), act="silu", bias=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ----------------------------------------------------------- 8-bit scales --
@pytest.mark.parametrize("rows,channels", [(7, 64), (4001, 24), (2600, 512), (2600, 1000), (2600, 4096), (7, 4096),
                                           (7, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_8_bit_scales_of_rows_without_a_norm(rows, channels, dtype):
    """Lane, block and ring forms: a row whose squares leave fp32's range, an infinity among them or not, has
    the scale infinity and gives no value; a NaN gives the scale NaN; the other rows know nothing of it."""
    g = gen(83)
    x = normal(g, rows, channels, dtype=DT[dtype])
    w = 1 + normal(g, channels, std=0.1)
    w[5] = 0.0
    q0, s0 = sc.sc_add_norm_fwd(x, w, e4m3=True)
    x[1, 3] = math.inf
    x[2, 3] = math.nan
    x[3, 5] = -math.inf  # where the weight is 0
    x[4] = 2e38
    x[5, 0], x[5, 7] = math.inf, math.nan
    q, s = sc.sc_add_norm_fwd(x, w, e4m3=True)
    for r in (1, 3, 4):
        assert float(s[r]) == math.inf, r
        assert (q[r].float() * s[r]).isnan().all(), r
    for r in (2, 5):
        assert s[r].isnan() and (q[r].float() * s[r]).isnan().all(), r
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[1:6] = False
    assert torch.equal(s[keep], s0[keep]) and torch.equal(q.view(torch.uint8)[keep], q0.view(torch.uint8)[keep])


# ---------------------------------------------------------------- clipping --
def test_clip_many_chunks_a_block():
    """Blocks walk runs of 32 KB chunks across gradients' ends: 70M values in 90 (the long table) and 41 gradients."""
    for count, seed in ((90, 5), (41, 6)):
        g = torch.Generator().manual_seed(seed)
        sizes = [int(10 ** (3 + 3.7 * float(torch.rand(1, generator=g)))) + 1 for _ in range(count)]
        dtypes = [["bf16", "f32", "f16"][i % 3] for i in range(count)]
        gg = gen(seed)
        grads = [normal(gg, n + 1, std=0.02, dtype=DT[d])[1:] if i % 4 == 1 else normal(gg, n, std=0.02, dtype=DT[d])
                 for i, (n, d) in enumerate(zip(sizes, dtypes))]
        norm, ref = clip_ref(grads, 1.0)
        out = [torch.empty_like(t) for t in grads]
        got = sc.sc_grad_clip(sc.GradList(grads, out=out), 1.0)
        assert abs(float(got) - norm) <= 64 * E * norm
        for o, r, d in zip(out, ref, dtypes):
            within(o, r, (U[d] + 4 * E) * r.abs() + TINY[d], "scaled")
        again = sc.sc_grad_clip(grads, 1.0)
        assert torch.equal(again, got) and all(torch.equal(t, o) for t, o in zip(grads, out))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clip_leaves_gradients_whose_norm_passes_fp32(dtype):
    """Finite values, a norm of 9.5e38: said as infinity, so nothing is scaled."""
    grads = [torch.full((7,), 3e38, device="cuda", dtype=DT[dtype]), torch.ones(70000, device="cuda"),
             torch.full((3,), -3e38, device="cuda", dtype=DT[dtype])]
    kept = [t.clone() for t in grads]
    out = [torch.zeros_like(t) for t in grads]
    assert float(sc.sc_grad_clip(sc.GradList(grads, out=out), 1.0)) == math.inf
    assert float(sc.sc_grad_clip(grads, 1.0)) == math.inf
    assert all(torch.equal(t, k) and torch.equal(o, k) for t, o, k in zip(grads, out, kept))


@pytest.mark.parametrize("largest", [1.0, 1e-3, 1e-30])
def test_clip_factors_below_the_normal_range(largest):
    g = gen(85)
    grads = [normal(g, 1000, std=3e36), normal(g, 33, std=3e36).bfloat16()]
    norm, ref = clip_ref(grads, largest)
    assert largest / norm < 2.0 ** -126
    got = sc.sc_grad_clip(grads, largest)
    assert abs(float(got) - norm) <= 64 * E * norm
    for t, r in zip(grads, ref):
        u = 4 * E if t.dtype is torch.float32 else U["bf16"] + 4 * E
        within(t, r, u * r.abs() + 2.0 ** -148, "scaled")


def test_clip_refuses_a_norm_among_the_gradients():
    t = torch.ones(64, device="cuda")
    o = torch.ones(64, device="cuda")
    L = sc.lib()
    for norm_at, out in ((t, t), (t, o), (o, o)):
        entry = (sc._Grad * 1)((t.data_ptr(), out.data_ptr(), 64, 0))
        assert L.sc_grad_clip(entry, 1, ctypes.c_float(1.0), norm_at.data_ptr() + 4 * 63, None) == 1
    torch.cuda.synchronize()
    assert (t == 1).all() and (o == 1).all()


# ------------------------------------------------------------ calls at once --
def test_blocks_at_once_from_threads():
    """Three of the example's blocks, each on a stream and a host thread of its own: convolution, norms, products
    in 16 and 8 bits, attention and clipping side by side on the SMs, the same bits as one after the other."""
    blocks = [small(20 + i, scans=2 + i, voxels=400 * (i + 1))[1:] for i in range(3)]

    def run(block, feats, gy):
        y = block.forward(feats)
        grads = block.backward(gy)[1:]  # the convolution's adds with atomics
        y8 = block.forward_e4m3(feats)
        norm = sc.sc_grad_clip(grads, 0.5)
        return [y, y8, norm] + grads

    for block, _, _ in blocks:
        block.quantise()
    want = [run(*b) for b in blocks]
    torch.cuda.synchronize()
    got, failed = [[] for _ in blocks], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(6):
                    got[i].append(run(*blocks[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert len(many) == 6
        for one in many:
            assert all(torch.equal(a, b) for a, b in zip(w, one))
    sc.sc_rows_check()
    sc.sc_attn_check()
