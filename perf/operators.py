"""What is measured of the operators for voxel and text tokens: the per-head norm of queries and
keys with the position rotation, and attention over packed sequences.

A case is one pass through an operator:

  rope         q and k of T tokens, normed per head and rotated (forward)
  rope_train   the same with its gradients
  attn         attention over packed sequences (forward)
  attn_train   the same with its gradients

``own`` false computes the plain form (elementary torch operations in 32 bits over sequences padded
to the longest), true calls the library.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def _rope(name, op, dtype, t, hq, hk, d, rot, axes, interleaved, norm, factor=1.0):
    return {"name": name, "op": op, "dtype": dtype, "t": t, "hq": hq, "hk": hk, "d": d, "rot": rot, "axes": axes,
            "interleaved": interleaved, "norm": norm, "factor": factor}


def _attn(name, op, dtype, seqs, q_lo, q_hi, k_lo, k_hi, hq, hk, d, causal, lens):
    """Lengths are drawn from the number `lens` between *_lo and *_hi; k_hi = 0: the keys are the queries' tokens."""
    return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "k_lo": k_lo,
            "k_hi": k_hi, "hq": hq, "hk": hk, "d": d, "causal": causal, "lens": lens}


def listed():
    return [
        # one decoding step of 32 sequences: latency
        _rope("rope_step_32", "rope", "bf16", 32, 32, 8, 128, 128, 1, False, True),
        # a packed prompt of 32k text tokens, frequencies scaled for a longer context
        _rope("rope_prompt_32k", "rope", "bf16", 32768, 32, 8, 128, 128, 1, False, True, 8.0),
        # training on a batch of four LiDAR scans of 120k voxels, 256 channels, rotated by x, y, z
        _rope("rope_voxels_480k_train", "rope_train", "f16", 480000, 4, 4, 64, 60, 3, False, True),
        # half of each head rotated, interleaved pairs, odd token count
        _rope("rope_partial_9973_train", "rope_train", "bf16", 9973, 12, 4, 96, 48, 1, True, True),
        # three short prompts of 1 to 64 tokens: latency
        _attn("attn_short", "attn", "f16", 3, 1, 64, 0, 0, 8, 2, 64, True, 5),
        # a batch of packed prompts of very different lengths
        _attn("attn_packed_prompts", "attn", "bf16", 10, 1, 4096, 0, 0, 32, 8, 128, True, 3),
        # one long prompt
        _attn("attn_prompt_16k", "attn", "bf16", 1, 16384, 16384, 0, 0, 32, 8, 128, True, 1),
        # a LiDAR scan's 120k voxels in windows of up to 1024 along their order, 256 channels
        _attn("attn_voxel_windows", "attn", "f16", 160, 500, 1000, 0, 0, 4, 4, 64, False, 7),
        # training on packed documents
        _attn("attn_train_packed", "attn_train", "bf16", 5, 100, 3500, 0, 0, 16, 4, 128, True, 9),
        # training on voxel windows with narrow heads
        _attn("attn_train_windows", "attn_train", "f16", 96, 300, 1000, 0, 0, 8, 8, 32, False, 11),
        # one decoding step of 64 sequences, each with its own length of keys and values
        _attn("attn_step_64", "attn", "bf16", 64, 1, 1, 1, 16384, 32, 8, 128, True, 13),
        # 100 query tokens of each of four scenes read all 120k voxels of their scene
        _attn("attn_scene_queries", "attn", "f16", 4, 100, 100, 115000, 125000, 8, 8, 64, False, 17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_train", "attn", "attn", "attn_train", "step"])
    if kind in ("rope", "rope_train"):
        d = rng.choice([32, 64, 80, 96, 128])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 1, 2, 3, 4, 8])
        axes = rng.choice([1, 1, 3])
        rot = 2 * axes * max(1, int(d // (2 * axes) * rng.choice([0.5, 0.75, 1.0])))
        dtype = rng.choice(["bf16", "f16", "f32"])
        top = 480000 * (256 if dtype == "f32" else 512) // ((hq + hk) * d)
        return _rope("", kind, dtype, _log(rng, 1, top), hq, hk, d, rot, axes,
                     rng.random() < 0.4, rng.random() < 0.75, rng.choice([1.0, 4.0, 8.0]))
    d = rng.choice([32, 64, 96, 128])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4])
    dtype = rng.choice(["bf16", "f16"])
    lens = rng.randrange(1, 1 << 20)
    if kind == "step":  # few queries, long keys
        q = rng.choice([1, 1, 1, 4, 60])
        seqs = _log(rng, 1, 100)
        k = _log(rng, 64, max(64, min(400000, 64 * 16384 * 8 // (seqs * hk))))
        return _attn("", "attn", dtype, seqs, q, q, max(q, k // 8), max(q, k), hq, hk, d, rng.random() < 0.5, lens)
    causal = rng.random() < 0.6
    most = 8192 if kind == "attn" else 3000
    hi = _log(rng, 1, most)
    room = (1 << 32) if kind == "attn" else (1 << 29)  # scores of the padded form
    seqs = _log(rng, 1, max(1, min(200, room // (hq * hi * hi))))
    return _attn("", kind, dtype, seqs, max(1, hi // 10), hi, 0, 0, hq, hk, d, causal, lens)


def lengths(case):
    """([queries], [keys]) of each sequence, from the case alone."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    q[r.randrange(len(q))] = case["q_hi"]
    if case["seqs"] > 2:
        q[r.randrange(len(q))] = case["q_lo"]
    if not case["k_hi"]:
        return q, list(q)
    k = [r.randint(case["k_lo"], case["k_hi"]) for _ in range(case["seqs"])]
    k[r.randrange(len(k))] = case["k_hi"]
    return q, k


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("rope"):
        rows = case["t"] * (case["hq"] + case["hk"])
        tensors = 2 if case["op"] == "rope" else 5  # x -> y; training: and gy, x -> gx
        return {"bytes": tensors * rows * case["d"] * e + 4 * case["t"] * case["axes"],
                "flops": (8 if case["op"] == "rope" else 24) * rows * case["d"]}
    q, k = lengths(case)
    if case["causal"]:  # query i sees keys 0 .. i + lk - lq
        pairs = sum(sum(min(b, max(0, i + b - a + 1)) for i in range(a)) for a, b in zip(q, k))
    else:
        pairs = sum(a * b for a, b in zip(q, k))
    d, hq, hk = case["d"], case["hq"], case["hk"]
    rows_q, rows_k = sum(q) * hq * d * e, sum(k) * hk * d * e
    if case["op"] == "attn":
        return {"bytes": 2 * rows_q + 2 * rows_k, "flops": 4 * d * hq * pairs}
    # forward, then gradients of q, k, v from q, k, v, out and gout
    return {"bytes": 5 * rows_q + 6 * rows_k, "flops": 14 * d * hq * pairs}


# ----------------------------------------------------------------- inputs --
def _offsets(lens, dev):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    d, hq, hk = case["d"], case["hq"], case["hk"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dt)

    if case["op"].startswith("rope"):
        t, rot, axes = case["t"], case["rot"], case["axes"]
        qkv = normal(t, (hq + 2 * hk), d, std=1.5)  # a fused projection's output: q, k, v side by side
        per = rot // 2 // axes
        i = torch.arange(rot // 2, device=dev, dtype=torch.float64) % per
        freq = (10000.0 ** (-i / per) / case["factor"]).float()
        if axes == 1:  # text: a packed batch's positions
            pos = (torch.arange(t, device=dev, dtype=torch.int32) + seed % 7) % 32768
            pos = pos.view(t, 1)
        else:  # voxel coordinates (batch, x, y, z): the last three columns
            c = torch.randint(0, 1440, (t, 4), generator=g, device=dev, dtype=torch.int32)
            pos = c[:, 1:]
        s = {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "pos": pos, "freq": freq, "wq": None,
             "wk": None, "amp": 1.0 + 0.1 * math.log(case["factor"])}
        if case["norm"]:
            s["wq"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=dev)
            s["wk"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=dev)
        if case["op"] == "rope_train":
            s["gq"] = normal(t, hq, d)
            s["gk"] = normal(t, hk, d)
        return s

    lq, lk = lengths(case)
    tq, tk = sum(lq), sum(lk)
    s = {"case": case, "q_off": _offsets(lq, dev), "k_off": _offsets(lk, dev), "max_q": max(lq), "max_k": max(lk),
         "scale": 1.0 / math.sqrt(d)}
    s["q"] = normal(tq, hq, d, std=1.7)  # after the norm and its weight
    s["k"] = normal(tk, hk, d)
    if case["k_hi"]:
        s["v"] = normal(tk, hk, d)
    else:  # v stays where the fused projection wrote it
        s["v"] = normal(tk, hq + 2 * hk, d)[:, hq + hk:]
    if case["op"] == "attn_train":
        s["gout"] = normal(tq, hq, d)
    return s


# -------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "rope":
        return _rope_plain(s)[:2]
    if op == "rope_train":
        yq, yk, *ctx = _rope_plain(s)
        return (yq, yk) + _rope_plain_grad(s, *ctx)
    if op == "attn":
        return _attn_plain(s)[0]
    return _attn_plain_train(s)


def _run_own(s, op):
    from submanifold_sparse_convolution_hash_gb300 import binding as sc
    c = s["case"]
    if op.startswith("rope"):
        kw = dict(wq=s["wq"], wk=s["wk"], eps=EPS, interleaved=c["interleaved"], amp=s["amp"])
        yq, yk = sc.sc_qk_norm_rope_fwd(s["q"], s["k"], s["pos"], s["freq"], **kw)
        if op == "rope":
            return yq, yk
        return (yq, yk) + tuple(x for x in sc.sc_qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["pos"],
                                                                  s["freq"], **kw) if x is not None)
    kw = dict(k_off=s["k_off"], causal=c["causal"], scale=s["scale"])
    if op == "attn":
        return sc.sc_attn_fwd(s["q"], s["k"], s["v"], s["q_off"], **kw)
    out, lse = sc.sc_attn_fwd(s["q"], s["k"], s["v"], s["q_off"], return_lse=True, **kw)
    return (out,) + sc.sc_attn_bwd(s["gout"], s["q"], s["k"], s["v"], out, lse, s["q_off"], **kw)


# ------------------------------------------------------------- plain forms --
def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _angles(s):
    c = s["case"]
    per = c["rot"] // 2 // c["axes"]
    # A 32-bit product of a position near 32k and a frequency is off by 1e-3 radians.  So the frequency
    # goes in two parts: 9 bits, whose product with a 15-bit position is exact, and the small rest.
    top = s["freq"].view(torch.int32).bitwise_and(-32768).view(torch.float32)
    pos = s["pos"].float().repeat_interleave(per, 1)
    x, y = pos * top, pos * (s["freq"] - top)
    cos = x.cos() * y.cos() - x.sin() * y.sin()
    sin = x.sin() * y.cos() + x.cos() * y.sin()
    return (cos * s["amp"]).unsqueeze(1), (sin * s["amp"]).unsqueeze(1)


def _rotate(z, cos, sin, c):
    a, b = _pairs(z, c["rot"], c["interleaved"])
    return _join(a * cos - b * sin, b * cos + a * sin, z[..., c["rot"]:], c["interleaved"])


def _rope_plain(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        x = x.float()
        if w is None:
            return _rotate(x, cos, sin, c), x, None
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _rotate(x * r * w, cos, sin, c), x * r, r

    yq, xq, rq = one(s["q"], s["wq"])
    yk, xk, rk = one(s["k"], s["wk"])
    dt = s["q"].dtype
    return yq.to(dt), yk.to(dt), cos, sin, xq, rq, xk, rk


def _rope_plain_grad(s, cos, sin, xq, rq, xk, rk):
    c = s["case"]
    dt = s["q"].dtype

    def one(gy, xn, r, w):
        g = _rotate(gy.float(), cos, -sin, c)
        if w is None:
            return g.to(dt), None
        h = g * w
        gx = r * (h - xn * (h * xn).mean(-1, keepdim=True))
        return gx.to(dt), (g * xn).sum((0, 1))

    gq, gwq = one(s["gq"], xq, rq, s["wq"])
    gk, gwk = one(s["gk"], xk, rk, s["wk"])
    return (gq, gk) if gwq is None else (gq, gk, gwq, gwk)


def _padded(x, off, longest):
    """[tokens, heads, d] -> float [sequences, heads, longest, d] with zeros, and which places hold a token."""
    at = torch.arange(longest, device=x.device)
    n = off[1:] - off[:-1]
    held = at < n.unsqueeze(1)
    row = torch.where(held, off[:-1].unsqueeze(1) + at, 0)
    return (x[row].float() * held[..., None, None]).transpose(1, 2), held, row


def _attn_scores(s):
    c = s["case"]
    q, held, row = _padded(s["q"], s["q_off"], s["max_q"])
    k, kheld, krow = _padded(s["k"], s["k_off"], s["max_k"])
    v, _, _ = _padded(s["v"], s["k_off"], s["max_k"])
    b, hk, lk, d = k.shape
    lq = q.shape[2]
    q = q.reshape(b, hk, -1, d)  # a key head's query heads, one after the other
    p = (q * s["scale"]) @ k.transpose(-1, -2)
    seen = kheld[:, None, :].expand(b, lq, lk)
    if c["causal"]:
        nq, nk = s["q_off"].diff(), s["k_off"].diff()
        last = torch.arange(lq, device=q.device) + (nk - nq).unsqueeze(1)
        seen = seen & (torch.arange(lk, device=q.device) <= last.unsqueeze(-1))
    sc = p.view(b, hk, -1, lq, lk)
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    sc.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = sc.sum(-1, keepdim=True)
    sc.div_(torch.where(total == 0, 1.0, total))
    return p, q, k, v, held, row, kheld, krow


def _packed(x, held):
    """[sequences, heads, longest, d] -> [tokens, heads, d]"""
    return x.transpose(1, 2)[held]


def _attn_plain(s):
    p, q, k, v, held, row, kheld, krow = _attn_scores(s)
    b, hk, lk, d = k.shape
    o = (p @ v).view(b, -1, s["max_q"], d)
    return _packed(o, held).to(s["q"].dtype), p, q, k, v, o, held, kheld


def _attn_plain_train(s):
    out, p, q, k, v, o, held, kheld = _attn_plain(s)
    b, hk, lk, d = k.shape
    lq, dt = s["max_q"], s["q"].dtype
    g, _, _ = _padded(s["gout"], s["q_off"], lq)
    delta = (g * o).sum(-1).view(b, hk, -1, 1)
    g = g.reshape(b, hk, -1, d)
    gv = p.transpose(-1, -2) @ g
    ds = (g @ v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(s["scale"])
    gq = (ds @ k).view(b, -1, lq, d)
    gk = ds.transpose(-1, -2) @ q
    return (out, _packed(gq, held).to(dt), _packed(gk, kheld).to(dt), _packed(gv, kheld).to(dt))


# ------------------------------------------------------- in 64 bits, apart --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rope"):
        return _rope_exact(s, case)
    q, k = lengths(case)
    if sum(a * b for a, b in zip(q, k)) * case["hq"] * case["d"] > 3e12:
        return None  # minutes in 64 bits
    return _attn_exact(s, case, q, k)


def _rope_exact(s, c):
    """The rotation as a complex product."""
    per = c["rot"] // 2 // c["axes"]
    phi = torch.cat([s["pos"][:, a:a + 1].double() * s["freq"][a * per:(a + 1) * per].double()
                     for a in range(c["axes"])], 1)
    turn = torch.polar(torch.full_like(phi, s["amp"]), phi)[:, None]

    def turned(z, by):
        if c["interleaved"]:
            head = torch.view_as_complex(z[..., :c["rot"]].unflatten(-1, (-1, 2)).contiguous()) * by
            head = torch.view_as_real(head).flatten(-2)
        else:
            h = c["rot"] // 2
            w = torch.complex(z[..., :h], z[..., h:2 * h]) * by
            head = torch.cat((w.real, w.imag), -1)
        return torch.cat((head, z[..., c["rot"]:]), -1)

    ys, gxs, gws = [], [], []
    for x, w, gy in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        x = x.double()
        n = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        z = x if w is None else x / n * w.double()
        ys.append(turned(z, turn))
        if gy is None:
            continue
        g = turned(gy.double(), turn.conj())
        if w is None:
            gxs.append(g)
            continue
        gws.append(torch.einsum("thd,thd->d", g, x / n))
        h = g * w.double()
        gxs.append(h / n - x * ((h * x).sum(-1, keepdim=True) / (c["d"] * n ** 3)))
    return tuple(ys) if c["op"] == "rope" else tuple(ys + gxs + gws)


def _attn_exact(s, c, lq, lk):
    """One sequence and one query head at a time, from logarithms of sums."""
    train = c["op"] == "attn_train"
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    gq = torch.zeros_like(out)
    gk, gv = (torch.zeros(k.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    a = b = 0
    for n, m in zip(lq, lk):
        for h in range(c["hq"]):
            j = h // (c["hq"] // c["hk"])
            qh, kh, vh = q[a:a + n, h].double(), k[b:b + m, j].double(), v[b:b + m, j].double()
            x = torch.einsum("id,jd->ij", qh, kh) * s["scale"]
            if c["causal"]:
                x = x.masked_fill(torch.ones(n, m, dtype=torch.bool, device=x.device).triu(m - n + 1), -math.inf)
            p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)).nan_to_num(0.0)
            out[a:a + n, h] = torch.einsum("ij,jd->id", p, vh)
            if train:
                g = s["gout"][a:a + n, h].double()
                gv[b:b + m, j] += torch.einsum("ij,id->jd", p, g)
                dp = torch.einsum("id,jd->ij", g, vh)
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
                gq[a:a + n, h] = torch.einsum("ij,jd->id", ds, kh)
                gk[b:b + m, j] += torch.einsum("ij,id->jd", ds, qh)
        a, b = a + n, b + m
    return (out, gq, gk, gv) if train else out
