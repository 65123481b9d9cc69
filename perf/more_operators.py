"""What is measured of the operators around attention on voxel and text tokens: the norm of rows
with the residual's addition (16-bit output, or 8 bits with scales), matrix products with their
epilogue, and the norm of all gradients with clipping.

A case is one pass through an operator:

  norm         rows normed after adding the residual (forward)
  norm_grad    the gradients of its rows and weights
  linear       product with bias, activation and residual (forward)
  linear_grad  the gradients of its rows, weights and bias
  clip         norm over many gradients and their scaling to a largest norm

``own`` false computes the plain form (elementary torch operations in 32 bits), true calls the
library.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases --
def _norm(name, op, dtype, rows, channels, residual, fp8=False, room=0):
    """room: channels between the rows (they are part of a wider buffer)."""
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "channels": channels, "residual": residual,
            "fp8": fp8, "room": room}


def _linear(name, op, dtype, rows, c_in, c_out, act, bias, residual, fp8=False, pre=False, room=0):
    """pre: the values before the activation are returned too (a training forward)."""
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "c_in": c_in, "c_out": c_out, "act": act,
            "bias": bias, "residual": residual, "fp8": fp8, "pre": pre, "room": room}


def _clip(name, dtype, tensors, total, largest, sizes):
    """`total` values in `tensors` gradients, their sizes drawn from the number `sizes`; dtype "mixed":
    every third is f32, the others bf16.  largest: the norm they are scaled to."""
    return {"name": name, "op": "clip", "dtype": dtype, "tensors": tensors, "total": total, "largest": largest,
            "sizes": sizes}


def listed():
    return [
        # one decoding step of 32 sequences: latency
        _norm("norm_step_32", "norm", "bf16", 32, 4096, True),
        # a packed prompt of 32k text tokens, quantised for the next product
        _norm("norm_prompt_32k_e4m3", "norm", "bf16", 32768, 4096, True, fp8=True),
        # training on a batch of four LiDAR scans of 120k voxels, 256 channels
        _norm("norm_voxels_480k_grad", "norm_grad", "f16", 480000, 256, True),
        # odd token count, a width that is no power of two, rows within wider ones
        _norm("norm_9973_grad", "norm_grad", "bf16", 9973, 2056, True, room=24),
        # one decoding step of 16 sequences through an output projection: the weights' bytes
        _linear("linear_step_16", "linear", "bf16", 16, 4096, 4096, "none", False, True),
        # a packed prompt through the first product of a wide MLP
        _linear("linear_prompt_8k", "linear", "bf16", 8192, 4096, 16384, "gelu", True, False),
        # the same tokens in 8 bits through an output projection
        _linear("linear_prompt_8k_e4m3", "linear", "bf16", 8192, 4096, 4096, "none", False, True, fp8=True),
        # a batch of four LiDAR scans through the first product of an MLP on 256 channels, training
        _linear("linear_voxels_480k", "linear", "f16", 480000, 256, 512, "silu", True, False, pre=True),
        # its gradients on one scan
        _linear("linear_voxels_120k_grad", "linear_grad", "f16", 120000, 256, 512, "silu", True, False),
        # odd sizes, rows within wider ones
        _linear("linear_9973_grad", "linear_grad", "bf16", 9973, 1992, 1048, "gelu", True, False, room=8),
        # a small network's gradients: latency
        _clip("clip_48_small", "f16", 48, 120001, 1.0, 3),
        # a large network's gradients, matrices in bf16, norms and biases in f32
        _clip("clip_300_mixed", "mixed", 300, 400000003, 1.0, 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "step", "linear_grad", "clip"])
    dtype = rng.choice(["bf16", "f16"])
    room = rng.choice([0, 0, 8, 40])
    if op in ("norm", "norm_grad"):
        channels = 8 * _log(rng, 2, 1024)
        fp8 = op == "norm" and rng.random() < 0.5
        dtype = rng.choice(["bf16", "f16", "f32"])
        rows = _log(rng, 1, 32768 * 4096 // (channels * (2 if dtype == "f32" else 1)))
        return _norm("", op, dtype, rows, channels, rng.random() < 0.7, fp8, room)
    if op == "clip":
        tensors = _log(rng, 1, 1000)
        total = max(tensors, _log(rng, 1000, 400000000))
        return _clip("", rng.choice(["bf16", "f16", "f32", "mixed"]), tensors, total,
                     rng.choice([1.0, 1.0, 0.25, 1e9]), rng.randrange(1, 1 << 20))
    fp8 = op != "linear_grad" and rng.random() < 0.35
    unit = 16 if fp8 else 8
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if op == "step":  # few rows, large weights
        c_in, c_out = unit * _log(rng, 256 // unit, 16384 // unit), unit * _log(rng, 256 // unit, 16384 // unit)
        return _linear("", "linear", dtype, _log(rng, 1, 128), c_in, c_out, act, rng.random() < 0.5,
                       rng.random() < 0.5, fp8, False, room * unit // 8)
    c_in, c_out = unit * _log(rng, 1, 8192 // unit), unit * _log(rng, 1, 8192 // unit)
    top = min(480000, (1 << 37) // (c_in * c_out), (1 << 29) // (c_in + c_out))
    return _linear("", op, dtype, _log(rng, 1, top), c_in, c_out, act, rng.random() < 0.6,
                   op == "linear" and rng.random() < 0.5, fp8, op == "linear" and act != "none" and rng.random() < 0.5,
                   room * unit // 8)


def sizes(case):
    """The gradients' sizes, from the case alone: shares spread over three decades."""
    r = random.Random(case["sizes"])
    n, spare = case["tensors"], case["total"] - case["tensors"]
    share = [10.0 ** r.uniform(-3, 0) for _ in range(n)]
    unit = spare / sum(share)
    out = [1 + int(s * unit) for s in share]
    out[r.randrange(n)] += case["total"] - sum(out)
    return out


def _parts(case):
    """[(dtype name, its gradients' sizes)]"""
    n = sizes(case)
    if case["dtype"] != "mixed":
        return [(case["dtype"], n)]
    parts = [("bf16", [x for i, x in enumerate(n) if i % 3 != 2]), ("f32", n[2::3])]
    return [p for p in parts if p[1]]


def work(case):
    if case["op"] == "clip":
        by = sum(sum(n) * (4 if dt == "f32" else 2) for dt, n in _parts(case))
        return {"bytes": 2 * by + 4, "flops": 3 * case["total"]}
    e = 4 if case["dtype"] == "f32" else 2
    rows = case["rows"]
    if case["op"] == "norm":
        c = case["channels"]
        per_row = c * e + (1 * c + 4 if case["fp8"] else c * e) + (2 * c * e if case["residual"] else 0)
        return {"bytes": rows * per_row + 4 * c, "flops": 6 * rows * c}
    if case["op"] == "norm_grad":  # gout, the rows and the residual's gradient in, the rows' gradient out
        c = case["channels"]
        return {"bytes": rows * c * e * (4 if case["residual"] else 3) + 8 * c, "flops": 12 * rows * c}
    c_in, c_out = case["c_in"], case["c_out"]
    if case["op"] == "linear":
        ei = 1 if case["fp8"] else 2
        outs = 1 + case["residual"] + case["pre"]
        by = rows * (c_in * ei + c_out * 2 * outs) + c_in * c_out * ei
        by += (4 * (rows + c_out) if case["fp8"] else 0) + (4 * c_out if case["bias"] else 0)
        return {"bytes": by, "flops": 2 * rows * c_in * c_out}
    # gout, pre and x in, their gradients and the weights', once each
    by = rows * 2 * (2 * c_in + (2 if case["act"] != "none" else 1) * c_out) + 4 * c_in * c_out
    return {"bytes": by + (4 * c_out if case["bias"] else 0), "flops": 4 * rows * c_in * c_out}


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std

    if case["op"] == "clip":
        return _prepare_clip(case, normal)
    dt, room, rows = DTYPES[case["dtype"]], case["room"], case["rows"]

    def wide(c, std=1.0):  # rows within wider ones
        return normal(rows, c + room, std=std).to(dt)[:, :c]

    if case["op"].startswith("norm"):
        c = case["channels"]
        s = {"case": case, "x": wide(c, 1.5), "w": 1.0 + 0.2 * normal(c), "res": None, "gout": None}
        s["x"] *= torch.exp(normal(rows, 1, std=0.5)).to(dt)  # tokens' sizes differ
        if case["op"] == "norm_grad":
            s["gout"] = normal(rows, c, std=0.3).to(dt)
        if case["residual"]:  # the other summand, or the gradient that arrives past the norm
            s["res"] = normal(rows, c, std=0.7).to(dt)
        return s
    c_in, c_out = case["c_in"], case["c_out"]
    s = {"case": case, "x": wide(c_in), "W": (normal(c_in, c_out) / math.sqrt(c_in)).to(dt), "bias": None,
         "res": None, "sx": None, "sw": None, "pre": None, "gout": None}
    if case["bias"]:
        s["bias"] = normal(c_out, std=0.5)
    if case["residual"]:
        s["res"] = normal(rows, c_out).to(dt)
    if case["op"] == "linear_grad":
        s["gout"] = normal(rows, c_out, std=0.3).to(dt)
        if case["act"] != "none":
            s["pre"] = normal(rows, c_out).to(dt)
    if case["fp8"]:  # as a quantising norm leaves the rows, and the weights laid out once
        s["x"], s["sx"] = _quantised(s["x"].float())
        s["W"], s["sw"] = _quantised(s["W"].float().t().contiguous())
        if room:  # the rows within wider ones
            buf = torch.zeros(rows, c_in + room, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
            buf.view(torch.uint8)[:, :c_in] = s["x"].view(torch.uint8)
            s["x"] = buf[:, :c_in]
    return s


def _prepare_clip(case, normal):
    s = {"case": case, "flat": [], "out": [], "grads": [], "outs": []}
    for name, n in _parts(case):
        total = sum(n)
        flat = normal(total, std=0.02).to(DTYPES[name])
        out = torch.empty_like(flat)
        s["flat"].append(flat)
        s["out"].append(out)
        s["grads"] += flat.split(n)  # each at its place, aligned to nothing
        s["outs"] += out.split(n)
    if own:  # the list a training program makes once
        from submanifold_sparse_convolution_hash_gb300 import binding as sc
        s["list"] = sc.GradList(s["grads"], out=s["outs"])
    return s


# -------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "linear": _linear_plain,
            "linear_grad": _linear_grad_plain, "clip": _clip_plain}[op](s)


def _run_own(s, op):
    from submanifold_sparse_convolution_hash_gb300 import binding as sc
    c = s["case"]
    if op == "norm":
        return sc.sc_add_norm_fwd(s["x"], s["w"], res=s["res"], eps=EPS, e4m3=c["fp8"])
    if op == "norm_grad":
        return sc.sc_add_norm_bwd(s["gout"], s["x"], s["w"], gsum=s["res"], eps=EPS)
    if op == "linear":
        return sc.sc_linear_fwd(s["x"], s["W"], bias=s["bias"], act=c["act"], res=s["res"], scale_x=s["sx"],
                                scale_w=s["sw"], dtype=DTYPES[c["dtype"]], return_pre=c["pre"])
    if op == "linear_grad":
        return sc.sc_linear_bwd(s["gout"], s["x"], s["W"], pre=s["pre"], act=c["act"], bias=c["bias"])
    norm = sc.sc_grad_clip(s["list"], c["largest"])
    return [norm] + s["out"]


# ------------------------------------------------------------- plain forms --
def _quantised(y):
    """(y in 8 bits, the scale of each row): the largest of a row becomes 448."""
    scale = y.abs().amax(-1, keepdim=True) / E4M3_MAX
    q = torch.where(scale > 0, y / scale, 0.0).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), scale.squeeze(-1)


def _norm_plain(s):
    c = s["case"]
    dt = s["x"].dtype
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    out = _quantised(y) if c["fp8"] else (y.to(dt),)
    return out + (h.to(dt),) if s["res"] is not None else out if c["fp8"] else out[0]


def _norm_grad_plain(s):
    x, g = s["x"].float(), s["gout"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, h = x * r, g * s["w"]
    gx = r * (h - n * (h * n).mean(-1, keepdim=True))
    if s["res"] is not None:
        gx = gx + s["res"].float()
    return gx.to(s["x"].dtype), (g * n).sum(0)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _linear_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["fp8"]:
        z = (s["x"].float() @ s["W"].float().t()) * s["sx"][:, None] * s["sw"]
    else:
        z = s["x"].float() @ s["W"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return (y.to(dt), z.to(dt)) if c["pre"] else y.to(dt)


def _linear_grad_plain(s):
    c = s["case"]
    dt = s["x"].dtype
    g = s["gout"].float()
    if c["act"] != "none":
        g = g * _act_slope(s["pre"].float(), c["act"])
    gx, gw = g @ s["W"].float().t(), s["x"].float().t() @ g
    return gx.to(dt), gw.to(dt), g.sum(0) if c["bias"] else None


def _clip_plain(s):
    norm = sum(f.float().square().sum(dtype=torch.float64) for f in s["flat"]).sqrt().float().view(1)
    by = torch.where(norm > s["case"]["largest"], s["case"]["largest"] / norm, 1.0)
    return [norm] + [(f.float() * by).to(f.dtype) for f in s["flat"]]


# ------------------------------------------------------- in 64 bits, apart --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        x = [f.double() for f in s["flat"]]
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(v) for v in x])).view(1)
        scale = min(1.0, case["largest"] / norm.item()) if norm.item() else 1.0
        return [norm] + [v.mul_(scale) for v in x]
    if case["op"] == "norm":
        x = s["x"].double() if s["res"] is None else torch.add(s["x"].double(), s["res"].double())
        y = torch.einsum("rc,r,c->rc", x, x.square().mean(1).add(EPS).pow(-0.5), s["w"].double())
        tail = () if s["res"] is None else (x,)
        if not case["fp8"]:
            return (y,) + tail if tail else y
        top = torch.linalg.vector_norm(y, ord=math.inf, dim=1)
        return (y * (E4M3_MAX / top.clamp(min=1e-300))[:, None], top / E4M3_MAX) + tail
    if case["op"] == "norm_grad":
        x, g, w = s["x"].double(), s["gout"].double(), s["w"].double()
        n = (x.square().mean(1) + EPS).sqrt()
        dot = torch.einsum("rc,rc,c->r", g, x, w)
        gx = torch.einsum("rc,c,r->rc", g, w, 1 / n) - torch.einsum("rc,r->rc", x, dot / (x.shape[1] * n ** 3))
        gw = torch.einsum("rc,rc,r->c", g, x, 1 / n)
        return (gx if s["res"] is None else gx + s["res"].double()), gw
    if case["rows"] * case["c_in"] * case["c_out"] > 1 << 42:
        return None  # minutes in 64 bits
    return _linear_exact(s, case)


def _linear_exact(s, c):
    """The activation from the normal and logistic distributions; its slope from their densities."""
    x, W = s["x"].double(), s["W"].double()
    if c["fp8"]:
        x, W = x * s["sx"].double()[:, None], (W * s["sw"].double()[:, None]).t()
    if c["op"] == "linear":
        z = torch.einsum("ri,io->ro", x, W)
        if s["bias"] is not None:
            z += s["bias"].double()
        y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0.0),
             "gelu": lambda: z * torch.special.ndtr(z), "silu": lambda: z * torch.sigmoid(z)}[c["act"]]()
        if s["res"] is not None:
            y = y + s["res"].double()
        return (y, z) if c["pre"] else y
    g = s["gout"].double()
    if c["act"] != "none":
        z = s["pre"].double()
        p = torch.sigmoid(z)
        g = g * {"relu": lambda: torch.heaviside(z, torch.zeros_like(z)),
                 "gelu": lambda: torch.special.ndtr(z) + z * torch.exp(torch.distributions.Normal(0., 1.).log_prob(z)),
                 "silu": lambda: torch.lerp(p, p + z * p, 1 - p)}[c["act"]]()
    return (torch.einsum("ro,io->ri", g, W), torch.einsum("ri,ro->io", x, g), g.sum(0) if c["bias"] else None)
