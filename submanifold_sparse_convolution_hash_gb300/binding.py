"""Thin ctypes binding over libsc (include/sc.h), with the same names.

Argument marshalling only: torch tensors become device pointers, sizes and a
stream; every step of the layer runs in libsc's CUDA kernels.  There is no
CPU path: if libsc.so is missing, or a tensor is not on a CUDA device, the
calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsc.so")
_lib = None

SC_RELU = 0x1
SC_VARIANT_FUSED = 0x10
SC_VARIANT_WS = 0x20
SC_VARIANT_SIMT = 0x40
SC_VARIANT_SPLIT = 0x80
SC_KMAP_NO_SYNC = 0x100
SC_KMAP_ORDER = 0x200
SC_KMAP_NO_ORDER = 0x400
SC_KMAP_SORT = 0x800
SC_KMAP_NO_SORT = 0x1000
SC_KMAP_TRANSPOSE = 0x2000
SC_KMAP_HALF = 0x4000
SC_KMAP_SPLIT = 0x8000
SC_KMAP_TILE_TABLE = 0x10000
SC_ROPE_INTERLEAVED = 0x1
SC_ATTN_CAUSAL = 0x1
SC_ACT = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
VARIANTS = {"fused": SC_VARIANT_FUSED, "ws": SC_VARIANT_WS, "simt": SC_VARIANT_SIMT, "split": SC_VARIANT_SPLIT}
VARIANT_NAMES = {v: k for k, v in VARIANTS.items()}
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_E4M3 = torch.float8_e4m3fn
_E4M3_CODE = 3
STATUS = {0: "SC_OK", 1: "SC_ERR_INVALID_ARG", 2: "SC_ERR_OUT_OF_RANGE", 3: "SC_ERR_DUPLICATE_COORD",
          4: "SC_ERR_TABLE_FULL", 5: "SC_ERR_UNSUPPORTED", 6: "SC_ERR_CUDA", 7: "SC_ERR_OOM",
          8: "SC_ERR_TIMEOUT"}


class ScError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded libsc.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libsc.so is not built: run `python -m submanifold_sparse_convolution_hash_gb300.build`"
                               " or __graft_entry__.build()")
        L = ctypes.CDLL(_LIB_PATH)
        P, I64, I32, U = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint
        F = ctypes.c_float
        sig = {
            "sc_hash_build": ([P, I64, P, P, P], I32),
            "sc_hash_query": ([P, P, I64, P, P], I32),
            "sc_hash_info": ([P, P, P], I32),
            "sc_hash_check": ([P, P], I32),
            "sc_hash_destroy": ([P, P], I32),
            "sc_hash_build_conv_out": ([P, I32, I32, I32, P, P, P, P], I32),
            "sc_hash_coords": ([P, P, P], I32),
            "sc_kmap_build_conv": ([P, P, I32, I32, I32, P, U, P, P, P], I32),
            "sc_kmap_build": ([P, I32, I32, P, U, P, P, P], I32),
            "sc_kmap_view": ([P, P, P, P, P, P], I32),
            "sc_kmap_info": ([P, P, P, P, P], I32),
            "sc_kmap_check": ([P, P], I32),
            "sc_kmap_export": ([P, P, P, P, P, P], I32),
            "sc_kmap_destroy": ([P, P], I32),
            "sc_subm_conv_fwd": ([P, P, P, P, I32, I32, I32, U, P], I32),
            "sc_subm_conv_bwd_data": ([P, P, P, P, I32, I32, I32, U, P], I32),
            "sc_subm_conv_bwd_weight": ([P, P, P, P, I32, I32, I32, U, P], I32),
            "sc_subm_conv_tune": ([P, P, P, P, I32, I32, I32, U, I32, P, P], I32),
            "sc_subm_conv_fwd_noalloc": ([P, P, P, P, I32, I32, I32, U, P], I32),
            "sc_qk_norm_rope_fwd": ([P] * 7 + [I64, I32, P, I64, I32, I32, I32, I32, F, F, I32, U, P], I32),
            "sc_qk_norm_rope_bwd": ([P] * 11 + [I64, I32, P, I64, I32, I32, I32, I32, F, F, I32, U, P], I32),
            "sc_attn_fwd": ([P] * 8 + [I64, I64, I64, I32, I32, I32, F, I32, U, P], I32),
            "sc_attn_bwd": ([P] * 11 + [I64, I64, I64, I32, I32, I32, F, I32, U, P], I32),
            "sc_attn_check": ([P], I32),
            "sc_add_norm_fwd": ([P] * 6 + [I64, I32, F, I32, I32, P], I32),
            "sc_add_norm_bwd": ([P] * 6 + [I64, I32, F, I32, P], I32),
            "sc_linear_fwd": ([P] * 8 + [I64, I32, I32, I32, I32, I32, P], I32),
            "sc_linear_bwd": ([P] * 7 + [I64, I32, I32, I32, I32, P], I32),
            "sc_rows_check": ([P], I32),
            "sc_grad_clip": ([P, I64, F, P, P], I32),
            "sc_set_allocator": ([P, P, P], I32),
            "sc_status_str": ([I32], ctypes.c_char_p),
            "sc_last_error": ([], ctypes.c_char_p),
            "sc_launch_count": ([], I64),
            "sc_profile_enable": ([I32], None),
            "sc_profile_only": ([ctypes.c_char_p], None),
            "sc_profile_collect": ([], I32),
            "sc_profile_reset": ([], None),
            "sc_profile_get": ([I32, P, P, P], I32),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def exported_symbols() -> list:
    return [n for n in ("sc_hash_build", "sc_hash_query", "sc_hash_info", "sc_hash_check", "sc_hash_destroy",
                        "sc_hash_build_conv_out", "sc_hash_coords", "sc_kmap_build_conv",
                        "sc_kmap_build", "sc_kmap_info", "sc_kmap_check", "sc_kmap_export", "sc_kmap_view",
                        "sc_kmap_destroy",
                        "sc_subm_conv_fwd", "sc_subm_conv_tune", "sc_subm_conv_fwd_noalloc",
                        "sc_subm_conv_bwd_data", "sc_subm_conv_bwd_weight", "sc_qk_norm_rope_fwd",
                        "sc_qk_norm_rope_bwd", "sc_attn_fwd", "sc_attn_bwd", "sc_attn_check", "sc_add_norm_fwd",
                        "sc_add_norm_bwd", "sc_linear_fwd", "sc_linear_bwd", "sc_rows_check", "sc_grad_clip",
                        "sc_set_allocator", "sc_status_str", "sc_last_error",
                        "sc_launch_count", "sc_profile_enable", "sc_profile_only", "sc_profile_collect",
                        "sc_profile_reset",
                        "sc_profile_get")]


def _check(st: int, what: str):
    if st != 0:
        raise ScError(st, f"{what}: {lib().sc_last_error().decode()}")


def _stream(stream=None):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the current stream's handle, without a Stream object around it
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


class Hash:
    """Handle of a coordinate hash table built by sc_hash_build."""

    def __init__(self, handle, n: int, capacity: int, device):
        self._h = handle
        self.n = n
        self.capacity = capacity
        self.device = device

    def query(self, coords: torch.Tensor, stream=None) -> torch.Tensor:
        """Row id of each (batch, x, y, z) query, -1 when absent (sc_hash_query)."""
        q = _dev(coords, "coords")
        rows = torch.empty(q.shape[0], dtype=torch.int32, device=q.device)
        _check(lib().sc_hash_query(self._h, _ptr(q), q.shape[0], _ptr(rows), _stream(stream)), "sc_hash_query")
        return rows

    def check(self, stream=None):
        _check(lib().sc_hash_check(self._h, _stream(stream)), "sc_hash_check")

    def coords(self, stream=None) -> torch.Tensor:
        """int32 [n, 4] (batch, x, y, z) of every row (sc_hash_coords)."""
        out = torch.empty((self.n, 4), dtype=torch.int32, device=self.device)
        _check(lib().sc_hash_coords(self._h, _ptr(out), _stream(stream)), "sc_hash_coords")
        return out

    def destroy(self, stream=None):
        if self._h:
            lib().sc_hash_destroy(self._h, _stream(stream))
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class KernelMap:
    """Handle of a kernel map built by sc_kmap_build."""

    def __init__(self, handle, n: int, ndim: int, K: int, dims, device, n_in: int | None = None,
                 stride: int = 1):
        self._h = handle
        self.n = n
        self.n_in = n if n_in is None else n_in
        self.stride = stride
        self.identity = n_in is None  # submanifold: the centre list is the identity
        self.ndim = ndim
        self.K = K
        self.volume = K ** ndim
        self.dims = tuple(dims)
        self.device = device

    def map_size(self, stream=None) -> int:
        """|M|, centre tuples included (sc_kmap_info)."""
        m = ctypes.c_int64(0)
        _check(lib().sc_kmap_info(self._h, None, None, ctypes.byref(m), _stream(stream)), "sc_kmap_info")
        return m.value

    def check(self, stream=None):
        _check(lib().sc_kmap_check(self._h, _stream(stream)), "sc_kmap_check")

    def nbr(self, stream=None) -> torch.Tensor:
        out = torch.empty((self.n, self.volume), dtype=torch.int32, device=self.device)
        _check(lib().sc_kmap_export(self._h, _ptr(out), None, None, None, _stream(stream)), "sc_kmap_export")
        return out

    def offsets(self, stream=None) -> torch.Tensor:
        out = torch.empty(self.volume + 1, dtype=torch.int64, device=self.device)
        _check(lib().sc_kmap_export(self._h, None, _ptr(out), None, None, _stream(stream)), "sc_kmap_export")
        return out

    def lists(self, stream=None):
        """(offs [V+1], in_rows [L], out_rows [L]): the per-offset lists (a
        submanifold map's centre segment is empty, its tuples implicit)."""
        offs = self.offsets(stream)
        L = self.map_size(stream) - (self.n if self.identity else 0)
        i = torch.empty(max(L, 0), dtype=torch.int32, device=self.device)
        o = torch.empty(max(L, 0), dtype=torch.int32, device=self.device)
        _check(lib().sc_kmap_export(self._h, None, None, _ptr(i) if L else None, _ptr(o) if L else None,
                                    _stream(stream)), "sc_kmap_export")
        return offs, i, o

    def view(self):
        """Borrowed, zero-copy device tensors of the products (sc_kmap_view):
        {"nbr": int32 [n, V], "offs": int64 [V+1], "in": int32 [L], "out":
        int32 [L], "map_size": |M|}.  They alias memory the handle owns: valid
        while this map is alive (each tensor keeps a reference to it), and not
        to be written."""
        nbr, offs, i, o = (ctypes.c_void_p() for _ in range(4))
        ms = ctypes.c_int64()
        _check(lib().sc_kmap_view(self._h, ctypes.byref(nbr), ctypes.byref(offs), ctypes.byref(i), ctypes.byref(o),
                                  ctypes.byref(ms)), "sc_kmap_view")
        L = ms.value - (self.n if self.identity else 0)

        def wrap(ptr, shape, typestr):
            n_el = 1
            for d in shape:
                n_el *= d
            if n_el == 0 or not ptr.value:
                return torch.empty(shape, dtype=torch.int64 if typestr == "<i8" else torch.int32, device=self.device)
            owner = self

            class _Borrowed:
                # torch takes only writable interfaces; the memory is read-only by contract
                __cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr, "data": (ptr.value, False),
                                            "version": 3, "strides": None}
                keep = owner  # the map outlives the tensor's view of it
            return torch.as_tensor(_Borrowed(), device=self.device)

        return {"nbr": wrap(nbr, (self.n, self.volume), "<i4"), "offs": wrap(offs, (self.volume + 1,), "<i8"),
                "in": wrap(i, (max(L, 0),), "<i4"), "out": wrap(o, (max(L, 0),), "<i4"), "map_size": ms.value}

    def destroy(self, stream=None):
        if self._h:
            lib().sc_kmap_destroy(self._h, _stream(stream))
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def sc_hash_build(coords: torch.Tensor, stream=None, allocator=None) -> Hash:
    """Hash table over int32 coords [N, 4] = (batch, x, y, z) on a CUDA device."""
    c = _dev(coords, "coords")
    if c.dtype != torch.int32 or c.dim() != 2 or c.shape[1] != 4:
        raise ValueError("coords must be int32 [N, 4]")
    h = ctypes.c_void_p()
    _check(lib().sc_hash_build(_ptr(c), c.shape[0], _alloc_arg(allocator), _stream(stream), ctypes.byref(h)),
           "sc_hash_build")
    n = ctypes.c_int64()
    cap = ctypes.c_int64()
    lib().sc_hash_info(h, ctypes.byref(n), ctypes.byref(cap))
    return Hash(h, n.value, cap.value, c.device)


def sc_kmap_build(h: Hash, ndim: int, K: int, dims, sync: bool = True, order: bool | None = None,
                  sort: bool | None = None, half: bool = False, split: bool = False, stream=None,
                  allocator=None, tile_table: bool = False) -> KernelMap:
    """Kernel map of a K^ndim submanifold convolution over the hashed points.

    order: True / False forces the locality order on / off; None leaves the
    library's default (on for n >= 262144).  sort: the same for the
    signature sort of the convolution's rows (default on for n >= 262144 when
    K^ndim <= 128).  half: build it by the half probe (mirror symmetry); the
    map is the same.  split: also compute the row orders of column splitting
    (K^ndim <= 32), which the "split" layer variant uses.  tile_table: also
    build the fused layer's tile-transposed index table (K^ndim <= 128),
    which pays when the map serves several layers."""
    d = (ctypes.c_int32 * 3)(*(list(dims) + [1] * (3 - len(dims))))
    m = ctypes.c_void_p()
    flags = 0 if sync else SC_KMAP_NO_SYNC
    if half:
        flags |= SC_KMAP_HALF
    if split:
        flags |= SC_KMAP_SPLIT
    if tile_table:
        flags |= SC_KMAP_TILE_TABLE
    if order is True:
        flags |= SC_KMAP_ORDER
    elif order is False:
        flags |= SC_KMAP_NO_ORDER
    if sort is True:
        flags |= SC_KMAP_SORT
    elif sort is False:
        flags |= SC_KMAP_NO_SORT
    _check(lib().sc_kmap_build(h._h, ndim, K, d, flags, _alloc_arg(allocator), _stream(stream), ctypes.byref(m)),
           "sc_kmap_build")
    return KernelMap(m, h.n, ndim, K, list(d), h.device)


def sc_hash_build_conv_out(h: Hash, ndim: int, K: int, stride: int, dims, stream=None, allocator=None) -> Hash:
    """Output set of a regular (stride 1: dilating) or strided layer over the
    points of `h`: every o with an input at stride * o + d (synchronises)."""
    d = (ctypes.c_int32 * 3)(*(list(dims) + [1] * (3 - len(dims))))
    o = ctypes.c_void_p()
    _check(lib().sc_hash_build_conv_out(h._h, ndim, K, stride, d, _alloc_arg(allocator), _stream(stream),
                                        ctypes.byref(o)),
           "sc_hash_build_conv_out")
    n = ctypes.c_int64()
    cap = ctypes.c_int64()
    lib().sc_hash_info(o, ctypes.byref(n), ctypes.byref(cap))
    return Hash(o, n.value, cap.value, h.device)


def sc_kmap_build_conv(h_in: Hash, h_out: Hash, ndim: int, K: int, stride: int, dims, sync: bool = True,
                       order: bool | None = None, sort: bool | None = None, transpose: bool = False, stream=None,
                       allocator=None, tile_table: bool = False) -> KernelMap:
    """Kernel map of a regular / strided layer: rows = the points of `h_out`,
    neighbours = rows of `h_in` at stride * o + d.  transpose: the transposed
    map (rows = the points of `h_in`, neighbours = the outputs whose windows
    hold them, at the mirrored offset), which sc_subm_conv_bwd_data takes.
    tile_table: as for sc_kmap_build."""
    d = (ctypes.c_int32 * 3)(*(list(dims) + [1] * (3 - len(dims))))
    m = ctypes.c_void_p()
    flags = 0 if sync else SC_KMAP_NO_SYNC
    if transpose:
        flags |= SC_KMAP_TRANSPOSE
    if tile_table:
        flags |= SC_KMAP_TILE_TABLE
    if order is True:
        flags |= SC_KMAP_ORDER
    elif order is False:
        flags |= SC_KMAP_NO_ORDER
    if sort is True:
        flags |= SC_KMAP_SORT
    elif sort is False:
        flags |= SC_KMAP_NO_SORT
    _check(lib().sc_kmap_build_conv(h_in._h, h_out._h, ndim, K, stride, d, flags, _alloc_arg(allocator),
                                    _stream(stream), ctypes.byref(m)),
           "sc_kmap_build_conv")
    if transpose:
        return KernelMap(m, h_in.n, ndim, K, list(d), h_in.device, n_in=h_out.n, stride=stride)
    return KernelMap(m, h_out.n, ndim, K, list(d), h_in.device, n_in=h_in.n, stride=stride)


def _conv_args(kmap, feats, W, out):
    f = _dev(feats, "feats")
    w = _dev(W, "W")
    if f.dtype not in _DTYPES or w.dtype != f.dtype:
        raise ValueError("feats and W must share one dtype: float32, float16 or bfloat16")
    if (w.dim() != 3 or w.shape[0] != kmap.volume or f.dim() != 2 or f.shape[1] != w.shape[1]
            or f.shape[0] != kmap.n_in):
        raise ValueError("shapes must be feats [N_in, C_in], W [K^ndim, C_in, C_out]")
    c_out = w.shape[2]
    if out is None:
        out = torch.empty((kmap.n, c_out), dtype=f.dtype, device=f.device)
    else:
        _dev(out, "out")
        if out.dtype != f.dtype or tuple(out.shape) != (kmap.n, c_out):
            raise ValueError("out must be [N, C_out] of the feats dtype")
    return f, w, out, f.shape[1], c_out, _DTYPES[f.dtype]


def sc_subm_conv_fwd(kmap: KernelMap, feats: torch.Tensor, W: torch.Tensor, out: torch.Tensor | None = None,
                     relu: bool = False, variant: str | None = None, stream=None) -> torch.Tensor:
    """out[q] = act(sum over map tuples (p, q, d) of feats[p] @ W[d]).  feats has
    the map's input rows (kmap.n_in), out its rows (kmap.n): the same for a
    submanifold map, the output set's for a regular / strided one."""
    f, w, out, c_in, c_out, dt = _conv_args(kmap, feats, W, out)
    flags = (SC_RELU if relu else 0) | (VARIANTS[variant] if variant else 0)
    _check(lib().sc_subm_conv_fwd(kmap._h, _ptr(f), _ptr(w), _ptr(out), c_in, c_out, dt, flags,
                                  _stream(stream)), "sc_subm_conv_fwd")
    return out


def sc_subm_conv_bwd_data(kmap: KernelMap, gout: torch.Tensor, W: torch.Tensor, gin: torch.Tensor | None = None,
                          variant: str | None = None, stream=None) -> torch.Tensor:
    """Gradient of a (ReLU-free) layer's loss with respect to its input
    features: gin[p] = sum over map tuples (p, q, d) of gout[q] @ W[d]^T.
    kmap: the layer's submanifold map, or the transposed map of a regular /
    strided layer (sc_kmap_build_conv(..., transpose=True)): gout has
    kmap.n_in rows (the layer's outputs), gin kmap.n (its inputs)."""
    g = _dev(gout, "gout")
    w = _dev(W, "W")
    if g.dtype not in _DTYPES or w.dtype != g.dtype:
        raise ValueError("gout and W must share one dtype: float32, float16 or bfloat16")
    if (w.dim() != 3 or w.shape[0] != kmap.volume or g.dim() != 2 or g.shape[1] != w.shape[2]
            or g.shape[0] != kmap.n_in):
        raise ValueError("shapes must be gout [N_out, C_out], W [K^ndim, C_in, C_out] (a submanifold map: "
                         "N_out = N; a transposed map: N_out = the layer's output count)")
    c_in, c_out = w.shape[1], w.shape[2]
    if gin is None:
        gin = torch.empty((kmap.n, c_in), dtype=g.dtype, device=g.device)
    elif gin.dtype != g.dtype or tuple(gin.shape) != (kmap.n, c_in):
        raise ValueError("gin must be [N, C_in] of the gout dtype")
    _check(lib().sc_subm_conv_bwd_data(kmap._h, _ptr(g), _ptr(w), _ptr(_dev(gin, "gin")), c_in, c_out,
                                       _DTYPES[g.dtype], VARIANTS[variant] if variant else 0, _stream(stream)),
           "sc_subm_conv_bwd_data")
    return gin


def sc_subm_conv_bwd_weight(kmap: KernelMap, feats: torch.Tensor, gout: torch.Tensor, dW: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Gradient with respect to the weights: dW[d] = sum over map tuples
    (p, q, d) of feats[p]^T gout[q]."""
    f = _dev(feats, "feats")
    g = _dev(gout, "gout")
    if f.dtype not in _DTYPES or g.dtype != f.dtype:
        raise ValueError("feats and gout must share one dtype: float32, float16 or bfloat16")
    if f.dim() != 2 or g.dim() != 2 or f.shape[0] != kmap.n_in or g.shape[0] != kmap.n:
        raise ValueError("shapes must be feats [N_in, C_in], gout [N, C_out]")
    c_in, c_out = f.shape[1], g.shape[1]
    if dW is None:
        dW = torch.empty((kmap.volume, c_in, c_out), dtype=f.dtype, device=f.device)
    elif dW.dtype != f.dtype or tuple(dW.shape) != (kmap.volume, c_in, c_out):
        raise ValueError("dW must be [K^ndim, C_in, C_out] of the feats dtype")
    _check(lib().sc_subm_conv_bwd_weight(kmap._h, _ptr(f), _ptr(g), _ptr(_dev(dW, "dW")), c_in, c_out,
                                         _DTYPES[f.dtype], 0, _stream(stream)), "sc_subm_conv_bwd_weight")
    return dW


def sc_subm_conv_tune(kmap: KernelMap, feats: torch.Tensor, W: torch.Tensor, out: torch.Tensor | None = None,
                      relu: bool = False, reps: int = 3, stream=None) -> str:
    """Times the variants on this map, caches the fastest, returns its name."""
    f, w, out, c_in, c_out, dt = _conv_args(kmap, feats, W, out)
    chosen = ctypes.c_uint(0)
    _check(lib().sc_subm_conv_tune(kmap._h, _ptr(f), _ptr(w), _ptr(out), c_in, c_out, dt,
                                   SC_RELU if relu else 0, reps, _stream(stream), ctypes.byref(chosen)),
           "sc_subm_conv_tune")
    return VARIANT_NAMES[chosen.value]


class _Heads(ctypes.Structure):
    """sc_heads / sc_heads_out: a strided view of rows [tokens, heads, head_dim]."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


# A call on few rows is bound by the host, so these wrappers read a tensor's
# properties once and pass plain integers (argtypes converts them).
def _heads(t, name: str, dtype=None, device=None, shape=None):
    """The view struct of a CUDA tensor [tokens, heads, head_dim] whose last
    dimension is contiguous (the other strides are free), by reference."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    stride = t.stride()
    if len(stride) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if dtype is not None and (t.dtype is not dtype or t.get_device() != device):
        raise ValueError(f"{name} must have the dtype and device of the other rows")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if stride[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return ctypes.byref(_Heads(t.data_ptr(), stride[0], stride[1]))


def _rows_out(t, name: str, like, shape, dtype, device):
    """(t, its view): where to write rows of `shape`, made here if t is None."""
    if t is not None:
        return t, _heads(t, name, dtype, device, shape)
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    return t, ctypes.byref(_Heads(t.data_ptr(), shape[1] * shape[2], shape[2]))


def _raw_stream(stream) -> int:
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _f32(t, name: str, n: int, device: int):
    """The address of a float32 [n] vector, or None."""
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype is not torch.float32
            or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 [{n}] tensor on the rows' device")
    return t.data_ptr()


def _positions(pos, freq, tokens, device):
    """(address, token stride, axes, frequencies' address, rot_dim)."""
    if freq is None:
        return None, 0, 1, None, 0
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise ValueError("freq must be a float32 vector")
    half = freq.shape[0]
    fp = _f32(freq, "freq", half, device)
    if not isinstance(pos, torch.Tensor) or pos.get_device() != device or pos.dtype is not torch.int32:
        raise ValueError("pos must be int32 on the rows' device")
    st, axes = pos.stride(), 1
    if len(st) not in (1, 2) or pos.shape[0] != tokens:
        raise ValueError("pos must be [tokens] or [tokens, axes]")
    if len(st) == 2:
        axes = pos.shape[1]
        if axes > 1 and st[1] != 1:
            raise ValueError("pos: the axes must be contiguous")
    return (pos.data_ptr() if half else None), st[0], axes, fp, 2 * half


def sc_qk_norm_rope_fwd(q, k, pos=None, freq=None, wq=None, wk=None, eps: float = 1e-6, interleaved: bool = False,
                        amp: float = 1.0, out_q=None, out_k=None, stream=None):
    """(q', k'): rows q [tokens, heads_q, head_dim] and k [tokens, heads_k,
    head_dim] (one of them may be None) normed per head by wq, wk (float32
    [head_dim], or None) and rotated by pos (int32 [tokens] or [tokens, axes])
    times freq (float32 [rot_dim / 2]; rope_frequencies makes them).  out_q,
    out_k: where to write (q and k themselves are allowed)."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("pass q, k or both")
    hq = hk = oq = ok = sq = sk = None
    nq = nk = 0
    if q is not None:
        hq = _heads(q, "q")
        sq = q.shape
        nq = sq[1]
    dtype, device = first.dtype, first.get_device()
    if k is not None:
        hk = _heads(k, "k", dtype, device)
        sk = k.shape
        nk = sk[1]
    tokens, _, d = sq or sk
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("rows must be float32, float16 or bfloat16")
    pp, stride, axes, fp, rot = _positions(pos, freq, tokens, device)
    wqp, wkp = _f32(wq, "wq", d, device), _f32(wk, "wk", d, device)
    if (wq is None) != (wk is None) and nq and nk:
        raise ValueError("pass both norm weights, or neither")
    if sq and sk and (sk[0] != tokens or sk[2] != d):
        raise ValueError("q and k must have the same tokens and head_dim")
    if sq:
        out_q, oq = _rows_out(out_q, "out_q", q, sq, dtype, device)
    if sk:
        out_k, ok = _rows_out(out_k, "out_k", k, sk, dtype, device)
    st = (_lib or lib()).sc_qk_norm_rope_fwd(hq, hk, oq, ok, wqp, wkp, pp, stride, axes, fp, tokens, nq, nk, d, rot,
                                             eps, amp, code, SC_ROPE_INTERLEAVED if interleaved else 0,
                                             _raw_stream(stream))
    if st:
        _check(st, "sc_qk_norm_rope_fwd")
    return out_q, out_k


def sc_qk_norm_rope_bwd(gout_q, gout_k, q=None, k=None, pos=None, freq=None, wq=None, wk=None, eps: float = 1e-6,
                        interleaved: bool = False, amp: float = 1.0, gin_q=None, gin_k=None, stream=None):
    """(gq, gk, gwq, gwk): the gradients of sc_qk_norm_rope_fwd's inputs and
    weights from those of its outputs.  q, k: the forward's inputs (read only
    with a norm); gwq, gwk are float32, None without a norm."""
    first = gout_q if gout_q is not None else gout_k
    if first is None:
        raise ValueError("pass gout_q, gout_k or both")
    gq = gk = hq = hk = iq = ik = sq = sk = gwq = gwk = None
    nq = nk = 0
    if gout_q is not None:
        gq = _heads(gout_q, "gout_q")
        sq = gout_q.shape
        nq = sq[1]
    dtype, device = first.dtype, first.get_device()
    if gout_k is not None:
        gk = _heads(gout_k, "gout_k", dtype, device)
        sk = gout_k.shape
        nk = sk[1]
    tokens, _, d = sq or sk
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("rows must be float32, float16 or bfloat16")
    pp, stride, axes, fp, rot = _positions(pos, freq, tokens, device)
    wqp, wkp = _f32(wq, "wq", d, device), _f32(wk, "wk", d, device)
    if (wq is None) != (wk is None) and nq and nk:
        raise ValueError("pass both norm weights, or neither")
    if sq and sk and (sk[0] != tokens or sk[2] != d):
        raise ValueError("gout_q and gout_k must have the same tokens and head_dim")
    norm = wq is not None or wk is not None
    if sq:
        gin_q, iq = _rows_out(gin_q, "gin_q", gout_q, sq, dtype, device)
        if norm:
            hq = _heads(q, "q", dtype, device, sq)
            if nq:
                gwq = torch.empty_like(wq)
    if sk:
        gin_k, ik = _rows_out(gin_k, "gin_k", gout_k, sk, dtype, device)
        if norm:
            hk = _heads(k, "k", dtype, device, sk)
            if nk:
                gwk = torch.empty_like(wk)
    st = (_lib or lib()).sc_qk_norm_rope_bwd(gq, gk, hq, hk, iq, ik, gwq.data_ptr() if gwq is not None else None,
                                             gwk.data_ptr() if gwk is not None else None, wqp, wkp, pp, stride, axes,
                                             fp, tokens, nq, nk, d, rot, eps, amp, code,
                                             SC_ROPE_INTERLEAVED if interleaved else 0, _raw_stream(stream))
    if st:
        _check(st, "sc_qk_norm_rope_bwd")
    return gin_q, gin_k, gwq, gwk


def rope_frequencies(rot_dim: int, axes: int = 1, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original: int = 8192, slow: float = 1.0, fast: float = 32.0, device=None):
    """(freq, amp) for sc_qk_norm_rope_*: float32 [rot_dim / 2] radians a
    position, pair i of an axis's n pairs turning by base^(-i/n), and the factor
    of the rotated values.

    scaling, for contexts `factor` times the `original` length:
      "none"    as they are
      "linear"  every frequency divided by factor
      "base"    the base raised so that the slowest pair slows by factor
      "parts"   pairs that make under `slow` turns over the original length are
                divided by factor, those over `fast` kept, a ramp between, and
                amp = 1 + 0.1 ln(factor)"""
    if axes < 1 or rot_dim < 2 or rot_dim % (2 * axes):
        raise ValueError("rot_dim must be a positive multiple of 2 * axes")
    if not factor >= 1.0 or not base > 1.0:
        raise ValueError("factor must be at least 1 and base above 1")
    n = rot_dim // 2 // axes
    i = torch.arange(n, dtype=torch.float64)
    amp = 1.0
    if scaling == "base" and n > 1:
        base = base * factor ** (n / (n - 1))
    freq = base ** (-i / n)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        if not fast > slow:
            raise ValueError("fast must be above slow")
        turns = original * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
        amp = 1.0 + 0.1 * math.log(factor)
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.float().repeat(axes).to(device), amp


def _offsets(off, name: str, device: int, n: int | None = None):
    """The address of an int32 vector (of n values)."""
    if (not isinstance(off, torch.Tensor) or off.get_device() != device or off.dtype is not torch.int32
            or off.dim() != 1 or not off.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 vector on the rows' device")
    if n is not None and off.shape[0] != n:
        raise ValueError(f"{name} must hold {n} values")
    return off.data_ptr()


def _attn_common(q, k, v, q_off, k_off, scale):
    hq = _heads(q, "q")
    dtype, device, sq = q.dtype, q.get_device(), q.shape
    hk = _heads(k, "k", dtype, device)
    sk = k.shape
    hv = _heads(v, "v", dtype, device, sk)
    if sk[2] != sq[2]:
        raise ValueError("q, k and v must have one head_dim")
    qp = kp = _offsets(q_off, "q_off", device)
    n = q_off.shape[0] - 1
    if n < 0:
        raise ValueError("q_off must hold one more offset than there are sequences")
    if k_off is not None:
        kp = _offsets(k_off, "k_off", device, n + 1)
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("rows must be float16 or bfloat16")
    if scale is None:
        scale = max(sq[2], 1) ** -0.5
    return hq, hk, hv, dtype, device, sq, sk, qp, kp, n, code, scale


def sc_attn_fwd(q, k, v, q_off, k_off=None, k_len=None, causal: bool = False, scale: float | None = None,
                return_lse: bool = False, out=None, stream=None):
    """out [t_q, heads_q, head_dim] = softmax(scale q k^T) v over packed
    sequences: q [t_q, heads_q, head_dim], k and v [t_k, heads_kv, head_dim]
    (any token and head strides), sequence s holding query rows q_off[s] ..
    q_off[s+1] and key rows k_off[s] .. k_off[s+1] (default: q_off), or k_len[s]
    rows from k_off[s] on.  causal: query i sees keys 0 .. i + keys - queries.
    scale: default head_dim^-0.5.  return_lse: (out, lse float32 [t_q, heads_q])."""
    hq, hk, hv, dtype, device, sq, sk, qp, kp, n, code, scale = _attn_common(q, k, v, q_off, k_off, scale)
    lp = None if k_len is None else _offsets(k_len, "k_len", device, n)
    out, ho = _rows_out(out, "out", q, sq, dtype, device)
    lse = torch.empty(sq[:2], dtype=torch.float32, device=q.device) if return_lse else None
    st = (_lib or lib()).sc_attn_fwd(hq, hk, hv, ho, lse.data_ptr() if return_lse else None, qp, kp, lp, n, sq[0],
                                     sk[0], sq[1], sk[1], sq[2], scale, code, SC_ATTN_CAUSAL if causal else 0,
                                     _raw_stream(stream))
    if st:
        _check(st, "sc_attn_fwd")
    return (out, lse) if return_lse else out


def sc_attn_bwd(gout, q, k, v, out, lse, q_off, k_off=None, causal: bool = False, scale: float | None = None,
                gq=None, gk=None, gv=None, stream=None):
    """(gq, gk, gv): gradients of sc_attn_fwd's inputs from gout, that of its
    output, with the forward's out and lse.  gq, gk, gv: where to write."""
    hq, hk, hv, dtype, device, sq, sk, qp, kp, n, code, scale = _attn_common(q, k, v, q_off, k_off, scale)
    hg, ho = _heads(gout, "gout", dtype, device, sq), _heads(out, "out", dtype, device, sq)
    if (not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32 or lse.get_device() != device
            or lse.shape != sq[:2] or not lse.is_contiguous()):
        raise ValueError("lse must be the forward's contiguous float32 [t_q, heads_q]")
    gq, oq = _rows_out(gq, "gq", q, sq, dtype, device)
    gk, ok = _rows_out(gk, "gk", k, sk, dtype, device)
    gv, ov = _rows_out(gv, "gv", v, sk, dtype, device)
    st = (_lib or lib()).sc_attn_bwd(hg, hq, hk, hv, ho, lse.data_ptr(), oq, ok, ov, qp, kp, n, sq[0], sk[0], sq[1],
                                     sk[1], sq[2], scale, code, SC_ATTN_CAUSAL if causal else 0, _raw_stream(stream))
    if st:
        _check(st, "sc_attn_bwd")
    return gq, gk, gv


def sc_attn_check(stream=None):
    """Synchronises and raises what the attention calls on the current device
    latched since the last check (offsets that leave the rows)."""
    _check(lib().sc_attn_check(_stream(stream)), "sc_attn_check")


class _Rows(ctypes.Structure):
    """sc_rows / sc_rows_out: a strided view of rows [rows, channels]."""
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


def _rows(t, name: str, dtype=None, device=None, shape=None):
    """The view struct of a CUDA tensor [rows, channels] whose channels are
    contiguous (the rows' stride is free), by reference."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    stride = t.stride()
    if len(stride) != 2:
        raise ValueError(f"{name} must be [rows, channels]")
    if dtype is not None and (t.dtype is not dtype or t.get_device() != device):
        raise ValueError(f"{name} must be {dtype} on the other rows' device")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if stride[1] != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    return ctypes.byref(_Rows(t.data_ptr(), stride[0]))


def _new_rows(t, name: str, shape, dtype, like):
    """(t, its view): where to write rows of `shape`, made here if t is None."""
    if t is not None:
        return t, _rows(t, name, dtype, like.get_device(), shape)
    t = torch.empty(shape, dtype=dtype, device=like.device)
    return t, ctypes.byref(_Rows(t.data_ptr(), shape[1]))


def _same_device(t, name: str) -> int:
    """The tensor's device, which has to be the current one: its stream is the call's."""
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} lies on device {device}, which is not the current one")
    return device


def sc_add_norm_fwd(x, w=None, res=None, eps: float = 1e-6, e4m3: bool = False, out=None, sum=None, stream=None):
    """The norm of rows after the residual's addition: h = x + res,
    y = w * h / sqrt(mean(h^2) + eps), for x and res [rows, channels] (any row
    stride) and w float32 [channels].

    Returns y, or (y, h) with res.  e4m3: y in 8 bits with a scale for each row
    (float32 [rows]; y is about out * scale; infinity: a row without values), as
    (out, scale) or (out, scale, h); w may then be None: h as it is.  out, sum: where to write y and h; sum
    may be x or res themselves, and so may out unless it has 8 bits."""
    hx = _rows(x, "x")
    shape, dtype, device = x.shape, x.dtype, _same_device(x, "x")
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("rows must be float32, float16 or bfloat16")
    hr = hs = scale = None
    if res is not None:
        hr = _rows(res, "res", dtype, device, shape)
        sum, hs = _new_rows(sum, "sum", shape, dtype, x)
    elif sum is not None:
        raise ValueError("sum is the sum with res: pass res too")
    wp = _f32(w, "w", shape[1], device)
    out, ho = _new_rows(out, "out", shape, _E4M3 if e4m3 else dtype, x)
    if e4m3:
        scale = torch.empty(shape[0], dtype=torch.float32, device=x.device)
    st = (_lib or lib()).sc_add_norm_fwd(hx, hr, hs, ho, scale.data_ptr() if e4m3 else None, wp, shape[0], shape[1],
                                         eps, code, _E4M3_CODE if e4m3 else code, _raw_stream(stream))
    if st:
        _check(st, "sc_add_norm_fwd")
    if e4m3:
        return (out, scale) if res is None else (out, scale, sum)
    return out if res is None else (out, sum)


def sc_add_norm_bwd(gout, h, w, gsum=None, eps: float = 1e-6, need_gw: bool = True, gin=None, stream=None):
    """(gin, gw): the gradients of sc_add_norm_fwd's rows (x and res alike) and
    weights (float32; None without need_gw), from gout, the gradient of y, and
    gsum, the gradient that reaches h past the norm.  h: the forward's sum, or
    its x without a residual.  gin: where to write, which may be gout, gsum or h."""
    hh = _rows(h, "h")
    shape, dtype, device = h.shape, h.dtype, _same_device(h, "h")
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("rows must be float32, float16 or bfloat16")
    hg = _rows(gout, "gout", dtype, device, shape)
    hs = None if gsum is None else _rows(gsum, "gsum", dtype, device, shape)
    if w is None:
        raise ValueError("w must be the forward's weights")
    wp = _f32(w, "w", shape[1], device)
    gin, hi = _new_rows(gin, "gin", shape, dtype, h)
    gw = torch.empty_like(w) if need_gw else None
    st = (_lib or lib()).sc_add_norm_bwd(hg, hh, hs, hi, gw.data_ptr() if need_gw else None, wp, shape[0], shape[1],
                                         eps, code, _raw_stream(stream))
    if st:
        _check(st, "sc_add_norm_bwd")
    return gin, gw


def _act_code(act) -> int:
    code = SC_ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(SC_ACT)}")
    return code


def _weights(W, dtype, device, shape):
    if (not isinstance(W, torch.Tensor) or W.get_device() != device or W.dtype is not dtype or W.dim() != 2
            or not W.is_contiguous() or (shape is not None and W.shape != shape)):
        raise ValueError("W must be a contiguous matrix of the rows' dtype, width and device")
    return W.data_ptr()


def sc_linear_fwd(x, W, bias=None, act: str = "none", res=None, scale_x=None, scale_w=None, dtype=None,
                  return_pre: bool = False, out=None, stream=None):
    """out = act(x W + bias) + res for x [rows, c_in] (any row stride), W
    [c_in, c_out] and bias float32 [c_out]; act: "none", "relu", "gelu" or
    "silu".  return_pre: (out, pre), pre being x W + bias for the backward pass.

    8 bits: x float8_e4m3fn with scale_x float32 [rows], as sc_add_norm_fwd(...,
    e4m3=True) gives them, and W float8_e4m3fn [c_out, c_in] with scale_w
    [c_out], which the same call without weights makes once of W's transpose.
    The outputs are then of `dtype` (default: res's, else bfloat16)."""
    hx = _rows(x, "x")
    (rows, c_in), kind, device = x.shape, x.dtype, _same_device(x, "x")
    code, e4m3 = _act_code(act), kind is _E4M3
    if e4m3:
        wp = _weights(W, kind, device, None)
        c_out = W.shape[0]
        if W.shape[1] != c_in:
            raise ValueError("W of 8 bits must be [c_out, c_in]")
        if scale_x is None or scale_w is None:
            raise ValueError("8 bits need scale_x and scale_w")
        xp, sp = _f32(scale_x, "scale_x", rows, device), _f32(scale_w, "scale_w", c_out, device)
        if dtype is None:
            dtype = torch.bfloat16 if res is None else res.dtype
        in_code = _E4M3_CODE
    else:
        if scale_x is not None or scale_w is not None:
            raise ValueError("scales are for 8 bits only")
        wp = _weights(W, kind, device, None)
        c_out = W.shape[1]
        if W.shape[0] != c_in:
            raise ValueError("W must be [c_in, c_out]")
        xp = sp = None
        if dtype is None:
            dtype = kind
        in_code = _DTYPES.get(kind)
    out_code = _DTYPES.get(dtype)
    if in_code is None or out_code is None:
        raise ValueError("rows must be float16, bfloat16 or float8_e4m3fn")
    shape = torch.Size((rows, c_out))
    bp = _f32(bias, "bias", c_out, device)
    hr = None if res is None else _rows(res, "res", dtype, device, shape)
    out, ho = _new_rows(out, "out", shape, dtype, x)
    pre, hp = _new_rows(None, "pre", shape, dtype, x) if return_pre else (None, None)
    st = (_lib or lib()).sc_linear_fwd(hx, wp, xp, sp, bp, hr, ho, hp, rows, c_in, c_out, code, in_code, out_code,
                                       _raw_stream(stream))
    if st:
        _check(st, "sc_linear_fwd")
    return (out, pre) if return_pre else out


def sc_linear_bwd(gout, x, W, pre=None, act: str = "none", bias: bool = False, need_gin: bool = True,
                  need_gW: bool = True, gin=None, stream=None):
    """(gin, gW, gbias): the gradients of sc_linear_fwd's x, W and bias (float32)
    from gout, that of its output (and of res), with the forward's x, W and, with
    an activation, pre.  None where not needed (bias: whether there is one).
    gin: where to write the rows'."""
    hg = _rows(gout, "gout")
    (rows, c_out), dtype, device = gout.shape, gout.dtype, _same_device(gout, "gout")
    code, kind = _act_code(act), _DTYPES.get(dtype)
    if kind is None:
        raise ValueError("rows must be float16 or bfloat16")
    hx = _rows(x, "x", dtype, device)
    c_in = x.shape[1]
    if x.shape[0] != rows:
        raise ValueError("x and gout must have the same rows")
    wp = _weights(W, dtype, device, torch.Size((c_in, c_out)))
    hp = None
    if code:
        hp = _rows(pre, "pre", dtype, device, gout.shape)
    hi = gw = gb = None
    if need_gin:
        gin, hi = _new_rows(gin, "gin", x.shape, dtype, gout)
    elif gin is not None:
        raise ValueError("gin is given but not needed")
    if need_gW:
        gw = torch.empty_like(W)
    if bias:
        gb = torch.empty(c_out, dtype=torch.float32, device=gout.device)
    st = (_lib or lib()).sc_linear_bwd(hg, hx, hp, wp, hi, gw.data_ptr() if need_gW else None,
                                       gb.data_ptr() if bias else None, rows, c_in, c_out, code, kind,
                                       _raw_stream(stream))
    if st:
        _check(st, "sc_linear_bwd")
    return gin, gw, gb


def sc_rows_check(stream=None):
    """Synchronises and raises what the calls on rows on the current device
    latched since the last check (a device-side wait that gave up)."""
    _check(lib().sc_rows_check(_stream(stream)), "sc_rows_check")


class _Grad(ctypes.Structure):
    """sc_grad: one gradient and where it goes."""
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int)]


class GradList:
    """A training program's gradients, looked over once: contiguous CUDA tensors
    (float32, float16 or bfloat16, mixed as they come) on one device, of any
    alignment, and where they go when scaled (`out`, tensors like them; default:
    in place).  Looking them over takes about 2 us a gradient (2.5 with outputs), so
    gradients that keep their places are put in a list once and for all.  Holds
    the tensors and their addresses; whoever replaces one, or its memory, makes a
    new list."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError("out must hold a tensor for each gradient")
        entries, spans = [], []
        self.device = None
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            for t in (g, o):
                if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.dtype not in _DTYPES:
                    raise ValueError(f"gradient {i} must be a contiguous float32, float16 or bfloat16 CUDA tensor")
            if o.dtype is not g.dtype or o.numel() != g.numel():
                raise ValueError(f"out[{i}] must have its gradient's dtype and size")
            if self.device is None:
                self.device = g.get_device()
            if g.get_device() != self.device or o.get_device() != self.device:
                raise ValueError("the gradients must lie on one device")
            n, size = g.numel(), g.element_size()
            entries.append((g.data_ptr(), o.data_ptr(), n, _DTYPES[g.dtype]))
            if n:
                spans.append((o.data_ptr(), o.data_ptr() + n * size, i))
                if o is not g and o.data_ptr() != g.data_ptr():
                    spans.append((g.data_ptr(), g.data_ptr() + n * size, -1))
        # what is written lies apart from all else, or two blocks would meet there
        spans.sort()
        high = high_w = -1  # the furthest end so far, of any run and of a written one
        for lo, hi, i in spans:
            if lo < (high if i >= 0 else high_w):
                raise ValueError("gradients that are written share memory with one another or with others")
            high = max(high, hi)
            if i >= 0:
                high_w = max(high_w, hi)
        self.entries = (_Grad * len(entries))(*entries)


def sc_grad_clip(grads, max_norm: float, stream=None):
    """The norm of all gradients together (float32 [1], before the scaling) and
    their scaling by min(1, max_norm / norm), in place or to a GradList's out;
    a norm that is not finite scales nothing.  grads: a GradList, or tensors, of
    which each call makes one anew (48 gradients: 115 us, of which the call with a
    list of them is 15).  No host synchronisation."""
    if not isinstance(grads, GradList):
        grads = GradList(grads)
    current = torch._C._cuda_getDevice()
    if grads.device is not None and grads.device != current:
        raise ValueError(f"the gradients lie on device {grads.device}, which is not the current one")
    norm = torch.empty(1, dtype=torch.float32, device="cuda")
    st = (_lib or lib()).sc_grad_clip(grads.entries, len(grads.entries), max_norm, norm.data_ptr(), _raw_stream(stream))
    if st:
        _check(st, "sc_grad_clip")
    return norm


_ALLOC_FN = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p)
_FREE_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)
_torch_allocator = None  # the callbacks stay alive: buffers they made are freed through them


class Allocator(ctypes.Structure):
    """sc_allocator: a caller's device allocator for one build call."""
    _fields_ = [("alloc", ctypes.c_void_p), ("free", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _alloc_arg(allocator):
    return ctypes.byref(allocator) if allocator is not None else None


def torch_allocator() -> Allocator:
    """An sc_allocator over PyTorch's caching allocator, for the allocator
    argument of the build calls (the callbacks live as long as the module)."""
    _torch_callbacks()
    return Allocator(ctypes.cast(_torch_allocator[0], ctypes.c_void_p).value,
                     ctypes.cast(_torch_allocator[1], ctypes.c_void_p).value, None)


def _torch_callbacks():
    global _torch_allocator
    if _torch_allocator is None:
        def _alloc(nbytes, stream, ctx):
            try:
                return torch.cuda.caching_allocator_alloc(int(nbytes), stream=int(stream or 0))
            except Exception:
                return None

        def _free(ptr, stream, ctx):
            torch.cuda.caching_allocator_delete(int(ptr))

        _torch_allocator = (_ALLOC_FN(_alloc), _FREE_FN(_free))
    return _torch_allocator


def use_torch_allocator(on: bool = True):
    """Route the library's device memory through PyTorch's caching allocator
    (on) or back to CUDA's stream-ordered pool (off) (sc_set_allocator)."""
    if not on:
        _check(lib().sc_set_allocator(None, None, None), "sc_set_allocator")
        return
    _torch_callbacks()
    a = ctypes.cast(_torch_allocator[0], ctypes.c_void_p)
    f = ctypes.cast(_torch_allocator[1], ctypes.c_void_p)
    _check(lib().sc_set_allocator(a, f, None), "sc_set_allocator")


def launch_count() -> int:
    return int(lib().sc_launch_count())


def profile_enable(on: bool = True):
    lib().sc_profile_enable(1 if on else 0)


def profile_only(name_prefix: str | None = None):
    """Time only kernels whose profile name starts with `name_prefix`."""
    lib().sc_profile_only(name_prefix.encode() if name_prefix else None)


def profile_reset():
    lib().sc_profile_reset()


def profile_collect() -> dict:
    """{kernel name: (launches, total ms)} accumulated since the last reset."""
    L = lib()
    _check(L.sc_profile_collect(), "sc_profile_collect")
    out = {}
    i = 0
    name = ctypes.c_char_p()
    n = ctypes.c_int64()
    ms = ctypes.c_double()
    while L.sc_profile_get(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms)) == 0:
        out[name.value.decode()] = (n.value, ms.value)
        i += 1
    return out
