/*
 * sc.h -- C ABI of libsc: submanifold sparse convolution on one GPU
 * (sm_103a).  Plain pointers and sizes only; no C++ or framework types.
 *
 * The layer (after "Sparse inputs and sparse convolution", sections "The fix"
 * and "The map is the computation", and the exam sheet "Sparse convolution
 * for point clouds", sections "Submanifold sparse convolution" and "The map
 * and the update rule"):
 *
 *   points   coords[i] = (batch, x, y, z), features feats[i, 0:C_in]
 *   offsets  d in [-r, r]^ndim, r = (K-1)/2, K odd, stride 1
 *   map      M = {(p, q, d) : coords[p] = coords[q] + d}       (P = Q + d)
 *   layer    out[q, :] = sum_{(p, q, d) in M} feats[p, :] @ W[d]
 *
 * The output point set equals the input point set (P_out = P_in): out has the
 * same N rows, in the same order, as feats.
 *
 * Offset index: lexicographic over (dx, dy[, dz]) with the first axis
 * slowest, idx = sum_k (d_k + r) * K^(ndim-1-k); the centre offset is
 * (V-1)/2 and the mirror of idx is V-1-idx, V = K^ndim.  In 2D (ndim = 2)
 * offsets move x and y only; z is carried unchanged as part of the key.
 *
 * Pointers.  Arguments named d_* are device pointers (cudaMalloc'd or
 * equivalent); the library never dereferences them on the host.  Arguments of
 * sc_kmap_export may be device or host pointers (UVA).  All calls are
 * asynchronous on the given stream unless stated.  Errors in the arguments
 * are returned synchronously; no call aborts, throws or traps.
 *
 * Memory.  Handles own their device buffers, allocated on the stream passed
 * at build time from the allocator passed to the build call (NULL: the
 * process-wide one, see sc_set_allocator; by default CUDA's stream-ordered
 * pool) and released stream-ordered on the stream passed to *_destroy, each
 * buffer to the allocator that made it.  The caller owns coords, feats, W and
 * out.
 */
#ifndef SC_H_
#define SC_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* sc_stream;

typedef enum {
  SC_OK = 0,
  SC_ERR_INVALID_ARG = 1,     /* bad pointer, size, alignment, K, ndim, dims */
  SC_ERR_OUT_OF_RANGE = 2,    /* a coordinate outside [0, dims) or batch outside [0, 65535) */
  SC_ERR_DUPLICATE_COORD = 3, /* two rows share one (batch, x, y, z) */
  SC_ERR_TABLE_FULL = 4,      /* hash insert gave up after probing every slot */
  SC_ERR_UNSUPPORTED = 5,     /* channel counts or dtype the kernels do not cover */
  SC_ERR_CUDA = 6,            /* a CUDA runtime call failed; see sc_last_error() */
  SC_ERR_OOM = 7,             /* device allocation failed */
  SC_ERR_TIMEOUT = 8          /* a bounded device-side wait gave up (kernel bug) */
} sc_status;

/* SC_E4M3 (8 bits, largest value 448): only where an entry point names it */
typedef enum { SC_F32 = 0, SC_F16 = 1, SC_BF16 = 2, SC_E4M3 = 3 } sc_dtype;

/* flags for sc_subm_conv_fwd / sc_subm_conv_tune */
#define SC_RELU 0x1u            /* max(out, 0) before the cast to the output dtype */
#define SC_VARIANT_FUSED 0x10u  /* force the output-stationary tcgen05 kernel */
#define SC_VARIANT_WS 0x20u     /* force the weight-stationary gather/GEMM/scatter kernels */
#define SC_VARIANT_SIMT 0x40u   /* force the CUDA-core kernel (the only one for SC_F32) */
#define SC_VARIANT_SPLIT 0x80u  /* force the fused kernel with column splitting (a map built with SC_KMAP_SPLIT) */
#define SC_VARIANT_MASK 0xF0u

/* flags for sc_kmap_build */
#define SC_KMAP_NO_SYNC 0x100u  /* do not synchronise; check errors later with sc_kmap_check */
#define SC_KMAP_ORDER 0x200u    /* always compute the locality order (default: n >= 262144) */
#define SC_KMAP_NO_ORDER 0x400u /* never compute it: tiles follow the input row order */
#define SC_KMAP_SORT 0x800u     /* always sort the convolution's rows by signature (default: n >= 262144, V <= 128) */
#define SC_KMAP_NO_SORT 0x1000u /* never sort them */
#define SC_KMAP_TRANSPOSE 0x2000u /* sc_kmap_build_conv: the transposed map (rows = the layer's inputs) */
#define SC_KMAP_HALF 0x4000u    /* sc_kmap_build: half probe by mirror symmetry (same map, another build) */
#define SC_KMAP_SPLIT 0x8000u   /* sc_kmap_build, K^ndim <= 32: row orders for column splitting (see below) */
#define SC_KMAP_TILE_TABLE 0x10000u /* K^ndim <= 128: also the fused layer's tile-transposed index table (see below) */

/* flags for sc_qk_norm_rope_fwd / sc_qk_norm_rope_bwd */
#define SC_ROPE_INTERLEAVED 0x1u /* pairs (2i, 2i+1); default: (i, i + rot_dim/2) */

/* flags for sc_attn_fwd / sc_attn_bwd */
#define SC_ATTN_CAUSAL 0x1u /* query i of a sequence sees its keys 0 .. i + (keys - queries) */

typedef struct sc_hash_s* sc_hash;
typedef struct sc_kmap_s* sc_kmap;

/*
 * A caller's device-memory allocator (see "Device memory" below).
 * alloc(bytes, stream, ctx) returns device memory of at least `bytes`,
 * 256-byte aligned, usable in stream order on `stream`, or NULL (the call
 * then fails with SC_ERR_OOM); free(ptr, stream, ctx) releases it after the
 * work queued on `stream`.  The callbacks run on the calling host thread and
 * must not call back into the library.
 */
typedef void* (*sc_alloc_fn)(size_t bytes, sc_stream stream, void* ctx);
typedef void (*sc_free_fn)(void* ptr, sc_stream stream, void* ctx);
typedef struct {
  sc_alloc_fn alloc;
  sc_free_fn free;
  void* ctx;
} sc_allocator;

/* ---------------------------------------------------------------- hash -- */

/*
 * Coordinate hash table: key (batch, x, y, z) -> row id i.
 * After "SparseConvNet: from hash table to rulebook", section 2 (each unique
 * input coordinate gets an incremental index) and "Sparse inputs and sparse
 * convolution", section "Gather, matmul, scatter" (the map is built on the
 * GPU, not copied from a CPU hash).
 *
 * d_coords  int32 [n, 4] row-major (batch, x, y, z), 16-byte aligned.
 *           batch in [0, 65535), x, y, z in [0, 65535).
 * n         number of points, 0 <= n < 2^31.
 * alloc     the allocator of the handle's buffers, or NULL (the process-wide
 *           one).  The struct is copied; its callbacks and ctx must stay
 *           valid until the handle is destroyed.
 * out       receives the handle.
 *
 * Keys are packed into 64 bits (16 bits per field, batch highest).  The
 * table is open addressing with linear probing over entries of one 2x2x2
 * block of voxels each: the block's key (the voxel key with the low bit of x,
 * y, z cleared) and the rows of its 8 voxels.  Capacity = next power of two
 * >= 2n entries (>= n when that would exceed 256 MB).  Asynchronous: a
 * duplicate or out-of-range coordinate is latched in the handle and reported
 * by sc_hash_check, sc_kmap_build or sc_kmap_check.
 */
sc_status sc_hash_build(const int32_t* d_coords, int64_t n, const sc_allocator* alloc, sc_stream stream,
                        sc_hash* out);

/* Row id of each query coordinate, -1 where it is not in the table.
 * d_query int32 [m, 4] (16-byte aligned), d_rows int32 [m]. Asynchronous. */
sc_status sc_hash_query(sc_hash h, const int32_t* d_query, int64_t m, int32_t* d_rows, sc_stream stream);

/* Number of points and table capacity in block entries (host values, no
 * synchronisation). */
sc_status sc_hash_info(sc_hash h, int64_t* n, int64_t* capacity);

/* Synchronises the stream and returns the latched insert status. */
sc_status sc_hash_check(sc_hash h, sc_stream stream);

/* Releases the handle's buffers stream-ordered on `stream`. */
sc_status sc_hash_destroy(sc_hash h, sc_stream stream);

/*
 * Output set of a regular (stride 1) or strided sparse convolution layer, as
 * a new hash handle over the output points.  "SparseConvNet: from hash table
 * to rulebook", section 2, gives the regular output definition: an output is
 * computed wherever the kernel window covers at least one active input, so
 * the active set grows (at stride 1, by the window: "Sparse inputs and sparse
 * convolution", section "What a dense convolution does to empty space");
 * section 3 relates input, output and offset under a stride.  Here output o
 * reads the input at stride * o + d, d in [-(K-1)/2, (K-1)/2]^ndim, and o is
 * an output iff one of those inputs is active.
 *
 * in       the input points' hash.
 * ndim     2 or 3; in 2D the offsets and the stride act on (x, y) and z is
 *          carried unchanged.
 * K        odd, in [1, 7].
 * stride   in [1, 64].
 * dims     the input grid's extents (x, y, z); the outputs lie on the grid
 *          of extents ceil(dims / stride) on the strided axes.
 * out      receives the output set: n = its point count (sc_hash_info),
 *          row ids 0 .. n - 1 in an unspecified order (their coordinates:
 *          sc_hash_coords).  It serves as the input hash of the next layer
 *          and as the output set of sc_kmap_build_conv.  The caller destroys
 *          it with sc_hash_destroy.
 *
 * Synchronises the stream (twice: the input hash's status, then the output
 * count).  Errors: the input hash's latched errors; SC_ERR_TABLE_FULL if the
 * output table would exceed 2^28 entries.  Device memory is allocated
 * stream-ordered on `stream` and owned by the handle.
 */
sc_status sc_hash_build_conv_out(sc_hash in, int ndim, int K, int stride, const int32_t dims[3],
                                 const sc_allocator* alloc, sc_stream stream, sc_hash* out);

/* Coordinates of every row of the hash: d_coords int32 [n, 4] = (batch, x,
 * y, z), device memory, 16-byte aligned, written asynchronously. */
sc_status sc_hash_coords(sc_hash h, int32_t* d_coords, sc_stream stream);

/* ---------------------------------------------------------- kernel map -- */

/*
 * Kernel map (rulebook) for a K^ndim submanifold convolution.
 * After "Sparse inputs and sparse convolution", section "The map is the
 * computation" (for each output q and offset d, look up q + d in the hash);
 * "TorchSparse optimizations", opening section (the centre offset maps every
 * point to itself at stride 1 and is not searched); "SparseConvNet: from hash
 * table to rulebook", section 3 (the rulebook is grouped by weight offset).
 *
 * ndim      2 or 3.
 * K         odd, K >= 1, with V = K^ndim <= 343 (K <= 7 in 3D, K <= 17 in 2D).
 * dims      spatial extents (x, y, z), each in [1, 65535]; every point must
 *           lie inside; neighbours outside are absent (zero padding).
 * flags     0, SC_KMAP_NO_SYNC, at most one of SC_KMAP_ORDER /
 *           SC_KMAP_NO_ORDER, at most one of SC_KMAP_SORT /
 *           SC_KMAP_NO_SORT, SC_KMAP_HALF (build by the half probe: the
 *           offsets after the centre are looked up and each hit is mirrored
 *           by symmetry, "Sparse inputs and sparse convolution", section "A
 *           symmetry you can check"; the same map), SC_KMAP_SPLIT (below),
 *           SC_KMAP_TILE_TABLE (below).
 *
 * Locality order: for n >= 262144 (or with SC_KMAP_ORDER) the build first
 * sorts the points into spatially compact groups (a counting sort on the top
 * 20 bits of a Morton code of (batch, x, y, z)); the convolution's 128-row
 * tiles are runs of that order, so they touch fewer offsets and reuse
 * neighbour rows.  It changes no result: outputs still land on their own
 * rows and nbr stays in input row order.
 *
 * Signature sort (V <= 128; for n >= 262144 or with SC_KMAP_SORT): inside
 * windows of 524288 consecutive rows of that order, the convolution's rows
 * are counting-sorted by a 20-bit signature, which of the 20 least frequent
 * features (over the whole map) the row has a neighbour under.  The
 * features are the offsets when V <= 32, else the 26 coarse directions
 * (sign(dx), sign(dy), sign(dz)), a feature's frequency being the tuple
 * count of its offsets.  Rows that touch the same rare features then share
 * 128-row tiles, and a tile walks fewer offsets (the bitmask reordering of
 * "TorchSparse optimizations", section "TorchSparse++").  It too changes no
 * result.
 *
 * Column splitting (SC_KMAP_SPLIT, V <= 32; implies the signature sort): the
 * offset range is cut at the centre into part 0 (offsets up to and including
 * the centre) and part 1 (the rest), and each part gets a row order of its
 * own, sorted by the signature of its own offsets, with tile masks of its
 * offsets only ("TorchSparse optimizations", section "TorchSparse++": the
 * column split that lets each part's tiles walk fewer offsets).  The layer
 * then uses them when run with SC_VARIANT_SPLIT (or when sc_subm_conv_tune
 * measured that variant fastest): two launches, the first storing fp32
 * partial sums, the second adding its own to them and rounding once.  The map
 * itself is unchanged.
 *
 * Tile table (SC_KMAP_TILE_TABLE, V <= 128, not with SC_KMAP_SPLIT): the
 * build also writes the fused layer's neighbour indices in that layer's row
 * order, transposed within each 128-row tile ([ceil(n/128)][V][128] int32,
 * 4 n V more bytes held by the handle), so that a tile's indices for one
 * offset are one contiguous 512-byte run.  Every fused layer (and input
 * gradient) on the map then reads them there instead of nbr.  Results are
 * unchanged.  It costs one pass over nbr after the build and pays when the
 * map serves several layers: on a batch of four 120k-point LiDAR scans
 * (3x3x3) eight layers 32 -> 256 took 2.37 ms instead of 2.65 ms for a 34 us
 * pass, while a single layer does not recover it (1M voxels 3x3x3: the layer
 * 25 us faster, the pass 60 us; 2M voxels 5x5x5: 100 us and 388 us).
 *
 * Products, owned by the handle:
 *   nbr      int32 [n, V]: nbr[q*V + idx(d)] = row p with coords[p] =
 *            coords[q] + d, or -1.  Column (V-1)/2 is the identity.
 *   offs     int64 [V+1]: per-offset segments of the (in, out) lists.  The
 *            centre segment is empty: its tuples are (i, i) for every i.
 *   in/out   int32 [offs[V]]: list entries (p, q).  The order of the
 *            entries inside a segment is not part of the result and may
 *            differ between builds (runs of up to 128 consecutive rows stay
 *            together, in row order).
 *   map size |M| = n + offs[V] tuples, centre included.
 *
 * Without SC_KMAP_NO_SYNC the call synchronises the stream once and returns
 * the hash's latched errors and its own (SC_ERR_OUT_OF_RANGE when a point
 * lies outside dims).  With it the call is fully asynchronous and errors
 * surface in sc_kmap_check.
 */
sc_status sc_kmap_build(sc_hash h, int ndim, int K, const int32_t dims[3], unsigned flags,
                        const sc_allocator* alloc, sc_stream stream, sc_kmap* out);

/*
 * Kernel map of a regular / strided layer: the rows are the points of
 * `out_set` (from sc_hash_build_conv_out with the same ndim, K, stride and
 * dims), and nbr[q*V + idx(d)] is the row p of `in` with coords[p] = stride *
 * coords[q] + d, or -1 (absent neighbours and the grid's edges: zero
 * padding).  The tuples (p, q, d) follow "SparseConvNet: from hash table to
 * rulebook", section 3 (rulebook grouped by offset).  Unlike a submanifold
 * map the centre offset is searched like the others and has its own list
 * segment; |M| = offs[V].  The map keeps neither hash: both stay owned by
 * the caller.  Flags as for sc_kmap_build (SC_KMAP_TILE_TABLE included)
 * except SC_KMAP_HALF and SC_KMAP_SPLIT (SC_ERR_UNSUPPORTED: submanifold maps
 * only); the locality
 * order and the signature sort apply to the map's rows (the outputs, or the
 * inputs of a transposed map) as for a submanifold map, except that the sort
 * is on by default only when V > 32 as well.
 *
 * sc_subm_conv_fwd and sc_subm_conv_bwd_weight take such a map: feats then
 * has the input's n_in rows and out / gout the map's n rows.  The
 * weight-stationary variant returns SC_ERR_UNSUPPORTED for it.
 *
 * With SC_KMAP_TRANSPOSE the map is transposed: its rows are the points of
 * `in` (the layer's inputs) and nbr[p*V + idx(-d)] is the row q of `out_set`
 * with stride * coords[q] + d = coords[p], or -1 (the outputs whose windows
 * contain p, at the mirrored offset).  sc_subm_conv_bwd_data takes the
 * transposed map of a layer, with d_gout [n_out, c_out] and d_gin [n, c_in]:
 * gin[p] = sum over those (q, d) of gout[q] @ W[idx(d)]^T, the layer's input
 * gradient, on the same kernels as the submanifold one.  A forward map
 * returns SC_ERR_UNSUPPORTED there.
 */
sc_status sc_kmap_build_conv(sc_hash in, sc_hash out_set, int ndim, int K, int stride, const int32_t dims[3],
                             unsigned flags, const sc_allocator* alloc, sc_stream stream, sc_kmap* out);

/* n, V and |M| (centre included).  Synchronises the stream when |M| is not
 * yet known on the host. */
sc_status sc_kmap_info(sc_kmap m, int64_t* n, int32_t* volume, int64_t* map_size, sc_stream stream);

/* Synchronises the stream and returns the latched hash and map status (it
 * reads the two status words only). */
sc_status sc_kmap_check(sc_kmap m, sc_stream stream);

/*
 * Copies the products into caller buffers (device or host pointers; any may
 * be NULL to skip): nbr int32 [n*V], offs int64 [V+1], in_rows and out_rows
 * int32 [offs[V]].  Asynchronous for device destinations.
 */
sc_status sc_kmap_export(sc_kmap m, int32_t* nbr, int64_t* offs, int32_t* in_rows, int32_t* out_rows,
                         sc_stream stream);

/*
 * Borrowed device pointers to the products (the rulebook grouped by weight
 * offset, "SparseConvNet: from hash table to rulebook", section 3; the map as
 * the computation, "Sparse inputs and sparse convolution", section "The map
 * is the computation"), in the layout sc_kmap_export writes:
 *   *d_nbr   int32 [n, V], rows in input row order (nbr[q*V + idx(d)]);
 *   *d_offs  int64 [V+1], the segments of the lists;
 *   *d_in, *d_out  int32 [offs[V]], the list entries (p, q) by segment;
 *   *map_size      |M| (host value).
 * Any output may be NULL to skip it.  The pointers stay valid, and their
 * contents unchanged, until the handle is destroyed; the caller must not
 * write through them.  The first call materialises the forms the handle does
 * not keep internally (rows back in input order when the locality order is
 * on; the lists compacted from their fixed per-offset strides) into buffers
 * the handle owns, from the handle's allocator, on the stream the map was
 * built on, and synchronises that stream (which must still exist); later
 * calls return the same pointers without device work.  Errors: the map's
 * latched status (as sc_kmap_check), SC_ERR_OOM, SC_ERR_CUDA.
 */
sc_status sc_kmap_view(sc_kmap m, const int32_t** d_nbr, const int64_t** d_offs, const int32_t** d_in,
                       const int32_t** d_out, int64_t* map_size);

/* Releases the handle's buffers stream-ordered on `stream`. */
sc_status sc_kmap_destroy(sc_kmap m, sc_stream stream);

/* ---------------------------------------------------------- convolution -- */

/*
 * One submanifold convolution layer on a built map:
 *   out[q, :] = act( sum_{(p, q, d) in M} feats[p, :] @ W[d] )
 * with fp32 accumulation and one rounding to the output dtype; act is
 * max(., 0) with SC_RELU, else the identity.  Update rule after the exam
 * sheet "Sparse convolution for point clouds", section "The map and the
 * update rule", and "Sparse inputs and sparse convolution", section "The map
 * is the computation".
 *
 * d_feats  [n, c_in] row-major, dtype; 16-byte aligned.
 * d_W      [V, c_in, c_out] row-major, dtype (W[idx(d)] is the c_in x c_out
 *          matrix of offset d); 16-byte aligned.
 * d_out    [n, c_out] row-major, dtype; 16-byte aligned; must not alias
 *          d_feats.  Every row is written exactly once.
 * c_in, c_out  multiples of 16 in [16, 256].
 * dtype    SC_F16 / SC_BF16 (tensor-core kernels) or SC_F32 (CUDA cores).
 * flags    SC_RELU, optionally one SC_VARIANT_* to force a kernel family.
 *
 * The fused kernel covers V <= 128; larger kernels use the weight-stationary
 * one.  SC_VARIANT_SPLIT (a map built with SC_KMAP_SPLIT) runs the fused
 * kernel with column splitting and an fp32 partial-sum buffer [n, c_out]
 * allocated for the call.  Variant: forced by flags, else the one sc_subm_conv_tune measured fastest
 * for (c_in, c_out, dtype) on this map, else the fused output-stationary
 * kernel (f16/bf16) or the CUDA-core kernel (f32).  The fused kernel reads
 * each weight slice by TMA straight from d_W (which must then be 16-byte
 * aligned; otherwise, and for output widths that fit no TMA box such as 48
 * or 80 channels, it repacks W into a temporary first) and allocates
 * nothing.  Temporary device memory of the other variants (packed weights,
 * the fp32 accumulator of the weight-stationary variant) is allocated and
 * freed stream-ordered on `stream`.
 */
sc_status sc_subm_conv_fwd(sc_kmap m, const void* d_feats, const void* d_W, void* d_out, int c_in,
                           int c_out, sc_dtype dtype, unsigned flags, sc_stream stream);

/*
 * Times every variant that supports (c_in, c_out, dtype) on this map with
 * CUDA events (`reps` runs each after one warm-up; synchronises), caches the
 * fastest in the handle for sc_subm_conv_fwd, and stores its SC_VARIANT_*
 * flag in *chosen.  d_out receives the last variant's result.
 */
sc_status sc_subm_conv_tune(sc_kmap m, const void* d_feats, const void* d_W, void* d_out, int c_in,
                            int c_out, sc_dtype dtype, unsigned flags, int reps, sc_stream stream,
                            unsigned* chosen);

/*
 * Backward pass of a layer computed by sc_subm_conv_fwd without SC_RELU (for
 * a ReLU layer, mask d_gout by the forward output first).  The layer is
 * linear in feats and in W, so both gradients come from the same map:
 *
 * sc_subm_conv_bwd_data: d_gin[p, :] = sum over the tuples (p, q, d) of
 *   d_gout[q, :] @ W[d]^T.  The tuple (p, q, d) of the forward map is the
 *   tuple (q, p, -d) of the same map (mirror symmetry), so this is a
 *   submanifold layer from c_out to c_in channels with weights
 *   W'[idx(d)] = W[idx(-d)]^T, and it runs on the forward kernels: the fused
 *   kernel reads each slice W[idx(-d)]^T by TMA straight from d_W (16-byte
 *   aligned, c_in at most 256), with no temporary; otherwise,
 *   and in the weight-stationary variant, the weight packing transposes and
 *   mirrors W into a temporary.
 *   d_gout [n, c_out], d_W [V, c_in, c_out] (the forward layer's weights),
 *   d_gin [n, c_in]; c_in and c_out are the forward layer's.  flags: 0 or one
 *   SC_VARIANT_*.
 *
 * sc_subm_conv_bwd_weight: d_dW[d] = sum over the tuples (p, q, d) of
 *   d_feats[p, :]^T d_gout[q, :], accumulated in fp32 from the map's
 *   per-offset lists (the identity for the centre) and rounded once to dtype.
 *   d_feats [n, c_in], d_gout [n, c_out], d_dW [V, c_in, c_out].  flags: 0.
 *   Synchronises once if the map's host counts are not yet known.
 *
 * The source pages show the forward layer only; these follow from it by
 * differentiation.  Argument rules as for sc_subm_conv_fwd.
 */
sc_status sc_subm_conv_bwd_data(sc_kmap m, const void* d_gout, const void* d_W, void* d_gin, int c_in, int c_out,
                                sc_dtype dtype, unsigned flags, sc_stream stream);
sc_status sc_subm_conv_bwd_weight(sc_kmap m, const void* d_feats, const void* d_gout, void* d_dW, int c_in,
                                  int c_out, sc_dtype dtype, unsigned flags, sc_stream stream);

/*
 * The layer of sc_subm_conv_fwd, computed by its fused tensor-core kernel,
 * without allocating any memory.  The source pages have no counterpart: this
 * entry point exists for callers that cannot call cudaMalloc (or any
 * allocator) at this point, such as programs that plan all device memory up
 * front and hand kernels fixed buffers, runtimes that own every allocation
 * themselves, or latency-critical code where an allocation that may block or
 * fail is not acceptable.
 *
 * This entry point always repacks the weights into the fused kernel's
 * shared-memory layout (rather than reading W by TMA as sc_subm_conv_fwd
 * does), into one fixed 4 MiB device array inside the library, present on
 * every GPU that loads the library until the process exits.  The caller still
 * passes every input and output.
 *
 * Limits: f16/bf16 only; V <= 128; V * c_in * c_out * 2 bytes <= 4 MiB
 * (4,194,304), else SC_ERR_UNSUPPORTED with a message in sc_last_error().
 * flags: 0 or SC_RELU.  Other arguments as for sc_subm_conv_fwd.
 *
 * The first call on each device looks up the array's device address with
 * cudaGetSymbolAddress while that device is current; make that first call
 * before any stream capture.  The address is cached per device and per CUDA
 * context: a call made after the device's context was replaced (for example
 * after cudaDeviceReset) looks it up again, so it too should come before any
 * capture.  Every call reuses the one array and overwrites
 * all of the packed weights it uses, so nothing carries over between calls
 * except stale bytes that are never read.  Calls whose GPU work overlaps (on
 * different streams, or from different threads) race on the array: order
 * them on one stream or synchronise between them.
 */
sc_status sc_subm_conv_fwd_noalloc(sc_kmap m, const void* d_feats, const void* d_W, void* d_out, int c_in,
                                   int c_out, sc_dtype dtype, unsigned flags, sc_stream stream);

/* ------------------------------------------------------------- tokens -- */

/*
 * Operators on token rows [tokens, heads, head_dim]: voxels packed scene after
 * scene (or window after window), or text tokens.  The source pages have no
 * counterpart; these are the layers that networks put beside the convolutions
 * to mix voxels at a distance.
 *
 * A strided view of such rows: element (t, h, i) lies at data + t *
 * token_stride + h * head_stride + i (strides in elements), so q, k and v may
 * be parts of one projection's output.  data is device memory, 16-byte
 * aligned, and both strides are multiples of 16 bytes.
 */
typedef struct {
  const void* data;
  int64_t token_stride;
  int64_t head_stride;
} sc_heads;
/* The same for rows that a call writes.  Rows must not share memory: every
 * token's heads lie apart. */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} sc_heads_out;

/*
 * Norm of each head of queries and keys, and the rotation by position, in one
 * pass.  For each row x (head_dim values) of q and of k:
 *   z = w * x / sqrt(mean(x^2) + eps), or z = x when both weights are NULL;
 *   pair i of the first rot_dim values turns by phi = pos[t, axis(i)] * freq[i],
 *   y_a = amp (z_a cos phi - z_b sin phi), y_b = amp (z_b cos phi + z_a sin phi);
 *   the values from rot_dim on are z.
 *
 * q, k        rows of heads_q and heads_k heads; either count may be 0 (its
 *             struct is then not read and may be NULL).
 * d_w_q, d_w_k  fp32 [head_dim], or both NULL (no norm).  A side without
 *             heads may pass NULL.
 * d_pos       int32: token t's position on axis a is d_pos[t * pos_stride + a]
 *             (any int32 value).  With axes = 3 and pos_stride = 4,
 *             d_pos = d_coords + 1 rotates by a voxel's x, y and z.
 * axes        in [1, 4]; rot_dim / 2 is a multiple of it, and pair i belongs to
 *             axis i / (rot_dim / 2 / axes).
 * d_freq      fp32 [rot_dim / 2], radians a position; scaled contexts scale
 *             these (and amp).  The angle keeps its fraction of a turn at any
 *             position.
 * rot_dim     even, in [0, head_dim]; 0: no rotation (d_pos, d_freq may be NULL).
 * head_dim    a multiple of 8 in [16, 256].
 * dtype       of q, k and the outputs: SC_F32, SC_F16 or SC_BF16.  The norm and
 *             the rotation run in fp32 and round once.
 * out_q, out_k  may be q and k themselves (the same pointer and strides); any
 *             other overlap is refused.
 * flags       0 or SC_ROPE_INTERLEAVED.
 */
sc_status sc_qk_norm_rope_fwd(const sc_heads* q, const sc_heads* k, const sc_heads_out* out_q,
                              const sc_heads_out* out_k, const float* d_w_q, const float* d_w_k,
                              const int32_t* d_pos, int64_t pos_stride, int axes, const float* d_freq,
                              int64_t tokens, int heads_q, int heads_k, int head_dim, int rot_dim, float eps,
                              float amp, sc_dtype dtype, unsigned flags, sc_stream stream);

/*
 * Its gradients: gin_q, gin_k from the outputs' gradients gout_q, gout_k and
 * the forward's inputs q, k (read only with a norm; else they may be NULL),
 * and with a norm d_gw_q, d_gw_k fp32 [head_dim] (either may be NULL), summed
 * over tokens and heads in an order that depends on the sizes alone, so that
 * the same inputs give the same bits.  gin may be gout itself.  The other
 * arguments as for the forward.
 */
sc_status sc_qk_norm_rope_bwd(const sc_heads* gout_q, const sc_heads* gout_k, const sc_heads* q, const sc_heads* k,
                              const sc_heads_out* gin_q, const sc_heads_out* gin_k, float* d_gw_q, float* d_gw_k,
                              const float* d_w_q, const float* d_w_k, const int32_t* d_pos, int64_t pos_stride,
                              int axes, const float* d_freq, int64_t tokens, int heads_q, int heads_k, int head_dim,
                              int rot_dim, float eps, float amp, sc_dtype dtype, unsigned flags, sc_stream stream);

/*
 * Attention over packed sequences.  Sequence s has the query rows
 * [d_q_off[s], d_q_off[s+1]) and the key and value rows [d_k_off[s],
 * d_k_off[s+1]), or [d_k_off[s], d_k_off[s] + d_k_len[s]) when d_k_len is not
 * NULL (key lists that grow in place, with room between them).  Query head h
 * reads key head h / (heads_q / heads_kv).  For each query row
 *   S_j = scale * q . k_j,  lse = log sum_j exp(S_j),
 *   out = sum_j exp(S_j - lse) v_j
 * over the keys it sees: all of its sequence, or with SC_ATTN_CAUSAL keys
 * j <= i + (keys - queries) for query i (the last query sees all).  A row that
 * sees no key gets out = 0 and lse = -inf.  Sums and statistics are fp32 (the
 * tensor cores cut a product off at 2^-25 of the sum that it is added to);
 * exp(S - max) is rounded to dtype for the second product (f16: a weight below
 * 2^-21 of the largest is off by up to 2^-32 of it), and out once.
 *
 * d_q_off, d_k_off  int32 [n_seq + 1], device memory, not decreasing;
 *             d_q_off[0] = 0 and d_q_off[n_seq] = t_q (every query row
 *             belongs to a sequence); keys within [0, t_k).  The arrays are
 *             read and checked on the device: a violation writes no output and
 *             is latched for sc_attn_check.  n_seq is below 2^20.
 * d_k_len     int32 [n_seq] or NULL.
 * heads_q     a multiple of heads_kv, at most 128 times it.
 * head_dim    a multiple of 8 in [16, 128].
 * d_lse       fp32 [t_q, heads_q], or NULL.
 * scale       positive, below 2^127.
 * dtype       SC_F16 or SC_BF16.
 * out         must not overlap q, k or v.
 *
 * Values of other sequences never reach a row, whatever they are (NaN
 * included).  Inside a sequence a masked value takes part with weight 0, so a
 * row is finite only if the keys and values after it in its 128-key block are.
 * Temporary device memory is allocated and freed stream-ordered on `stream`: lists of
 * 48 bytes a query tile and, where queries are few and keys may be cut, fp32 partial
 * results of up to 256 MB (a decoding step takes all of it: the size is set by the
 * largest tile, whatever the sequences hold).
 */
sc_status sc_attn_fwd(const sc_heads* q, const sc_heads* k, const sc_heads* v, const sc_heads_out* out,
                      float* d_lse, const int32_t* d_q_off, const int32_t* d_k_off, const int32_t* d_k_len,
                      int64_t n_seq, int64_t t_q, int64_t t_k, int heads_q, int heads_kv, int head_dim, float scale,
                      sc_dtype dtype, unsigned flags, sc_stream stream);

/*
 * Its gradients, from the forward's inputs, out and d_lse and the gradient
 * gout of out:
 *   P = exp(S - lse), delta = gout . out, dS = P * (gout . v - delta),
 *   gq_i = scale sum_j dS_ij k_j, gk_j = scale sum_i dS_ij q_i, gv_j = sum_i P_ij gout_i,
 * gk and gv also summed over the query heads that share the key head.  P and
 * dS are rounded to dtype for the products (f16: held times powers of two, dS's
 * from its sequence's largest values of gout and v, so that small weights and
 * gradients keep their bits), sums are fp32, and each gradient is rounded once.
 * No sum depends on an order of arrival: the same inputs give the same bits.
 *
 * P comes from the fp32 lse, so a weight is off by up to 2^-22 |lse| of itself:
 * beyond the rounding to dtype from |lse| of 2^11 (f16) or 2^14 (bf16) on.  From
 * 2^17 on it is taken low, so that none is above 1 and finite scores and products
 * give finite gradients, if within dtype's range.  As in the forward, a masked
 * query or key inside a sequence takes part with weight 0, so a row of gk or gv
 * is finite only if the queries of the 128-row tiles that it is seen from are.
 *
 * Here the key lists are packed too: d_k_off[0] = 0 and d_k_off[n_seq] = t_k, so
 * that every row of gk and gv is written.  The outputs must not overlap the
 * inputs.
 */
sc_status sc_attn_bwd(const sc_heads* gout, const sc_heads* q, const sc_heads* k, const sc_heads* v,
                      const sc_heads* out, const float* d_lse, const sc_heads_out* gq, const sc_heads_out* gk,
                      const sc_heads_out* gv, const int32_t* d_q_off, const int32_t* d_k_off, int64_t n_seq,
                      int64_t t_q, int64_t t_k, int heads_q, int heads_kv, int head_dim, float scale,
                      sc_dtype dtype, unsigned flags, sc_stream stream);

/* Synchronises the stream, returns the status latched by the attention calls
 * on the current device since the last check (SC_ERR_OUT_OF_RANGE: offsets
 * that break the rules above; SC_ERR_TIMEOUT) and clears it. */
sc_status sc_attn_check(sc_stream stream);

/* --------------------------------------------------------------- rows -- */

/*
 * Operators on rows [rows, channels]: the features of voxels or text tokens
 * between the convolutions and the attention.  The source pages have no
 * counterpart; with these a whole block of such a network, its training step
 * and its inference in 8 bits run on the library.
 *
 * A strided view of rows: channel c of row r lies at data + r * stride + c
 * (stride in elements), so rows may be parts of wider ones.  data is device
 * memory, 16-byte aligned, and the stride a multiple of 16 bytes.
 */
typedef struct {
  const void* data;
  int64_t stride;
} sc_rows;
/* The same for rows that a call writes; they must not overlap one another. */
typedef struct {
  void* data;
  int64_t stride;
} sc_rows_out;

/*
 * The residual's addition and the norm of rows, in one pass:
 *   h = x + res,  y = d_w * h / sqrt(mean(h^2) + eps)
 * and with out_dtype SC_E4M3 the row's scale s = max |y| / 448 and out = y / s
 * in 8 bits, rounded to nearest, so that y is about out * s.
 *
 * res       NULL: h = x.
 * sum       where h goes, in dtype (the next residual), or NULL.
 * d_w       fp32 [channels], 16-byte aligned; NULL: y = h, for SC_E4M3 only
 *           (rows, or weights laid out as rows, quantised as they are).
 * d_scale   fp32 [rows], 4-byte aligned; SC_E4M3 only.
 * channels  a multiple of 8 in [8, 16384].  (sc_linear_fwd takes 8-bit rows and
 *           weights of up to 65536: wider ones than 16384 come from elsewhere.)
 * dtype     of x, res and sum: SC_F32, SC_F16 or SC_BF16.
 * out_dtype dtype or SC_E4M3 (whose out may be aligned, and its rows strided, by
 *           multiples of 8 bytes).
 *
 * Squares are summed in fp32 from the unrounded h, and each output is rounded
 * once.  A row whose squares pass fp32's range (an infinity among them) has
 * r = 0: values 0, and NaN where h is infinite.  A row whose max |y| / 448 is
 * below 2^-126 is written as zeros with scale 0.  An infinity, or with weights
 * squares past fp32's range, leaves its row of 8-bit values without any: scale
 * inf, values 0 or NaN.  With weights a NaN makes its whole row and the scale
 * NaN; without them it is one value of a row that keeps the others' scale.
 * sum may be x or res themselves (the same pointer and
 * stride), and so may out where it has their dtype; any other overlap is
 * refused.
 */
sc_status sc_add_norm_fwd(const sc_rows* x, const sc_rows* res, const sc_rows_out* sum, const sc_rows_out* out,
                          float* d_scale, const float* d_w, int64_t rows, int channels, float eps, sc_dtype dtype,
                          sc_dtype out_dtype, sc_stream stream);

/*
 * Its gradients.  h: the forward's sum (or x, without a residual); gout: the
 * gradient of y; gsum: the gradient that reaches h past the norm, or NULL.
 *   n = h / sqrt(mean(h^2) + eps),  z = d_w * gout,
 *   gin = (z - n mean(z n)) / sqrt(mean(h^2) + eps) + gsum,  d_gw = sum over rows of gout * n
 * gin is the gradient of x and of res alike.  d_gw fp32 [channels], or NULL;
 * summed in fp32 in an order that depends on the sizes alone, so that the same
 * inputs give the same bits.  gin may be gout, gsum or h themselves; any other
 * overlap is refused.  The other arguments as for the forward.
 */
sc_status sc_add_norm_bwd(const sc_rows* gout, const sc_rows* h, const sc_rows* gsum, const sc_rows_out* gin,
                          float* d_gw, const float* d_w, int64_t rows, int channels, float eps, sc_dtype dtype,
                          sc_stream stream);

/* activations of sc_linear_fwd / sc_linear_bwd */
typedef enum {
  SC_ACT_NONE = 0,
  SC_ACT_RELU = 1, /* max(z, 0) */
  SC_ACT_GELU = 2, /* z (1 + erf(z / sqrt 2)) / 2 */
  SC_ACT_SILU = 3  /* z / (1 + exp(-z)) */
} sc_act;

/*
 * Matrix product with its epilogue:
 *   z = x W + d_bias,  out = act(z) + res
 * on the tensor cores, with fp32 sums; out and pre are rounded once.
 *
 * x         [rows, c_in]; in_dtype SC_F16, SC_BF16 or SC_E4M3.  Its rows, and
 *           res's, must not overlap one another (a stride of 0 is refused).
 * d_W       in_dtype, 16-byte aligned, contiguous: [c_in, c_out]; of SC_E4M3
 *           laid out once as [c_out, c_in].
 * d_scale_x, d_scale_w  fp32 [rows] and [c_out] (this one 16-byte aligned),
 *           SC_E4M3 only (as sc_add_norm_fwd writes them): z = d_scale_x[r] d_scale_w[c] sum_i
 *           x[r, i] W[c, i] + d_bias[c], the scales multiplied first, in fp32.
 * d_bias    fp32 [c_out], 16-byte aligned, or NULL.
 * res       [rows, c_out] in dtype, or NULL.
 * out       [rows, c_out] in dtype; may be res itself (the same pointer and
 *           stride); any other overlap is refused.
 * pre       where z goes, in dtype, for the backward pass, or NULL.
 * rows      in [0, 2^31 - 256].
 * c_in, c_out  multiples of 8 (c_in of 16 for SC_E4M3) up to 65536.
 * dtype     SC_F16 or SC_BF16; in_dtype's unless that is SC_E4M3.
 *
 * Few rows take a form that reads the weights once, spread over the card.
 * Temporary device memory, where sums are cut along c_in, is allocated and
 * freed stream-ordered on `stream`.  No sum depends on an order of arrival; where
 * sums are cut may depend, beside the sizes, on which operands' rows begin on
 * 128-byte lines.
 */
sc_status sc_linear_fwd(const sc_rows* x, const void* d_W, const float* d_scale_x, const float* d_scale_w,
                        const float* d_bias, const sc_rows* res, const sc_rows_out* out, const sc_rows_out* pre,
                        int64_t rows, int c_in, int c_out, sc_act act, sc_dtype in_dtype, sc_dtype dtype,
                        sc_stream stream);

/*
 * Its gradients, of the 16-bit forms, from gout, the gradient of out (which is
 * also that of res), and the forward's x, W and pre:
 *   gz = gout * act'(pre),  gin = gz W^T,  d_gW = x^T gz,  d_gbias = sum over rows of gz
 * gin, d_gW [c_in, c_out] (dtype) and d_gbias (fp32) may each be NULL: not
 * computed; what only they read may then be NULL too.  pre is read only with
 * an activation.  gz is rounded to dtype for the products; d_gbias sums it
 * unrounded.  The rows of gout and x must not overlap one another.  relu'(0) = 0.
 * All sums are fp32, in an order that depends on the sizes and, as cuts of k are
 * chosen, on which operands' rows begin on 128-byte lines: the same inputs in
 * places alike give the same bits.  The outputs must not overlap the inputs that
 * are read, or each other.
 */
sc_status sc_linear_bwd(const sc_rows* gout, const sc_rows* x, const sc_rows* pre, const void* d_W,
                        const sc_rows_out* gin, void* d_gW, float* d_gbias, int64_t rows, int c_in, int c_out,
                        sc_act act, sc_dtype dtype, sc_stream stream);

/* Synchronises the stream, returns the status latched by the calls on rows on
 * the current device since the last check (SC_ERR_TIMEOUT: a bounded
 * device-side wait gave up and outputs are not whole) and clears it. */
sc_status sc_rows_check(sc_stream stream);

/* One gradient: n values at data (device memory, aligned to the type), which
 * go to out (data itself: in place). */
typedef struct {
  const void* data;
  void* out;
  int64_t n;
  sc_dtype dtype; /* SC_F32, SC_F16 or SC_BF16 */
} sc_grad;

/*
 * The norm of all gradients together, and their scaling to a largest norm:
 *   norm = sqrt(sum of squares over all values),  out = data * min(1, max_norm / norm)
 * A norm that is not finite, or is past fp32's range and so written as infinity,
 * leaves the values as they are (copied where out is not data); so does max_norm
 * = infinity.
 *
 * grads     host array of `count` entries, read during the call only.  The
 *           entries' dtypes may differ.  Outputs must not overlap each other
 *           or another entry's data, which is the caller's to see to.
 * max_norm  not negative, or infinity.
 * d_norm    fp32 [1], 4-byte aligned, apart from every entry's data and output: the
 *           norm before the scaling.
 *
 * No host synchronisation.  Values whose squares leave fp32's range are squared
 * in 64 bits, and the sums of 65 squares or fewer are added in 64 bits, in an
 * order that depends on the sizes and on where each gradient lies within its
 * 128-byte line: the same inputs in places alike give the same bits.  The factor
 * is rounded to fp32, and each output once.
 */
sc_status sc_grad_clip(const sc_grad* grads, int64_t count, float max_norm, float* d_norm, sc_stream stream);

/* ------------------------------------------------------- device memory -- */

/*
 * Where the library's device memory comes from: the buffers a hash or map
 * handle owns and the temporaries of a call (packed weights, accumulators).
 * By default CUDA's stream-ordered pool (cudaMallocAsync / cudaFreeAsync on
 * the call's stream; the pool keeps freed blocks for reuse).  With
 * sc_set_allocator the library asks the caller's allocator instead, so an
 * application can keep all device memory in one pool (the Python binding
 * offers PyTorch's caching allocator).  A build call (sc_hash_build,
 * sc_hash_build_conv_out, sc_kmap_build, sc_kmap_build_conv) given a non-NULL
 * sc_allocator uses that one for the handle it makes, whatever the
 * process-wide setting is; the handle keeps a copy for the buffers it
 * allocates later (sc_kmap_view).  The source pages have no counterpart.
 *
 * alloc(bytes, stream, ctx) returns device memory of at least `bytes`,
 * 256-byte aligned, usable in stream order on `stream` (the stream of the
 * call that allocates), or NULL (the call then fails with SC_ERR_OOM).
 * free(ptr, stream, ctx) releases it; `stream` is the stream of the call
 * that frees (a handle's destroy, or the allocating call for temporaries),
 * after whose queued work the memory may be reused.  A buffer goes back to
 * the allocator that made it, whatever is set when it is freed.  Pass
 * NULL, NULL to return to the stream-ordered pool; both or neither must be
 * set (else SC_ERR_INVALID_ARG).  The setting is global to the process and
 * thread-safe; the callbacks run on the thread of the library call and must
 * not call back into the library.  sc_subm_conv_fwd_noalloc allocates
 * nothing either way.
 */
sc_status sc_set_allocator(sc_alloc_fn alloc, sc_free_fn free_fn, void* ctx);

/* ---------------------------------------------------------- diagnostics -- */

const char* sc_status_str(sc_status s);

/* Text of the last error raised on the calling host thread ("" if none). */
const char* sc_last_error(void);

/* Total number of kernels this library has launched in this process. */
int64_t sc_launch_count(void);

/*
 * Per-kernel device timing.  While enabled, every launch is bracketed with a
 * pair of CUDA events on its stream.  sc_profile_collect synchronises those
 * events and folds them into per-kernel totals; sc_profile_get reads entry
 * `index` (0-based; returns SC_ERR_INVALID_ARG past the end).
 */
void sc_profile_enable(int on);
/* Restrict the bracketing to kernels whose profile name starts with
 * `name_prefix` (for example "subm_conv"), so that timing one kernel adds no
 * events around the others.  NULL or "" restores all kernels.  The string is
 * copied. */
void sc_profile_only(const char* name_prefix);
sc_status sc_profile_collect(void);
void sc_profile_reset(void);
sc_status sc_profile_get(int index, const char** name, int64_t* launches, double* total_ms);

#ifdef __cplusplus
}
#endif

#endif /* SC_H_ */
