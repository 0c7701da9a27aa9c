/*
 * dbs.h — dual-view blocked sparse matrix x sparse vector multiplication
 * (DB-SpMSpV) with BFS and sparse-decode drivers, for AMD Instinct MI355X
 * (gfx950).
 *
 * The method is the one of "DB-SpMSpV: Dual-View Blocked Sparse Matrix-Sparse
 * Vector Multiplication for Dynamic GPU Workloads" (arXiv 2608.16308):
 *   section 2.1      the product y = A x with push (column-driven) and pull
 *                    (row-driven) formulations, Algorithm 1;
 *   section 3.2      the dual-view blocked format: 16x16 tiles, block-level
 *                    CSR and CSC index views over one shared tile payload,
 *                    five tile formats, 16-element vector blocks with masks;
 *   section 3.3      the two-level adaptive engine: push/pull selection from
 *                    the nonzero-block ratio, per-tile microkernels, load
 *                    balancing and hierarchical writeback;
 *   section 4.1      on-GPU construction of the vector-block metadata;
 *   section 4.2      DB-BFS (frontier = sparse x, visited mask);
 *   section 4.3      DB-Decoding (dense activation -> activation masks).
 *
 * Conventions for every entry point
 *   - Matrix and vector pointers are DEVICE pointers (memory from hipMalloc or
 *     any allocator of the current device), unless stated otherwise.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls are stream-ordered and asynchronous unless stated otherwise.
 *   - The caller owns all input and output buffers.  The handle owns the
 *     blocked format and the transient scratch it uses.  Inputs are never
 *     written.  Outputs are overwritten completely on every call.
 *   - Errors are reported by the return code only; nothing is thrown across
 *     the ABI.  On an error return no output has been written, except where
 *     a device-side check is documented.
 *   - A handle may be used by one stream at a time: calls on one handle that
 *     overlap in time race on its scratch.
 */
#ifndef DBS_H
#define DBS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dbs_matrix *dbs_handle; /* opaque */

typedef enum {
  DBS_OK = 0,
  DBS_ERR_INVALID_ARG = 1,   /* null pointer, bad size, bad enum, dtype/semiring mismatch */
  DBS_ERR_BAD_CSR = 2,       /* row_ptr not monotone / not starting at 0 / not ending at nnz,
                                column out of range, columns not strictly increasing in a row */
  DBS_ERR_OUT_OF_MEMORY = 3, /* a device allocation failed; nothing is leaked */
  DBS_ERR_DEVICE = 4,        /* a HIP runtime call failed */
  DBS_ERR_UNSUPPORTED = 5,   /* valid request this library does not implement */
  DBS_ERR_BAD_VECTOR = 6,    /* check mode found x_idx not strictly increasing */
  DBS_ERR_TOO_LARGE = 7      /* the problem needs more than the fixed scratch of an
                                allocation-free call (DBS_NOALLOC_SCRATCH_BYTES) */
} dbs_status;

/* value type of the matrix (and of x for DBS_PLUS_TIMES) */
typedef enum { DBS_F32 = 0, DBS_BF16 = 1, DBS_PATTERN = 2 } dbs_dtype;

/* PLUS_TIMES: y_i = sum_j a_ij x_j over active j, fp32 output, fp32 accumulation.
 * OR_AND:     y_i = 1 iff row i has a stored entry in an active column (values
 *             ignored, explicitly stored zeros count), uint8 0/1 output. */
typedef enum { DBS_PLUS_TIMES = 0, DBS_OR_AND = 1 } dbs_semiring;

/* Tile formats of section 3.2.1 (Figure 5(b)). */
typedef enum {
  DBS_TILE_COO = 0,       /* nnz < th0: packed (row<<4 | col) bytes + values */
  DBS_TILE_DENSE = 1,     /* nnz > th1: 256 values, row-major */
  DBS_TILE_FORCE_CSR = 2, /* column skew > th2 x row skew: row masks + row pointers */
  DBS_TILE_FORCE_CSC = 3, /* row skew > th2 x column skew: column masks + column pointers */
  DBS_TILE_CSR = 4        /* otherwise: patched CSR (row view + col_ptr + row_idx_csc2csr) */
} dbs_tile_format;

/* ------------------------------------------------------------------------
 * Build-time options (section 3.2.1 thresholds, section 3.3.2 segment weights).
 * ------------------------------------------------------------------------ */
typedef struct {
  int32_t th0;            /* COO below this nnz (default 32) */
  int32_t th1;            /* Dense above this nnz (default 128) */
  int32_t th2_num;        /* skew ratio threshold th2 = th2_num / th2_den (default 2/1) */
  int32_t th2_den;
  int32_t force_format;   /* -1 = adaptive (default); a dbs_tile_format value stores every
                             tile in that format (the format ablation of Figure 10) */
  int32_t seg_w_dense;    /* pull segment weights: Dense (default 4) */
  int32_t seg_w_csr;      /*   ForceCSR / ForceCSC / CSR (default 2) */
  int32_t seg_w_coo;      /*   COO (default 1) */
  int32_t seg_cap;        /* a segment closes at the tile bringing its weight to >= cap.
                             0 (default): 64 for value matrices, 256 for pattern matrices
                             (one 64-lane wave works on a segment, one tile per lane for
                             value matrices, four for pattern matrices; the pages'
                             32-lane warps use 16).  Explicit range 1..64 (value) or
                             1..256 (pattern): a segment holds at most seg_cap tiles;
                             other values give DBS_ERR_INVALID_ARG. */
} dbs_build_options;

/* Fills `opt` with the defaults above.  Never fails for a non-NULL pointer. */
dbs_status dbs_build_options_default(dbs_build_options *opt);

/*
 * dbs_build — convert a CSR matrix into the dual-view blocked format
 * (section 3.2.1, Figure 5(b)); the conversion runs on the GPU.
 *
 *   m, n      rows and columns, 1 <= m, n < 2^31
 *   nnz       stored entries, 0 <= nnz < 2^31
 *   row_ptr   device int32[m+1], row_ptr[0] = 0, non-decreasing, row_ptr[m] = nnz
 *   col_idx   device int32[nnz], strictly increasing within each row, in [0, n)
 *   val       device values: float[nnz] (DBS_F32), bf16 bit patterns uint16[nnz]
 *             (DBS_BF16) or NULL (DBS_PATTERN: structure only)
 *   opt       build options, or NULL for the defaults
 *   stream    hipStream_t; the call is SYNCHRONOUS on it (it reads sizes back)
 *   out       receives the new handle; untouched on error
 *
 * The CSR arrays may be freed once the call returns.  Returns DBS_ERR_BAD_CSR
 * for an invalid CSR (checked on the device before any other work), and
 * DBS_ERR_UNSUPPORTED for a format the kernels cannot address with their
 * 32-bit byte offsets: a tile payload of more than 4,294,967,024 bytes (4 GiB -
 * 272), or more than 536,870,910 tiles.
 */
dbs_status dbs_build(int32_t m, int32_t n, int64_t nnz, const int32_t *row_ptr,
                     const int32_t *col_idx, const void *val, dbs_dtype dtype,
                     const dbs_build_options *opt, void *stream, dbs_handle *out);

/*
 * dbs_spmspv — y = A x for a sparse x (sections 3.3, 4.1).
 *
 *   nnz_x     number of listed entries, 0 <= nnz_x <= n
 *   x_idx     device int32[nnz_x], strictly increasing.  Listed positions form
 *             the active set; an index outside [0, n) contributes nothing.
 *   x_val     device values of the matrix dtype (float or bf16 bits), required
 *             for DBS_PLUS_TIMES, ignored (may be NULL) for DBS_OR_AND.
 *   sr        DBS_PLUS_TIMES (not allowed on a DBS_PATTERN matrix) or DBS_OR_AND
 *   y         device float[m] (PLUS_TIMES) or uint8[m] holding 0/1 (OR_AND)
 *
 * One call launches the vector-metadata kernel and the SpMSpV kernel; the
 * push/pull choice (push iff N_nzblk / N_blk < th3) is taken on the device.
 * DBS_PLUS_TIMES on a DBS_F32 matrix of more than 1,073,741,808 columns, or a
 * DBS_BF16 one of more than 2,147,483,632 (x block-padded past 4 GiB - 16
 * bytes), returns DBS_ERR_UNSUPPORTED; so do the dense calls below.
 * In check mode (DBS_OPT_CHECK) a non-increasing x_idx is flagged on the
 * device and reported by the next dbs_get_stats as DBS_ERR_BAD_VECTOR;
 * without check mode such input gives unspecified (but memory-safe) y.
 */
dbs_status dbs_spmspv(dbs_handle A, int32_t nnz_x, const int32_t *x_idx, const void *x_val,
                      dbs_semiring sr, void *y, void *stream);

/*
 * dbs_spmspv_dense — y = A x for a dense x whose zeros are inactive, the
 * single-token decode case (section 4.3).  The activation masks are built on
 * the GPU from x (section 4.1): x_j is active iff x_j != 0 (+0 and -0 are
 * inactive).
 *
 *   x   device float[n] (DBS_F32) or bf16 bits uint16[n] (DBS_BF16); for
 *       DBS_OR_AND on a DBS_PATTERN matrix, float[n]
 *   y   as for dbs_spmspv
 */
dbs_status dbs_spmspv_dense(dbs_handle A, const void *x, dbs_semiring sr, void *y,
                            void *stream);

/*
 * dbs_spmspv_dense_threshold — decode with the activation sparsified in the
 * metadata kernel: y = A x' with x'_j = x_j when |x_j| > threshold, else 0
 * (magnitude thresholding, the activation sparsity of the decoding
 * evaluation, section 5.4).  The masks (section 4.1) come from x' and the
 * multiply reads x' only; x itself is not written.  threshold = 0 gives
 * dbs_spmspv_dense, except that a NaN entry of x is dropped here (every
 * comparison with NaN is false).
 *
 *   x          as for dbs_spmspv_dense
 *   threshold  finite and >= 0, else DBS_ERR_INVALID_ARG
 *   y          as for dbs_spmspv
 */
dbs_status dbs_spmspv_dense_threshold(dbs_handle A, const void *x, float threshold, dbs_semiring sr,
                                      void *y, void *stream);

/*
 * dbs_bfs — single-source BFS levels (section 4.2, Algorithm 5).  Each level
 * is one masked OR_AND SpMSpV y = A f with the frontier f as the sparse
 * vector; push or pull is chosen per level from the frontier's nonzero-block
 * ratio with the same rule as dbs_spmspv.  Vertex i is reached from j when
 * A_ij is stored (for a symmetric A this is the usual undirected BFS).
 *
 *   A        square (m == n) matrix of any dtype (values are ignored)
 *   src      source vertex, 0 <= src < m
 *   levels   device int32[m]: hop distance from src, -1 if unreachable
 *
 * SYNCHRONOUS on `stream`: the levels are launched in batches of eight and
 * the host reads the frontier sizes of a batch once (one stream
 * synchronization per eight levels); the levels of the last batch that come
 * after the first empty frontier return at once.  Uses device scratch that
 * the handle allocates on the first call (bitmaps, block lists, counters).
 */
dbs_status dbs_bfs(dbs_handle A, int32_t src, int32_t *levels, void *stream);

/*
 * dbs_bfs_noalloc — dbs_bfs for callers that cannot allocate memory (code
 * that must not call hipMalloc, tight serving loops, harnesses that forbid
 * allocation).  Same arguments, same levels, same kernels; the run's device
 * scratch comes from a fixed array of DBS_NOALLOC_SCRATCH_BYTES that each
 * device holds for the life of the process (set up on the first call on a
 * device), and the frontier sizes go to a host buffer on the call's stack.
 * The call makes no allocation of its own (no hipMalloc, hipHostMalloc,
 * hipFree).
 *
 *   Scratch needed: the 256-B-aligned sum of 4 (3 ceil(nb/2) + 1) (frontier
 *   bitmaps), 4 (ceil(nb/2) + 1) (visited), 4 (3 nb + 1) (block lists) and
 *   4 (25 + 8) (counters) bytes, about 20 nb bytes (nb = ceil(n/16)): up to
 *   about 26 million vertices.  When a push level could need chunk lists cut
 *   ahead (a forced push with nb > 6144, or th3 above 6144 / nb), 8 (3
 *   (T/64 + nb + 1) + 1) bytes more.  A larger problem returns
 *   DBS_ERR_TOO_LARGE before any work.
 *
 *   The array is shared by every call on the device and keeps the last
 *   call's contents (each call clears what it needs at its start): calls that
 *   overlap in time on one device race.  The current device must be the
 *   handle's (else DBS_ERR_INVALID_ARG).  dbs_stats.bfs_reached is not
 *   counted for this call (it stays -1): the visited bitmap it would be
 *   counted from lives in the shared array.
 */
#define DBS_NOALLOC_SCRATCH_BYTES (32u << 20)
dbs_status dbs_bfs_noalloc(dbs_handle A, int32_t src, int32_t *levels, void *stream);

/* Per-handle run-time options (dbs_set_option / dbs_get_option). */
enum {
  DBS_OPT_PATH = 0,              /* 0 auto (default), 1 force push, 2 force pull */
  DBS_OPT_TH3_NUM = 1,           /* th3 = num / den (default 1 / 100): push iff */
  DBS_OPT_TH3_DEN = 2,           /*   N_nzblk * den < N_blk * num              */
  DBS_OPT_LOCAL_PUSH_CUTOFF = 3, /* patched-CSR tiles use the column (push) microkernel
                                    when popcount(blk_x_mask) < cutoff (default 0: always
                                    the row microkernel, the faster one on this GPU) */
  DBS_OPT_TIMING = 4,            /* 1: time the kernels of each call with HIP events (setting
                                    it, to 0 or 1, also clears the sums in dbs_stats) */
  DBS_OPT_CHECK = 5,             /* 1: validate x_idx ordering on the device */
  DBS_OPT_PULL_WIDTH = 6,        /* PLUS_TIMES pull of a value matrix, segments per wave
                                    step: 0 auto (default: four when every resident wave
                                    gets several steps, else one), 1 or 4 forced */
  DBS_OPT_PULL_SHARE = 7         /* PLUS_TIMES pull with one segment per step: waves that
                                    share a segment, each taking a range of its tiles:
                                    0 auto (default: enough to give every resident wave
                                    work, at most 4), 1, 2 or 4 forced.  Ignored with four
                                    segments per step.  Both options change only the work
                                    split (and the fp32 summation order), not the result's
                                    bound; they exist to test and measure every variant */
};
dbs_status dbs_set_option(dbs_handle A, int32_t option, int64_t value);
dbs_status dbs_get_option(dbs_handle A, int32_t option, int64_t *value);

typedef struct {
  /* format (fixed at build time) */
  int32_t m, n, mb, nb;            /* rows, columns, row blocks, column blocks */
  int64_t nnz, tiles;
  int64_t tiles_by_format[5];      /* indexed by dbs_tile_format */
  int64_t nnz_by_format[5];
  int64_t segments;                /* pull segments */
  int64_t payload_bytes;           /* tile payload arena */
  int64_t index_bytes;             /* block-CSR + block-CSC views and tile metadata */
  int64_t format_bytes;            /* payload + index + segment descriptors + (pattern
                                      matrices) the Boolean pull's own arrays */
  int64_t build_peak_bytes;        /* peak device memory held during dbs_build */
  /* last dbs_spmspv / dbs_spmspv_dense call (reading them synchronizes its stream) */
  int32_t last_path;               /* 0 push, 1 pull, -1 no call yet */
  int32_t last_n_nzblk;            /* nonzero vector blocks */
  int64_t last_push_chunks;        /* 64-tile work chunks listed ahead for push (0 when the
                                      pushing kernel takes them from the block list itself) */
  float last_meta_ms;              /* metadata kernel time (DBS_OPT_TIMING), else -1 */
  float last_compute_ms;           /* SpMSpV kernel time (DBS_OPT_TIMING), else -1 */
  /* sums over the SpMSpV calls made since DBS_OPT_TIMING was last set to 1 (HIP
     events recorded on each call's stream around each of its two kernels) */
  int64_t timed_calls;
  double sum_meta_ms;
  double sum_compute_ms;
  /* last dbs_bfs call */
  int32_t bfs_levels;              /* levels run (including the empty last one) */
  int32_t bfs_push_levels;         /* of which push */
  int64_t bfs_reached;             /* vertices with a level >= 0 (counted from the handle's
                                      visited bitmap when dbs_get_stats is called) */
  float bfs_ms;                    /* whole BFS (DBS_OPT_TIMING), else -1 */
  float bfs_kernel_ms;             /* sum of the level kernels (DBS_OPT_TIMING), else -1 */
} dbs_stats;

/* Fills `out`; synchronizes the stream of the last call.  Returns
 * DBS_ERR_BAD_VECTOR (and still fills `out`) if check mode flagged the last call. */
dbs_status dbs_get_stats(dbs_handle A, dbs_stats *out);

/* Internal arrays of the format, copied to HOST memory for inspection and
 * tests.  `bytes_out` (may be NULL) receives the array's size; `dst` may be
 * NULL to query the size only; otherwise `capacity` must be at least that
 * size.  Synchronous.  Layouts are described in the library's design notes. */
enum {
  DBS_ARR_RB_PTR = 0,      /* uint32[mb+1]   global_block_csr_row_ptr */
  DBS_ARR_T_CB = 1,        /* uint32[T]      global_block_csr_col_idx */
  DBS_ARR_T_META = 2,      /* uint64[T]      payload offset | (nnz-1)<<40 | format<<48
                                             | inline<<51 | pattern: row block in its
                                             Boolean-pull segment<<52 */
  DBS_ARR_CB_PTR = 3,      /* uint32[nb+1]   global_block_csc_col_ptr */
  DBS_ARR_CSC_RB = 4,      /* uint32[T]      global_block_csc_row_idx */
  DBS_ARR_CSC2CSR = 5,     /* uint32[T]      global_block_csc2csr */
  DBS_ARR_PAYLOAD = 6,     /* uint8[]        tile payload arena */
  DBS_ARR_SEGMENTS = 7,    /* uint32[4*S]    {row block | split<<31 | drain<<30 | slot
                                             class<<28, t0, t1, partial slot + 1 or 0}:
                                             value matrices: the segments of class 3 first, by
                                             first column block, then the others by row block */
  DBS_ARR_XMASK = 8,       /* uint16[nb]     blk_x_mask of the last call */
  DBS_ARR_ACTIVE = 9,      /* uint32[N_nzblk] nonzero vector blocks of the last call (any order) */
  DBS_ARR_CSC_CM = 10,     /* uint16[T]      columns of each tile that hold entries, CSC order */
  DBS_ARR_PAT_SEGS = 11,   /* uint32[4*S']   pattern matrices: Boolean-pull segments {first row
                                             block, t0, t1, row blocks}, in launch order */
  DBS_ARR_T_CBX = 12,      /* uint32[T]      pattern matrices, the Boolean pull's column-block
                                             words: at most 2^19 column blocks: column block |
                                             row block in its Boolean-pull segment<<19 | (one
                                             entry<<23 | that entry's (row<<4 | column)<<24, or
                                             else the tile's index among its segment's tiles of
                                             more than one entry<<24); more: column block | that
                                             row block<<27 */
  DBS_ARR_META2 = 13,      /* uint64[T']     pattern matrices: the T_META words of the tiles
                                             without bit 23 in T_CBX, in tile order */
  DBS_ARR_PAT_M2 = 14      /* uint32[2*S']   per Boolean-pull segment (PAT_SEGS order): its
                                             first entry in META2, and its entries */
};
dbs_status dbs_copy_array(dbs_handle A, int32_t which, void *dst, int64_t capacity,
                          int64_t *bytes_out);

/* Releases the handle and everything it owns (synchronizes its last stream).
 * NULL is accepted. */
dbs_status dbs_free(dbs_handle A);

/* Static description of a status code. */
const char *dbs_status_string(dbs_status s);

/*
 * dbs_probe_read — a measurement helper, not part of the method: reads the
 * `bytes` bytes at device address `buf` once, with 16-byte vector loads from
 * a grid of eight 256-thread workgroups per compute unit, and writes nothing
 * unless the XOR of some thread's words equals `never` (then that value goes
 * to the device word *sink; pick a value the data cannot produce).  Timing it
 * on a stream gives the streaming-read bandwidth of the device, the yardstick
 * beside the published HBM peak for the byte-model roofline of the SpMSpV
 * kernels.  `buf` 16-byte aligned, `bytes` a positive multiple of 16, `sink`
 * a device uint32; else DBS_ERR_INVALID_ARG.  Asynchronous on `stream`.
 */
dbs_status dbs_probe_read(const void *buf, int64_t bytes, uint32_t *sink, uint32_t never, void *stream);

/* ------------------------------------------------------------------------
 * The layers and steps of a decoded token around the sparse products: 4-bit
 * weights, logits, rotary positions.  Vectors of several tokens are rows
 * [token][element] whose row stride is given in elements; `*_dtype` is
 * DBS_F32 or DBS_BF16.  The calls allocate nothing and use no scratch, so
 * they may run on several streams at once and be captured into a graph; they
 * run on the current device, which must hold all their buffers.  No output
 * may overlap an input, from its first byte to its last, except where stated.
 * Sums are in fp32; nothing depends on timing, so a call on the same inputs
 * gives the same bits again.
 * ------------------------------------------------------------------------ */
typedef struct dbs_q4_matrix *dbs_q4_handle; /* opaque */

/* tokens of one call, rows (row numbers of a last workgroup stay below 2^31) and columns (offsets in a
 * row of tiles stay below 2^32) at most */
#define DBS_Q4_MAX_TOKENS 524288
#define DBS_Q4_MAX_ROWS 2147483520
#define DBS_Q4_MAX_COLUMNS 268435456

/*
 * dbs_q4_build — lay out an m x n matrix held in 4 bits with group scales:
 *
 *   W_ij = scale[i][j / group] * (code_ij - zero[i][j / group])
 *
 *   group       32, 64 or 128 columns (the last group of a row may be cut)
 *   codes       device uint8[m][ceil(n/2)]: code of an even column in the low
 *               nibble, of the odd column after it in the high one
 *   scales      device [m][ceil(n/group)], float (DBS_F32) or bf16 (DBS_BF16)
 *   zeros       device uint8[m][ceil(n/group)], each at most 15, or NULL: 8
 *   stream      the call is SYNCHRONOUS on it (it reads a check flag back)
 *   out         receives the new handle; untouched on error
 *
 * The inputs may be freed once the call returns.  A zero point above 15 gives
 * DBS_ERR_INVALID_ARG.  Handles are read only after the build: calls on one
 * handle may overlap in time.
 */
dbs_status dbs_q4_build(int32_t m, int32_t n, int32_t group, const uint8_t *codes, const void *scales,
                        dbs_dtype scale_dtype, const uint8_t *zeros, void *stream, dbs_q4_handle *out);

/* Device bytes that the handle holds. */
dbs_status dbs_q4_bytes(dbs_q4_handle A, int64_t *bytes);

/* Releases the handle (waits for the device).  NULL is accepted. */
dbs_status dbs_q4_free(dbs_q4_handle A);

/*
 * dbs_q4_product — y_t = W x_t for `tokens` vectors, fp32 accumulation, one
 * rounding to y's type.
 *
 *   tokens   0 <= tokens <= DBS_Q4_MAX_TOKENS; made for one to 64 (up to 32 at a time, each time
 *            going through the weights, which come from memory once if the tokens are few)
 *   x        device [tokens][n], row stride ldx >= n elements
 *   y        device [tokens][m], row stride ldy >= m elements
 *
 * Infinities and NaN in x or the scales spread as in the formula, to the
 * tokens and rows whose sums hold them.  Results that are not finite are
 * computed a second time, weight by weight, which takes far longer (28672 x
 * 8192, 64 tokens of bf16: 56 us, 0.96 ms with a NaN in one token, 15 ms with
 * one in each): what pads a batch is better finite, or fewer tokens.
 *
 * A group's part of y is scale (sum (16 + code) x - (16 + zero) sum x), each
 * sum rounded for itself: before its rounding to y's type, y_ti is off by at
 * most
 *
 *   (387 + groups of a row) 2^-24 sum_j |scale x_j| (32 + code + zero)
 *
 * (and, for fp32 x, by what its bits below 2^-133 stand for, which are left out),
 * which is relative to these magnitudes, not to |W_ij x_j| (on ordinary data
 * a few 2^-24 of them, since roundings go either way).  A group of a row whose
 * codes all equal its zero point adds nothing: a row of such groups (pruned
 * or padding) is exactly 0 for finite x.  Other results that the formula makes 0 by
 * cancelling, or by zeros in x under nonzero weights, may come out as such a
 * small number.
 */
dbs_status dbs_q4_product(dbs_q4_handle A, int32_t tokens, const void *x, dbs_dtype x_dtype, int64_t ldx,
                          void *y, dbs_dtype y_dtype, int64_t ldy, void *stream);

/*
 * dbs_q4_product_masked — the same where token t wants only the rows i whose
 * bit i % 32 of row_mask[t][i / 32] is set (a grammar's allowed tokens at the
 * head): y_ti = fill elsewhere, whatever x holds.  A workgroup's rows are not
 * read if none of its tokens wants any of them: 16 rows for up to four
 * tokens; for more, up to 32 tokens and 16, 32, 64 or 128 rows, the more the
 * larger the call, so that a few wanted rows of a large matrix may have as
 * many read for each.  Bits at m and above are ignored.
 *
 *   row_mask   device uint32[tokens][ceil(m/32)], row stride ldmask words
 *   fill       any float, -INFINITY for logits
 */
dbs_status dbs_q4_product_masked(dbs_q4_handle A, int32_t tokens, const void *x, dbs_dtype x_dtype,
                                 int64_t ldx, const uint32_t *row_mask, int64_t ldmask, float fill, void *y,
                                 dbs_dtype y_dtype, int64_t ldy, void *stream);

/* activations of dbs_q4_gated: g / (1 + exp(-g)); g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)));
 * max(g, 0) (whose zeros a following dbs_spmspv_dense skips; a gate that the formula makes 0 by cancelling may be within
 * the product's error above 0 instead, which dbs_spmspv_dense_threshold drops) */
typedef enum { DBS_ACT_SILU = 0, DBS_ACT_GELU_TANH = 1, DBS_ACT_RELU = 2 } dbs_activation;

/*
 * dbs_q4_gated — y_t = act(G x_t) * (U x_t), elementwise: the gate and up
 * layers in one pass, products and activation in fp32, one rounding to y's
 * type.  G and U have the same m, n, group and scale type (one handle may be
 * given twice).  Arguments as for dbs_q4_product.
 */
dbs_status dbs_q4_gated(dbs_q4_handle G, dbs_q4_handle U, dbs_activation act, int32_t tokens, const void *x,
                        dbs_dtype x_dtype, int64_t ldx, void *y, dbs_dtype y_dtype, int64_t ldy,
                        void *stream);

/* rows of one dbs_logits_adjust call at most */
#define DBS_LOGITS_MAX_ROWS 65535

/*
 * dbs_logits_adjust — penalties, biases and a mask on rows of logits, in fp32
 * with one rounding to the output's type.  Per row b and token v, in order:
 *
 *   1. v anywhere in the row's history:  l = l > 0 ? l / repetition : l * repetition
 *   2. l -= frequency * c, and l -= presence if c > 0, where c counts v among
 *      the history's entries from hist_new[b] on (the generated ones)
 *   3. l += the row's bias of v (of several entries of one v the last counts)
 *   4. mask bit v % 32 of mask[b][v / 32] clear:  l = -inf, whatever l was
 *
 * Every step whose pointer is NULL is left out.  Ids outside [0, vocab)
 * contribute nothing, and the lists' pointers are clamped to the lists, so
 * bad ones are memory-safe.  A row whose mask is empty is -inf throughout.
 */
typedef struct {
  const int32_t *hist_ptr;   /* device int32[rows+1]: row b's history is hist[hist_ptr[b] .. hist_ptr[b+1]) */
  const int32_t *hist;       /* device int32[hist_len] token ids */
  int64_t hist_len;
  const int32_t *hist_new;   /* device int32[rows], positions within the row's history; NULL: 0 */
  const float *repetition;   /* device float[rows], > 0 */
  const float *frequency;    /* device float[rows] */
  const float *presence;     /* device float[rows] */
  const int32_t *bias_ptr;   /* device int32[rows+1] */
  const int32_t *bias_idx;   /* device int32[bias_len] token ids */
  const float *bias_val;     /* device float[bias_len] */
  int64_t bias_len;
  const uint32_t *mask;      /* device uint32[rows][ceil(vocab/32)], row stride ldmask words */
  int64_t ldmask;
} dbs_logits_params;

/*
 *   rows, vocab   0 <= rows <= DBS_LOGITS_MAX_ROWS, vocab >= 1
 *   logits        device [rows][vocab], row stride ld_in >= vocab
 *   out           device [rows][vocab], row stride ld_out >= vocab; may be `logits` itself (same
 *                 type and stride)
 * hist_ptr and hist go together, as do bias_ptr, bias_idx and bias_val;
 * repetition, frequency, presence or hist_new without a history is
 * DBS_ERR_INVALID_ARG.
 */
dbs_status dbs_logits_adjust(int32_t rows, int32_t vocab, const void *logits, dbs_dtype in_dtype, int64_t ld_in,
                             const dbs_logits_params *params, void *out, dbs_dtype out_dtype, int64_t ld_out,
                             void *stream);

/* pairs of a rotated head: element i with i + rot_dim/2, or 2i with 2i + 1 */
typedef enum { DBS_ROPE_HALF = 0, DBS_ROPE_INTERLEAVED = 1 } dbs_rope_layout;

/* largest rot_dim, and heads * head_dim */
#define DBS_ROPE_MAX_DIM 1024
#define DBS_ROPE_MAX_ELEMENTS 1073741824

/*
 * dbs_rope — rotary positions: in each head of each token, pair i (a, b) of
 * the first rot_dim elements becomes
 *
 *   (scale (a cos p - b sin p), scale (a sin p + b cos p)),  p = pos[token] * freq[i]
 *
 * and the elements from rot_dim on are copied.  p is formed and reduced in
 * 64 bits, so far positions keep their phase.
 *
 *   tokens, heads  >= 0;  head_dim >= 1;  rot_dim even, 0 <= rot_dim <= head_dim
 *   pos            device int32[tokens]; a negative position marks padding: the token's
 *                  rows of `out` are left as they are
 *   freq           device double[rot_dim/2], radians per position (dbs_rope_frequencies)
 *   inverse        nonzero: rotate by -p (undoes a rotation; the gradient with respect to x
 *                  is this rotation of the output's gradient)
 *   x, out         device, element (t, h, d) at t * token stride + h * head stride + d;
 *                  `out` may be `x` itself (same type and strides), else they share no element;
 *                  if one has elements between those of the other, as parts of one buffer, they
 *                  have the same token or head stride in bytes, and where the other stride differs
 *                  the rows along it, with what stands between them, are apart.
 *                  Strides of x are free; of out, one is at least head_dim and the other leaves
 *                  room for all that the first one spans (either order, either sign)
 */
dbs_status dbs_rope(int32_t tokens, int32_t heads, int32_t head_dim, int32_t rot_dim, dbs_rope_layout layout,
                    const int32_t *pos, const double *freq, float scale, int32_t inverse, const void *x,
                    dbs_dtype x_dtype, int64_t x_token_stride, int64_t x_head_stride, void *out,
                    dbs_dtype out_dtype, int64_t out_token_stride, int64_t out_head_stride, void *stream);

/* How frequencies f_i = base^(-2i/rot_dim) are scaled for contexts longer than the model's own. */
typedef enum {
  DBS_ROPE_PLAIN = 0,   /* not at all */
  DBS_ROPE_LINEAR = 1,  /* f / factor */
  DBS_ROPE_BASE = 2,    /* base * factor^(rot_dim / (rot_dim - 2)) in place of base */
  DBS_ROPE_BANDS = 3,   /* by the turns t = context * f / (2 pi) that pair i makes over the model's own
                           context: t < low: f / factor; t > high: f; between them f ((1 - w) / factor + w),
                           w = (t - low) / (high - low) */
  DBS_ROPE_RAMP = 4     /* by pair index: f up to pair `first`, f / factor from pair `last`, a linear ramp
                           between, first = max(floor(d(high)), 0), last = min(ceil(d(low)), rot_dim - 1),
                           d(t) = rot_dim ln(context / (2 pi t)) / (2 ln base); if last <= first,
                           f / factor behind pair `first`; *scale = 0.1 ln(factor) + 1 */
} dbs_rope_scaling;

typedef struct {
  int32_t rot_dim;   /* even, 2 <= rot_dim <= DBS_ROPE_MAX_DIM */
  int32_t scaling;   /* a dbs_rope_scaling */
  double base;       /* > 1 */
  double factor;     /* >= 1, all but PLAIN */
  double low, high;  /* 0 < low < high, BANDS and RAMP */
  double context;    /* > 0, BANDS and RAMP: positions of the model's own context */
} dbs_rope_options;

/* Fills freq[rot_dim/2] (HOST memory) and *scale (may be NULL; 1 but for RAMP).  Touches no device. */
dbs_status dbs_rope_frequencies(const dbs_rope_options *opt, double *freq, float *scale);

/* one part of dbs_norm_rope: the query or the key heads of the tokens, as dbs_rope's x and out */
typedef struct {
  const void *x;
  int64_t x_token_stride, x_head_stride;
  void *out;
  int64_t out_token_stride, out_head_stride;
  int32_t heads;        /* >= 0 */
  const void *weight;   /* device [head_dim], or NULL: ones */
} dbs_norm_part;

/*
 * dbs_norm_rope — the root mean square norm of each head, then its rotary
 * positions, in one pass over one or two parts (queries and keys):
 *
 *   y = w * x / sqrt(mean(x^2) + eps),  then y as dbs_rope's x
 *
 * in fp32 with one rounding to the output's type; the mean is over the
 * head's head_dim elements.  A sum of squares past fp32 (elements around 2^63
 * and above) makes the head's finite elements 0; with eps = 0 the mean has to be
 * one that fp32 holds (elements around 2^-63 and above), or results are
 * infinite, and those of zeros NaN.  A weight that is held as its distance from 1 is
 * given as 1 + w.  head_dim <= DBS_ROPE_MAX_DIM, eps >= 0 and finite; a
 * negative position leaves the token's rows as they are.  A part's out may
 * be its x itself; otherwise, and between the parts, outputs share nothing
 * with inputs or each other: parts of one buffer, as the queries and keys
 * of a fused projection's rows, have the same token stride, and what a token
 * of one spans from its first head to its last lies apart from the other's.
 */
dbs_status dbs_norm_rope(int32_t tokens, int32_t head_dim, int32_t rot_dim, dbs_rope_layout layout,
                         const int32_t *pos, const double *freq, float scale, float eps,
                         const dbs_norm_part *parts, int32_t count, dbs_dtype x_dtype, dbs_dtype out_dtype,
                         dbs_dtype weight_dtype, void *stream);

/* ------------------------------------------------------------------------
 * A paged cache of keys and values in 4 bits, and the attention over it.  As
 * above, the calls allocate nothing, run on the current device, may be
 * captured and give the same bits for the same arguments; what scratch the attention
 * uses is the caller's workspace.
 *
 * A group (32, 64 or 128 channels of a head of a token; the last one may be
 * cut) is held as codes q, a scale s and an offset b, and stands for
 *
 *   x = half(s q + b),  b = half(min), s = half((max - b) (1/15)),
 *                       q = rint((x - b) (1/s)) within 0 .. 15,  0 where s = 0
 *
 * each step in fp32, so that the bytes depend on nothing but x.  Values
 * above DBS_KV4_MAX_VALUE in size, infinities and NaN make their group NaN.
 *
 * The pool is the caller's: `pages` pages of page_tokens tokens each, all
 * key heads of them, dbs_kv4_page_bytes bytes (one layer's; the layers of a
 * model are several pools, or one with the layers' pages side by side).
 * Page p of sequence b is table[b][p]; nobody reads the entries of pages that no
 * new token sees, so the pages that a window has left may be freed and their
 * entries hold anything.  An entry outside [0, pages) stands for no page: what a call would
 * store there is dropped, and its tokens are seen by nobody.
 *
 * The new tokens of a call are the last ones of their sequences: row
 * new_ptr[b] + i of the call is token lens[b] - n + i of sequence b, i < n =
 * new_ptr[b+1] - new_ptr[b]; without new_ptr, n = tokens / sequences for all.
 * lens counts the new tokens.  A length is taken as at most what the table
 * has room for.  Tokens before the first (lens[b] < n) are stored nowhere and see nothing.
 *
 * Layout of a page, for each key head in turn (d = head_dim rounded up to
 * 64, 96, 128, 192 or 256, whose last channels have codes 0; a word has eight
 * nibbles e, the lowest first):
 *   key codes      uint32[page_tokens][4 g][d/32 k]     nibble e: channel 32 k + 8 g + e
 *   key records    half[page_tokens][d/group][2]        s, b
 *   value codes    uint32[page_tokens/8][16 c][d/16 n]  nibble e: channel 16 n + c of token 8 t + e
 *   value records  half[page_tokens/8][d/group][2][8]   s, b; of tokens 0 4 1 5 2 6 3 7
 * ------------------------------------------------------------------------ */
#define DBS_KV4_MAX_VALUE 65024.0f
#define DBS_KV4_MAX_DIM 256
/* tokens that a row of the table has room for, sequences, and tokens * heads of a call at most */
#define DBS_KV4_MAX_CONTEXT 1073741824
#define DBS_KV4_MAX_SEQUENCES 1048576
#define DBS_KV4_MAX_ROWS 16777216
/* bytes of the attention's workspace at most */
#define DBS_KV4_MAX_WORKSPACE 536870912

typedef struct {
  void *pool;              /* device, 16-byte aligned */
  int64_t page_stride;     /* bytes from page to page, a multiple of 16, >= dbs_kv4_page_bytes */
  int32_t pages;
  int32_t page_tokens;     /* 16, 32, 64, 128 or 256 */
  int32_t key_heads;
  int32_t head_dim;        /* 8 to DBS_KV4_MAX_DIM, a multiple of 8 */
  int32_t group;           /* 32, 64 or 128, a divisor of d */
  int32_t sequences;
  int32_t table_pages;     /* entries of a row of the table */
  const int32_t *table;    /* device int32[sequences][table_pages], row stride ldtable */
  int64_t ldtable;
  const int32_t *lens;     /* device int32[sequences] */
  const int32_t *new_ptr;  /* device int32[sequences+1], not decreasing; NULL: as many new tokens each */
} dbs_kv4_cache;

/* Bytes of a page of one layer.  Touches no device. */
dbs_status dbs_kv4_page_bytes(int32_t key_heads, int32_t head_dim, int32_t group, int32_t page_tokens,
                              int64_t *bytes);

/*
 * dbs_kv4_store — keys and values of the new tokens into their pages, which
 * must be there.  k and v are [tokens][key_heads][head_dim] with free token
 * and head strides.  k_out and v_out, if not NULL, receive what the cache
 * now stands for, rounded to their type (also for what is stored nowhere), so
 * that a prompt's attention can be computed elsewhere from what later steps
 * will read; they may be k and v themselves (same type and strides), else they share no element with them.
 * No page that is written may stand twice in the rows of the table.
 */
dbs_status dbs_kv4_store(const dbs_kv4_cache *cache, int32_t tokens, const void *k, int64_t k_token_stride,
                         int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                         dbs_dtype x_dtype, void *k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                         void *v_out, int64_t v_out_token_stride, int64_t v_out_head_stride,
                         dbs_dtype out_dtype, void *stream);

/*
 * dbs_kv4_attention — softmax attention of the new tokens, stored before, over
 * their sequences:
 *
 *   out_ih = sum_j p_ihj v_j,  p_ih. = softmax over the tokens j that i sees of scale q_ih k_j
 *
 * where query head h reads key head h / (heads / key_heads) and the token at position i
 * sees j <= i and, if window > 0, of these j > i - window and j < sinks (a few
 * first tokens that stay visible).  A row that sees nothing is 0, rows of no sequence
 * (before new_ptr[0], new_ptr[sequences] and behind) are left as they are.  What a row does not
 * see takes no part in it, whatever it holds.  A row that sees a group of values of which a code would be no finite half
 * has NaN, or what the formula gives, in that group's channels.
 *
 *   heads      a multiple of key_heads, tokens * heads <= DBS_KV4_MAX_ROWS; sequences * key_heads and what
 *              tokens * heads / 64 adds stay within 2^23, else DBS_ERR_UNSUPPORTED
 *   q, out     device [tokens][heads][head_dim], free token and head strides, apart
 *   scale      > 0, finite when multiplied by log2 e, usually 1/sqrt(head_dim)
 *   max_len    the host's bound of lens, or 0: the table's room.  It only tells how the work is cut:
 *              longer sequences are right, and slower, and so are those that are far shorter (one
 *              token of 1500 in a table of 131072: 19 us, 9.4 with a bound of 1500)
 *   workspace  device, 16-byte aligned, of dbs_kv4_attention_workspace bytes for these arguments (DBS_KV4_MAX_WORKSPACE at most); with
 *              fewer (NULL and 0 among them) the work is not cut along the tokens, which is slower for long ones and few
 *              rows.  Calls that may overlap in time need workspaces of their own.
 *
 * Keys and values enter the matrix cores as the halves that the cache stands for, q as a half
 * with its row's largest element below 2^15 and exponentials as halves, of which both are in
 * two parts where q or out is fp32.  Sums, maxima and the output are held in fp32.  What a weight loses
 * as halves is at most 2^-11 of it (2^-23 in two parts), or 2^-35 of its row's largest: beside one that is far above
 * all others, a weight below 2^-35 of it counts as 0.
 */
dbs_status dbs_kv4_attention_workspace(const dbs_kv4_cache *cache, int32_t tokens, int32_t heads,
                                       dbs_dtype q_dtype, dbs_dtype out_dtype, int32_t window, int32_t sinks,
                                       int32_t max_len, int64_t *bytes);
dbs_status dbs_kv4_attention(const dbs_kv4_cache *cache, int32_t tokens, int32_t heads, const void *q,
                             dbs_dtype q_dtype, int64_t q_token_stride, int64_t q_head_stride, void *out,
                             dbs_dtype out_dtype, int64_t out_token_stride, int64_t out_head_stride, float scale,
                             int32_t window, int32_t sinks, int32_t max_len, void *workspace,
                             int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DBS_H */
