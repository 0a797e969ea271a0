/*
 * w12.h - C ABI of libw12: the W12 lossless 12-bit BF16 weight format on MI355X (gfx950).
 *
 * The format (SpecPilot, arXiv 2611.02501; summary page, method bullet of section 4.1, and
 * the news article part "(1) W12"): a 12-bit record per BF16 weight,
 *   sign (1 bit) | exponent minus the channel's window base (4 bits, a window of 16
 *   binades per output channel) | top 7 mantissa bits,
 * plus an exact side list (the escapes) for weights the record cannot hold: exponents
 * outside the window, zeros, subnormals and inf/NaN.  Loading compares each decoded tensor
 * with its source bit for bit (summary page, result bullet of section 4.1); the GEMM decodes
 * records in registers and reduces its K split in a fixed order, so its bits repeat from run
 * to run (method bullet of section 4.1).
 *
 * Logical format (what every result is defined on):
 *   base[n]        window base exponent field b_n in 1..239; the window is [b_n, b_n+15].
 *                  b_n is the smallest b that maximises the number of in-window weights.
 *   rec[n][k]      (s << 11) | ((e - b_n) << 7) | m for in-window weights, 0 at escapes.
 *   esc_ptr[N+1]   exclusive prefix sum of per-channel escape counts (esc_ptr[0] = 0).
 *   esc[E]         (k << 16) | bf16_bits, channel after channel, ascending k in a channel.
 *
 * Physical layout W12_LAYOUT_RB16_K16 (this library's choice; w12_unpack_records gives the
 * logical records back).  Rows are grouped in row blocks of 16 (Nb = ceil(N/16)) and k in
 * chunks of 16 (Kc = ceil(K/16)); rows >= N and k >= K are padding with record 0.
 *   hi: uint8 [Nb][Kc][16 rows][16]  byte j of row r = rec >> 4 = s | off(4) | m[6:4]
 *       (also the nested 8-bit view of each weight).
 *   lo: uint8 [Nb][Kc][16 rows][8]   the low mantissa nibbles rec & 0xF of the 16 weights:
 *       byte 4d+i (d = 0,1; i = 0..3) holds weight 8d+i in its high nibble and weight
 *       8d+4+i in its low nibble.
 *
 * Conventions for every call:
 *   - All pointers are device pointers owned by the caller; the library never allocates
 *     and never frees.  BF16 data is passed as uint16_t bit patterns.
 *   - Every call that takes a stream only validates on the host and enqueues kernels on
 *     that stream; it returns before the GPU work finishes.  No call synchronises.
 *   - Return value: W12_OK (0) or a negative W12_ERR_* code.  Arguments are validated
 *     before any HIP call; on an error nothing is enqueued.  w12_last_error() gives a
 *     message for the last failing call of the calling thread.
 *   - Row pitches (ldw, ldx, ldo, ldr, ldy) are in elements.  BF16 matrices read or
 *     written with vector accesses (W, X, decode output, verify reference) need a
 *     16-byte aligned base pointer and a pitch that is a multiple of 8 elements.
 *   - Shapes: 1 <= N <= 2^24, 1 <= K <= 65536 (k fits the 16-bit field of an escape
 *     entry), N*K < 2^32 (escape counts are 32-bit); 1 <= M <= 4096 for the GEMM, whose
 *     X and Y must each span fewer than 2^29 elements ((M-1)*pitch + row length).
 */
#ifndef W12_H
#define W12_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define W12_OK 0
#define W12_ERR_INVALID_ARG (-1)          /* null pointer, bad pitch, bad descriptor        */
#define W12_ERR_UNSUPPORTED_SHAPE (-2)    /* N, K or M outside the supported ranges          */
#define W12_ERR_WORKSPACE_TOO_SMALL (-3)  /* ws_bytes below w12_gemm_workspace_size          */
#define W12_ERR_HIP (-4)                  /* a HIP runtime call or kernel launch failed      */
#define W12_ERR_MISALIGNED (-5)           /* a vector-accessed pointer or pitch is unaligned */
#define W12_ERR_IO (-6)                   /* a checkpoint file could not be read or written  */

#define W12_LAYOUT_RB16_K16 1

/* Descriptor of an encoded tensor.  All arrays are device memory owned by the caller. */
typedef struct w12_tensor {
  int32_t N, K;          /* logical shape of W[N][K]                                     */
  int32_t layout;        /* W12_LAYOUT_RB16_K16                                          */
  int32_t reserved;      /* must be 0                                                    */
  int64_t num_escapes;   /* E = esc_ptr[N], below 2^30                                   */
  uint8_t *base;         /* [N]                                                          */
  uint8_t *hi;           /* [w12_layout_bytes().hi_bytes]                                */
  uint8_t *lo;           /* [w12_layout_bytes().lo_bytes]                                */
  uint32_t *esc_ptr;     /* [N+1]                                                        */
  uint32_t *esc;         /* [E] (may be NULL when E == 0)                                */
} w12_tensor;

/* Sizes of the hi and lo planes of the physical layout for W[N][K].  Host only. */
int w12_layout_bytes(int32_t N, int32_t K, uint64_t *hi_bytes, uint64_t *lo_bytes);

/*
 * Encode pass 1 (window choice, summary page method bullet of section 4.1; news article
 * "(1) W12": exponents cluster within a channel).  For every channel n of the BF16 matrix
 * W (row pitch ldw) computes base[n] (or copies forced_base[n] when forced_base is not
 * NULL - a test hook; each value must be in 1..239) and writes
 *   esc_ptr[0] = 0, esc_ptr[n+1] = sum_{i<=n} (K - in-window count of channel i).
 * The caller reads E = esc_ptr[N] back to size esc[] before w12_encode_emit.
 * forced_base values outside 1..239 are clamped into range by the kernel (the host
 * cannot inspect device memory without synchronising).
 */
int w12_encode_count(const uint16_t *W, int32_t N, int32_t K, int64_t ldw,
                     const uint8_t *forced_base, uint8_t *base, uint32_t *esc_ptr,
                     hipStream_t stream);

/*
 * Encode pass 2 (records and escape list, summary page method bullet of section 4.1).
 * Reads W and t->base / t->esc_ptr written by w12_encode_count and writes t->hi, t->lo
 * (padding included) and t->esc.  Escapes of a channel are compacted in ascending k with
 * wavefront prefix sums.  t->num_escapes must equal esc_ptr[N].
 */
int w12_encode_emit(const uint16_t *W, int64_t ldw, const w12_tensor *t, hipStream_t stream);

/*
 * Full-tensor decode (summary page result bullet of section 4.1: decoded tensors are the
 * original weights bit for bit).  Writes out[n][k] (row pitch ldo) for n < N, k < K.
 * The escape list must be well formed (ascending k < K per channel); w12_verify checks it.
 */
int w12_decode(const w12_tensor *t, uint16_t *out, int64_t ldo, hipStream_t stream);

/*
 * Load-time bit-for-bit check (summary page result bullet of section 4.1).  Decodes t and
 * compares with ref (row pitch ldr).  Writes, on the device,
 *   d_result[0] = number of positions (n,k) whose decoded bits differ from ref[n][k]
 *                 plus the number of malformed escape entries (k >= K, k not above the k
 *                 of the entry before it in its channel, non-zero record under an escape) plus
 *                 the number of inconsistent pointers (esc_ptr[0] != 0, a decreasing
 *                 step, esc_ptr[N] != num_escapes);
 *   d_result[1] = smallest flat index n*K + k of a differing position, or
 *                 0xFFFFFFFFFFFFFFFF if there is none.
 * d_result must point to 2 device uint64 values; the call resets them first.
 */
int w12_verify(const w12_tensor *t, const uint16_t *ref, int64_t ldr,
               unsigned long long *d_result, hipStream_t stream);

/* Test aid: writes the logical 12-bit records rec[n][k] (row pitch ldr, uint16) of the
 * physical planes, so parity with an implementation of the logical format does not
 * depend on this library's layout. */
int w12_unpack_records(const w12_tensor *t, uint16_t *rec, int64_t ldr, hipStream_t stream);

/* Bytes of device workspace w12_gemm needs for M rows of X against W[N][K]. Host only.
 * The workspace starts with a 16 KB region of 32-bit arrival counters (split-K bookkeeping;
 * the same region for every plan, single or grouped) followed by the FP32 slice partials
 * and, where the plan needs it, a copy of X that the call writes itself: for M >= 65 X
 * rearranged into the matrix cores' operand order, otherwise, for K % 16 != 0, X padded
 * with zeros to whole 16-k chunks.
 * The size follows the plan, so a change of W12_GEMV_MAX_M between sizing and calling can
 * make the workspace too small (reported as W12_ERR_WORKSPACE_TOO_SMALL). */
int w12_gemm_workspace_size(int32_t M, int32_t N, int32_t K, uint64_t *bytes);

/* Zero-fill a GEMM workspace of ws_bytes bytes on `stream`.  Call it once after allocating
 * the workspace: w12_gemm needs the counter region to be zero on entry and leaves it zero
 * when it completes, so the workspace can then serve any sequence of w12_gemm calls on one
 * stream.  Calls that overlap in time on one workspace race. */
int w12_gemm_workspace_init(void *ws, uint64_t ws_bytes, hipStream_t stream);

/*
 * Y[m][n] = sum_k X[m][k] * W[n][k] for m < M, n < N (summary page method bullet of
 * section 4.1: the GEMM decodes W12 records in registers and reduces in a fixed order).
 * X: BF16 [M][ldx]; Y: FP32 [M][ldy], every Y[m][n] (n < N) is written.  Accumulation is
 * FP32; the result is within 2^-12 * sum_k |x w| of the exact sum and bitwise identical
 * from run to run on the same device for the same (M, N, K).  M <= 2 runs a wavefront
 * GEMV (FP32 dot2 products and a fixed-order wavefront reduction), larger M runs bf16 MFMA
 * tiles; the environment variable W12_GEMV_MAX_M (0..8, read at each call) moves that
 * boundary, and W12_MAX_GRID (read at each call) caps the number of work-groups.  The K range may be split over several work-groups;
 * the last one to finish a tile sums the slice partials in increasing slice order (no
 * floating-point atomics).  ws: device workspace of at least w12_gemm_workspace_size bytes,
 * initialised once with w12_gemm_workspace_init (only its counter region must be zero; the
 * partial region may hold anything on entry).
 */
int w12_gemm(const uint16_t *X, int32_t M, int64_t ldx, const w12_tensor *t,
             float *Y, int64_t ldy, void *ws, uint64_t ws_bytes, hipStream_t stream);

/*
 * The Q pass of two-level verification (news article, two-level verification part: the
 * first pass verifies at low precision with the 8-bit weight view nested in W12 and accepts
 * nothing).  Y = X . Wq^T, where Wq is W with every in-window weight read through the
 * record's top byte (sign, exponent offset, three mantissa bits), i.e. truncated toward zero
 * to four significant bits, and every escaped weight exact.  Only the hi plane of the records
 * is read (1 byte per weight).  Same arguments, layouts, workspace, errors, tolerance (against
 * the FP64 product with Wq) and run-to-run determinism as w12_gemm.
 */
int w12_gemm_q(const uint16_t *X, int32_t M, int64_t ldx, const w12_tensor *t,
               float *Y, int64_t ldy, void *ws, uint64_t ws_bytes, hipStream_t stream);

/*
 * w12_gemm for callers that cannot allocate device memory: code under stream capture, tight
 * serving loops, harnesses that forbid hipMalloc.  Same arguments (minus the workspace),
 * layouts, errors, tolerance and result as w12_gemm: Y is bitwise identical to w12_gemm's for
 * the same operands.  The workspace is a 32 MiB array held by the library on each device (kept
 * until the process ends); it covers every M <= 64 (the streaming tiles) with K <= 64,000 at the
 * default launch shape, and a product whose plan needs more is rejected with W12_ERR_WORKSPACE_TOO_SMALL (call w12_gemm
 * with a workspace instead).  Nothing is allocated: the first call on a device looks up the
 * array's address and clears its counter region on `stream` (a kernel launch); every call
 * leaves it clear.  All calls on one device share the one array, so calls that overlap in time
 * on one device (on different streams or host threads) race.
 */
int w12_gemm_noalloc(const uint16_t *X, int32_t M, int64_t ldx, const w12_tensor *t,
                     float *Y, int64_t ldy, hipStream_t stream);

/*
 * Grouped launch: several independent products of the same M in one launch (summary page
 * method bullet of section 4.1: the W12 GEMM is a stream-K GEMM whose split is reduced in a
 * fixed order).  items[i] asks for Y_i = X_i . W_i^T exactly as w12_gemm would (same operand
 * layouts, pitches and alignment rules, the same tolerance); the launch streams the W12 records
 * of all count products under one stream-K schedule over their concatenated work units, so the
 * pipeline fill, the tail and the split-K fixups are paid once per launch rather than once per
 * product.  Each Y_i is bitwise identical from run to run for the same (M, shapes, order of the
 * items), though not in general bitwise equal to w12_gemm's result (the K split points differ).
 * The products must not depend on one another: no Y_i may overlap any X_j or W_j of the group.
 * Limits: 1 <= count <= W12_GROUP_MAX; 1 <= M <= 64; every K a multiple of 16.  Outside them
 * the call returns W12_ERR_UNSUPPORTED_SHAPE.  items and the descriptors they point to are host
 * memory read during the call only.  ws: at least w12_gemm_group_workspace_size bytes,
 * initialised once with w12_gemm_workspace_init (counters at its start; every call leaves them
 * zero).  Up to W12_GROUP_INLINE products travel in the kernel arguments; a larger group (a
 * whole model, say) first stores its per-product argument blocks (about 200 bytes each) at the
 * end of the workspace, with one small kernel per W12_GROUP_INLINE products on `stream`, so the
 * workspace of such a group carries that region too.  W12_GEMV_MAX_M, W12_GROUPS_PER_CU and
 * W12_MAX_GRID apply as for w12_gemm.
 */
#define W12_GROUP_MAX 1024
#define W12_GROUP_INLINE 8
typedef struct w12_gemm_item {
  const uint16_t *X;     /* BF16 [M][ldx], device                                          */
  int64_t ldx;
  const w12_tensor *t;   /* host descriptor of W_i (device planes)                         */
  float *Y;              /* FP32 [M][ldy], device                                          */
  int64_t ldy;
} w12_gemm_item;
int w12_gemm_group_workspace_size(int32_t M, int32_t count, const w12_gemm_item *items, uint64_t *bytes);
int w12_gemm_group(int32_t M, int32_t count, const w12_gemm_item *items, void *ws, uint64_t ws_bytes,
                   hipStream_t stream);
/* The Q pass (as w12_gemm_q) of every product of a group, in one launch. */
int w12_gemm_group_q(int32_t M, int32_t count, const w12_gemm_item *items, void *ws, uint64_t ws_bytes,
                     hipStream_t stream);

/* How w12_gemm will run (M, N, K).  Host only. */
typedef struct w12_gemm_plan_info {
  int32_t path;              /* 1 = wavefront GEMV, 2 = MFMA tiles, 3 = wide MFMA tiles  */
  int32_t splits;            /* most K slices (partial sums) of one output tile          */
  int32_t rows_per_block;    /* rows of W per work-group tile                            */
  int32_t m_tile;            /* rows of X per work-group tile                            */
  int64_t grid;              /* work-groups launched                                     */
  uint64_t workspace_bytes;  /* == w12_gemm_workspace_size                               */
  uint64_t counter_bytes;    /* leading bytes of the workspace holding the counters (the
                                same for every plan)                                      */
} w12_gemm_plan_info;
int w12_gemm_plan(int32_t M, int32_t N, int32_t K, w12_gemm_plan_info *info);

/*
 * W12 checkpoint files (summary page, result bullet of section 4.1: converted layers are
 * checked bit for bit when they are loaded).  A file holds named encoded tensors in the
 * physical layout above: a 64-byte header (magic "W12CKPT1", version 1, tensor count), one
 * 128-byte index entry per tensor, then per tensor its base, esc_ptr, esc, hi and lo arrays,
 * each starting on a 256-byte boundary.  Integers are little-endian.
 */
typedef struct w12_file_entry {
  char name[64];         /* NUL-terminated (at most 63 characters are stored)           */
  int32_t N, K;
  int32_t layout;        /* W12_LAYOUT_RB16_K16                                          */
  int32_t reserved;
  int64_t num_escapes;
  uint64_t offset;       /* file offset of the tensor's data                             */
  uint64_t bytes;        /* bytes of the tensor's data (sections and their padding)      */
} w12_file_entry;

/* Write count tensors to path (created or truncated).  Every array of host_tensors[i] is HOST
 * memory (copy the planes back from the device first); names[i] are C strings.  Synchronous;
 * W12_ERR_IO on a failed open or write. */
int w12_file_write(const char *path, int32_t count, const char *const *names, const w12_tensor *host_tensors);

/* Read the index of path: *count receives the number of tensors; when entries is not NULL the
 * first *count entries are written (W12_ERR_INVALID_ARG if *count > max_entries).  Synchronous. */
int w12_file_index(const char *path, int32_t *count, w12_file_entry *entries, int32_t max_entries);

/*
 * Streamed load.  For i < count, copies tensor which[i] of the file into the device arrays of
 * dst[i] (N, K, layout and num_escapes must equal the index entry; the caller sizes the arrays
 * from the entry).  The file is read on the calling thread in pieces of staging_bytes / 2
 * into alternating halves of `staging` (pinned host memory of at least 512 bytes), each piece
 * copied to the device on `stream`; a half is refilled only after its previous copy has
 * completed.  When refs is not NULL and refs[i] is not NULL, the load-time check of dst[i]
 * against the BF16 matrix refs[i] (device, row pitch ldr[i]) is enqueued on `stream` right
 * after the tensor's copies, with w12_verify's semantics, into d_results[2i], d_results[2i+1]
 * (device; 2*count values).  The call returns once every copy has been enqueued and the
 * staging buffer is no longer read; the checks may still be running.  Creates and destroys
 * two HIP events; allocates no memory.  W12_ERR_IO on a read failure or a malformed file.
 */
int w12_file_load(const char *path, int32_t count, const int32_t *which, const w12_tensor *dst,
                  void *staging, uint64_t staging_bytes, const uint16_t *const *refs, const int64_t *ldr,
                  unsigned long long *d_results, hipStream_t stream);

/*
 * Measurement aid (not part of the format): a plain streaming read of buf[0, bytes) by
 * groups_per_cu 256-thread work-groups per compute unit, each reading a contiguous share with
 * 16-byte loads (1 KB of consecutive bytes per wave instruction) and keeping loads_per_lane
 * (1, 2, 4, 8 or 16) loads in flight per lane.  It gives the practical HBM read ceiling that the
 * GEMM's bytes moved per second are compared with.  buf: device, 16-byte aligned; bytes: a
 * multiple of 16, 16 <= bytes <= 2^31; groups_per_cu: 1..16; sink: device, at least
 * groups_per_cu * (compute units) uint32 values, never written in practice (the loaded data
 * is folded into a value that is stored only if it equals a fixed constant).
 */
int w12_read_probe(const void *buf, uint64_t bytes, int32_t loads_per_lane, int32_t groups_per_cu,
                   uint32_t *sink, hipStream_t stream);

/*
 * Operators around the products in one step of speculative decoding: a layer's residual addition
 * and RMS norm, rotary positions with the write into a paged cache, attention of a chain or tree
 * of drafted tokens over that cache, and an 8-bit product for layers that are kept in 8 bits (a
 * drafter's; the target's weights are W12).  All conventions above apply.  Matrices here are
 * accessed with 16-byte vectors: base pointers are 16-byte aligned and pitches are multiples of
 * 16 bytes unless an argument says otherwise.  Nothing past the last element of a row is written;
 * what lies between rows, or in the 16-byte step that holds an operand's last element, may be read
 * and never counts.  E4M3 is the 8-bit OCP format with 3 mantissa bits (largest value 448).
 */
#define W12_DTYPE_BF16 0
#define W12_DTYPE_F32 1
#define W12_DTYPE_E4M3 2
#define W12_QUANT_BLOCK 128   /* values that share a scale along a row */

/*
 * r = residual + delta (delta NULL: r = residual), y[m][n] = r[m][n] / sqrt(mean_n(r[m]^2) + eps)
 * * weight[n].  Sums and the norm are FP32; the norm takes r before it is rounded for storage.
 *   residual_out  r rounded to the residual's type; NULL: not stored; may be residual itself
 *                 (in place) but may not overlap it otherwise.
 *   y             BF16 (an operand of w12_gemm), or NULL.
 *   yq, yq_scale  E4M3 with one FP32 scale per row and block of 128 columns (an operand of
 *                 w12_gemm_e4m3), or both NULL: yq_scale[m][b] = max|y| of the block / 448 (1
 *                 where that is 0 in FP32: a block of zeros, or of nothing above 3.1e-43),
 *                 yq = y / yq_scale rounded to nearest even, cut off at +-448 (a scale below the
 *                 normal range is rounded coarsely).  y is taken before it is rounded to BF16.  A
 *                 NaN or infinity in a block makes its scale NaN or infinite.
 * At least one of y, yq and residual_out with a delta is wanted.  1 <= M <= 2^20, 1 <= N <= 65536.
 */
typedef struct w12_norm_args {
  int32_t M, N;
  int32_t residual_dtype;        /* W12_DTYPE_BF16 or W12_DTYPE_F32: residual, residual_out */
  int32_t delta_dtype;           /* W12_DTYPE_BF16 or W12_DTYPE_F32                          */
  const void *residual;          /* [M][ld_residual]                                         */
  int64_t ld_residual;
  const void *delta;             /* [M][ld_delta] or NULL                                    */
  int64_t ld_delta;
  const uint16_t *weight;        /* BF16 [N]                                                 */
  void *residual_out;            /* [M][ld_residual_out] or NULL                             */
  int64_t ld_residual_out;
  uint16_t *y;                   /* BF16 [M][ldy] or NULL                                    */
  int64_t ldy;
  uint8_t *yq;                   /* E4M3 [M][ldyq] or NULL                                   */
  int64_t ldyq;
  float *yq_scale;               /* [M][ld_scale], ld_scale >= ceil(N / 128), 4-byte aligned */
  int64_t ld_scale;
  float eps;                     /* >= 0                                                     */
  int32_t reserved;              /* must be 0                                                */
} w12_norm_args;
int w12_add_rmsnorm(const w12_norm_args *a, hipStream_t stream);

/*
 * A paged key / value cache.  Element (page p, token t of the page, head h, i) of K and of V is at
 * p * page_stride + t * token_stride + h * head_stride + i elements (so tokens or heads may come
 * first in a page).  E4M3 caches hold value / scale[h]; the scales are fixed when the cache is made.
 */
typedef struct w12_kv_cache {
  int32_t dtype;                 /* W12_DTYPE_BF16 or W12_DTYPE_E4M3                         */
  int32_t pages;                 /* 1 .. 2^31 - 1                                            */
  int32_t page_size;             /* tokens of a page: a power of two, 1 .. 1024              */
  int32_t heads;                 /* 1 .. 1024                                                */
  int32_t dim;                   /* 64, 128 or 256                                           */
  int32_t reserved;              /* must be 0                                                */
  int64_t page_stride, token_stride, head_stride;   /* elements, multiples of 16 bytes, >= 0  */
  void *k, *v;
  const float *k_scale, *v_scale;                   /* [heads], E4M3 only                     */
} w12_kv_cache;

/*
 * Takes T rows of a QKV product (q_heads query heads, then the cache's heads of K, then of V),
 * turns Q and K by their positions, stores Q as BF16 and puts K and V into the cache at
 * slots[t] = page * page_size + token of the page.  Rows whose slot is negative or past the cache
 * are not put (their Q is stored all the same).  The other slots must differ from one another.
 * Pair i of the first rot_dim elements of a head is (i, i + rot_dim / 2), or (2i, 2i + 1) with
 * adjacent != 0; it is turned by positions[axis[i]][t] * inv_freq[i], an angle formed in FP64 (far
 * positions keep their phase).  Several axes serve images and video (time, height, width); axis
 * NULL takes axis 0 throughout, a value past the last axis takes the last.  Elements past rot_dim
 * are copied.  E4M3 caches: value / scale[h] rounded to nearest even, cut off at +-448, NaN kept.
 * 1 <= T <= 2^20, rot_dim even, 0 <= rot_dim <= dim, 1 <= axes <= 8, 1 <= q_heads <= 4096.
 */
typedef struct w12_rope_args {
  int32_t T, q_heads;
  int32_t src_dtype;             /* W12_DTYPE_F32 (a w12_gemm result) or W12_DTYPE_BF16      */
  int32_t rot_dim, axes, adjacent;
  const void *qkv;               /* [T][ld_qkv]                                              */
  int64_t ld_qkv;
  const int32_t *positions;      /* [axes][ld_positions], ld_positions >= T                  */
  int64_t ld_positions;
  const int64_t *slots;          /* [T]                                                      */
  const double *inv_freq;        /* [rot_dim / 2], radians per position                      */
  const uint8_t *axis;           /* [rot_dim / 2] or NULL                                    */
  uint16_t *q;                   /* BF16 [T][ldq], q_heads * dim of a row written            */
  int64_t ldq;
} w12_rope_args;
int w12_rope_append(const w12_rope_args *a, const w12_kv_cache *cache, hipStream_t stream);

/*
 * Attention of drafted tokens.  Request b has the rows (nodes) node_ptr[b] .. node_ptr[b+1] - 1 of
 * q, its first ctx_len[b] tokens are in the cache, and its node i is the cache's token ctx_len[b] + i
 * (w12_rope_append put it there).  Token t of a request is in page page_table[b][t / page_size].
 * Node i attends every token before ctx_len[b], and of the nodes those whose bit is set in its
 * row of tree_mask (bit j % 64 of word j / 64 for node j; its own bit is not implied; nodes past
 * the words are not attended), or with tree_mask NULL the nodes 0..i (a chain).  Query head h
 * reads cache head h / (q_heads / heads).
 *   out[row][h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q . k_t - max).
 *   lse[row][h] = log sum_t exp(scale * q . k_t), if lse is not NULL.
 * Scores, p_t and all sums are FP32; for its product with v_t each p_t is rounded to BF16 (by up to 2^-8 of
 * itself), so that out may be off by 2^-8 of sum_t p_t |v_t| / sum_t p_t beside its own rounding.  lse has no such part.
 * What a row does not attend never reaches it, NaN and infinity included.  A row that attends
 * nothing, or whose scores are all -inf, gives zeros and lse -inf.  Tokens past max_pages * page_size, and
 * tokens whose page is not in 0 .. pages - 1, count as absent.  Rows outside every request are left as they are;
 * ranges of node_ptr are cut to 0..T and must not decrease (where they do, out and lse of the rows hold
 * anything, and nothing else is written); negative lengths count as 0.
 * node_ptr, ctx_len, page_table and tree_mask are device memory read by the kernels (a captured
 * graph follows their values).  The result is bitwise the same from run to run.
 * 1 <= T <= 2^20, 1 <= requests <= 1024, q_heads a multiple of heads (at most 64 times heads),
 * 1 <= mask_words <= 64, max_pages * page_size < 2^30.
 * ws: w12_tree_attention_workspace_size bytes, 16-byte aligned, any content; calls that overlap in
 * time need workspaces of their own.
 */
typedef struct w12_attention_args {
  int32_t T, requests, q_heads, max_pages;
  int32_t mask_words;            /* words of a tree_mask row (0 with tree_mask NULL)         */
  float scale;
  const uint16_t *q;             /* BF16 [T][ldq], head h at h * dim                         */
  int64_t ldq;
  const int32_t *node_ptr;       /* [requests + 1]                                           */
  const int32_t *ctx_len;        /* [requests]                                               */
  const int32_t *page_table;     /* [requests][ld_table]                                     */
  int64_t ld_table;
  const uint64_t *tree_mask;     /* [T][ld_mask] or NULL, 8-byte aligned                     */
  int64_t ld_mask;
  uint16_t *out;                 /* BF16 [T][ldo], head h at h * dim                         */
  int64_t ldo;
  float *lse;                    /* [T][ld_lse] or NULL, 4-byte aligned                      */
  int64_t ld_lse;
} w12_attention_args;
int w12_tree_attention_workspace_size(int32_t T, int32_t requests, int32_t q_heads, const w12_kv_cache *cache,
                                      uint64_t *bytes);
int w12_tree_attention(const w12_attention_args *a, const w12_kv_cache *cache, void *ws, uint64_t ws_bytes,
                       hipStream_t stream);

/*
 * Y[m][n] = sum_k (X[m][k] x_scale[m][k / 128]) (W[n][k] w_scale[n / 128][k / 128]) with E4M3 X and
 * W, FP32 scales, sums and Y: one scale per row and block of 128 of X (as w12_add_rmsnorm gives
 * them), one per block of 128 x 128 of W.  Bitwise the same from run to run for the same (M, N, K).
 * ldx and ldw are multiples of 16 bytes; ldxs, ldws >= ceil(K / 128), (M - 1) * ldxs + ceil(K / 128)
 * < 2^29; Y is 4-byte aligned.
 * 1 <= M <= 4096, N and K as for w12_gemm.  ws: as for w12_gemm (w12_gemm_e4m3_workspace_size bytes,
 * which serve every number of rows up to M over the same N and K; initialised once with
 * w12_gemm_workspace_init, of which the counters matter; every call leaves them zero).  A call that
 * needs less, or none, is not refused for a smaller one.  The two scales of a block are multiplied
 * first, in FP32: their product has to be a normal number or 0.
 */
int w12_gemm_e4m3_workspace_size(int32_t M, int32_t N, int32_t K, uint64_t *bytes);
int w12_gemm_e4m3(const uint8_t *X, int32_t M, int64_t ldx, const float *x_scale, int64_t ldxs, const uint8_t *W,
                  int32_t N, int32_t K, int64_t ldw, const float *w_scale, int64_t ldws, float *Y, int64_t ldy,
                  void *ws, uint64_t ws_bytes, hipStream_t stream);

/*
 * Operators of a hybrid target in speculative decoding: its recurrent layers (a short causal
 * convolution and the gated delta rule, for prompts, single tokens, and chains or trees of drafted
 * tokens) and the verification of drafted tokens.  All conventions above apply.
 *
 * Which rows of a call belong to which sequence, and where the sequences' states are.  Token i of
 * sequence b is row ptr[b] + i of the call's matrices, or row rows[ptr[b] + i] of them, for
 * i < ptr[b + 1] - ptr[b], and with lens for i < lens[b] besides.  A row outside 0 .. T - 1 counts
 * as zeros in every input, and has no output.  Outputs overlap no input.  A sequence starts from the state in slot src[b] (zeros for
 * a slot outside 0 .. slots - 1) and its new state goes to slot dst[b] (nowhere for a slot outside),
 * which may be src[b]; a sequence without tokens has its old state put there.  dst NULL: no state is stored.
 * Slots of dst must differ from one another, and from the src of other sequences; several may share
 * a src.  Where outputs are wanted, no row may be named twice.
 * Ranges of ptr are cut to 0..T and must not decrease (where they do, the outputs and the new
 * states hold anything, and nothing else is written); negative lengths count as 0.  Rows of no
 * sequence are left as they are.
 *
 * tree_mask makes every range a tree of drafted tokens in drafting order (dst, rows and lens are
 * then NULL): row r's bits below its own place name its ancestors (bit j for node j of its range,
 * as in w12_attention_args; its own bit and those above count as set and unset).  A node follows its
 * ancestors only; of a range more than 64 nodes long the rest is left as it is.  The ancestors have to be a path: a
 * node's are those of its nearest ancestor, and that ancestor (where they are not, the range's outputs hold anything).
 *
 * ptr, lens, rows, src, dst and tree_mask are device memory read by the kernels (a captured graph
 * follows their values).  1 <= T <= 2^20, 1 <= count <= 1024, 1 <= slots <= 2^20, 1 <= mask_words <= 64.
 */
#define W12_TREE_NODES 64
typedef struct w12_sequences {
  int32_t T, count;
  const int32_t *ptr;            /* [count + 1]                                              */
  const int32_t *lens;           /* [count] or NULL                                          */
  const int32_t *rows;           /* [T] or NULL                                              */
  const int32_t *src, *dst;      /* [count]; dst may be NULL                                 */
  const uint64_t *tree_mask;     /* [T][ld_mask] or NULL, 8-byte aligned                     */
  int64_t ld_mask;
  int32_t mask_words;            /* words of a tree_mask row (0 with tree_mask NULL)         */
  int32_t slots;                 /* places of the state array                                */
} w12_sequences;

/*
 * Short causal convolution of every channel: y_t = act(bias + sum_j weight[c][j] x_{t - (width - 1) + j}),
 * FP32 sums; the tokens before the sequence's first are its state, the last width - 1 rows of x (in x's
 * type, oldest first).  act: SiLU, y / (1 + exp(-y)), with silu != 0, else none.  In a tree the tokens before a node are its
 * ancestors, nearest last.  y NULL: only the states move on.  What is not in a row's window never reaches it.
 * 1 <= channels <= 2^17, 2 <= width <= 4.
 */
typedef struct w12_conv_args {
  int32_t channels, width;
  int32_t dtype;                 /* W12_DTYPE_F32 (a w12_gemm result) or W12_DTYPE_BF16: x, state */
  int32_t silu;
  const void *x;                 /* [T][ldx]                                                 */
  int64_t ldx;
  const uint16_t *weight;        /* BF16 [channels][width], 16-byte aligned                  */
  const uint16_t *bias;          /* BF16 [channels] or NULL                                  */
  void *state;                   /* [slots][width - 1][channels], 16-byte aligned            */
  int64_t slot_stride, tap_stride;   /* elements, multiples of 16 bytes; tap_stride >= channels  */
  uint16_t *y;                   /* BF16 [T][ldy] or NULL                                    */
  int64_t ldy;
} w12_conv_args;
int w12_short_conv(const w12_conv_args *a, const w12_sequences *s, hipStream_t stream);

/*
 * The gated delta rule.  Every value head h of a sequence has a state S of dk x dv, kept transposed:
 * state[slot][h][j][i] = S[i][j], FP32.  A token with key k (of key head h / (v_heads / k_heads)), value v,
 * log decay g, strength beta and query q turns it into
 *   S' = exp(g) S + k (beta (v - exp(g) S^T k))^T      and gives      out = scale S'^T q.
 * With l2norm, k and q are divided by sqrt(sum of squares + eps) first.  In a tree S is the state behind the node's parent.
 * The states are FP32 throughout.  Tokens of a tree or a long range are taken 64 at a time, as a triangular system
 *   u_i + beta_i sum_{j before i} exp(G_i - G_j) (k_i . k_j) u_j = beta_i (v_i - exp(G_i) S^T k_i),  G_i the sum of g up to i,
 * with BF16 matrix instructions: q, k and v are exact in them, what is FP32 (S, u, the system's inverse and the q . k factors) goes
 * in as two BF16 values, off by 2^-16 of each value at most; out is rounded once, as token by token.  Sums of squares are FP32:
 * a key whose sum passes that is no number, and with l2norm also a key or query whose sum + eps is under 2^-126 (eps 0).
 * g <= 0 is expected.  The rule itself grows without bound where beta |k|^2 passes 2.  A NaN or infinity in a row reaches
 * that row and those that come after it in its sequence (in a tree: its descendants), and the new state; nothing else.
 * (Finite values whose u passes FP32 may reach tokens before theirs among the 64 that are taken together.)
 * q and out NULL: only the states move on.  The result is bitwise the same from run to run.
 * dk: 64 or 128, dv: 64, 128 or 256, v_heads a multiple of k_heads, at most 1024.
 * ws: w12_gated_delta_workspace_size bytes for T rows in count sequences (or more), 16-byte aligned, any content; calls
 * that overlap in time need workspaces of their own.  A call with a tree or of T >= W12_DELTA_CHUNK_FROM * count rows (with lens:
 * W12_DELTA_CHUNK_FROM_LENS * count) has to have it, and one without lens and with T - count + 1 >= W12_DELTA_CHUNK_LONG, in which a sequence can be
 * long beside short ones, should.  Such a call takes trees, and each sequence that has W12_DELTA_CHUNK_FROM tokens or more itself (after lens),
 * 64 at a time and the others token by token: a sequence's result does not depend, bit for bit, on those that share the call.  Every
 * other call, and one of fewer than W12_DELTA_CHUNK_FROM * count rows whose ws is NULL or too small, takes all tokens one by one and needs no
 * workspace.  Either form rounds out once.
 */
#define W12_DELTA_CHUNK_FROM 12
#define W12_DELTA_CHUNK_FROM_LENS 65
#define W12_DELTA_CHUNK_LONG 64
typedef struct w12_delta_args {
  int32_t k_heads, v_heads, dk, dv;
  int32_t l2norm;
  float eps, scale;              /* eps >= 0, scale finite                                   */
  int32_t reserved;              /* must be 0                                                */
  const uint16_t *q;             /* BF16 [T][ldq], head h at h * dk; or NULL                 */
  int64_t ldq;
  const uint16_t *k;             /* BF16 [T][ldk], head h at h * dk                          */
  int64_t ldk;
  const uint16_t *v;             /* BF16 [T][ldv], head h at h * dv                          */
  int64_t ldv;
  const float *g;                /* [T][ldg]                                                 */
  int64_t ldg;
  const float *beta;             /* [T][ldbeta]                                              */
  int64_t ldbeta;
  float *state;                  /* [slots][v_heads][dv][dk], slots slot_stride apart        */
  int64_t slot_stride;           /* elements, a multiple of 4                                */
  uint16_t *out;                 /* BF16 [T][ldo], head h at h * dv; or NULL                 */
  int64_t ldo;
} w12_delta_args;
int w12_gated_delta_workspace_size(int32_t T, int32_t count, int32_t v_heads, int32_t dk, int32_t dv, uint64_t *bytes);
int w12_gated_delta(const w12_delta_args *a, const w12_sequences *s, void *ws, uint64_t ws_bytes, hipStream_t stream);

/*
 * Verification of drafted tokens.  Request b has the nodes node_ptr[b] .. node_ptr[b + 1] - 1; node 0 is
 * its last known token, tokens[r] is row r's token, and logits[r] (of vocab tokens) is what the target says after row
 * r's node: p_r = softmax(logits[r] / temperature[b]), at temperature 0 (or less, or NaN) all of it on the largest (the lowest index of
 * equals).  A node's parent is the nearest of its ancestors in tree_mask (its bits below its own place; a node without any, but for node 0, is never
 * reached), with tree_mask NULL the node before it.  Random numbers are inputs in [0, 1): u[r] takes the first token whose
 * cumulative weight, in the order of the tokens, passes u[r] times the total.
 *   q NULL: row r's token is taken from p_r by u[r].  From node 0 on, the walk goes to the child that has the token taken at
 *     its node (the first of several), until there is none; next is the last node's token.
 *   q (chains only): q[r] is the distribution that row r's token was drawn from.  Node i is accepted where accept_u[r] q[r][x] < p[x],
 *     x its token and p the distribution after the node before it.  After the first that is not, next is taken by u of the last
 *     accepted row from max(p - q[r], 0) (from p where that is 0 throughout); after the last node, from its p.
 * path[node_ptr[b] + i], i < count[b], are the rows of the walk (node 0 first) and -1 behind them up to the request's
 * last row; count[b] their number, next_token[b] the token that follows.  path and count serve as rows and lens of w12_sequences.
 * Weights, sums and comparisons are FP64.  Logits of -inf and NaN have no weight; where one or more are
 * +inf, the first of them has all of it; a row without any weight takes no token (-1), and no child follows it.  A token outside
 * 0 .. vocab - 1 is never accepted.  u is cut to 0 .. 1 - 2^-24; NaN counts as 0.
 * A request without nodes gets count 0 and next_token -1; of one with more than 4096 nodes, the first 4096 count.  Rows of no request
 * have their path left as it is; ranges as in w12_sequences.
 * 1 <= T <= 2^20, 1 <= requests <= 1024, 1 <= vocab <= 2^24, T * vocab < 2^40.
 * ws: w12_verify_draft_workspace_size bytes for T rows (or more), 16-byte aligned, any content; calls that overlap in time need
 * workspaces of their own.
 */
#define W12_VERIFY_NODES 4096
typedef struct w12_verify_draft_args {
  int32_t T, requests, vocab;
  int32_t logits_dtype;          /* W12_DTYPE_F32 (a w12_gemm result) or W12_DTYPE_BF16      */
  const void *logits;            /* [T][ld_logits]                                           */
  int64_t ld_logits;
  const float *q;                /* [T][ldq] or NULL                                         */
  int64_t ldq;
  const int32_t *tokens;         /* [T]                                                      */
  const int32_t *node_ptr;       /* [requests + 1]                                           */
  const uint64_t *tree_mask;     /* [T][ld_mask] or NULL, 8-byte aligned                     */
  int64_t ld_mask;
  int32_t mask_words;            /* words of a tree_mask row (0 with tree_mask NULL)         */
  int32_t reserved;              /* must be 0                                                */
  const float *u;                /* [T]                                                      */
  const float *accept_u;         /* [T], with q                                              */
  const float *temperature;      /* [requests] or NULL: 1 throughout                         */
  int32_t *path;                 /* [T]                                                      */
  int32_t *count, *next_token;   /* [requests]                                               */
} w12_verify_draft_args;
int w12_verify_draft_workspace_size(int32_t T, int32_t requests, int32_t vocab, uint64_t *bytes);
int w12_verify_draft(const w12_verify_draft_args *a, void *ws, uint64_t ws_bytes, hipStream_t stream);

/* Stored bits per weight: (1.5*N*K + N + 4*(N+1) + 4*E) * 8 / (N*K).  -1 for N < 1, K < 1
 * or E < 0. */
double w12_bits_per_weight(int32_t N, int32_t K, int64_t E);

/* Bytes of the logical format for W[N][K] with E escapes: ceil(12 N K / 8) record bytes, one
 * base byte per channel, (N + 1) 4-byte escape pointers and 4 bytes per escape.  0 for N < 1,
 * K < 1 or E < 0.  (The device planes are padded to whole 16 x 16 chunks: w12_layout_bytes.) */
uint64_t w12_tensor_bytes(int32_t N, int32_t K, int64_t E);

const char *w12_status_string(int status);
const char *w12_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* W12_H */
