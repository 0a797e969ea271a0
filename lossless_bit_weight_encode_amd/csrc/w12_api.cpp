// C ABI of libw12: argument validation (host only, before any HIP call), planning and
// launches.  The declarations and their contracts are in include/w12.h.
#include <stdarg.h>
#include <stdio.h>

#include <vector>

#include "w12_device.h"
#include "w12_gemm_common.h"
#include "w12_kernels.h"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  g_err[0] = '\0';
  return W12_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxN = int64_t(1) << 24;
constexpr int64_t kMaxK = 65536;
constexpr int32_t kMaxM = 4096;

int check_shape(int64_t N, int64_t K) {
  if (N < 1 || N > kMaxN) return fail(W12_ERR_UNSUPPORTED_SHAPE, "N=%lld outside 1..%lld", (long long)N, (long long)kMaxN);
  if (K < 1 || K > kMaxK) return fail(W12_ERR_UNSUPPORTED_SHAPE, "K=%lld outside 1..65536", (long long)K);
  if (N * K >= (int64_t(1) << 32)) return fail(W12_ERR_UNSUPPORTED_SHAPE, "N*K=%lld must be below 2^32", (long long)(N * K));
  // the GEMM addresses the hi plane with 32-bit buffer offsets
  if (w12::num_row_blocks(N) * w12::num_chunks(K) * w12::kHiChunkBytes >= (int64_t(1) << 32))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "padded N x K too large for 32-bit plane offsets");
  return W12_OK;
}

// A BF16 matrix accessed with 16-byte vector loads/stores: aligned base, pitch >= cols and
// a multiple of 8 elements.
int check_bf16_matrix(const void* p, int64_t ld, int64_t cols, const char* what) {
  if (!p) return fail(W12_ERR_INVALID_ARG, "%s is NULL", what);
  if (ld < cols) return fail(W12_ERR_INVALID_ARG, "%s pitch %lld < %lld columns", what, (long long)ld, (long long)cols);
  if (!aligned(p, 16)) return fail(W12_ERR_MISALIGNED, "%s must be 16-byte aligned", what);
  if (ld % 8) return fail(W12_ERR_MISALIGNED, "%s pitch %lld must be a multiple of 8 elements", what, (long long)ld);
  return W12_OK;
}

int check_tensor(const w12_tensor* t) {
  if (!t) return fail(W12_ERR_INVALID_ARG, "tensor descriptor is NULL");
  int rc = check_shape(t->N, t->K);
  if (rc) return rc;
  if (t->layout != W12_LAYOUT_RB16_K16) return fail(W12_ERR_INVALID_ARG, "unknown layout %d", t->layout);
  if (t->reserved != 0) return fail(W12_ERR_INVALID_ARG, "reserved field must be 0");
  if (!t->base || !t->hi || !t->lo || !t->esc_ptr) return fail(W12_ERR_INVALID_ARG, "tensor has a NULL plane");
  if (t->num_escapes < 0 || t->num_escapes > (int64_t)t->N * t->K)
    return fail(W12_ERR_INVALID_ARG, "num_escapes=%lld outside 0..N*K", (long long)t->num_escapes);
  // the kernels address the escape list with 32-bit byte offsets
  if (t->num_escapes >= (int64_t(1) << 30))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "num_escapes=%lld must be below 2^30", (long long)t->num_escapes);
  if (t->num_escapes > 0 && !t->esc) return fail(W12_ERR_INVALID_ARG, "esc is NULL with num_escapes > 0");
  if (!aligned(t->hi, 16) || !aligned(t->lo, 16)) return fail(W12_ERR_MISALIGNED, "hi and lo must be 16-byte aligned");
  if (!aligned(t->esc_ptr, 4) || (t->esc && !aligned(t->esc, 4))) return fail(W12_ERR_MISALIGNED, "esc_ptr/esc must be 4-byte aligned");
  return W12_OK;
}

// Prefix the current message with the index of the group item it concerns.
int item_fail(int code, int i) {
  char msg[sizeof(g_err)];
  snprintf(msg, sizeof(msg), "%s", g_err);
  return fail(code, "item %d: %s", i, msg);
}

int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(W12_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

int w12_layout_bytes(int32_t N, int32_t K, uint64_t* hi_bytes, uint64_t* lo_bytes) {
  int rc = check_shape(N, K);
  if (rc) return rc;
  if (!hi_bytes || !lo_bytes) return fail(W12_ERR_INVALID_ARG, "output pointer is NULL");
  const uint64_t chunks = (uint64_t)w12::num_row_blocks(N) * (uint64_t)w12::num_chunks(K);
  *hi_bytes = chunks * w12::kHiChunkBytes;
  *lo_bytes = chunks * w12::kLoChunkBytes;
  return ok();
}

int w12_encode_count(const uint16_t* W, int32_t N, int32_t K, int64_t ldw, const uint8_t* forced_base,
                     uint8_t* base, uint32_t* esc_ptr, hipStream_t stream) {
  int rc = check_shape(N, K);
  if (rc) return rc;
  if ((rc = check_bf16_matrix(W, ldw, K, "W"))) return rc;
  if (!base || !esc_ptr) return fail(W12_ERR_INVALID_ARG, "base or esc_ptr is NULL");
  if (!aligned(esc_ptr, 4)) return fail(W12_ERR_MISALIGNED, "esc_ptr must be 4-byte aligned");
  return hip_status(w12::launch_encode_count(W, N, K, ldw, forced_base, base, esc_ptr, stream), "encode_count");
}

int w12_encode_emit(const uint16_t* W, int64_t ldw, const w12_tensor* t, hipStream_t stream) {
  int rc = check_tensor(t);
  if (rc) return rc;
  if ((rc = check_bf16_matrix(W, ldw, t->K, "W"))) return rc;
  return hip_status(w12::launch_encode_emit(W, ldw, t, stream), "encode_emit");
}

int w12_decode(const w12_tensor* t, uint16_t* out, int64_t ldo, hipStream_t stream) {
  int rc = check_tensor(t);
  if (rc) return rc;
  if ((rc = check_bf16_matrix(out, ldo, t->K, "out"))) return rc;
  return hip_status(w12::launch_decode(t, out, ldo, stream), "decode");
}

int w12_verify(const w12_tensor* t, const uint16_t* ref, int64_t ldr, unsigned long long* d_result,
               hipStream_t stream) {
  int rc = check_tensor(t);
  if (rc) return rc;
  if ((rc = check_bf16_matrix(ref, ldr, t->K, "ref"))) return rc;
  if (!d_result) return fail(W12_ERR_INVALID_ARG, "d_result is NULL");
  if (!aligned(d_result, 8)) return fail(W12_ERR_MISALIGNED, "d_result must be 8-byte aligned");
  return hip_status(w12::launch_verify(t, ref, ldr, d_result, stream), "verify");
}

int w12_unpack_records(const w12_tensor* t, uint16_t* rec, int64_t ldr, hipStream_t stream) {
  int rc = check_tensor(t);
  if (rc) return rc;
  if (!rec) return fail(W12_ERR_INVALID_ARG, "rec is NULL");
  if (ldr < t->K) return fail(W12_ERR_INVALID_ARG, "rec pitch %lld < K", (long long)ldr);
  if (!aligned(rec, 2)) return fail(W12_ERR_MISALIGNED, "rec must be 2-byte aligned");
  return hip_status(w12::launch_unpack(t, rec, ldr, stream), "unpack_records");
}

int w12_gemm_workspace_size(int32_t M, int32_t N, int32_t K, uint64_t* bytes) {
  int rc = check_shape(N, K);
  if (rc) return rc;
  if (M < 1 || M > kMaxM) return fail(W12_ERR_UNSUPPORTED_SHAPE, "M=%d outside 1..%d", M, kMaxM);
  if (!bytes) return fail(W12_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = w12::plan_gemm(M, N, K).ws_bytes;
  return ok();
}

int w12_gemm_plan(int32_t M, int32_t N, int32_t K, w12_gemm_plan_info* info) {
  int rc = check_shape(N, K);
  if (rc) return rc;
  if (M < 1 || M > kMaxM) return fail(W12_ERR_UNSUPPORTED_SHAPE, "M=%d outside 1..%d", M, kMaxM);
  if (!info) return fail(W12_ERR_INVALID_ARG, "info is NULL");
  const w12::GemmPlan p = w12::plan_gemm(M, N, K);
  info->path = p.path;
  info->splits = p.splits;
  info->rows_per_block = p.rb * w12::kRowsPerBlock;
  info->m_tile = p.m_tile;
  info->grid = p.grid;
  info->workspace_bytes = p.ws_bytes;
  info->counter_bytes = p.counter_bytes;
  return ok();
}

int w12_gemm_workspace_init(void* ws, uint64_t ws_bytes, hipStream_t stream) {
  if (ws_bytes == 0) return ok();
  if (!ws) return fail(W12_ERR_INVALID_ARG, "ws is NULL");
  if (!aligned(ws, 16)) return fail(W12_ERR_MISALIGNED, "ws must be 16-byte aligned");
  return hip_status(w12::init_gemm_workspace(ws, ws_bytes, stream), "gemm_workspace_init");
}

static int gemm_call(const uint16_t* X, int32_t M, int64_t ldx, const w12_tensor* t, float* Y, int64_t ldy, void* ws,
                     uint64_t ws_bytes, bool qpass, hipStream_t stream) {
  int rc = check_tensor(t);
  if (rc) return rc;
  if (M < 1 || M > kMaxM) return fail(W12_ERR_UNSUPPORTED_SHAPE, "M=%d outside 1..%d", M, kMaxM);
  if ((rc = check_bf16_matrix(X, ldx, t->K, "X"))) return rc;
  if (((int64_t)M - 1) * ldx + t->K + 16 >= (int64_t(1) << 30))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "X spans too many elements for 31-bit buffer offsets");
  if (!Y) return fail(W12_ERR_INVALID_ARG, "Y is NULL");
  if (ldy < t->N) return fail(W12_ERR_INVALID_ARG, "Y pitch %lld < N", (long long)ldy);
  if (((int64_t)M - 1) * ldy + t->N >= (int64_t(1) << 29))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "Y spans too many elements for 31-bit buffer offsets");
  if (!aligned(Y, 4)) return fail(W12_ERR_MISALIGNED, "Y must be 4-byte aligned");
  const w12::GemmPlan p = w12::plan_gemm(M, t->N, t->K);
  if (ws_bytes < p.ws_bytes)
    return fail(W12_ERR_WORKSPACE_TOO_SMALL, "workspace %llu bytes < %llu needed", (unsigned long long)ws_bytes,
                (unsigned long long)p.ws_bytes);
  if (p.ws_bytes && !ws) return fail(W12_ERR_INVALID_ARG, "ws is NULL");
  if (ws && !aligned(ws, 16)) return fail(W12_ERR_MISALIGNED, "ws must be 16-byte aligned");
  return hip_status(w12::launch_gemm(p, X, M, ldx, t, Y, ldy, ws, qpass, stream), qpass ? "gemm_q" : "gemm");
}

int w12_gemm(const uint16_t* X, int32_t M, int64_t ldx, const w12_tensor* t, float* Y, int64_t ldy, void* ws,
             uint64_t ws_bytes, hipStream_t stream) {
  return gemm_call(X, M, ldx, t, Y, ldy, ws, ws_bytes, false, stream);
}

int w12_gemm_q(const uint16_t* X, int32_t M, int64_t ldx, const w12_tensor* t, float* Y, int64_t ldy, void* ws,
               uint64_t ws_bytes, hipStream_t stream) {
  return gemm_call(X, M, ldx, t, Y, ldy, ws, ws_bytes, true, stream);
}

int w12_gemm_noalloc(const uint16_t* X, int32_t M, int64_t ldx, const w12_tensor* t, float* Y, int64_t ldy,
                     hipStream_t stream) {
  int rc = check_tensor(t);
  if (rc) return rc;
  if (M < 1 || M > kMaxM) return fail(W12_ERR_UNSUPPORTED_SHAPE, "M=%d outside 1..%d", M, kMaxM);
  const w12::GemmPlan p = w12::plan_gemm(M, t->N, t->K);
  if (p.ws_bytes > w12::kScratchBytes)
    return fail(W12_ERR_WORKSPACE_TOO_SMALL,
                "M=%d, N=%d, K=%d needs %llu bytes of workspace, above the library's %llu-byte scratch; "
                "call w12_gemm with a workspace", M, t->N, t->K, (unsigned long long)p.ws_bytes,
                (unsigned long long)w12::kScratchBytes);
  void* ws = nullptr;
  const hipError_t e = w12::scratch_workspace(&ws, stream);
  if (e != hipSuccess) return hip_status(e, "gemm_noalloc scratch");
  return gemm_call(X, M, ldx, t, Y, ldy, ws, w12::kScratchBytes, false, stream);
}

// Validates a group and plans it; on success fills tiles_of / upt_of and *plan.
static int group_plan(int32_t M, int32_t count, const w12_gemm_item* items, w12::GemmPlan* plan, int64_t* tiles_of,
                      int64_t* upt_of) {
  if (count < 1 || count > W12_GROUP_MAX)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "group of %d products outside 1..%d", count, W12_GROUP_MAX);
  if (M < 1 || M > 64) return fail(W12_ERR_UNSUPPORTED_SHAPE, "grouped M=%d outside 1..64", M);
  if (!items) return fail(W12_ERR_INVALID_ARG, "items is NULL");
  std::vector<int32_t> N((size_t)count), K((size_t)count);
  for (int i = 0; i < count; ++i) {
    int rc = check_tensor(items[i].t);
    if (rc) return item_fail(rc, i);
    if (items[i].t->K % w12::kChunkK)
      return fail(W12_ERR_UNSUPPORTED_SHAPE, "item %d: K=%d is not a multiple of 16", i, items[i].t->K);
    N[i] = items[i].t->N;
    K[i] = items[i].t->K;
  }
  *plan = w12::plan_gemm_group(M, count, N.data(), K.data(), tiles_of, upt_of);
  return W12_OK;
}

int w12_gemm_group_workspace_size(int32_t M, int32_t count, const w12_gemm_item* items, uint64_t* bytes) {
  w12::GemmPlan p;
  std::vector<int64_t> tiles_of(W12_GROUP_MAX), upt_of(W12_GROUP_MAX);
  int rc = group_plan(M, count, items, &p, tiles_of.data(), upt_of.data());
  if (rc) return rc;
  if (!bytes) return fail(W12_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = p.ws_bytes;
  return ok();
}

static int gemm_group_call(int32_t M, int32_t count, const w12_gemm_item* items, void* ws, uint64_t ws_bytes,
                           bool qpass, hipStream_t stream) {
  w12::GemmPlan p;
  std::vector<int64_t> tiles_of(W12_GROUP_MAX), upt_of(W12_GROUP_MAX);
  int rc = group_plan(M, count, items, &p, tiles_of.data(), upt_of.data());
  if (rc) return rc;
  for (int i = 0; i < count; ++i) {
    const w12_gemm_item& it = items[i];
    if ((rc = check_bf16_matrix(it.X, it.ldx, it.t->K, "X"))) return item_fail(rc, i);
    if (((int64_t)M - 1) * it.ldx + it.t->K + 16 >= (int64_t(1) << 30))
      return fail(W12_ERR_UNSUPPORTED_SHAPE, "item %d: X spans too many elements for 31-bit buffer offsets", i);
    if (!it.Y) return fail(W12_ERR_INVALID_ARG, "item %d: Y is NULL", i);
    if (it.ldy < it.t->N) return fail(W12_ERR_INVALID_ARG, "item %d: Y pitch %lld < N", i, (long long)it.ldy);
    if (((int64_t)M - 1) * it.ldy + it.t->N >= (int64_t(1) << 29))
      return fail(W12_ERR_UNSUPPORTED_SHAPE, "item %d: Y spans too many elements for 31-bit buffer offsets", i);
    if (!aligned(it.Y, 4)) return fail(W12_ERR_MISALIGNED, "item %d: Y must be 4-byte aligned", i);
  }
  if (ws_bytes < p.ws_bytes)
    return fail(W12_ERR_WORKSPACE_TOO_SMALL, "workspace %llu bytes < %llu needed", (unsigned long long)ws_bytes,
                (unsigned long long)p.ws_bytes);
  if (!ws) return fail(W12_ERR_INVALID_ARG, "ws is NULL");
  if (!aligned(ws, 16)) return fail(W12_ERR_MISALIGNED, "ws must be 16-byte aligned");
  return hip_status(w12::launch_gemm_group(p, M, count, items, tiles_of.data(), upt_of.data(), ws, qpass, stream),
                    qpass ? "gemm_group_q" : "gemm_group");
}

int w12_gemm_group(int32_t M, int32_t count, const w12_gemm_item* items, void* ws, uint64_t ws_bytes,
                   hipStream_t stream) {
  return gemm_group_call(M, count, items, ws, ws_bytes, false, stream);
}

int w12_gemm_group_q(int32_t M, int32_t count, const w12_gemm_item* items, void* ws, uint64_t ws_bytes,
                     hipStream_t stream) {
  return gemm_group_call(M, count, items, ws, ws_bytes, true, stream);
}

int w12_file_write(const char* path, int32_t count, const char* const* names, const w12_tensor* host_tensors) {
  if (!path || !names || !host_tensors) return fail(W12_ERR_INVALID_ARG, "path, names or host_tensors is NULL");
  if (count < 1) return fail(W12_ERR_INVALID_ARG, "count=%d must be at least 1", count);
  for (int i = 0; i < count; ++i) {
    if (!names[i]) return fail(W12_ERR_INVALID_ARG, "names[%d] is NULL", i);
    int rc = check_tensor(&host_tensors[i]);
    if (rc) return item_fail(rc, i);
  }
  char err[256];
  if (w12::file_write(path, count, names, host_tensors, err, sizeof(err))) return fail(W12_ERR_IO, "%s", err);
  return ok();
}

int w12_file_index(const char* path, int32_t* count, w12_file_entry* entries, int32_t max_entries) {
  if (!path || !count) return fail(W12_ERR_INVALID_ARG, "path or count is NULL");
  char err[256];
  if (entries && max_entries < 0) return fail(W12_ERR_INVALID_ARG, "max_entries < 0");
  int32_t n = 0;
  if (w12::file_index(path, &n, nullptr, 0, err, sizeof(err))) return fail(W12_ERR_IO, "%s", err);
  *count = n;
  if (!entries) return ok();
  if (n > max_entries) return fail(W12_ERR_INVALID_ARG, "file holds %d tensors, room for %d", n, max_entries);
  if (w12::file_index(path, &n, entries, max_entries, err, sizeof(err))) return fail(W12_ERR_IO, "%s", err);
  return ok();
}

int w12_file_load(const char* path, int32_t count, const int32_t* which, const w12_tensor* dst, void* staging,
                  uint64_t staging_bytes, const uint16_t* const* refs, const int64_t* ldr,
                  unsigned long long* d_results, hipStream_t stream) {
  if (!path || !which || !dst) return fail(W12_ERR_INVALID_ARG, "path, which or dst is NULL");
  if (count < 1) return fail(W12_ERR_INVALID_ARG, "count=%d must be at least 1", count);
  if (!staging || staging_bytes < 512) return fail(W12_ERR_INVALID_ARG, "staging must hold at least 512 bytes");
  char err[256];
  int32_t n = 0;
  if (w12::file_index(path, &n, nullptr, 0, err, sizeof(err))) return fail(W12_ERR_IO, "%s", err);
  std::vector<w12_file_entry> idx(n);
  if (n && w12::file_index(path, &n, idx.data(), n, err, sizeof(err))) return fail(W12_ERR_IO, "%s", err);
  for (int i = 0; i < count; ++i) {
    if (which[i] < 0 || which[i] >= n) return fail(W12_ERR_INVALID_ARG, "which[%d]=%d outside 0..%d", i, which[i], n - 1);
    int rc = check_tensor(&dst[i]);
    if (rc) return item_fail(rc, i);
    const w12_file_entry& e = idx[which[i]];
    if (e.N != dst[i].N || e.K != dst[i].K || e.layout != dst[i].layout || e.num_escapes != dst[i].num_escapes)
      return fail(W12_ERR_INVALID_ARG, "item %d: descriptor does not match file entry %d (%s)", i, which[i], e.name);
    if (refs && refs[i]) {
      if (!ldr) return fail(W12_ERR_INVALID_ARG, "ldr is NULL");
      if ((rc = check_bf16_matrix(refs[i], ldr[i], dst[i].K, "ref"))) return item_fail(rc, i);
      if (!d_results) return fail(W12_ERR_INVALID_ARG, "d_results is NULL");
      if (!aligned(d_results, 8)) return fail(W12_ERR_MISALIGNED, "d_results must be 8-byte aligned");
    }
  }
  const int rc = w12::file_load(path, count, which, dst, staging, staging_bytes, refs, ldr, d_results, stream, err,
                                sizeof(err));
  if (rc == -1) return fail(W12_ERR_IO, "%s", err);
  if (rc) return fail(W12_ERR_HIP, "%s", err);
  return ok();
}

int w12_read_probe(const void* buf, uint64_t bytes, int32_t loads_per_lane, int32_t groups_per_cu, uint32_t* sink,
                   hipStream_t stream) {
  if (!buf || !sink) return fail(W12_ERR_INVALID_ARG, "buf or sink is NULL");
  // the kernel marks loads past a work-group's share with offset 2^31, which must stay past the buffer
  if (bytes < 16 || bytes % 16 || bytes > (uint64_t(1) << 31))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "bytes=%llu must be a multiple of 16 in 16..2^31", (unsigned long long)bytes);
  if (loads_per_lane != 1 && loads_per_lane != 2 && loads_per_lane != 4 && loads_per_lane != 8 && loads_per_lane != 16)
    return fail(W12_ERR_INVALID_ARG, "loads_per_lane=%d is not 1, 2, 4, 8 or 16", loads_per_lane);
  if (groups_per_cu < 1 || groups_per_cu > 16) return fail(W12_ERR_INVALID_ARG, "groups_per_cu=%d outside 1..16", groups_per_cu);
  if (!aligned(buf, 16)) return fail(W12_ERR_MISALIGNED, "buf must be 16-byte aligned");
  if (!aligned(sink, 4)) return fail(W12_ERR_MISALIGNED, "sink must be 4-byte aligned");
  const int64_t grid = (int64_t)w12::device_cus() * groups_per_cu;
  return hip_status(w12::launch_read_probe(buf, bytes, loads_per_lane, grid, sink, stream), "read_probe");
}

// A matrix accessed with 16-byte vectors: aligned base, rows of whole 16-byte steps, and (where rows
// have to hold cols) a pitch of at least cols.
static int check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int elem_bytes, const char* what) {
  if (!p) return fail(W12_ERR_INVALID_ARG, "%s is NULL", what);
  if (ld < cols) return fail(W12_ERR_INVALID_ARG, "%s pitch %lld < %lld columns", what, (long long)ld, (long long)cols);
  if (!aligned(p, 16)) return fail(W12_ERR_MISALIGNED, "%s must be 16-byte aligned", what);
  if (ld % (16 / elem_bytes))
    return fail(W12_ERR_MISALIGNED, "%s pitch %lld must be a multiple of 16 bytes", what, (long long)ld);
  if (rows > 1 && ld > (int64_t(1) << 40) / rows)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "%s pitch %lld is too large", what, (long long)ld);
  return W12_OK;
}

// An array of 4- or 8-byte values with a pitch of at least cols.
static int check_table(const void* p, int64_t ld, int64_t rows, int64_t cols, int elem_bytes, const char* what) {
  if (!p) return fail(W12_ERR_INVALID_ARG, "%s is NULL", what);
  if (ld < cols) return fail(W12_ERR_INVALID_ARG, "%s pitch %lld < %lld columns", what, (long long)ld, (long long)cols);
  if (!aligned(p, elem_bytes)) return fail(W12_ERR_MISALIGNED, "%s must be %d-byte aligned", what, elem_bytes);
  if (rows > 1 && ld > (int64_t(1) << 40) / rows)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "%s pitch %lld is too large", what, (long long)ld);
  return W12_OK;
}

static constexpr int32_t kMaxRows = 1 << 20;   // rows of the operators that stream rows

static bool float_dtype(int32_t d) { return d == W12_DTYPE_BF16 || d == W12_DTYPE_F32; }

int w12_add_rmsnorm(const w12_norm_args* a, hipStream_t stream) {
  if (!a) return fail(W12_ERR_INVALID_ARG, "arguments are NULL");
  if (a->reserved != 0) return fail(W12_ERR_INVALID_ARG, "reserved field must be 0");
  if (a->M < 1 || a->M > kMaxRows) return fail(W12_ERR_UNSUPPORTED_SHAPE, "M=%d outside 1..%d", a->M, kMaxRows);
  if (a->N < 1 || a->N > kMaxK) return fail(W12_ERR_UNSUPPORTED_SHAPE, "N=%d outside 1..65536", a->N);
  if (!float_dtype(a->residual_dtype) || (a->delta && !float_dtype(a->delta_dtype)))
    return fail(W12_ERR_INVALID_ARG, "residual and delta are BF16 or FP32");
  if (!(a->eps >= 0.0f)) return fail(W12_ERR_INVALID_ARG, "eps must not be negative");
  const int rb = a->residual_dtype == W12_DTYPE_F32 ? 4 : 2;
  int rc = check_matrix(a->residual, a->ld_residual, a->M, a->N, rb, "residual");
  if (rc) return rc;
  if (a->delta && (rc = check_matrix(a->delta, a->ld_delta, a->M, a->N, a->delta_dtype == W12_DTYPE_F32 ? 4 : 2, "delta")))
    return rc;
  if (!a->weight) return fail(W12_ERR_INVALID_ARG, "weight is NULL");
  if (!aligned(a->weight, 16)) return fail(W12_ERR_MISALIGNED, "weight must be 16-byte aligned");
  if (a->residual_out) {
    if ((rc = check_matrix(a->residual_out, a->ld_residual_out, a->M, a->N, rb, "residual_out"))) return rc;
    if (a->residual_out == a->residual && a->ld_residual_out != a->ld_residual)
      return fail(W12_ERR_INVALID_ARG, "residual_out in place needs the residual's pitch");
  }
  if (a->y && (rc = check_matrix(a->y, a->ldy, a->M, a->N, 2, "y"))) return rc;
  if (a->yq) {
    if ((rc = check_matrix(a->yq, a->ldyq, a->M, a->N, 1, "yq"))) return rc;
    if ((rc = check_table(a->yq_scale, a->ld_scale, a->M, w12::ceil_div(a->N, W12_QUANT_BLOCK), 4, "yq_scale"))) return rc;
  } else if (a->yq_scale) {
    return fail(W12_ERR_INVALID_ARG, "yq_scale without yq");
  }
  if (!a->y && !a->yq && !(a->residual_out && a->delta)) return fail(W12_ERR_INVALID_ARG, "no output is wanted");
  return hip_status(w12::launch_add_rmsnorm(*a, stream), "add_rmsnorm");
}

static int check_cache(const w12_kv_cache* c) {
  if (!c) return fail(W12_ERR_INVALID_ARG, "cache is NULL");
  if (c->reserved != 0) return fail(W12_ERR_INVALID_ARG, "cache: reserved field must be 0");
  if (c->dtype != W12_DTYPE_BF16 && c->dtype != W12_DTYPE_E4M3)
    return fail(W12_ERR_INVALID_ARG, "cache: type %d is neither BF16 nor E4M3", c->dtype);
  if (c->pages < 1) return fail(W12_ERR_UNSUPPORTED_SHAPE, "cache: %d pages", c->pages);
  if (c->page_size < 1 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "cache: page size %d is not a power of two in 1..1024", c->page_size);
  if (c->heads < 1 || c->heads > 1024) return fail(W12_ERR_UNSUPPORTED_SHAPE, "cache: %d heads outside 1..1024", c->heads);
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "cache: head dimension %d is not 64, 128 or 256", c->dim);
  if (!c->k || !c->v) return fail(W12_ERR_INVALID_ARG, "cache: k or v is NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(W12_ERR_MISALIGNED, "cache: k and v must be 16-byte aligned");
  const int64_t step = c->dtype == W12_DTYPE_BF16 ? 8 : 16;
  const int64_t strides[3] = {c->page_stride, c->token_stride, c->head_stride};
  for (int64_t s : strides) {
    if (s < 0) return fail(W12_ERR_INVALID_ARG, "cache: negative stride");
    if (s % step) return fail(W12_ERR_MISALIGNED, "cache: stride %lld must be a multiple of 16 bytes", (long long)s);
  }
  if (c->page_stride > (int64_t(1) << 42) / c->pages || c->token_stride > (int64_t(1) << 32) / c->page_size ||
      c->head_stride > (int64_t(1) << 32) / c->heads)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "cache: strides too large");
  if (c->dtype == W12_DTYPE_E4M3) {
    if (!c->k_scale || !c->v_scale) return fail(W12_ERR_INVALID_ARG, "cache: an E4M3 cache needs k_scale and v_scale");
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
      return fail(W12_ERR_MISALIGNED, "cache: scales must be 4-byte aligned");
  }
  return W12_OK;
}

int w12_rope_append(const w12_rope_args* a, const w12_kv_cache* cache, hipStream_t stream) {
  if (!a) return fail(W12_ERR_INVALID_ARG, "arguments are NULL");
  int rc = check_cache(cache);
  if (rc) return rc;
  if (a->T < 1 || a->T > kMaxRows) return fail(W12_ERR_UNSUPPORTED_SHAPE, "T=%d outside 1..%d", a->T, kMaxRows);
  if (a->q_heads < 1 || a->q_heads > 4096) return fail(W12_ERR_UNSUPPORTED_SHAPE, "q_heads=%d outside 1..4096", a->q_heads);
  if (!float_dtype(a->src_dtype)) return fail(W12_ERR_INVALID_ARG, "qkv is BF16 or FP32");
  if (a->rot_dim < 0 || a->rot_dim > cache->dim || a->rot_dim % 2)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "rot_dim=%d is not an even number in 0..%d", a->rot_dim, cache->dim);
  if (a->axes < 1 || a->axes > 8) return fail(W12_ERR_UNSUPPORTED_SHAPE, "axes=%d outside 1..8", a->axes);
  const int64_t width = (int64_t)(a->q_heads + 2 * cache->heads) * cache->dim;
  if ((rc = check_matrix(a->qkv, a->ld_qkv, a->T, width, a->src_dtype == W12_DTYPE_F32 ? 4 : 2, "qkv"))) return rc;
  if ((rc = check_matrix(a->q, a->ldq, a->T, (int64_t)a->q_heads * cache->dim, 2, "q"))) return rc;
  if (a->rot_dim) {
    if ((rc = check_table(a->positions, a->ld_positions, a->axes, a->T, 4, "positions"))) return rc;
    if (!a->inv_freq) return fail(W12_ERR_INVALID_ARG, "inv_freq is NULL");
    if (!aligned(a->inv_freq, 8)) return fail(W12_ERR_MISALIGNED, "inv_freq must be 8-byte aligned");
  }
  if (!a->slots) return fail(W12_ERR_INVALID_ARG, "slots is NULL");
  if (!aligned(a->slots, 8)) return fail(W12_ERR_MISALIGNED, "slots must be 8-byte aligned");
  return hip_status(w12::launch_rope_append(*a, *cache, stream), "rope_append");
}

static int check_attention_shape(int32_t T, int32_t requests, int32_t q_heads, const w12_kv_cache* cache) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (T < 1 || T > kMaxRows) return fail(W12_ERR_UNSUPPORTED_SHAPE, "T=%d outside 1..%d", T, kMaxRows);
  if (requests < 1 || requests > 1024) return fail(W12_ERR_UNSUPPORTED_SHAPE, "requests=%d outside 1..1024", requests);
  if (q_heads < 1 || q_heads % cache->heads || q_heads / cache->heads > 64)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "q_heads=%d is not 1..64 times the cache's %d heads", q_heads, cache->heads);
  return W12_OK;
}

int w12_tree_attention_workspace_size(int32_t T, int32_t requests, int32_t q_heads, const w12_kv_cache* cache,
                                      uint64_t* bytes) {
  int rc = check_attention_shape(T, requests, q_heads, cache);
  if (rc) return rc;
  if (!bytes) return fail(W12_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = w12::attention_workspace_bytes(T, requests, q_heads, *cache);
  return ok();
}

int w12_tree_attention(const w12_attention_args* a, const w12_kv_cache* cache, void* ws, uint64_t ws_bytes,
                       hipStream_t stream) {
  if (!a) return fail(W12_ERR_INVALID_ARG, "arguments are NULL");
  int rc = check_attention_shape(a->T, a->requests, a->q_heads, cache);
  if (rc) return rc;
  const int64_t width = (int64_t)a->q_heads * cache->dim;
  if ((rc = check_matrix(a->q, a->ldq, a->T, width, 2, "q"))) return rc;
  if ((rc = check_matrix(a->out, a->ldo, a->T, width, 2, "out"))) return rc;
  if (a->max_pages < 1 || (int64_t)a->max_pages * cache->page_size >= (int64_t(1) << 30))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "max_pages=%d: a request holds 1 .. 2^30 - 1 tokens", a->max_pages);
  if ((rc = check_table(a->page_table, a->ld_table, a->requests, a->max_pages, 4, "page_table"))) return rc;
  if (!a->node_ptr || !a->ctx_len) return fail(W12_ERR_INVALID_ARG, "node_ptr or ctx_len is NULL");
  if (!aligned(a->node_ptr, 4) || !aligned(a->ctx_len, 4))
    return fail(W12_ERR_MISALIGNED, "node_ptr and ctx_len must be 4-byte aligned");
  if (a->tree_mask) {
    if (a->mask_words < 1 || a->mask_words > 64)
      return fail(W12_ERR_UNSUPPORTED_SHAPE, "mask_words=%d outside 1..64", a->mask_words);
    if ((rc = check_table(a->tree_mask, a->ld_mask, a->T, a->mask_words, 8, "tree_mask"))) return rc;
  } else if (a->mask_words != 0) {
    return fail(W12_ERR_INVALID_ARG, "mask_words without tree_mask");
  }
  if (a->lse && (rc = check_table(a->lse, a->ld_lse, a->T, a->q_heads, 4, "lse"))) return rc;
  if (!(a->scale > 0.0f) || a->scale > 1e30f) return fail(W12_ERR_INVALID_ARG, "scale must be positive and finite");
  const uint64_t need = w12::attention_workspace_bytes(a->T, a->requests, a->q_heads, *cache);
  if (ws_bytes < need)
    return fail(W12_ERR_WORKSPACE_TOO_SMALL, "workspace %llu bytes < %llu needed", (unsigned long long)ws_bytes,
                (unsigned long long)need);
  if (need && !ws) return fail(W12_ERR_INVALID_ARG, "ws is NULL");
  if (ws && !aligned(ws, 16)) return fail(W12_ERR_MISALIGNED, "ws must be 16-byte aligned");
  return hip_status(w12::launch_tree_attention(*a, *cache, ws, stream), "tree_attention");
}

int w12_gemm_e4m3_workspace_size(int32_t M, int32_t N, int32_t K, uint64_t* bytes) {
  int rc = check_shape(N, K);
  if (rc) return rc;
  if (M < 1 || M > kMaxM) return fail(W12_ERR_UNSUPPORTED_SHAPE, "M=%d outside 1..%d", M, kMaxM);
  if (!bytes) return fail(W12_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = w12::gemm_e4m3_workspace_bytes(M, N, K);
  return ok();
}

int w12_gemm_e4m3(const uint8_t* X, int32_t M, int64_t ldx, const float* x_scale, int64_t ldxs, const uint8_t* W,
                  int32_t N, int32_t K, int64_t ldw, const float* w_scale, int64_t ldws, float* Y, int64_t ldy,
                  void* ws, uint64_t ws_bytes, hipStream_t stream) {
  int rc = check_shape(N, K);
  if (rc) return rc;
  if (M < 1 || M > kMaxM) return fail(W12_ERR_UNSUPPORTED_SHAPE, "M=%d outside 1..%d", M, kMaxM);
  const int64_t kb = w12::ceil_div(K, W12_QUANT_BLOCK);
  if ((rc = check_matrix(X, ldx, M, K, 1, "X"))) return rc;
  if ((rc = check_matrix(W, ldw, N, K, 1, "W"))) return rc;
  if ((rc = check_table(x_scale, ldxs, M, kb, 4, "x_scale"))) return rc;
  if ((rc = check_table(w_scale, ldws, w12::ceil_div(N, W12_QUANT_BLOCK), kb, 4, "w_scale"))) return rc;
  if ((rc = check_table(Y, ldy, M, N, 4, "Y"))) return rc;
  // the kernels address each operand with 32-bit buffer offsets
  if (((int64_t)M - 1) * ldx + K >= (int64_t(1) << 31))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "X spans too many bytes for 31-bit buffer offsets");
  if (((int64_t)M - 1) * ldxs + kb >= (int64_t(1) << 29))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "x_scale spans too many elements for 31-bit buffer offsets");
  if (((int64_t)N - 1) * ldw + K >= (int64_t(1) << 32) - 16)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "W spans too many bytes for 32-bit buffer offsets");
  if (((int64_t)M - 1) * ldy + N >= (int64_t(1) << 29))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "Y spans too many elements for 31-bit buffer offsets");
  const uint64_t need = w12::gemm_e4m3_call_bytes(M, N, K);
  if (ws_bytes < need)
    return fail(W12_ERR_WORKSPACE_TOO_SMALL, "workspace %llu bytes < %llu needed", (unsigned long long)ws_bytes,
                (unsigned long long)need);
  if (need && !ws) return fail(W12_ERR_INVALID_ARG, "ws is NULL");
  if (ws && !aligned(ws, 16)) return fail(W12_ERR_MISALIGNED, "ws must be 16-byte aligned");
  return hip_status(w12::launch_gemm_e4m3(X, M, ldx, x_scale, ldxs, W, N, K, ldw, w_scale, ldws, Y, ldy, ws, stream),
                    "gemm_e4m3");
}

// The rows and states of a call: a state array's address is checked by the caller.
static int check_sequences(const w12_sequences* s) {
  if (!s) return fail(W12_ERR_INVALID_ARG, "sequences are NULL");
  if (s->T < 1 || s->T > kMaxRows) return fail(W12_ERR_UNSUPPORTED_SHAPE, "T=%d outside 1..%d", s->T, kMaxRows);
  if (s->count < 1 || s->count > 1024) return fail(W12_ERR_UNSUPPORTED_SHAPE, "count=%d outside 1..1024", s->count);
  if (s->slots < 1 || s->slots > kMaxRows) return fail(W12_ERR_UNSUPPORTED_SHAPE, "slots=%d outside 1..%d", s->slots, kMaxRows);
  if (!s->ptr || !s->src) return fail(W12_ERR_INVALID_ARG, "ptr or src is NULL");
  if (!aligned(s->ptr, 4) || !aligned(s->lens, 4) || !aligned(s->rows, 4) || !aligned(s->src, 4) || !aligned(s->dst, 4))
    return fail(W12_ERR_MISALIGNED, "ptr, lens, rows, src and dst must be 4-byte aligned");
  if (s->tree_mask) {
    if (s->dst || s->rows || s->lens) return fail(W12_ERR_INVALID_ARG, "a tree has no dst, rows or lens");
    if (s->mask_words < 1 || s->mask_words > 64)
      return fail(W12_ERR_UNSUPPORTED_SHAPE, "mask_words=%d outside 1..64", s->mask_words);
    return check_table(s->tree_mask, s->ld_mask, s->T, s->mask_words, 8, "tree_mask");
  }
  if (s->mask_words != 0) return fail(W12_ERR_INVALID_ARG, "mask_words without tree_mask");
  return W12_OK;
}

// A state array of `each` elements a slot.
static int check_state(const void* p, int64_t slot_stride, int64_t each, int32_t slots, int elem_bytes) {
  if (!p) return fail(W12_ERR_INVALID_ARG, "state is NULL");
  if (!aligned(p, 16)) return fail(W12_ERR_MISALIGNED, "state must be 16-byte aligned");
  if (slot_stride < each)
    return fail(W12_ERR_INVALID_ARG, "slot stride %lld < %lld elements of a state", (long long)slot_stride, (long long)each);
  if (slot_stride % (16 / elem_bytes))
    return fail(W12_ERR_MISALIGNED, "slot stride %lld must be a multiple of 16 bytes", (long long)slot_stride);
  if (slot_stride > (int64_t(1) << 42) / slots) return fail(W12_ERR_UNSUPPORTED_SHAPE, "slot stride too large");
  return W12_OK;
}

int w12_short_conv(const w12_conv_args* a, const w12_sequences* s, hipStream_t stream) {
  if (!a) return fail(W12_ERR_INVALID_ARG, "arguments are NULL");
  int rc = check_sequences(s);
  if (rc) return rc;
  if (a->channels < 1 || a->channels > (1 << 17))
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "channels=%d outside 1..%d", a->channels, 1 << 17);
  if (a->width < 2 || a->width > 4) return fail(W12_ERR_UNSUPPORTED_SHAPE, "width=%d outside 2..4", a->width);
  if (!float_dtype(a->dtype)) return fail(W12_ERR_INVALID_ARG, "x and state are BF16 or FP32");
  const int eb = a->dtype == W12_DTYPE_F32 ? 4 : 2;
  if ((rc = check_matrix(a->x, a->ldx, s->T, a->channels, eb, "x"))) return rc;
  if (!a->weight) return fail(W12_ERR_INVALID_ARG, "weight is NULL");
  if (!aligned(a->weight, 16) || !aligned(a->bias, 2)) return fail(W12_ERR_MISALIGNED, "weight must be 16-byte, bias 2-byte aligned");
  if (a->tap_stride < a->channels)
    return fail(W12_ERR_INVALID_ARG, "tap stride %lld < %d channels", (long long)a->tap_stride, a->channels);
  if (a->tap_stride % (16 / eb))
    return fail(W12_ERR_MISALIGNED, "tap stride %lld must be a multiple of 16 bytes", (long long)a->tap_stride);
  if (a->tap_stride > (int64_t(1) << 40)) return fail(W12_ERR_UNSUPPORTED_SHAPE, "tap stride too large");
  if ((rc = check_state(a->state, a->slot_stride, (a->width - 2) * a->tap_stride + a->channels, s->slots, eb))) return rc;
  if (a->y && (rc = check_matrix(a->y, a->ldy, s->T, a->channels, 2, "y"))) return rc;
  if (!a->y && !s->dst) return fail(W12_ERR_INVALID_ARG, "neither outputs nor states are wanted");
  return hip_status(w12::launch_short_conv(*a, *s, stream), "short_conv");
}

static int check_delta_shape(int32_t T, int32_t count, int32_t v_heads, int32_t dk, int32_t dv) {
  if (T < 1 || T > kMaxRows) return fail(W12_ERR_UNSUPPORTED_SHAPE, "T=%d outside 1..%d", T, kMaxRows);
  if (count < 1 || count > 1024) return fail(W12_ERR_UNSUPPORTED_SHAPE, "count=%d outside 1..1024", count);
  if (v_heads < 1 || v_heads > 1024) return fail(W12_ERR_UNSUPPORTED_SHAPE, "v_heads=%d outside 1..1024", v_heads);
  if (dk != 64 && dk != 128) return fail(W12_ERR_UNSUPPORTED_SHAPE, "dk=%d is not 64 or 128", dk);
  if (dv != 64 && dv != 128 && dv != 256) return fail(W12_ERR_UNSUPPORTED_SHAPE, "dv=%d is not 64, 128 or 256", dv);
  return W12_OK;
}

int w12_gated_delta_workspace_size(int32_t T, int32_t count, int32_t v_heads, int32_t dk, int32_t dv, uint64_t* bytes) {
  int rc = check_delta_shape(T, count, v_heads, dk, dv);
  if (rc) return rc;
  if (!bytes) return fail(W12_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = w12::gated_delta_workspace_bytes(T, count, v_heads, dk, dv);
  return ok();
}

int w12_gated_delta(const w12_delta_args* a, const w12_sequences* s, void* ws, uint64_t ws_bytes, hipStream_t stream) {
  if (!a) return fail(W12_ERR_INVALID_ARG, "arguments are NULL");
  int rc = check_sequences(s);
  if (rc) return rc;
  if ((rc = check_delta_shape(s->T, s->count, a->v_heads, a->dk, a->dv))) return rc;
  if (a->reserved != 0) return fail(W12_ERR_INVALID_ARG, "reserved field must be 0");
  if (a->k_heads < 1 || a->v_heads % a->k_heads)
    return fail(W12_ERR_UNSUPPORTED_SHAPE, "v_heads=%d is not a multiple of k_heads=%d", a->v_heads, a->k_heads);
  if (!(a->eps >= 0.0f)) return fail(W12_ERR_INVALID_ARG, "eps must not be negative");
  if (!(a->scale >= -1e30f && a->scale <= 1e30f)) return fail(W12_ERR_INVALID_ARG, "scale must be finite");
  const int64_t kw = (int64_t)a->k_heads * a->dk, vw = (int64_t)a->v_heads * a->dv;
  if ((a->q == nullptr) != (a->out == nullptr)) return fail(W12_ERR_INVALID_ARG, "q and out go together");
  if (a->q && (rc = check_matrix(a->q, a->ldq, s->T, kw, 2, "q"))) return rc;
  if ((rc = check_matrix(a->k, a->ldk, s->T, kw, 2, "k"))) return rc;
  if ((rc = check_matrix(a->v, a->ldv, s->T, vw, 2, "v"))) return rc;
  if ((rc = check_table(a->g, a->ldg, s->T, a->v_heads, 4, "g"))) return rc;
  if ((rc = check_table(a->beta, a->ldbeta, s->T, a->v_heads, 4, "beta"))) return rc;
  if ((rc = check_state(a->state, a->slot_stride, vw * a->dk, s->slots, 4))) return rc;
  if (a->out && (rc = check_matrix(a->out, a->ldo, s->T, vw, 2, "out"))) return rc;
  if (!a->out && !s->dst) return fail(W12_ERR_INVALID_ARG, "neither outputs nor states are wanted");
  const uint64_t need = w12::gated_delta_call_bytes(*s, a->v_heads);
  if (ws_bytes < need)
    return fail(W12_ERR_WORKSPACE_TOO_SMALL, "workspace %llu bytes < %llu needed", (unsigned long long)ws_bytes,
                (unsigned long long)need);
  if (need && !ws) return fail(W12_ERR_INVALID_ARG, "ws is NULL");
  if (ws && !aligned(ws, 16)) return fail(W12_ERR_MISALIGNED, "ws must be 16-byte aligned");
  return hip_status(w12::launch_gated_delta(*a, *s, ws, ws_bytes, stream), "gated_delta");
}

static int check_verify_draft_shape(int32_t T, int32_t requests, int32_t vocab) {
  if (T < 1 || T > kMaxRows) return fail(W12_ERR_UNSUPPORTED_SHAPE, "T=%d outside 1..%d", T, kMaxRows);
  if (requests < 1 || requests > 1024) return fail(W12_ERR_UNSUPPORTED_SHAPE, "requests=%d outside 1..1024", requests);
  if (vocab < 1 || vocab > (1 << 24)) return fail(W12_ERR_UNSUPPORTED_SHAPE, "vocab=%d outside 1..2^24", vocab);
  if ((int64_t)T * vocab >= (int64_t(1) << 40)) return fail(W12_ERR_UNSUPPORTED_SHAPE, "T * vocab must be below 2^40");
  return W12_OK;
}

int w12_verify_draft_workspace_size(int32_t T, int32_t requests, int32_t vocab, uint64_t* bytes) {
  int rc = check_verify_draft_shape(T, requests, vocab);
  if (rc) return rc;
  if (!bytes) return fail(W12_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = w12::verify_draft_workspace_bytes(T, requests, vocab);
  return ok();
}

int w12_verify_draft(const w12_verify_draft_args* a, void* ws, uint64_t ws_bytes, hipStream_t stream) {
  if (!a) return fail(W12_ERR_INVALID_ARG, "arguments are NULL");
  int rc = check_verify_draft_shape(a->T, a->requests, a->vocab);
  if (rc) return rc;
  if (a->reserved != 0) return fail(W12_ERR_INVALID_ARG, "reserved field must be 0");
  if (!float_dtype(a->logits_dtype)) return fail(W12_ERR_INVALID_ARG, "logits are BF16 or FP32");
  if ((rc = check_matrix(a->logits, a->ld_logits, a->T, a->vocab, a->logits_dtype == W12_DTYPE_F32 ? 4 : 2, "logits"))) return rc;
  if (a->q) {
    if (a->tree_mask) return fail(W12_ERR_INVALID_ARG, "q goes with chains, not with a tree_mask");
    if ((rc = check_matrix(a->q, a->ldq, a->T, a->vocab, 4, "q"))) return rc;
  }
  if ((a->q == nullptr) != (a->accept_u == nullptr)) return fail(W12_ERR_INVALID_ARG, "q and accept_u go together");
  if (a->tree_mask) {
    if (a->mask_words < 1 || a->mask_words > 64)
      return fail(W12_ERR_UNSUPPORTED_SHAPE, "mask_words=%d outside 1..64", a->mask_words);
    if ((rc = check_table(a->tree_mask, a->ld_mask, a->T, a->mask_words, 8, "tree_mask"))) return rc;
  } else if (a->mask_words != 0) {
    return fail(W12_ERR_INVALID_ARG, "mask_words without tree_mask");
  }
  if (!a->tokens || !a->node_ptr || !a->u || !a->path || !a->count || !a->next_token)
    return fail(W12_ERR_INVALID_ARG, "tokens, node_ptr, u, path, count or next_token is NULL");
  const void* words[] = {a->tokens, a->node_ptr, a->u, a->accept_u, a->temperature, a->path, a->count, a->next_token};
  for (const void* p : words)
    if (!aligned(p, 4))
      return fail(W12_ERR_MISALIGNED, "tokens, node_ptr, random numbers, temperature and outputs must be 4-byte aligned");
  const uint64_t need = w12::verify_draft_workspace_bytes(a->T, a->requests, a->vocab);
  if (ws_bytes < need)
    return fail(W12_ERR_WORKSPACE_TOO_SMALL, "workspace %llu bytes < %llu needed", (unsigned long long)ws_bytes,
                (unsigned long long)need);
  if (!ws) return fail(W12_ERR_INVALID_ARG, "ws is NULL");
  if (!aligned(ws, 16)) return fail(W12_ERR_MISALIGNED, "ws must be 16-byte aligned");
  return hip_status(w12::launch_verify_draft(*a, ws, stream), "verify_draft");
}

double w12_bits_per_weight(int32_t N, int32_t K, int64_t E) {
  if (N < 1 || K < 1 || E < 0) return -1.0;
  const double nk = (double)N * (double)K;
  return (1.5 * nk + (double)N + 4.0 * ((double)N + 1.0) + 4.0 * (double)E) * 8.0 / nk;
}

#ifdef W12_TIMELINE
#include "w12_timeline.h"
int w12_timeline_copy(void* host, uint64_t bytes) {
  if (!host) return fail(W12_ERR_INVALID_ARG, "host is NULL");
  if (bytes == 0 || bytes > (uint64_t)w12::kMaxGrid * 16 * 8)
    return fail(W12_ERR_INVALID_ARG, "bytes=%llu outside 1..%llu", (unsigned long long)bytes,
                (unsigned long long)w12::kMaxGrid * 16 * 8);
  return hip_status(w12::timeline_copy(host, bytes), "timeline_copy");
}
#endif

uint64_t w12_tensor_bytes(int32_t N, int32_t K, int64_t E) {
  if (N < 1 || K < 1 || E < 0) return 0;
  const uint64_t nk = (uint64_t)N * (uint64_t)K;
  return (12 * nk + 7) / 8 + (uint64_t)N + 4 * ((uint64_t)N + 1) + 4 * (uint64_t)E;
}

const char* w12_status_string(int status) {
  switch (status) {
    case W12_OK: return "ok";
    case W12_ERR_INVALID_ARG: return "invalid argument";
    case W12_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case W12_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case W12_ERR_HIP: return "HIP error";
    case W12_ERR_MISALIGNED: return "misaligned pointer or pitch";
    case W12_ERR_IO: return "checkpoint file error";
    default: return "unknown status";
  }
}

const char* w12_last_error(void) { return g_err; }

}  // extern "C"
