// Attention of drafted tokens over a paged cache.
//
// The rows of a request that read one cache head (node i, query head g: row i * group + g) are cut
// into blocks of 128, the tokens into tiles of 64 and the tiles into chunks.  A work-group takes one
// block over one chunk; the length of a chunk is the same for all requests, chosen on the device: of one
// request so that the items make whole rounds of the chip, of several one round, or, if they are many, so that
// they fill it about evenly (unequal lengths give unequal numbers of items).  Items are numbered
// request, head, chunk, block, and neighbouring numbers run on one XCD: the blocks of a chunk read its
// keys and values together, once from memory.  Blocks of several chunks leave partial results, which
// k_join adds in the order of the chunks.
//
// A wave holds 32 rows: S^T = K Q^T by 32x32x16 matrix instructions leaves a row's scores in the
// two lanes of its column, so the softmax needs one exchange between lanes, and the registers of
// P^T are already the operand of O^T = V^T P^T (a sum over tokens, taken in the order in which the
// registers hold them; V is read from LDS transposed in the same order).  With a running maximum m,
//   p = exp2(c s - c m),  l = sum p,  O = sum p v,
// l and O are scaled only when a score passes m by 2^8 (p stays below 2^8).  P is rounded to BF16
// for the product (relative error 2^-8 of each p at most); everything else is FP32.
//
// Tiles go to LDS (double-buffered, 16-byte pieces swizzled by token so that both reads are free of
// bank conflicts) while the previous tile is computed on: directly where a tile of a BF16 cache lies in one page,
// else through registers, in which E4M3 caches become BF16 (exactly); their scales go into c and the result.
//
// Bound (40 heads on 8 cache heads of 128): a long cache by the matrix instructions, their operand reads from LDS
// and the exponentials, which run partly beside each other (64 nodes over 131001 tokens: 223 to 238 us, 720 to 770 TFLOP/s,
// 2.4 TB/s); a short one by the loop's start, the partial results, the second launch and work-groups without an item: the
// grid is what any lengths may need, as the host does not know them (63 nodes over 8191: 29 us, 2080 work-groups for 456
// items; one over 509: 11).  A chain is computed above its diagonal too, and those products are dropped.
#include <type_traits>

#include "w12_attention_plan.h"
#include "w12_device.h"
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4a __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kAttnThreads = 256;
constexpr int kMaxRequests = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;       // log2 of the largest p that a stale maximum may give

// One request: its rows and lengths, cut to what is there.
struct Request {
  int start, nodes, ctx, len;
};

__device__ __forceinline__ Request request_of(const w12_attention_args& a, int page_size, int b) {
  Request r;
  r.start = min(max(a.node_ptr[b], 0), a.T);
  r.nodes = min(max(a.node_ptr[b + 1], r.start), a.T) - r.start;
  const int room = a.max_pages * page_size;
  r.ctx = min(max(a.ctx_len[b], 0), room);
  r.len = (int)min((int64_t)r.ctx + r.nodes, (int64_t)room);
  return r;
}

__device__ __forceinline__ Blocks blocks_of(const Request& r, int group) { return blocks_of(r.nodes * group, r.len); }

// Running sums over the requests, value(b) of each, into LDS (before[b], before[requests] the total).
template <typename F>
__device__ __forceinline__ int64_t prefix_requests(int requests, int64_t* before, int64_t* wave_sums, F value) {
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  int64_t carry = 0;
  for (int b0 = 0; b0 < requests; b0 += kAttnThreads) {
    const int64_t v = b0 + t < requests ? value(b0 + t) : 0;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t u = __shfl_up(s, o);
      if (lane >= o) s += u;
    }
    if (lane == 63) wave_sums[w] = s;
    __syncthreads();
    int64_t off = carry;
    for (int i = 0; i < w; ++i) off += wave_sums[i];
    if (b0 + t < requests) before[b0 + t] = off + s - v;
    for (int i = 0; i < kAttnThreads / 64; ++i) carry += wave_sums[i];
    __syncthreads();
  }
  if (t == 0) before[requests] = carry;
  __syncthreads();
  return carry;
}

// The last request whose sum does not pass x (x is below the total).
__device__ __forceinline__ int find_request(const int64_t* before, int requests, int64_t x) {
  int lo = 0, hi = requests;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// The value of the lane 32 away.  Each lane picks its result: given one value twice, or the larger of both
// results asked for, the compiler takes the two results for the same.
__device__ __forceinline__ float other_half(float v) {
  uint32_t a = __builtin_bit_cast(uint32_t, v), b = a;
  asm("" : "+v"(b));
  const auto sw = __builtin_amdgcn_permlane32_swap(a, b, false, false);   // (low halves, high halves)
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? sw[0] : sw[1]);
}

// The items of a call.  `before` (LDS) holds the number of items before each request; one request needs none.
__device__ __forceinline__ Plan plan_items(const w12_attention_args& a, const w12_kv_cache& c, int group, int target, int64_t* before,
                                           int64_t* sums) {
  return plan_of(
      a.requests, c.heads, a.T * group, target, [&](int b) { return blocks_of(request_of(a, c.page_size, b), group); },
      [&](auto value) { return uniform(prefix_requests(a.requests, before, sums, value)); });
}

__host__ __device__ constexpr int64_t slot_floats(int D, int row_groups) { return (int64_t)row_groups * 32 * (D + 2); }

// Where a thread's part of a tile comes from and goes to.
template <int D, bool F8>
struct Tile {
  static constexpr int kRowBytes = D * 2;                       // BF16 in LDS
  static constexpr int kPieces = D / 8;                         // 16-byte pieces of a row in LDS
  static constexpr int kSrc = F8 ? D / 16 : D / 8;              // 16-byte loads of a row
  static constexpr int kRows = kAttnThreads / kSrc;             // rows of a load instruction of the work-group
  static constexpr int kPass = kTile / kRows;
  // Reads of K take one piece of 32 tokens, reads of V 4 pieces of 8 tokens: the swizzles spread
  // each over all banks.
  __device__ static int k_swizzle(int token) { return D == 64 ? token >> 1 & 7 : token & 15; }
  __device__ static int v_swizzle(int token) { return D == 64 ? (token >> 1 & 1) << 2 : (token & 3) << 2; }
};

// LDS: K and V of two tiles, and per tile and token whether it is there.
template <int D>
struct Lds {
  u32x4a kv[2][2][kTile * D / 8];
  uint8_t there[2][kTile];
  uint32_t bad;        // drafted tokens of this segment had values that are infinite or NaN
  int64_t before[kMaxRequests + 1];
  int64_t sums[kAttnThreads / 64];
};

// Whether one of a piece's values is infinite or NaN: an exponent of ones (BF16), all bits but the sign (E4M3).
// Such a field is the only one that a carry leaves when 1 is added at its foot.
template <bool F8>
__device__ __forceinline__ bool not_finite(u32x4a u) {
  constexpr uint32_t field = F8 ? 0x7F7F7F7Fu : 0x7F807F80u, foot = F8 ? 0x01010101u : 0x00800080u, top = F8 ? 0x80808080u : 0x80008000u;
  const u32x4a c = ((u & field) + foot) & top;
  return (c[0] | c[1] | c[2] | c[3]) != 0;
}

// E4M3 to BF16: 8 bytes.
__device__ __forceinline__ u32x4a widen(uint32_t lo, uint32_t hi) {
  return u32x4a{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
}

// The tiles of a segment on their way from the cache to LDS.  WHOLE: a tile lies in one page (pages of 64
// tokens or more), so its page and address are scalars and a thread's offsets the same for every tile.
// Nothing here is loaded under a branch: tokens that are not there read what is (the first page, the last
// token) and are marked; the compiler then knows how many loads are in flight and waits for no more than it needs.
template <int D, bool F8, bool WHOLE>
struct Stream {
  using T = Tile<D, F8>;
  const w12_attention_args& a;
  const w12_kv_cache& c;
  Lds<D>& lds;
  const int32_t* table;      // the request's pages
  int page_bits, ctx, len;
  int64_t head_bytes;
  uint32_t off[WHOLE ? T::kPass : 1];
  u32x4a k[T::kPass], v[T::kPass];
  int page[WHOLE ? 1 : T::kPass];      // of the tile that is fetched next
  uint32_t there;                      // bit i: the token of pass i of the fetched tile is there

  __device__ __forceinline__ int row() const { return threadIdx.x / T::kSrc; }
  __device__ __forceinline__ int piece() const { return threadIdx.x % T::kSrc; }

  __device__ __forceinline__ void begin(int b, int h, const Request& rq) {
    table = a.page_table + b * a.ld_table;
    ctx = rq.ctx;
    len = rq.len;
    head_bytes = (int64_t)h * c.head_stride * (F8 ? 1 : 2);
    if constexpr (WHOLE) {
#pragma unroll
      for (int i = 0; i < T::kPass; ++i)
        off[i] = (uint32_t)(i * T::kRows + row()) * (uint32_t)(c.token_stride * (F8 ? 1 : 2)) + piece() * 16;
    }
  }

  __device__ __forceinline__ void look_up(int tile) {
    if constexpr (WHOLE) {
      page[0] = table[min(tile * kTile, len - 1) >> page_bits];
    } else {
#pragma unroll
      for (int i = 0; i < T::kPass; ++i) page[i] = table[min(tile * kTile + i * T::kRows + row(), len - 1) >> page_bits];
    }
  }

  // Starts the loads of the tile whose pages are looked up.
  __device__ __forceinline__ void fetch(int tile) {
    if constexpr (WHOLE) {
      const int p = uniform(page[0]);
      const bool in = (uint32_t)p < (uint32_t)c.pages;
      const int64_t base = ((int64_t)(in ? p : 0) * c.page_stride + (int64_t)(tile * kTile & (c.page_size - 1)) * c.token_stride) *
                               (F8 ? 1 : 2) + head_bytes;
      const char* kp = static_cast<const char*>(c.k) + base;
      const char* vp = static_cast<const char*>(c.v) + base;
      there = 0;
#pragma unroll
      for (int i = 0; i < T::kPass; ++i) {
        k[i] = *reinterpret_cast<const u32x4a*>(kp + off[i]);
        v[i] = *reinterpret_cast<const u32x4a*>(vp + off[i]);
        there |= (in && tile * kTile + i * T::kRows + row() < len ? 1u : 0u) << i;
      }
    } else {
      there = 0;
#pragma unroll
      for (int i = 0; i < T::kPass; ++i) {
        const int token = tile * kTile + i * T::kRows + row();
        const bool in = (uint32_t)page[i] < (uint32_t)c.pages;
        const int64_t e = (int64_t)(in ? page[i] : 0) * c.page_stride + (int64_t)(token & (c.page_size - 1)) * c.token_stride;
        const int64_t at = e * (F8 ? 1 : 2) + head_bytes + piece() * 16;
        k[i] = *reinterpret_cast<const u32x4a*>(static_cast<const char*>(c.k) + at);
        v[i] = *reinterpret_cast<const u32x4a*>(static_cast<const char*>(c.v) + at);
        there |= (in && token < len ? 1u : 0u) << i;
      }
    }
  }

  // Puts the fetched tile into a buffer.  Values of tokens that are not there, and values of drafted tokens
  // that are infinite or NaN, are taken out (a row that does not attend the token would meet them as
  // 0 * inf); the latter are marked, and added by add_bad_tokens to the rows that attend them.
  __device__ __forceinline__ void put(int tile, int buf) {
    if ((tile + 1) * kTile > ctx) put_values<true>(tile, buf);
    else put_values<false>(tile, buf);
  }

  template <bool DRAFTED>
  __device__ __forceinline__ void put_values(int tile, int buf) {
#pragma unroll
    for (int i = 0; i < T::kPass; ++i) {
      const int r = i * T::kRows + row();
      const bool in = there >> i & 1;
      if (piece() == 0) lds.there[buf][r] = in;
      uint32_t keep = in ? ~0u : 0u;
      if constexpr (DRAFTED) {
        const bool bad = in && tile * kTile + r >= ctx && not_finite<F8>(v[i]);
        const uint64_t mine = ((1ull << T::kSrc) - 1) << ((threadIdx.x & 63) / T::kSrc * T::kSrc);
        const uint64_t any = __ballot(bad);
        if (any) lds.bad = 1;
        keep = any & mine ? 0u : keep;
      }
      const u32x4a kept = v[i] & keep;
      u32x4a* const kd = lds.kv[buf][0] + r * T::kPieces;
      u32x4a* const vd = lds.kv[buf][1] + r * T::kPieces;
      if constexpr (F8) {
        kd[(2 * piece()) ^ T::k_swizzle(r)] = widen(k[i][0], k[i][1]);
        kd[(2 * piece() + 1) ^ T::k_swizzle(r)] = widen(k[i][2], k[i][3]);
        vd[(2 * piece()) ^ T::v_swizzle(r)] = widen(kept[0], kept[1]);
        vd[(2 * piece() + 1) ^ T::v_swizzle(r)] = widen(kept[2], kept[3]);
      } else {
        kd[piece() ^ T::k_swizzle(r)] = k[i];
        vd[piece() ^ T::v_swizzle(r)] = kept;
      }
    }
  }
};

// A tile in one page of a BF16 cache goes from memory to LDS without passing through registers: a lane names the
// 16 bytes that belong in its place of a row (the swizzle is in the addresses).  The page table is read through the
// scalar cache, so nothing in the loop waits for a load but the barrier that ends it.  Tiles that have drafted or
// missing tokens (few) are gone over in LDS before they are used.
template <int D>
struct Direct {
  using T = Tile<D, false>;
  typedef __attribute__((address_space(4))) const int32_t scalar_i32;
  const w12_attention_args& a;
  const w12_kv_cache& c;
  Lds<D>& lds;
  scalar_i32* table;
  int page_bits, ctx, len;
  int64_t head_bytes;
  uint32_t koff[T::kPass], voff[T::kPass];

  __device__ __forceinline__ int row() const { return threadIdx.x / T::kSrc; }
  __device__ __forceinline__ int place() const { return threadIdx.x % T::kSrc; }

  __device__ __forceinline__ void begin(int b, int h, const Request& rq) {
    table = (scalar_i32*)(uintptr_t)(a.page_table + b * a.ld_table);
    ctx = rq.ctx;
    len = rq.len;
    head_bytes = (int64_t)h * c.head_stride * 2;
#pragma unroll
    for (int i = 0; i < T::kPass; ++i) {
      const int r = i * T::kRows + row();
      koff[i] = (uint32_t)r * (uint32_t)(c.token_stride * 2) + (place() ^ T::k_swizzle(r)) * 16;
      voff[i] = (uint32_t)r * (uint32_t)(c.token_stride * 2) + (place() ^ T::v_swizzle(r)) * 16;
    }
  }

  __device__ __forceinline__ int page_of(int tile) const { return table[uniform(tile * kTile >> page_bits)]; }
  __device__ __forceinline__ bool is_page(int p) const { return (uint32_t)p < (uint32_t)c.pages; }
  // Whether a tile has tokens to look at one by one.
  __device__ __forceinline__ bool special(int tile) const { return (tile + 1) * kTile > ctx || !is_page(page_of(tile)); }

  // Starts a tile's way into a buffer; wait_vm_all ends it.
  __device__ __forceinline__ void fetch(int tile, int buf) {
    const int p = page_of(tile);
    const int64_t base = ((int64_t)(is_page(p) ? p : 0) * c.page_stride + (int64_t)(tile * kTile & (c.page_size - 1)) * c.token_stride) * 2 +
                         head_bytes;
    const uint64_t kp = (uint64_t)(uintptr_t)c.k + base, vp = (uint64_t)(uintptr_t)c.v + base;
    const uint32_t wave_at = (uint32_t)wave_id() * 1024u;
#pragma unroll
    for (int i = 0; i < T::kPass; ++i) {
      to_lds(kp, koff[i], lds_off(lds.kv[buf][0]) + i * (kAttnThreads * 16) + wave_at);
      to_lds(vp, voff[i], lds_off(lds.kv[buf][1]) + i * (kAttnThreads * 16) + wave_at);
    }
  }
  // 16 bytes a lane from base + off to the wave's 1 KB of LDS at `at`.  Not through the builtin: the compiler would
  // wait for it before every read of LDS.
  __device__ __forceinline__ static void to_lds(uint64_t base, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(uniform((int)at)), "v"(off), "s"(base) : "memory", "m0");
  }

  // What put() does in Stream, in place.
  __device__ __forceinline__ void look_over(int tile, int buf) {
    const bool in_page = is_page(page_of(tile));
#pragma unroll
    for (int i = 0; i < T::kPass; ++i) {
      const int r = i * T::kRows + row();
      const bool in = in_page && tile * kTile + r < len;
      if (place() == 0) lds.there[buf][r] = in;
      u32x4a* const v = lds.kv[buf][1] + r * T::kPieces + place();
      const u32x4a was = *v;
      const bool bad = in && tile * kTile + r >= ctx && not_finite<false>(was);
      const uint64_t mine = ((1ull << T::kSrc) - 1) << ((threadIdx.x & 63) / T::kSrc * T::kSrc);
      const uint64_t any = __ballot(bad);
      if (any) lds.bad = 1;
      if (!in || (any & mine)) *v = u32x4a{0, 0, 0, 0};
    }
  }
};

// A wave's 32 rows (a lane: its row's elements of the query and result, shared with the lane 32 away).
template <int D>
struct Rows {
  bf16x8 q[D / 16];
  f32x16 o[D / 32];
  float m, l;        // m in score units (before the scale); l: this lane's half of the tokens
};

// Bits t of the 32 tokens from tok0 that the lane's row attends; valid: the tokens that are there.
__device__ __forceinline__ uint32_t attended(const w12_attention_args& a, int ctx, int row, int node, int tok0,
                                             uint32_t valid) {
  const int nb = tok0 - ctx;      // node number of the first token
  if (nb <= -32) return valid;
  const uint32_t cached = nb < 0 ? (1u << -nb) - 1 : 0;
  uint32_t sees;
  if (a.tree_mask) {
    const uint64_t* words = a.tree_mask + row * a.ld_mask;
    const int first = max(nb, 0), w = first >> 6, sh = first & 63;
    uint64_t bits = w < a.mask_words ? words[w] >> sh : 0;
    if (sh > 32 && w + 1 < a.mask_words) bits |= words[w + 1] << (64 - sh);
    sees = nb < 0 ? (uint32_t)bits << -nb : (uint32_t)bits;
  } else {
    const int count = node + 1 - nb;
    sees = count <= 0 ? 0 : count >= 32 ? ~0u : (1u << count) - 1;
  }
  return valid & (cached | sees);
}

// NS blocks of 32 tokens (from block `sub` of the tile in `buf`) for the wave's rows.  special: tokens may be missing
// or drafted.
template <int D, int NS, typename T>
__device__ __forceinline__ void attend(const w12_attention_args& a, const Lds<D>& lds, Rows<D>& x, int ctx, int tile, int buf,
                                       int sub, int row, int node, float scale, bool special) {
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5;
  constexpr int KS = D / 16, DB = D / 32;
  f32x16 sc[NS];
  // a lane's K operand: its token's row; the piece 2 ks + hi is the one for ks = 0 with bits of ks flipped
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(lds.kv[buf][0]) + (sub * 32 + col) * T::kRowBytes;
  const uint32_t kpiece = (uint32_t)(hi ^ T::k_swizzle(col)) * 16;
  // operands are read kAhead instructions before their use (left to itself the compiler reads them right before it)
  constexpr int kAhead = 4;
  u32x4a kf[kAhead];
  auto read_k = [&](int i) {
    kf[i % kAhead] = *reinterpret_cast<const u32x4a*>(kbase + i / KS * 32 * T::kRowBytes + (kpiece ^ (i % KS * 32u)));
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) read_k(i);
#pragma unroll
  for (int n = 0; n < NS; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[n][i] = 0.0f;
#pragma unroll
  for (int i = 0; i < NS * KS; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    sc[i / KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[i % kAhead]), x.q[i % KS], sc[i / KS], 0, 0, 0);
    if (i + kAhead < NS * KS) read_k(i + kAhead);
  }
  // a lane's V operand: 4 elements of one token, which the transposing read exchanges among 16 lanes
  const int g = lane >> 4, t4 = (lane & 15) >> 2;
  const int vtoken = 4 * (g >> 1) + t4;
  const uint8_t* vbase = reinterpret_cast<const uint8_t*>(lds.kv[buf][1]) + (sub * 32 + vtoken) * T::kRowBytes + (lane & 1) * 8;
  const uint32_t vpiece = (uint32_t)((2 * (g & 1) + ((lane & 3) >> 1)) ^ T::v_swizzle(vtoken)) * 16;
  constexpr int kVAhead = 4;
  s16x8 vf[kVAhead];
  auto read_v = [&](int i) {      // of 16 tokens i / DB, elements 32 (i % DB) .. + 31
    const uint8_t* at = vbase + i / DB * 16 * T::kRowBytes + (vpiece ^ (i % DB * 64u));
    const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
    const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 8 * T::kRowBytes));
    vf[i % kVAhead] = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
  };
#pragma unroll
  for (int i = 0; i < kVAhead; ++i) read_v(i);
  if (special) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int tok0 = tile * kTile + (sub + n) * 32;
      const uint32_t valid = (uint32_t)__ballot(lds.there[buf][(sub + n) * 32 + col] != 0);
      if (valid != ~0u || tok0 + 32 > ctx) {
        const uint32_t mine = attended(a, ctx, row, node, tok0, valid) >> (4 * hi);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!(mine >> (8 * (r >> 2) + (r & 3)) & 1)) sc[n][r] = -INFINITY;
      }
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int n = 0; n < NS; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[n][r]);
  top = fmaxf(top, other_half(top));
  // each row decides by itself, so that its result does not depend on the rows beside it
  const bool move = (top - x.m) * scale > kSlack;       // also true for the first finite score
  if (__any(move)) {
    const float m = move ? top : x.m;
    const float corr = move ? __builtin_amdgcn_exp2f((x.m - m) * scale) : 1.0f;
    x.m = m;
    x.l *= corr;
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) x.o[db][r] *= corr;
  }
  const float base = x.m == -INFINITY ? 0.0f : x.m * scale;
  // 16 tokens (u) at a time, and beside each of their matrix instructions a part of the next 16 tokens' exponentials: a
  // wave issues in order, so what is to run under a matrix instruction has to stand right behind it
  constexpr int kEach = 8 / DB > 0 ? 8 / DB : 1;
  u32x4a p[2];
  auto weigh = [&](int u, int i) {      // score i of 8
    float& l = x.l;
    const float e = __builtin_amdgcn_exp2f(sc[u / 2][8 * (u % 2) + i] * scale - base);
    l += e;
    sc[u / 2][8 * (u % 2) + i] = e;
    if (i % 2) p[u % 2][i / 2] = bf16_pair(sc[u / 2][8 * (u % 2) + i - 1], e);
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) weigh(0, i);
#pragma unroll
  for (int u = 0; u < 2 * NS; ++u)
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      const int i = u * DB + db;
      __builtin_amdgcn_sched_barrier(0);
      x.o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf[i % kVAhead]),
                                                        __builtin_bit_cast(bf16x8, p[u % 2]), x.o[db], 0, 0, 0);
      if (i + kVAhead < 2 * NS * DB) read_v(i + kVAhead);
      if (u + 1 < 2 * NS) {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (db * kEach + j < 8) weigh(u + 1, db * kEach + j);
      }
    }
}

// Drafted tokens of tiles [first, last) whose values were taken out (infinities, NaN): added one by one, element by
// element, to the rows of this wave that attend them (their weights are in l already).
template <int D, bool F8>
__device__ __forceinline__ void add_bad_tokens(const w12_attention_args& a, const w12_kv_cache& c, const Request& rq, int b, int h,
                                            int first, int last, int half, int row, int node, float scale, Rows<D>& x) {
  const int lane = threadIdx.x & 63, hi = lane >> 5, page_bits = 31 - __builtin_clz(c.page_size);
  auto at = [](const void* p, int64_t i) {
    if constexpr (F8) return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(p)[i], 0);
    else return bf16_float(static_cast<const uint16_t*>(p)[i]);
  };
  const float base = x.m == -INFINITY ? 0.0f : x.m * scale;
  for (int token = max(rq.ctx, first * kTile); token < min(rq.len, last * kTile); ++token) {
    if (half >= 0 && (token >> 5 & 1) != half) continue;
    const int page = a.page_table[b * a.ld_table + (token >> page_bits)];
    if ((uint32_t)page >= (uint32_t)c.pages) continue;
    const int64_t e = (int64_t)page * c.page_stride + (int64_t)(token & (c.page_size - 1)) * c.token_stride + (int64_t)h * c.head_stride;
    bool bad = false;
    for (int i = lane; i < D; i += 64) bad |= !(fabsf(at(c.v, e + i)) < INFINITY);
    if (!__any(bad)) continue;
    float s = 0.0f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s += (float)x.q[ks][i] * at(c.k, e + ks * 16 + hi * 8 + i);
      __builtin_amdgcn_sched_barrier(0);      // few loads at a time: registers are short here, time is not
    }
    s += other_half(s);
    if (!(attended(a, rq.ctx, row, node, token, 1u) & 1)) continue;
    const float p = __builtin_amdgcn_exp2f(s * scale - base);
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        x.o[db][r] += p * at(c.v, e + 32 * db + 8 * (r >> 2) + 4 * hi + (r & 3));
        if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
  }
}

template <int D, bool F8, bool WHOLE>
__global__ __launch_bounds__(kAttnThreads, D == 256 ? 1 : 2) void k_tree_attention(w12_attention_args a, w12_kv_cache c,
                                                                                    float* ws, int row_groups, int target, int64_t most) {
  using T = Tile<D, F8>;
  __shared__ Lds<D> lds;
  const int group = a.q_heads / c.heads;
  const int lane = threadIdx.x & 63, wave = wave_id(), col = lane & 31, hi = lane >> 5;
  const Plan plan = plan_items(a, c, group, target, lds.before, lds.sums);
  // physical work-group p runs on XCD p % 8, whose items are neighbours
  const int64_t x8 = blockIdx.x % 8, q8 = plan.items / 8, r8 = plan.items % 8, i8 = blockIdx.x / 8;
  if (i8 >= q8 + (x8 < r8)) return;
  const int64_t item = x8 * q8 + min(x8, r8) + i8;
  if (item >= most) return;      // ranges of node_ptr that decrease overlap: more items than the workspace has places for
  const int b = a.requests == 1 ? 0 : uniform(find_request(lds.before, a.requests, item));
  const Request rq = request_of(a, c.page_size, b);
  const Blocks bl = blocks_of(rq, group);
  const int chunks = (bl.tiles + plan.chunk - 1) / plan.chunk;
  const int in = (int)(item - (a.requests == 1 ? 0 : uniform(lds.before[b])));
  const int rb = in % bl.count(), chunk = in / bl.count() % chunks, h = in / bl.count() / chunks;
  const int w = rb < bl.full ? 4 : bl.rest;
  const int first = chunk * plan.chunk, last = min(first + plan.chunk, bl.tiles);
  constexpr bool kDirect = WHOLE && !F8;
  std::conditional_t<kDirect, Direct<D>, Stream<D, F8, WHOLE>> s{a, c, lds};
  s.page_bits = 31 - __builtin_clz(c.page_size);
  // this wave's rows: in a block of 4 every wave has 32 rows and all tokens, in one of 2 the waves
  // are two groups of rows by two halves of each tile
  const int rg = w == 4 ? wave : wave & 1, half = wave >> 1;
  const int rows = rq.nodes * group;
  const int r = rb * kBlockRows + rg * 32 + col;
  const bool active = rb * kBlockRows + rg * 32 < rows;      // uniform
  const bool mine = r < rows;
  const int node = mine ? r / group : 0;
  const int head = h * group + (mine ? r % group : 0);
  const int row = rq.start + node;
  const float scale = a.scale * kLog2e * (F8 ? c.k_scale[h] : 1.0f);
  s.begin(b, h, rq);
  if constexpr (kDirect) s.fetch(first, 0);
  else s.look_up(first);
  Rows<D> x;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    u32x4a q = {0, 0, 0, 0};
    if (mine) q = *reinterpret_cast<const u32x4a*>(a.q + row * a.ldq + head * D + ks * 16 + hi * 8);
    x.q[ks] = __builtin_bit_cast(bf16x8, q);
  }
  if constexpr (!kDirect) {
    s.fetch(first);
    s.look_up(min(first + 1, last - 1));
  }
#pragma unroll
  for (int db = 0; db < D / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) x.o[db][i] = 0.0f;
  x.m = -INFINITY;
  x.l = 0.0f;
  if (threadIdx.x == 0) lds.bad = 0;
  if constexpr (kDirect) {
    wait_vm_all();
    lds_barrier();
  } else {
    lds_barrier();
    s.put(first, 0);
    lds_barrier();
  }
  // The query is here before the loop: a load that is first used inside it would be waited for there, every time.
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) asm volatile("" : "+v"(x.q[ks]));
  // one loop for each kind of wave: paths that meet inside a loop cost copies of the result's registers
  auto run = [&](auto blocks, int sub) {
    for (int tile = first; tile < last; ++tile) {
      const int buf = (tile - first) & 1, next = min(tile + 1, last - 1);      // past the end: what the caches hold
      bool special = true;
      if constexpr (kDirect) {
        special = s.special(tile);
        if (special) {
          s.look_over(tile, buf);
          lds_barrier();
        }
        s.fetch(next, buf ^ 1);
      } else {
        s.fetch(next);
        s.look_up(min(tile + 2, last - 1));
      }
      if constexpr (blocks.value > 0) attend<D, blocks.value, T>(a, lds, x, rq.ctx, tile, buf, sub, row, node, scale, special);
      if constexpr (kDirect) wait_vm_all();
      else s.put(next, buf ^ 1);
      lds_barrier();
    }
  };
  if (!active) run(std::integral_constant<int, 0>(), 0);
  else if (w == 4) run(std::integral_constant<int, 2>(), 0);
  else run(std::integral_constant<int, 1>(), half);
  if (lds.bad && active) add_bad_tokens<D, F8>(a, c, rq, b, h, first, last, w == 4 ? -1 : half, row, node, scale, x);

  x.l += other_half(x.l);
  // two halves of the tokens: the second's rows go to the first's through LDS
  if (w != 4) {
    lds_barrier();      // lds.bad is read
    float* mine_at = reinterpret_cast<float*>(lds.kv) + (int64_t)(wave & 1) * 64 * (D / 2 + 2);
    if (active && half) {
#pragma unroll
      for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) mine_at[(db * 16 + i) * 64 + lane] = x.o[db][i];
      mine_at[(D / 2) * 64 + lane] = x.m;
      mine_at[(D / 2 + 1) * 64 + lane] = x.l;
    }
    lds_barrier();
    if (active && !half) {
      const float m2 = mine_at[(D / 2) * 64 + lane], l2 = mine_at[(D / 2 + 1) * 64 + lane];
      const float m = fmaxf(x.m, m2), base = m == -INFINITY ? 0.0f : m;
      const float f1 = exp2f((x.m - base) * scale), f2 = exp2f((m2 - base) * scale);
      x.m = m;
      x.l = x.l * f1 + l2 * f2;
#pragma unroll
      for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) x.o[db][i] = x.o[db][i] * f1 + mine_at[(db * 16 + i) * 64 + lane] * f2;
    }
  }
  if (!active || (w != 4 && half)) return;

  const float ms = x.m == -INFINITY ? -INFINITY : x.m * scale;
  if (chunks == 1) {
    const float inv = x.l == 0.0f ? 0.0f : (F8 ? c.v_scale[h] : 1.0f) / x.l;
    if (mine) {
#pragma unroll
      for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint2 v;
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = x.l == 0.0f ? 0.0f : x.o[db][4 * i + j] * inv;
          v.x = bf16_pair(e[0], e[1]);
          v.y = bf16_pair(e[2], e[3]);
          *reinterpret_cast<uint2*>(a.out + row * a.ldo + head * D + 32 * db + 8 * i + 4 * hi) = v;
        }
      if (a.lse && hi == 0) a.lse[row * a.ld_lse + head] = x.l == 0.0f ? -INFINITY : (ms + log2f(x.l)) / kLog2e;
    }
  } else {
    float* slot = ws + item * slot_floats(D, row_groups);
    float4* o4 = reinterpret_cast<float4*>(slot) + rg * (D / 8) * 64 + lane;
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o4[(db * 4 + i) * 64] = make_float4(x.o[db][4 * i], x.o[db][4 * i + 1], x.o[db][4 * i + 2], x.o[db][4 * i + 3]);
    if (hi == 0) {
      float2* ml = reinterpret_cast<float2*>(slot + (int64_t)row_groups * 32 * D);
      ml[rg * 32 + col] = make_float2(ms, x.l);
    }
  }
}

// Joins the partial results of blocks of several chunks: 32 rows and 8 elements at a time, the parts in the order of
// the chunks, eight in flight.  With few rows (SPLIT) each wave of a work-group takes a quarter of the parts and
// the first adds the quarters in their order; with many each wave has elements of its own.  Either way
// the order is the same every time, and with it every bit.
template <int D, bool F8, bool SPLIT>
__global__ __launch_bounds__(kAttnThreads) void k_join(w12_attention_args a, w12_kv_cache c, const float* ws,
                                                       int row_groups, int target, int64_t most) {
  constexpr int kWaves = kAttnThreads / 64;
  __shared__ int64_t before[kMaxRequests + 1], rows_before[kMaxRequests + 1], sums[kWaves];
  __shared__ float quarter[SPLIT ? kWaves : 1][6][64];
  const int group = a.q_heads / c.heads;
  const Plan plan = plan_items(a, c, group, target, before, sums);
  const int64_t x = blockIdx.x;
  int b = 0;
  if (a.requests > 1) {
    const int64_t all = prefix_requests(a.requests, rows_before, sums, [&](int i) {
      return (int64_t)(request_of(a, c.page_size, i).nodes * group + 31) / 32;
    });
    if (x >= all) return;
    b = uniform(find_request(rows_before, a.requests, x));
  }
  const Request rq = request_of(a, c.page_size, b);
  const Blocks bl = blocks_of(rq, group);
  const int chunks = (bl.tiles + plan.chunk - 1) / plan.chunk;
  const int rgx = (int)(x - (a.requests > 1 ? uniform(rows_before[b]) : 0)), rb = rgx / 4, rg = rgx % 4;
  if (chunks <= 1 || rgx * 32 >= rq.nodes * group) return;      // written whole, or no rows
  const int h = blockIdx.y, wave = wave_id();
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5;
  // the block's items: one a chunk, count() apart
  const int64_t item0 = (a.requests > 1 ? uniform(before[b]) : 0) + (int64_t)h * chunks * bl.count() + rb;
  if (item0 + (int64_t)(chunks - 1) * bl.count() >= most) return;
  const int64_t slot = slot_floats(D, row_groups) * 4, step = slot * bl.count();
  const char* part = reinterpret_cast<const char*>(ws) + item0 * slot;
  const uint32_t ml_off = (uint32_t)(row_groups * 32 * D * 4 + (rg * 32 + col) * 8);
  const int r = rgx * 32 + col;
  const int64_t row = rq.start + r / group;
  const int head = h * group + r % group;
  const int quad = SPLIT ? blockIdx.z : blockIdx.z * kWaves + wave;
  const uint32_t o_off = (uint32_t)((rg * (D / 8) + quad) * 64 + lane) * 16u;
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  auto add = [&](float m2, float l2, float4 o2) {
    const float mn = fmaxf(m, m2), base = mn == -INFINITY ? 0.0f : mn;
    const float f1 = exp2f(m - base), f2 = exp2f(m2 - base);
    m = mn;
    l = l * f1 + l2 * f2;
    o.x = o.x * f1 + o2.x * f2;
    o.y = o.y * f1 + o2.y * f2;
    o.z = o.z * f1 + o2.z * f2;
    o.w = o.w * f1 + o2.w * f2;
  };
  const int begin = SPLIT ? chunks * wave / kWaves : 0, end = SPLIT ? chunks * (wave + 1) / kWaves : chunks;
  for (int i0 = begin; i0 < end; i0 += 8) {
    float4 p[8];
    float2 ml[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const char* at = part + min(i0 + u, end - 1) * step;
      ml[u] = *reinterpret_cast<const float2*>(at + ml_off);
      p[u] = *reinterpret_cast<const float4*>(at + o_off);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u < end) add(ml[u].x, ml[u].y, p[u]);
  }
  if constexpr (SPLIT) {
    if (wave) {
      const float v[6] = {m, l, o.x, o.y, o.z, o.w};
#pragma unroll
      for (int i = 0; i < 6; ++i) quarter[wave][i][lane] = v[i];
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
      const float* q = &quarter[i][0][lane];
      add(q[0], q[64], make_float4(q[128], q[192], q[256], q[320]));
    }
  }
  if (r >= rq.nodes * group) return;
  const float inv = l == 0.0f ? 0.0f : (F8 ? c.v_scale[h] : 1.0f) / l;
  uint2 v = make_uint2(0, 0);
  if (l != 0.0f) {
    v.x = bf16_pair(o.x * inv, o.y * inv);
    v.y = bf16_pair(o.z * inv, o.w * inv);
  }
  *reinterpret_cast<uint2*>(a.out + row * a.ldo + head * D + 8 * quad + 4 * hi) = v;
  if (a.lse && quad == 0 && hi == 0) a.lse[row * a.ld_lse + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) / kLog2e;
}

// Items of four waves of two rounds of the work-groups that the chip holds at once (two a compute unit, one where a head
// of 256 takes its LDS).
static int attention_target(int D) { return 2 * device_cus() * (D == 256 ? 1 : 2); }
// Groups of 32 rows that a block can hold.
static int attention_row_groups(int32_t T, int32_t q_heads, const w12_kv_cache& c) {
  const int64_t rows = (int64_t)T * (q_heads / c.heads);
  return (int)(rows >= kBlockRows ? kBlockRows / 32 : ceil_div(rows, 32));
}
static int64_t attention_most_items(int32_t T, int32_t requests, int32_t q_heads, const w12_kv_cache& c) {
  return most_items((int64_t)T * (q_heads / c.heads), requests, c.heads, attention_target(c.dim));
}

uint64_t attention_workspace_bytes(int32_t T, int32_t requests, int32_t q_heads, const w12_kv_cache& c) {
  return (uint64_t)(attention_most_items(T, requests, q_heads, c) * slot_floats(c.dim, attention_row_groups(T, q_heads, c)) * 4);
}

template <int D, bool F8>
static hipError_t launch_attention(const w12_attention_args& a, const w12_kv_cache& c, float* ws, hipStream_t stream) {
  const int64_t groups = attention_most_items(a.T, a.requests, a.q_heads, c);
  const int target = attention_target(D);
  const int rg = attention_row_groups(a.T, a.q_heads, c);
  // tiles inside one page, with a thread's offsets in 32 bits (looked up token by token instead: 63 nodes over 32767
  // tokens 80 us for 68, with heads of 256 over 8191 44 for 32)
  const bool whole = c.page_size >= kTile && c.token_stride <= (int64_t(1) << 24);
  const dim3 g((unsigned)groups), t(kAttnThreads);
  if (whole) hipLaunchKernelGGL((k_tree_attention<D, F8, true>), g, t, 0, stream, a, c, ws, rg, target, groups);
  else hipLaunchKernelGGL((k_tree_attention<D, F8, false>), g, t, 0, stream, a, c, ws, rg, target, groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t row_blocks = ceil_div((int64_t)a.T * (a.q_heads / c.heads), 32) + a.requests;
  // few rows: waves share the parts (12 nodes over 8191 tokens 19.0 us, else 22.2; one node 16.4 and 19.9); many: they
  // share the work of finding the request, and a wave's parts are few (16 requests of 24 nodes, BF16, 93 us, else 116)
  const unsigned x = (unsigned)row_blocks, y = (unsigned)c.heads;
  if (row_blocks * c.heads < device_cus())
    hipLaunchKernelGGL((k_join<D, F8, true>), dim3(x, y, D / 8), t, 0, stream, a, c, (const float*)ws, rg, target, groups);
  else
    hipLaunchKernelGGL((k_join<D, F8, false>), dim3(x, y, D / 32), t, 0, stream, a, c, (const float*)ws, rg, target, groups);
  return hipGetLastError();
}

hipError_t launch_tree_attention(const w12_attention_args& a, const w12_kv_cache& c, void* ws, hipStream_t stream) {
  float* p = static_cast<float*>(ws);
  const bool f8 = c.dtype == W12_DTYPE_E4M3;
  switch (c.dim) {
    case 64: return f8 ? launch_attention<64, true>(a, c, p, stream) : launch_attention<64, false>(a, c, p, stream);
    case 128: return f8 ? launch_attention<128, true>(a, c, p, stream) : launch_attention<128, false>(a, c, p, stream);
    default: return f8 ? launch_attention<256, true>(a, c, p, stream) : launch_attention<256, false>(a, c, p, stream);
  }
}

}  // namespace w12
