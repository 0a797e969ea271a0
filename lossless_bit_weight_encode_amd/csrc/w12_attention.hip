// Attention of drafted tokens over a paged cache.
//
// The rows of a request that read one cache head (node i, query head g: row i * group + g) are cut
// into blocks of 128, the tokens into tiles of 64.  A block's tiles are a run of cost units (2 a tile
// for a block of up to 64 rows, 4 above); the runs of all heads, blocks and requests laid end to end
// are cut into equal shares, one a work-group, so unequal lengths load the chip evenly and a single
// request fills it.  A block whose tiles fall to several work-groups leaves partial results, which
// k_join adds in the order of the work-groups.
//
// A wave holds 32 rows: S^T = K Q^T by 32x32x16 matrix instructions leaves a row's scores in the
// two lanes of its column, so the softmax needs one exchange between lanes, and the registers of
// P^T are already the operand of O^T = V^T P^T (a sum over tokens, taken in the order in which the
// registers hold them; V is read from LDS transposed in the same order).  With a running maximum m,
//   p = exp2(c s - c m),  l = sum p,  O = sum p v,
// l and O are scaled only when a score passes m by 2^8 (p stays below 2^8).  P is rounded to BF16
// for the product (relative error 2^-8 of each p at most); everything else is FP32.
//
// Tiles go global -> registers -> LDS (double-buffered, 16-byte pieces swizzled by token so that
// both reads are free of bank conflicts) while the previous tile is computed on; E4M3 caches become BF16
// (exactly) on the way, their scales go into c and the result.
#include "w12_device.h"
#include "w12_gemm_common.h"
#include "w12_kernels.h"
#include "w12_rows.h"

namespace w12 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kAttnThreads = 256;
constexpr int kTile = 64;            // tokens of a tile
constexpr int kBlockRows = 128;      // rows of a block
constexpr int kMaxRequests = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;       // log2 of the largest p that a stale maximum may give
constexpr int kMinCost = 4;          // least cost units of a share (128 tokens of up to 64 rows)

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

struct Costs {
  int64_t head;    // cost units of one cache head
  int tiles, full, rest;   // tiles of a block; blocks of 128 rows; units a tile of the last, smaller block (0: none)
};

__device__ __forceinline__ Costs costs_of(const Request& r, int group) {
  Costs c;
  const int rows = r.nodes * group, rem = rows % kBlockRows;
  c.tiles = (r.len + kTile - 1) / kTile;
  c.full = rows / kBlockRows;
  c.rest = rem == 0 ? 0 : rem <= kBlockRows / 2 ? 2 : 4;
  c.head = (int64_t)c.tiles * (4 * c.full + c.rest);
  return c;
}

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

// The value of the lane 32 away.  The copy is kept apart from v: given one value twice, the
// compiler takes both results of the exchange for the same.
__device__ __forceinline__ float other_half(float v) {
  uint32_t a = __builtin_bit_cast(uint32_t, v), b = a;
  asm("" : "+v"(b));
  const auto sw = __builtin_amdgcn_permlane32_swap(a, b, false, false);   // (low halves, high halves)
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? sw[0] : sw[1]);
}

// Cost units of a work-group's share.
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t groups) {
  return max((total + groups - 1) / groups, (int64_t)kMinCost);
}

// Tiles [first, last) of a block (units from c0, w a tile) in the share [r0, r1).
__device__ __forceinline__ void tiles_in(int64_t c0, int w, int tiles, int64_t r0, int64_t r1, int* first, int* last) {
  const int sh = w == 4 ? 2 : 1;
  *first = (int)max((r0 - c0 + w - 1) >> sh, (int64_t)0);
  *last = (int)min((r1 - c0 + w - 1) >> sh, (int64_t)tiles);
}

__host__ __device__ constexpr int64_t slot_floats(int D, int row_groups) { return (int64_t)row_groups * 32 * (D + 2); }

template <int D, bool F8>
struct Tile {
  static constexpr int kRowBytes = D * 2;                       // BF16 in LDS
  static constexpr int kPieces = D / 8;                         // 16-byte pieces of a row in LDS
  static constexpr int kSrc = F8 ? D / 16 : D / 8;              // 16-byte loads of a row
  static constexpr int kRows = kAttnThreads / kSrc;             // rows of a load instruction of the work-group
  static constexpr int kPass = kTile / kRows;
  static constexpr int kBytes = kTile * kRowBytes;              // K or V of a tile
  // Reads of K take one piece of 32 tokens, reads of V 4 pieces of 8 tokens: the swizzles spread
  // each over all banks.
  __device__ static int k_piece(int token, int piece) { return piece ^ (token & (D == 64 ? 7 : 15)); }
  __device__ static int v_piece(int token, int piece) {
    return D == 64 ? piece ^ (((token >> 1) & 1) << 2) : piece ^ ((token & 3) << 2);
  }
};

// LDS: K and V of two tiles, then per tile and token whether it is there (bit 0) and whether its
// values were taken out for being infinite or NaN (bit 1).
template <int D>
struct Lds {
  uint4 kv[2][2][kTile * D / 8];
  uint8_t state[2][kTile];
  int64_t before[kMaxRequests + 1];
  int64_t sums[kAttnThreads / 64];
};

template <int D, bool F8>
struct Attention {
  using T = Tile<D, F8>;
  const w12_attention_args& a;
  const w12_kv_cache& c;
  Lds<D>& lds;
  int group, page_bits;
  // the segment
  int b, h;
  Request rq;
  // a thread's pieces of the next tile
  uint4 kreg[T::kPass], vreg[T::kPass];
  int page[T::kPass];
  uint32_t there;      // bit i: the token of pass i is there

  __device__ __forceinline__ int row_in_pass() const { return threadIdx.x / T::kSrc; }
  __device__ __forceinline__ int piece() const { return threadIdx.x % T::kSrc; }

  // The pages of a tile's tokens.
  __device__ __forceinline__ void look_up(int tile) {
#pragma unroll
    for (int i = 0; i < T::kPass; ++i) {
      const int token = tile * kTile + i * T::kRows + row_in_pass();
      page[i] = token < rq.len ? a.page_table[b * a.ld_table + (token >> page_bits)] : -1;
    }
  }

  // Start the loads of a tile whose pages are looked up.
  __device__ __forceinline__ void fetch(int tile) {
    there = 0;
#pragma unroll
    for (int i = 0; i < T::kPass; ++i) {
      const int token = tile * kTile + i * T::kRows + row_in_pass();
      kreg[i] = vreg[i] = make_uint4(0, 0, 0, 0);
      if ((uint32_t)page[i] < (uint32_t)c.pages) {
        there |= 1u << i;
        const int64_t e = (int64_t)page[i] * c.page_stride + (int64_t)(token & (c.page_size - 1)) * c.token_stride +
                          (int64_t)h * c.head_stride;
        const int64_t at = e * (F8 ? 1 : 2) + piece() * 16;
        kreg[i] = *reinterpret_cast<const uint4*>(static_cast<const char*>(c.k) + at);
        vreg[i] = *reinterpret_cast<const uint4*>(static_cast<const char*>(c.v) + at);
      }
    }
  }

  __device__ static bool not_finite(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F8) {
#pragma unroll
        for (int s = 0; s < 32; s += 8) bad |= ((w[i] >> s) & 0x7F) == 0x7F;
      } else {
        bad |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
      }
    }
    return bad;
  }

  // E4M3 to BF16: 16 bytes become two pieces.
  __device__ static void widen(uint4 u, uint4 out[2]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true));
    }
    out[0] = make_uint4(r[0], r[1], r[2], r[3]);
    out[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }

  // Put the fetched tile into a buffer.  Values of drafted tokens that are infinite or NaN are taken
  // out (a row that does not attend the token would meet them as 0 * inf) and marked.
  __device__ __forceinline__ void put(int tile, int buf) {
    const bool drafted = (tile + 1) * kTile > rq.ctx;
#pragma unroll
    for (int i = 0; i < T::kPass; ++i) {
      const int r = i * T::kRows + row_in_pass();
      uint32_t st = there >> i & 1;
      if (drafted) {
        const bool bad = tile * kTile + r >= rq.ctx && not_finite(vreg[i]);
        const uint64_t all = __ballot(bad);
        const int lane = threadIdx.x & 63;
        const uint64_t mine = T::kSrc == 64 ? ~0ull : ((1ull << T::kSrc) - 1) << (lane / T::kSrc * T::kSrc);
        if (all & mine) {
          vreg[i] = make_uint4(0, 0, 0, 0);
          st |= 2;
        }
      }
      if (piece() == 0) lds.state[buf][r] = (uint8_t)st;
      if constexpr (F8) {
        uint4 k2[2], v2[2];
        widen(kreg[i], k2);
        widen(vreg[i], v2);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          lds.kv[buf][0][r * T::kPieces + T::k_piece(r, 2 * piece() + j)] = k2[j];
          lds.kv[buf][1][r * T::kPieces + T::v_piece(r, 2 * piece() + j)] = v2[j];
        }
      } else {
        lds.kv[buf][0][r * T::kPieces + T::k_piece(r, piece())] = kreg[i];
        lds.kv[buf][1][r * T::kPieces + T::v_piece(r, piece())] = vreg[i];
      }
    }
  }
};

// A wave's 32 rows.
template <int D>
struct Rows {
  bf16x8 q[D / 16];
  f32x16 o[D / 32];
  float m, l;        // m in score units (before the scale); l: this lane's half of the tokens
};

// Bits t of the 32 tokens from tok0 that the lane's row attends; valid: the tokens that are there.
__device__ __forceinline__ uint32_t attended(const w12_attention_args& a, const Request& rq, int row, int node, int tok0,
                                             uint32_t valid) {
  const int nb = tok0 - rq.ctx;      // node number of the first token
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

// NS blocks of 32 tokens (from block `sub` of the tile in `buf`) for the wave's rows.
template <int D, bool F8, int NS>
__device__ __forceinline__ void attend(Attention<D, F8>& s, Rows<D>& x, int tile, int buf, int sub, int row, int node,
                                       float scale) {
  using T = Tile<D, F8>;
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5;
  f32x16 sc[NS];
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(s.lds.kv[buf][0]);
#pragma unroll
  for (int n = 0; n < NS; ++n) {
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[n][i] = 0.0f;
    const int token = (sub + n) * 32 + col;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint4 k = *reinterpret_cast<const uint4*>(kbase + token * T::kRowBytes + T::k_piece(token, 2 * ks + hi) * 16);
      sc[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, k), x.q[ks], sc[n], 0, 0, 0);
    }
  }
  // masks: needed where a token is missing or a drafted one is among them
  uint32_t sees[NS], bad[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    const int tok0 = tile * kTile + (sub + n) * 32;
    const uint8_t st = s.lds.state[buf][(sub + n) * 32 + col];
    const uint32_t valid = (uint32_t)__ballot(st & 1);
    bad[n] = (uint32_t)__ballot(st & 2);
    sees[n] = ~0u;
    if (valid != ~0u || tok0 + 32 > s.rq.ctx) {
      sees[n] = attended(s.a, s.rq, row, node, tok0, valid);
      const uint32_t mine = sees[n] >> (4 * hi);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (!(mine >> (8 * (r >> 2) + (r & 3)) & 1)) sc[n][r] = -INFINITY;
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
    const float corr = move ? exp2f((x.m - m) * scale) : 1.0f;
    x.m = m;
    x.l *= corr;
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) x.o[db][r] *= corr;
  }
  const float base = x.m == -INFINITY ? 0.0f : x.m * scale;
#pragma unroll
  for (int n = 0; n < NS; ++n) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      sc[n][r] = __builtin_amdgcn_exp2f(sc[n][r] * scale - base);
      x.l += sc[n][r];
    }
  }
  const uint8_t* vbase = reinterpret_cast<const uint8_t*>(s.lds.kv[buf][1]);
  const int g = lane >> 4, t4 = (lane & 15) >> 2;
#pragma unroll
  for (int n = 0; n < NS; ++n) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = bf16_pair(sc[n][8 * ks + 2 * i], sc[n][8 * ks + 2 * i + 1]);
      const bf16x8 pb = __builtin_bit_cast(bf16x8, make_uint4(p[0], p[1], p[2], p[3]));
#pragma unroll
      for (int db = 0; db < D / 32; ++db) {
        s16x4 v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int token = (sub + n) * 32 + 16 * ks + 8 * j + 4 * (g >> 1) + t4;
          const int pc = 4 * db + 2 * (g & 1) + ((lane & 3) >> 1);
          const uint8_t* at = vbase + token * T::kRowBytes + T::v_piece(token, pc) * 16 + (lane & 1) * 8;
          v[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
        }
        const uint2 lo = __builtin_bit_cast(uint2, v[0]), up = __builtin_bit_cast(uint2, v[1]);
        x.o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, up.x, up.y)), pb,
                                                          x.o[db], 0, 0, 0);
      }
    }
  }
  // drafted tokens whose values were taken out: added element by element to the rows that attend them
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    if (bad[n] == 0) continue;
    for (int t = 0; t < 32; ++t) {
      if (!(bad[n] >> t & 1)) continue;
      float p = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if ((t >> 3) == (r >> 2) && (t & 3) == (r & 3)) p = sc[n][r];
      p = __shfl(p, col + 32 * (t >> 2 & 1));
      const int token = tile * kTile + (sub + n) * 32 + t;
      const int page = s.a.page_table[s.b * s.a.ld_table + (token >> s.page_bits)];
      const int64_t e = (int64_t)page * s.c.page_stride + (int64_t)(token & (s.c.page_size - 1)) * s.c.token_stride +
                        (int64_t)s.h * s.c.head_stride;
      if (sees[n] >> t & 1) {
#pragma unroll
        for (int db = 0; db < D / 32; ++db)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int64_t i = e + 32 * db + 8 * (r >> 2) + 4 * hi + (r & 3);
            float v;
            if constexpr (F8) v = __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(s.c.v)[i], 0);
            else v = bf16_float(static_cast<const uint16_t*>(s.c.v)[i]);
            x.o[db][r] += p * v;
          }
      }
    }
  }
}

template <int D, bool F8>
__global__ __launch_bounds__(kAttnThreads, D == 256 ? 1 : 2) void k_tree_attention(w12_attention_args a, w12_kv_cache c,
                                                                                    float* ws, int row_groups) {
  using T = Tile<D, F8>;
  __shared__ Lds<D> lds;
  Attention<D, F8> s{a, c, lds};
  s.group = a.q_heads / c.heads;
  s.page_bits = 31 - __builtin_clz(c.page_size);
  const int lane = threadIdx.x & 63, wave = wave_id(), col = lane & 31, hi = lane >> 5;
  const int64_t total = uniform(prefix_requests(a.requests, lds.before, lds.sums, [&](int b) {
    return costs_of(request_of(a, c.page_size, b), s.group).head * c.heads;
  }));
  const int64_t share = share_of(total, gridDim.x);
  const int64_t g = logical_wg(blockIdx.x, gridDim.x);
  const int64_t r0 = g * share, r1 = min(r0 + share, total);
  int64_t at = r0;
  while (at < r1) {
    // the block that unit `at` belongs to
    s.b = uniform(find_request(lds.before, a.requests, at));
    s.rq = request_of(a, c.page_size, s.b);
    const Costs cs = costs_of(s.rq, s.group);
    const int64_t b0 = uniform(lds.before[s.b]);
    int64_t in = at - b0;
    s.h = (int)(in / cs.head);
    in -= s.h * cs.head;
    const int rb = (int)min(in / (4 * (int64_t)cs.tiles), (int64_t)cs.full);
    const int w = rb < cs.full ? 4 : cs.rest;
    const int64_t c0 = b0 + s.h * cs.head + (int64_t)rb * 4 * cs.tiles;
    const int64_t c1 = c0 + (int64_t)w * cs.tiles;
    int first, last;
    tiles_in(c0, w, cs.tiles, r0, r1, &first, &last);
    at = c1;
    if (first >= last) continue;

    // this wave's rows: with 4 units a tile every wave has 32 rows and all tokens, with 2 the waves
    // are two groups of rows by two halves of each tile
    const int rg = w == 4 ? wave : wave & 1, half = wave >> 1;
    const int rows = s.rq.nodes * s.group;
    const int r = rb * kBlockRows + rg * 32 + col;
    const bool active = rb * kBlockRows + rg * 32 < rows;      // uniform
    const bool mine = r < rows;
    const int node = mine ? r / s.group : 0;
    const int head = s.h * s.group + (mine ? r % s.group : 0);
    const int row = s.rq.start + node;
    const float scale = a.scale * kLog2e * (F8 ? c.k_scale[s.h] : 1.0f);
    Rows<D> x;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (mine) q = *reinterpret_cast<const uint4*>(a.q + row * a.ldq + head * D + ks * 16 + hi * 8);
      x.q[ks] = __builtin_bit_cast(bf16x8, q);
    }
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int i = 0; i < 16; ++i) x.o[db][i] = 0.0f;
    x.m = -INFINITY;
    x.l = 0.0f;

    s.look_up(first);
    s.fetch(first);
    s.look_up(first + 1);
    s.put(first, 0);
    lds_barrier();
    for (int tile = first; tile < last; ++tile) {
      const int buf = (tile - first) & 1;
      const bool more = tile + 1 < last;
      if (more) {
        s.fetch(tile + 1);
        s.look_up(tile + 2);
      }
      if (active) {
        if (w == 4) attend<D, F8, 2>(s, x, tile, buf, 0, row, node, scale);
        else attend<D, F8, 1>(s, x, tile, buf, half, row, node, scale);
      }
      if (more) s.put(tile + 1, buf ^ 1);
      lds_barrier();
    }

    {
      const float other = other_half(x.l);
      x.l = hi ? other + x.l : x.l + other;
    }
    // two halves of the tokens: the second's rows go to the first's through LDS
    if (w != 4) {
      float* park = reinterpret_cast<float*>(lds.kv);
      float* mine_at = park + (int64_t)(wave & 1) * 64 * (D / 2 + 2);
      if (active && half) {
#pragma unroll
        for (int db = 0; db < D / 32; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) mine_at[(db * 16 + i) * 64 + lane] = x.o[db][i];
        mine_at[(D / 2) * 64 + lane] = x.m;
        mine_at[(D / 2 + 1) * 64 + lane] = x.l;
      }
      __syncthreads();
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
      __syncthreads();
    }
    if (!active || (w != 4 && half)) continue;

    const float ms = x.m == -INFINITY ? -INFINITY : x.m * scale;
    if (first == 0 && last == cs.tiles) {
      const float inv = x.l == 0.0f ? 0.0f : (F8 ? c.v_scale[s.h] : 1.0f) / x.l;
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
      // a share meets at most two blocks that it does not hold whole: the one it starts in and the one it ends in
      float* slot = ws + (2 * g + (c0 > r0)) * slot_floats(D, row_groups);
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
}

// Joins the partial results of blocks that several work-groups share: a wave takes 32 rows and 8
// elements, and adds the parts in the order of the work-groups (bitwise the same every time).
template <int D, bool F8>
__global__ __launch_bounds__(kAttnThreads) void k_join(w12_attention_args a, w12_kv_cache c, const float* ws,
                                                       int row_groups, int64_t groups) {
  __shared__ int64_t before[kMaxRequests + 1], rows_before[kMaxRequests + 1], sums[kAttnThreads / 64];
  const int group = a.q_heads / c.heads;
  const int64_t total = prefix_requests(a.requests, before, sums, [&](int b) {
    return costs_of(request_of(a, c.page_size, b), group).head * c.heads;
  });
  const int64_t all = prefix_requests(a.requests, rows_before, sums, [&](int b) {
    return (int64_t)(request_of(a, c.page_size, b).nodes * group + 31) / 32;
  });
  const int64_t x = blockIdx.x;
  if (x >= all) return;
  const int h = blockIdx.y, quad = blockIdx.z * (kAttnThreads / 64) + wave_id();
  const int lane = threadIdx.x & 63, col = lane & 31, hi = lane >> 5;
  const int b = find_request(rows_before, a.requests, x);
  const Request rq = request_of(a, c.page_size, b);
  const Costs cs = costs_of(rq, group);
  const int rgx = (int)(x - rows_before[b]), rb = rgx / 4, rg = rgx % 4;
  const int w = rb < cs.full ? 4 : cs.rest;
  const int64_t c0 = before[b] + h * cs.head + (int64_t)rb * 4 * cs.tiles, c1 = c0 + (int64_t)w * cs.tiles;
  const int64_t share = share_of(total, groups);
  const int64_t g0 = c0 / share, g1 = (c1 - 1) / share;
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  for (int64_t g = g0; g <= g1; ++g) {
    int first, last;
    tiles_in(c0, w, cs.tiles, g * share, min((g + 1) * share, total), &first, &last);
    if (first == 0 && last == cs.tiles) return;        // whole: already written
    if (first >= last) continue;
    const float* slot = ws + (2 * g + (c0 > g * share)) * slot_floats(D, row_groups);
    const float4 p = reinterpret_cast<const float4*>(slot)[(rg * (D / 8) + quad) * 64 + lane];
    const float2 ml = reinterpret_cast<const float2*>(slot + (int64_t)row_groups * 32 * D)[rg * 32 + col];
    const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.0f : mn;
    const float f1 = exp2f(m - base), f2 = exp2f(ml.x - base);
    m = mn;
    l = l * f1 + ml.y * f2;
    o.x = o.x * f1 + p.x * f2;
    o.y = o.y * f1 + p.y * f2;
    o.z = o.z * f1 + p.z * f2;
    o.w = o.w * f1 + p.w * f2;
  }
  const int r = rgx * 32 + col;
  if (r >= rq.nodes * group) return;
  const int64_t row = rq.start + r / group;
  const int head = h * group + r % group;
  const float inv = l == 0.0f ? 0.0f : (F8 ? c.v_scale[h] : 1.0f) / l;
  uint2 v = make_uint2(0, 0);
  if (l != 0.0f) {
    v.x = bf16_pair(o.x * inv, o.y * inv);
    v.y = bf16_pair(o.z * inv, o.w * inv);
  }
  *reinterpret_cast<uint2*>(a.out + row * a.ldo + head * D + 8 * quad + 4 * hi) = v;
  if (a.lse && quad == 0 && hi == 0) a.lse[row * a.ld_lse + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) / kLog2e;
}

// Work-groups of a call: two a compute unit (one where a head of 256 takes its LDS).
static int64_t attention_groups(int D) { return (int64_t)device_cus() * (D == 256 ? 1 : 2); }
// Groups of 32 rows that a block can hold.
static int attention_row_groups(int32_t T, int32_t q_heads, const w12_kv_cache& c) {
  const int64_t rows = (int64_t)T * (q_heads / c.heads);
  return (int)(rows >= kBlockRows ? kBlockRows / 32 : ceil_div(rows, 32));
}

uint64_t attention_workspace_bytes(int32_t T, int32_t, int32_t q_heads, const w12_kv_cache& c) {
  return (uint64_t)(2 * attention_groups(c.dim) * slot_floats(c.dim, attention_row_groups(T, q_heads, c)) * 4);
}

template <int D, bool F8>
static hipError_t launch_attention(const w12_attention_args& a, const w12_kv_cache& c, float* ws, hipStream_t stream) {
  const int64_t groups = attention_groups(D);
  const int rg = attention_row_groups(a.T, a.q_heads, c);
  hipLaunchKernelGGL((k_tree_attention<D, F8>), dim3((unsigned)groups), dim3(kAttnThreads), 0, stream, a, c, ws, rg);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t row_blocks = ceil_div((int64_t)a.T * (a.q_heads / c.heads), 32) + a.requests;
  const dim3 grid((unsigned)row_blocks, (unsigned)c.heads, D / 8 / (kAttnThreads / 64));
  hipLaunchKernelGGL((k_join<D, F8>), grid, dim3(kAttnThreads), 0, stream, a, c, (const float*)ws, rg, groups);
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
