// What the two attention kernels share: operands from codes, row blocks, and
// the last workgroup's sum over the parts of a row block.
#pragma once

#include "device.hpp"

namespace mid {
namespace {

constexpr int kRsrcWord3 = 0x00020000;
constexpr int kDeviceScope = 16;  // cache policy SC1
constexpr float kTiny = 0x1p-24f;  // int8 codes as operands are in units of this
// Weights as operands go up to binary16's upper end: m is kept kBelow under the
// largest exponent that it was set by, and set again when a weight would pass
// 2^kMost.  So weights down to 2^-26 of the largest have all 11 bits and vanish
// below 2^-37 (a long flat context beside one dominant token: with weights of
// at most 1, those below 2^-14 lost bits and those below 2^-25 everything).
constexpr float kBelow = 12.f, kMost = 15.f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ inline f32x16 mma(h8 a, h8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
__device__ inline f32x4 mma(h8 a, h8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// over the lanes that share lane % 16
template <typename F>
__device__ inline float join16(float x, F f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t a0 = a[0], a1 = a[1];
  const uint32_t w = __builtin_bit_cast(uint32_t, f(__builtin_bit_cast(float, a0), __builtin_bit_cast(float, a1)));
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const uint32_t b0 = b[0], b1 = b[1];
  return f(__builtin_bit_cast(float, b0), __builtin_bit_cast(float, b1));
}
__device__ inline float max16(float x) { return join16(x, [](float a, float b) { return fmaxf(a, b); }); }
__device__ inline float sum16(float x) { return join16(x, [](float a, float b) { return a + b; }); }
__device__ inline int lane_value(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ inline float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// What a row of bf16 queries is multiplied by to become binary16: its largest
// magnitude goes to [2^15, 2^16).  Channels down to 2^-32 of that one keep their
// 8 bits then, and they vanish below 2^-40.  binary16 queries stay as they are.
__device__ inline float query_unit(float top) {
  const int ex = top > 0.f && top < INFINITY ? (int)(__builtin_bit_cast(uint32_t, top) >> 23) : 142;
  return __builtin_bit_cast(float, (uint32_t)min(269 - ex, 254) << 23);
}

// An infinite key scale makes its codes' values infinite or NaN (0), and the
// logits of a page with both NaN; infinity times the sum of codes would have a
// sign, and a negative one would drop the token.
__device__ inline float key_scale(float k) { return fabsf(k) < INFINITY ? k : NAN; }

// A page's value scale as 2^log times rest.  rest is 1 for scales of at least
// 2^-80; smaller ones count as 2^-80 (no logarithm for 0, and no weight that
// leaves binary32), and it has the sign and whatever is not finite.
struct ValueScale {
  float log, rest;
};
__device__ inline ValueScale value_scale(float v) {
  const bool finite = fabsf(v) < INFINITY, small = fabsf(v) < 0x1p-80f;
  return {small ? -80.f : finite ? __builtin_amdgcn_logf(fabsf(v)) : 0.f,
          small ? v * 0x1p80f : finite ? copysignf(1.f, v) : v};
}
// 2^10 / 2^log: sums of weights are in units of 2^-10, which keeps them within
// binary32 for scales from 2^-80 (and a million tokens) to 2^128.
__device__ inline float inverse(float log) { return __builtin_amdgcn_exp2f(10.f - log); }
// What a sum of weights times codes is multiplied by, to go over such a sum of weights.
template <int CODE>
constexpr float kUnit = CODE == MI_DECODE_INT8 ? 0x1p10f / kTiny : 0x1p10f;

// Two bytes code + 128 in 16-bit slots as two numbers code 2^-24.
__device__ inline uint32_t centred(uint32_t w) {
  const _Float16 off = (_Float16)(-128.f * kTiny);
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, w) + h2{off, off});
}

// Eight codes of one token as eight numbers, in order.
template <int CODE>
__device__ inline h8 along(uint32_t w0, uint32_t w1) {
  u32x4 o;
  if constexpr (CODE == MI_DECODE_INT8) {
    w0 ^= 0x80808080u, w1 ^= 0x80808080u;
    o[0] = centred(__builtin_amdgcn_perm(0u, w0, 0x0c010c00u));
    o[1] = centred(__builtin_amdgcn_perm(0u, w0, 0x0c030c02u));
    o[2] = centred(__builtin_amdgcn_perm(0u, w1, 0x0c010c00u));
    o[3] = centred(__builtin_amdgcn_perm(0u, w1, 0x0c030c02u));
  } else {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true));
  }
  return __builtin_bit_cast(h8, o);
}

// Channels 2 B and 2 B + 1 of eight tokens' words as eight numbers each, in token order.
template <int CODE, int B>
__device__ inline void across(const uint32_t (&w)[8], h8& even, h8& odd) {
  u32x4 e, o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t0 = w[2 * i], t1 = w[2 * i + 1];
    if constexpr (CODE == MI_DECODE_INT8) {
      e[i] = centred(__builtin_amdgcn_perm(t1, t0, 0x0c040c00u + 0x00020002u * B));
      o[i] = centred(__builtin_amdgcn_perm(t1, t0, 0x0c050c01u + 0x00020002u * B));
    } else {
      const uint32_t y = __builtin_amdgcn_perm(t1, t0, 0x05010400u + 0x02020202u * B);
      e[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.f, false));
      o[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.f, true));
    }
  }
  even = __builtin_bit_cast(h8, e);
  odd = __builtin_bit_cast(h8, o);
}

// One row block of one sequence.
template <int TILE>
struct Block {
  int first, rows;  // the sequence's first token, the block's rows
  int r0;           // the block's first row
  int start;        // position of the sequence's first query token
  int plo, phi;     // positions of the block's first and last row
  int ns, lo;       // tiles of sinks, and the first tile after them
  int tiles;        // 0: no rows
  int b;            // the sequence
  __device__ int token(int t) const { return TILE * (t < ns ? t : lo + t - ns); }
  __device__ Block of_lane(int l) const {
    Block k;
    k.first = __builtin_amdgcn_readlane(first, l), k.rows = __builtin_amdgcn_readlane(rows, l);
    k.r0 = __builtin_amdgcn_readlane(r0, l), k.start = __builtin_amdgcn_readlane(start, l);
    k.plo = __builtin_amdgcn_readlane(plo, l), k.phi = __builtin_amdgcn_readlane(phi, l);
    k.ns = __builtin_amdgcn_readlane(ns, l), k.lo = __builtin_amdgcn_readlane(lo, l);
    k.tiles = __builtin_amdgcn_readlane(tiles, l), k.b = __builtin_amdgcn_readlane(b, l);
    return k;
  }
};
//
// In a tree every row may see up to the sequence's last token, and `plo` is the
// last position that the drafts' bits do not speak of: rows stand at plo + 1 at
// least, which moves a window's border by one in what is loaded, and what is
// seen of that goes by each row's own position.
template <int TILE, bool TREE>
__device__ inline Block<TILE> block_of(const AttendArgs& p, int G, int block_rows, int blocks, int pair, int pairs) {
  Block<TILE> k = {};
  if (pair >= pairs) return k;
  const int b = blocks == 1 ? pair : pair / blocks, rb = pair - b * blocks;
  k.b = b;
  const int held = p.batch.lens[b];  // requested before the tokens' bounds are waited for
  const Span sp = span_of(p.batch, b);
  const int64_t cap = (int64_t)p.batch.table_cols * p.cache.page_size;
  const int len = (int)min((int64_t)max(held, 0), cap);
  k.first = sp.first;
  k.r0 = rb * block_rows;
  const int64_t all = (int64_t)min(sp.n, p.batch.max_tokens) * G;
  k.rows = (int)min((int64_t)block_rows, all - k.r0);
  k.start = len - sp.n;
  k.plo = k.start + k.r0 / G;
  k.phi = k.start + (k.r0 + k.rows - 1) / G;
  if (TREE) k.plo = k.start - 1, k.phi = len - 1;
  if (p.window) {
    const int lo = max(0, k.plo - p.window + 1);
    k.lo = lo / TILE;
    k.ns = min((int)(((int64_t)min(p.sinks, max(k.phi + 1, 0)) + TILE - 1) / TILE), k.lo);
  }
  k.tiles = k.rows <= 0 ? 0 : max(1, k.ns + max(k.phi, 0) / TILE + 1 - k.lo);
  return k;
}

// A row of a tree: its token of the call, and with a window the first position
// of the context that is in it.
struct TreeRow {
  int token;  // -1: there is no row
  int from;
};
__device__ inline uint32_t seen_word(const AttendArgs& p, int token, int w) {
  return w < p.seen_words ? (uint32_t)p.seen[token * p.seen_stride + w] : 0u;
}
// Token `i` of the n drafted ones, which lie from position start on and begin with token `first` of the call.
__device__ inline TreeRow tree_row(const AttendArgs& p, int first, int i, int n, int start, bool in) {
  TreeRow t = {in ? first + i : -1, 0};
  if (p.window && in) {
    int others = 0;
    for (int w = 0; 32 * w < n; ++w) {
      uint32_t x = seen_word(p, t.token, w);
      if (n - 32 * w < 32) x &= (1u << (n - 32 * w)) - 1;
      if (i / 32 == w) x &= ~(1u << (i % 32));
      others += __builtin_popcount(x);
    }
    t.from = start + others - p.window + 1;
  }
  return t;
}
// Which of the positions at .. at + 31 a row sees, as bits.
__device__ inline uint32_t tree_bits32(const AttendArgs& p, const TreeRow& t, int n, int start, int at) {
  auto ones = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
  if (t.token < 0) return 0;
  const int off = at - start;
  uint32_t drafts = 0;
  if (off > -32 && off < n) {
    const uint32_t lo = seen_word(p, t.token, max(off, 0) / 32), hi = seen_word(p, t.token, off / 32 + 1);
    drafts = (off < 0 ? lo << -off : __builtin_amdgcn_alignbit(hi, lo, off % 32)) & ones(n - off);
  }
  uint32_t context = ones(-off);
  if (p.window) context &= ~ones(t.from - at) | ones(p.sinks - at);
  return context | drafts;
}
// At .. at + 63.
__device__ inline uint64_t tree_bits64(const AttendArgs& p, const TreeRow& t, int n, int start, int at) {
  return tree_bits32(p, t, n, start, at) | (uint64_t)tree_bits32(p, t, n, start, at + 32) << 32;
}

// Four channels of a row's result: row r of the sequence whose first token is
// `first`, key-value head h.
__device__ inline void store_row(const AttendArgs& p, int first, int r, int h, int G, int d, f32x4 x, float sum) {
  uint16_t* out = static_cast<uint16_t*>(p.out.data) + (first + r / G) * p.out.token_stride +
                  (h * G + r % G) * p.out.head_stride + d;
  u32x2 y = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float v = sum == 0.f ? 0.f : x[k] / sum;
    y[k / 2] |= (uint32_t)(p.bf16 ? to16<true>(v) : to16<false>(v)) << (16 * (k % 2));
  }
  *reinterpret_cast<u32x2*>(out) = y;
}

// A part in the workspace: sums of ROWS x D, then m and l of each row.
__host__ __device__ constexpr uint32_t part_bytes(int rows, int D) { return 4 * (uint32_t)rows * (D + 2); }

// Counts a workgroup in whose part is stored; true in the last of `parts`.
//
// Workgroups of one item run on XCDs whose L2 caches are not coherent.  Parts
// are stored and loaded with device scope, past those caches, and counted when
// their stores are acknowledged; fences would write back and drop whole caches
// instead (15 to 25 us between the two).
__device__ inline bool last_to_arrive(int* cnt, int parts, int* flag) {
  __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8));  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0) *flag = __hip_atomic_fetch_add(cnt, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
  __syncthreads();
  return *flag;
}

// A row block in parts: part 0 lies at `head`, part n at `tail` + (n - 1) `step`.
__device__ inline uint32_t part_at(const JoinItem& it, int n) { return n == 0 ? it.head : it.tail + (uint32_t)(n - 1) * it.step; }

// Adds the parts of rows r0 .. r0 + rows - 1 of a block in order and stores the
// result; smem: room for 6 THREADS floats.
//
// A thread adds four channels of a row over every groups-th part; where there
// are few rows, groups of threads share the parts.  DEPTH parts' loads are in
// flight at a time: one after the other, a part costs the memory's latency (32
// parts of 4 rows: 45 us).
template <int D, int THREADS, int DEPTH, typename Rsrc>
__device__ inline void join_parts(const AttendArgs& p, const Rsrc& parts_rsrc, const JoinItem& it, int block_rows,
                                  int r0, int rows, float* smem) {
  const int tid = threadIdx.x, G = p.q_heads / p.cache.kv_heads, parts = it.parts;
  const int all = rows * (D / 4);
  int groups = 1;
  while (groups < 8 && 2 * groups * all <= THREADS && 2 * groups <= parts) groups *= 2;
  const int per = THREADS / groups, grp = tid / per;
  for (int e = tid % per; e < all; e += per) {
    const int rr = r0 + e / (D / 4), d = e % (D / 4) * 4;
    float top = -INFINITY, sum = 0.f;
    f32x4 x = {0, 0, 0, 0};
    for (int n = grp; n < parts; n += DEPTH * groups) {
      float pm[DEPTH], pl[DEPTH];
      f32x4 px[DEPTH];
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        const uint32_t s = part_at(it, min(n + k * groups, parts - 1));
        const f32x2 ml = __builtin_bit_cast(
            f32x2, __builtin_amdgcn_raw_buffer_load_b64(parts_rsrc, s + 4 * (block_rows * D + 2 * rr), 0, kDeviceScope));
        pm[k] = ml[0], pl[k] = ml[1];
        px[k] = __builtin_bit_cast(
            f32x4, __builtin_amdgcn_raw_buffer_load_b128(parts_rsrc, s + 4 * (rr * D + d), 0, kDeviceScope));
      }
      float t1 = top;
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) t1 = fmaxf(t1, pm[k]);
      const float base = t1 == -INFINITY ? 0.f : t1, down = __builtin_amdgcn_exp2f(top - base);
      top = t1, x *= down, sum *= down;
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        if (n + k * groups >= parts) break;
        const float f = __builtin_amdgcn_exp2f(pm[k] - base);
        sum += f * pl[k];
        x += f * px[k];
      }
    }
    if (groups > 1) {  // then every thread has one element at most
      float* mine = smem + 6 * tid;
      mine[0] = top, mine[1] = sum;
      mine[2] = x[0], mine[3] = x[1], mine[4] = x[2], mine[5] = x[3];
    } else {
      store_row(p, it.first, it.r0 + rr, it.h, G, d, x, sum);
    }
  }
  if (groups > 1) {
    __syncthreads();
    for (int e = tid; e < all; e += THREADS) {
      float top = -INFINITY, sum = 0.f;
      f32x4 x = {0, 0, 0, 0};
      for (int k = 0; k < groups; ++k) top = fmaxf(top, smem[6 * (k * per + e)]);
      const float base = top == -INFINITY ? 0.f : top;
      for (int k = 0; k < groups; ++k) {
        const float* s = smem + 6 * (k * per + e);
        const float f = __builtin_amdgcn_exp2f(s[0] - base);
        sum += f * s[1];
        x += f * f32x4{s[2], s[3], s[4], s[5]};
      }
      store_row(p, it.first, it.r0 + r0 + e / (D / 4), it.h, G, e % (D / 4) * 4, x, sum);
    }
  }
}

}  // namespace
}  // namespace mid
