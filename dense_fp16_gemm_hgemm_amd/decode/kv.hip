// Appending keys and values to the paged 8-bit cache, and reading values back.
//
// Append.  With x the new row of a (page, head), rotated by its position:
//   s' = max(s, max |x| / QMAX),  code = rne(x / s'),
// and, where s' > s, the codes the page held become rne(code * s / s').  The
// maximum is over the page's new tokens, so one workgroup owns one (page,
// head) of K or of V: no atomics, and the result does not depend on order.
// The same launch turns the queries, in workgroups of their own.
//
// Work lies on lines of pages and of tokens, on which a wave finds its sequence
// with one load a lane: a grid of the longest sequence for each of a ragged
// batch would mostly start workgroups that find nothing (8 prompts of up to
// 4096 tokens, 4.9 k in all: 44 us in two launches, 26 so).
//
// Bounds: a call for one token of 64 sequences is latency (lengths, page, scale
// and row one after the other, 5.7 us); prompts move 110 MB at 4.2 TB/s, where
// a large copy reaches 5.0.  Divisions are exact, as codes at a border depend
// on the last bit; they stay below the loads' time.
#include "device.hpp"

namespace mid {
namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// Sixteen channels of one row: 8 and their 8 partners under rotation.
struct Chunk {
  f32x8 a, b;
};

// Where chunk c of a row lies: first channels of a and b, and whether it turns.
struct Place {
  int a, b;
  bool turns;
};
__device__ __forceinline__ Place place_of(int c, int rot_dim, bool interleaved) {
  if (16 * c >= rot_dim || interleaved) return {16 * c, 16 * c + 8, 16 * c < rot_dim};
  return {8 * c, rot_dim / 2 + 8 * c, true};
}

template <bool BF16>
__device__ __forceinline__ void load8(f32x8& x, const uint16_t* p) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = from16<BF16>((uint16_t)(w[i] & 0xffff));
    x[2 * i + 1] = from16<BF16>((uint16_t)(w[i] >> 16));
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(uint16_t* p, const f32x8& x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to16<BF16>(x[2 * i]) | (uint32_t)to16<BF16>(x[2 * i + 1]) << 16;
  *reinterpret_cast<u32x4*>(p) = w;
}

// The cosines and sines that a chunk's pairs are turned by.
struct Angles {
  f32x8 co, si;
};
__device__ __forceinline__ Angles load_angles(const AppendArgs& p, int c, int64_t pos) {
  Angles g;
  const float* row = p.rope + max(min(pos, p.rope_rows - 1), (int64_t)0) * p.rot_dim + 8 * c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(row + 4 * i);
    const f32x4 w = *reinterpret_cast<const f32x4*>(row + p.rot_dim / 2 + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) g.co[4 * i + e] = u[e], g.si[4 * i + e] = w[e];
  }
  return g;
}
// The row of rope for token t of the call, which comes to position pos.
__device__ __forceinline__ int64_t rope_row(const AppendArgs& p, int64_t t, int64_t pos) {
  return p.positions ? p.positions[t] : pos;
}
__device__ __forceinline__ void turn(Chunk& x, const Angles& g, bool interleaved) {
  if (!interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x.a[e], b = x.b[e];
      x.a[e] = a * g.co[e] - b * g.si[e];
      x.b[e] = b * g.co[e] + a * g.si[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = x.a[2 * e], b = x.a[2 * e + 1];
      x.a[2 * e] = a * g.co[e] - b * g.si[e];
      x.a[2 * e + 1] = b * g.co[e] + a * g.si[e];
      a = x.b[2 * e], b = x.b[2 * e + 1];
      x.b[2 * e] = a * g.co[4 + e] - b * g.si[4 + e];
      x.b[2 * e + 1] = b * g.co[4 + e] + a * g.si[4 + e];
    }
  }
}

// A chunk of a new key (turned) or value row: token t of the call, for position pos.
template <bool BF16>
__device__ __forceinline__ Chunk load_chunk(const AppendArgs& p, const uint16_t* row, int c, int64_t t, int64_t pos, bool rotate) {
  Chunk x;
  const Place at = place_of(c, rotate ? p.rot_dim : 0, p.interleaved);
  load8<BF16>(x.a, row + at.a);
  load8<BF16>(x.b, row + at.b);
  if (at.turns) turn(x, load_angles(p, c, rope_row(p, t, pos)), p.interleaved);
  return x;
}

// The sequence that token t of the call belongs to, by a whole wave: the last
// one that starts at t or before.
__device__ inline int sequence_of(const mi_decode_batch_t& k, int t) {
  if (k.cu == nullptr) return t;
  const int lane = threadIdx.x & 63;
  int b = 0;
  for (int at = 0; at < k.batch; at += 64) {
    const uint64_t m = __ballot(at + lane < k.batch && k.cu[min(at + lane, k.batch - 1)] <= t);
    if (m == 0) break;
    b = at + 63 - __builtin_clzll(m);
    if (m != ~0ull) break;
  }
  return b;
}
// The same from sequence b of an earlier token on.
__device__ inline int sequence_after(const mi_decode_batch_t& k, int b, int t) {
  if (k.cu == nullptr) return t;
  while (b + 1 < k.batch && k.cu[b + 1] <= t) ++b;
  return b;
}

// |x| as bits: their order is that of the values, infinities and NaN above.
__device__ inline uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// Eight codes, the nearest ones to y.
template <int CODE>
__device__ __forceinline__ u32x2 codes8(const f32x8& y) {
  u32x2 w = {0, 0};
  if constexpr (CODE == MI_DECODE_INT8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 4] |= (uint32_t)to_code<CODE>(y[e]) << (8 * (e % 4));
  } else {
    f32x8 z;
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = fminf(fmaxf(y[e], -448.f), 448.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * i], z[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z[4 * i + 2], z[4 * i + 3], v, true);
    }
  }
  return w;
}
template <int CODE>
__device__ __forceinline__ u32x2 pack8(const f32x8& x, float s) {
  f32x8 y;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = s > 0.f || s != s ? x[e] / s : 0.f;
  return codes8<CODE>(y);
}

// One (page, head) of K or V, page `line` of the call's.  D / 16 threads to a
// row; a thread's first KEEP rows stay in registers between the maximum and the
// codes.
template <int CODE, bool BF16, int D>
__device__ __forceinline__ void append_page(const AppendArgs& p, int line, int h, bool is_k) {
  constexpr int TPR = D / 16, KEEP = 2;
  const int ps = p.cache.page_size, H = p.cache.kv_heads, lane = threadIdx.x & 63;
  const int64_t cap = (int64_t)p.batch.table_cols * ps;
  // lane i knows sequence `at` + i and the line up to its pages
  int b = 0, j = 0;
  if (p.batch.max_tokens == 1) {
    b = line;
  } else {
    int before = 0;
    for (int at = 0;; at += 64) {
      int pages = 0;
      if (at + lane < p.batch.batch) {
        const Span sp = span_of(p.batch, at + lane);
        const int64_t past = min(max((int64_t)p.batch.lens[at + lane], (int64_t)0), cap);
        if (sp.n > 0) pages = (int)((past % ps + sp.n - 1) / ps) + 1;
      }
      int upto = pages;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
      }
      const uint64_t m = __ballot(before + upto > line);
      if (m) {
        const int l = __builtin_ctzll(m);
        b = at + l;
        j = line - before - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(pages, l));
        break;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
      if (at + 64 >= p.batch.batch) return;
    }
  }
  const Span sp = span_of(p.batch, b);
  const int64_t past = min(max((int64_t)p.batch.lens[b], (int64_t)0), cap);
  const int64_t col = past / ps + j;
  const int64_t start = col * ps;
  const int64_t lo = max(start, past), hi = min(start + ps, past + sp.n);
  if (lo >= hi) return;
  const int page = page_of(p.cache, p.batch, b, (int)min(col, (int64_t)p.batch.table_cols));
  if (page < 0) return;
  const int fill = (int)(lo - start);  // tokens that the page holds already

  const int64_t token_stride = is_k ? p.k.token_stride : p.v.token_stride;
  const uint16_t* base = static_cast<const uint16_t*>(is_k ? p.k.data : p.v.data) +
                         h * (is_k ? p.k.head_stride : p.v.head_stride);
  uint8_t* codes = static_cast<uint8_t*>(is_k ? p.cache.k : p.cache.v) + ((int64_t)page * H + h) * ps * D;
  float* scale = (is_k ? p.cache.k_scale : p.cache.v_scale) + (int64_t)page * H + h;

  const int tid = threadIdx.x, c = tid % TPR, r0 = tid / TPR, rows = blockDim.x / TPR;
  const int n = (int)(hi - lo);
  const int64_t t0 = sp.first + (lo - past);
  const float old = fill ? *scale : 0.f;
  auto fetch = [&](int r) { return load_chunk<BF16>(p, base + (t0 + r) * token_stride, c, t0 + r, lo + r, is_k); };
  uint32_t m = 0;
  auto widen = [&](const Chunk& x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, max(abs_bits(x.a[e]), abs_bits(x.b[e])));
  };
  Chunk kept[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) kept[k] = fetch(min(r0 + k * rows, n - 1));  // past the end the last row again
#pragma unroll
  for (int k = 0; k < KEEP; ++k) widen(kept[k]);
  for (int r = r0 + KEEP * rows; r < n; r += rows) widen(fetch(r));
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if (blockDim.x > 64) {
    __shared__ uint32_t part[4];
    if (tid % 64 == 0) part[tid / 64] = m;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 64; ++w) m = max(m, part[w]);
  }
  const float mine = __builtin_bit_cast(float, m) / kQmax<CODE>;
  const float s = abs_bits(mine) > abs_bits(old) ? mine : old;
  if (tid == 0) *scale = s;

  const Place at = place_of(c, is_k ? p.rot_dim : 0, p.interleaved);
  auto put = [&](int r, const Chunk& x) {
    uint8_t* to = codes + (fill + r) * D;
    *reinterpret_cast<u32x2*>(to + at.a) = pack8<CODE>(x.a, s);
    *reinterpret_cast<u32x2*>(to + at.b) = pack8<CODE>(x.b, s);
  };
#pragma unroll
  for (int k = 0; k < KEEP; ++k)
    if (r0 + k * rows < n) put(r0 + k * rows, kept[k]);
  for (int r = r0 + KEEP * rows; r < n; r += rows) put(r, fetch(r));
  if (fill && abs_bits(s) > abs_bits(old)) {
    const float ratio = old / s;
    const int all = fill * (D / 16);  // 16 codes at a time, four of them in flight
    for (int i = tid; i < all; i += 4 * blockDim.x) {
      u32x4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * (int)blockDim.x < all) w[k] = reinterpret_cast<const u32x4*>(codes)[i + k * blockDim.x];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i + k * (int)blockDim.x >= all) continue;
        u32x4 out;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          f32x8 y;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = from_code<CODE>((uint8_t)(w[k][2 * g + e / 4] >> (8 * (e % 4)))) * ratio;
          const u32x2 o = codes8<CODE>(y);
          out[2 * g] = o[0], out[2 * g + 1] = o[1];
        }
        reinterpret_cast<u32x4*>(codes)[i + k * blockDim.x] = out;
      }
    }
  }
}

// Queries turned by their positions: a thread takes a chunk of four heads, whose
// angles are the same.
template <bool BF16, int D>
__device__ __forceinline__ void turn_queries(const AppendArgs& p, int64_t item) {
  constexpr int TPR = D / 16, HEADS = 4;
  const int groups = (p.q_heads + HEADS - 1) / HEADS, per = TPR * groups;
  const int64_t t64 = item / per, first = (item - (threadIdx.x & 63)) / per;  // the thread's token, and its wave's
  int b = sequence_of(p.batch, (int)min(first, (int64_t)p.batch.tokens - 1));
  if (t64 >= p.batch.tokens) return;
  const int t = (int)t64, c = (int)(item % TPR), h0 = (int)(item % per) / TPR * HEADS;
  b = sequence_after(p.batch, b, t);
  const Span sp = span_of(p.batch, b);
  if (t < sp.first || t >= sp.first + sp.n) return;
  const int64_t cap = (int64_t)p.batch.table_cols * p.cache.page_size;
  const int64_t pos = min(max((int64_t)p.batch.lens[b], (int64_t)0), cap) + (t - sp.first);
  const Place at = place_of(c, p.rot_dim, p.interleaved);
  const uint16_t* row = static_cast<const uint16_t*>(p.q.data) + t * p.q.token_stride;
  uint16_t* to = static_cast<uint16_t*>(p.q_out.data) + t * p.q_out.token_stride;
  Angles g;
  if (at.turns) g = load_angles(p, c, rope_row(p, t, pos));
  Chunk x[HEADS];
#pragma unroll
  for (int k = 0; k < HEADS; ++k)
    if (h0 + k < p.q_heads) {
      load8<BF16>(x[k].a, row + (h0 + k) * p.q.head_stride + at.a);
      load8<BF16>(x[k].b, row + (h0 + k) * p.q.head_stride + at.b);
    }
#pragma unroll
  for (int k = 0; k < HEADS; ++k)
    if (h0 + k < p.q_heads) {
      if (at.turns) turn(x[k], g, p.interleaved);
      store8<BF16>(to + (h0 + k) * p.q_out.head_stride + at.a, x[k].a);
      store8<BF16>(to + (h0 + k) * p.q_out.head_stride + at.b, x[k].b);
    }
}

// Workgroups 0 .. page_blocks - 1 append, the others turn queries.
template <int CODE, bool BF16, int D>
__global__ __launch_bounds__(256, 4) void append_kernel(AppendArgs p, int page_blocks) {
  const int id = blockIdx.x;
  if (id < page_blocks) {
    const int each = 2 * p.cache.kv_heads;
    append_page<CODE, BF16, D>(p, id / each, id % each / 2, id & 1);
  } else {
    turn_queries<BF16, D>(p, (int64_t)(id - page_blocks) * blockDim.x + threadIdx.x);
  }
}

// Values of cached tokens, 16 to a thread.
template <int CODE, bool BF16>
__global__ __launch_bounds__(256) void read_kernel(ReadArgs p) {
  const int H = p.cache.kv_heads, D = p.cache.head_dim, ps = p.cache.page_size;
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = H * D / 16;
  const int64_t t64 = item / per, first = (item - (threadIdx.x & 63)) / per;
  int b = sequence_of(p.batch, (int)min(first, (int64_t)p.batch.tokens - 1));
  if (t64 >= p.batch.tokens) return;
  const int t = (int)t64, at = (int)(item % per) * 16, h = at / D, d = at % D;
  b = sequence_after(p.batch, b, t);
  const Span sp = span_of(p.batch, b);
  if (t < sp.first || t >= sp.first + sp.n) return;
  const int64_t pos = (int64_t)p.batch.lens[b] + (t - sp.first);
  const int page = pos < 0 ? -1 : page_of(p.cache, p.batch, b, (int)min(pos / ps, (int64_t)INT32_MAX));
  u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
  float sk = 0.f, sv = 0.f;
  if (page >= 0) {
    const int64_t ph = (int64_t)page * H + h;
    const int64_t off = (ph * ps + pos % ps) * D + d;
    k = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p.cache.k) + off);
    v = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p.cache.v) + off);
    sk = p.cache.k_scale[ph], sv = p.cache.v_scale[ph];
  }
  const int64_t to = (int64_t)t * H * D + at;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    f32x8 x, y;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = from_code<CODE>((uint8_t)(k[2 * g + e / 4] >> (8 * (e % 4)))) * sk;
      y[e] = from_code<CODE>((uint8_t)(v[2 * g + e / 4] >> (8 * (e % 4)))) * sv;
    }
    store8<BF16>(static_cast<uint16_t*>(p.k_out) + to + 8 * g, x);
    store8<BF16>(static_cast<uint16_t*>(p.v_out) + to + 8 * g, y);
  }
}

template <int CODE, bool BF16, int D>
hipError_t append(const AppendArgs& a, hipStream_t s) {
  const int ps = a.cache.page_size;
  // A sequence's n tokens lie on n / ps + 1 pages at most, or one more.
  const int64_t pages = a.batch.max_tokens == 1 ? a.batch.batch : a.batch.tokens / ps + 2 * (int64_t)a.batch.batch;
  const int64_t page_blocks = 2 * (int64_t)a.cache.kv_heads * pages;
  const int threads = a.batch.max_tokens <= 1024 / D ? 64 : 256;
  const int64_t items = (int64_t)a.batch.tokens * ((a.q_heads + 3) / 4) * (D / 16);
  const int64_t blocks = page_blocks + (a.q_heads ? (items + threads - 1) / threads : 0);
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  return launch(append_kernel<CODE, BF16, D>, dim3((unsigned)blocks), threads, 0, s, a, (int)page_blocks);
}

template <int CODE, bool BF16>
hipError_t append(const AppendArgs& a, hipStream_t s) {
  switch (a.cache.head_dim) {
    case 64: return append<CODE, BF16, 64>(a, s);
    case 128: return append<CODE, BF16, 128>(a, s);
    default: return append<CODE, BF16, 256>(a, s);
  }
}

template <int CODE, bool BF16>
hipError_t read(const ReadArgs& a, hipStream_t s) {
  const int64_t items = (int64_t)a.batch.tokens * a.cache.kv_heads * (a.cache.head_dim / 16);
  const int64_t x = (items + 255) / 256;
  if (x > INT32_MAX) return hipErrorInvalidConfiguration;
  return launch(read_kernel<CODE, BF16>, dim3((unsigned)x), 256, 0, s, a);
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
  if (a.cache.code == MI_DECODE_INT8)
    return a.bf16 ? append<MI_DECODE_INT8, true>(a, s) : append<MI_DECODE_INT8, false>(a, s);
  return a.bf16 ? append<MI_DECODE_E4M3, true>(a, s) : append<MI_DECODE_E4M3, false>(a, s);
}

hipError_t launch_read(const ReadArgs& a, hipStream_t s) {
  if (a.cache.code == MI_DECODE_INT8)
    return a.bf16 ? read<MI_DECODE_INT8, true>(a, s) : read<MI_DECODE_INT8, false>(a, s);
  return a.bf16 ? read<MI_DECODE_E4M3, true>(a, s) : read<MI_DECODE_E4M3, false>(a, s);
}

}  // namespace mid
