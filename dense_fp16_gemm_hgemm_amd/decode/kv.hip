// Appending keys and values to the paged 8-bit cache, and reading values back.
//
// Append.  With x the new row of a (page, head), rotated by its position:
//   s' = max(s, max |x| / QMAX),  code = rne(x / s'),
// and, where s' > s, the codes the page held become rne(code * s / s').  The
// maximum is over the page's new tokens, so one workgroup owns one (page,
// head) of K or of V: no atomics, and the result does not depend on order.
#include "device.hpp"

namespace mid {
namespace {

// Sixteen channels of one row: 8 and their 8 partners under rotation.
struct Chunk {
  float a[8], b[8];
};

// Where chunk c of a row lies: first channels of a and b, and whether it turns.
struct Place {
  int a, b;
  bool turns;
};
__device__ inline Place place_of(int c, int rot_dim, bool interleaved) {
  if (16 * c >= rot_dim || interleaved) return {16 * c, 16 * c + 8, 16 * c < rot_dim};
  return {8 * c, rot_dim / 2 + 8 * c, true};
}

template <bool BF16>
__device__ inline void load8(float (&x)[8], const uint16_t* p) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = from16<BF16>((uint16_t)(w[i] & 0xffff));
    x[2 * i + 1] = from16<BF16>((uint16_t)(w[i] >> 16));
  }
}
template <bool BF16>
__device__ inline void store8(uint16_t* p, const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to16<BF16>(x[2 * i]) | (uint32_t)to16<BF16>(x[2 * i + 1]) << 16;
  *reinterpret_cast<u32x4*>(p) = w;
}

// a, b turned by the angles whose cosines and sines lie in `rope`'s row.
__device__ inline void turn(Chunk& x, const float* row, int half, int c, bool interleaved) {
  float co[8], si[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(row + 8 * c + 4 * i);
    const f32x4 w = *reinterpret_cast<const f32x4*>(row + half + 8 * c + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) co[4 * i + e] = u[e], si[4 * i + e] = w[e];
  }
  if (!interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x.a[e], b = x.b[e];
      x.a[e] = a * co[e] - b * si[e];
      x.b[e] = b * co[e] + a * si[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = x.a[2 * e], b = x.a[2 * e + 1];
      x.a[2 * e] = a * co[e] - b * si[e];
      x.a[2 * e + 1] = b * co[e] + a * si[e];
      a = x.b[2 * e], b = x.b[2 * e + 1];
      x.b[2 * e] = a * co[4 + e] - b * si[4 + e];
      x.b[2 * e + 1] = b * co[4 + e] + a * si[4 + e];
    }
  }
}

template <bool BF16>
__device__ inline Chunk load_chunk(const AppendArgs& p, const uint16_t* row, int c, int64_t pos, bool rotate) {
  Chunk x;
  const Place at = place_of(c, rotate ? p.rot_dim : 0, p.interleaved);
  load8<BF16>(x.a, row + at.a);
  load8<BF16>(x.b, row + at.b);
  if (at.turns) {
    const int64_t r = pos < p.rope_rows ? pos : p.rope_rows - 1;
    turn(x, p.rope + r * p.rot_dim, p.rot_dim / 2, c, p.interleaved);
  }
  return x;
}

// |x| as bits: their order is that of the values, infinities and NaN above.
__device__ inline uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

template <int CODE>
__device__ inline u32x2 pack8(const float (&x)[8], float s) {
  u32x2 w = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t c = s > 0.f || s != s ? to_code<CODE>(x[e] / s) : 0u;
    w[e / 4] |= c << (8 * (e % 4));
  }
  return w;
}

// One (page, head) of K or V.  Block: any multiple of 64 up to 256 threads,
// D / 16 threads to a row.
template <int CODE, bool BF16, int D>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs p, int pages_each) {
  constexpr int TPR = D / 16;
  const int ps = p.cache.page_size, H = p.cache.kv_heads;
  int id = blockIdx.x;
  const bool is_k = id & 1;
  id >>= 1;
  const int h = id % H;
  id /= H;
  const int j = id % pages_each, b = id / pages_each;
  const Span sp = span_of(p.batch, b);
  const int64_t cap = (int64_t)p.batch.table_cols * ps;
  const int64_t past = min(max((int64_t)p.batch.lens[b], (int64_t)0), cap);
  const int64_t col = past / ps + j;
  const int64_t start = col * ps;
  const int64_t lo = max(start, past), hi = min(start + ps, past + sp.n);
  if (lo >= hi) return;
  const int page = page_of(p.cache, p.batch, b, (int)min(col, (int64_t)p.batch.table_cols));
  if (page < 0) return;
  const int fill = (int)(lo - start);  // tokens that the page holds already

  const mi_decode_rows_t& src = is_k ? p.k : p.v;
  const uint16_t* base = static_cast<const uint16_t*>(src.data) + h * src.head_stride;
  uint8_t* codes = static_cast<uint8_t*>(is_k ? p.cache.k : p.cache.v) + ((int64_t)page * H + h) * ps * D;
  float* scale = (is_k ? p.cache.k_scale : p.cache.v_scale) + (int64_t)page * H + h;

  const int tid = threadIdx.x, c = tid % TPR, r0 = tid / TPR, rows = blockDim.x / TPR;
  const int n = (int)(hi - lo);
  const int64_t t0 = sp.first + (lo - past);
  uint32_t m = 0;
  for (int r = r0; r < n; r += rows) {
    const Chunk x = load_chunk<BF16>(p, base + (t0 + r) * src.token_stride, c, lo + r, is_k);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, max(abs_bits(x.a[e]), abs_bits(x.b[e])));
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  __shared__ uint32_t part[4];
  const float old = fill ? *scale : 0.f;
  if (tid % 64 == 0) part[tid / 64] = m;
  __syncthreads();
  for (int w = 0; w < (int)blockDim.x / 64; ++w) m = max(m, part[w]);
  const float mine = __builtin_bit_cast(float, m) / kQmax<CODE>;
  const float s = abs_bits(mine) > abs_bits(old) ? mine : old;
  if (tid == 0) *scale = s;

  for (int r = r0; r < n; r += rows) {
    const Chunk x = load_chunk<BF16>(p, base + (t0 + r) * src.token_stride, c, lo + r, is_k);
    const Place at = place_of(c, is_k ? p.rot_dim : 0, p.interleaved);
    uint8_t* to = codes + (fill + r) * D;
    *reinterpret_cast<u32x2*>(to + at.a) = pack8<CODE>(x.a, s);
    *reinterpret_cast<u32x2*>(to + at.b) = pack8<CODE>(x.b, s);
  }
  if (fill && abs_bits(s) > abs_bits(old)) {
    const float ratio = old / s;
    for (int i = tid; i < fill * (D / 8); i += blockDim.x) {
      u32x2* at = reinterpret_cast<u32x2*>(codes + i * 8);
      const u32x2 w = *at;
      u32x2 out = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        out[e / 4] |= (uint32_t)to_code<CODE>(from_code<CODE>((uint8_t)(w[e / 4] >> (8 * (e % 4)))) * ratio)
                      << (8 * (e % 4));
      *at = out;
    }
  }
}

// Queries turned by their positions.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void turn_kernel(AppendArgs p) {
  constexpr int TPR = D / 16;
  const int b = blockIdx.y;
  const Span sp = span_of(p.batch, b);
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int c = (int)(item % TPR), h = (int)(item / TPR % p.q_heads);
  const int64_t i = item / TPR / p.q_heads;
  if (i >= sp.n) return;
  const int64_t cap = (int64_t)p.batch.table_cols * p.cache.page_size;
  const int64_t pos = min(max((int64_t)p.batch.lens[b], (int64_t)0), cap) + i;
  const uint16_t* row = static_cast<const uint16_t*>(p.q.data) + (sp.first + i) * p.q.token_stride + h * p.q.head_stride;
  uint16_t* to = static_cast<uint16_t*>(p.q_out.data) + (sp.first + i) * p.q_out.token_stride + h * p.q_out.head_stride;
  const Chunk x = load_chunk<BF16>(p, row, c, pos, true);
  const Place at = place_of(c, p.rot_dim, p.interleaved);
  store8<BF16>(to + at.a, x.a);
  store8<BF16>(to + at.b, x.b);
}

// Values of cached tokens, 8 to a thread.
template <int CODE, bool BF16>
__global__ __launch_bounds__(256) void read_kernel(ReadArgs p) {
  const int b = blockIdx.y, H = p.cache.kv_heads, D = p.cache.head_dim, ps = p.cache.page_size;
  const Span sp = span_of(p.batch, b);
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = H * D / 8;
  const int64_t i = item / per;
  if (i >= sp.n) return;
  const int at = (int)(item % per) * 8, h = at / D, d = at % D;
  const int64_t pos = (int64_t)p.batch.lens[b] + i;
  const int page = pos < 0 ? -1 : page_of(p.cache, p.batch, b, (int)min(pos / ps, (int64_t)INT32_MAX));
  float x[8] = {}, y[8] = {};
  if (page >= 0) {
    const int64_t ph = (int64_t)page * H + h;
    const int64_t off = (ph * ps + pos % ps) * D + d;
    const u32x2 k = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(p.cache.k) + off);
    const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(p.cache.v) + off);
    const float sk = p.cache.k_scale[ph], sv = p.cache.v_scale[ph];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = from_code<CODE>((uint8_t)(k[e / 4] >> (8 * (e % 4)))) * sk;
      y[e] = from_code<CODE>((uint8_t)(v[e / 4] >> (8 * (e % 4)))) * sv;
    }
  }
  const int64_t to = (sp.first + i) * H * D + at;
  store8<BF16>(static_cast<uint16_t*>(p.k_out) + to, x);
  store8<BF16>(static_cast<uint16_t*>(p.v_out) + to, y);
}

template <int CODE, bool BF16, int D>
hipError_t append(const AppendArgs& a, hipStream_t s) {
  const int ps = a.cache.page_size;
  const int pages_each = (a.batch.max_tokens + ps - 2) / ps + 1;
  const int64_t blocks = 2 * (int64_t)a.cache.kv_heads * pages_each * a.batch.batch;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  const int threads = a.batch.max_tokens <= 1024 / D ? 64 : 256;
  append_kernel<CODE, BF16, D><<<dim3((unsigned)blocks), threads, 0, s>>>(a, pages_each);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.q_heads == 0) return e;
  const int64_t items = (int64_t)a.batch.max_tokens * a.q_heads * (D / 16);
  const int64_t x = (items + 255) / 256;
  if (x > INT32_MAX) return hipErrorInvalidConfiguration;
  turn_kernel<BF16, D><<<dim3((unsigned)x, a.batch.batch), 256, 0, s>>>(a);
  return hipGetLastError();
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
  const int64_t items = (int64_t)a.batch.max_tokens * a.cache.kv_heads * (a.cache.head_dim / 8);
  const int64_t x = (items + 255) / 256;
  if (x > INT32_MAX) return hipErrorInvalidConfiguration;
  read_kernel<CODE, BF16><<<dim3((unsigned)x, a.batch.batch), 256, 0, s>>>(a);
  return hipGetLastError();
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
