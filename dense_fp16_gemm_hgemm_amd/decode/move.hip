// Pages that are copied, and drafted tokens that are kept.
#include "device.hpp"

namespace mid {
namespace {

// ------------------------------------------------------------------ copy --

constexpr int kPiece = 16384;  // bytes of a page that a workgroup copies

__global__ __launch_bounds__(256) void copy_kernel(CopyArgs p, int pieces) {
  const int64_t pair = blockIdx.x / (2 * pieces);
  const int rest = blockIdx.x % (2 * pieces), at = rest >> 1, is_v = rest & 1, H = p.cache.kv_heads;
  const int64_t bytes = (int64_t)H * p.cache.page_size * p.cache.head_dim;
  const int src = p.src[pair], dst = p.dst[pair];
  if (src < 0 || dst < 0 || src >= p.cache.pages || dst >= p.cache.pages || src == dst) return;
  uint8_t* base = static_cast<uint8_t*>(is_v ? p.cache.v : p.cache.k);
  const u32x4* from = reinterpret_cast<const u32x4*>(base + src * bytes + (int64_t)at * kPiece);
  u32x4* to = reinterpret_cast<u32x4*>(base + dst * bytes + (int64_t)at * kPiece);
  const int units = (int)min((int64_t)kPiece, bytes - (int64_t)at * kPiece) / 16;
  u32x4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((int)threadIdx.x + 256 * i < units) x[i] = from[threadIdx.x + 256 * i];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((int)threadIdx.x + 256 * i < units) to[threadIdx.x + 256 * i] = x[i];
  if (at == 0) {
    float* scale = is_v ? p.cache.v_scale : p.cache.k_scale;
    for (int h = threadIdx.x; h < H; h += 256) scale[(int64_t)dst * H + h] = scale[(int64_t)src * H + h];
  }
}

// ------------------------------------------------------------------ keep --

// |x| as bits: their order is that of the values, infinities and NaN above.
__device__ inline uint64_t abs_bits(double x) { return __builtin_bit_cast(uint64_t, x) & 0x7fffffffffffffffull; }

// Sixteen codes times ratio, to the nearest codes.  Scales of two pages are often
// in a simple ratio, as the largest code sets the new one, and their products lie
// on the border between two codes then: in binary64 the rounding to binary32
// that follows takes the ratio's error away, and the border goes to even.
template <int CODE>
__device__ inline u32x4 rescaled(u32x4 w, double ratio) {
  u32x4 o = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    o[e / 4] |= (uint32_t)to_code<CODE>((float)(from_code<CODE>((uint8_t)(w[e / 4] >> (8 * (e % 4)))) * ratio)) << (8 * (e % 4));
  return o;
}

// One workgroup moves the kept tokens of a sequence in one head of K or of V,
// page by page in the order of positions: a token comes from its own place or a
// later one, so what a page reads no earlier page has written.
template <int CODE>
__global__ __launch_bounds__(256) void keep_kernel(KeepArgs p) {
  __shared__ uint64_t part[4];
  const int H = p.cache.kv_heads, D = p.cache.head_dim, ps = p.cache.page_size;
  const int b = blockIdx.x / (2 * H), h = blockIdx.x % (2 * H) >> 1, is_v = blockIdx.x & 1;
  const Span sp = span_of(p.batch, b);
  const int n = min(sp.n, p.batch.max_tokens);
  if (n <= 0) return;
  const int64_t cap = (int64_t)p.batch.table_cols * ps;
  const int64_t past = min(max((int64_t)p.batch.lens[b], (int64_t)0), cap);
  uint8_t* codes = static_cast<uint8_t*>(is_v ? p.cache.v : p.cache.k);
  float* scales = is_v ? p.cache.v_scale : p.cache.k_scale;
  const int per = D / 16, rows = 256 / per, r0 = threadIdx.x / per, c = threadIdx.x % per;
  auto row_at = [&](int page, int slot) {
    return reinterpret_cast<u32x4*>(codes + (((int64_t)page * H + h) * ps + slot) * D) + c;
  };

  const int64_t upto = min(past + n, cap);
  for (int64_t start = past - past % ps; start < upto; start += ps) {
    const int page = page_of(p.cache, p.batch, b, (int)(start / ps));
    if (page < 0) continue;
    const int lo = (int)(max(start, past) - past), hi = (int)(min(start + ps, upto) - past);  // tokens that come here
    const float old = scales[(int64_t)page * H + h];
    // where token i comes from: its page, or `page` and its own slot
    struct Source {
      int page, slot;
    };
    auto source = [&](int i) {
      const int k = p.keep[sp.first + i];
      const int64_t pos = past + k;
      const int from = k < i ? -1 : page_of(p.cache, p.batch, b, (int)min(pos / ps, (int64_t)p.batch.table_cols));
      return from < 0 ? Source{page, (int)((past + i) % ps)} : Source{from, (int)(pos % ps)};
    };
    uint64_t m = 0;
    for (int i = lo + r0; i < hi; i += rows) {
      const Source s = source(i);
      if (s.page == page) continue;
      const double by = scales[(int64_t)s.page * H + h];
      const u32x4 w = *row_at(s.page, s.slot);
#pragma unroll
      for (int e = 0; e < 16; ++e) m = max(m, abs_bits(from_code<CODE>((uint8_t)(w[e / 4] >> (8 * (e % 4)))) * by));
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) m = max(m, (uint64_t)__shfl_xor((unsigned long long)m, d));
    __syncthreads();  // the last page's maximum has been read
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = max(m, part[w]);
    const double mine = __builtin_bit_cast(double, m) * (1. / kQmax<CODE>);
    const bool grows = abs_bits(mine) > abs_bits(old);
    const double s1 = grows ? mine : old;

    // tokens in order, `rows` at a time: all of them are read before any is written
    for (int i0 = lo; i0 < hi; i0 += rows) {
      const int i = i0 + r0;
      bool put = false;
      u32x4 w;
      if (i < hi) {
        const Source s = source(i);
        const double by = s.page == page ? old : scales[(int64_t)s.page * H + h];
        put = grows || s.page != page || s.slot != (int)((past + i) % ps);
        if (put) {
          w = *row_at(s.page, s.slot);
          const double ratio = by / s1;
          if (s1 == 0.) w = u32x4{0, 0, 0, 0};
          else if (ratio != 1. && (grows || s.page != page)) w = rescaled<CODE>(w, ratio);
        }
      }
      __syncthreads();
      if (put) *row_at(page, (int)((past + i) % ps)) = w;
    }
    if (grows) {
      const int held = (int)(past + lo - start);
      const double ratio = old / s1;
      for (int r = r0; r < held; r += rows) *row_at(page, r) = rescaled<CODE>(*row_at(page, r), ratio);
      if (threadIdx.x == 0) scales[(int64_t)page * H + h] = (float)s1;
    }
  }
}

}  // namespace

hipError_t launch_copy(const CopyArgs& a, hipStream_t s) {
  const int64_t bytes = (int64_t)a.cache.kv_heads * a.cache.page_size * a.cache.head_dim;
  const int64_t pieces = (bytes + kPiece - 1) / kPiece;
  if (a.pairs > INT32_MAX / (2 * pieces)) return hipErrorInvalidConfiguration;
  return launch(copy_kernel, dim3((unsigned)(a.pairs * 2 * pieces)), 256, 0, s, a, (int)pieces);
}

hipError_t launch_keep(const KeepArgs& a, hipStream_t s) {
  const int64_t blocks = 2 * (int64_t)a.cache.kv_heads * a.batch.batch;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks);
  if (a.cache.code == MI_DECODE_INT8) return launch(keep_kernel<MI_DECODE_INT8>, grid, 256, 0, s, a);
  return launch(keep_kernel<MI_DECODE_E4M3>, grid, 256, 0, s, a);
}

}  // namespace mid
