// Norm with the residual's addition, into 8-bit floats with a scale for 128 columns:
//   t = round(x + r),  y = t / sqrt(mean t^2 + eps) * g,  s_j = max |y| / 448,  code = rne(y / s_j).
//
// One pass: a thread keeps its columns of t in registers, the row's sum of squares
// is one exchange over its threads, and a block's maximum one over sixteen lanes
// (sixteen threads hold 128 columns).  y is not rounded before it is divided by the
// scale.  Above 16384 columns t is read again, from the caches for the most part.
//
// Bound: for many rows the bytes, x, r, t and codes (8192 x 4096 bf16, 235 MB: 48.4 us
// in a trace, 4.9 TB/s, and 52 as nodes of a graph; the same read again instead of
// kept 58, a wave to a row 67), and beside them vector instructions, the division of
// each y by its scale among them, which issue in all of its cycles.  For few rows
// launch, one round of loads, the exchanges and the division (1 x 4096 3.7 us, an empty
// kernel 3.3).  Rows that do not begin at multiples of 16 bytes, or do not end at one
// of 8 columns, take eight loads of 2 bytes and eight byte stores a thread, whose
// number is the bound then: 1, 512 and 8192 x 4095 6.6, 12.2 and 149 us where 4096
// columns take 3.7, 6.6 and 52.
#include "device.hpp"

namespace mid {
namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ inline uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// What a row's values are multiplied by: 2^-shift, then `by`.
struct Root {
  int shift;
  double by;
};

// The largest of |x| or a sum over the T threads of a row.
template <int T, typename V, typename F>
__device__ inline V over_row(V x, V* room, F f) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = f(x, __shfl_xor(x, d));
  if constexpr (T > 64) {
    __syncthreads();  // the last one's values have been read
    if (threadIdx.x % 64 == 0) room[threadIdx.x / 64] = x;
    __syncthreads();
    x = room[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) x = f(x, room[w]);
  }
  return x;
}

// Eight values from column k on, 0 past K; WIDE: all eight are there and aligned.
template <bool BF16, bool WIDE>
__device__ inline f32x8 load8(const void* base, int k, int K) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + k;
  f32x8 x;
  if constexpr (WIDE) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = from16<BF16>((uint16_t)(w[e / 2] >> (16 * (e % 2))));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = k + e < K ? from16<BF16>(p[e]) : 0.f;
  }
  return x;
}

// T threads to a row; thread t has eight columns from 8 t + 8 T i on, i < C (C 0:
// any number of them, which are read again instead of kept).
template <bool BF16, bool WIDE, int T, int C>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_kernel(NormArgs p) {
  constexpr int ROWS = T < 256 ? 256 / T : 1;
  __shared__ float sums[T / 64];
  __shared__ uint32_t tops[T / 64];
  const int tid = threadIdx.x % T, K = p.K;
  const int64_t m = (int64_t)blockIdx.x * ROWS + threadIdx.x / T;
  if (T == 64 && m >= p.M) return;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + m * p.ldx;
  const uint16_t* r = p.residual ? static_cast<const uint16_t*>(p.residual) + m * p.ldr : nullptr;
  uint16_t* total = p.total ? static_cast<uint16_t*>(p.total) + m * p.ldt : nullptr;
  const int steps = C ? C : (K + 8 * T - 1) / (8 * T);

  auto fetch = [&](int k) {
    f32x8 t = load8<BF16, WIDE>(x, k, K);
    if (r) {
      t += load8<BF16, WIDE>(r, k, K);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = from16<BF16>(to16<BF16>(t[e]));
    }
    return t;
  };
  f32x8 kept[C ? C : 1];
  float sum = 0.f;
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int k = 8 * (tid + T * i);
      kept[i] = f32x8{};
      if (k < K) kept[i] = fetch(k);
    }
  }
#pragma unroll(C ? C : 1)
  for (int i = 0; i < steps; ++i) {
    const int k = 8 * (tid + T * i);
    if (k >= K) continue;
    const f32x8 t = C ? kept[C ? i : 0] : fetch(k);
    if (total) {
      if constexpr (WIDE) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = to16<BF16>(t[2 * e]) | (uint32_t)to16<BF16>(t[2 * e + 1]) << 16;
        *reinterpret_cast<u32x4*>(total + k) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k + e < K) total[k + e] = to16<BF16>(t[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(t[e], t[e], sum);
  }
  // a total that took x's or r's place is read from there again
  if (C == 0 && total) x = total, r = nullptr;
  sum = over_row<T>(sum, sums, [](float a, float b) { return a + b; });

  bool rare = false;  // the same in a row's threads
  // Squares of values up to 2^128 (bf16) leave binary32: then once more, with the
  // row's largest magnitude in [1, 2).  Small ones matter where eps is no larger.
  Root root = {0, 0.};
  float by = 1.f / __builtin_sqrtf(sum / (float)K + p.eps);
  if (!(sum < INFINITY) || (sum < 0x1p-80f && p.eps < 0x1p-80f)) {
    uint32_t top = 0;
#pragma unroll(C ? C : 1)
    for (int i = 0; i < steps; ++i) {
      const int k = 8 * (tid + T * i);
      if (k >= K) continue;
      const f32x8 t = C ? kept[C ? i : 0] : fetch(k);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, abs_bits(t[e]));
    }
    top = over_row<T>(top, tops, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    if (top != 0 && top < 0x7f800000u) {
      root.shift = __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, top)) - 1;
      sum = 0.f;
#pragma unroll(C ? C : 1)
      for (int i = 0; i < steps; ++i) {
        const int k = 8 * (tid + T * i);
        if (k >= K) continue;
        const f32x8 t = C ? kept[C ? i : 0] : fetch(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = __builtin_ldexpf(t[e], -root.shift);
          sum = __builtin_fmaf(u, u, sum);
        }
      }
      sum = over_row<T>(sum, sums, [](float a, float b) { return a + b; });
      rare = true;
      root.by = 1. / __builtin_sqrt((double)sum / K + __builtin_ldexp((double)p.eps, -2 * root.shift));
    }
  }

  rare = __builtin_amdgcn_readfirstlane(rare);
#pragma unroll(C ? C : 1)
  for (int i = 0; i < steps; ++i) {
    const int k = 8 * (tid + T * i);
    f32x8 y = {};
    if (k < K) {
      y = C ? kept[C ? i : 0] : fetch(k);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = rare ? (float)(__builtin_ldexpf(y[e], -root.shift) * root.by) : y[e] * by;
      if (p.weight) y *= load8<BF16, WIDE>(p.weight, k, K);
    }
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, k + e < K ? abs_bits(y[e]) : 0u);
#pragma unroll
    for (int d = 8; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (k >= K) continue;
    const float s = __builtin_bit_cast(float, top) / 448.f;
    if (tid % 16 == 0) p.scales[m * p.lds + k / 128] = s;
    uint8_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = to_code<MI_DECODE_E4M3>(s > 0.f || s != s ? y[e] / s : 0.f);
    uint8_t* to = p.codes + m * p.ldc + k;
    if constexpr (WIDE) {
      u32x2 w = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e / 4] |= (uint32_t)c[e] << (8 * (e % 4));
      *reinterpret_cast<u32x2*>(to) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < K) to[e] = c[e];
    }
  }
}

template <bool BF16, bool WIDE, int T, int C>
hipError_t run(const NormArgs& a, hipStream_t s) {
  constexpr int ROWS = T < 256 ? 256 / T : 1;
  return launch(norm_kernel<BF16, WIDE, T, C>, dim3((unsigned)((a.M + ROWS - 1) / ROWS)), T < 256 ? 256 : T, 0, s, a);
}

// Up to 512 rows take many threads with one or two groups of columns each, as
// the time is one thread's chain; more rows take fewer threads, so that several
// rows share a compute unit.  us as nodes of a graph, more threads and fewer: 1, 512
// and 8192 rows of 1024 columns 3.5, 4.1, 21.3 (256 threads) and 4.5, 5.1, 19.7 (64);
// of 4096 3.7, 6.6, 55.6 (512) and 4.7, 7.3, 52.5 (256); 1, 512 and 4096 rows of 8192
// 4.4, 10.3, 56.5 (1024) and 7.4, 11.8, 56.5 (256); 1, 512 and 2048 rows of 16384 6.6,
// 18.5, 53.4 (1024) and 8.1, 19.5, 56.6 (512).
template <bool BF16, bool WIDE>
hipError_t pick(const NormArgs& a, hipStream_t s) {
  const bool few = a.M <= 512;
  if (a.K <= 512) return run<BF16, WIDE, 64, 1>(a, s);
  if (a.K <= 1024) return few ? run<BF16, WIDE, 256, 1>(a, s) : run<BF16, WIDE, 64, 2>(a, s);
  if (a.K <= 2048) return run<BF16, WIDE, 256, 1>(a, s);
  if (a.K <= 4096) return few ? run<BF16, WIDE, 512, 1>(a, s) : run<BF16, WIDE, 256, 2>(a, s);
  if (a.K <= 8192) return few ? run<BF16, WIDE, 1024, 1>(a, s) : run<BF16, WIDE, 256, 4>(a, s);
  if (a.K <= 16384) return few ? run<BF16, WIDE, 1024, 2>(a, s) : run<BF16, WIDE, 512, 4>(a, s);
  return run<BF16, WIDE, 1024, 0>(a, s);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const bool wide = a.K % 8 == 0 && a.ldx % 8 == 0 && a.ldr % 8 == 0 && a.ldt % 8 == 0 && a.ldc % 8 == 0 &&
                    aligned(a.x, 16) && aligned(a.residual, 16) && aligned(a.weight, 16) && aligned(a.total, 16) &&
                    aligned(a.codes, 8);
  if (a.bf16) return wide ? pick<true, true>(a, s) : pick<true, false>(a, s);
  return wide ? pick<false, true>(a, s) : pick<false, false>(a, s);
}

}  // namespace mid
