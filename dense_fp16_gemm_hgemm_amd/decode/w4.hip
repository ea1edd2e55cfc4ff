// Linear layer with 4-bit weights for few tokens:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] (c[n][k] - z[n][g]) + bias[n].
//
// A workgroup owns 16 NT rows of weights and all its waves split K: wave w
// takes the 128-column blocks w, w + W, w + 2 W, ..., each one contiguous KiB
// (a 16-byte load per lane) per 16 rows, which is the operand of four 16x16x32
// matrix instructions.  U blocks are in flight per wave, and the waves' sums
// are added in wave order through LDS at the end: one pass over the weights,
// one launch, the same bits every time.
//
// Codes become matrix operands without arithmetic: code c placed under the
// exponent of 16 is the number 16 + c (fp16: bits 6..9 of 0x4c00, bf16: bits
// 3..6 of 0x4180), so a shift and an and-or make two operands.  The offset
// leaves the sum again per group:
//   sum x (c - z) = sum x (16 + c) - (16 + z) sum x,
// where sum x is one more matrix product, by ones, shared by the NT tiles.
// Both products are exact in binary32 and the offset at most doubles to
// quadruples the terms' size, so this costs about two of binary32's 24 bits.
#include "device.hpp"

namespace mid {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int kRsrcWord3 = 0x00020000;
constexpr uint32_t kOOB = 0x80000000u;

template <bool BF16>
__device__ inline f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// Eight codes as eight numbers 16 + c, in k order.
template <bool BF16>
__device__ inline u32x4 unpack(uint32_t w) {
  if constexpr (BF16) {
    constexpr uint32_t mask = 0x00780078u, base = 0x41804180u;
    return u32x4{(w << 3 & mask) | base, (w >> 1 & mask) | base, (w >> 5 & mask) | base, (w >> 9 & mask) | base};
  } else {
    constexpr uint32_t mask = 0x03c003c0u, base = 0x4c004c00u;
    return u32x4{(w << 6 & mask) | base, (w << 2 & mask) | base, (w >> 2 & mask) | base, (w >> 6 & mask) | base};
  }
}

// MT x NT tiles of 16 tokens by 16 rows of weights to a wave, U blocks of 128
// columns in flight.  PER: matrix instructions (32 columns each) to a group's
// sum.  WIDE: x's rows are 16-byte aligned and of whole 16-byte pieces.
template <bool BF16, int MT, int NT, int U, int PER, bool WIDE>
__global__ __launch_bounds__(512) void w4_kernel(W4Args p) {
  constexpr int FL = 4 / PER;  // group sums to a block
  extern __shared__ float red[];
  const int lane = threadIdx.x & 63, W = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int NB = (p.N + 15) >> 4, KB = (p.K + 127) >> 7;
  const int64_t np = (int64_t)NB * 16;
  const int nb0 = blockIdx.x * NT, m0 = blockIdx.y * (16 * MT);

  const u32x4* wp[NT];
  int64_t sn[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int nb = min(nb0 + t, NB - 1);
    wp[t] = reinterpret_cast<const u32x4*>(p.qw) + (int64_t)nb * KB * 64 + lane;
    sn[t] = nb * 16 + r;
  }
  const uint16_t* xb = static_cast<const uint16_t*>(p.x) + m0 * p.ldx;
  uint32_t xo[MT];  // byte offset of the lane's row, or out of range
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xo[m] = m0 + m * 16 + r < p.M ? (uint32_t)((m * 16 + r) * p.ldx * 2) : kOOB;
  const auto xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(xb), (short)0, (int)0x7fffffff, kRsrcWord3);

  u32x4 wq[U][NT], xq[U][4][MT];
  uint16_t sq[U][FL][NT];
  uint8_t zq[U][FL][NT];

  auto load = [&](int u, int kb) {
    const int at = min(kb, KB - 1);
#pragma unroll
    for (int t = 0; t < NT; ++t) wq[u][t] = wp[t][(int64_t)at * 64];
#pragma unroll
    for (int f = 0; f < FL; ++f) {
      const int g = min(at * 128 + f * (32 * PER), p.K - 1) / p.group;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sq[u][f][t] = static_cast<const uint16_t*>(p.scales)[g * np + sn[t]];
        zq[u][f][t] = p.zeros ? p.zeros[g * np + sn[t]] : 8;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = kb * 128 + j * 32 + c * 8;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if constexpr (WIDE) {
          const uint32_t off = k < p.K ? xo[m] + (uint32_t)k * 2 : kOOB;
          xq[u][j][m] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, off | (xo[m] & kOOB), 0, 0));
        } else {
          const uint16_t* row = xb + (int64_t)(m * 16 + r) * p.ldx;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool row_in = m0 + m * 16 + r < p.M;
            const uint32_t lo = row_in && k + 2 * i < p.K ? row[k + 2 * i] : 0;
            const uint32_t hi = row_in && k + 2 * i + 1 < p.K ? row[k + 2 * i + 1] : 0;
            xq[u][j][m][i] = lo | hi << 16;
          }
        }
      }
    }
  };

  f32x4 total[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) total[m][t] = f32x4{0, 0, 0, 0};
  const u32x4 ones = BF16 ? u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}
                          : u32x4{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};

#pragma unroll
  for (int u = 0; u < U; ++u) load(u, wave + u * W);
  for (int base = wave; base < KB; base += U * W) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * W >= KB) break;
#pragma unroll
      for (int f = 0; f < FL; ++f) {
        f32x4 rs[MT], ps[MT][NT];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int j = f * PER + i;
          const f32x4 zero = {0, 0, 0, 0};
#pragma unroll
          for (int m = 0; m < MT; ++m) rs[m] = mma<BF16>(xq[u][j][m], ones, i ? rs[m] : zero);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const u32x4 b = unpack<BF16>(wq[u][t][j]);
#pragma unroll
            for (int m = 0; m < MT; ++m) ps[m][t] = mma<BF16>(xq[u][j][m], b, i ? ps[m][t] : zero);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float s = from16<BF16>(sq[u][f][t]), z = -16.f - (float)zq[u][f][t];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) total[m][t][e] += s * __builtin_fmaf(z, rs[m][e], ps[m][t][e]);
        }
      }
      load(u, base + (u + U) * W);
    }
  }

  // red[wave][m][t][lane] as 4 tokens each; summed in wave order
  constexpr int PART = MT * NT * 64;
  f32x4* part = reinterpret_cast<f32x4*>(red);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) part[wave * PART + (m * NT + t) * 64 + lane] = total[m][t];
  __syncthreads();
  // thread -> (m, t, l): lanes of 16 neighbours hold 16 neighbouring columns of four tokens
  for (int i = threadIdx.x; i < PART; i += blockDim.x) {
    f32x4 y = part[i];
    for (int w = 1; w < W; ++w) y += part[w * PART + i];
    const int l = i & 63, t = (i >> 6) % NT, m = (i >> 6) / NT;
    const int n = (nb0 + t) * 16 + (l & 15);
    if (n >= p.N) continue;
    const float b = p.bias ? from16<BF16>(static_cast<const uint16_t*>(p.bias)[n]) : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = m0 + m * 16 + (l >> 4) * 4 + e;
      if (row < p.M) static_cast<uint16_t*>(p.y)[row * p.ldy + n] = to16<BF16>(y[e] + b);
    }
  }
}

// K = 0: the bias, or zeros.
template <bool BF16>
__global__ __launch_bounds__(256) void w4_bias_kernel(W4Args p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * p.N) return;
  const int n = (int)(i % p.N);
  static_cast<uint16_t*>(p.y)[i / p.N * p.ldy + n] = p.bias ? static_cast<const uint16_t*>(p.bias)[n] : (uint16_t)0;
}

template <bool BF16, int MT, int NT, int U, int PER, bool WIDE>
hipError_t run(const W4Args& a, hipStream_t s) {
  const int NB = (a.N + 15) / 16, KB = (a.K + 127) / 128;
  const int W = KB < 8 ? KB : 8;
  const dim3 grid((NB + NT - 1) / NT, (a.M + 16 * MT - 1) / (16 * MT));
  if (grid.y > 65535) return hipErrorInvalidConfiguration;
  w4_kernel<BF16, MT, NT, U, PER, WIDE><<<grid, 64 * W, W * MT * NT * 1024, s>>>(a);
  return hipGetLastError();
}

template <bool BF16, int PER>
hipError_t wide(const W4Args& a, hipStream_t s) {
  if (a.M <= 8) return run<BF16, 1, 1, 4, PER, true>(a, s);
  if (a.M <= 16) return run<BF16, 1, 2, 4, PER, true>(a, s);
  if (a.M <= 32) return run<BF16, 2, 2, 2, PER, true>(a, s);
  return run<BF16, 4, 4, 1, PER, true>(a, s);
}

template <bool BF16>
hipError_t pick(const W4Args& a, hipStream_t s) {
  if (a.K == 0) {
    const int64_t blocks = ((int64_t)a.M * a.N + 255) / 256;
    if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
    w4_bias_kernel<BF16><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
    return hipGetLastError();
  }
  // 16-byte rows, and tile rows that a 31-bit byte offset reaches
  if ((reinterpret_cast<uintptr_t>(a.x) & 15) || a.ldx % 8 || a.K % 8 || a.ldx > (1 << 23) || a.K > (1 << 23))
    return run<BF16, 1, 1, 1, 1, false>(a, s);
  if (a.group % 128 == 0) return wide<BF16, 4>(a, s);
  if (a.group % 64 == 0 && 128 % a.group == 0) return wide<BF16, 2>(a, s);
  return wide<BF16, 1>(a, s);
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t s) { return a.bf16 ? pick<true>(a, s) : pick<false>(a, s); }

}  // namespace mid
