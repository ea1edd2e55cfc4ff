// Linear layer with 4-bit weights for few tokens:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] (c[n][k] - z[n][g]) + bias[n].
//
// A workgroup owns 16 NT rows of weights and its waves split K: wave w of W
// takes the 128-column blocks w, w + W, w + 2 W, ..., each one contiguous KiB
// (a 16-byte load per lane) per 16 rows, which is the operand of four 16x16x32
// matrix instructions.  U blocks are in flight per wave, and the waves' sums
// are added in wave order through LDS at the end: one pass over the weights,
// one launch, the same bits every time.  W is as large as lets every workgroup
// run at once (7 x 5003 x 4072: 8.1 us; with 12 waves and two rounds 11.4).
//
// Bounds, measured with weights that change from call to call: up to 8 tokens
// latency and then the weights' bytes (1 x 4096 x 4096 4.7 us, of which an
// empty launch takes 3.4; 1 x 32768 x 4096 17.3 us, 4.0 TB/s); from 32 tokens
// each wave's chain of unpacking, products and group sums, about 290 vector
// instructions beside 40 matrix ones for 128 columns, at two or three waves a
// SIMD (64 x 14336 x 4096 18.2 us: vector instructions in 55 % of the busy
// cycles, matrix pipes 28 %; two waves unpack the same codes there).
//
// Codes become matrix operands without arithmetic: code c placed under the
// exponent of 16 is the number 16 + c (fp16: bits 6..9 of 0x4c00, bf16: bits
// 3..6 of 0x4180), so a shift and an and-or make two operands.  The offset
// leaves the sum again per group:
//   sum x (c - z) = sum x (16 + c) - (16 + z) sum x,
// where sum x is one more matrix product, by ones, shared by the NT tiles.
// Both products are exact in binary32 and the offset at most doubles to
// quadruples the terms' size, so this costs about two of binary32's 24 bits.
// Where x is infinite, or the offset takes a sum past binary32, the difference
// is NaN: results that are not finite are summed again, term by term, by the
// wave that has them, unless x holds a NaN (1 x 4096 x 4096 4.5 us, with a NaN
// 7.2, with an infinity 60; 64 x 14336 x 4096 with one such row 18.9, 21.5, 76).
#include "device.hpp"

namespace mid {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at any element

template <bool BF16>
__device__ inline f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// Eight codes as eight numbers 16 + c, in k order: a shift and an and-or make
// two.  The and-or takes one constant from a scalar register at most, so the
// exponent's bits come in a vector register.
template <bool BF16>
__device__ inline u32x4 unpack(uint32_t w, uint32_t base) {
  if constexpr (BF16) {
    constexpr uint32_t mask = 0x00780078u;
    return u32x4{(w << 3 & mask) | base, (w >> 1 & mask) | base, (w >> 5 & mask) | base, (w >> 9 & mask) | base};
  } else {
    constexpr uint32_t mask = 0x03c003c0u;
    return u32x4{(w << 6 & mask) | base, (w << 2 & mask) | base, (w >> 2 & mask) | base, (w >> 6 & mask) | base};
  }
}

// Orders a wave's accesses to its piece of shared memory: what its lanes stored
// before is what they load after, and the other way round.  The hardware keeps
// a wave's order; this keeps the compiler's, and costs no instruction.
__device__ inline void wave_shared() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// sum_k x[m][k] ((c - z) s), one term after the other, over every step-th word
// of eight columns; the loads of four words are in flight at a time.
template <bool BF16>
__device__ inline float sum_terms(const W4Args& p, int64_t m, int n, int first, int step) {
  constexpr int DEPTH = 4;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + m * p.ldx;
  const uint16_t* scales = static_cast<const uint16_t*>(p.scales) + n;
  const int64_t np = (int64_t)((p.N + 15) >> 4) * 16;
  const uint32_t* tiles = p.qw + (int64_t)(n >> 4) * ((p.K + 127) >> 7) * 256 + 4 * (n & 15);
  const int words = (p.K + 7) >> 3;
  float y = 0.f;
  for (int at = first; at < words; at += DEPTH * step) {
    uint32_t w[DEPTH];
    uint16_t s[DEPTH], v[DEPTH][8];
    int z[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int k0 = 8 * min(at + d * step, words - 1);
      const int64_t group = k0 / p.group * np;
      w[d] = tiles[(int64_t)(k0 >> 7) * 256 + (k0 >> 3 & 3) * 64 + (k0 >> 5 & 3)];
      s[d] = scales[group];
      z[d] = p.zeros ? p.zeros[group + n] : 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[d][e] = x[min(k0 + e, p.K - 1)];
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * (at + d * step) + e < p.K)
          y = __builtin_fmaf(from16<BF16>(v[d][e]),
                             (float)((int)(w[d] >> (4 * (e / 2) + 16 * (e % 2)) & 15) - z[d]) * from16<BF16>(s[d]), y);
  }
  return y;
}

// Whether row m of x holds a NaN, by a whole wave: its results are NaN then.
template <bool BF16>
__device__ inline bool has_nan(const W4Args& p, int64_t m, int lane) {
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + m * p.ldx;
  bool nan = false;
  for (int k0 = lane; k0 < p.K; k0 += 8 * 64) {
    uint16_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x[min(k0 + 64 * e, p.K - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) nan |= (v[e] & 0x7fff) > (BF16 ? 0x7f80 : 0x7c00);
  }
  return __any(nan);
}

// MT x NT tiles of 16 tokens by 16 rows of weights to a wave, U blocks of 128
// columns in flight.  MW waves share a block and take 16 MT tokens each; the
// other way round, waves that differ in K add their sums.  PER: matrix
// instructions (32 columns each) to a group's sum.  R: loads of 4 tokens that
// hold a wave's tokens.
//
// x comes in rows of 256 bytes (16 lanes), and goes through a piece of shared
// memory that belongs to the wave: loaded as the matrix instruction wants it,
// neighbouring lanes are in different rows, and each such load takes as many
// cache lookups as it has lanes (16 x 4096 x 11008:
// 15.6 us, through shared memory 12.7).
template <bool BF16, int MT, int NT, int U, int PER, int R, int MW, int WMAX>
__global__ __launch_bounds__(64 * WMAX) void w4_kernel(W4Args p) {
  constexpr int FL = 4 / PER;  // group sums to a block
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int lane = threadIdx.x & 63, KW = (int)(blockDim.x >> 6) / MW;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave / MW, mw = wave % MW;
  const int r = lane & 15, c = lane >> 4;
  const int NB = (p.N + 15) >> 4, KB = (p.K + 127) >> 7;
  const int64_t np = (int64_t)NB * 16;
  const int nb0 = blockIdx.x * NT, m0 = blockIdx.y * (16 * MT * MW) + mw * (16 * MT);

  const u32x4* wp[NT];  // the tile row's first entry, the same in every lane
#pragma unroll
  for (int t = 0; t < NT; ++t)
    wp[t] = reinterpret_cast<const u32x4*>(p.qw) + (int64_t)min(nb0 + t, NB - 1) * KB * 64;
  // Lane l holds the 16-byte piece l % 16 of tokens l / 16, l / 16 + 4, ...;
  // rows may begin at any element (the hardware takes such loads as they are).
  // Tokens past M read the last one's row and are not stored; a piece that
  // crosses K is read 8 columns before K and shifted, one past K is zero.
  // Distances are counted in 32 bits, so only to the last of the wave's own
  // rows (31 rows of 2^25 elements at most), however many rows follow.
  const int xrow = lane >> 4, xcol = lane & 15;
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(p.x) + m0 * p.ldx);
  const uint32_t last = (uint32_t)(min(max(p.M - 1 - m0, 0), 16 * MT - 1) * p.ldx * 2), x0 = (uint32_t)(xrow * p.ldx * 2), x4 = (uint32_t)(p.ldx * 8);
  if (m0 >= p.M) xb = static_cast<const uint8_t*>(p.x);
  // the wave's [16 MT][16] pieces; piece q of row i lies at q ^ (i % 16), so
  // that eight rows' pieces of one column do not meet in a bank
  u32x4* xs = reinterpret_cast<u32x4*>(red) + wave * (MT * 256);
#pragma unroll
  for (int i = R; i < 4 * MT; ++i) xs[(4 * i + xrow) * 16 + xcol] = u32x4{0, 0, 0, 0};

  // without zeros their loads go to the scales and are not used: a branch
  // around them would make every later wait a wait for all loads
  const uint8_t* zp = p.zeros ? p.zeros : static_cast<const uint8_t*>(p.scales);
  const bool has_z = p.zeros != nullptr;

  u32x4 wq[U][NT], xq[U][R];
  uint16_t sq[U][FL][NT];
  uint8_t zq[U][FL][NT];

  auto load = [&](int u, int kb) {
    const int at = min(kb, KB - 1);
#pragma unroll
    for (int t = 0; t < NT; ++t) wq[u][t] = wp[t][(int64_t)at * 64 + lane];
#pragma unroll
    for (int f = 0; f < FL; ++f) {
      // the 32-column unit over the group's units: a product by the
      // reciprocal is the quotient or one below it
      const uint32_t unit = min(at * 4 + f * PER, (p.K - 1) >> 5);
      uint32_t g = __umulhi(unit, p.group_inv);
      if ((g + 1) * (uint32_t)(p.group >> 5) <= unit) ++g;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int64_t row = g * np + min(nb0 + t, NB - 1) * 16;
        sq[u][f][t] = (static_cast<const uint16_t*>(p.scales) + row)[r];
        zq[u][f][t] = (zp + row)[r];
      }
    }
    const uint32_t piece = (uint32_t)min(at * 128 + xcol * 8, p.K - 8) * 2;
#pragma unroll
    for (int i = 0; i < R; ++i) xq[u][i] = *reinterpret_cast<const loose*>(xb + (min(x0 + i * x4, last) + piece));
  };
  // what the piece of block kb that lies past K brought, taken out
  auto trim = [&](u32x4 w, int kb) {
    const int by = min(max(kb * 128 + xcol * 8 + 8 - p.K, 0), 8);  // columns past K
    uint64_t lo = w[0] | (uint64_t)w[1] << 32, hi = w[2] | (uint64_t)w[3] << 32;
    if (by & 4) lo = hi, hi = 0;
    const int bits = 16 * (by & 3);
    lo = bits ? lo >> bits | hi << (64 - bits) : lo;
    hi >>= bits;
    if (by == 8) lo = hi = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  };

  f32x4 total[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) total[m][t] = f32x4{0, 0, 0, 0};
  uint32_t expo = BF16 ? 0x41804180u : 0x4c004c00u;
  asm("" : "+v"(expo));
  const u32x4 ones = BF16 ? u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}
                          : u32x4{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};

#pragma unroll
  for (int u = 0; u < U; ++u) load(u, kw + u * KW);
  for (int base = kw; base < KB; base += U * KW) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * KW >= KB) break;
      const int kb = base + u * KW;
      if (kb * 128 + 128 > p.K) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          xq[u][i] = trim(xq[u][i], kb);
          __builtin_amdgcn_sched_barrier(0);  // one at a time: together they need 8 R more registers
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) xs[(4 * i + xrow) * 16 + (xcol ^ ((4 * i + xrow) & 15))] = xq[u][i];
      wave_shared();
      u32x4 xf[4][MT];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) xf[j][m] = xs[(16 * m + r) * 16 + ((4 * j + c) ^ r)];
      wave_shared();
      u32x4 w[NT];
      float sc[FL][NT], of[FL][NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        w[t] = wq[u][t];
#pragma unroll
        for (int f = 0; f < FL; ++f) {
          sc[f][t] = from16<BF16>(sq[u][f][t]);
          of[f][t] = has_z ? -16.f - (float)zq[u][f][t] : -24.f;
        }
      }
      load(u, base + (u + U) * KW);
#pragma unroll
      for (int f = 0; f < FL; ++f) {
        f32x4 rs[MT];
        const f32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m) rs[m] = mma<BF16>(xf[f * PER + i][m], ones, i ? rs[m] : zero);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          f32x4 ps[MT];
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const u32x4 b = unpack<BF16>(w[t][f * PER + i], expo);
#pragma unroll
            for (int m = 0; m < MT; ++m) ps[m] = mma<BF16>(xf[f * PER + i][m], b, i ? ps[m] : zero);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) total[m][t][e] = __builtin_fmaf(sc[f][t], __builtin_fmaf(of[f][t], rs[m][e], ps[m][e]), total[m][t][e]);
        }
      }
    }
  }

  // red[kw][mw][m][t][lane] as 4 tokens each; summed in the order of kw
  constexpr int PART = MT * NT * 64;
  f32x4* part = reinterpret_cast<f32x4*>(red);
  __syncthreads();  // every wave is done with its piece
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) part[wave * PART + (m * NT + t) * 64 + lane] = total[m][t];
  __syncthreads();
  // thread -> (mw, m, t, l): lanes of 16 neighbours hold 16 neighbouring columns of four tokens
  for (int i = threadIdx.x; i < MW * PART; i += blockDim.x) {
    f32x4 y = part[i];
    for (int w = 1; w < KW; ++w) y += part[w * MW * PART + i];
    const int l = i & 63, t = (i >> 6) % NT, m = (i >> 6) / NT;  // m counts over the MW waves' tiles
    const int n = (nb0 + t) * 16 + (l & 15), row0 = blockIdx.y * (16 * MT * MW) + m * 16;
    float odd = 0.f;  // NaN if one of the four is not finite; scales past N may be anything
#pragma unroll
    for (int e = 0; e < 4; ++e) odd = __builtin_fmaf(y[e], 0.f, odd);
    if (__any(n < p.N && odd != 0.f)) {
      // the wave takes one token after the other: 16 columns, a quarter of K to a lane
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool bad = n < p.N && !(fabsf(y[e]) < INFINITY);
        const uint64_t where = __ballot(bad);
        for (int q = 0; q < 4; ++q) {
          const int row = row0 + 4 * q + e;
          if ((where >> (16 * q) & 0xffff) == 0 || row >= p.M || has_nan<BF16>(p, row, l)) continue;
          float sum = n < p.N ? sum_terms<BF16>(p, row, n, l >> 4, 4) : 0.f;
          sum += __shfl_xor(sum, 16);
          sum += __shfl_xor(sum, 32);
          if (bad && (l >> 4) == q) y[e] = sum;
        }
      }
    }
    if (n >= p.N) continue;
    const float b = p.bias ? from16<BF16>(static_cast<const uint16_t*>(p.bias)[n]) : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = row0 + (l >> 4) * 4 + e;
      if (row < p.M) static_cast<uint16_t*>(p.y)[row * p.ldy + n] = to16<BF16>(y[e] + b);
    }
  }
}

// K below 8, where no whole piece of a row exists: one result to a thread.
template <bool BF16>
__global__ __launch_bounds__(256) void w4_short_kernel(W4Args p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * p.N) return;
  const int n = (int)(i % p.N);
  const int64_t m = i / p.N;
  float y = sum_terms<BF16>(p, m, n, 0, 1);
  if (p.bias) y += from16<BF16>(static_cast<const uint16_t*>(p.bias)[n]);
  static_cast<uint16_t*>(p.y)[m * p.ldy + n] = to16<BF16>(y);
}

// WMAX: the waves of one workgroup, and of all workgroups on a compute unit,
// that the instance's registers allow.  K is split over as many waves as let
// all workgroups run at once.
template <bool BF16, int MT, int NT, int U, int PER, int R, int MW, int WMAX>
hipError_t run(const W4Args& a, hipStream_t s) {
  static_assert(NT <= 4 && WMAX * MT * 4096 <= 160 << 10, "the sums lie where x was");
  const int NB = (a.N + 15) / 16, KB = (a.K + 127) / 128;
  const dim3 grid((NB + NT - 1) / NT, (a.M + 16 * MT * MW - 1) / (16 * MT * MW));
  if (grid.y > 65535) return hipErrorInvalidConfiguration;
  const int64_t each = ((int64_t)grid.x * grid.y + a.cus - 1) / a.cus;
  int kw = each < WMAX / MW ? WMAX / MW / (int)each : 1;
  if (kw < 4 / MW) kw = 4 / MW;
  if (kw > KB) kw = KB;
  return launch(w4_kernel<BF16, MT, NT, U, PER, R, MW, WMAX>, grid, 64 * kw * MW, kw * MW * MT * 4096, s, a);
}

// One or two tiles of weight rows to a workgroup, by their number (us with one
// and two, 4096 columns, groups of 128): 1 token, 512 tiles 6.2 and 6.8, 1024
// tiles 9.4 and 9.8, 2048 tiles 18.6 and 17.0; 8 tokens, 1024 tiles 9.9 and
// 10.0, 1376 tiles 15.7 and 15.1, 2048 tiles 22.5 and 18.3; 16 tokens, 512
// tiles 7.7 and 7.2, 896 tiles 11.4 and 11.9, 1376 tiles 20.2 and 15.5.
template <bool BF16, int PER, int R>
hipError_t few(const W4Args& a, hipStream_t s) {
  const int NB = (a.N + 15) / 16;
  if (NB < 1024) return run<BF16, 1, 1, 2, PER, R, 1, 16>(a, s);
  return run<BF16, 1, 2, 2, PER, R, 1, R == 4 || PER == 1 ? 12 : 16>(a, s);
}

// From 17 tokens on the border is 512 tiles (us below and above it, groups of
// 128): 32 tokens, 256 tiles 7.4 and 7.1, 512 tiles 11.0 and 8.1, 896 tiles 17.4
// and 12.8; 64 tokens, 256 tiles 10.4 and 16.0, 512 tiles 16.5 and 16.5, 896
// tiles 28.9 and 17.5; groups of 32 and 64 tokens, 256 tiles 11.8 and 15.7, 512
// tiles 18.5 and 16.2.
template <bool BF16, int PER>
hipError_t sized(const W4Args& a, hipStream_t s) {
  const int NB = (a.N + 15) / 16;
  if (a.M <= 4) return few<BF16, PER, 1>(a, s);
  if (a.M <= 8) return few<BF16, PER, 2>(a, s);
  if (a.M <= 16) return few<BF16, PER, 4>(a, s);
  if (a.M <= 32) {
    if (NB < 512) return run<BF16, 2, 1, 1, PER, 8, 1, 16>(a, s);
    return run<BF16, 2, 2, 1, PER, 8, 1, PER == 1 ? 8 : 12>(a, s);
  }
  if (NB < 512) return run<BF16, 2, 1, 1, PER, 8, 2, 16>(a, s);
  if constexpr (PER == 4) return run<BF16, 2, 4, 1, PER, 8, 2, 8>(a, s);
  else return run<BF16, 2, 2, 1, PER, 8, 2, PER == 1 ? 8 : 12>(a, s);
}

template <bool BF16>
hipError_t pick(const W4Args& a, hipStream_t s) {
  if (a.K < 8) {
    const int64_t blocks = ((int64_t)a.M * a.N + 255) / 256;
    if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
    return launch(w4_short_kernel<BF16>, dim3((unsigned)blocks), 256, 0, s, a);
  }
  if (a.group % 128 == 0) return sized<BF16, 4>(a, s);
  if (a.group % 64 == 0 && 128 % a.group == 0) return sized<BF16, 2>(a, s);
  return sized<BF16, 1>(a, s);
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t s) { return a.bf16 ? pick<true>(a, s) : pick<false>(a, s); }

}  // namespace mid
