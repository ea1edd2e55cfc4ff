// Linear layer of 8-bit floats with block scales:
//   y[m][n] = sum_j (xs[m][j] ws[n / 128][j]) sum_{k in block j} x[m][k] w[n][k] + bias[n].
//
// A block of 128 columns is the depth of one 16x16x128 matrix instruction, so a
// block's sum is one instruction from zero, and its scales enter as one
// multiply-add for each of the four results in a lane.  Weights are the left
// operand: a lane holds four neighbouring n of one token, whose scale is one
// number of the lane's, and ws is the same for a wave's whole 16-row tile.
// Which column of a block stands where in the operands does not matter as long
// as it is the same for both.
#include "device.hpp"

namespace mid {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(1)));  // 16 bytes at any address

__device__ inline f32x4 mma(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1) {
  i32x8 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = a0[i], a[4 + i] = a1[i], b[i] = b0[i], b[4 + i] = b1[i];
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

template <bool BF16>
__device__ inline float bias_of(const F8Args& p, int n) {
  return p.bias ? from16<BF16>(static_cast<const uint16_t*>(p.bias)[n]) : 0.f;
}

// Four results of token m from column n on.
template <bool BF16>
__device__ inline void store4(const F8Args& p, int m, int n, f32x4 y, bool whole) {
  uint16_t* to = static_cast<uint16_t*>(p.y) + m * p.ldy + n;
  if (m >= p.M) return;
  if (whole) {  // N and the rows' distance are multiples of 4, and y is aligned
    if (n >= p.N) return;
    u32x2 w = {0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e / 2] |= (uint32_t)to16<BF16>(y[e] + bias_of<BF16>(p, n + e)) << (16 * (e % 2));
    *reinterpret_cast<u32x2*>(to) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) to[e] = to16<BF16>(y[e] + bias_of<BF16>(p, n + e));
  }
}

// -------------------------------------------------------------- few tokens --

// MT x NT tiles of 16 tokens by 16 weight rows to a workgroup, whose waves split
// K: wave w of W takes blocks w, w + W, ...; U of them are in flight.
template <bool BF16, int MT, int NT, int U>
__global__ __launch_bounds__(1024) void f8_few_kernel(F8Args p, int whole) {
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int lane = threadIdx.x & 63, W = (int)(blockDim.x >> 6);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, KB = (p.K + 127) >> 7;
  const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
  const uint8_t* wp[NT];
  const uint8_t* xp[MT];
  const float* sp[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) wp[t] = p.w + (int64_t)min(n0 + 16 * t + r, p.N - 1) * p.ldw;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t row = min(m0 + 16 * t + r, p.M - 1);
    xp[t] = p.x + row * p.ldx;
    sp[t] = p.xs + row * p.ldxs;
  }
  u32x4 wq[U][NT][2], xq[U][MT][2];
  float xs[U][MT], ws[U][NT];
  auto load = [&](int u, int kb) {
    const int at = min(kb, KB - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // a piece that crosses K is read 16 columns before K and shifted
      const int k = min(128 * at + 32 * g + 16 * i, p.K - 16);
#pragma unroll
      for (int t = 0; t < NT; ++t) wq[u][t][i] = *reinterpret_cast<const loose*>(wp[t] + k);
#pragma unroll
      for (int t = 0; t < MT; ++t) xq[u][t][i] = *reinterpret_cast<const loose*>(xp[t] + k);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) ws[u][t] = p.ws[min(n0 + 16 * t, p.N - 1) / 128 * p.ldws + at];
#pragma unroll
    for (int t = 0; t < MT; ++t) xs[u][t] = sp[t][at];
  };
  // without the bytes that lie past K
  auto trim = [&](u32x4 w, int k) {
    const int by = min(max(k + 16 - p.K, 0), 16), bits = 8 * (by & 7);
    uint64_t lo = w[0] | (uint64_t)w[1] << 32, hi = w[2] | (uint64_t)w[3] << 32;
    if (by & 8) lo = hi, hi = 0;
    lo = bits ? lo >> bits | hi << (64 - bits) : lo;
    hi >>= bits;
    if (by == 16) lo = hi = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  };
  f32x4 total[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) total[m][t] = f32x4{0, 0, 0, 0};

#pragma unroll
  for (int u = 0; u < U; ++u) load(u, wave + u * W);
  for (int base = wave; base < KB; base += U * W) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = base + u * W;
      if (kb >= KB) break;
      if (128 * kb + 128 > p.K) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = 128 * kb + 32 * g + 16 * i;
#pragma unroll
          for (int t = 0; t < NT; ++t) wq[u][t][i] = trim(wq[u][t][i], k);
#pragma unroll
          for (int t = 0; t < MT; ++t) xq[u][t][i] = trim(xq[u][t][i], k);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const f32x4 d = mma(wq[u][t][0], wq[u][t][1], xq[u][m][0], xq[u][m][1]);
          const float s = xs[u][m] * ws[u][t];
#pragma unroll
          for (int e = 0; e < 4; ++e) total[m][t][e] = __builtin_fmaf(d[e], s, total[m][t][e]);
        }
      load(u, base + (u + U) * W);
    }
  }
  // the waves' sums, added in their order
  constexpr int PART = MT * NT * 64;
  f32x4* part = reinterpret_cast<f32x4*>(red);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) part[wave * PART + (m * NT + t) * 64 + lane] = total[m][t];
  __syncthreads();
  for (int i = threadIdx.x; i < PART; i += blockDim.x) {
    f32x4 y = part[i];
    for (int w = 1; w < W; ++w) y += part[w * PART + i];
    const int l = i & 63, t = (i >> 6) % NT, m = (i >> 6) / NT;
    store4<BF16>(p, m0 + 16 * m + (l & 15), n0 + 16 * t + 4 * (l >> 4), y, whole);
  }
}

// K below 16, where no whole piece of a row exists: one result to a thread.
template <bool BF16>
__global__ __launch_bounds__(256) void f8_short_kernel(F8Args p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * p.N) return;
  const int n = (int)(i % p.N), m = (int)(i / p.N);
  float y = 0.f;
  for (int k = 0; k < p.K; ++k)
    y = __builtin_fmaf(from_code<MI_DECODE_E4M3>(p.x[m * p.ldx + k]), from_code<MI_DECODE_E4M3>(p.w[n * p.ldw + k]), y);
  if (p.K > 0) y *= p.xs[m * p.ldxs] * p.ws[n / 128 * p.ldws];
  static_cast<uint16_t*>(p.y)[m * p.ldy + n] = to16<BF16>(y + bias_of<BF16>(p, n));
}

// ------------------------------------------------------------- many tokens --

constexpr uint32_t kOutside = 0x80000000u;  // past every descriptor's end: reads zero
constexpr int kRsrcWord3 = 0x00020000;

__device__ inline u32x4 raw_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, (uint32_t)kRsrcWord3};
}
__device__ inline uint32_t lds_at(const void* p) { return (uint32_t)reinterpret_cast<uint64_t>(p); }
// A lane's 16 or 4 bytes at voff + soff go to shared memory at lds + 16 or 4 times the lane.
__device__ inline void copy16(const u32x4& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory", "m0");
}
__device__ inline void copy4(const u32x4& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory", "m0");
}

// Tile (tm, tn) of workgroup id: neighbouring ids go to different XCDs, so each
// of the eight gets a run of tiles, which go down GROUP tile rows at a time.
__device__ inline void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GROUP = 8;
  const int all = tiles_m * tiles_n, q = all >> 3, rest = all & 7, x = id & 7;
  id = x * q + min(x, rest) + (id >> 3);
  const int band = id / (GROUP * tiles_n), rows = min(GROUP, tiles_m - band * GROUP), in = id - band * GROUP * tiles_n;
  tm = band * GROUP + in % rows;
  tn = in / rows;
}

// BM tokens by BN weight rows to a workgroup of WM x WN waves; a stage is one
// block of 128 columns, rows of 128 bytes whose 16-byte pieces are exchanged by
// (row / 2) % 8, so that eight rows' reads of one piece meet no bank twice.
template <bool BF16, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void f8_tile_kernel(F8Args p, int whole) {
  constexpr int W = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int XB = BM * 128, WB = BN * 128, STAGE = XB + WB + BM * 4 + 256;
  static_assert(128 % TN == 0 && BM % 64 == 0 && BM / 64 < W, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, g = lane >> 4;
  const int KB = (p.K + 127) >> 7;
  int tm, tn;
  tile_of(blockIdx.x, (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int xrows = min(BM, p.M - m0), wrows = min(BN, p.N - n0), b0 = n0 / 128, brows = (n0 + wrows - 1) / 128 - b0 + 1;
  const u32x4 rx = raw_rsrc(p.x + m0 * p.ldx, (uint32_t)((xrows - 1) * p.ldx + p.K));
  const u32x4 rw = raw_rsrc(p.w + n0 * p.ldw, (uint32_t)((wrows - 1) * p.ldw + p.K));
  const u32x4 rxs = raw_rsrc(p.xs + m0 * p.ldxs, (uint32_t)(4 * ((xrows - 1) * p.ldxs + KB)));
  const u32x4 rws = raw_rsrc(p.ws + b0 * p.ldws, (uint32_t)(4 * ((brows - 1) * p.ldws + KB)));
  const uint32_t base = lds_at(lds);
  const int crow = lane >> 3;
  auto copy = [&](int st, int kb) {
    const uint32_t to = base + st * STAGE;
#pragma unroll
    for (int i = 0; i < BM / 8 / W; ++i) {
      const int blk = wave * (BM / 8 / W) + i, row = 8 * blk + crow, ch = (lane & 7) ^ ((row >> 1) & 7);
      const bool in = row < xrows && 128 * kb + 16 * ch < p.K;
      copy16(rx, in ? (uint32_t)(row * p.ldx + 16 * ch) : kOutside, 128u * kb, to + 1024 * blk);
    }
#pragma unroll
    for (int i = 0; i < BN / 8 / W; ++i) {
      const int blk = wave * (BN / 8 / W) + i, row = 8 * blk + crow, ch = (lane & 7) ^ ((row >> 1) & 7);
      const bool in = row < wrows && 128 * kb + 16 * ch < p.K;
      copy16(rw, in ? (uint32_t)(row * p.ldw + 16 * ch) : kOutside, 128u * kb, to + XB + 1024 * blk);
    }
    if (wave < BM / 64) {
      const int row = 64 * wave + lane;
      copy4(rxs, row < xrows ? (uint32_t)(4 * row * p.ldxs) : kOutside, 4u * kb, to + XB + WB + 256 * wave);
    } else if (wave == W - 1) {
      copy4(rws, lane < brows ? (uint32_t)(4 * lane * p.ldws) : kOutside, 4u * kb, to + XB + WB + 4 * BM);
    }
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};

  const int sw = (r >> 1) & 7;
  copy(0, 0);
  for (int kb = 0; kb < KB; ++kb) {
    __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8));  // vmcnt(0)
    __syncthreads();
    if (kb + 1 < KB) copy((kb + 1) & 1, kb + 1);
    const uint8_t* at = lds + (kb & 1) * STAGE;
    const float* sc = reinterpret_cast<const float*>(at + XB + WB);
    const float ws = sc[BM + ((n0 & 127) + wn * TN) / 128];
    u32x4 wf[FN][2];
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        wf[n][i] = *reinterpret_cast<const u32x4*>(at + XB + (wn * TN + 16 * n + r) * 128 + 16 * ((g + 4 * i) ^ sw));
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      u32x4 xf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        xf[i] = *reinterpret_cast<const u32x4*>(at + (wm * TM + 16 * m + r) * 128 + 16 * ((g + 4 * i) ^ sw));
      const float s = sc[wm * TM + 16 * m + r] * ws;
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const f32x4 d = mma(wf[n][0], wf[n][1], xf[0], xf[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][n][e] = __builtin_fmaf(d[e], s, acc[m][n][e]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n)
      store4<BF16>(p, m0 + wm * TM + 16 * m + r, n0 + wn * TN + 16 * n + 4 * g, acc[m][n], whole);
}

// 256 x 256 tiles for eight waves in two groups that take turns at the matrix
// pipes: in each phase one group multiplies a block of 128 columns while the
// other reads its operands of its next block and issues copies.  Group g owns
// token rows 128 g .. 128 g + 127, its wave w weight rows 64 w .. 64 w + 63.
// Block kb is multiplied by group 0 in phase 2 kb, by group 1 in phase 2 kb + 1.
// Weights, scales and half of a group's tokens are read in the phase before, the
// other half while the first is multiplied.  Both operands have two stages: w and
// group 0's half of x are free after phase 2 kb, and group 0 refills them in
// phase 2 kb + 1; group 1's half is free after that, and group 1 refills it in
// phase 2 kb + 2.  Each waits for its copies at the end of its next
// multiplication, before the barrier behind which they are first read.
template <bool BF16>
__global__ __launch_bounds__(512) void f8_turns_kernel(F8Args p, int whole) {
  constexpr int BM = 256, BN = 256, FM = 8, FN = 4, XB = BM * 128, WB = BN * 128, STAGE = XB + WB + 4 * BM + 256;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = wave >> 2, w4 = wave & 3, r = lane & 15, g = lane >> 4;
  const int KB = (p.K + 127) >> 7;
  int tm, tn;
  tile_of(blockIdx.x, (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int xrows = min(BM, p.M - m0), wrows = min(BN, p.N - n0), b0 = n0 / 128, brows = (n0 + wrows - 1) / 128 - b0 + 1;
  const u32x4 rx = raw_rsrc(p.x + m0 * p.ldx, (uint32_t)((xrows - 1) * p.ldx + p.K));
  const u32x4 rw = raw_rsrc(p.w + n0 * p.ldw, (uint32_t)((wrows - 1) * p.ldw + p.K));
  const u32x4 rxs = raw_rsrc(p.xs + m0 * p.ldxs, (uint32_t)(4 * ((xrows - 1) * p.ldxs + KB)));
  const u32x4 rws = raw_rsrc(p.ws + b0 * p.ldws, (uint32_t)(4 * ((brows - 1) * p.ldws + KB)));
  const uint32_t base = lds_at(lds);
  // A copy is 8 rows; a lane's row of it, and its 16-byte piece in even and odd
  // ones.  Rows past the tile's end read past the descriptor's, so does a piece past K.
  const int crow = lane >> 3, ch0 = (lane & 7) ^ (lane >> 4), ch1 = ch0 ^ 4;
  const uint32_t x0 = (uint32_t)(crow * p.ldx + 16 * ch0), x1 = (uint32_t)(crow * p.ldx + 16 * ch1);
  const uint32_t w0 = (uint32_t)(crow * p.ldw + 16 * ch0), w1 = (uint32_t)(crow * p.ldw + 16 * ch1);
  auto copy_x = [&](int half, int kb) {
    const bool in0 = 128 * kb + 16 * ch0 < p.K, in1 = 128 * kb + 16 * ch1 < p.K;
    const uint32_t to = base + (kb & 1) * STAGE;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int blk = 16 * half + 4 * w4 + i;
      copy16(rx, i & 1 ? (in1 ? x1 : kOutside) : (in0 ? x0 : kOutside), (uint32_t)(8 * blk * p.ldx) + 128u * kb, to + 1024 * blk);
    }
    if (w4 < 2) {
      const int row = 128 * half + 64 * w4 + lane;
      copy4(rxs, row < xrows && kb < KB ? (uint32_t)(4 * row * p.ldxs) : kOutside, 4u * kb, to + XB + WB + 4 * (128 * half + 64 * w4));
    }
  };
  auto copy_w = [&](int kb) {
    const bool in0 = 128 * kb + 16 * ch0 < p.K, in1 = 128 * kb + 16 * ch1 < p.K;
    const uint32_t to = base + (kb & 1) * STAGE;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int blk = 8 * w4 + i;
      copy16(rw, i & 1 ? (in1 ? w1 : kOutside) : (in0 ? w0 : kOutside), (uint32_t)(8 * blk * p.ldw) + 128u * kb, to + XB + 1024 * blk);
    }
    if (w4 == 3) copy4(rws, lane < brows && kb < KB ? (uint32_t)(4 * lane * p.ldws) : kOutside, 4u * kb, to + XB + WB + 4 * BM);
  };
  auto landed = []() { __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8)); };  // vmcnt(0)

  const int sw = (r >> 1) & 7, p0 = 16 * (g ^ sw), p1 = p0 ^ 64;
  const uint8_t* xat = lds + (128 * grp + r) * 128;
  const uint8_t* wat = lds + XB + (64 * w4 + r) * 128;
  u32x4 xf[4][2], wf[FN][2];
  float sc[FM];
  auto read_x = [&](const uint8_t* at, int m) {
    xf[m & 3][0] = *reinterpret_cast<const u32x4*>(at + 2048 * m + p0);
    xf[m & 3][1] = *reinterpret_cast<const u32x4*>(at + 2048 * m + p1);
  };
  auto read = [&](int kb) {
    const int st = (kb & 1) * STAGE;
    const float* scales = reinterpret_cast<const float*>(lds + st + XB + WB);
    const float ws = scales[BM + w4 / 2];
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      wf[n][0] = *reinterpret_cast<const u32x4*>(wat + st + 2048 * n + p0);
      wf[n][1] = *reinterpret_cast<const u32x4*>(wat + st + 2048 * n + p1);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) read_x(xat + st, m);
#pragma unroll
    for (int m = 0; m < FM; ++m) sc[m] = scales[128 * grp + 16 * m + r] * ws;
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
  auto multiply = [&](int kb) {
    const uint8_t* at = xat + (kb & 1) * STAGE;
    __builtin_amdgcn_s_setprio(1);
    f32x4 d[3];
    auto add = [&](int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[i / FN][i % FN][e] = __builtin_fmaf(d[i % 3][e], sc[i / FN], acc[i / FN][i % FN][e]);
    };
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) {
      const int m = i / FN, n = i % FN;
      d[i % 3] = mma(wf[n][0], wf[n][1], xf[m & 3][0], xf[m & 3][1]);
      if (i >= 2) add(i - 2);
      if (n == FN - 1 && m + 4 < FM) read_x(at, m + 4);
      __builtin_amdgcn_sched_barrier(0);
    }
    add(FM * FN - 2), add(FM * FN - 1);
    __builtin_amdgcn_s_setprio(0);
  };

  copy_x(grp, 0);
  if (grp == 0) copy_w(0);
  landed();
  __syncthreads();
  if (grp == 1) __syncthreads();  // phase -1
  for (int kb = 0; kb < KB; ++kb) {
    copy_x(grp, kb + 1);
    if (grp == 0) copy_w(kb + 1);
    read(kb);
    __syncthreads();
    multiply(kb);
    landed();
    __syncthreads();
  }
  if (grp == 0) __syncthreads();
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n)
      store4<BF16>(p, m0 + 128 * grp + 16 * m + r, n0 + 64 * w4 + 16 * n + 4 * g, acc[m][n], whole);
}

// ----------------------------------------------------------------- choice --

template <bool BF16, int MT, int NT, int U>
hipError_t few(const F8Args& a, int whole, hipStream_t s) {
  const int KB = (a.K + 127) / 128;
  const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.M + 16 * MT - 1) / (16 * MT));
  if (grid.y > 65535) return hipErrorInvalidConfiguration;
  const int64_t each = ((int64_t)grid.x * grid.y + a.cus - 1) / a.cus;
  int waves = each < 16 ? 16 / (int)each : 1;
  if (waves < 4) waves = 4;
  if (waves > KB) waves = KB;
  return launch(f8_few_kernel<BF16, MT, NT, U>, grid, 64 * waves, waves * MT * NT * 1024, s, a, whole);
}

template <bool BF16, int BM, int BN, int WM, int WN>
hipError_t tiles(const F8Args& a, int whole, hipStream_t s) {
  const int64_t all = ((int64_t)a.M + BM - 1) / BM * (((int64_t)a.N + BN - 1) / BN);
  if (all > INT32_MAX) return hipErrorInvalidConfiguration;
  return launch(f8_tile_kernel<BF16, BM, BN, WM, WN>, dim3((unsigned)all), 64 * WM * WN, 0, s, a, whole);
}

template <bool BF16>
hipError_t pick(const F8Args& a, hipStream_t s) {
  if (a.K < 16) {
    const int64_t blocks = ((int64_t)a.M * a.N + 255) / 256;
    if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
    return launch(f8_short_kernel<BF16>, dim3((unsigned)blocks), 256, 0, s, a);
  }
  const int whole = a.N % 4 == 0 && a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 8 == 0;
  // a tile's rows lie within 2^31 bytes, and begin at multiples of 16
  const bool tiled = a.K % 16 == 0 && a.ldx % 16 == 0 && a.ldw % 16 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && a.ldx <= 1 << 22 && a.ldw <= 1 << 22 &&
                     a.ldxs <= 1 << 20 && a.ldws <= 1 << 20;
  if (a.M <= 16) return few<BF16, 1, 1, 2>(a, whole, s);
  if (a.M <= 32) return few<BF16, 2, 1, 2>(a, whole, s);
  if (a.M <= 64 || !tiled) return few<BF16, 4, 1, 1>(a, whole, s);
  if (a.M >= 256 && (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256) >= a.cus / 2) {
    const int64_t all = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
    if (all > INT32_MAX) return hipErrorInvalidConfiguration;
    return launch(f8_turns_kernel<BF16>, dim3((unsigned)all), 512, 0, s, a, whole);
  }
  return tiles<BF16, 128, 128, 2, 2>(a, whole, s);
}

}  // namespace

hipError_t launch_f8(const F8Args& a, hipStream_t s) { return a.bf16 ? pick<true>(a, s) : pick<false>(a, s); }

}  // namespace mid
