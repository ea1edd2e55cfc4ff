// Linear layer of 8-bit floats with block scales:
//   y[m][n] = sum_j (xs[m][j] ws[n / 128][j]) sum_{k in block j} x[m][k] w[n][k] + bias[n].
//
// A block of 128 columns is the depth of one 16x16x128 matrix instruction, so a
// block's sum is one instruction from zero, and its scales enter as one
// multiply-add for each of the four results in a lane.  Weights are the left
// operand: a lane holds four neighbouring n of one token, whose scale is one
// number of the lane's, and ws is the same for a wave's whole 16-row tile.
// Which 8 columns of a block stand where in the operands does not matter as long
// as it is the same for both.
//
// Precision.  Every matrix instruction for 8-bit floats adds the products of 8
// neighbouring columns in units of 2^-13 of the largest one's power of two, cut off
// towards zero (measured: beside 2^16 and -2^16, 2^3 is kept and 2^2 is not), and
// the sums of these in binary32.  Results of random operands are off by 2^-14 of
// their size for it, an eighth of what binary16 rounds off.  Operands in binary16
// would keep all bits, at half the rate and with a conversion of each.
#include <type_traits>
#include <utility>

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

__device__ __forceinline__ f32x4& add(f32x4& to, f32x4 d, float by) {
#pragma unroll
  for (int e = 0; e < 4; ++e) to[e] = __builtin_fmaf(d[e], by, to[e]);
  return to;
}
// Sums are done here, and not where they are used next.
__device__ __forceinline__ void here(f32x4& x) {
  asm volatile("" : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]));
}
// The N products of a block and their scaled additions: a product's results come
// 8 to 11 issue slots after it, so its additions follow the next LAG products
// (right behind the next one each product waits 3 to 6 slots: 8192 x 4096 x 11008
// 322 us, here 310).  `more` is what else is done meanwhile, such as reads.
template <int N, typename Mul, typename Add, typename More>
__device__ __forceinline__ void products(Mul mul, Add add, More more) {
  constexpr int LAG = 3;
  f32x4 d[LAG + 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    d[i % (LAG + 1)] = mul(i);
    __builtin_amdgcn_sched_barrier(0);
    if (i >= LAG) here(add(i - LAG, d[(i - LAG) % (LAG + 1)]));
    more(i);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = N < LAG ? 0 : N - LAG; i < N; ++i) here(add(i, d[i % (LAG + 1)]));
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

// ------------------------------------------------------- rows at any byte --

// A piece of 16 bytes from column k on, which was read 16 columns before K where it
// crosses K, without the bytes that lie past K.
__device__ inline u32x4 trim_bytes(u32x4 w, int k, int K) {
  const int by = min(max(k + 16 - K, 0), 16), bits = 8 * (by & 7);
  uint64_t lo = w[0] | (uint64_t)w[1] << 32, hi = w[2] | (uint64_t)w[3] << 32;
  if (by & 8) lo = hi, hi = 0;
  lo = bits ? lo >> bits | hi << (64 - bits) : lo;
  hi >>= bits;
  if (by == 16) lo = hi = 0;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// For few tokens and weight rows that do not begin at multiples of 4 bytes, or lie
// very far apart: 16 tokens by 16 weight rows to a workgroup, whose waves split K
// and load operands from memory: wave w of W takes blocks w, w + W, ..., U in flight.
template <bool BF16>
__global__ __launch_bounds__(1024) void f8_any_kernel(F8Args p, int whole) {
  constexpr int U = 2;
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int lane = threadIdx.x & 63, W = (int)(blockDim.x >> 6);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, KB = (p.K + 127) >> 7;
  const int n0 = blockIdx.x * 16;
  const uint8_t* wp = p.w + (int64_t)min(n0 + r, p.N - 1) * p.ldw;
  const uint8_t* xp = p.x + (int64_t)min(r, p.M - 1) * p.ldx;
  const float* sp = p.xs + (int64_t)min(r, p.M - 1) * p.ldxs;
  u32x4 wq[U][2], xq[U][2];
  float xs[U], ws[U];
  auto load = [&](int u, int kb) {
    const int at = min(kb, KB - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = min(128 * at + 32 * g + 16 * i, p.K - 16);
      wq[u][i] = *reinterpret_cast<const loose*>(wp + k);
      xq[u][i] = *reinterpret_cast<const loose*>(xp + k);
    }
    ws[u] = p.ws[n0 / 128 * p.ldws + at], xs[u] = sp[at];
  };
  f32x4 total = {0, 0, 0, 0};
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
          wq[u][i] = trim_bytes(wq[u][i], k, p.K), xq[u][i] = trim_bytes(xq[u][i], k, p.K);
        }
      }
      add(total, mma(wq[u][0], wq[u][1], xq[u][0], xq[u][1]), xs[u] * ws[u]);
      load(u, base + (u + U) * W);
    }
  }
  // the waves' sums, added in their order
  f32x4* part = reinterpret_cast<f32x4*>(red);
  part[threadIdx.x] = total;
  __syncthreads();
  if (wave) return;
  f32x4 y = part[lane];
  for (int w = 1; w < W; ++w) y += part[64 * w + lane];
  store4<BF16>(p, r, n0 + 4 * g, y, whole);
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
// A lane's 16 or 4 bytes at voff + soff go to shared memory at lds + PLUS + 16 or 4 times the lane.
// A copy reads m0 one wait state after it is written at the earliest, which the
// compiler sees to for its own copies and not within asm.
template <int PLUS>
__device__ __forceinline__ void copy16(const u32x4& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc), "s"(soff), "n"(PLUS)
               : "memory", "m0", "scc");
}
template <int PLUS>
__device__ __forceinline__ void copy4(const u32x4& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc), "s"(soff), "n"(PLUS)
               : "memory", "m0", "scc");
}
__device__ __forceinline__ uint32_t uniform(int64_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
// A number at compile time for each i below N.
template <int N, typename F, int... I>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each<N>(f, std::make_integer_sequence<int, N>{});
}

// Where a lane's 16-byte pieces of the next block to be copied lie: rows of an
// operand go to shared memory eight at a time, with their pieces exchanged by
// (row / 2) % 8, so `at` differs in even and odd copies.  Rows past the last one
// lie past the descriptor's end; pieces past K are sent there, and one that
// crosses K (a multiple of 4) is read 16 columns before K, for `trim`.
struct Walk {
  uint32_t at[2];
  int ch[2];
  __device__ Walk(int64_t ld, int lane) {
    ch[0] = (lane & 7) ^ (lane >> 4), ch[1] = ch[0] ^ 4;
    at[0] = (uint32_t)((lane >> 3) * ld + 16 * ch[0]), at[1] = (uint32_t)((lane >> 3) * ld + 16 * ch[1]);
  }
  __device__ void begin(int kb, int K) {
    at[0] += 128u * kb, at[1] += 128u * kb;
    cut(kb, K);
  }
  // kb: the block that comes next, `by` blocks further on
  __device__ void next(int kb, int by, int K) {
    at[0] += 128u * by, at[1] += 128u * by;
    cut(kb, K);
  }
  __device__ void cut(int kb, int K) {
    if (128 * kb + 128 <= K) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (128 * kb + 16 * ch[i] >= K) at[i] = kOutside;
      else at[i] -= max(128 * kb + 16 * ch[i] + 16 - K, 0);
  }
};

// A piece from column k on that crosses K: its last columns, in their place, and zeros.
__device__ __forceinline__ void trim(u32x4& w, int k, int K) {
  const int by = k < K && k + 16 > K ? (k + 16 - K) / 4 : 0;
  if (by & 1) w = u32x4{w[1], w[2], w[3], 0};
  if (by & 2) w = u32x4{w[2], w[3], 0, 0};
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

// For rows at any byte, or far apart: BM tokens by BN weight rows to a workgroup of
// WM x WN waves.  Copies into shared memory need rows at multiples of 4 bytes, so a
// block of 128 columns is loaded into registers while the one before is
// multiplied, and stored from there, pieces exchanged as in f8_tile_kernel.
//
// Bound: latency, one block ahead (77 x 5003 x 4071 28 us, 26 with two; 512 x 4096 x
// 4095 32 and 35; 4096^3 less one column 160, 860 TFLOP/s, matrix pipes busy in 21 % of
// the cycles).  Each wave for itself with
// operands from memory, as above, takes 69, 450 (345 with four strips of tokens) and 2700.
template <bool BF16, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void f8_loose_kernel(F8Args p, int whole) {
  constexpr int T = 64 * WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16, PX = BM * 8 / T, PW = BN * 8 / T;
  constexpr int XB = BM * 128, STAGE = XB + BN * 128 + BM * 4;
  static_assert(PX * T == BM * 8 && PW * T == BN * 8 && BM <= T && 128 % BN == 0 && 2 * STAGE <= 160 << 10, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, g = lane >> 4, KB = (p.K + 127) >> 7;
  int tm, tn;
  tile_of(blockIdx.x, (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  // piece i of a thread: row (tid + T i) / 8, columns 16 c and on
  const int c = tid & 7;
  const uint8_t *xp[PX], *wp[PW];
#pragma unroll
  for (int i = 0; i < PX; ++i) xp[i] = p.x + (int64_t)min(m0 + (tid + T * i) / 8, p.M - 1) * p.ldx;
#pragma unroll
  for (int i = 0; i < PW; ++i) wp[i] = p.w + (int64_t)min(n0 + (tid + T * i) / 8, p.N - 1) * p.ldw;
  const float* sp = p.xs + (int64_t)min(m0 + min(tid, BM - 1), p.M - 1) * p.ldxs;
  const float* ws_row = p.ws + n0 / 128 * p.ldws;
  u32x4 xq[PX], wq[PW];
  float sq, ws;
  auto load = [&](int kb) {
    const int k = min(128 * kb + 16 * c, p.K - 16);
#pragma unroll
    for (int i = 0; i < PX; ++i) xq[i] = *reinterpret_cast<const loose*>(xp[i] + k);
#pragma unroll
    for (int i = 0; i < PW; ++i) wq[i] = *reinterpret_cast<const loose*>(wp[i] + k);
    sq = sp[kb], ws = ws_row[kb];
  };
  auto store = [&](int kb) {
    uint8_t* to = lds + (kb & 1) * STAGE;
    const int k = 128 * kb + 16 * c;
    if (128 * kb + 128 > p.K) {
#pragma unroll
      for (int i = 0; i < PX; ++i) xq[i] = trim_bytes(xq[i], k, p.K);
#pragma unroll
      for (int i = 0; i < PW; ++i) wq[i] = trim_bytes(wq[i], k, p.K);
    }
    auto at = [&](int i) {
      const int row = (tid + T * i) / 8;
      return 128 * row + 16 * (c ^ ((row >> 1) & 7));
    };
#pragma unroll
    for (int i = 0; i < PX; ++i) *reinterpret_cast<u32x4*>(to + at(i)) = xq[i];
#pragma unroll
    for (int i = 0; i < PW; ++i) *reinterpret_cast<u32x4*>(to + XB + at(i)) = wq[i];
    if (tid < BM) reinterpret_cast<float*>(to + XB + BN * 128)[tid] = sq * ws;
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
  const int sw = (r >> 1) & 7, p0 = 128 * r + 16 * (g ^ sw), p1 = p0 ^ 64;
  load(0);
  for (int kb = 0; kb < KB; ++kb) {
    store(kb);  // who still reads the block before does so in the other stage
    __syncthreads();
    if (kb + 1 < KB) load(kb + 1);
    const uint8_t *x = lds + (kb & 1) * STAGE + wm * TM * 128, *w = lds + (kb & 1) * STAGE + XB + wn * TN * 128;
    const float* sc = reinterpret_cast<const float*>(lds + (kb & 1) * STAGE + XB + BN * 128) + wm * TM + r;
    u32x4 wf[FN][2], xf[FM][2];
    float s[FM];
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      wf[n][0] = *reinterpret_cast<const u32x4*>(w + 2048 * n + p0);
      wf[n][1] = *reinterpret_cast<const u32x4*>(w + 2048 * n + p1);
    }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      xf[m][0] = *reinterpret_cast<const u32x4*>(x + 2048 * m + p0);
      xf[m][1] = *reinterpret_cast<const u32x4*>(x + 2048 * m + p1);
      s[m] = sc[16 * m];
    }
    products<FM * FN>(
        [&](int i) { return mma(wf[i % FN][0], wf[i % FN][1], xf[i / FN][0], xf[i / FN][1]); },
        [&](int i, f32x4 d) -> f32x4& { return add(acc[i / FN][i % FN], d, s[i / FN]); },
        [](int) {});
  }
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n)
      store4<BF16>(p, m0 + wm * TM + 16 * m + r, n0 + wn * TN + 16 * n + 4 * g, acc[m][n], whole);
}

// BM tokens by BN weight rows to a workgroup of WM x WN waves; a stage of the
// ring is one block of 128 columns, rows of 128 bytes whose 16-byte pieces are
// exchanged by (row / 2) % 8, so that eight rows' reads of one piece meet no bank
// twice.
//
// Bound: copies, reads and products side by side, none of them alone; the smaller the
// tile, the more copies to a product (matrix pipes busy in 13 % of the cycles at 77 x
// 5003 x 4072 with 64 x 64, 22 at 512 x 4096 x 4096 with 64 x 128, 35 at 1024 with 128 x
// 128, 47 at 2048 with 128 x 256).  1024 x 4096
// x 4096 took 41 us with a stage's copies issued together and 28 with them spread
// between its products; on the way, at 32, leaving out the copies, the reads or the
// products (a copy, for timing) left 22, 24 and 26.  Two, three or four stages
// make no difference.  Copies of what lies in an XCD's cache reach 128 GB/s for a
// compute unit, from the last-level cache 28, so workgroups that run together on an XCD
// share rows of tiles (tile_of).
template <bool BF16, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) void f8_tile_kernel(F8Args p, int whole) {
  constexpr int W = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int XB = BM * 128, WB = BN * 128, STAGE = XB + WB + BM * 4 + 256;
  constexpr int CX = BM / 8 / W, CW = BN / 8 / W, COPIES = CX + CW + 1;
  static_assert(128 % TN == 0 && BM % 64 == 0 && BM / 64 < W && CX * W * 8 == BM && CW * W * 8 == BN && S * STAGE <= 160 << 10, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * STAGE];
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
  static_assert(CX % 2 == 0 && CW % 2 == 0, "a wave's first copy is an even one");
  Walk xw(p.ldx, lane), ww(p.ldw, lane);
  const bool of_x = wave < BM / 64;  // scales: of 64 tokens, or of the weights (the same from each of those waves)
  const u32x4 rs = of_x ? rxs : rws;
  const int srow = of_x ? 64 * wave + lane : lane;
  uint32_t sat = srow < (of_x ? xrows : brows) ? (uint32_t)(4 * srow * (of_x ? p.ldxs : p.ldws)) : kOutside;
  const uint32_t xbase = base + 1024 * CX * wave, wbase = base + XB + 1024 * CW * wave, sbase = base + XB + WB + (of_x ? 256 * wave : 4 * BM);
  const uint32_t xrow = uniform(8 * CX * wave * p.ldx), wrow = uniform(8 * CW * wave * p.ldw);
  const uint32_t x8 = uniform(8 * p.ldx), w8 = uniform(8 * p.ldw);
  // copy i of a wave's COPIES ones
  auto copy = [&](auto ic, int st) {
    constexpr int i = decltype(ic)::value;
    if constexpr (i < CX) copy16<1024 * i>(rx, xw.at[i & 1], xrow + i * x8, xbase + st * STAGE);
    else if constexpr (i < CX + CW) copy16<1024 * (i - CX)>(rw, ww.at[i & 1], wrow + (i - CX) * w8, wbase + st * STAGE);
    else copy4<0>(rs, sat, 0, sbase + st * STAGE);
  };
  auto next = [&](int kb) {  // the copies that follow are of block kb
    xw.next(kb, 1, p.K), ww.next(kb, 1, p.K);
    sat = kb < KB ? sat + 4 : kOutside;
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};

  const int sw = (r >> 1) & 7, p0 = 128 * r + 16 * (g ^ sw), p1 = p0 ^ 64;
  struct Operands {
    u32x4 w[FN][2], x[FM][2];
    float s[FM], ws;
  };
  constexpr int READS = 2 * FN + 3 * FM + 1;
  // read i of READS
  auto read = [&](int i, Operands& o, int st) {
    const uint8_t* at = lds + st * STAGE;
    const float* sc = reinterpret_cast<const float*>(at + XB + WB);
    if (i < 2 * FN) o.w[i / 2][i & 1] = *reinterpret_cast<const u32x4*>(at + XB + (wn * TN + 16 * (i / 2)) * 128 + (i & 1 ? p1 : p0));
    else if (i < 2 * (FN + FM)) o.x[i / 2 - FN][i & 1] = *reinterpret_cast<const u32x4*>(at + (wm * TM + 16 * (i / 2 - FN)) * 128 + (i & 1 ? p1 : p0));
    else if (i < 2 * FN + 3 * FM) o.s[i - 2 * (FN + FM)] = sc[wm * TM + 16 * (i - 2 * (FN + FM)) + r];
    else o.ws = sc[BM + ((n0 & 127) + wn * TN) / 128];
  };
  auto landed = [](auto blocks) {  // all but the last `blocks` ones, and what was read is in registers
    constexpr int left = decltype(blocks)::value * COPIES;
    static_assert(left < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((left & 15) | ((left >> 4) << 14) | (0x7 << 4));
  };
  xw.begin(0, p.K), ww.begin(0, p.K);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    each<COPIES>([&](auto i) { copy(i, s); });
    next(s + 1);
  }
  landed(std::integral_constant<int, S - 1>{});
  __syncthreads();
  // While a block is multiplied, the next one's operands are read and the copies
  // of the block S further on go where it was: a few of them behind each product.
  int st = 0;
  auto step = [&](Operands& now, Operands& ahead, int kb) {
    landed(std::integral_constant<int, S - 2>{});  // block kb + 1
    __syncthreads();
    const int old = st;
    if (++st == S) st = 0;
    if (kb == KB - 1 && p.K % 16) {
#pragma unroll
      for (int n = 0; n < FN; ++n) trim(now.w[n][0], 128 * kb + 16 * g, p.K), trim(now.w[n][1], 128 * kb + 64 + 16 * g, p.K);
#pragma unroll
      for (int m = 0; m < FM; ++m) trim(now.x[m][0], 128 * kb + 16 * g, p.K), trim(now.x[m][1], 128 * kb + 64 + 16 * g, p.K);
    }
#pragma unroll
    for (int m = 0; m < FM; ++m) now.s[m] *= now.ws;
    constexpr int N = FM * FN;
    products<N>(
        [&](int i) { return mma(now.w[i % FN][0], now.w[i % FN][1], now.x[i / FN][0], now.x[i / FN][1]); },
        [&](int i, f32x4 d) -> f32x4& { return add(acc[i / FN][i % FN], d, now.s[i / FN]); },
        [&](int i) {
#pragma unroll
          for (int j = i * READS / N; j < (i + 1) * READS / N; ++j) read(j, ahead, st);
          each<COPIES>([&](auto j) {
            if (decltype(j)::value >= i * COPIES / N && decltype(j)::value < (i + 1) * COPIES / N) copy(j, old);
          });
        });
    next(kb + S + 1);
  };
  Operands a, b;
#pragma unroll
  for (int i = 0; i < READS; ++i) read(i, a, 0);
  for (int kb = 0; kb < KB; kb += 2) {
    step(a, b, kb);
    if (kb + 1 < KB) step(b, a, kb + 1);
  }
  __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8));  // vmcnt(0): no copy outlives the workgroup
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
//
// Bound: matrix instructions.  8192 x 4096 x 11008 310 to 323 us on different boards,
// 2290 to 2380 TFLOP/s, where a large library product with one scale for each operand
// reaches 2590; matrix pipes are busy in 64 % of the cycles.  A scaled addition is four
// vector instructions to 32 cycles of the matrix pipe.
template <bool BF16, int BN>
__global__ __launch_bounds__(512) void f8_turns_kernel(F8Args p, int whole) {
  constexpr int BM = 256, TN = BN / 4, FM = 8, FN = TN / 16, XB = BM * 128, WB = BN * 128, STAGE = XB + WB + 4 * BM + 256;
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
  Walk xw(p.ldx, lane), ww(p.ldw, lane);
  const int srow = 128 * grp + 64 * w4 + lane;
  uint32_t xs_at = w4 < 2 && srow < xrows ? (uint32_t)(4 * srow * p.ldxs) : kOutside;
  uint32_t ws_at = lane < brows ? (uint32_t)(4 * lane * p.ldws) : kOutside;
  const uint32_t xbase = base + 1024 * (16 * grp + 4 * w4), wbase = base + XB + BN / 32 * 1024 * w4;
  const uint32_t xrow = uniform(8 * (16 * grp + 4 * w4) * p.ldx), wrow = uniform(BN / 4 * w4 * p.ldw);
  const uint32_t x8 = uniform(8 * p.ldx), w8 = uniform(8 * p.ldw);
  // the group's half of x, and group 0's weights, of the block where the walks stand
  auto copy = [&](int kb) {
    const uint32_t st = (kb & 1) * STAGE;
    if (grp == 0) {
      each<BN / 32>([&](auto i) { copy16<1024 * decltype(i)::value>(rw, ww.at[i & 1], wrow + i * w8, wbase + st); });
      if (w4 == 3) copy4<XB + WB + 4 * BM>(rws, ws_at, 0, base + st);
    }
    each<4>([&](auto i) { copy16<1024 * decltype(i)::value>(rx, xw.at[i & 1], xrow + i * x8, xbase + st); });
    if (w4 < 2) copy4<XB + WB>(rxs, xs_at, 0, base + st + 4 * (128 * grp + 64 * w4));
    xw.next(kb + 1, 1, p.K), ww.next(kb + 1, 1, p.K);
    xs_at = kb + 1 < KB ? xs_at + 4 : kOutside;
    ws_at = kb + 1 < KB ? ws_at + 4 : kOutside;
  };
  auto landed = []() { __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8)); };  // vmcnt(0)

  const int sw = (r >> 1) & 7, p0 = 16 * (g ^ sw), p1 = p0 ^ 64;
  const uint8_t* xat = lds + (128 * grp + r) * 128;
  const uint8_t* wat = lds + XB + (TN * w4 + r) * 128;
  u32x4 xf[4][2], wf[FN][2];
  float sc[FM];
  auto read_x = [&](const uint8_t* at, int m) {
    xf[m & 3][0] = *reinterpret_cast<const u32x4*>(at + 2048 * m + p0);
    xf[m & 3][1] = *reinterpret_cast<const u32x4*>(at + 2048 * m + p1);
  };
  auto read = [&](int kb) {
    const int st = (kb & 1) * STAGE;
    const float* scales = reinterpret_cast<const float*>(lds + st + XB + WB);
    const float ws = scales[BM + ((n0 & 127) + TN * w4) / 128];
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
    products<FM * FN>(
        [&](int i) { return mma(wf[i % FN][0], wf[i % FN][1], xf[i / FN & 3][0], xf[i / FN & 3][1]); },
        [&](int i, f32x4 d) -> f32x4& { return add(acc[i / FN][i % FN], d, sc[i / FN]); },
        [&](int i) {
          if (i % FN == FN - 1 && i / FN + 4 < FM) read_x(at, i / FN + 4);
        });
    __builtin_amdgcn_s_setprio(0);
  };

  xw.begin(0, p.K), ww.begin(0, p.K);
  copy(0);
  landed();
  __syncthreads();
  if (grp == 1) __syncthreads();  // phase -1
  for (int kb = 0; kb < KB; ++kb) {
    copy(kb + 1);
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
      store4<BF16>(p, m0 + 128 * grp + 16 * m + r, n0 + TN * w4 + 16 * n + 4 * g, acc[m][n], whole);
}

// --------------------------------------------------- strips of weight rows --

// 16 NT weight rows by up to 16 MT tokens to a workgroup whose W waves split K:
// wave w takes blocks w, w + W, ... through a ring of S stages of its own in
// shared memory, so that no wave waits for another before the sums are added.
//
// Bound: launch and one or two rounds of loads for small weights (1 x 4096 x 4096
// 5.7 us with weights from memory, 4.8 from the last-level cache), the weights' bytes
// for large ones (1 x 14336 x 4096 14.9, 3.9 TB/s).  With operands in registers
// instead, which hold fewer loads in flight, 64 x 4096 x 4096 took 22 us; here 9.3.
// Towards 64 tokens, copies of x: each wave copies all tokens' columns of its own
// blocks, and each workgroup does so again, four fifths of the copied bytes with
// strips of 16 rows and half with 64 (matrix pipes busy in 5 and 11 % of the cycles).
template <bool BF16, int MT, int NT, int S, int W>
__global__ __launch_bounds__(64 * W) void f8_strip_kernel(F8Args p, int whole) {
  constexpr int SCALES = (MT + 3) / 4, STAGE = 2048 * (MT + NT) + 256 * SCALES, COPIES = 2 * (MT + NT) + SCALES;
  constexpr int PART = MT * NT * 64;
  static_assert(W * S * STAGE <= 160 << 10 && W * PART * 16 <= W * S * STAGE && S >= 2 && S <= 4 && 8 % NT == 0, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * S * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, KB = (p.K + 127) >> 7;
  const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
  const int xrows = min(16 * MT, p.M - m0), wrows = min(16 * NT, p.N - n0);
  const u32x4 rx = raw_rsrc(p.x + m0 * p.ldx, (uint32_t)((xrows - 1) * p.ldx + p.K));
  const u32x4 rw = raw_rsrc(p.w + n0 * p.ldw, (uint32_t)((wrows - 1) * p.ldw + p.K));
  const u32x4 rxs = raw_rsrc(p.xs + m0 * p.ldxs, (uint32_t)(4 * ((xrows - 1) * p.ldxs + KB)));
  const float* ws_row = p.ws + n0 / 128 * p.ldws;
  const uint32_t base = lds_at(lds) + wave * (S * STAGE);
  const uint8_t* mine = lds + wave * (S * STAGE);
  Walk xw(p.ldx, lane), ww(p.ldw, lane);
  uint32_t sat[SCALES];
#pragma unroll
  for (int i = 0; i < SCALES; ++i) sat[i] = 64 * i + lane < xrows ? (uint32_t)(4 * ((64 * i + lane) * p.ldxs + wave)) : kOutside;
  const uint32_t x8 = uniform(8 * p.ldx), w8 = uniform(8 * p.ldw);
  // the block where the walks stand, and on to kb
  auto copy = [&](int st, int kb) {
    const uint32_t to = base + st * STAGE;
    each<2 * NT>([&](auto i) { copy16<1024 * decltype(i)::value>(rw, ww.at[i & 1], i * w8, to); });
    each<2 * MT>([&](auto i) { copy16<2048 * NT + 1024 * decltype(i)::value>(rx, xw.at[i & 1], i * x8, to); });
    each<SCALES>([&](auto i) {
      copy4<2048 * (NT + MT) + 256 * decltype(i)::value>(rxs, sat[i], 0, to);
      sat[i] += sat[i] < kOutside ? 4 * W : 0;
    });
    xw.next(kb, W, p.K), ww.next(kb, W, p.K);
  };
  auto landed = [](auto left) {  // all but the copies of the last `left` blocks
    constexpr int n = decltype(left)::value * COPIES;
    static_assert(n < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (0x7 << 4) | (0xf << 8));
  };
  f32x4 total[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) total[m][t] = f32x4{0, 0, 0, 0};

  // lane l knows the weights' scale of the wave's block `from` + l
  const int blocks = wave < KB ? (KB - wave + W - 1) / W : 0;
  float ws = lane < blocks ? ws_row[wave + W * lane] : 0.f;
  xw.begin(wave, p.K), ww.begin(wave, p.K);
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < blocks) copy(s, wave + W * (s + 1));
  const int sw = (r >> 1) & 7, p0 = 128 * r + 16 * (g ^ sw), p1 = p0 ^ 64;
  int st = 0;
  for (int i = 0; i < blocks; ++i) {
    if (i && (i & 63) == 0) {
      ws = i + lane < blocks ? ws_row[wave + W * (i + lane)] : 0.f;
    }
    if (i + S - 1 < blocks) {
      landed(std::integral_constant<int, S - 1>{});
    } else if (S > 3 && i + 2 < blocks) {
      landed(std::integral_constant<int, S == 4 ? 2 : 0>{});
    } else if (S > 2 && i + 1 < blocks) {
      landed(std::integral_constant<int, 1>{});
    } else {
      landed(std::integral_constant<int, 0>{});
    }
    const uint8_t* at = mine + st * STAGE;
    u32x4 wf[NT][2], xf[MT][2];
    float s[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wf[t][0] = *reinterpret_cast<const u32x4*>(at + 2048 * t + p0);
      wf[t][1] = *reinterpret_cast<const u32x4*>(at + 2048 * t + p1);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      xf[m][0] = *reinterpret_cast<const u32x4*>(at + 2048 * (NT + m) + p0);
      xf[m][1] = *reinterpret_cast<const u32x4*>(at + 2048 * (NT + m) + p1);
      s[m] = reinterpret_cast<const float*>(at + 2048 * (NT + MT))[16 * m + r];
    }
    const int kb = wave + W * i;
    if (kb == KB - 1 && p.K % 16) {
#pragma unroll
      for (int t = 0; t < NT; ++t) trim(wf[t][0], 128 * kb + 16 * g, p.K), trim(wf[t][1], 128 * kb + 64 + 16 * g, p.K);
#pragma unroll
      for (int m = 0; m < MT; ++m) trim(xf[m][0], 128 * kb + 16 * g, p.K), trim(xf[m][1], 128 * kb + 64 + 16 * g, p.K);
    }
    __builtin_amdgcn_s_waitcnt(0xf | (3 << 14) | (0x7 << 4));  // lgkmcnt(0): the stage has been read
    if (i + S < blocks) copy(st, wave + W * (i + S + 1));
    const float wi = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ws), i & 63));
#pragma unroll
    for (int m = 0; m < MT; ++m) s[m] *= wi;
    products<MT * NT>(
        [&](int i) { return mma(wf[i % NT][0], wf[i % NT][1], xf[i / NT][0], xf[i / NT][1]); },
        [&](int i, f32x4 d) -> f32x4& { return add(total[i / NT][i % NT], d, s[i / NT]); },
        [](int) {});
    if (++st == S) st = 0;
  }
  // the waves' sums, added in their order
  f32x4* part = reinterpret_cast<f32x4*>(lds);
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) part[wave * PART + (m * NT + t) * 64 + lane] = total[m][t];
  __syncthreads();
  for (int i = threadIdx.x; i < PART; i += 64 * W) {
    f32x4 y = part[i];
#pragma unroll
    for (int w = 1; w < W; ++w) y += part[w * PART + i];
    const int l = i & 63, t = (i >> 6) % NT, m = (i >> 6) / NT;
    store4<BF16>(p, m0 + 16 * m + (l & 15), n0 + 16 * t + 4 * (l >> 4), y, whole);
  }
}

// ----------------------------------------------------------------- choice --

template <bool BF16>
hipError_t any(const F8Args& a, int whole, hipStream_t s) {
  const int KB = (a.K + 127) / 128, waves = KB < 16 ? KB : 16;
  return launch(f8_any_kernel<BF16>, dim3((a.N + 15) / 16), 64 * waves, waves * 1024, s, a, whole);
}

template <bool BF16, int BM, int BN, int WM, int WN>
hipError_t loosely(const F8Args& a, int whole, hipStream_t s) {
  const int64_t all = ((int64_t)a.M + BM - 1) / BM * (((int64_t)a.N + BN - 1) / BN);
  if (all > INT32_MAX) return hipErrorInvalidConfiguration;
  return launch(f8_loose_kernel<BF16, BM, BN, WM, WN>, dim3((unsigned)all), 64 * WM * WN, 0, s, a, whole);
}

template <bool BF16, int BM, int BN, int WM, int WN, int S>
hipError_t tiles(const F8Args& a, int whole, hipStream_t s) {
  const int64_t all = ((int64_t)a.M + BM - 1) / BM * (((int64_t)a.N + BN - 1) / BN);
  if (all > INT32_MAX) return hipErrorInvalidConfiguration;
  return launch(f8_tile_kernel<BF16, BM, BN, WM, WN, S>, dim3((unsigned)all), 64 * WM * WN, 0, s, a, whole);
}

template <bool BF16, int BN>
hipError_t turns(const F8Args& a, int whole, hipStream_t s) {
  const int64_t all = ((int64_t)a.M + 255) / 256 * (((int64_t)a.N + BN - 1) / BN);
  if (all > INT32_MAX) return hipErrorInvalidConfiguration;
  return launch(f8_turns_kernel<BF16, BN>, dim3((unsigned)all), 512, 0, s, a, whole);
}

template <bool BF16, int MT, int NT, int S, int W>
hipError_t strips(const F8Args& a, int whole, hipStream_t s) {
  const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.M + 16 * MT - 1) / (16 * MT));
  if (grid.y > 65535) return hipErrorInvalidConfiguration;
  return launch(f8_strip_kernel<BF16, MT, NT, S, W>, grid, 64 * W, 0, s, a, whole);
}

template <bool BF16>
hipError_t pick(const F8Args& a, hipStream_t s) {
  if (a.K < 16) {
    const int64_t blocks = ((int64_t)a.M * a.N + 255) / 256;
    if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
    return launch(f8_short_kernel<BF16>, dim3((unsigned)blocks), 256, 0, s, a);
  }
  const int whole = a.N % 4 == 0 && a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 8 == 0;
  // Copies into shared memory: rows begin at multiples of 4 bytes, and those of
  // a tile lie within 2^31 bytes.
  auto multiple = [&](int n) {
    return a.K % n == 0 && a.ldx % n == 0 && a.ldw % n == 0 && reinterpret_cast<uintptr_t>(a.x) % n == 0 &&
           reinterpret_cast<uintptr_t>(a.w) % n == 0;
  };
  const bool narrow = (a.N + 15) / 16 <= a.cus;
  if (!multiple(4) || a.ldx > 1 << 22 || a.ldw > 1 << 22 || a.ldxs > 1 << 20 || a.ldws > 1 << 20) {
    // us with strips and tiles: 1 token, K 4095, N 4096 18 and 23, N 14336 41 and 33;
    // 16 tokens 32 and 28, 77 and 36; 8 tokens, N 500, K 11007 44 and 70.  Tiles of
    // 64 and 128 rows: 512 tokens, K 4095, N 4096 32 and 45, N 14336 123 and 95; 4096
    // tokens, N 4096 246 and 164.
    if (a.M <= 16 && narrow) return any<BF16>(a, whole, s);
    const int64_t small = ((int64_t)a.M + 63) / 64 * (((int64_t)a.N + 63) / 64);
    return small <= 3 * a.cus ? loosely<BF16, 64, 64, 2, 2>(a, whole, s) : loosely<BF16, 128, 128, 2, 4>(a, whole, s);
  }
  // Up to 64 tokens: one strip of 16 weight rows to a compute unit while there are
  // no more, else wider strips (us with strips of 16 rows and wider ones, K 4096:
  // 1 token, N 4096 6.0 and 6.4, N 14336 17.3 and 15.3; 32 tokens, N 4096 6.9 and
  // 11.4, N 14336 24.5 and 18.5; 64 tokens, N 4096 9.8 and 15.3, N 14336 36 and 20.7).
  if (a.M <= 16) return narrow ? strips<BF16, 1, 1, 2, 16>(a, whole, s) : strips<BF16, 1, 2, 2, 12>(a, whole, s);
  if (a.M <= 32) return narrow ? strips<BF16, 2, 1, 2, 12>(a, whole, s) : strips<BF16, 2, 4, 3, 4>(a, whole, s);
  if (a.M <= 64) return narrow ? strips<BF16, 4, 1, 2, 6>(a, whole, s) : strips<BF16, 4, 4, 2, 4>(a, whole, s);
  // More: the tile with the least time by the rounds of workgroups that it takes.
  // `us` is what a round of 256 took with K 4096 beyond a launch.
  struct Tile {
    int bm, bn;
    float us;
  };
  constexpr Tile kTiles[] = {{64, 32, 6.5f}, {64, 64, 10.f}, {64, 128, 14.f}, {128, 128, 24.f}, {128, 256, 39.5f}, {256, 256, 70.f}};
  int best = 0;
  float least = INFINITY;
  for (int i = 0; i < 6; ++i) {
    const int64_t all = ((int64_t)a.M + kTiles[i].bm - 1) / kTiles[i].bm * (((int64_t)a.N + kTiles[i].bn - 1) / kTiles[i].bn);
    const float us = (float)((all + a.cus - 1) / a.cus) * kTiles[i].us;
    if (us <= least && (i < 5 || multiple(16)) && (i > 0 || a.M <= 64 * 65535)) best = i, least = us;
  }
  switch (best) {
    case 0: return strips<BF16, 4, 2, 2, 6>(a, whole, s);
    case 1: return tiles<BF16, 64, 64, 2, 2, 4>(a, whole, s);
    case 2: return tiles<BF16, 64, 128, 2, 2, 3>(a, whole, s);
    case 3: return tiles<BF16, 128, 128, 2, 4, 4>(a, whole, s);
    case 4: return tiles<BF16, 128, 256, 2, 4, 3>(a, whole, s);
    default: return turns<BF16, 256>(a, whole, s);
  }
}

}  // namespace

hipError_t launch_f8(const F8Args& a, hipStream_t s) { return a.bf16 ? pick<true>(a, s) : pick<false>(a, s); }

}  // namespace mid
