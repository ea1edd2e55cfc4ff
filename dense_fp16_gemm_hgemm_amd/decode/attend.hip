// Attention over the paged 8-bit cache, one pass over keys and values with the
// running maximum m and sum l of a softmax (base 2), a page's value scale v in
// the exponent: y = z + log2 v,
//   m' = max(m, y),  l' = l 2^{m-m'} + sum 2^{y-m'} / v,  o' = o 2^{m-m'} + sum 2^{y-m'} code.
// Weights become binary16 operands in a unit of the row's own then, whatever
// other rows see (a unit for the workgroup, the largest scale of its pages,
// lost rows that do not see that page).
//
// Rows.  The G query heads of a key-value head and a sequence's n query tokens
// are one matrix of G n rows (row r: token r / G, head r % G) against the same
// keys, cut into blocks of 16 NT rows.  An item is one row block of one
// sequence and key-value head; its work is the list of 32-token tiles that any
// of its rows sees (the sinks' tiles, then the window's).
//
// Split.  All items' tiles lie on one line, which the workgroups cut into equal
// pieces whatever the sequences' lengths are.  A piece that ends inside an item
// leaves (m, l, o) in the workspace, and the item's last workgroup to arrive
// adds the parts in the order of the line: the same bits every time.
//
// A wave takes every fourth tile of a piece.  Keys are the left operand (16
// tokens by 32 channels), so the product's columns are query rows and a lane
// holds four tokens' logits of one row: these, rounded to binary16, are in place
// as the right operand of the second product, whose left operand are values
// transposed with byte permutes from 8 tokens' loads.  Eleven bits of a weight
// are what an output in binary16 has, and roundings of many weights largely
// cancel (1 x 4096 tokens in binary16: 2.5e-4 from the exact result, of which
// the output's own rounding is 2.1e-4); as two numbers a weight would double
// the second product.
//
// Codes become binary16 operands in about one instruction each: e4m3 by the
// conversion instruction; int8 as the subnormal (code + 128) 2^-24, which is a
// byte in a 16-bit slot, less 128 2^-24 (packed, exact).  Leaving the offset to
// the sums instead saves that subtraction, but costs the small results of a
// sum whose large terms are zero: 128 of them take the place of its low bits.
//
// Bounds: long contexts run at the rate of a large read (32 x 131149 tokens of
// 8 heads: 1.41 ms, 6.1 TB/s), ragged ones near it (64 sequences to 16384 tokens
// 58 us, 4.4 TB/s), short ones at their latencies (1 x 4096 tokens 12.4 us).
#include "attend.hpp"

namespace mid {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;
// Bytes of parts that an item may have up to which its last workgroup adds them
// itself; beyond, a second kernel does.  us inside and beyond: 41 KB (4 x 2048
// tokens, 8 rows) 14.8 and 15.8, 82 KB (16 rows) 19.1 and 17.0, 147 KB (1 x
// 8192, 16 rows) 22.1 and 17.6.
constexpr int64_t kJoinInside = 80 << 10;
constexpr int kItem = 16;   // what starting and ending an item costs, in tiles
constexpr int kShort = 16;  // tiles of an item that is not worth cutting

// Keeps the compiler's order of a wave's accesses to its piece of shared memory, as the hardware does.
__device__ inline void wave_shared() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

template <int CODE, int D, int NT, bool TREE>
__global__ __launch_bounds__(64 * kWaves, NT * D > 384 ? 1 : 2) void attend_kernel(AttendArgs p, int blocks) {
  constexpr int ROWS = 16 * NT, KS = D / 32, DT = D / 16, VW = D / 64;  // VW: 32-bit words of a token's values in a lane
  constexpr int OS = D + 4;
  __shared__ float obuf[kWaves][16][OS];
  __shared__ float mbuf[kWaves][ROWS], lbuf[kWaves][ROWS];
  __shared__ u32x4 qbuf[NT > 1 ? NT * KS * 64 : 1];
  __shared__ int last_flag;
  // of a tree's rows, for each wave: where a window begins, and what they see of the wave's tile
  __shared__ int from_of[TREE ? kWaves : 1][64];
  __shared__ uint32_t bits_of[TREE ? kWaves : 1][64];

  const int lane = threadIdx.x & 63, tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int H = p.cache.kv_heads, G = p.q_heads / H, ps = p.cache.page_size, log_ps = __builtin_ctz((unsigned)ps);
  const int pairs = p.batch.batch * blocks;

  // the line's length, and where this workgroup's piece begins; lane i knows
  // row block `at` + i, and the wave takes its numbers from there
  int at = 0;
  Block<kTile> mine = block_of<kTile, TREE>(p, G, ROWS, blocks, lane, pairs);
  int64_t total = 0, items = 0;
  int alike = 0;       // not 0: every item has this length on the line
  uint32_t ahead = 0;  // line of the blocks up to the lane's own, for one head
  int most = 0;        // the most tiles of a block
  auto length = [&](int tiles) { return (uint32_t)(alike ? alike : tiles + kItem); };
  auto extend = [&]() {
    ahead = mine.tiles > 0 ? length(mine.tiles) : 0u;
    most = max(most, mine.tiles);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)ahead, d);
      most = max(most, __shfl_xor(most, d));
      if (lane >= d) ahead += o;
    }
    return (uint32_t)lane_value((int)ahead, 63);
  };
  while (true) {
    total += extend();
    items += __builtin_popcountll(__ballot(mine.tiles > 0));
    if (at + 64 >= pairs) break;
    at += 64;
    mine = block_of<kTile, TREE>(p, G, ROWS, blocks, at + lane, pairs);
  }
  total *= H, items *= H;
  most = __builtin_amdgcn_readfirstlane(most);
  const int64_t each = (int64_t)((double)total / (double)(int)gridDim.x) + 1;
  // Two to four tiles for a wave, so that a short line is not cut into more
  // parts than joining them is worth (1 x 4096 tokens: 32 parts 15.1 us, 16
  // parts 12.6; 1 x 8192: 32 parts 17.1, 16 parts 14.7).
  int chunk = max((int)((each + kWaves - 1) / kWaves) * kWaves, min(max(most / 16 & ~3, 8), 16));
  // Items that are short, or not much longer than a piece, are not cut: with
  // one item to a workgroup nothing is joined (us cut and whole: 64 x 256 tokens
  // 17.0 and 11.2, 16 x 512 14.6 and 10.4, 1 x 512 9.6 and 10.2).
  if (items <= (int64_t)gridDim.x && (most <= kShort || 4 * (int64_t)(most + kItem) <= 7 * each)) {
    alike = chunk = most + kItem;
    total = items * alike;
    if (at == 0) extend();
  }
  const int64_t begin = (int64_t)blockIdx.x * chunk, end = min(begin + chunk, total);
  if (p.join && tid == 0) p.join[blockIdx.x].parts = 0;
  if (begin >= end) return;
  int64_t before = 0;
  if (at > 0) {
    at = 0;
    while (true) {
      mine = block_of<kTile, TREE>(p, G, ROWS, blocks, at + lane, pairs);
      const uint32_t more = extend();
      if ((before + more) * H > begin) break;
      before += more;
      at += 64;
    }
  }
  int who = __builtin_ctzll(__ballot((before + ahead) * H > begin));  // the block's lane
  Block<kTile> blk = mine.of_lane(who);
  int h, v0;  // head, and where in the item's line the piece begins
  {
    const uint32_t len = length(blk.tiles);
    const uint32_t off = (uint32_t)(begin - (before + (uint32_t)lane_value((int)ahead, who) - len) * H);
    h = (int)(off / len);
    v0 = (int)(off % len);
  }
  int64_t left = end - begin;

  // a part: sums of ROWS x D, then m and l of each row
  constexpr uint32_t kPart = part_bytes(ROWS, D);
  const auto parts_at = __builtin_amdgcn_make_buffer_rsrc(p.ws, (short)0, (int)MI_DECODE_WORKSPACE_BYTES, kRsrcWord3);

  auto item = [&](const Block<kTile>& blk, int h, int s0, int s1) {
    const int32_t* table = p.batch.table + (int64_t)blk.b * p.batch.table_stride;

    // the block's queries: rows as columns of the right operand.  Of several
    // 16-row tiles each wave prepares one
    const int qt = NT == 1 ? 0 : wave;
    u32x4 qraw[KS];
    {
      const int r = blk.r0 + qt * 16 + c;
      const uint16_t* q = static_cast<const uint16_t*>(p.q.data) + (blk.first + r / G) * p.q.token_stride +
                          (h * G + r % G) * p.q.head_stride + 16 * g;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qraw[s] = u32x4{0, 0, 0, 0};
        if (qt * 16 + c < blk.rows) qraw[s] = *reinterpret_cast<const u32x4*>(q + 64 * (s / 2) + 8 * (s % 2));
      }
    }

    // pages and scales of the wave's next 64 tiles, one to a lane, for each half of a tile
    int pg[2];
    float ks[2], vlog[2];
    uint64_t odd, plain;  // tiles with a page whose scales are not finite, or leave a rest; with no such page and none missing
    auto pages = [&](int tile) {
      const int t = tile + kWaves * lane;
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int tok = blk.token(t) + 16 * st;
        const bool some = t < s1 && tok <= blk.phi &&
                          (p.window == 0 || tok + 15 > blk.plo - p.window || tok < p.sinks);
        pg[st] = -1;
        if (some) pg[st] = table[tok >> log_ps];
      }
#pragma unroll
      for (int st = 0; st < 2; ++st)
        if (pg[st] < 0 || (int64_t)pg[st] >= p.cache.pages) pg[st] = -1;
    };
    auto scales = [&]() {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        ks[st] = 0.f, vlog[st] = 0.f;
        if (pg[st] >= 0) {
          const int64_t at = (int64_t)pg[st] * H + h;
          ks[st] = p.cache.k_scale[at];
          vlog[st] = p.cache.v_scale[at];
        }
      }
    };
    // once the scales are there: not before the first tile is requested
    auto logarithms = [&]() {
      bool some = false;
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const ValueScale vs = value_scale(vlog[st]);
        vlog[st] = vs.log;
        some |= pg[st] >= 0 && (vs.rest != 1.f || !(fabsf(ks[st]) < INFINITY));
      }
      odd = __ballot(some);
      plain = __ballot(pg[0] >= 0 && pg[1] >= 0) & ~odd;
    };

    u32x4 kraw[2][KS / 2];
    uint32_t vraw[8][VW];
    const uint32_t koff = c * D + g * 16, voff = g * 4 * D + c * (D / 16);
    // the bytes of 16 tokens; where there is no page, readable memory that is masked later
    auto place = [&](const void* base, int i, int tile, int st) {
      const int page = lane_value(pg[st], i);
      const int64_t at = (((int64_t)page * H + h) * ps + ((blk.token(tile) + 16 * st) & (ps - 1))) * D;
      return page >= 0 ? static_cast<const uint8_t*>(base) + at : reinterpret_cast<const uint8_t*>(p.ws);
    };
    auto load_k = [&](int i, int tile) {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const uint8_t* k = place(p.cache.k, i, tile, st);
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) kraw[st][j] = *reinterpret_cast<const u32x4*>(k + koff + 64 * j);
      }
    };
    auto load_v = [&](int i, int tile) {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const uint8_t* v = place(p.cache.v, i, tile, st) + voff;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (VW == 1) vraw[4 * st + e][0] = *reinterpret_cast<const uint32_t*>(v + e * D);
          else if constexpr (VW == 2) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(v + e * D);
            vraw[4 * st + e][0] = w[0], vraw[4 * st + e][1] = w[1];
          } else {
            const u32x4 w = *reinterpret_cast<const u32x4*>(v + e * D);
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) vraw[4 * st + e][i2 % VW] = w[i2];
          }
        }
      }
    };
    int tile = s0 + wave, i = 0;
    pages(tile);
    scales();
    load_k(0, tile);
    load_v(0, tile);

    h8 qf[NT == 1 ? KS : 1];
    float fac[NT];
    int pos[NT];
    auto token_of = [&]() { return lane < blk.rows ? (blk.r0 + lane) / G : -1; };  // of the block's row `lane`
    __syncthreads();  // the last item's reads of shared memory are over
    {
      float x[KS][8], top = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint16_t v = (uint16_t)(qraw[s][e / 2] >> (16 * (e % 2)));
          x[s][e] = p.bf16 ? from16<true>(v) : from16<false>(v);
          top = fmaxf(top, fabsf(x[s][e]));
        }
      top = max16(top);
      const float down = p.bf16 ? query_unit(top) : 1.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        h8 f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (_Float16)(x[s][e] * down);
        if constexpr (NT == 1) qf[s] = f;
        else if (qt < NT) qbuf[(qt * KS + s) * 64 + lane] = __builtin_bit_cast(u32x4, f);
      }
      float f = p.scale * 1.44269504088896340736f / down;
      if (CODE == MI_DECODE_INT8) f *= 1.f / kTiny;
      if (top == INFINITY) f = NAN;  // every logit is infinite, and no softmax is left
      if constexpr (NT == 1) {
        fac[0] = f;
      } else {
        if (qt < NT && g == 0) mbuf[0][qt * 16 + c] = f;
        __syncthreads();
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (NT > 1) fac[nt] = mbuf[0][nt * 16 + c];
        pos[nt] = nt * 16 + c < blk.rows ? blk.start + (blk.r0 + nt * 16 + c) / G : -1;
      }
      if (NT > 1) __syncthreads();
    }

    if (TREE && p.window) {  // read by the lane that writes it
      const int i = token_of();
      if (i >= 0) from_of[wave][lane] = tree_row(p, blk.first, i, blk.phi + 1 - blk.start, blk.start, true).from;
    }

    float m[NT], l[NT];
    f32x4 o[NT][DT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY, l[nt] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[nt][d] = f32x4{0, 0, 0, 0};
    }

    logarithms();
    for (; tile < s1; tile += kWaves) {
      const int tok0 = blk.token(tile);
      float ks0 = lane_value(ks[0], i), ks1 = lane_value(ks[1], i);
      const float log0 = lane_value(vlog[0], i), log1 = lane_value(vlog[1], i);
      const float inv0 = inverse(log0), inv1 = inverse(log1);
      const bool is_plain = plain >> i & 1;
      int pg0 = 0, pg1 = 0;
      float rest0 = 1.f, rest1 = 1.f;
      if (!is_plain) {
        pg0 = lane_value(pg[0], i), pg1 = lane_value(pg[1], i);
        if (odd >> i & 1) {  // read once more: kept, it would take registers from all tiles
          ks0 = key_scale(ks0), ks1 = key_scale(ks1);
          if (pg0 >= 0) rest0 = value_scale(p.cache.v_scale[(int64_t)pg0 * H + h]).rest;
          if (pg1 >= 0) rest1 = value_scale(p.cache.v_scale[(int64_t)pg1 * H + h]).rest;
        }
      }
      const bool whole = is_plain && tok0 + kTile - 1 <= blk.plo &&
                         (p.window == 0 || tok0 > blk.phi - p.window || tok0 + kTile - 1 < p.sinks);
      // whether a row of tile nt sees the lane's token c: constants against
      // numbers of the tile, which otherwise stay in registers as tokens
      const int from = tok0 + 4 * g;
      // one lane finds a row's bits; kept in registers until they are used, in
      // its or in every lane, they cost spills (48 rows of 128 channels)
      if (TREE && !whole) {
        const int i = token_of();
        wave_shared();
        bits_of[wave][lane] = i < 0 ? 0u : tree_bits32(p, {blk.first + i, p.window ? from_of[wave][lane] : 0},
                                                       blk.phi + 1 - blk.start, blk.start, tok0);
        wave_shared();
      }
      auto sees = [&](int nt) { return TREE ? bits_of[wave][16 * nt + c] >> (4 * g) : 0u; };
      auto seen = [&](int c, int nt, uint32_t bits) {
        if constexpr (TREE) return (bits >> c & 1) != 0;
        const int upto = pos[nt] - from;
        return c <= upto && (p.window == 0 || c > upto - p.window || c < p.sinks - from);
      };
      const int next = tile + kWaves;
      if (++i == 64) {
        i = 0;
        pages(next);
        scales();
        logarithms();
      }

      f32x4 z[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int st = 0; st < 2; ++st)
          z[nt][st] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        h8 kf[2];
#pragma unroll
        for (int st = 0; st < 2; ++st)
          kf[st] = along<CODE>(kraw[st][s / 2][2 * (s % 2)], kraw[st][s / 2][2 * (s % 2) + 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          h8 q;
          if constexpr (NT == 1) q = qf[s];
          else q = __builtin_bit_cast(h8, qbuf[(nt * KS + s) * 64 + lane]);
#pragma unroll
          for (int st = 0; st < 2; ++st) z[nt][st] = mma(kf[st], q, z[nt][st]);
        }
        if (NT > 1) __builtin_amdgcn_sched_barrier(0);
      }
      load_k(i, next);  // past the piece's end there is no page

      h8 pf[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float f0 = fac[nt] * ks0, f1 = fac[nt] * ks1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[nt][0][e] = __builtin_fmaf(z[nt][0][e], f0, log0);
          z[nt][1][e] = __builtin_fmaf(z[nt][1][e], f1, log1);
        }
        if (!whole) {
          const uint32_t bits = sees(nt);
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((st ? pg1 : pg0) < 0 || !seen(16 * st + e, nt, bits)) z[nt][st][e] = -INFINITY;
        }
        float top = fmaxf(fmaxf(fmaxf(z[nt][0][0], z[nt][0][1]), fmaxf(z[nt][0][2], z[nt][0][3])),
                          fmaxf(fmaxf(z[nt][1][0], z[nt][1][1]), fmaxf(z[nt][1][2], z[nt][1][3])));
        // m is 12 below the largest y and moves when weights would pass 2^15
        if (__any(top > m[nt] + kMost)) {
          const float m1 = fmaxf(m[nt], max16(top) - kBelow);
          const float down = m[nt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[nt] - m1);
          m[nt] = m1;
          l[nt] *= down;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[nt][d] *= down;
        }
        const float base = m[nt] == -INFINITY ? 0.f : m[nt];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float w = __builtin_amdgcn_exp2f(z[nt][st][e] - base);
            sum += w;
            if (!whole) w = z[nt][st][e] == -INFINITY ? 0.f : w * (st ? rest1 : rest0);
            pf[nt][4 * st + e] = (_Float16)w;
          }
          l[nt] = __builtin_fmaf(sum, st ? inv1 : inv0, l[nt]);
        }
      }

      if (CODE == MI_DECODE_E4M3 && !whole) {
        // codes that no row sees may be NaN, and one that some rows see is NaN to those alone
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int tok = tok0 + 16 * (e / 4) + 4 * g + e % 4;
          const bool any = (e < 4 ? pg0 : pg1) >= 0 && tok <= blk.phi &&
                           (p.window == 0 || tok > blk.plo - p.window || tok < p.sinks);
          bool nan = false;
#pragma unroll
          for (int x = 0; x < VW; ++x) {
            if (!any) vraw[e][x] = 0;
            nan |= (((vraw[e][x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
          }
          const uint64_t bad = __ballot(nan);
          if (bad) {
            const bool mine = (bad >> (16 * g)) & 0xffff;  // the token's row has a NaN
#pragma unroll
            for (int x = 0; x < VW; ++x)
              if (mine) vraw[e][x] = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t bits = sees(nt);
              if (mine && seen(16 * (e / 4) + e % 4, nt, bits)) pf[nt][e] = (_Float16)NAN;
            }
          }
        }
      }
      // o += V^T P^T over the tile's 32 tokens
#pragma unroll
      for (int x = 0; x < VW; ++x) {
        uint32_t col[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) col[e] = CODE == MI_DECODE_INT8 ? vraw[e][x] ^ 0x80808080u : vraw[e][x];
        h8 a0, a1, a2, a3;
        across<CODE, 0>(col, a0, a1);
        across<CODE, 1>(col, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][4 * x] = mma(a0, pf[nt], o[nt][4 * x]);
          o[nt][4 * x + 1] = mma(a1, pf[nt], o[nt][4 * x + 1]);
          o[nt][4 * x + 2] = mma(a2, pf[nt], o[nt][4 * x + 2]);
          o[nt][4 * x + 3] = mma(a3, pf[nt], o[nt][4 * x + 3]);
        }
        if (NT > 1) __builtin_amdgcn_sched_barrier(0);
      }
      load_v(i, next);
    }

    auto store = [&](int rr, int d, f32x4 x, float sum) { store_row(p, blk.first, blk.r0 + rr, h, G, d, x, sum); };

    // the four waves' sums to one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float sum = sum16(l[nt]);
      if (g == 0) mbuf[wave][nt * 16 + c] = m[nt], lbuf[wave][nt * 16 + c] = sum;
    }
    const bool whole_item = s0 == 0 && s1 == blk.tiles;
    const uint32_t slot = (uint32_t)(2 * blockIdx.x + (s0 == 0)) * kPart;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt * 16 >= blk.rows) break;
      if (nt) __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int d = 0; d < DT; d += 4) {
          f32x4 x;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            x[y] = o[nt][d + y][e] * kUnit<CODE>;
          }
          *reinterpret_cast<f32x4*>(&obuf[wave][c][(4 * g + e) * DT + d]) = x;
        }
      __syncthreads();
      for (int e = tid; e < 16 * (D / 4); e += 64 * kWaves) {
        const int row = e / (D / 4), d = e % (D / 4) * 4, rr = nt * 16 + row;
        if (rr >= blk.rows) break;
        float top = mbuf[0][rr];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, mbuf[w][rr]);
        const float base = top == -INFINITY ? 0.f : top;
        f32x4 x = {0, 0, 0, 0};
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(mbuf[w][rr] - base);
          sum += f * lbuf[w][rr];
          x += f * *reinterpret_cast<const f32x4*>(&obuf[w][row][d]);
        }
        if (whole_item) {
          store(rr, d, x, sum);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), parts_at, slot + 4 * (rr * D + d), 0, kDeviceScope);
          if (d == 0)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{top, sum}), parts_at,
                                                  slot + 4 * (ROWS * D + 2 * rr), 0, kDeviceScope);
        }
      }
    }

    if (!whole_item) {
      const int earlier = (s0 + chunk - 1) / chunk, later = (blk.tiles - s1 + chunk - 1) / chunk;
      const int first = (int)blockIdx.x - earlier, parts = earlier + 1 + later;
      const JoinItem it = {blk.first, blk.r0, blk.rows, h, parts, (uint32_t)(2 * first + 1) * kPart,
                           (uint32_t)(2 * first + 2) * kPart, 2 * kPart};
      if (p.join) {
        if (s0 == 0 && tid == 0) p.join[blockIdx.x] = it;  // one item that goes on in other workgroups
      } else if (last_to_arrive(p.cnt + first, parts, &last_flag)) {
        join_parts<D, 64 * kWaves, 16>(p, parts_at, it, ROWS, 0, blk.rows, &obuf[0][0][0]);
        if (tid == 0) __hip_atomic_store(p.cnt + first, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  };

  while (true) {
    const int v1 = (int)min((int64_t)length(blk.tiles), v0 + left);
    const int s0 = max(v0 - kItem, 0), s1 = min(max(v1 - kItem, 0), blk.tiles);
    if (s1 > s0) item(blk, h, s0, s1);
    left -= v1 - v0;
    if (left <= 0) break;
    v0 = 0;
    if (++h < H) continue;
    h = 0;
    do {
      if (++who == 64) {
        who = 0, at += 64;
        mine = block_of<kTile, TREE>(p, G, ROWS, blocks, at + lane, pairs);
      }
      blk = mine.of_lane(who);
    } while (blk.tiles == 0);
  }
}

template <int CODE, int D, int NT, bool TREE>
hipError_t run_as(const AttendArgs& a, hipStream_t s) {
  constexpr int ROWS = 16 * NT;
  const int64_t rows = (int64_t)(a.q_heads / a.cache.kv_heads) * a.batch.max_tokens;
  const int64_t blocks = (rows + ROWS - 1) / ROWS;
  if (blocks * a.batch.batch > INT32_MAX) return hipErrorInvalidConfiguration;
  int grid = (NT * D > 384 ? 1 : 2) * (a.cus < 304 ? a.cus : 304);
  static_assert(sizeof(float) * ROWS * (D + 2) * 2 * 2 * 304 <= MI_DECODE_WORKSPACE_BYTES, "partial results");
  const double tiles = (double)blocks * a.batch.batch * a.cache.kv_heads * (a.max_len / kTile + 1);
  if (tiles < grid) grid = (int)tiles;
  // An item has grid / kv_heads parts at most, as a sequence's heads are alike,
  // and no part but the ends is below 8 tiles, or a sixteenth of 256.
  const int64_t reach = a.max_len / kTile + 1, cut = reach >= 256 ? 16 : 8;
  const int64_t by_grid = grid / a.cache.kv_heads + 1, by_len = reach / cut + 2;
  const int64_t part_rows = (by_grid < by_len ? by_grid : by_len) * (rows < ROWS ? rows : ROWS);
  AttendArgs b = a;
  if (part_rows * D * 4 <= kJoinInside) b.join = nullptr;
  const hipError_t e = launch(attend_kernel<CODE, D, NT, TREE>, grid, 64 * kWaves, 0, s, b, (int)blocks);
  return e != hipSuccess || !b.join ? e : launch_join(b, grid, ROWS, s);
}

template <int CODE, int D, int NT>
hipError_t run(const AttendArgs& a, hipStream_t s) {
  // Three tiles of 128 channels and a tree's bits spill 80 bytes a lane with e4m3 and 28
  // with int8, four do not.  us with three and four: e4m3, 12 drafts of 4 heads to a
  // key-value head after 1000, 4096 and 16000 tokens 20.6, 23.0, 36.0 and 21.0, 23.8, 34.0,
  // 16 such sequences after 4096 53.8 and 60.0; int8 19.4, 21.5, 34.3 and 20.5, 23.4, 33.7,
  // 48.7 and 61.0.  e4m3 takes four, as no kernel here keeps more than 64 bytes in
  // scratch memory.  (With 256 channels one tile spills 12 to 24.)
  constexpr int TREE_NT = CODE == MI_DECODE_E4M3 && D == 128 && NT == 3 ? 4 : NT;
  return a.seen ? run_as<CODE, D, TREE_NT, true>(a, s) : run_as<CODE, D, NT, false>(a, s);
}

template <int CODE, int D>
hipError_t rows_of(const AttendArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)(a.q_heads / a.cache.kv_heads) * a.batch.max_tokens;
  if (rows <= 16) return run<CODE, D, 1>(a, s);
  if constexpr (D == 256) {
    return run<CODE, D, 2>(a, s);
  } else {
    if (rows <= 32) return run<CODE, D, 2>(a, s);
    if (rows <= 48) return run<CODE, D, 3>(a, s);
    return run<CODE, D, 4>(a, s);
  }
}

template <int CODE>
hipError_t dims_of(const AttendArgs& a, hipStream_t s) {
  if (a.cache.head_dim == 64) return rows_of<CODE, 64>(a, s);
  if (a.cache.head_dim == 128) return rows_of<CODE, 128>(a, s);
  return rows_of<CODE, 256>(a, s);
}

}  // namespace

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)(a.q_heads / a.cache.kv_heads) * a.batch.max_tokens;
  // us, here and there.  32 x 8 items against 4096 tokens: 64 rows of 128 channels
  // 94 and 117, 80 rows 196 and 120; 64 rows of 64 channels 68 and 98, 80 rows 95
  // and 101, 128 rows 95 and 105 (2 x 8 items, 8192 tokens: 64 rows 28 and 23, 80
  // rows 32 and 24).  256 channels, 1 x 8 items against 8192 tokens: 128 rows 42
  // and 50, 256 rows 62 and 63, 512 rows 99 and 95; with 32 x 8 items against
  // 4096 tokens 64 rows 194 and 280, 80 rows 313 and 280, 512 rows 1397 and 1143.
  bool tile = rows > (a.cache.head_dim == 256 ? 511 : 64);
  // Trees of a batch differ in size, and rows that no sequence has cost nothing here:
  // by the rows that a sequence has on the mean.  us here and there, 32 sequences to
  // 2048 tokens: 64 channels, 128 rows each 59 and 82, 192 rows 102 and 76; 128
  // channels, 80 rows 121 and 80, up to 128 rows and 66 on the mean (to 12000 tokens)
  // 84 and 108; 256 channels, 80 rows 180 and 166, 256 rows 428 and 334, up to 256
  // rows and 116 on the mean (to 8000 tokens) 189 and 263.
  if (a.seen && rows > 64) {
    const int64_t mean = (int64_t)(a.q_heads / a.cache.kv_heads) * a.batch.tokens / a.batch.batch;
    tile = a.cache.head_dim == 64 ? mean > 150 : a.cache.head_dim == 128 ? mean > 68 : tile || 5 * mean > 3 * rows;
  }
  if (tile) return launch_attend_tile(a, s);
  return a.cache.code == MI_DECODE_INT8 ? dims_of<MI_DECODE_INT8>(a, s) : dims_of<MI_DECODE_E4M3>(a, s);
}

}  // namespace mid
