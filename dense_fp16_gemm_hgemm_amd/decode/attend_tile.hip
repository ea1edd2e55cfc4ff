// Attention over the paged 8-bit cache for many query rows of one sequence and
// key-value head (pieces of prompts): the same sums as in attend.hip, but the
// codes of a 64-token stage become binary16 operands once, in shared memory,
// for all the workgroup's rows.
//
// A wave owns 32 rows; a stage is two products of 32 tokens by 32 rows and two
// of D channels by 32 rows with 32x32x16 matrix instructions.  Rows are the
// columns again, so a lane holds 16 of a stage half's logits of one row, and
// the values' tokens lie in shared memory in the order in which the weights
// leave the first product.  Stage n + 1 is converted into the other buffer
// while stage n is used (one barrier a stage); its codes were requested a stage
// earlier, and its page numbers two.  The second half of the waves converts
// first and multiplies then, so that of the two waves of a SIMD one has vector
// work while the other has matrix work.
//
// Bound: each wave's chain of products, exponentials and conversions, with two
// waves a SIMD (registers).  2 x 2048 queries of 32 heads against 8192 tokens:
// 510 to 538 us on different boards, 900 to 940 TFLOP/s; matrix pipes are busy
// 41 % of it, vector instructions issue in 61 %, and shared memory works 41 %,
// a third of that for bank conflicts (by their addresses, of the value writes).
// Products with fragments read just before use 600 us, page numbers and
// addresses per lane 567.
//
// Scales.  A page's value scale goes into the exponent here too, and the sum of
// weights takes it out again once for 8 of them.  Each wave takes the logarithms
// of a stage's four scales itself (528 us; taken once, by the wave that loads
// them, before it converts, 545 to 557).
#include "attend.hpp"

namespace mid {
namespace {

constexpr int kStage = 64;

// What a stage's buffer says of one of its four 16-token parts.
struct alignas(16) Part {
  float ks, vs;  // scales of its page, 0 where there is none
  int page;      // the page, or -1
};

// Channels of a token lie in 16-byte pieces, the first halves of all 16-channel
// groups before the second ones: a thread that converts 16 codes then writes
// into different banks than its neighbours.
template <int D>
__device__ inline int piece_channel(int piece) {
  return piece < D / 16 ? 16 * piece : 16 * (piece - D / 16) + 8;
}

// The order of N products and the reads of their left operands, AHEAD reads in front.
template <int N, int AHEAD>
__device__ inline void schedule_reads() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 0);
}

// The parts of a tree's items.  Sequences differ in length, and their drafts all
// see the whole of it, so an item (row block, sequence, head) has as many parts as
// its length asks for, of `chunk` stages at most.  A workgroup finds its part by a
// scan over the row blocks, 64 at a time; those of items in parts come first, as
// the others are the shorter ones and fill what is left (32 sequences to 12000
// tokens with up to 64 drafts: one item to a workgroup 428 us, parts for one round
// of workgroups in the items' order 137, so 112; one line that the workgroups cut
// into equal pieces 163, where the loop over a piece's items takes 20 % longer for
// each stage).
constexpr int kLeast = 4;  // stages of a part: joining it costs about two
__host__ __device__ inline int room_of(uint32_t part) { return (int)(MI_DECODE_WORKSPACE_BYTES / part); }
__device__ inline bool place_on_line(const AttendArgs& p, int G, int blocks, int block_rows, uint32_t part, Block<kStage>& blk,
                                     int& h, int& j, int& parts, int& item, int& slot) {
  const int lane = threadIdx.x & 63, H = p.cache.kv_heads, pairs = p.batch.batch * blocks, room = room_of(part);
  auto sum_up_to = [&](int x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(x, d);
      if (lane >= d) x += o;
    }
    return x;
  };
  Block<kStage> mine;
  int loaded = -1;
  auto load = [&](int at) {
    if (at != loaded) mine = block_of<kStage, true>(p, G, block_rows, blocks, at + lane, pairs);
    loaded = at;
  };
  // a block without rows has a part too: its workgroup writes that nothing is joined
  auto parts_of = [&](int at, int chunk) { return at + lane < pairs ? max(1, (mine.tiles + chunk - 1) / chunk) : 0; };
  int64_t total = 0;
  int most = 0;
  for (int at = 0; at < pairs; at += 64) {
    load(at);
    total += lane_value(sum_up_to(mine.tiles), 63);
    most = max(most, mine.tiles);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) most = max(most, __shfl_xor(most, d));
  // Whole items, parts for one round of workgroups, or for two, by how many stages
  // it takes until the last one ends; starting a part costs about three, joining four.
  const float cus = (float)p.cus, items = (float)(pairs * H), all = (float)(total * H);
  auto until = [&](float chunk, float parts) { return parts <= cus ? chunk + 3.f : (all + 3.f * parts) / cus + 0.5f * chunk; };
  auto chunk_of = [&](int want) { return min(most, max(kLeast, (int)((total * H + want - 1) / want))); };
  int chunk = most;
  float least = until((float)most, items);
  for (int rounds = 2; rounds >= 1; --rounds) {
    const int c = chunk_of(rounds * p.cus);
    const float u = until((float)c, all / (float)c + (rounds == 1 ? 0.f : items)) + 4.f;
    if (c > 0 && u < least) chunk = c, least = u;
  }
  // Of t stages, an item in parts has more than chunk and so fewer than 2 tiles / chunk
  // parts: with t / chunk at most half the room all have a place.
  int many = 0;  // parts of items in parts
  auto count = [&]() {
    many = 0;
    for (int at = 0; at < pairs; at += 64) {
      load(at);
      const int n = parts_of(at, chunk);
      many += lane_value(sum_up_to(n > 1 ? n * H : 0), 63);
    }
  };
  chunk = max(chunk, 1);
  count();
  if (many > room) {
    chunk = max(chunk_of(min(p.cus, room / 2)), 1);
    count();
  }
  const bool first = (int)blockIdx.x < many;  // of an item in parts
  int before = first ? 0 : many;
  for (int at = 0; at < pairs; at += 64) {
    load(at);
    const int n = parts_of(at, chunk), upto = sum_up_to((n > 1) == first ? n * H : 0);
    const uint64_t m = __ballot(before + upto > (int)blockIdx.x);
    if (m) {
      const int l = __builtin_ctzll(m);
      blk = mine.of_lane(l);
      parts = lane_value(n, l);
      const int off = (int)blockIdx.x - before - (lane_value(upto, l) - parts * H);
      h = off / parts, j = off % parts;
      item = (at + l) * H + h;
      slot = (int)blockIdx.x - j;
      if (blk.tiles == 0) parts = 0;
      return true;
    }
    before += lane_value(upto, 63);
  }
  return false;
}

template <int CODE, int D, int NW, bool TREE>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attend_tile_kernel(AttendArgs p, int blocks, int splits) {
  constexpr int ROWS = 32 * NW, KS = D / 16, DT = D / 32, T = 64 * NW;
  constexpr int UNITS = kStage * D / 16, UN = (UNITS + T - 1) / T;  // 16-byte units of a stage, and a thread's
  constexpr uint32_t kPart = part_bytes(ROWS, D);
  constexpr int VD = D / 4;                                         // groups of 4 channels
  __shared__ u32x4 kbuf[2][kStage * D / 8];
  __shared__ u32x4 vbuf[2][D * kStage / 8];
  __shared__ Part part_of[2][4];
  __shared__ unsigned long long nans[3];  // tokens of a stage with a NaN among their values' codes

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hi = lane >> 5;
  const int H = p.cache.kv_heads, G = p.q_heads / H, ps = p.cache.page_size;

  // Workgroups of one sequence and head are a multiple of their number apart:
  // with a multiple of 8 they share an XCD's L2.  The last rows, which see
  // most, come first.
  const int heads = p.batch.batch * H, bh = blockIdx.x % heads, rest = blockIdx.x / heads;
  int j = rest % splits, h = bh % H, parts = 1, item, slot;
  Block<kStage> blk;
  if (TREE && p.join) {
    if (!place_on_line(p, G, blocks, ROWS, kPart, blk, h, j, parts, item, slot)) return;
  } else {
    const int rb = blocks - 1 - rest / splits;
    blk = block_of<kStage, TREE>(p, G, ROWS, blocks, bh / H * blocks + rb, p.batch.batch * blocks);
    parts = blk.tiles == 0 ? 0 : min(splits, max(1, blk.tiles / 4)), item = rb * heads + bh, slot = item * splits;
  }
  if ((TREE ? p.join != nullptr : splits > 1) && j == 0 && tid == 0) {
    const uint32_t at = (uint32_t)slot * kPart;
    p.join[item] = parts > 1 ? JoinItem{blk.first, blk.r0, blk.rows, h, parts, at, at + kPart, kPart} : JoinItem{};
  }
  if (j >= parts) return;
  const int s0 = (int)((int64_t)blk.tiles * j / parts), s1 = (int)((int64_t)blk.tiles * (j + 1) / parts);
  const int32_t* table = p.batch.table + (int64_t)blk.b * p.batch.table_stride;

  // What a wave loads and converts belongs to one 16-token part for each i, so
  // pages and addresses are the same in all its lanes: units of 16 codes of a
  // token's key, and of 4 tokens by 4 channels of values.
  const bool loader = UNITS >= T || wave < UNITS / 64;
  const int log_ps = __builtin_ctz((unsigned)ps);
  const uint32_t head_bytes = (uint32_t)(ps * D);  // a page's bytes fit 32 bits: 65535 heads of 256 x 256
  const uint32_t page_bytes = (uint32_t)H * head_bytes;
  const uint32_t koff = (tid / (D / 16) & 15) * D + tid % (D / 16) * 16;
  const uint32_t voff = (tid / VD & 3) * 4 * D + tid % VD * 4;
  auto part = [&](int i) { return (64 * wave + T * i) / D; };
  int entry[UN];  // table entries, one stage ahead of the loads; -1: no row sees the part
  u32x4 kraw[UN];
  uint32_t vraw[UN][4];
  Part got[UN];
  auto entries = [&](int n) {
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int at = blk.token(n) + 16 * part(i);
      entry[i] = -1;
      if (loader && n < s1 && at <= blk.phi && (p.window == 0 || at + 15 > blk.plo - p.window || at < p.sinks))
        entry[i] = table[at >> log_ps];
    }
  };
  auto loads = [&](int n) {
    if (!loader) return;
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      int page = __builtin_amdgcn_readfirstlane(entry[i]);
      if ((int64_t)page >= p.cache.pages) page = -1;
      const int slot = (blk.token(n) + 16 * part(i)) & (ps - 1);
      const uint64_t at = (uint64_t)(uint32_t)page * page_bytes + (uint32_t)h * head_bytes + (uint32_t)(slot * D);
      // where there is no page, readable memory that is masked later
      const uint8_t* k = page >= 0 ? static_cast<const uint8_t*>(p.cache.k) + at : reinterpret_cast<const uint8_t*>(p.ws);
      const uint8_t* v = page >= 0 ? static_cast<const uint8_t*>(p.cache.v) + at : reinterpret_cast<const uint8_t*>(p.ws);
      kraw[i] = *reinterpret_cast<const u32x4*>(k + koff);
#pragma unroll
      for (int e = 0; e < 4; ++e) vraw[i][e] = *reinterpret_cast<const uint32_t*>(v + voff + e * D);
      got[i] = Part{0.f, 0.f, page};
      if (page >= 0 && (64 * wave + T * i) % D == 0) {  // the part's first wave
        got[i].ks = p.cache.k_scale[(int64_t)page * H + h];
        got[i].vs = p.cache.v_scale[(int64_t)page * H + h];
      }
    }
  };
  // codes of a stage to operands in buffer b
  auto convert = [&](int b, int n3) {
    if (!loader) return;
    bool any_nan = false;
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      if (lane == 0 && (64 * wave + T * i) % D == 0) part_of[b][part(i)] = got[i];
      const int u = tid + T * i;
      const int tok = u / (D / 16), c = u % (D / 16);
      u32x4* row = &kbuf[b][tok * (D / 8)];
      row[c ^ (tok & 7)] = __builtin_bit_cast(u32x4, along<CODE>(kraw[i][0], kraw[i][1]));
      row[(c + D / 16) ^ (tok & 7)] = __builtin_bit_cast(u32x4, along<CODE>(kraw[i][2], kraw[i][3]));
      const int tg = u / VD, d = u % VD * 4;
      if constexpr (CODE == MI_DECODE_E4M3) {
        // a NaN code's token is kept in a list and its code becomes zero: rows
        // that do not see the token would have 0 times NaN
#pragma unroll
        for (int e = 0; e < 4; ++e) any_nan |= (((vraw[i][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
        if (__any(any_nan)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t bad = ((vraw[i][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
            if (bad) {
              vraw[i][e] &= ~((bad >> 7) * 0xffu);
              atomicOr(&nans[n3], 1ull << (4 * tg + e));
            }
          }
        }
      }
      // 4 tokens of 4 channels: channel d + y's at its row's piece for the
      // tokens' group of 16, in the order that the first product leaves
      uint32_t lo[4], hi4[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if constexpr (CODE == MI_DECODE_INT8) {
          const uint32_t t0 = vraw[i][0] ^ 0x80808080u, t1 = vraw[i][1] ^ 0x80808080u;
          const uint32_t t2 = vraw[i][2] ^ 0x80808080u, t3 = vraw[i][3] ^ 0x80808080u;
          lo[y] = centred(__builtin_amdgcn_perm(t1, t0, 0x0c040c00u + 0x00010001u * y));
          hi4[y] = centred(__builtin_amdgcn_perm(t3, t2, 0x0c040c00u + 0x00010001u * y));
        }
      }
      if constexpr (CODE == MI_DECODE_E4M3) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t a = __builtin_amdgcn_perm(vraw[i][1], vraw[i][0], 0x05010400u + 0x02020202u * y);
          const uint32_t z = __builtin_amdgcn_perm(vraw[i][3], vraw[i][2], 0x05010400u + 0x02020202u * y);
          lo[2 * y] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false));
          lo[2 * y + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true));
          hi4[2 * y] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(z, 1.f, false));
          hi4[2 * y + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(z, 1.f, true));
        }
      }
      const int piece = 2 * (tg / 4) + (tg & 1), half = (tg >> 1) & 1;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int dim = d + y;
        u32x2* to = reinterpret_cast<u32x2*>(&vbuf[b][dim * (kStage / 8) + (piece ^ ((dim ^ (dim >> 3)) & 7))]) + half;
        *to = u32x2{lo[y], hi4[y]};
      }
    }
  };

  // the wave's queries: rows as columns of the right operand, with the scale's sign
  const int row = 32 * wave + col;
  const bool in = row < blk.rows;
  const int pos = in ? blk.start + (blk.r0 + row) / G : -1;
  TreeRow tree;
  if constexpr (TREE) tree = tree_row(p, blk.first, (blk.r0 + row) / G, blk.phi + 1 - blk.start, blk.start, in);
  entries(s0);
  u32x4 qraw[KS];
  {
    const int r = blk.r0 + row;
    const uint16_t* q = static_cast<const uint16_t*>(p.q.data) + (blk.first + r / G) * p.q.token_stride +
                        (h * G + r % G) * p.q.head_stride;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      qraw[s] = u32x4{0, 0, 0, 0};
      if (in) qraw[s] = *reinterpret_cast<const u32x4*>(q + piece_channel<D>(2 * s + hi));
    }
  }
  if (tid < 3) nans[tid] = 0;
  loads(s0);
  entries(s0 + 1);
  h8 qf[KS];
  float fac;
  {
    float top = 0.f;
    auto value = [&](int s, int e) {
      const uint16_t v = (uint16_t)(qraw[s][e / 2] >> (16 * (e % 2)));
      return p.bf16 ? from16<true>(v) : from16<false>(v);
    };
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(value(s, e)));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float down = p.bf16 ? query_unit(top) : 1.f;
    const float by = p.scale < 0.f ? -down : down;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      // converted anew: the compiler would keep the first pass's 8 KS floats
      asm("" : "+v"(qraw[s]));
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[s][e] = (_Float16)(value(s, e) * by);
    }
    fac = fabsf(p.scale) * 1.44269504088896340736f / down;
    if (CODE == MI_DECODE_INT8) fac *= 1.f / kTiny;
    if (top == INFINITY) fac = NAN;  // every logit is infinite, and no softmax is left
  }
  __syncthreads();
  convert(0, 0);
  loads(s0 + 1);
  entries(s0 + 2);
  __syncthreads();

  float m = -INFINITY, l = 0.f;
  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = f32x16{};

  // rows of the wave that exist, and their positions
  const int wrows = min(32, blk.rows - 32 * wave);
  const int wlo = TREE ? blk.plo : blk.start + (blk.r0 + 32 * wave) / G;
  const int whi = TREE ? blk.phi : blk.start + (blk.r0 + 32 * wave + wrows - 1) / G;
  // pieces of the operands: the key's of token `col`, the value's of channel `col`
  // for four of them; the others are whole steps away
  int kx[4], vx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    kx[i] = col * (D / 8) + ((2 * i + hi) ^ (col & 7));
    vx[i] = col * (kStage / 8) + ((2 * i + hi) ^ ((col ^ (col >> 3)) & 7));
  }

  auto rescale = [&](float down) {
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] *= down;
  };
  auto use = [&](int n, int b, int n3) {
    const int t0 = blk.token(n);
    if (wrows <= 0 || t0 > whi) return;
    if (p.window && t0 + kStage - 1 <= wlo - p.window && t0 >= p.sinks) return;
    // Lane i knows part i % 4; read before the first product's operands, used after it.
    const Part mine = part_of[b][lane & 3];
    __builtin_amdgcn_sched_barrier(0);
    const u32x4 *kb = kbuf[b], *vb = vbuf[b];
    f32x16 z[2] = {};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const u32x4 k = kb[kx[s % 4] + (x * 32 * (D / 8) + s / 4 * 8)];
        z[x] = mma(__builtin_bit_cast(h8, k), qf[s], z[x]);
      }
    // operands are read six products ahead of their use
    schedule_reads<2 * KS, 6>();
    const ValueScale vs = value_scale(mine.vs);
    const float inv = inverse(vs.log);
    // Token c after the lane's first one (constants, compared with numbers of
    // the stage: left as tokens, 32 of them would stay in registers).
    const int upto = pos - t0 - 4 * hi, after = p.window ? upto - p.window : -1, sink = p.sinks - t0 - 4 * hi;
    uint64_t sees = 0;
    auto seen = [&](int c) {
      if constexpr (TREE) return (sees >> c & 1) != 0;
      return c <= upto && (c > after || c < sink);
    };
    const int valid = __ballot(mine.page >= 0) & 15;
    const bool plain = vs.rest == 1.f && mine.ks >= 0.f && mine.ks < INFINITY;
    const bool whole = valid == 15 && __all(plain) && t0 + kStage - 1 <= wlo &&
                       (p.window == 0 || t0 > whi - p.window || t0 + kStage - 1 < p.sinks);
    if (TREE && !(whole && (CODE == MI_DECODE_INT8 || nans[n3] == 0))) sees = tree_bits64(p, tree, blk.phi + 1 - blk.start, blk.start, t0) >> (4 * hi);
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = fac * lane_value(mine.ks, i);
    float top = -INFINITY;
    if (whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float t = z[i / 2][8 * (i % 2)];
#pragma unroll
        for (int e = 1; e < 8; ++e) t = fmaxf(t, z[i / 2][8 * (i % 2) + e]);
        top = fmaxf(top, __builtin_fmaf(t, f[i], lane_value(vs.log, i)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lv = lane_value(vs.log, i), fi = key_scale(f[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool ok = (valid >> i & 1) && seen(16 * i + 8 * (e / 4) + e % 4);
          const float y = ok ? __builtin_fmaf(z[i / 2][8 * (i % 2) + e], fi, lv) : -INFINITY;
          z[i / 2][8 * (i % 2) + e] = y;
          top = fmaxf(top, y);
        }
      }
    }
    // m is 12 below the largest y and moves when weights would pass 2^15
    if (__any(top > m + kMost)) {
      const float m1 = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)) - kBelow);
      const float by = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - m1);
      m = m1;
      l *= by;
      rescale(by);
    }
    h8 pf[4];
    if (whole) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = lane_value(vs.log, i) - m;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(z[i / 2][8 * (i % 2) + e], f[i], c));
          sum += w;
          pf[i][e] = (_Float16)w;
        }
        l = __builtin_fmaf(sum, lane_value(inv, i), l);
      }
    } else {
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float iv = lane_value(inv, i), rest = lane_value(vs.rest, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = z[i / 2][8 * (i % 2) + e], w = __builtin_amdgcn_exp2f(y - base);
          l = __builtin_fmaf(w, iv, l);
          pf[i][e] = y == -INFINITY ? (_Float16)0 : (_Float16)(w * rest);
        }
      }
    }
    if (CODE == MI_DECODE_E4M3 && nans[n3]) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = 16 * i + 8 * (e / 4) + e % 4;
          if ((nans[n3] >> (4 * hi) >> at & 1) && (valid >> i & 1) && seen(at)) pf[i][e] = (_Float16)NAN;
        }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const u32x4 v = vb[vx[i ^ (2 * (d & 1))] + d * 32 * (kStage / 8)];
        o[d] = mma(__builtin_bit_cast(h8, v), pf[i], o[d]);
      }
    schedule_reads<4 * DT, 6>();
  };

  const bool first_half = wave < NW / 2;
  for (int n = s0, n3 = 0; n < s1; ++n) {
    const int b = (n - s0) & 1, next3 = n3 == 2 ? 0 : n3 + 1;
    auto stage = [&]() {
      if (n + 1 >= s1) return;
      convert(b ^ 1, next3);
      loads(n + 2);
      entries(n + 3);
    };
    if (!first_half) stage();
    use(n, b, n3);
    if (first_half) stage();
    // of three lists one is used, one is filled and one is emptied
    if (CODE == MI_DECODE_E4M3 && tid == 0) nans[next3 == 2 ? 0 : next3 + 1] = 0;
    __syncthreads();
    n3 = next3;
  }

  // o as rows: lane (col, hi) holds channels 32 d + 8 a + 4 hi + 0..3 of row col
  l += __shfl_xor(l, 32);
  constexpr float unit = kUnit<CODE>;
  if (parts == 1) {
    if (in)
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const f32x4 x = {o[d][4 * a], o[d][4 * a + 1], o[d][4 * a + 2], o[d][4 * a + 3]};
          store_row(p, blk.first, blk.r0 + row, h, G, 32 * d + 8 * a + 4 * hi, x * unit, l);
        }
    return;
  }
  const auto parts_at = __builtin_amdgcn_make_buffer_rsrc(p.ws, (short)0, (int)MI_DECODE_WORKSPACE_BYTES, kRsrcWord3);
  const uint32_t to = (uint32_t)(slot + j) * kPart;
  if (in) {
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const f32x4 x = {o[d][4 * a], o[d][4 * a + 1], o[d][4 * a + 2], o[d][4 * a + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x * unit), parts_at,
                                               to + 4 * (row * D + 32 * d + 8 * a + 4 * hi), 0, kDeviceScope);
      }
    if (hi == 0)
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{m, l}), parts_at,
                                            to + 4 * (ROWS * D + 2 * row), 0, kDeviceScope);
  }
}

template <int CODE, int D, int NW, bool TREE>
hipError_t run_as(const AttendArgs& a, hipStream_t s) {
  constexpr int ROWS = 32 * NW;
  const int64_t rows = (int64_t)(a.q_heads / a.cache.kv_heads) * a.batch.max_tokens;
  const int64_t blocks = (rows + ROWS - 1) / ROWS;
  const int64_t items = blocks * a.batch.batch * a.cache.kv_heads;
  if (items > INT32_MAX) return hipErrorInvalidConfiguration;
  // Few items: their stages are split so that every compute unit has a piece.
  int64_t splits = items < a.cus && items <= kJoins ? a.cus / items : 1;
  const int64_t stages = a.max_len / kStage + 1;
  if (splits > stages / 4) splits = stages / 4 > 0 ? stages / 4 : 1;
  if (items * splits * part_bytes(ROWS, D) > MI_DECODE_WORKSPACE_BYTES) splits = 1;
  AttendArgs b = a;
  int64_t grid = items * splits;
  if (TREE) {
    splits = 1, grid = items;
    // The list of joins has its length: beyond it an item is one workgroup's, however
    // long (128 sequences of 8 heads, one to 12000 tokens and the others to 300, with 24
    // drafts each 127 us, 129 of them 322).
    if (stages <= kLeast || items > kJoins) b.join = nullptr;
    else grid = items + 2 * a.cus;
  }
  const hipError_t e =
      launch(attend_tile_kernel<CODE, D, NW, TREE>, (unsigned)grid, 64 * NW, 0, s, b, (int)blocks, (int)splits);
  return e != hipSuccess || (TREE ? !b.join : splits == 1) ? e : launch_join(b, (int)items, ROWS, s);
}

template <int CODE, int D, int NW>
hipError_t run(const AttendArgs& a, hipStream_t s) {
  return a.seen ? run_as<CODE, D, NW, true>(a, s) : run_as<CODE, D, NW, false>(a, s);
}

// 256 channels: a row's sums, queries and logits need more registers than two
// waves of a SIMD have.
template <int CODE>
hipError_t dims_of(const AttendArgs& a, hipStream_t s) {
  if (a.cache.head_dim == 64) return run<CODE, 64, 8>(a, s);
  if (a.cache.head_dim == 128) return run<CODE, 128, 8>(a, s);
  return run<CODE, 256, 4>(a, s);
}

}  // namespace

hipError_t launch_attend_tile(const AttendArgs& a, hipStream_t s) {
  return a.cache.code == MI_DECODE_INT8 ? dims_of<MI_DECODE_INT8>(a, s) : dims_of<MI_DECODE_E4M3>(a, s);
}

}  // namespace mid
