// Pages that are copied, and drafted tokens that are kept.
#include "device.hpp"

namespace mid {
namespace {

// ------------------------------------------------------------------ copy --

constexpr int kPiece = 16384;  // bytes of a page that a workgroup copies

// A workgroup copies 16 KiB of a page's keys or values, a thread's four loads
// in flight at once; the page's first one takes its scales along.
//
// Bound: bytes.  2048 pages of 8 heads x 64 tokens x 128 channels are 105 us, 5.1 TB/s
// of 537 MB of reads and writes (torch's copy of 2 GiB reaches 4.9); one page is
// 3.6 us, an empty kernel 3.3.
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
// that follows takes the ratio's error away, and the border goes to even.  A NaN
// stays one (to_code's bounds would make a number of it).
template <int CODE>
__device__ inline u32x4 rescaled(u32x4 w, double ratio) {
  u32x4 o = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    o[e / 4] |= (uint32_t)to_code<CODE>((float)(from_code<CODE>((uint8_t)(w[e / 4] >> (8 * (e % 4)))) * ratio)) << (8 * (e % 4));
  if constexpr (CODE == MI_DECODE_E4M3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t nan = (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
      o[i] |= nan * 0x7fu;
    }
  }
  return o;
}

// The largest of sixteen codes' magnitudes times by, as bits.
template <int CODE>
__device__ inline uint64_t largest(u32x4 w, double by) {
  uint64_t m = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = max(m, abs_bits(from_code<CODE>((uint8_t)(w[e / 4] >> (8 * (e % 4)))) * by));
  return m;
}

// Every load before it has brought its value when a wave passes, so that what
// other waves store behind it cannot be what is loaded.
__device__ inline void all_read() {
  __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8));  // vmcnt(0)
  __syncthreads();
}

// One workgroup moves the kept tokens of a sequence in one head of K or of V.
//
// Where all of them fit into its registers they are all read before any is
// written, and the pages' maxima lie in shared memory: one chain of dependent
// loads (lengths, index, pages, codes and scales).  Otherwise page by page in the
// order of positions: a token comes from its own place or a later one, so what a
// page reads no earlier page has written.
//
// Bound: those latencies, 4 us for one sequence and, 128 sequences of 8 heads with
// paths of a dozen tokens over pages of 16, 9.7 us (page by page, with its loads for
// each page in turn, 14.6).  Their 2048 workgroups are resident all at once (up to 64
// registers), their bytes are few, and vector instructions (binary64) issue in 42 % of
// the cycles.  In a trace of fresh caches 1, 16, 64 and 128
// sequences take 5.9, 6.8, 8.5 and 13.4 us; the 128 take 10.8 where no scale grows, and
// 12.1 where the path begins a page, so that no older rows of it are read, rescaled
// and stored behind the barrier.  Page by page 200 tokens take 23 us over pages of 64
// and 56 over pages of 16.
template <int CODE>
__global__ __launch_bounds__(256) void keep_kernel(KeepArgs p) {
  constexpr int KEEP = 2, PAGES = KEEP * 64 / 16 + 1;  // pages of 16 that KEEP rows a thread of 64 channels lie on
  __shared__ unsigned long long top[PAGES];
  const int H = p.cache.kv_heads, D = p.cache.head_dim, ps = p.cache.page_size;
  const int b = blockIdx.x / (2 * H), h = blockIdx.x % (2 * H) >> 1, is_v = blockIdx.x & 1;
  const Span sp = span_of(p.batch, b);
  const int64_t held_now = p.batch.lens[b];
  const int n = min(sp.n, p.batch.max_tokens);
  if (n <= 0) return;
  const int64_t cap = (int64_t)p.batch.table_cols * ps;
  const int64_t past = min(max(held_now, (int64_t)0), cap);
  uint8_t* codes = static_cast<uint8_t*>(is_v ? p.cache.v : p.cache.k);
  float* scales = is_v ? p.cache.v_scale : p.cache.k_scale;
  const int per = D / 16, rows = 256 / per, r0 = threadIdx.x / per, c = threadIdx.x % per;
  auto row_at = [&](int page, int slot) {
    return reinterpret_cast<u32x4*>(codes + (((int64_t)page * H + h) * ps + slot) * D) + c;
  };
  auto page_at = [&](int64_t pos) { return page_of(p.cache, p.batch, b, (int)min(pos / ps, (int64_t)p.batch.table_cols)); };
  // where token i comes from: its page, or `page` and its own slot
  struct Source {
    int page, slot;
  };
  auto source = [&](int i, int page) {
    const int k = p.keep[sp.first + i];
    const int64_t pos = past + k;
    const int from = k < i ? -1 : page_at(pos);
    return from < 0 ? Source{page, (int)((past + i) % ps)} : Source{from, (int)(pos % ps)};
  };
  // a page's new scale from the bits of the largest that comes
  struct Scale {
    double s;
    bool grows;
  };
  auto scale_of = [&](uint64_t m, float old) {
    const double mine = __builtin_bit_cast(double, m) * (1. / kQmax<CODE>);
    const bool grows = abs_bits(mine) > abs_bits(old);
    return Scale{grows ? mine : old, grows};
  };
  // the codes of a token as they are on a page of scale s
  auto changed = [&](u32x4 w, double by, double s, bool moved_in) {
    if (s == 0.) return u32x4{0, 0, 0, 0};
    const double ratio = by / s;
    return ratio != 1. && moved_in ? rescaled<CODE>(w, ratio) : w;
  };
  const int64_t upto = min(past + n, cap), start0 = past - past % ps;

  if (n <= KEEP * rows) {
    const int pages = (int)((upto - 1 - start0) / ps) + 1;
    if ((int)threadIdx.x < PAGES) top[threadIdx.x] = 0;
    u32x4 w[KEEP];
    int to[KEEP], slot[KEEP], in[KEEP];  // page and slot, which of the pages, and whether the code comes from another
    bool stays[KEEP], other[KEEP];
    float by[KEEP], old[KEEP];
    for (int k = 0; k < KEEP; ++k) to[k] = -1;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      const int i = r0 + k * rows;
      if (i >= n || past + i >= cap) continue;
      to[k] = page_at(past + i);
      if (to[k] < 0) continue;
      const Source s = source(i, to[k]);
      slot[k] = (int)((past + i) % ps), in[k] = (int)((past + i - start0) / ps);
      other[k] = s.page != to[k], stays[k] = !other[k] && s.slot == slot[k];
      w[k] = *row_at(s.page, s.slot);
      by[k] = scales[(int64_t)s.page * H + h], old[k] = scales[(int64_t)to[k] * H + h];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (to[k] >= 0 && other[k]) atomicMax(&top[in[k]], (unsigned long long)largest<CODE>(w[k], by[k]));
    // the first page's scale for the tokens before the path, and every page's to be stored
    const int mine = (int)threadIdx.x < pages ? page_at(start0 + (int64_t)threadIdx.x * ps) : -1;
    const float mine_old = mine >= 0 ? scales[(int64_t)mine * H + h] : 0.f;
    const int first = page_at(start0);
    const float first_old = first >= 0 ? scales[(int64_t)first * H + h] : 0.f;
    all_read();
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      if (to[k] < 0) continue;
      const Scale s = scale_of(top[in[k]], old[k]);
      if (s.grows || !stays[k]) *row_at(to[k], slot[k]) = changed(w[k], by[k], s.s, s.grows || other[k]);
    }
    if (mine >= 0) {
      const Scale s = scale_of(top[threadIdx.x], mine_old);
      if (s.grows) scales[(int64_t)mine * H + h] = (float)s.s;
    }
    if (first >= 0) {
      const Scale s = scale_of(top[0], first_old);
      if (s.grows)
        for (int r = r0; r < (int)(past - start0); r += rows) *row_at(first, r) = changed(*row_at(first, r), first_old, s.s, true);
    }
    return;
  }

  for (int64_t start = start0; start < upto; start += ps) {
    const int page = page_at(start);
    if (page < 0) continue;
    const int lo = (int)(max(start, past) - past), hi = (int)(min(start + ps, upto) - past);  // tokens that come here
    const float old = scales[(int64_t)page * H + h];
    __syncthreads();  // the last page's maximum has been read
    if (threadIdx.x == 0) top[0] = 0;
    __syncthreads();
    uint64_t m = 0;
    for (int i = lo + r0; i < hi; i += rows) {
      const Source s = source(i, page);
      if (s.page != page) m = max(m, largest<CODE>(*row_at(s.page, s.slot), scales[(int64_t)s.page * H + h]));
    }
    if (m) atomicMax(&top[0], (unsigned long long)m);
    __syncthreads();
    const Scale sc = scale_of(top[0], old);
    // tokens in order, `rows` at a time: all of them are read before any is written
    for (int i0 = lo; i0 < hi; i0 += rows) {
      const int i = i0 + r0;
      bool put = false;
      u32x4 w;
      if (i < hi) {
        const Source s = source(i, page);
        put = sc.grows || s.page != page || s.slot != (int)((past + i) % ps);
        if (put)
          w = changed(*row_at(s.page, s.slot), s.page == page ? old : scales[(int64_t)s.page * H + h], sc.s,
                      sc.grows || s.page != page);
      }
      all_read();
      if (put) *row_at(page, (int)((past + i) % ps)) = w;
    }
    if (sc.grows) {
      for (int r = r0; r < (int)(past + lo - start); r += rows) *row_at(page, r) = changed(*row_at(page, r), old, sc.s, true);
      if (threadIdx.x == 0) scales[(int64_t)page * H + h] = (float)sc.s;
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
