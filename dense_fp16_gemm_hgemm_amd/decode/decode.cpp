// The C ABI of libmi_decode: argument checks, the handle and its workspace.
#include <cstring>
#include <mutex>
#include <new>

#include "internal.h"

using namespace mid;

namespace {
constexpr const char* kArch = "gfx950";

struct DeviceGuard {
  int old = -1;
  bool switched = false;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&old) == hipSuccess && old != dev) switched = hipSetDevice(dev) == hipSuccess;
  }
  ~DeviceGuard() {
    if (switched) (void)hipSetDevice(old);
  }
};

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is16(int dtype) { return dtype == MI_DECODE_F16 || dtype == MI_DECODE_BF16; }

constexpr int64_t kFar = int64_t(1) << 30;  // rows' distances: 2^31 of them stay within 64 bits

struct Extent {
  uintptr_t lo, hi;  // bytes [lo, hi)
};
Extent extent(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, p && bytes > 0 ? a + (uintptr_t)bytes : a};
}
bool overlap(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

// [tokens][heads][D] rows: bytes from the first to past the last element.
Extent extent(const mi_decode_rows_t& r, int64_t tokens, int64_t heads, int64_t D) {
  return extent(r.data, 2 * ((tokens - 1) * r.token_stride + (heads - 1) * r.head_stride + D));
}

// Whether an element of a is one of b: [tokens][heads][D] rows of either.
// Fused projections put both into one buffer, a token's heads side by side.
bool meet(const mi_decode_rows_t& a, int64_t heads_a, const mi_decode_rows_t& b, int64_t heads_b, int64_t tokens,
          int64_t D) {
  if (!overlap(extent(a, tokens, heads_a, D), extent(b, tokens, heads_b, D))) return false;
  if (tokens > 1 && (a.token_stride != b.token_stride || a.token_stride == 0)) return true;  // no fused layout
  const int64_t S = a.token_stride, delta = ((intptr_t)b.data - (intptr_t)a.data) / 2;
  // [0, la) of a token, and [off, off + lb) of the same one or another
  auto touch = [&](int64_t la, int64_t off, int64_t lb) {
    if (tokens == 1) return off < la && off + lb > 0;
    const int64_t r = ((off % S) + S) % S;
    return r < la || r + lb > S;
  };
  if (!touch((heads_a - 1) * a.head_stride + D, delta, (heads_b - 1) * b.head_stride + D)) return false;
  for (int64_t i = 0; i < heads_a; ++i)
    for (int64_t j = 0; j < heads_b; ++j)
      if (touch(D, delta + j * b.head_stride - i * a.head_stride, D)) return true;
  return false;
}
}  // namespace

struct mi_decode_ctx {
  int device = -1;
  int cus = 0;
  bool no_device = false;
  float* ws = nullptr;
  int* cnt = nullptr;  // counters, then the list of joins
  int last_hip_error = 0;
  std::mutex mu;  // guards last_hip_error
};

namespace {
mi_decode_status_t done(mi_decode_ctx* h, hipError_t e) {
  if (e == hipSuccess) return MI_DECODE_OK;
  if (e == hipErrorInvalidConfiguration) return MI_DECODE_ERR_UNSUPPORTED;  // more workgroups than a launch can have
  std::lock_guard<std::mutex> lk(h->mu);
  h->last_hip_error = (int)e;
  return MI_DECODE_ERR_HIP;
}

mi_decode_status_t check_cache(const mi_decode_cache_t* c) {
  if (!c) return MI_DECODE_ERR_INVALID_ARG;
  if (c->pages < 0 || c->kv_heads < 1) return MI_DECODE_ERR_INVALID_ARG;
  if (c->code != MI_DECODE_INT8 && c->code != MI_DECODE_E4M3) return MI_DECODE_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MI_DECODE_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 &&
      c->page_size != 256)
    return MI_DECODE_ERR_UNSUPPORTED;
  if (c->kv_heads > 65535 || c->pages > INT32_MAX) return MI_DECODE_ERR_UNSUPPORTED;
  if (c->pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return MI_DECODE_ERR_UNSUPPORTED;
  return MI_DECODE_OK;
}

mi_decode_status_t check_batch(const mi_decode_cache_t* c, const mi_decode_batch_t* t) {
  if (!t || t->batch < 0 || t->tokens < 0 || t->max_tokens < 0 || t->table_cols < 0)
    return MI_DECODE_ERR_INVALID_ARG;
  if (t->batch == 0 || t->tokens == 0) return MI_DECODE_OK;
  if (!t->lens || (t->table_cols > 0 && !t->table) || t->table_stride < t->table_cols || t->max_tokens < 1)
    return MI_DECODE_ERR_INVALID_ARG;
  if (!t->cu && (t->tokens != t->batch || t->max_tokens != 1)) return MI_DECODE_ERR_INVALID_ARG;
  if ((int64_t)t->table_cols * c->page_size > (int64_t(1) << 30)) return MI_DECODE_ERR_UNSUPPORTED;
  return MI_DECODE_OK;
}

// Rows are read and written 16 bytes at a time.
mi_decode_status_t check_rows(const mi_decode_rows_t* r, int64_t heads, int64_t D) {
  if (!r || !r->data || r->token_stride < 0 || r->head_stride < 0) return MI_DECODE_ERR_INVALID_ARG;
  if (heads > 1 && r->head_stride < D) return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(r->data, 16) || r->token_stride % 8 || r->head_stride % 8) return MI_DECODE_ERR_UNSUPPORTED;
  return MI_DECODE_OK;
}
}  // namespace

#define TRY(x)                                       \
  do {                                               \
    const mi_decode_status_t st_ = (x);              \
    if (st_ != MI_DECODE_OK) return st_;             \
  } while (0)

// Both forms of attention; seen is nullptr for the one in order.
static mi_decode_status_t attend(mi_decode_handle_t h, const mi_decode_cache_t* cache, mi_decode_dtype_t dtype,
                                 const mi_decode_batch_t* batch, int64_t max_len, int32_t q_heads,
                                 const mi_decode_rows_t* q, const mi_decode_rows_t* out, const int32_t* seen,
                                 int64_t seen_stride, int32_t seen_words, float scale, int32_t window,
                                 int32_t sinks, void* stream) {
  if (!h) return MI_DECODE_ERR_INVALID_ARG;
  TRY(check_cache(cache));
  TRY(check_batch(cache, batch));
  if (!is16(dtype)) return MI_DECODE_ERR_UNSUPPORTED;
  if (max_len < 0 || q_heads < 1 || window < 0 || sinks < 0 || !(scale == scale) || scale - scale != 0.f)
    return MI_DECODE_ERR_INVALID_ARG;
  if (q_heads % cache->kv_heads) return MI_DECODE_ERR_INVALID_ARG;
  if ((int64_t)q_heads / cache->kv_heads * (batch->max_tokens > 0 ? batch->max_tokens : 1) > (1 << 24))
    return MI_DECODE_ERR_UNSUPPORTED;
  if (batch->batch == 0 || batch->tokens == 0) return MI_DECODE_OK;
  // a sequence's heads on the line of work are counted in 32 bits
  if (((int64_t)batch->table_cols * cache->page_size / 32 + 32) * cache->kv_heads > INT32_MAX)
    return MI_DECODE_ERR_UNSUPPORTED;
  TRY(check_rows(q, q_heads, cache->head_dim));
  TRY(check_rows(out, q_heads, cache->head_dim));
  if (batch->tokens > 1 && out->token_stride < cache->head_dim) return MI_DECODE_ERR_INVALID_ARG;
  if (overlap(extent(*out, batch->tokens, q_heads, cache->head_dim),
              extent(*q, batch->tokens, q_heads, cache->head_dim)))
    return MI_DECODE_ERR_INVALID_ARG;
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  AttendArgs a = {};
  a.cache = *cache;
  a.batch = *batch;
  a.bf16 = dtype == MI_DECODE_BF16;
  a.q = *q;
  a.out = *out;
  a.max_len = max_len;
  a.q_heads = q_heads;
  // positions are below 2^30: a longer window hides nothing, and the kernels'
  // differences of positions and these stay within 32 bits
  a.window = window < (1 << 30) ? window : 0;
  a.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
  a.scale = scale;
  a.seen = seen;
  a.seen_stride = seen_stride;
  a.seen_words = seen_words;
  a.ws = h->ws;
  a.cnt = h->cnt;
  a.join = reinterpret_cast<JoinItem*>(h->cnt + kCounters);
  a.cus = h->cus;
  DeviceGuard g(h->device);
  return done(h, launch_attend(a, (hipStream_t)stream));
}

extern "C" {

mi_decode_status_t mi_decode_create(mi_decode_handle_t* out, uint32_t flags) {
  if (!out) return MI_DECODE_ERR_INVALID_ARG;
  *out = nullptr;
  mi_decode_ctx* h = new (std::nothrow) mi_decode_ctx();
  if (!h) return MI_DECODE_ERR_HIP;
  if (flags & MI_DECODE_CREATE_NO_DEVICE) {
    h->no_device = true;
    *out = h;
    return MI_DECODE_OK;
  }
  int count = 0;
  hipDeviceProp_t prop;
  if (hipGetDeviceCount(&count) != hipSuccess || count < 1 || hipGetDevice(&h->device) != hipSuccess ||
      hipGetDeviceProperties(&prop, h->device) != hipSuccess ||
      std::strncmp(prop.gcnArchName, kArch, std::strlen(kArch)) != 0) {
    (void)hipGetLastError();
    delete h;
    return MI_DECODE_ERR_NO_DEVICE;
  }
  void* ws = nullptr;
  void* cnt = nullptr;
  if (hipMalloc(&ws, MI_DECODE_WORKSPACE_BYTES) != hipSuccess ||
      hipMalloc(&cnt, kCounters * sizeof(int) + kJoins * sizeof(JoinItem)) != hipSuccess ||
      hipMemset(cnt, 0, kCounters * sizeof(int)) != hipSuccess || hipDeviceSynchronize() != hipSuccess) {
    if (ws) (void)hipFree(ws);
    if (cnt) (void)hipFree(cnt);
    (void)hipGetLastError();
    delete h;
    return MI_DECODE_ERR_HIP;
  }
  h->cus = prop.multiProcessorCount;
  h->ws = static_cast<float*>(ws);
  h->cnt = static_cast<int*>(cnt);
  *out = h;
  return MI_DECODE_OK;
}

mi_decode_status_t mi_decode_destroy(mi_decode_handle_t h) {
  if (!h) return MI_DECODE_OK;
  if (!h->no_device) {
    DeviceGuard g(h->device);
    (void)hipFree(h->ws);
    (void)hipFree(h->cnt);
  }
  delete h;
  return MI_DECODE_OK;
}

int mi_decode_device(mi_decode_handle_t h) { return h ? h->device : -1; }

const char* mi_decode_status_string(mi_decode_status_t s) {
  switch (s) {
    case MI_DECODE_OK: return "MI_DECODE_OK";
    case MI_DECODE_ERR_INVALID_ARG: return "MI_DECODE_ERR_INVALID_ARG";
    case MI_DECODE_ERR_UNSUPPORTED: return "MI_DECODE_ERR_UNSUPPORTED";
    case MI_DECODE_ERR_NO_DEVICE: return "MI_DECODE_ERR_NO_DEVICE";
    case MI_DECODE_ERR_HIP: return "MI_DECODE_ERR_HIP";
  }
  return "unknown status";
}

int mi_decode_last_hip_error(mi_decode_handle_t h) {
  if (!h) return 0;
  std::lock_guard<std::mutex> lk(h->mu);
  return h->last_hip_error;
}

mi_decode_status_t mi_decode_w4_linear(mi_decode_handle_t h, mi_decode_dtype_t dtype, int64_t M,
                                       int64_t N, int64_t K, int64_t group, const void* x,
                                       int64_t ldx, const void* qweight, const void* scales,
                                       const void* zeros, const void* bias, void* y, int64_t ldy,
                                       void* stream) {
  if (!h || M < 0 || N < 0 || K < 0 || group < 1) return MI_DECODE_ERR_INVALID_ARG;
  if (!is16(dtype) || group % 32) return MI_DECODE_ERR_UNSUPPORTED;
  if (M > INT32_MAX || N > INT32_MAX - 15 || K > (1 << 30)) return MI_DECODE_ERR_UNSUPPORTED;
  if ((M > 1 && ldx < K) || (M > 1 && ldy < N)) return MI_DECODE_ERR_INVALID_ARG;
  if (M > 1 && ldx > (int64_t(1) << 25)) return MI_DECODE_ERR_UNSUPPORTED;  // 32 rows' bytes are counted in 32 bits
  if (M == 0 || N == 0) return MI_DECODE_OK;
  if (!y || (K > 0 && (!x || !qweight || !scales))) return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(qweight, 16) || !aligned(x, 2) || !aligned(y, 2) || !aligned(scales, 2) || !aligned(bias, 2))
    return MI_DECODE_ERR_UNSUPPORTED;
  const int64_t nb = (N + 15) / 16, kb = (K + 127) / 128, groups = (K + group - 1) / group;
  const Extent ey = extent(y, 2 * ((M - 1) * ldy + N));
  if (overlap(ey, extent(x, K > 0 ? 2 * ((M - 1) * ldx + K) : 0)) || overlap(ey, extent(qweight, nb * kb * 1024)) ||
      overlap(ey, extent(scales, groups * nb * 32)) || overlap(ey, extent(zeros, groups * nb * 16)) ||
      overlap(ey, extent(bias, 2 * N)))
    return MI_DECODE_ERR_INVALID_ARG;
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  W4Args a;
  a.x = x;
  a.qw = static_cast<const uint32_t*>(qweight);
  a.scales = scales;
  a.zeros = static_cast<const uint8_t*>(zeros);
  a.bias = bias;
  a.y = y;
  a.ldx = M > 1 ? ldx : 0;
  a.ldy = ldy;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  a.group = (int32_t)(group < INT32_MAX ? group : INT32_MAX / 32 * 32);
  a.cus = h->cus;
  a.group_inv = a.group == 32 ? UINT32_MAX : (uint32_t)((uint64_t(1) << 32) / (a.group / 32));
  a.bf16 = dtype == MI_DECODE_BF16;
  DeviceGuard g(h->device);
  return done(h, launch_w4(a, (hipStream_t)stream));
}

mi_decode_status_t mi_decode_kv_append(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                       mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                       const mi_decode_rows_t* k, const mi_decode_rows_t* v,
                                       const float* rope, int64_t rope_rows, int32_t rot_dim,
                                       int32_t interleaved, int32_t q_heads,
                                       const mi_decode_rows_t* q, const mi_decode_rows_t* q_out,
                                       void* stream) {
  return mi_decode_kv_append_at(h, cache, dtype, batch, k, v, rope, rope_rows, rot_dim, interleaved,
                                nullptr, q_heads, q, q_out, stream);
}

mi_decode_status_t mi_decode_kv_append_at(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                          mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                          const mi_decode_rows_t* k, const mi_decode_rows_t* v,
                                          const float* rope, int64_t rope_rows, int32_t rot_dim,
                                          int32_t interleaved, const int32_t* positions,
                                          int32_t q_heads, const mi_decode_rows_t* q,
                                          const mi_decode_rows_t* q_out, void* stream) {
  if (!h) return MI_DECODE_ERR_INVALID_ARG;
  TRY(check_cache(cache));
  TRY(check_batch(cache, batch));
  if (!is16(dtype)) return MI_DECODE_ERR_UNSUPPORTED;
  if (q_heads < 0 || rope_rows < 0 || rot_dim < 0) return MI_DECODE_ERR_INVALID_ARG;
  const int32_t D = cache->head_dim;
  if (rope) {
    const int64_t least = positions ? 1 : (int64_t)batch->table_cols * cache->page_size;
    if (rot_dim > D || rope_rows < least || rope_rows < 1) return MI_DECODE_ERR_INVALID_ARG;
    if (!aligned(positions, 4)) return MI_DECODE_ERR_UNSUPPORTED;
    if (rot_dim % 16 || rot_dim == 0 || !aligned(rope, 16)) return MI_DECODE_ERR_UNSUPPORTED;
  }
  if (batch->batch == 0 || batch->tokens == 0) return MI_DECODE_OK;
  TRY(check_rows(k, cache->kv_heads, D));
  TRY(check_rows(v, cache->kv_heads, D));
  AppendArgs a = {};
  if (q && q_heads > 0) {
    TRY(check_rows(q, q_heads, D));
    TRY(check_rows(q_out, q_heads, D));
    if (batch->tokens > 1 && q_out->token_stride < D) return MI_DECODE_ERR_INVALID_ARG;
    const bool same = q->data == q_out->data && q->token_stride == q_out->token_stride &&
                      q->head_stride == q_out->head_stride;
    const Extent eq = extent(*q_out, batch->tokens, q_heads, D);
    if (!same && overlap(eq, extent(*q, batch->tokens, q_heads, D))) return MI_DECODE_ERR_INVALID_ARG;
    // a q turned in place may share its rows' buffer with k and v (a fused
    // projection), but none of their elements; any other place may not
    for (const mi_decode_rows_t* x : {k, v})
      if (same ? meet(*q_out, q_heads, *x, cache->kv_heads, batch->tokens, D)
               : overlap(eq, extent(*x, batch->tokens, cache->kv_heads, D)))
        return MI_DECODE_ERR_INVALID_ARG;
    a.q = *q;
    a.q_out = *q_out;
    a.q_heads = q_heads;
  }
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  a.cache = *cache;
  a.batch = *batch;
  a.bf16 = dtype == MI_DECODE_BF16;
  a.k = *k;
  a.v = *v;
  a.rope = rope;
  a.rope_rows = rope_rows;
  a.positions = positions;
  a.rot_dim = rope ? rot_dim : 0;
  a.interleaved = interleaved != 0;
  DeviceGuard g(h->device);
  return done(h, launch_append(a, (hipStream_t)stream));
}

mi_decode_status_t mi_decode_kv_read(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                     mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                     void* k_out, void* v_out, void* stream) {
  if (!h) return MI_DECODE_ERR_INVALID_ARG;
  TRY(check_cache(cache));
  TRY(check_batch(cache, batch));
  if (!is16(dtype)) return MI_DECODE_ERR_UNSUPPORTED;
  if (batch->batch == 0 || batch->tokens == 0) return MI_DECODE_OK;
  if (!k_out || !v_out) return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return MI_DECODE_ERR_UNSUPPORTED;
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  ReadArgs a = {};
  a.cache = *cache;
  a.batch = *batch;
  a.bf16 = dtype == MI_DECODE_BF16;
  a.k_out = k_out;
  a.v_out = v_out;
  DeviceGuard g(h->device);
  return done(h, launch_read(a, (hipStream_t)stream));
}

mi_decode_status_t mi_decode_kv_attend(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                       mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                       int64_t max_len, int32_t q_heads, const mi_decode_rows_t* q,
                                       const mi_decode_rows_t* out, float scale, int32_t window,
                                       int32_t sinks, void* stream) {
  return attend(h, cache, dtype, batch, max_len, q_heads, q, out, nullptr, 0, 0, scale, window, sinks, stream);
}

mi_decode_status_t mi_decode_kv_attend_tree(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                            mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                            int64_t max_len, int32_t q_heads,
                                            const mi_decode_rows_t* q, const mi_decode_rows_t* out,
                                            const int32_t* seen, int64_t seen_stride,
                                            int32_t seen_words, float scale, int32_t window,
                                            int32_t sinks, void* stream) {
  if (!h || !batch || seen_words < 0 || seen_stride < seen_words) return MI_DECODE_ERR_INVALID_ARG;
  if (batch->batch > 0 && batch->tokens > 0) {
    if (!seen || (int64_t)seen_words * 32 < batch->max_tokens) return MI_DECODE_ERR_INVALID_ARG;
    if (!aligned(seen, 4)) return MI_DECODE_ERR_UNSUPPORTED;
  }
  return attend(h, cache, dtype, batch, max_len, q_heads, q, out, seen, seen_stride, seen_words, scale, window,
                sinks, stream);
}

mi_decode_status_t mi_decode_kv_keep(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                     const mi_decode_batch_t* batch, const int32_t* keep,
                                     void* stream) {
  if (!h) return MI_DECODE_ERR_INVALID_ARG;
  TRY(check_cache(cache));
  TRY(check_batch(cache, batch));
  if (batch->batch == 0 || batch->tokens == 0) return MI_DECODE_OK;
  if (!keep) return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(keep, 4)) return MI_DECODE_ERR_UNSUPPORTED;
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  KeepArgs a = {};
  a.cache = *cache;
  a.batch = *batch;
  a.keep = keep;
  DeviceGuard g(h->device);
  return done(h, launch_keep(a, (hipStream_t)stream));
}

mi_decode_status_t mi_decode_kv_copy(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                     const int32_t* src, const int32_t* dst, int64_t pairs,
                                     void* stream) {
  if (!h || pairs < 0) return MI_DECODE_ERR_INVALID_ARG;
  TRY(check_cache(cache));
  if (pairs == 0 || cache->pages == 0) return MI_DECODE_OK;
  if (!src || !dst) return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return MI_DECODE_ERR_UNSUPPORTED;
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  CopyArgs a = {*cache, src, dst, pairs};
  DeviceGuard g(h->device);
  return done(h, launch_copy(a, (hipStream_t)stream));
}

mi_decode_status_t mi_decode_rms_norm_f8(mi_decode_handle_t h, mi_decode_dtype_t dtype, int64_t M,
                                         int64_t K, const void* x, int64_t ldx,
                                         const void* residual, int64_t ldr, const void* weight,
                                         float eps, void* codes, int64_t ldc, float* scales,
                                         int64_t lds, void* total, int64_t ldt, void* stream) {
  if (!h || M < 0 || K < 0 || !(eps >= 0.f) || eps - eps != 0.f) return MI_DECODE_ERR_INVALID_ARG;
  if (!is16(dtype) || M > INT32_MAX || K > (1 << 30)) return MI_DECODE_ERR_UNSUPPORTED;
  for (const int64_t ld : {ldx, ldr, ldc, lds, ldt})
    if (ld > kFar) return MI_DECODE_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) return MI_DECODE_OK;
  const int64_t blocks = (K + 127) / 128;
  if (!x || !codes || !scales || (total && !residual)) return MI_DECODE_ERR_INVALID_ARG;
  if (M > 1 && (ldx < K || ldc < K || lds < blocks || (residual && ldr < K) || (total && ldt < K)))
    return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(total, 2) || !aligned(scales, 4))
    return MI_DECODE_ERR_UNSUPPORTED;
  auto rows = [&](const void* p, int64_t ld, int64_t n, int64_t size) { return extent(p, size * ((M - 1) * ld + n)); };
  const Extent in[3] = {rows(x, ldx, K, 2), rows(residual, ldr, K, 2), extent(weight, 2 * K)};
  const Extent out[3] = {rows(codes, ldc, K, 1), rows(scales, lds, blocks, 4), rows(total, ldt, K, 2)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MI_DECODE_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j) {
      // a row is read before its total is written, element by element
      const bool same = i == 2 && ((j == 0 && total == x && (M == 1 || ldt == ldx)) ||
                                   (j == 1 && total == residual && (M == 1 || ldt == ldr)));
      if (!same && overlap(out[i], in[j])) return MI_DECODE_ERR_INVALID_ARG;
    }
  }
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.total = total;
  a.ldx = M > 1 ? ldx : 0;
  a.ldr = M > 1 ? ldr : 0;
  a.ldc = M > 1 ? ldc : 0;
  a.lds = M > 1 ? lds : 0;
  a.ldt = M > 1 ? ldt : 0;
  a.M = M;
  a.K = (int32_t)K;
  a.eps = eps;
  a.bf16 = dtype == MI_DECODE_BF16;
  DeviceGuard g(h->device);
  return done(h, launch_norm(a, (hipStream_t)stream));
}

mi_decode_status_t mi_decode_f8_linear(mi_decode_handle_t h, mi_decode_dtype_t dtype, int64_t M,
                                       int64_t N, int64_t K, const void* x, int64_t ldx,
                                       const float* xs, int64_t ldxs, const void* w, int64_t ldw,
                                       const float* ws, int64_t ldws, const void* bias, void* y,
                                       int64_t ldy, void* stream) {
  if (!h || M < 0 || N < 0 || K < 0) return MI_DECODE_ERR_INVALID_ARG;
  // row numbers of whole tiles fit in 32 bits
  if (!is16(dtype) || M > INT32_MAX - 255 || N > INT32_MAX - 255 || K > (1 << 30)) return MI_DECODE_ERR_UNSUPPORTED;
  for (const int64_t ld : {ldx, ldxs, ldw, ldws, ldy})
    if (ld > kFar) return MI_DECODE_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MI_DECODE_OK;
  const int64_t kb = (K + 127) / 128, nb = (N + 127) / 128;
  if (!y || (K > 0 && (!x || !xs || !w || !ws))) return MI_DECODE_ERR_INVALID_ARG;
  if ((M > 1 && (ldx < K || ldxs < kb || ldy < N)) || (N > 1 && ldw < K) || (nb > 1 && ldws < kb))
    return MI_DECODE_ERR_INVALID_ARG;
  if (!aligned(xs, 4) || !aligned(ws, 4) || !aligned(bias, 2) || !aligned(y, 2)) return MI_DECODE_ERR_UNSUPPORTED;
  const Extent ey = extent(y, 2 * ((M - 1) * ldy + N));
  if (K > 0 && (overlap(ey, extent(x, (M - 1) * ldx + K)) || overlap(ey, extent(w, (N - 1) * ldw + K)) ||
                overlap(ey, extent(xs, 4 * ((M - 1) * ldxs + kb))) || overlap(ey, extent(ws, 4 * ((nb - 1) * ldws + kb)))))
    return MI_DECODE_ERR_INVALID_ARG;
  if (overlap(ey, extent(bias, 2 * N))) return MI_DECODE_ERR_INVALID_ARG;
  if (h->no_device) return MI_DECODE_ERR_NO_DEVICE;
  F8Args a = {};
  a.x = static_cast<const uint8_t*>(x);
  a.w = static_cast<const uint8_t*>(w);
  a.xs = xs;
  a.ws = ws;
  a.bias = bias;
  a.y = y;
  a.ldx = M > 1 ? ldx : 0;
  a.ldxs = M > 1 ? ldxs : 0;
  a.ldw = N > 1 ? ldw : 0;
  a.ldws = nb > 1 ? ldws : 0;
  a.ldy = M > 1 ? ldy : 0;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  a.cus = h->cus;
  a.bf16 = dtype == MI_DECODE_BF16;
  DeviceGuard g(h->device);
  return done(h, launch_f8(a, (hipStream_t)stream));
}

}  // extern "C"
