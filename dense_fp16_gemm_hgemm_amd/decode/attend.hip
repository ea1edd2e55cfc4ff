// Attention over the paged 8-bit cache.  One wave to a query and head: lanes
// take positions for the logits and channels for the sum, with the running
// maximum m and sum l of a softmax:
//   m' = max(m, logits),  l' = l e^{m-m'} + sum e^{logit-m'},  o' = o e^{m-m'} + sum e^{logit-m'} v.
#include "device.hpp"

namespace mid {
namespace {

template <int CODE, bool BF16>
__global__ __launch_bounds__(64) void attend_kernel(AttendArgs p) {
  const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x;
  const Span sp = span_of(p.batch, b);
  const int i = blockIdx.x;
  if (i >= sp.n) return;
  const int H = p.cache.kv_heads, D = p.cache.head_dim, ps = p.cache.page_size, kh = h / (p.q_heads / H);
  const int64_t cap = (int64_t)p.batch.table_cols * ps;
  const int len = (int)min((int64_t)max(p.batch.lens[b], 0), cap);
  const int pos = len - sp.n + i;
  __shared__ float qs[256];
  const uint16_t* q = static_cast<const uint16_t*>(p.q.data) + (sp.first + i) * p.q.token_stride + h * p.q.head_stride;
  for (int d = lane; d < D; d += 64) qs[d] = from16<BF16>(q[d]) * p.scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[4] = {};
  for (int j0 = 0; j0 <= pos; j0 += 64) {
    const int j = j0 + lane;
    const bool seen = j <= pos && (p.window == 0 || j > pos - p.window || j < p.sinks);
    const int page = seen ? page_of(p.cache, p.batch, b, j / ps) : -1;
    const int64_t ph = (int64_t)page * H + kh, off = (ph * ps + j % ps) * D;
    float logit = -INFINITY, vs = 0.f;
    if (page >= 0) {
      const uint8_t* k = static_cast<const uint8_t*>(p.cache.k) + off;
      float dot = 0.f;
      for (int d = 0; d < D; ++d) dot += qs[d] * from_code<CODE>(k[d]);
      logit = dot * p.cache.k_scale[ph];
      vs = p.cache.v_scale[ph];
    }
    float top = logit;
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const bool any = __any(page >= 0);
    if (!any) continue;
    const float m1 = fmaxf(m, top);
    const float keep = m == -INFINITY ? 0.f : expf(m - m1);
    const float w = page >= 0 ? expf(logit - m1) : 0.f;
    float sum = w;
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    l = l * keep + sum;
    for (int e = 0; e < D / 64; ++e) o[e] *= keep;
    for (int t = 0; t < 64; ++t) {
      const int pg = __shfl(page, t);
      if (pg < 0) continue;
      const float wt = __shfl(w, t) * __shfl(vs, t);
      const uint8_t* v = static_cast<const uint8_t*>(p.cache.v) + (((int64_t)pg * H + kh) * ps + (j0 + t) % ps) * D;
      for (int e = 0; e < D / 64; ++e) o[e] += wt * from_code<CODE>(v[lane + 64 * e]);
    }
    m = m1;
  }
  uint16_t* out = static_cast<uint16_t*>(p.out.data) + (sp.first + i) * p.out.token_stride + h * p.out.head_stride;
  for (int e = 0; e < D / 64; ++e) out[lane + 64 * e] = to16<BF16>(l == 0.f ? 0.f : o[e] / l);
}

}  // namespace

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
  const dim3 grid(a.batch.max_tokens, a.q_heads, a.batch.batch);
  if (a.cache.code == MI_DECODE_INT8) {
    if (a.bf16) attend_kernel<MI_DECODE_INT8, true><<<grid, 64, 0, s>>>(a);
    else attend_kernel<MI_DECODE_INT8, false><<<grid, 64, 0, s>>>(a);
  } else {
    if (a.bf16) attend_kernel<MI_DECODE_E4M3, true><<<grid, 64, 0, s>>>(a);
    else attend_kernel<MI_DECODE_E4M3, false><<<grid, 64, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace mid
