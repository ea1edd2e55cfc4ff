// Linear layer with 4-bit weights for few tokens:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] (c[n][k] - z[n][g]) + bias[n].
// One thread to an output, in binary32.
#include "device.hpp"

namespace mid {
namespace {

template <bool BF16>
__global__ __launch_bounds__(256) void w4_kernel(W4Args p) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int n = (int)(id % p.N), m = (int)(id / p.N);
  if (m >= p.M) return;
  const int kb = (p.K + 127) / 128, np = (p.N + 15) / 16 * 16;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + m * p.ldx;
  float sum = 0.f;
  for (int g = 0, k = 0; k < p.K; ++g) {
    float part = 0.f;
    const int64_t at = (int64_t)g * np + n;
    const float z = p.zeros ? p.zeros[at] : 8;
    for (const int end = (int)min((int64_t)p.K, (int64_t)k + p.group); k < end; ++k) {
      const int64_t word = ((int64_t)(n / 16) * kb + k / 128) * 256 + ((k / 8 % 4) * 16 + n % 16) * 4 + k / 32 % 4;
      const int c = p.qw[word] >> (4 * (k % 8 / 2) + 16 * (k % 2)) & 15;
      part += from16<BF16>(x[k]) * ((float)c - z);
    }
    sum += part * from16<BF16>(static_cast<const uint16_t*>(p.scales)[at]);
  }
  if (p.bias) sum += from16<BF16>(static_cast<const uint16_t*>(p.bias)[n]);
  static_cast<uint16_t*>(p.y)[m * p.ldy + n] = to16<BF16>(sum);
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.M * a.N + 255) / 256;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  if (a.bf16) w4_kernel<true><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
  else w4_kernel<false><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace mid
