// Conversions and cache addressing that the decode kernels share.
#pragma once

#include "internal.h"

namespace mid {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 16-bit storage to binary32 and back, to nearest even.
template <bool BF16>
__device__ inline float from16(uint16_t v) {
  if constexpr (BF16) return __builtin_bit_cast(float, uint32_t(v) << 16);
  else return (float)__builtin_bit_cast(_Float16, v);
}
template <bool BF16>
__device__ inline uint16_t to16(float x) {
  if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
  else return __builtin_bit_cast(uint16_t, (_Float16)x);
}

// A code's value.
template <int CODE>
__device__ inline float from_code(uint8_t c) {
  if constexpr (CODE == MI_DECODE_INT8) return (float)(int8_t)c;
  else return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}
// The nearest code (ties to even) of a value within +-QMAX.
template <int CODE>
__device__ inline uint8_t to_code(float x) {
  if constexpr (CODE == MI_DECODE_INT8) {
    x = fminf(fmaxf(x, -127.f), 127.f);
    return (uint8_t)(int8_t)(int)__builtin_rintf(x);
  } else {
    x = fminf(fmaxf(x, -448.f), 448.f);
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, 0.f, 0, false) & 0xff);
  }
}
template <int CODE>
constexpr float kQmax = CODE == MI_DECODE_INT8 ? 127.f : 448.f;

// Tokens [first, first + n) of sequence b, clamped to the call's tokens.
struct Span {
  int first, n;
};
__device__ inline Span span_of(const mi_decode_batch_t& t, int b) {
  if (t.cu == nullptr) return {b, b < t.tokens ? 1 : 0};
  const int lo = min(max(t.cu[b], 0), t.tokens);
  const int hi = min(max(t.cu[b + 1], lo), t.tokens);
  return {lo, hi - lo};
}

// The page of table column c of sequence b, or -1 where the entry names none.
__device__ inline int page_of(const mi_decode_cache_t& k, const mi_decode_batch_t& t, int b, int c) {
  if (c < 0 || c >= t.table_cols) return -1;
  const int p = t.table[(int64_t)b * t.table_stride + c];
  return (p >= 0 && (int64_t)p < k.pages) ? p : -1;
}

}  // namespace mid
