// What the files of libmi_decode share: the kernels' arguments and launchers.
#pragma once

#include <hip/hip_runtime.h>

#include "mi_decode.h"

namespace mid {

struct W4Args {
  const void* x;
  const uint32_t* qw;
  const void* scales;
  const uint8_t* zeros;  // nullptr: 8 everywhere
  const void* bias;      // nullptr: none
  void* y;
  int64_t ldx, ldy;
  int32_t M, N, K, group;
  int32_t cus;         // the device's compute units
  uint32_t group_inv;  // floor(2^32 / (group / 32)), 2^32 - 1 for 32
  int32_t bf16;
};

struct KvArgs {
  mi_decode_cache_t cache;
  mi_decode_batch_t batch;
  int32_t bf16;
};

struct AppendArgs : KvArgs {
  mi_decode_rows_t k, v, q, q_out;
  const float* rope;  // nullptr: no rotation
  int64_t rope_rows;
  const int32_t* positions;  // [tokens] rows of rope, nullptr: those of the tokens' places
  int32_t rot_dim, interleaved, q_heads;
};

struct ReadArgs : KvArgs {
  void* k_out;
  void* v_out;
};

// A row block whose result lies in parts (parts 0: none): rows r0 .. r0 + rows - 1
// of the sequence whose first token is `first`, of key-value head h.
struct JoinItem {
  int32_t first, r0, rows, h, parts;
  uint32_t head, tail, step;  // bytes in the workspace: part 0, part 1, and from part to part
};

struct AttendArgs : KvArgs {
  mi_decode_rows_t q, out;
  int64_t max_len;
  int32_t q_heads, window, sinks;
  float scale;
  float* ws;  // partial results, MI_DECODE_WORKSPACE_BYTES
  int* cnt;   // arrival counters, zero between launches
  JoinItem* join;  // what a second kernel joins, or nullptr: the last workgroup does
  int cus;    // the device's compute units
  const int32_t* seen;  // drafted tokens that a token sees, nullptr: it sees all up to itself
  int64_t seen_stride;
  int32_t seen_words;
};

struct KeepArgs : KvArgs {
  const int32_t* keep;
};

struct CopyArgs {
  mi_decode_cache_t cache;
  const int32_t* src;
  const int32_t* dst;
  int64_t pairs;
};

struct NormArgs {
  const void* x;
  const void* residual;  // nullptr: none
  const void* weight;    // nullptr: 1
  uint8_t* codes;
  float* scales;
  void* total;  // nullptr: not wanted
  int64_t ldx, ldr, ldc, lds, ldt, M;
  int32_t K;
  float eps;
  int32_t bf16;
};

struct F8Args {
  const uint8_t* x;
  const uint8_t* w;
  const float* xs;
  const float* ws;
  const void* bias;  // nullptr: none
  void* y;
  int64_t ldx, ldxs, ldw, ldws, ldy;
  int32_t M, N, K;
  int32_t cus;  // the device's compute units
  int32_t bf16;
};

// Enqueues a kernel and returns its own launch's status: the runtime's last error
// may be another call's, from before.  A launch counts its threads in 32 bits.
template <typename... P, typename... A>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t shared, hipStream_t s, A... a) {
  if ((uint64_t)grid.x * block.x > UINT32_MAX) return hipErrorInvalidConfiguration;
  return [&](P... p) {
    void* args[] = {&p...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, args, shared, s);
  }(a...);
}

// Each enqueues its kernel for arguments that have been checked; none is empty.
hipError_t launch_w4(const W4Args& a, hipStream_t s);
hipError_t launch_append(const AppendArgs& a, hipStream_t s);
hipError_t launch_read(const ReadArgs& a, hipStream_t s);
hipError_t launch_attend(const AttendArgs& a, hipStream_t s);       // any number of rows
hipError_t launch_attend_tile(const AttendArgs& a, hipStream_t s);  // many rows a sequence
hipError_t launch_keep(const KeepArgs& a, hipStream_t s);
hipError_t launch_copy(const CopyArgs& a, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_f8(const F8Args& a, hipStream_t s);

// Adds the parts of `items` listed blocks of at most block_rows rows.
hipError_t launch_join(const AttendArgs& a, int items, int block_rows, hipStream_t s);

constexpr int kCounters = 1024, kJoins = 1024;  // workgroups or row blocks with parts

}  // namespace mid
