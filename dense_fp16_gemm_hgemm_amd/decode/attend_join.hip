// Row blocks whose parts several workgroups left in the workspace: four rows
// to a workgroup.  One workgroup for a whole block reads parts at what one
// compute unit can load, 32 parts of 256 rows in 130 us.
#include "attend.hpp"

namespace mid {
namespace {

constexpr int kRows = 4;

template <int D>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs p, int block_rows) {
  __shared__ float smem[6 * 256];
  const JoinItem it = p.join[blockIdx.x];
  const int r0 = blockIdx.y * kRows;
  if (it.parts == 0 || r0 >= it.rows) return;
  const auto parts_at = __builtin_amdgcn_make_buffer_rsrc(p.ws, (short)0, (int)MI_DECODE_WORKSPACE_BYTES, kRsrcWord3);
  join_parts<D, 256, 8>(p, parts_at, it, block_rows, r0, min(kRows, it.rows - r0), smem);
}

}  // namespace

hipError_t launch_join(const AttendArgs& a, int items, int block_rows, hipStream_t s) {
  const int64_t rows = (int64_t)(a.q_heads / a.cache.kv_heads) * a.batch.max_tokens;
  const dim3 grid(items, (unsigned)(((rows < block_rows ? rows : block_rows) + kRows - 1) / kRows));
  switch (a.cache.head_dim) {
    case 64: return launch(join_kernel<64>, grid, 256, 0, s, a, block_rows);
    case 128: return launch(join_kernel<128>, grid, 256, 0, s, a, block_rows);
    default: return launch(join_kernel<256>, grid, 256, 0, s, a, block_rows);
  }
}

}  // namespace mid
