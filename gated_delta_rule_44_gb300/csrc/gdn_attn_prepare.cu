// gdn_attn_prepare.cu -- the step before full attention: per-head RMS norm of
// q and k, rotary positions, and the new k and v rows into the paged cache, in
// one pass over the projection rows.
//
// Per token t (sequence s, position p) and head, over the head's D values:
//   x^ = x / sqrt(mean_d x_d^2 + eps) * w_d                 (when w is given)
//   (y_j, y_{j+R/2}) = (x^_j c_j - x^_{j+R/2} s_j, x^_{j+R/2} c_j + x^_j s_j)
// for j < R/2 with (c, s) the table row [cos | sin] of the rotary position;
// the other dims are copied.  q goes to q_out; k to k_out and / or the cache
// row p % page of page table[s, p / page]; v to the cache.  All arithmetic in
// f32, one rounding at the store.
//
// HBM-bound: every row is read and written once.  D / 8 lanes own one token and
// 8 dims each: of the rotated ones 4 and their 4 partners R / 2 further on, so that
// a rotation stays inside a lane; of the others 8 in a row.  The table row and the
// norm weights stay in registers while the lanes walk a range of the token's
// heads.  What binds before HBM is the number of instructions of a row: with
// partners fetched by shuffles and addresses multiplied out per head, 222 of them
// took 44 us where HBM takes 25 (four 2048-token prompts of 16 + 2 + 2 heads of
// 256); now about 100 take 37, 67 % of the copy rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_attn_prepare.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

using namespace attn_prepare;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 4) attn_prepare_kernel(
    const __grid_constant__ AttnPrepareLaunch p, int heads, int heads_per_group, int token_ctas) {
  prepare_rows<T, D>(p, heads, heads_per_group, token_ctas, (int)blockIdx.x, (int)blockIdx.y);
}

template <typename T, int D>
cudaError_t launch(const AttnPrepareLaunch& p, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / 8);
  // Without a cache the v heads have nowhere to go.
  const int used = p.Hq + (p.table ? 2 : 1) * p.Hkv;
  const unsigned gx = (unsigned)((p.T + GROUPS - 1) / GROUPS);
  // Heads per group: all of them once that leaves two CTAs per SM, fewer before:
  // what a group does before its first head (sequence, position, table rows) is a
  // chain of loads and as many instructions as four heads.  (Four 2048-token
  // prompts: 39, 42, 47 and 50 us with 20, 10, 5 and 4 heads; 512 single tokens
  // of 40 heads: 13, 12, 13 and 15 us with 8, 4, 2 and 1; the rule takes 20 and 3.)
  int per = used;
  while (per > 1 && (int64_t)gx * ((used + per - 1) / per) < 2 * 152) per = (per + 1) / 2;
  const unsigned checks = p.cu == nullptr ? 0 : (unsigned)((p.N + kCheckSeqs - 1) / kCheckSeqs);
  const dim3 grid(gx + checks, (unsigned)((used + per - 1) / per));
  attn_prepare_kernel<T, D><<<grid, kThreads, 0, st>>>(p, used, per, (int)gx);
  note_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_dim(const AttnPrepareLaunch& p, cudaStream_t st) {
  switch (p.D) {
    case 32: return launch<T, 32>(p, st);
    case 64: return launch<T, 64>(p, st);
    case 128: return launch<T, 128>(p, st);
    default: return launch<T, 256>(p, st);
  }
}

}  // namespace

cudaError_t launch_attn_prepare(const AttnPrepareLaunch& p, cudaStream_t st) {
  return p.bf16 ? by_dim<__nv_bfloat16>(p, st) : by_dim<float>(p, st);
}

}  // namespace gdn
