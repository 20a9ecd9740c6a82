// gdn_attn_simt.cu -- full attention on CUDA cores, in f32 throughout: every
// supported size, type, page size and stride.  It serves f32 activations and
// what the tensor-core kernel does not take.
//
// A CTA owns 64 rows (tokens x the query heads of one kv head, so that a key
// read once serves the whole group) and walks its keys 64 at a time with a
// running maximum m and sum l per row:
//   S = scale log2(e) Q K^T;  m' = max(m, max S);  P = 2^(S - m')
//   l = l 2^(m - m') + sum P;  O = O 2^(m - m') + P V;   out = O / l
// 256 threads hold a 4 x 4 piece of S and 4 x D/16 of O in registers; Q, K, V
// and P tiles are in shared memory.  Bound by f32 FMA issue (about 12
// shared-memory wavefronts to 64 FMAs).  With few CTAs a sequence's keys are
// cut into ranges over blockIdx.y, whose sums a second kernel joins.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

using namespace attn;

constexpr int BM = 64, BN = 64, kThreads = 256;
constexpr int kMaxSplits = 64;

template <int D>
struct Smem {
  static constexpr int kLd = D + 4;   // padded rows: float4 columns fall on distinct banks
  static constexpr int kLdP = BN + 4;
  float q[BM][kLd], k[BN][kLd], v[BN][D], p[BM][kLdP];
  float m[BM], l[BM], f[BM];
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(const __grid_constant__ AttnLaunch p,
                                                             int splits) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  constexpr int NC = D / 16;              // O columns per thread
  constexpr int VW = NC < 4 ? NC : 4;     // in vectors of VW
  constexpr int NJ = NC / VW;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int G = p.Hq / p.Hkv, TT = BM / G;
  // The longest rows first: the last tiles of a sequence see the most keys.
  const int id = (int)(gridDim.x / p.Hkv) - 1 - (int)(blockIdx.x / p.Hkv);
  const int hkv = blockIdx.x % p.Hkv;
  const SeqTile tile = find_tile(p, id, TT);
  if (tile.bad && tid == 0) atomicOr(p.status, kStatusBadSeqlens);
  if (tile.nt == 0) return;
  const int base = cu_at(p.cu, tile.s);
  const int rows = tile.nt * G;
  // Keys any row of the tile sees, and this CTA's range of them.
  const int hi = max(0, tile.pos0 + tile.nt);
  const int blocks = (hi + BN - 1) / BN;
  const int kb0 = (int)((int64_t)blocks * blockIdx.y / splits);
  const int kb1 = (int)((int64_t)blocks * (blockIdx.y + 1) / splits);
  const float c = p.scale * kLog2e;

  for (int i = tid; i < BM * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      x = load4(static_cast<const T*>(p.q.p) + (int64_t)(tile.t0 + r / G) * p.q.ts +
                (int64_t)(hkv * G + r % G) * p.q.hs + d);
    *reinterpret_cast<float4*>(&sm.q[r][d]) = x;
  }
  if (tid < BM) {
    sm.m[tid] = -INFINITY;
    sm.l[tid] = 0.0f;
  }
  float o[4][NC];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) o[i][j] = 0.0f;

  for (int kb = kb0; kb < kb1; ++kb) {
    const int j0 = kb * BN, nk = min(BN, hi - j0);
    __syncthreads();
    for (int i = tid; i < BN * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (r < nk) {
        const int64_t ko = key_offset(p, false, tile.s, base, hkv, j0 + r);
        const int64_t vo = key_offset(p, true, tile.s, base, hkv, j0 + r);
        if (ko >= 0) x = load4(static_cast<const T*>(key_base(p, false)) + ko + d);
        if (vo >= 0) y = load4(static_cast<const T*>(key_base(p, true)) + vo + d);
        if (ko < 0 && d == 0) atomicOr(p.status, kStatusBadIndex);
      }
      *reinterpret_cast<float4*>(&sm.k[r][d]) = x;
      *reinterpret_cast<float4*>(&sm.v[r][d]) = y;
    }
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&sm.q[ty * 4 + i][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
          s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
          s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
          s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
        }
    }
    // The 16 lanes of a row (half a warp) share its maximum and sum.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      const int last = tile.pos0 + r / G;  // the row's last visible key
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = (j0 + tx + 16 * j <= last) ? s[i][j] * c : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mo = sm.m[r], mn = fmaxf(mo, mx);
      const float ref = mn == -INFINITY ? 0.0f : mn;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - ref);
        sum += s[i][j];
        sm.p[r][tx + 16 * j] = s[i][j];
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      const float f = exp2f(mo - ref);
      __syncwarp();
      if (tx == 0) {
        sm.m[r] = mn;
        sm.l[r] = fmaf(sm.l[r], f, sum);
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) o[i][j] *= f;
    }
    __syncwarp();  // a warp's own 8 rows of P are all it reads below
#pragma unroll 2
    for (int j = 0; j < BN; j += 4) {
      float4 pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(&sm.p[ty * 4 + i][j]);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
          float v[VW];
          const float* vp = &sm.v[j + jj][n * 16 * VW + tx * VW];
          if constexpr (VW == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(vp);
          else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(vp);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = jj == 0 ? pr[i].x : jj == 1 ? pr[i].y : jj == 2 ? pr[i].z : pr[i].w;
#pragma unroll
            for (int e = 0; e < VW; ++e) o[i][n * VW + e] = fmaf(w, v[e], o[i][n * VW + e]);
          }
        }
      }
    }
  }

  // The rows' sums into shared memory (over Q), a warp's 8 rows by that warp.
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < NJ; ++n)
#pragma unroll
      for (int e = 0; e < VW; ++e) sm.q[ty * 4 + i][n * 16 * VW + tx * VW + e] = o[i][n * VW + e];
  __syncwarp();
  const int lane = tid & 31;
  constexpr int E = D / 32;
  for (int r = (tid >> 5) * 8; r < (tid >> 5) * 8 + 8 && r < rows; ++r) {
    const int t = tile.t0 + r / G, h = hkv * G + r % G;
    float acc[E], m = sm.m[r], l = sm.l[r];
    bool finite = isfinite(l);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      acc[e] = sm.q[r][lane * E + e];
      finite = finite && isfinite(acc[e]);
    }
    if (!__all_sync(0xffffffffu, finite))
      exact_row<T, D>(p, tile.s, base, t, h, kb0 * BN, min(kb1 * BN, tile.pos0 + r / G + 1), acc, m,
                      l);
    if (splits > 1) {
      const Partials part(p.ws, (int64_t)gridDim.x * splits, BM, D);
      const int64_t slot = ((int64_t)id * p.Hkv + hkv) * splits + blockIdx.y;
      part.put<E>(slot, r, lane, acc, m, l);
    } else {
      finish_row<T, D>(p, t, h, lane, acc, m, l);
    }
  }
}

// Joins the key ranges of a row: out = sum_z 2^(m_z - M) O_z / sum_z 2^(m_z - M) l_z.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const __grid_constant__ AttnLaunch p,
                                                             int splits, int bm, int TT) {
  const int G = p.Hq / p.Hkv;
  const int id = (int)(blockIdx.x / p.Hkv), hkv = blockIdx.x % p.Hkv;
  const SeqTile tile = find_tile(p, id, TT);
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5);
  if (r >= tile.nt * G) return;
  const Partials part(p.ws, (int64_t)gridDim.x * splits, bm, D);
  constexpr int E = D / 32;
  float acc[E] = {}, m = -INFINITY, l = 0.0f;
  const int64_t slot = ((int64_t)id * p.Hkv + hkv) * splits;
  for (int z = 0; z < splits; ++z) part.add<E>(slot + z, r, lane, acc, m, l);
  finish_row<T, D>(p, tile.t0 + r / G, hkv * G + r % G, lane, acc, m, l);
}

int pick_splits(int64_t ctas, int64_t max_kv) {
  // Twice the SMs in flight, ranges of at least 4 key blocks.
  const int64_t want = (2 * 152 + ctas - 1) / ctas, most = max_kv / (4 * BN);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, kMaxSplits}));
}

template <typename T, int D>
cudaError_t launch(const AttnLaunch& p, cudaStream_t st) {
  const int G = p.Hq / p.Hkv, TT = BM / G;
  const int64_t ctas = tile_bound(p.T, p.N, TT) * p.Hkv;
  const int64_t max_kv = p.table ? (int64_t)p.max_pages * p.page_size : 0;
  const int splits = pick_splits(ctas, max_kv);
  static const cudaError_t attr = cudaFuncSetAttribute(
      attn_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
  if (attr != cudaSuccess) return attr;
  attn_simt_kernel<T, D><<<dim3((unsigned)ctas, splits), kThreads, sizeof(Smem<D>), st>>>(p, splits);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  return launch_attn_join(p, splits, BM, TT, st);
}

template <typename T>
cudaError_t by_dim(const AttnLaunch& p, cudaStream_t st) {
  switch (p.D) {
    case 32: return launch<T, 32>(p, st);
    case 64: return launch<T, 64>(p, st);
    case 128: return launch<T, 128>(p, st);
    default: return launch<T, 256>(p, st);
  }
}

}  // namespace

size_t attn_simt_workspace_bytes(int64_t T, int64_t N, int64_t Hq, int64_t Hkv, int64_t D) {
  const int64_t ctas = tile_bound(T, N, BM / (Hq / Hkv)) * Hkv;
  const int splits = pick_splits(ctas, INT64_MAX);
  return splits > 1 ? Partials::bytes(ctas * splits, BM, D) : 0;
}

cudaError_t launch_attn_join(const AttnLaunch& p, int splits, int bm, int TT, cudaStream_t st) {
  const dim3 grid((unsigned)(tile_bound(p.T, p.N, TT) * p.Hkv), (bm + kThreads / 32 - 1) / (kThreads / 32));
  if (p.bf16) {
    if (p.D == 32) attn_join_kernel<__nv_bfloat16, 32><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
    else if (p.D == 64) attn_join_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
    else if (p.D == 128) attn_join_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
    else attn_join_kernel<__nv_bfloat16, 256><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
  } else {
    if (p.D == 32) attn_join_kernel<float, 32><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
    else if (p.D == 64) attn_join_kernel<float, 64><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
    else if (p.D == 128) attn_join_kernel<float, 128><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
    else attn_join_kernel<float, 256><<<grid, kThreads, 0, st>>>(p, splits, bm, TT);
  }
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_attn_simt(const AttnLaunch& p, cudaStream_t st) {
  return p.bf16 ? by_dim<__nv_bfloat16>(p, st) : by_dim<float>(p, st);
}

}  // namespace gdn
