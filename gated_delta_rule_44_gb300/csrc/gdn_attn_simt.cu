// gdn_attn_simt.cu -- full attention on CUDA cores, in f32 throughout: every
// supported size, type, page size and stride.  It serves f32 activations and
// what the tensor-core kernel does not take.
//
// Tile kernel.  A tile is 64 rows (tokens x the query heads of one kv head, so
// that a key read once serves the whole group); its keys come 64 at a time with a
// running maximum m and sum l per row:
//   S = scale log2(e) Q K^T;  m' = max(m, max S);  P = 2^(S - m')
//   l = l 2^(m - m') + sum P;  O = O 2^(m - m') + P V;   out = O / l
// 256 threads hold a 4 x 4 piece of S and 4 x D/16 of O in registers; Q, P and one
// of K and V at a time are in shared memory, so that two CTAs fit an SM (the other is
// on its way in registers for D <= 64).  Bound by f32 FMA issue.  A cluster of
// CTAs shares a tile: each takes every so many key blocks, and the sums are joined
// through distributed shared memory, so that few or unequal tiles still fill the
// SMs.
//
// Row kernel, for a few rows per kv head (decode, drafts): a warp takes 8 keys at
// a time with the dims over its lanes, each key and value read once and straight
// from global memory; the 8 x rows partial dot products of the lanes are summed
// by one transposing butterfly.  Bound by HBM.  Key ranges over the warps of a CTA
// are joined in shared memory, over CTAs by a second kernel.
//
// Measured on GB300, f32, heads of 128: a 1024-token prompt, 8 + 2 heads, 100 us
// (21 TFLOP/s, about 28 % of the FMA rate; the shared-memory loads of the 4 x 4
// pieces and the barriers between a block's phases bind; packed two-lane FMAs
// changed nothing).  8 single tokens over up to 4097 keys: 24 us a call, of which
// the chains of loads of a few steps per warp and the join take most.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

using namespace attn;
namespace cg = cooperative_groups;

constexpr int BM = 64, BN = 64, kThreads = 256;
constexpr int kMaxCluster = 8;

template <int D>
struct Smem {
  static constexpr int kLd = D + 4;   // padded rows: float4 columns fall on distinct banks
  static constexpr int kLdP = BN + 4;
  float q[BM][kLd], kv[BN][kLd], p[BM][kLdP];
  float m[BM], l[BM];
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

template <typename T, int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, D <= 128 ? 2 : 1)
    attn_simt_kernel(const __grid_constant__ AttnLaunch p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  constexpr int NC = D / 16;              // O columns per thread
  constexpr int VW = NC < 4 ? NC : 4;     // in vectors of VW
  constexpr int NJ = NC / VW;
  constexpr int NL = BN * (D / 4) / kThreads;  // float4 of a K or V block per thread
  // The next block waits in registers where there are enough (D = 128: 536 instead
  // of 570 us without, 1536 tokens of 32 heads).
  constexpr bool kAhead = D <= 64;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int G = p.Hq / p.Hkv, TT = BM / G;
  // The longest rows first: the last tiles of a sequence see the most keys.
  const int item = blockIdx.x / ranks;
  const int id = (int)(gridDim.x / ranks / p.Hkv) - 1 - item / p.Hkv;
  const int hkv = item % p.Hkv;
  const SeqTile tile = find_tile(p, id, TT);
  if ((tid == 0 && tile.bad) || (tid == kThreads - 1 && rank == 0 && hkv == 0 && own_range_bad(p, id)))
    atomicOr(p.status, kStatusBadSeqlens);
  if (tile.nt == 0) return;  // the whole cluster
  const int base = cu_at(p.cu, tile.s);
  const int rows = tile.nt * G;
  const int hi = max(0, tile.pos0 + tile.nt);  // keys any row of the tile sees
  const int blocks = (hi + BN - 1) / BN;
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

  // This thread's vectors of block kb of K or V; rows past the last visible key
  // and bad pages are zeros.
  float4 next[kAhead ? NL : 1];
  auto fetch1 = [&](bool of_v, int kb, int n) -> float4 {
    const int i = tid + n * kThreads, r = i / (D / 4), d = i % (D / 4) * 4, j = kb * BN + r;
    if (j >= hi) return make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (PAGED) {
      const int64_t at = key_offset(p, of_v, tile.s, base, hkv, j);
      if (at < 0) {
        if (d == 0) atomicOr(p.status, kStatusBadIndex);
        return make_float4(0.f, 0.f, 0.f, 0.f);
      }
      return load4(static_cast<const T*>(key_base(p, of_v)) + at + d);
    } else {
      const AttnRows& x = of_v ? p.v : p.k;
      return load4(static_cast<const T*>(x.p) + (int64_t)(base + j) * x.ts + (int64_t)hkv * x.hs + d);
    }
  };
  auto fetch = [&](bool of_v, int kb) {
    if constexpr (kAhead) {
#pragma unroll
      for (int n = 0; n < NL; ++n) next[n] = fetch1(of_v, kb, n);
    }
  };
  auto place = [&](bool of_v, int kb) {
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const int i = tid + n * kThreads;
      const float4 x = kAhead ? next[kAhead ? n : 0] : fetch1(of_v, kb, n);
      *reinterpret_cast<float4*>(&sm.kv[i / (D / 4)][i % (D / 4) * 4]) = x;
    }
  };
  if (rank < blocks) fetch(false, rank);
  for (int kb = rank; kb < blocks; kb += ranks) {
    const int j0 = kb * BN;
    __syncthreads();
    place(false, kb);
    __syncthreads();
    fetch(true, kb);
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
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(&sm.kv[tx + 16 * j][d]);
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
    __syncthreads();  // K has been read
    place(true, kb);
    __syncthreads();
    if (kb + ranks < blocks) fetch(false, kb + ranks);
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
          const float* vp = &sm.kv[j + jj][n * 16 * VW + tx * VW];
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

  // The rows' sums into shared memory, over Q, for the whole cluster to see.
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < NJ; ++n)
#pragma unroll
      for (int e = 0; e < VW; ++e) sm.q[ty * 4 + i][n * 16 * VW + tx * VW + e] = o[i][n * VW + e];
  cluster.sync();
  const int lane = tid & 31;
  constexpr int E = D / 32;
  for (int r = rank * (kThreads / 32) + (tid >> 5); r < rows; r += ranks * (kThreads / 32)) {
    const int t = tile.t0 + r / G, h = hkv * G + r % G;
    float acc[E] = {}, m = -INFINITY, l = 0.0f;
    for (int z = 0; z < ranks; ++z) {  // the same order in every call
      const Smem<D>& other = *cluster.map_shared_rank(&sm, z);
      const float mz = other.m[r];
      const float mn = fmaxf(m, mz);
      // A share without a key (m = -inf) adds its l = 0, or the NaN of a row all of
      // whose scores are NaN.
      const float f = m == -INFINITY ? 0.0f : exp2f(m - mn);
      const float g = mz == -INFINITY ? 1.0f : exp2f(mz - mn);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, g * other.q[r][lane * E + e]);
      l = fmaf(l, f, g * other.l[r]);
      m = mn;
    }
    bool finite = isfinite(l);
#pragma unroll
    for (int e = 0; e < E; ++e) finite = finite && isfinite(acc[e]);
    if (!__all_sync(0xffffffffu, finite))
      exact_row<T, D>(p, tile.s, base, t, h, 0, min(hi, tile.pos0 + r / G + 1), acc, m, l);
    finish_row<T, D>(p, t, h, lane, acc, m, l);
  }
  cluster.sync();  // no CTA leaves while its sums may be read
}

// Sums v[0 .. 31] of every lane over the warp: lane i is left with the sum of
// v[i].  Each step halves the values: a lane keeps the half its bit names and
// sends the other.
__device__ __forceinline__ float butterfly(float (&v)[32], int lane) {
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
    }
  }
  return v[0];
}

constexpr int kKeys = 8;   // keys of a warp's step

// RB rows at most: RB * kKeys / 32 butterflies per step.
template <typename T, int D, int RB>
__global__ void __launch_bounds__(kThreads, RB * D <= 512 ? 2 : 1) attn_rows_kernel(const __grid_constant__ AttnLaunch p,
                                                             int splits) {
  constexpr int E = D / 32, W = kThreads / 32, NB = RB * kKeys / 32;
  __shared__ float so[W][RB][D];
  __shared__ float2 sml[W][RB];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.Hq / p.Hkv, TT = RB / G;
  const int id = blockIdx.x / p.Hkv, hkv = blockIdx.x % p.Hkv;
  start_next_kernel();
  const SeqTile tile = find_tile(p, id, TT);
  if ((threadIdx.x == 0 && tile.bad) ||
      (threadIdx.x == kThreads - 1 && blockIdx.y == 0 && hkv == 0 && own_range_bad(p, id)))
    atomicOr(p.status, kStatusBadSeqlens);
  if (tile.nt == 0) return;
  const int base = cu_at(p.cu, tile.s), rows = tile.nt * G;
  const int hi = max(0, tile.pos0 + tile.nt);
  const int steps = (hi + kKeys - 1) / kKeys;
  const int k0 = (int)((int64_t)steps * blockIdx.y / splits) * kKeys;
  const int k1 = min(hi, (int)((int64_t)steps * (blockIdx.y + 1) / splits) * kKeys);
  const float c = p.scale * kLog2e;

  auto loadE = [&](const T* x, float (&v)[E]) {
    if constexpr (E == 1) {
      v[0] = to_f(x[lane]);
    } else if constexpr (E % 4 == 0) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 f = load4(x + lane * E + e);
        v[e] = f.x; v[e + 1] = f.y; v[e + 2] = f.z; v[e + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = to_f(x[lane * E + e]);
    }
  };
  float q[RB][E], acc[RB][E], m[RB], l[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[r][e] = acc[r][e] = 0.0f;
    if (r < rows)
      loadE(static_cast<const T*>(p.q.p) + (int64_t)(tile.t0 + r / G) * p.q.ts +
                (int64_t)(hkv * G + r % G) * p.q.hs, q[r]);
  }
  // Lane i < kKeys finds key i of a step, one step ahead.
  int64_t next_k = -1, next_v = -1;
  auto find = [&](int j) {
    next_k = next_v = -1;
    if (lane < kKeys && j < k1) {
      next_k = key_offset(p, false, tile.s, base, hkv, j);
      next_v = key_offset(p, true, tile.s, base, hkv, j);
      if (next_k < 0) atomicOr(p.status, kStatusBadIndex);
    }
  };
  find(k0 + warp * kKeys + lane);
#pragma unroll 1
  for (int j0 = k0 + warp * kKeys; j0 < k1; j0 += W * kKeys) {
    float k[kKeys][E], v[kKeys][E];
    const int64_t ko = next_k, vo = next_v;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int64_t a = __shfl_sync(0xffffffffu, ko, i), b = __shfl_sync(0xffffffffu, vo, i);
#pragma unroll
      for (int e = 0; e < E; ++e) k[i][e] = v[i][e] = 0.0f;
      if (a >= 0) loadE(static_cast<const T*>(key_base(p, false)) + a, k[i]);
      if (b >= 0) loadE(static_cast<const T*>(key_base(p, true)) + b, v[i]);
    }
    find(j0 + W * kKeys + lane);
    // Dot products: value rr * kKeys + i of a butterfly is row rr, key i.
    float s[NB];  // this lane's row and key of each butterfly
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float x[32];
#pragma unroll
      for (int z = 0; z < 32; ++z) {
        const int r = n * (32 / kKeys) + z / kKeys, i = z % kKeys;
        float d = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) d = fmaf(q[r][e], k[i][e], d);
        x[z] = d;
      }
      s[n] = butterfly(x, lane);
      const int r = n * (32 / kKeys) + lane / kKeys, j = j0 + lane % kKeys;
      s[n] = (j < k1 && j <= tile.pos0 + r / G) ? s[n] * c : -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float mx = s[n];  // over the row's 8 lanes
#pragma unroll
      for (int w = kKeys / 2; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
#pragma unroll
      for (int rr = 0; rr < 32 / kKeys; ++rr) {
        const int r = n * (32 / kKeys) + rr;
        const float mn = fmaxf(m[r], __shfl_sync(0xffffffffu, mx, rr * kKeys));
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2f(m[r] - ref);
        m[r] = mn;
        l[r] *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] *= f;
        const float w = exp2f(s[n] - ref);  // of this lane's key, if it is of row r
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, rr * kKeys + i);
          l[r] += wi;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[r][e] = fmaf(wi, v[i][e], acc[r][e]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RB; ++r) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][r][lane * E + e] = acc[r][e];
    if (lane == 0) sml[warp][r] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  for (int r = warp; r < rows; r += W) {
    float a[E] = {}, mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < W; ++w) {
      const float2 x = sml[w][r];
      const float mn = fmaxf(mm, x.x);
      const float f = mm == -INFINITY ? 0.0f : exp2f(mm - mn);
      const float g = x.x == -INFINITY ? 1.0f : exp2f(x.x - mn);  // (0, or a NaN: kept)
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = fmaf(a[e], f, g * so[w][r][lane * E + e]);
      ll = fmaf(ll, f, g * x.y);
      mm = mn;
    }
    const int t = tile.t0 + r / G, h = hkv * G + r % G;
    bool finite = isfinite(ll);
#pragma unroll
    for (int e = 0; e < E; ++e) finite = finite && isfinite(a[e]);
    if (!__all_sync(0xffffffffu, finite))
      exact_row<T, D>(p, tile.s, base, t, h, k0, min(k1, tile.pos0 + r / G + 1), a, mm, ll);
    if (splits > 1) {
      const Partials part(p.ws, (int64_t)gridDim.x * splits, RB, D);
      part.put<E>(((int64_t)id * p.Hkv + hkv) * splits + blockIdx.y, r, lane, a, mm, ll);
    } else {
      finish_row<T, D>(p, t, h, lane, a, mm, ll);
    }
  }
}

// Joins the key ranges of the rows of each tile, RW warps to a row.
template <typename T, int D, int RW>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const __grid_constant__ AttnLaunch p,
                                                             int splits, int bm, int TT) {
  wait_for_previous_kernel();
  const int G = p.Hq / p.Hkv;
  const int id = (int)(blockIdx.x / p.Hkv), hkv = blockIdx.x % p.Hkv;
  const SeqTile tile = find_tile(p, id, TT);
  const int r = (blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5)) / RW;
  const Partials part(p.ws, (int64_t)gridDim.x * splits, bm, D);
  const int64_t slot = ((int64_t)id * p.Hkv + hkv) * splits;
  join_row<T, D, RW>(p, part, splits, [&](int z) { return slot + z; }, r, r < tile.nt * G,
                     tile.t0 + r / G, hkv * G + r % G);
}

// Rows of the row kernel's CTA that hold `need` of them; 0: too many (its warps'
// sums, 8 x rows x D, take 32 KB of shared memory at most, and the registers).
int row_block(int64_t need, int64_t D) {
  for (int rb = 4; rb <= 16 && rb * D <= 1024; rb <<= 1)
    if (need <= rb) return rb;
  return 0;
}

int row_splits(int64_t ctas, int64_t max_kv) {
  // Four CTAs per SM (about half the tile numbers are empty), two at a time: unequal
  // sequences even out.  Ranges of at least 32 keys a warp: each costs the join a step.
  // (f32, 8 + 2 heads of 128; two per SM, 64 ranges at most, against this: one sequence of
  // 100000 keys 99 and 72 us, 32 of 1 .. 8192 99 and 93, 128 of 1 .. 4096 181 and 165, 4
  // of up to 7000 33 and 34; with ranges of 8 keys a warp the last takes 38.)
  const int64_t want = (8 * 152 + ctas - 1) / ctas, most = max_kv / 256;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 256}));
}

template <typename T, int D, int RB>
cudaError_t launch_rows(const AttnLaunch& p, cudaStream_t st) {
  const int TT = RB / (p.Hq / p.Hkv);
  const int64_t ctas = tile_bound(p.T, p.N, TT) * p.Hkv;
  const int splits = row_splits(ctas, (int64_t)p.max_pages * p.page_size);
  attn_rows_kernel<T, D, RB><<<dim3((unsigned)ctas, splits), kThreads, 0, st>>>(p, splits);
  note_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  return launch_attn_join(p, splits, RB, TT, st);
}

template <typename T, int D, bool PAGED>
cudaError_t launch_tiles(const AttnLaunch& p, int64_t items, int ranks, cudaStream_t st) {
  static const cudaError_t attr =
      cudaFuncSetAttribute(attn_simt_kernel<T, D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)sizeof(Smem<D>));
  if (attr != cudaSuccess) return attr;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ranks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(items * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem<D>);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_simt_kernel<T, D, PAGED>, p);
  note_launch();
  return e;
}

template <typename T, int D>
cudaError_t launch(const AttnLaunch& p, cudaStream_t st) {
  const int G = p.Hq / p.Hkv, TT = BM / G;
  if (p.table != nullptr) {
    switch (row_block((int64_t)p.max_q * G, D)) {
      case 4: return launch_rows<T, D, 4>(p, st);
      case 8:
        if constexpr (D <= 128) return launch_rows<T, D, 8>(p, st);
        break;
      case 16:
        if constexpr (D <= 64) return launch_rows<T, D, 16>(p, st);
        break;
    }
  }
  const int64_t items = tile_bound(p.T, p.N, TT) * p.Hkv;
  // A cluster per tile, large enough for two CTAs per SM.  (1024 tokens, 8 heads,
  // D = 128: 187, 122, 103 and 154 us with 1, 2, 4 and 8; the rule takes 4.)
  int ranks = 1;
  while (ranks < kMaxCluster && items * ranks < 2 * 152) ranks <<= 1;
  return p.table != nullptr ? launch_tiles<T, D, true>(p, items, ranks, st)
                            : launch_tiles<T, D, false>(p, items, ranks, st);
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

size_t attn_simt_workspace_bytes(int64_t T, int64_t N, int64_t Hq, int64_t Hkv, int64_t D,
                                 int64_t max_q) {
  const int64_t G = Hq / Hkv;
  const int rb = row_block(max_q * G, D);
  if (rb == 0) return 0;
  const int64_t ctas = tile_bound(T, N, rb / G) * Hkv;
  const int splits = row_splits(ctas, INT64_MAX);
  return splits > 1 ? Partials::bytes(ctas * splits, rb, D) : 0;
}

namespace {

template <typename T, int D>
cudaError_t join(const AttnLaunch& p, int splits, int bm, int TT, cudaStream_t st) {
  const int64_t ctas = tile_bound(p.T, p.N, TT) * p.Hkv;
  const int rows = TT * (p.Hq / p.Hkv);
  // Eight warps to a row when there is a range for each (5 instead of 16 us for 16
  // ranges of 8 rows), else a warp.
  if (splits >= 8)
    return launch_after(attn_join_kernel<T, D, 8>, dim3((unsigned)ctas, rows), kThreads, st, p, splits,
                        bm, TT);
  return launch_after(attn_join_kernel<T, D, 1>, dim3((unsigned)ctas, (rows + 7) / 8), kThreads, st, p,
                      splits, bm, TT);
}

template <typename T>
cudaError_t join_by_dim(const AttnLaunch& p, int splits, int bm, int TT, cudaStream_t st) {
  switch (p.D) {
    case 32: return join<T, 32>(p, splits, bm, TT, st);
    case 64: return join<T, 64>(p, splits, bm, TT, st);
    case 128: return join<T, 128>(p, splits, bm, TT, st);
    default: return join<T, 256>(p, splits, bm, TT, st);
  }
}

}  // namespace

cudaError_t launch_attn_join(const AttnLaunch& p, int splits, int bm, int TT, cudaStream_t st) {
  return p.bf16 ? join_by_dim<__nv_bfloat16>(p, splits, bm, TT, st)
                : join_by_dim<float>(p, splits, bm, TT, st);
}

cudaError_t launch_attn_simt(const AttnLaunch& p, cudaStream_t st) {
  return p.bf16 ? by_dim<__nv_bfloat16>(p, st) : by_dim<float>(p, st);
}

}  // namespace gdn
