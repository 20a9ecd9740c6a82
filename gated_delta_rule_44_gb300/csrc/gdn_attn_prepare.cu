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
// HBM-bound: every row is read and written once in 16-byte vectors.  D / 8
// lanes own one token and 8 dims each, so the norm is a shuffle reduction, the
// rotary partner (R / 2 dims away, a whole number of lanes) is one shuffle,
// and the table row and the norm weights stay in registers while the lanes
// walk a range of the token's heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // heads whose loads are in flight before the first is used

template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 r;
  __device__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ void copy(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ static void store(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ void copy(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

// The last sequence s with cu[s] <= t.  A decode batch (t = s) and a single
// sequence are tried first: a binary search is a chain of dependent loads.
__device__ __forceinline__ int find_seq(const int32_t* cu, int N, int t) {
  if (cu == nullptr) return t;
  if (t < N && cu[t] == t && cu[t + 1] == t + 1) return t;
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_prepare_kernel(
    const __grid_constant__ AttnPrepareLaunch p, int heads, int heads_per_group) {
  constexpr int LG = D / 8;               // lanes of a token
  constexpr int GROUPS = kThreads / LG;   // tokens of a CTA
  const int lane = threadIdx.x % LG, d0 = lane * 8;
  const int t = blockIdx.x * GROUPS + threadIdx.x / LG;
  const bool live = t < p.T;
  const int h0 = blockIdx.y * heads_per_group, h1 = min(heads, h0 + heads_per_group);
  const unsigned grp = (LG == 32) ? 0xffffffffu
                                  : ((1u << (LG & 31)) - 1u) << ((threadIdx.x & 31) / LG * LG);

  auto src = [&](int h) -> const T* {
    if (h < p.Hq) return static_cast<const T*>(p.q.p) + (int64_t)t * p.q.ts + (int64_t)h * p.q.hs;
    h -= p.Hq;
    if (h < p.Hkv) return static_cast<const T*>(p.k.p) + (int64_t)t * p.k.ts + (int64_t)h * p.k.hs;
    h -= p.Hkv;
    return static_cast<const T*>(p.v.p) + (int64_t)t * p.v.ts + (int64_t)h * p.v.hs;
  };
  if (!live) return;  // whole groups leave: the shuffles below stay inside a group

  Vec8<T> raw[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (h0 + i < h1) raw[i].load(src(h0 + i) + d0);

  // The token's sequence, position, table row and cache row.
  const int s = find_seq(p.cu, p.N, t);
  const int a = attn::cu_at(p.cu, s), b = attn::cu_at(p.cu, s + 1);
  unsigned bad = 0;
  if (s >= p.N || a > t || b <= t || b > p.T || (s == 0 && a != 0) || (s == p.N - 1 && b != p.T))
    bad |= kStatusBadSeqlens;
  int pos = -1;  // place in the sequence
  if (!bad) {
    const int kv = p.kv_lens ? p.kv_lens[s] : b - a;
    if (kv < 0) bad |= kStatusBadSeqlens;
    else pos = kv - (b - t);
  }
  int64_t page = -1;
  int row = 0;
  if (p.table != nullptr && pos >= 0) {
    const int pi = pos / p.page_size;
    row = pos - pi * p.page_size;
    if (pi >= p.max_pages) {
      bad |= kStatusBadSeqlens;
    } else {
      page = p.table[(int64_t)s * p.table_stride + pi];
      if (page < 0 || page >= p.num_pages) {
        bad |= kStatusBadIndex;
        page = -1;
      }
    }
  }
  float c8[8], s8[8];
  const int half = p.rot >> 1;
  const bool rotates = d0 < p.rot;
  bool shown = pos >= 0;  // a token without a position gives a zero q and k
  if (p.rot > 0 && shown) {
    const int rp = p.positions ? p.positions[t] : pos;
    if (rp < 0 || rp >= p.max_pos) {
      bad |= kStatusBadIndex;
      shown = false;
      page = -1;
    } else if (rotates) {
      const float* cs = p.cos_sin + (int64_t)rp * p.rot + (d0 < half ? d0 : d0 - half);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(&c8[i]) = *reinterpret_cast<const float4*>(cs + i);
        *reinterpret_cast<float4*>(&s8[i]) = *reinterpret_cast<const float4*>(cs + half + i);
      }
      // The lower half of a pair subtracts its partner's sine term.
      if (d0 < half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s8[i] = -s8[i];
      }
    }
  }
  if (bad && lane == 0) atomicOr(p.status, bad);
  // The lane (of the whole warp) that holds the partner dims, R / 2 away.
  const int wl = threadIdx.x & 31;
  const int partner = !rotates ? wl : (d0 < half ? wl + half / 8 : wl - half / 8);

  float qw[8], kw[8];
  if (p.q_w && h0 < p.Hq) {
    Vec8<T> w;
    w.load(static_cast<const T*>(p.q_w) + d0);
    w.get(qw);
  }
  if (p.k_w && h1 > p.Hq) {
    Vec8<T> w;
    w.load(static_cast<const T*>(p.k_w) + d0);
    w.get(kw);
  }

  for (int hb = h0; hb < h1; hb += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = hb + i;
      if (h >= h1) break;
      if (h >= p.Hq + p.Hkv) {  // v: copied
        if (page >= 0)
          raw[i].copy(static_cast<T*>(p.vc.p) + page * p.vc.ps +
                      (int64_t)(h - p.Hq - p.Hkv) * p.vc.hs + (int64_t)row * p.vc.ts + d0);
        continue;
      }
      const bool is_q = h < p.Hq;
      float x[8];
      raw[i].get(x);
      if (is_q ? p.q_w != nullptr : p.k_w != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(grp, ss, o);
        const float inv = math::rms_inv(ss, 1.0f / D, p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv * (is_q ? qw[e] : kw[e]);
      }
      if (p.rot > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = __shfl_sync(grp, x[e], partner);
          if (rotates) x[e] = fmaf(x[e], c8[e], y * s8[e]);
        }
      }
      if (!shown) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.0f;
      }
      if (is_q) {
        Vec8<T>::store(static_cast<T*>(p.q_out) + ((int64_t)t * p.Hq + h) * D + d0, x);
      } else {
        const int hk = h - p.Hq;
        if (p.k_out)
          Vec8<T>::store(static_cast<T*>(p.k_out) + ((int64_t)t * p.Hkv + hk) * D + d0, x);
        if (page >= 0)
          Vec8<T>::store(static_cast<T*>(p.kc.p) + page * p.kc.ps + (int64_t)hk * p.kc.hs +
                             (int64_t)row * p.kc.ts + d0, x);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (hb + kAhead + i < h1) raw[i].load(src(hb + kAhead + i) + d0);
  }
}

template <typename T, int D>
cudaError_t launch(const AttnPrepareLaunch& p, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / 8);
  // Without a cache the v heads have nowhere to go.
  const int used = p.Hq + (p.table ? 2 : 1) * p.Hkv;
  const unsigned gx = (unsigned)((p.T + GROUPS - 1) / GROUPS);
  // Heads per group: 8 once that still leaves a few CTAs per SM, fewer before.
  int per = 8;
  while (per > 1 && (int64_t)gx * ((used + per - 1) / per) < 4 * 152) per >>= 1;
  const dim3 grid(gx, (unsigned)((used + per - 1) / per));
  attn_prepare_kernel<T, D><<<grid, kThreads, 0, st>>>(p, used, per);
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
