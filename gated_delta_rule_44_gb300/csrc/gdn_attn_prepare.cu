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

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kDepth = 2;  // heads on their way while as many are worked on (4: 43 for 39 us)

// 8 values of a row: 4 at lo, 4 at hi.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint2 a, b;
  __device__ void load(const __nv_bfloat16* p, int lo, int hi) {
    a = *reinterpret_cast<const uint2*>(p + lo);
    b = *reinterpret_cast<const uint2*>(p + hi);
  }
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static Vec8 of(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return {make_uint2(w[0], w[1]), make_uint2(w[2], w[3])};
  }
  __device__ void store(__nv_bfloat16* p, int lo, int hi) const {
    *reinterpret_cast<uint2*>(p + lo) = a;
    *reinterpret_cast<uint2*>(p + hi) = b;
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p, int lo, int hi) {
    a = *reinterpret_cast<const float4*>(p + lo);
    b = *reinterpret_cast<const float4*>(p + hi);
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ static Vec8 of(const float (&x)[8]) {
    return {make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7])};
  }
  __device__ void store(float* p, int lo, int hi) const {
    *reinterpret_cast<float4*>(p + lo) = a;
    *reinterpret_cast<float4*>(p + hi) = b;
  }
};

// The last sequence s with cu[s] <= t, for the warp's first token t: 32 probes at
// a time, a lane each, so that the chain of dependent loads is log32 N long.  A
// decode batch's answer, s = t, is tried beside the first probes.
__device__ __forceinline__ int find_seq(const int32_t* cu, int N, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = N;  // the answer is in lo .. lo + n - 1
  const bool guess = t < N && cu[t] == t && cu[t + 1] == t + 1;
  for (;;) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < lo + n && cu[at] <= t);
    if (guess) return t;
    // cu rises, so the lanes below are the first ones (of malformed offsets any
    // answer will do: the caller checks it).
    lo += max(0, __popc(below) - 1) * step;
    n = min(step, N - lo);
    if (step == 1) return lo;
  }
}

// The search takes rising offsets as given, and of others may never land on the
// sequence that falls, so every sequence's are looked at once: by CTAs of their own,
// which delay none of the others.
constexpr int kCheckSeqs = 2048;  // sequences of such a CTA

__device__ void check_offsets(const AttnPrepareLaunch& p, int cta) {
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  unsigned bad = 0;
  const int s1 = min(p.N, (cta + 1) * kCheckSeqs);
#pragma unroll 4
  for (int s = cta * kCheckSeqs + threadIdx.x; s < s1; s += kThreads) {
    const int a = p.cu[s], b = p.cu[s + 1], kv = p.kv_lens ? p.kv_lens[s] : 0;
    if (a < 0 || b < a || b > p.T || (s == 0 && a != 0) || (s == p.N - 1 && b != p.T) || kv < 0 ||
        (p.table != nullptr && kv > cap))
      bad = kStatusBadSeqlens;
  }
  if (bad) atomicOr(p.status, bad);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 4) attn_prepare_kernel(
    const __grid_constant__ AttnPrepareLaunch p, int heads, int heads_per_group, int token_ctas) {
  constexpr int LG = D / 8;               // lanes of a token
  constexpr int GROUPS = kThreads / LG;   // tokens of a CTA
  if ((int)blockIdx.x >= token_ctas) {
    if (blockIdx.y == 0) check_offsets(p, blockIdx.x - token_ctas);
    return;
  }
  const int lane = threadIdx.x % LG;
  const int t = blockIdx.x * GROUPS + threadIdx.x / LG;
  const int t_first = blockIdx.x * GROUPS + (threadIdx.x & ~31) / LG;  // the warp's first token
  if (t_first >= p.T) return;
  const int h0 = blockIdx.y * heads_per_group, h1 = min(heads, h0 + heads_per_group);
  const unsigned grp = (LG == 32) ? 0xffffffffu
                                  : ((1u << (LG & 31)) - 1u) << ((threadIdx.x & 31) / LG * LG);
  // This lane's dims.
  const bool rotates = lane < p.rot / 8;
  const int lo = rotates ? lane * 4 : lane * 8, hi = rotates ? p.rot / 2 + lane * 4 : lane * 8 + 4;

  // The token's sequence, position, table row and cache row.
  int s = p.cu == nullptr ? t : find_seq(p.cu, p.N, t_first);
  if (t >= p.T) return;  // whole groups leave: the shuffles below stay inside a group
  if (p.cu != nullptr)   // the warp's later tokens may be in later sequences
    while (s + 1 < p.N && p.cu[s + 1] <= t) ++s;
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
  float c4[4], s4[4];
  bool shown = pos >= 0;  // a token without a position gives a zero q and k
  if (p.rot > 0 && shown) {
    const int rp = p.positions ? p.positions[t] : pos;
    if (rp < 0 || rp >= p.max_pos) {
      bad |= kStatusBadIndex;
      shown = false;
      page = -1;
    } else if (rotates) {
      const float* cs = p.cos_sin + (int64_t)rp * p.rot + lo;
      *reinterpret_cast<float4*>(c4) = *reinterpret_cast<const float4*>(cs);
      *reinterpret_cast<float4*>(s4) = *reinterpret_cast<const float4*>(cs + p.rot / 2);
    }
  }
  if (bad && lane == 0) atomicOr(p.status, bad);

  // Heads first .. last - 1 of q or k: norm, rotation, store to one or two places.
  auto rows = [&](const AttnRows& r, const void* weight, int first, int last, T* out, T* cache,
                  int64_t cache_hs) {
    if (first >= last) return;
    const T* in = static_cast<const T*>(r.p) + (int64_t)t * r.ts + (int64_t)first * r.hs;
    if (out != nullptr) out += (int64_t)first * D;
    if (cache != nullptr) cache += (int64_t)first * cache_hs;
    Vec8<T> next[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
      if (first + i < last) next[i].load(in + i * r.hs, lo, hi);
    float w[8];
    if (weight != nullptr) {
      Vec8<T> v;
      v.load(static_cast<const T*>(weight), lo, hi);
      v.get(w);
    }
#pragma unroll 1
    for (int hb = first; hb < last; hb += kDepth) {
      Vec8<T> cur[kDepth];
      in += kDepth * r.hs;
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        cur[i] = next[i];
        if (hb + kDepth + i < last) next[i].load(in + i * r.hs, lo, hi);
      }
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        if (hb + i >= last) break;
        float x[8];
        cur[i].get(x);
        if (weight != nullptr) {
          float ss = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(grp, ss, o);
          const float inv = math::rms_inv(ss, 1.0f / D, p.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv * w[e];
        }
        if (rotates) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = x[e], v = x[e + 4];
            x[e] = fmaf(u, c4[e], -v * s4[e]);
            x[e + 4] = fmaf(v, c4[e], u * s4[e]);
          }
        }
        if (!shown) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        }
        const Vec8<T> y = Vec8<T>::of(x);
        if (out != nullptr) {
          y.store(out, lo, hi);
          out += D;
        }
        if (cache != nullptr) {
          y.store(cache, lo, hi);
          cache += cache_hs;
        }
      }
    }
  };
  rows(p.q, p.q_w, h0, min(h1, p.Hq), static_cast<T*>(p.q_out) + (int64_t)t * p.Hq * D, nullptr, 0);
  const int k0 = max(h0 - p.Hq, 0), k1 = min(h1 - p.Hq, p.Hkv);
  rows(p.k, p.k_w, k0, k1, p.k_out ? static_cast<T*>(p.k_out) + (int64_t)t * p.Hkv * D : nullptr,
       page >= 0 ? static_cast<T*>(p.kc.p) + page * p.kc.ps + (int64_t)row * p.kc.ts : nullptr,
       p.kc.hs);
  if (page >= 0) {
    const T* in = static_cast<const T*>(p.v.p) + (int64_t)t * p.v.ts;
    T* out = static_cast<T*>(p.vc.p) + page * p.vc.ps + (int64_t)row * p.vc.ts;
    for (int h = max(h0 - p.Hq - p.Hkv, 0); h < h1 - p.Hq - p.Hkv; ++h) {
      Vec8<T> v;
      v.load(in + (int64_t)h * p.v.hs, lane * 8, lane * 8 + 4);
      v.store(out + (int64_t)h * p.vc.hs, lane * 8, lane * 8 + 4);
    }
  }
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
