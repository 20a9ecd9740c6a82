// gdn_attn8_prepare.cu -- the step before full attention over a cache in 8 bits: norm and
// rotary positions of q and k as in gdn_attn_prepare.cu, and the new k and v rows as e4m3
// codes with a scale for each block of `block` rows and kv head.
//
// A block's scale is a power of two, S = 2^e: the smallest with max |x| <= 448 2^e over the
// finite new values of the block (e >= -64), and at least the scale that rows from earlier
// calls have there.  Where it grows, those rows' codes are rounded again at the new scale;
// being powers of two, the scales shift a code exactly unless it falls below the format's
// normal range.  code = e4m3(x / S), to nearest even; what is not finite becomes the
// format's NaN.
//
// Work.  Items of (block of a sequence's positions, kv head, k or v), each one team's: the
// team reads its new rows, keeps the rotated values in registers (the first kKeep rows a
// lane; later ones are computed twice) until the block's maximum is known, and stores.
// A team is a warp where the calls bring a few tokens a sequence and a CTA of 256 threads
// where they bring many.  Beside the items, further CTAs of the same launch do the rows of
// q (and of k for k_out).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_prepare.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

using namespace attn_prepare;
using attn::E4;

constexpr int kKeep = 4;
constexpr int kMinExp = -64;

// Item numbers of a sequence: its new rows lie in at most floor((n + B - 2) / B) + 1 <=
// floor(n / B) + 2 blocks, so numbers from floor(cu[s] / B) + 2 s on have room for them
// (as for the tiles of attn::find_tile).
__device__ __forceinline__ int64_t first_number(const int32_t* cu, int s, int B) {
  return (int64_t)(cu[s] / B) + 2 * (int64_t)s;
}

// The last sequence whose first number is <= id: 32 probes at a time by a whole warp.
__device__ __forceinline__ int find_block_seq(const int32_t* cu, int N, int B, int64_t id) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = N;
  for (;;) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned below =
        __ballot_sync(0xffffffffu, at < lo + n && first_number(cu, at, B) <= id);
    lo += max(0, __popc(below) - 1) * step;
    n = min(step, N - lo);
    if (step == 1) return lo;
  }
}

// 2^e with the smallest e >= kMinExp that brings amax (finite, >= 0) within 448 = 1.75 2^8.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = max(kMinExp, (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0));
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <int TEAM>
__device__ __forceinline__ float team_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if constexpr (TEAM > 32) {
    __shared__ float part[TEAM / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = part[threadIdx.x & (TEAM / 32 - 1)];
#pragma unroll
    for (int o = TEAM / 64; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  }
  return x;
}

template <typename T, int D, int TEAM>
__device__ __forceinline__ void block_item(const AttnPrepareLaunch& p, int64_t item) {
  constexpr int LG = D / 8, RG = TEAM / LG;  // lanes of a row, rows of a pass
  const int in_team = threadIdx.x % TEAM, lane = in_team % LG, row_of = in_team / LG;
  const int B = p.block, h2 = (int)(item % (2 * p.Hkv));
  const int64_t id = item / (2 * p.Hkv);
  const bool of_v = h2 >= p.Hkv;
  const int h = of_v ? h2 - p.Hkv : h2;

  // The block: rows first .. first + rows - 1 of the sequence, `before` earlier ones.
  int s = (int)id, nth = 0;
  if (p.cu != nullptr) {
    s = find_block_seq(p.cu, p.N, B, id);
    nth = (int)(id - first_number(p.cu, s, B));
  }
  if (s >= p.N) return;
  const int a = attn::cu_at(p.cu, s), b = attn::cu_at(p.cu, s + 1);
  if (a < 0 || b <= a || b > p.T || nth < 0) return;  // (raised by the checks of q's CTAs)
  const int kv = p.kv_lens ? p.kv_lens[s] : b - a;
  const int pos0 = kv - (b - a);
  const int64_t start = ((int64_t)(max(pos0, 0) / B) + nth) * B;
  if (start >= kv) return;
  const int first = max(pos0, (int)start), rows = (int)min((int64_t)kv, start + B) - first;
  const int before = first - (int)start;
  const int pi = first / p.page_size;
  if (pi >= p.max_pages) {
    if (in_team == 0) atomicOr(p.status, kStatusBadSeqlens);
    return;
  }
  const int64_t pg = p.table[(int64_t)s * p.table_stride + pi];
  if (pg < 0 || pg >= p.num_pages) {
    if (in_team == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  const int in_page = first - pi * p.page_size;
  const AttnPages& c = of_v ? p.vc : p.kc;
  unsigned char* codes = static_cast<unsigned char*>(c.p) + pg * c.ps + (int64_t)h * c.hs +
                         (int64_t)in_page * c.ts;  // of row `first`
  float* scale_p = (of_v ? p.vs : p.ks) + attn::scale_at(p.Hkv, p.page_size, B, pg, h, in_page);
  const int t0 = a + (first - pos0);

  const AttnRows& src = of_v ? p.v : p.k;
  const bool rotates = !of_v && lane < p.rot / 8;
  const int lo = rotates ? lane * 4 : lane * 8, hi = rotates ? p.rot / 2 + lane * 4 : lane * 8 + 4;
  const void* weight = of_v ? nullptr : p.k_w;
  float w[8];
  if (weight != nullptr) {
    Vec8<T> v;
    v.load(static_cast<const T*>(weight), lo, hi);
    v.get(w);
  }
  // Row i of the block's new ones, normed and rotated; false: none (its values are 0).
  auto value = [&](int i, float (&x)[8]) -> bool {
    bool live = i < rows;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    float c4[4], s4[4];
    if (live) {
      if (!of_v && p.rot > 0) {
        const int rp = p.positions ? p.positions[t0 + i] : first + i;
        live = rp >= 0 && rp < p.max_pos;  // (raised with the rows of q)
        if (live && rotates) {
          const float* cs = p.cos_sin + (int64_t)rp * p.rot + lo;
          *reinterpret_cast<float4*>(c4) = *reinterpret_cast<const float4*>(cs);
          *reinterpret_cast<float4*>(s4) = *reinterpret_cast<const float4*>(cs + p.rot / 2);
        }
      } else if (of_v && p.rot > 0) {  // a row without a rotary position is not written at all
        const int rp = p.positions ? p.positions[t0 + i] : first + i;
        live = rp >= 0 && rp < p.max_pos;
      }
    }
    if (live) {
      Vec8<T> v;
      v.load(static_cast<const T*>(src.p) + (int64_t)(t0 + i) * src.ts + (int64_t)h * src.hs, lo, hi);
      v.get(x);
    }
    if (weight != nullptr) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = math::rms_inv(ss, 1.0f / D, p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv * w[e];
    }
    if (live && rotates) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[e], v = x[e + 4];
        x[e] = fmaf(u, c4[e], -v * s4[e]);
        x[e + 4] = fmaf(v, c4[e], u * s4[e]);
      }
    }
    return live;
  };
  float amax = 0.0f;
  auto take = [&](const float (&x)[8], bool live) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = fabsf(x[e]);
      if (live && m <= 3.402823466e38f) amax = fmaxf(amax, m);
    }
  };
  const int passes = (rows + RG - 1) / RG;  // the same for the whole team
  float keep[kKeep][8];
  unsigned lives = 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    if (k < passes) {
      const bool live = value(k * RG + row_of, keep[k]);
      lives |= live ? 1u << k : 0u;
      take(keep[k], live);
    }
  }
  for (int k = kKeep; k < passes; ++k) {
    float x[8];
    const bool live = value(k * RG + row_of, x);
    take(x, live);
  }
  amax = team_max<TEAM>(amax);
  // One thread reads the scale that earlier rows have, and replaces it.
  float scale = block_scale(amax), ratio = 1.0f;
  if (before > 0) {
    float old = 0.0f;
    if constexpr (TEAM == 32) {
      if (in_team == 0) old = *scale_p;
      old = __shfl_sync(0xffffffffu, old, 0);
    } else {
      __shared__ float was;
      if (in_team == 0) was = *scale_p;
      __syncthreads();
      old = was;
    }
    ratio = old / fmaxf(old, scale);
    scale = fmaxf(old, scale);
  }
  if (in_team == 0) *scale_p = scale;
  const float inv = 1.0f / scale;
  auto code2 = [&](float x, float y) -> uint32_t {
    // (x - x is NaN for what is not finite)
    return attn::f_to_e4x2(fmaf(x, inv, x - x), fmaf(y, inv, y - y));
  };
  auto store = [&](int i, const float (&x)[8]) {
    unsigned char* to = codes + (int64_t)i * c.ts;
    *reinterpret_cast<uint32_t*>(to + lo) = code2(x[0], x[1]) | code2(x[2], x[3]) << 16;
    *reinterpret_cast<uint32_t*>(to + hi) = code2(x[4], x[5]) | code2(x[6], x[7]) << 16;
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (lives >> k & 1u) store(k * RG + row_of, keep[k]);
  for (int k = kKeep; k < passes; ++k) {
    float x[8];
    const bool live = value(k * RG + row_of, x);
    if (live) store(k * RG + row_of, x);
  }
  if (ratio != 1.0f) {  // earlier rows at the new scale (ratio NaN: of a scale that is none)
    for (int i = in_team; i < before * (D / 16); i += TEAM) {
      uint4* at = reinterpret_cast<uint4*>(codes + (int64_t)(i / (D / 16) - before) * c.ts + i % (D / 16) * 16);
      uint4 v = *at;
      uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = attn::e4x2_to_f(u[e] & 0xffffu), y = attn::e4x2_to_f(u[e] >> 16);
        u[e] = attn::f_to_e4x2(x.x * ratio, x.y * ratio) | attn::f_to_e4x2(y.x * ratio, y.y * ratio) << 16;
      }
      *at = v;
    }
  }
}

template <typename T, int D, int TEAM>
__global__ void __launch_bounds__(kThreads, 3) attn8_prepare_kernel(
    const __grid_constant__ AttnPrepareLaunch p, const __grid_constant__ AttnPrepareLaunch q_rows,
    int64_t items, int item_ctas, int heads, int heads_per_group, int token_ctas, int gx) {
  if ((int)blockIdx.x < item_ctas) {
    const int64_t item = (int64_t)blockIdx.x * (kThreads / TEAM) + threadIdx.x / TEAM;
    if (item < items) block_item<T, D, TEAM>(p, item);
    return;
  }
  const int i = (int)blockIdx.x - item_ctas;
  prepare_rows<T, D>(q_rows, heads, heads_per_group, token_ctas, i % gx, i / gx);
}

template <typename T, int D, int TEAM>
cudaError_t launch_team(const AttnPrepareLaunch& p, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / 8);
  const int64_t numbers = p.cu == nullptr ? p.N : p.T / p.block + 2 * (int64_t)p.N;
  const int64_t items = numbers * 2 * p.Hkv, per_cta = kThreads / TEAM;
  const int64_t item_ctas = (items + per_cta - 1) / per_cta;
  // The rows of q, and of k where they are asked for: no cache.
  AttnPrepareLaunch q = p;
  q.table = nullptr;
  if (q.k_out == nullptr) q.Hkv = 0;
  const int used = q.Hq + q.Hkv;
  const unsigned gx = (unsigned)((p.T + GROUPS - 1) / GROUPS);
  int per = used;  // heads per group, as in gdn_attn_prepare.cu
  while (per > 1 && (int64_t)gx * ((used + per - 1) / per) < 2 * 152) per = (per + 1) / 2;
  const unsigned checks = p.cu == nullptr ? 0 : (unsigned)((p.N + kCheckSeqs - 1) / kCheckSeqs);
  const int64_t q_ctas = (int64_t)(gx + checks) * ((used + per - 1) / per);
  if (item_ctas + q_ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  attn8_prepare_kernel<T, D, TEAM><<<(unsigned)(item_ctas + q_ctas), kThreads, 0, st>>>(
      p, q, items, (int)item_ctas, used, per, (int)gx, (int)(gx + checks));
  note_launch();
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch(const AttnPrepareLaunch& p, cudaStream_t st) {
  // A warp per item where sequences bring four tokens or fewer on average.
  if (p.T <= 4 * (int64_t)p.N) return launch_team<T, D, 32>(p, st);
  return launch_team<T, D, kThreads>(p, st);
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

cudaError_t launch_attn8_prepare(const AttnPrepareLaunch& p, cudaStream_t st) {
  return p.bf16 ? by_dim<__nv_bfloat16>(p, st) : by_dim<float>(p, st);
}

}  // namespace gdn
