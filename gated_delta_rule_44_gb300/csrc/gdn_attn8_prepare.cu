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
// The code is that of the exact x: it is taken from an f32 evaluation, and where a change by
// what that may be off would change it (2^-19 of x and its partner; some one row of 256
// values in 50), the row is evaluated again in pairs of f32, hi + lo, and rounded from
// those.  What is kept of a key for the whole sequence then does not hang on the order of a
// sum.
//
// Work.  Items of (block of a sequence's positions, kv head, k or v), each one team's: the
// team reads its new rows, keeps the rotated values in registers (the first few rows of a
// lane; later ones are computed twice) until the block's maximum is known, and stores.
// A team is the D / 8 lanes of one row where the calls bring a few tokens a sequence, and a
// CTA of 256 threads where they bring many.  Beside the items, further CTAs of the same
// launch do the rows of q (and of k for k_out).
//
// Four prompts of 2048, 16 + 2 heads of 256 (161 MB, 24 us) take 40 us, bound by the instructions
// of the rows of q as in gdn_attn_prepare.cu (57 % of the issue rate); with the values of k and v
// kept in shared memory instead of computed twice, or three or five CTAs per SM, 40, 43.5
// and 43.7.  512 single tokens take 10.5 us of kernel time, two chains of dependent loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_prepare.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

using namespace attn_prepare;
using attn::E4;

constexpr int kMinExp = -64;

// Item numbers of a sequence: its new rows lie in at most floor((n + B - 2) / B) + 1 <=
// floor(n / B) + 2 blocks, so numbers from floor(cu[s] / B) + 2 s on have room for them
// (as for the tiles of attn::find_tile).
__device__ __forceinline__ int64_t first_number(const int32_t* cu, int s, int B) {
  return (int64_t)(cu[s] / B) + 2 * (int64_t)s;
}

// The last sequence whose first number is <= id: 32 probes at a time by a whole warp.  A
// decode batch's answer (cu[s] = s) is tried beside the first probes.
__device__ __forceinline__ int find_block_seq(const int32_t* cu, int N, int B, int64_t id) {
  const int lane = threadIdx.x & 31;
  const int64_t g = id * B / (2 * B + 1);
  const bool guess = g + 1 < N && first_number(cu, (int)g, B) <= id && first_number(cu, (int)g + 1, B) > id;
  int lo = 0, n = N;
  for (;;) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned below =
        __ballot_sync(0xffffffffu, at < lo + n && first_number(cu, at, B) <= id);
    if (guess) return (int)g;
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
__device__ __forceinline__ float team_max(float x, unsigned mask) {
#pragma unroll
  for (int o = (TEAM < 32 ? TEAM : 32) / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(mask, x, o));
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

// ---- a row in pairs of f32 ----
// Sums and products with their rounding errors, which f32 arithmetic gives exactly (Knuth's
// two-sum; a product's by an fma).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair sum_of(float a, float b) {
  const float s = a + b, z = s - a;
  return {s, (a - (s - z)) + (b - z)};
}
__device__ __forceinline__ Pair product_of(float a, float b) {
  const float p = a * b;
  return {p, fmaf(a, b, -p)};
}
__device__ __forceinline__ Pair times(Pair a, float b) {
  const Pair p = product_of(a.hi, b);
  return {p.hi, fmaf(a.lo, b, p.lo)};
}
__device__ __forceinline__ Pair plus(Pair a, Pair b) {
  const Pair s = sum_of(a.hi, b.hi);
  return {s.hi, s.lo + (a.lo + b.lo)};
}
// The f32 next to the pair whose last bit is set where the pair is none: it rounds to any
// shorter format as the pair does (midpoints between shorter numbers end in 0).
__device__ __forceinline__ float to_odd(Pair a) {
  const float h = a.hi + a.lo, l = a.lo - (h - a.hi);
  int b = __float_as_int(h);
  if (l != 0.0f && (b & 1) == 0 && h - h == 0.0f) b += (l > 0.0f) == (h > 0.0f) ? 1 : -1;
  return __int_as_float(b);
}
// (x - x is NaN for what is not finite)
__device__ __forceinline__ uint32_t code2(float x, float y, float f) {
  return attn::f_to_e4x2(fmaf(x, f, x - x), fmaf(y, f, y - y));
}
// The codes, at 1 / scale = inv, of 8 values of a row of D, 4 at lo and 4 at hi: normed
// (weight not null) and rotated (cs, the row's cosines at lo, not null; its sines rot / 2
// further on).  By the row's lanes, `mask`.  It reads everything again: passed in registers,
// the rare case would cost the others theirs.
template <typename T, int D>
__device__ __noinline__ uint2 exact_codes(const T* row, const T* weight, const float* cs, int rot, int lo, int hi,
                                          float eps, float inv, unsigned mask) {
  float x[8];
  Vec8<T> v;
  v.load(row, lo, hi);
  v.get(x);
  Pair y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = {x[e], 0.0f};
  if (weight != nullptr) {
    float w[8];
    v.load(weight, lo, hi);
    v.get(w);
    Pair ss{0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = plus(ss, product_of(x[e], x[e]));
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1)
      ss = plus(ss, {__shfl_xor_sync(mask, ss.hi, o), __shfl_xor_sync(mask, ss.lo, o)});
    // r = 1 / sqrt(m): an approximation and a Newton step, r (1 + (1 - m r^2) / 2).
    const Pair m = plus({ss.hi * (1.0f / D), ss.lo * (1.0f / D)}, {eps, 0.0f});
    const float r = rsqrtf(m.hi);
    const Pair r2 = product_of(r, r), p = product_of(m.hi, r2.hi);
    const float e1 = (1.0f - p.hi) - (p.lo + fmaf(m.hi, r2.lo, m.lo * r2.hi));
    const float r_lo = 0.5f * r * e1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Pair xw = product_of(x[e], w[e]);
      y[e] = times(xw, r);
      y[e].lo = fmaf(xw.hi, r_lo, y[e].lo);
    }
  }
  if (cs != nullptr) {
    const float4 c = *reinterpret_cast<const float4*>(cs), s = *reinterpret_cast<const float4*>(cs + rot / 2);
    const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const Pair u = y[e], w = y[e + 4];
      y[e] = plus(times(u, c4[e]), times(w, -s4[e]));
      y[e + 4] = plus(times(w, c4[e]), times(u, s4[e]));
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = to_odd(y[e]);
  return make_uint2(code2(x[0], x[1], inv) | code2(x[2], x[3], inv) << 16,
                    code2(x[4], x[5], inv) | code2(x[6], x[7], inv) << 16);
}

// TEAM: the D / 8 lanes of a row (a warp's teams then have the same block), or 256 threads.
template <typename T, int D, int TEAM>
__device__ __forceinline__ void block_item(const AttnPrepareLaunch& p, int64_t id, int h2) {
  constexpr int LG = D / 8, RG = TEAM / LG;  // lanes of a row, rows of a pass
  constexpr int kKeep = TEAM > 32 ? 2 : 1;
  const int in_team = threadIdx.x % TEAM, lane = in_team % LG, row_of = in_team / LG;
  const int B = p.block;
  const unsigned mask =  // the row's lanes
      LG == 32 ? 0xffffffffu : ((1u << (LG & 31)) - 1u) << ((threadIdx.x & 31) / LG * LG);

  // The block: rows first .. first + rows - 1 of the sequence, `before` earlier ones.
  int s = (int)id, nth = 0;
  if (p.cu != nullptr) {
    s = find_block_seq(p.cu, p.N, B, id);
    nth = (int)(id - first_number(p.cu, s, B));
  }
  if (s >= p.N || h2 >= 2 * p.Hkv) return;
  const bool of_v = h2 >= p.Hkv;
  const int h = of_v ? h2 - p.Hkv : h2;
  const int a = attn::cu_at(p.cu, s), b = attn::cu_at(p.cu, s + 1);
  const int kv_len = p.kv_lens ? p.kv_lens[s] : 0;
  if (a < 0 || b <= a || b > p.T || nth < 0) return;  // (raised by the checks of q's CTAs)
  const int kv = p.kv_lens ? kv_len : b - a;
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
  const int64_t pg = p.table[(int64_t)s * p.table_stride + pi];  // (looked at below)
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
  auto row_at = [&](int i) {
    return static_cast<const T*>(src.p) + (int64_t)(t0 + i) * src.ts + (int64_t)h * src.hs;
  };
  auto table_at = [&](int i) {
    return p.cos_sin + (int64_t)(p.positions ? p.positions[t0 + i] : first + i) * p.rot + lo;
  };
  // Row i of the block's new ones, normed and rotated; false: none (its values are 0).
  auto value = [&](int i, float (&x)[8]) -> bool {
    bool live = i < rows;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    float c4[4], s4[4];
    if (live && p.rot > 0) {  // a row without a rotary position is not written at all
      const int rp = p.positions ? p.positions[t0 + i] : first + i;
      live = rp >= 0 && rp < p.max_pos;  // (raised with the rows of q)
      if (live && rotates) {
        const float* cs = table_at(i);
        *reinterpret_cast<float4*>(c4) = *reinterpret_cast<const float4*>(cs);
        *reinterpret_cast<float4*>(s4) = *reinterpret_cast<const float4*>(cs + p.rot / 2);
      }
    }
    if (live) {
      Vec8<T> v;
      v.load(row_at(i), lo, hi);
      v.get(x);
    }
    if (weight != nullptr) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float inv = math::rms_inv(ss, 1.0f / D, p.eps);
      scale_pairs(x, inv, w);
    }
    if (live && rotates) rotate_pairs(x, c4, s4);
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
  if (pg < 0 || pg >= p.num_pages) {  // (the same for the whole team)
    if (in_team == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  const int in_page = first - pi * p.page_size;
  const AttnPages& c = of_v ? p.vc : p.kc;
  unsigned char* codes = static_cast<unsigned char*>(c.p) + pg * c.ps + (int64_t)h * c.hs +
                         (int64_t)in_page * c.ts;  // of row `first`
  float* scale_p = (of_v ? p.vs : p.ks) + attn::scale_at(p.Hkv, p.page_size, B, pg, h, in_page);
  // One thread reads the scale that earlier rows have, and replaces it.
  float old = 0.0f;
  if (before > 0 && in_team == 0) old = *scale_p;
  amax = team_max<TEAM>(amax, mask);
  float scale = block_scale(amax), ratio = 1.0f;
  if (before > 0) {
    if constexpr (TEAM <= 32) {
      old = __shfl_sync(mask, old, (threadIdx.x & 31) / LG * LG);
    } else {
      __shared__ float was;
      if (in_team == 0) was = old;
      __syncthreads();
      old = was;
    }
    ratio = old / fmaxf(old, scale);
    scale = fmaxf(old, scale);
  }
  if (in_team == 0) *scale_p = scale;
  const float inv = 1.0f / scale;
  const bool computed = weight != nullptr || (!of_v && p.rot > 0);  // its rows are not as they came
  auto store = [&](int i, const float (&x)[8]) {
    uint32_t u[2];
    u[0] = code2(x[0], x[1], inv) | code2(x[2], x[3], inv) << 16;
    u[1] = code2(x[4], x[5], inv) | code2(x[6], x[7], inv) << 16;
    if (computed) {
      // How far f32 may be off: 11 steps for the norm and 3 for the rotation, relative to
      // |u| + |v|, which a (scaled) rotation keeps to within sqrt(2).
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        d[e] = 0x1p-19f * (rotates ? fabsf(x[e]) + fabsf(x[e ^ 4]) : fabsf(x[e]));
      const uint32_t a0 = code2(x[0] + d[0], x[1] + d[1], inv) | code2(x[2] + d[2], x[3] + d[3], inv) << 16;
      const uint32_t a1 = code2(x[4] + d[4], x[5] + d[5], inv) | code2(x[6] + d[6], x[7] + d[7], inv) << 16;
      const uint32_t b0 = code2(x[0] - d[0], x[1] - d[1], inv) | code2(x[2] - d[2], x[3] - d[3], inv) << 16;
      const uint32_t b1 = code2(x[4] - d[4], x[5] - d[5], inv) | code2(x[6] - d[6], x[7] - d[7], inv) << 16;
      if (__any_sync(mask, a0 != b0 || a1 != b1)) {
        const uint2 e = exact_codes<T, D>(row_at(i), static_cast<const T*>(weight),
                                          rotates ? table_at(i) : nullptr, p.rot, lo, hi, p.eps, inv, mask);
        u[0] = e.x;
        u[1] = e.y;
      }
    }
    unsigned char* to = codes + (int64_t)i * c.ts;
    *reinterpret_cast<uint32_t*>(to + lo) = u[0];
    *reinterpret_cast<uint32_t*>(to + hi) = u[1];
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
__global__ void __launch_bounds__(kThreads, 4) attn8_prepare_kernel(
    const __grid_constant__ AttnPrepareLaunch p, const __grid_constant__ AttnPrepareLaunch q_rows,
    int64_t items, int item_ctas, int heads, int heads_per_group, int token_ctas, int gx) {
  attn::start_next_kernel();
  attn::wait_for_previous_kernel();
  if ((int)blockIdx.x < item_ctas) {
    // Items of a warp (a CTA): the heads' k, then v, of a block, a team each.
    constexpr int kUnit = TEAM > 32 ? kThreads : 32, kTeams = kUnit / TEAM;
    const int per_block = (2 * p.Hkv + kTeams - 1) / kTeams;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / kUnit) + threadIdx.x / kUnit;
    if (item < items)
      block_item<T, D, TEAM>(p, item / per_block, (int)(item % per_block) * kTeams + threadIdx.x % kUnit / TEAM);
    return;
  }
  const int i = (int)blockIdx.x - item_ctas;
  prepare_rows<T, D>(q_rows, heads, heads_per_group, token_ctas, i % gx, i / gx);
}

template <typename T, int D, int TEAM>
cudaError_t launch_team(const AttnPrepareLaunch& p, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / 8);
  constexpr int kUnit = TEAM > 32 ? kThreads : 32, kTeams = kUnit / TEAM;
  const int64_t numbers = p.cu == nullptr ? p.N : p.T / p.block + 2 * (int64_t)p.N;
  const int64_t items = numbers * ((2 * p.Hkv + kTeams - 1) / kTeams), per_cta = kThreads / kUnit;
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
  return attn::launch_after(attn8_prepare_kernel<T, D, TEAM>, dim3((unsigned)(item_ctas + q_ctas)), kThreads, st,
                            0, p, q, items, (int)item_ctas, used, per, (int)gx, (int)(gx + checks));
}

template <typename T, int D>
cudaError_t launch(const AttnPrepareLaunch& p, cudaStream_t st) {
  // A row's lanes per item where sequences bring four tokens or fewer on average.
  if (p.T <= 4 * (int64_t)p.N) return launch_team<T, D, D / 8>(p, st);
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
