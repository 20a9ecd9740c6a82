// gdn_attn_common.cuh -- what the full-attention kernels share: the tile map
// of packed new tokens, key addresses in packed rows and in paged caches, the
// scalar tail of an output row, and the exact form of one row.
//
// New tokens.  Sequence s owns tokens cu[s] .. cu[s+1]-1 (q_len of them) and a
// context of L = kv_lens[s] keys that ends with them: token i sits at position
// L - q_len + i and sees the keys at positions 0 .. L - q_len + i.  A token at
// a negative position (q_len > L) sees nothing: its output is 0, its lse -inf.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_math.cuh"

namespace gdn {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int cu_at(const int32_t* cu, int s) { return cu ? cu[s] : s; }

// Tiles of TT tokens, each inside one sequence, numbered without a prefix sum:
// sequence s owns the numbers from floor(cu[s] / TT) + s on.  Its ceil(q_len /
// TT) tiles fit below the next sequence's first number because
// floor((a + n) / TT) - floor(a / TT) >= floor(n / TT) >= ceil(n / TT) - 1.
// The numbers in use are below floor(T / TT) + N; the rest are empty.
__host__ __device__ inline int64_t tile_bound(int64_t T, int64_t N, int64_t TT) {
  return T / TT + N;
}

// Sequence s as the device sees it: tokens a .. b-1 and its context length,
// clamped to what the tables hold.  bad: cu_seqlens or kv_lens cannot be right
// (with offsets outside 0 .. T the sequence is taken as empty).
struct SeqRange {
  int a, b, kv;
  int bad;
};
__device__ inline SeqRange seq_range(const AttnLaunch& p, int s) {
  SeqRange r;
  r.a = cu_at(p.cu, s);
  r.b = cu_at(p.cu, s + 1);
  r.bad = r.a < 0 || r.b < r.a || r.b > p.T ||
          (!p.part && ((s == 0 && r.a != 0) || (s == p.N - 1 && r.b != p.T)));
  if (r.a < 0 || r.b < r.a || r.b > p.T) {
    r.a = r.b = r.kv = 0;
    return r;
  }
  r.kv = r.b - r.a;
  if (p.kv_lens != nullptr) {
    r.kv = p.kv_lens[s];
    const int64_t cap = (int64_t)p.max_pages * p.page_size;
    if (r.kv < 0 || r.kv > cap) {
      r.bad = 1;
      r.kv = r.kv < 0 ? 0 : (int)cap;
    }
  }
  if (p.table != nullptr && r.b - r.a > p.max_q) r.bad = 1;
  return r;
}

// The search of find_tile takes rising offsets as given, and of others may never land
// on the sequence that falls. So sequence `id`, where there is one, is looked at with
// tile number `id` as well: the numbers reach N and all are asked for.
__device__ __forceinline__ bool own_range_bad(const AttnLaunch& p, int id) {
  return id < p.N && seq_range(p, id).bad;
}

struct SeqTile {
  int s;       // sequence
  int t0;      // first token of the tile
  int nt;      // its tokens (0: an empty number)
  int pos0;    // position of the first token (may be negative)
  int bad;
};

__device__ inline SeqTile find_tile(const AttnLaunch& p, int id, int TT) {
  int lo = 0, hi = p.N - 1;  // the last s whose first number is <= id
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu_at(p.cu, mid) / TT + mid <= id) lo = mid;
    else hi = mid - 1;
  }
  const SeqRange q = seq_range(p, lo);
  SeqTile r{lo, 0, 0, 0, q.bad};
  const int64_t off = (int64_t)(id - (q.a / TT + lo)) * TT;
  if (off < 0 || off >= q.b - q.a) return r;
  r.t0 = q.a + (int)off;
  r.nt = min(TT, q.b - r.t0);
  r.pos0 = q.kv - (q.b - r.t0);
  return r;
}

// Element offset of key row j of sequence s: of its page's row j % page_size,
// or of packed token base + j.  -1 when the page number is outside the cache
// (the row then reads as zeros and the status word is raised).
__device__ __forceinline__ int64_t page_of(const AttnLaunch& p, int s, int page_idx) {
  const int pg = p.table[(int64_t)s * p.table_stride + page_idx];
  return (pg >= 0 && pg < p.num_pages) ? pg : -1;
}
__device__ __forceinline__ int64_t key_offset(const AttnLaunch& p, bool of_v, int s, int base,
                                              int hkv, int j) {
  if (p.table == nullptr) {
    const AttnRows& r = of_v ? p.v : p.k;
    return (int64_t)(base + j) * r.ts + (int64_t)hkv * r.hs;
  }
  const AttnPages& c = of_v ? p.vc : p.kc;
  const int64_t pg = page_of(p, s, j / p.page_size);
  if (pg < 0) return -1;
  return pg * c.ps + (int64_t)hkv * c.hs + (int64_t)(j % p.page_size) * c.ts;
}
__device__ __forceinline__ const void* key_base(const AttnLaunch& p, bool of_v) {
  return p.table == nullptr ? (of_v ? p.v.p : p.k.p) : (of_v ? p.vc.p : p.kc.p);
}

// ---- caches in 8 bits ----
// A value is its e4m3 code times the f32 scale of its block of rows and kv head.
struct E4 {
  unsigned char code;
};
// Two codes (the first in the low byte) as floats, exact; a NaN code gives NaN.
__device__ __forceinline__ float2 e4x2_to_f(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}\n" : "=r"(h) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float to_f(E4 x) { return e4x2_to_f(x.code).x; }
// (a, b) rounded to the nearest codes, a in the low byte; NaN stays NaN, larger magnitudes
// than 448 become 448.
__device__ __forceinline__ uint32_t f_to_e4x2(float a, float b) {
  unsigned short c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}
// The place of row `row` of page pg in the scales.
__device__ __forceinline__ int64_t scale_at(int Hkv, int page_size, int block, int64_t pg, int hkv,
                                            int row) {
  return (pg * Hkv + hkv) * (page_size / block) + row / block;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// The scale of key row j of sequence s; 0 for a page outside the cache.
__device__ __forceinline__ float key_scale(const AttnLaunch& p, bool of_v, int s, int hkv, int j) {
  const int64_t pg = page_of(p, s, j / p.page_size);
  if (pg < 0) return 0.0f;
  return (of_v ? p.vs : p.ks)[scale_at(p.Hkv, p.page_size, p.block, pg, hkv, j % p.page_size)];
}

__device__ __forceinline__ float sigmoid_gate(float z) { return math::norm_gate(z, true); }

// The sums of a row over a range of its keys, kept in a workspace until the
// ranges are joined: O [slots][rows][D], then (m, l) [slots][rows] pairs, f32.
struct Partials {
  float* o;
  float2* ml;
  int rows, D;
  __host__ __device__ Partials(void* ws, int64_t slots, int rows_, int D_)
      : o(static_cast<float*>(ws)),
        ml(reinterpret_cast<float2*>(static_cast<float*>(ws) + slots * rows_ * D_)),
        rows(rows_),
        D(D_) {}
  static size_t bytes(int64_t slots, int rows, int64_t D) {
    return (size_t)(slots * rows * (D + 2)) * sizeof(float);
  }
#ifdef __CUDACC__
  // One warp, E = D / 32 dims per lane.
  template <int E>
  __device__ void put(int64_t slot, int r, int lane, const float (&acc)[E], float m, float l) const {
    float* d = o + (slot * rows + r) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = acc[e];
    if (lane == 0) ml[slot * rows + r] = make_float2(m, l);
  }
#endif
};

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// The tail of a row by one warp: normalise, gate, round once, store; the lse
// of the scaled scores from their base-2 form.  A row without a key: 0, -inf.
template <typename T, int D>
__device__ __forceinline__ void finish_row(const AttnLaunch& p, int t, int h, int lane,
                                           const float (&acc)[D / 32], float m, float l) {
  constexpr int E = D / 32;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  T* out = static_cast<T*>(p.out) + ((int64_t)t * p.Hq + h) * D + lane * E;
  const T* gate = p.gate.p == nullptr ? nullptr
                                      : static_cast<const T*>(p.gate.p) + (int64_t)t * p.gate.ts +
                                            (int64_t)h * p.gate.hs + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float x = acc[e] * inv;
    if (gate != nullptr) x *= sigmoid_gate(to_f(gate[e]));
    out[e] = from_f<T>(x);
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[(int64_t)t * p.Hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// A joining kernel is launched with programmatic dependence on the kernel whose
// sums it joins: its launch is prepared while that one runs.
__device__ __forceinline__ void start_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}
template <typename... K, typename... A>
cudaError_t launch_after(void (*kernel)(K...), dim3 grid, int threads, cudaStream_t st, size_t shared,
                         const A&... a) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a...);
  note_launch();
  return e;
}

// Lets a kernel have `bytes` of dynamic shared memory on the current device: every device has
// attributes of its own.  `done`: the kernel's, a bit for each of the first 64 devices.
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & bit) != 0) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Joins the n ranges of a row,
//   out = sum_z 2^(m_z - M) O_z / sum_z 2^(m_z - M) l_z,
// whose sums are in the blocks slot_of(z) (negative: none), by RW warps of a CTA
// of 8: warp w takes z = w, w + RW, ...: the (m, l) of 32 ranges first, a lane
// each, then their weighted O, AHEAD loads in flight (8 for 76 ranges of a row; for two or
// three the wide cache's drafts take 353 us with 8, 350.5 with 4).  The order of the sums
// depends on n alone.
template <typename T, int D, int RW, int AHEAD = 8, typename SlotOf>
__device__ __forceinline__ void join_row(const AttnLaunch& p, const Partials& part, int n,
                                         SlotOf slot_of, int r, bool live, int t, int h) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % RW;
  float acc[E] = {}, m = -INFINITY, l = 0.0f;
  for (int z0 = 0; live && w + z0 * RW < n; z0 += 32) {
    const int z = w + (z0 + lane) * RW;
    const int64_t slot = z < n ? slot_of(z) : -1;
    const float2 ml = slot >= 0 ? part.ml[slot * part.rows + r] : make_float2(-INFINITY, 0.0f);
    float mn = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mn = fmaxf(mn, m);
    if (mn == -INFINITY) continue;
    const float f = exp2f(m - mn);  // 0 for m = -inf
    const float wt = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - mn);
    float lw = ml.x == -INFINITY ? 0.0f : wt * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    l = fmaf(l, f, lw);
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
    unsigned todo = __ballot_sync(0xffffffffu, ml.x != -INFINITY);
    while (todo) {
      float x[AHEAD][E], wk[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        wk[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] = 0.0f;
        if (todo) {
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          wk[k] = __shfl_sync(0xffffffffu, wt, src);
          const int64_t sk = __shfl_sync(0xffffffffu, slot, src);
          const float* o = part.o + (sk * part.rows + r) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) x[k][e] = o[e];
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wk[k], x[k][e], acc[e]);
    }
  }
  if constexpr (RW > 1) {
    __shared__ float so[8][D];
    __shared__ float2 sml[8];
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (w != 0) return;
    for (int k = 1; k < RW; ++k) {
      const float2 x = sml[warp + k];
      if (x.x == -INFINITY) continue;
      const float mn = fmaxf(m, x.x);
      const float f = m == -INFINITY ? 0.0f : exp2f(m - mn), g = exp2f(x.x - mn);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, g * so[warp + k][lane * E + e]);
      l = fmaf(l, f, g * x.y);
      m = mn;
    }
  }
  if (live) finish_row<T, D>(p, t, h, lane, acc, m, l);
}

// One row (token t, query head h) over the keys [k0, k1) of its sequence, by
// one warp, key after key in f32 with a running maximum: D / 32 dims per lane.
// m is the maximum of the scaled scores times log2(e), acc and l the sums at
// that reference.  The tiled kernels multiply a masked key's weight 0 into its
// v row, which is not 0 when that v is infinite or NaN; a row whose tiled
// result is not finite is therefore evaluated here, where a masked key is not
// touched at all, and one that scores -inf adds nothing.  bad pages read as
// zeros, as in the tiled kernels.  `progress` (may be null) counts on every 2^14
// keys, for others that wait.  C: the cache's type (T, or E4 with scales).
template <typename T, int D, typename C = T>
__device__ __noinline__ void exact_row(const AttnLaunch& p, int s, int base, int t, int h, int k0,
                                       int k1, float (&acc)[D / 32], float& m, float& l,
                                       int* progress = nullptr) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int hkv = h / (p.Hq / p.Hkv);
  const T* q = static_cast<const T*>(p.q.p) + (int64_t)t * p.q.ts + (int64_t)h * p.q.hs + lane * E;
  float qv[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f(q[e]);
    acc[e] = 0.0f;
  }
  m = -INFINITY;
  l = 0.0f;
  const float c = p.scale * kLog2e;
  for (int j = k0; j < k1; ++j) {
    if (progress != nullptr && lane == 0 && (j & 0x3fff) == 0) atomicAdd(progress, 1);
    const int64_t ko = key_offset(p, false, s, base, hkv, j);
    const int64_t vo = key_offset(p, true, s, base, hkv, j);
    float dot = 0.0f;
    if (ko >= 0) {
      const C* kr = static_cast<const C*>(key_base(p, false)) + ko + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) dot = fmaf(qv[e], to_f(kr[e]), dot);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    float x = dot * c;
    float vscale = 1.0f;
    if constexpr (std::is_same<C, E4>::value) {
      x *= key_scale(p, false, s, hkv, j);
      vscale = key_scale(p, true, s, hkv, j);
    }
    if (x != x) {  // no weight of the row is a number
      m = 0.0f;
      l = x;
      return;
    }
    if (x == -INFINITY) continue;  // weight 0: no part, as of a masked key, whatever its v
    const float mn = fmaxf(m, x);
    const float f = (m == -INFINITY) ? 0.0f : exp2f(m - mn);
    const float w = exp2f(x - mn);
    m = mn;
    l = fmaf(l, f, w);
    const C* vr = static_cast<const C*>(key_base(p, true)) + (vo < 0 ? 0 : vo) + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e)
      acc[e] = fmaf(acc[e], f, w * (vo < 0 ? 0.0f : to_f(vr[e]) * vscale));
  }
}

}  // namespace attn
}  // namespace gdn
