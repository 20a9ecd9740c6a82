// gdn_beam.cu -- beam search's selection: the K best continuations (beam, token) of each
// group of W beams,
//   s[w, v] = score[w] + x[w, v] - ln sum_u e^{x[w, u]},
// in one pass over the logits.
//
// Row kernel.  A CTA has a segment of a row.  Each thread keeps a running maximum and sum of
// exponentials (f32; the threads' sums are joined in f64), and the segment's K largest
// logits are collected on the way: in the first chunk every warp sorts its lanes' maxima,
// and the smallest of the warps' ceil(K / 8)-th ones is a value that at least K logits of
// the segment reach; from then on only logits that reach it are put aside (some K to 10 K
// of them), and the segment's list is the K first of them, sorted.  A segment in which more
// reach it than there is room for (rows of equal logits) is read again, once for each of
// the K places.
//
// Join kernel.  A CTA per group joins the segments' sums into f64 log-sums, turns list
// entries into 64-bit scores (beams are compared at 2^-53: two f32 roundings of a score of
// -12 already span what separates neighbours), and sorts those that reach the K-th best
// head of a list.  Order: score, then the lower w V + v; keys are integers, since f64
// comparisons are a sixty-fourth of their rate.
//
// Bound by the read of the logits; 64 x 8 rows of 131072 bf16 are 134 MB, 20 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;      // 16-byte vectors of a thread per chunk
constexpr int kRoom = 2048;     // logits put aside
constexpr int kMaxSegs = 32;
constexpr float kLog2e = 1.4426950408889634f;

// What a segment leaves: count entries of its list (value key, ~index), its maximum and sum.
struct SegSum {
  float m;
  int count;
  double sum;
};
struct Ws {
  SegSum* sums;               // [rows][segs]
  unsigned long long* list;   // [rows][segs][K]
};
__host__ __device__ inline Ws carve(void* ws, int64_t lists) {
  Ws w;
  w.sums = static_cast<SegSum*>(ws);
  w.list = reinterpret_cast<unsigned long long*>(w.sums + lists);
  return w;
}

// A float's order as an unsigned number; -0 is 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_of(double x) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double value_of(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k & 0x7fffffffffffffffull : ~k));
}
// An entry: larger is better; of equal values the lower index.
__device__ __forceinline__ unsigned long long entry(float x, uint32_t index) {
  return (unsigned long long)order_of(x) << 32 | (uint32_t)~index;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  uint4 r;
  __device__ void load(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  float4 r;
  __device__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ void get(float (&x)[4]) const {
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
  }
};

// Sorts the first n entries (padded with 0 up to a power of two; `size` of them have room)
// in falling order, by the whole CTA.
__device__ __forceinline__ void sort_falling(unsigned long long* a, int n) {
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) a[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int lo = 2 * j * (i / j) + i % j, hi = lo + j;
        const unsigned long long x = a[lo], y = a[hi];
        if ((x < y) == ((lo & k) == 0)) {
          a[lo] = y;
          a[hi] = x;
        }
      }
      __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 6) beam_rows_kernel(const __grid_constant__ BeamLaunch p,
                                                                int segs, int seg_len) {
  attn::start_next_kernel();
  __shared__ unsigned long long aside[kRoom];
  __shared__ float bound[kWarps];
  __shared__ float wm[kWarps];
  __shared__ double wsum[kWarps];
  __shared__ unsigned long long best[kWarps];
  __shared__ int count;
  using V = Vec<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / segs, seg = blockIdx.x % segs;
  const int K = p.K;
  const Ws ws = carve(p.ws, (int64_t)p.B * p.W * segs);
  SegSum* sum_out = ws.sums + blockIdx.x;
  unsigned long long* list = ws.list + (int64_t)blockIdx.x * K;
  const float score = p.scores[row];
  if (!(fabsf(score) <= 3.402823466e38f) || (p.finished != nullptr && p.finished[row] != 0)) {
    if (tid == 0) *sum_out = SegSum{-INFINITY, 0, 0.0};
    return;
  }
  const T* x = static_cast<const T*>(p.logits) + (int64_t)(row / p.W) * p.batch_stride +
               (int64_t)(row % p.W) * p.beam_stride;
  const int v0 = min((int64_t)p.V, (int64_t)seg * seg_len), v1 = (int)min((int64_t)p.V, (int64_t)v0 + seg_len);
  if (tid == 0) count = 0;
  // The row's 16-byte boundaries: logits before the first and behind the last go one by one.
  const int mis = (int)((reinterpret_cast<uintptr_t>(x + v0) & 15u) / sizeof(T));
  const int head = min(v1 - v0, mis ? V::N - mis : 0);
  const int vecs = (v1 - v0 - head) / V::N;
  const int tail0 = v0 + head + vecs * V::N;
  const T* body = x + v0 + head;
  float m = -INFINITY, sum = 0.0f, ref = 0.0f;  // ref = m log2(e), 0 while m is -inf
  float floor_ = -INFINITY;                     // logits below it are not among the segment's K
  auto add = [&](float y) { sum += ex2(fmaf(y, kLog2e, -ref)); };
  auto raise = [&](float top) {
    if (top > m) {
      const float r = top * kLog2e;
      sum *= m == -INFINITY ? 1.0f : ex2(ref - r);  // (a sum of NaN stays one)
      m = top;
      ref = r;
    }
  };
  auto put = [&](float y, int v) {
    if (y >= floor_ && y > -INFINITY) {
      const int at = atomicAdd(&count, 1);
      if (at < kRoom) aside[at] = entry(y, (uint32_t)v);
    }
  };
  __syncthreads();
  for (int base = 0; base < vecs; base += kThreads * kUnroll) {
    V r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kThreads + tid;
      if (i < vecs) r[u].load(body + (int64_t)i * V::N);
    }
    float tops[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      tops[u] = -INFINITY;
      if (base + u * kThreads + tid >= vecs) continue;
      float y[V::N];
      r[u].get(y);
#pragma unroll
      for (int e = 0; e < V::N; ++e) tops[u] = fmaxf(tops[u], y[e]);
      raise(tops[u]);
#pragma unroll
      for (int e = 0; e < V::N; ++e) add(y[e]);
    }
    if (floor_ == -INFINITY) {  // the same in all threads
      float t = -INFINITY;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) t = fmaxf(t, tops[u]);
      // The warp's maxima in falling order over the lanes.
#pragma unroll
      for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
          const float o = __shfl_xor_sync(0xffffffffu, t, j);
          const bool larger = ((lane & k) == 0) == ((lane & j) == 0);
          t = larger ? fmaxf(t, o) : fminf(t, o);
        }
      t = __shfl_sync(0xffffffffu, t, (K + kWarps - 1) / kWarps - 1);
      if (lane == 0) bound[warp] = t;
      __syncthreads();
      t = bound[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) t = fminf(t, bound[w]);
      floor_ = t;
      __syncthreads();  // `bound` may be written again
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kThreads + tid;
      if (i >= vecs || tops[u] < floor_ || tops[u] == -INFINITY) continue;
      float y[V::N];
      r[u].get(y);
#pragma unroll
      for (int e = 0; e < V::N; ++e) put(y[e], v0 + head + i * V::N + e);
    }
  }
  if (tid < head + (v1 - tail0)) {  // fewer than 16 of them
    const int v = tid < head ? v0 + tid : tail0 + tid - head;
    const float y = attn::to_f(x[v]);
    raise(y);
    add(y);
    put(y, v);
  }
  // The threads' sums.
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) wm[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, wm[w]);
  double d = m == -INFINITY ? (double)sum : (double)(sum * ex2(ref - top * kLog2e));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) wsum[warp] = d;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) d += wsum[w];
    *sum_out = SegSum{top, min(count, K), d};
  }
  if (count <= kRoom) {
    sort_falling(aside, count);
    for (int i = tid; i < min(count, K); i += kThreads) list[i] = aside[i];
    return;
  }
  // Too many: place after place, the largest entry below the last one.
  unsigned long long last = ~0ull;
  for (int k = 0; k < K; ++k) {
    unsigned long long mine = 0;
    for (int v = v0 + tid; v < v1; v += kThreads) {
      const float y = attn::to_f(x[v]);
      if (y > -INFINITY) {
        const unsigned long long e = entry(y, (uint32_t)v);
        if (e < last && e > mine) mine = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, mine, o);
      mine = other > mine ? other : mine;
    }
    if (lane == 0) best[warp] = mine;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) mine = best[w] > mine ? best[w] : mine;
    last = mine;
    if (tid == 0) list[k] = mine;
    __syncthreads();
  }
}

// Sorts scores and their indices in falling order of score, rising of index.
__device__ __forceinline__ void sort_scores(unsigned long long* key, uint32_t* index, int n) {
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) {
    key[i] = 0;
    index[i] = 0xffffffffu;
  }
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int lo = 2 * j * (i / j) + i % j, hi = lo + j;
        const unsigned long long x = key[lo], y = key[hi];
        const uint32_t a = index[lo], b = index[hi];
        const bool less = x < y || (x == y && a > b);
        if (less == ((lo & k) == 0)) {
          key[lo] = y;
          key[hi] = x;
          index[lo] = b;
          index[hi] = a;
        }
      }
      __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const __grid_constant__ BeamLaunch p, int segs) {
  __shared__ unsigned long long key[kRoom];
  __shared__ uint32_t index[kRoom];
  __shared__ double base[kBeamMaxW];  // score - log sum of each beam; NaN: takes no part
  __shared__ int count;
  const int tid = threadIdx.x, b = blockIdx.x, K = p.K;
  const int lists = p.W * segs;  // at most kRoom
  attn::wait_for_previous_kernel();
  const Ws ws = carve(p.ws, (int64_t)p.B * lists);
  const SegSum* sums = ws.sums + (int64_t)b * lists;
  const unsigned long long* list = ws.list + (int64_t)b * lists * K;
  for (int w = tid; w < p.W; w += kThreads) {
    const double score = p.scores[(int64_t)b * p.W + w];
    float top = -INFINITY;
    for (int s = 0; s < segs; ++s) top = fmaxf(top, sums[w * segs + s].m);
    double total = 0.0;
    for (int s = 0; s < segs; ++s) {
      const SegSum x = sums[w * segs + s];
      total += x.m == -INFINITY ? x.sum : x.sum * exp((double)x.m - (double)top);
    }
    // Nothing in the row, an infinity or a NaN: no score of it is finite.
    base[w] = score - ((double)top + log(total));
  }
  __syncthreads();
  auto score_of = [&](int l, unsigned long long e) -> unsigned long long {
    const double s = base[l / segs] + (double)value_of((uint32_t)(e >> 32));
    return s - s == 0.0 ? order_of(s) : 0ull;
  };
  // The K-th best head of a list is a score that K entries reach.
  unsigned long long floor_ = 0;
  if (lists >= K) {
    for (int l = tid; l < lists; l += kThreads) {
      key[l] = sums[l].count > 0 ? score_of(l, list[(int64_t)l * K]) : 0ull;
      index[l] = (uint32_t)l;
    }
    sort_scores(key, index, lists);
    floor_ = key[K - 1];
  }
  __syncthreads();
  int kept = 0;
  const int64_t all = (int64_t)lists * K;
  // Beams that ended come first: one entry each.
  if (tid == 0) count = 0;
  __syncthreads();
  for (int w = tid; w < p.W; w += kThreads) {
    const float s = p.scores[(int64_t)b * p.W + w];
    if (p.finished != nullptr && p.finished[(int64_t)b * p.W + w] != 0 && fabsf(s) <= 3.402823466e38f) {
      const int at = atomicAdd(&count, 1);
      key[at] = order_of((double)s);
      index[at] = (uint32_t)(w * p.V + p.pad);
    }
  }
  __syncthreads();
  kept = count;
  const int room = kRoom - kBeamMaxK;  // new ones of a pass; W <= kBeamMaxW <= kBeamMaxK
  for (int64_t at0 = 0; at0 < all; at0 += room) {
    for (int64_t i = at0 + tid; i < min(all, at0 + room); i += kThreads) {
      const int l = (int)(i / K), k = (int)(i % K);
      if (k >= sums[l].count) continue;
      const unsigned long long e = list[i], s = score_of(l, e);
      if (s != 0 && s >= floor_) {
        const int at = atomicAdd(&count, 1);
        key[at] = s;
        index[at] = (uint32_t)(l / segs * p.V) + ~(uint32_t)e;
      }
    }
    __syncthreads();
    const int n = count;
    if (n > kept || at0 == 0) {
      sort_scores(key, index, n);
      kept = min(n, K);
    }
    __syncthreads();
    if (tid == 0) count = kept;
    __syncthreads();
  }
  for (int k = tid; k < K; k += kThreads) {
    const bool some = k < kept;
    const int64_t to = (int64_t)b * K + k;
    p.parents[to] = some ? (int32_t)(index[k] / (uint32_t)p.V) : -1;
    p.tokens[to] = some ? (int32_t)(index[k] % (uint32_t)p.V) : -1;
    p.out_scores[to] = some ? (float)value_of(key[k]) : -INFINITY;
  }
}

// Segments of a row.  Twenty-four CTAs for each SM (six at a time) even out, while a
// segment of fewer than 4096 logits spends its time on the sorts; the sums depend on the
// sizes alone.
int segments(int64_t rows, int64_t V) {
  const int64_t want = (24 * 152 + rows - 1) / rows, most = (V + 4095) / 4096;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, kMaxSegs}));
}

}  // namespace

size_t beam_workspace_bytes(int64_t B, int64_t W, int64_t V, int64_t K) {
  const int64_t lists = B * W * segments(B * W, V);
  return (size_t)(lists * ((int64_t)sizeof(SegSum) + 8 * K));
}

cudaError_t launch_beam(const BeamLaunch& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.W;
  const int segs = segments(rows, p.V);
  // Whole vectors, so that only a row's own ends are ragged.
  const int seg_len = ((p.V + segs - 1) / segs + 7) & ~7;
  const unsigned grid = (unsigned)(rows * segs);
  if (p.bf16)
    beam_rows_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p, segs, seg_len);
  else
    beam_rows_kernel<float><<<grid, kThreads, 0, st>>>(p, segs, seg_len);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return attn::launch_after(beam_join_kernel, dim3((unsigned)p.B), kThreads, st, p, segs);
}

}  // namespace gdn
