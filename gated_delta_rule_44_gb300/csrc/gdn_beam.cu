// gdn_beam.cu -- beam search's selection: the K best continuations (beam, token) of each
// group of W beams,
//   s[w, v] = score[w] + x[w, v] - ln sum_u e^{x[w, u]},
// in one pass over the logits.
//
// Row kernel.  A CTA has a segment of a row.  Each thread keeps a running sum of
// 2^(H x - ref) (f32), H = log2(e) rounded to f32 and ref a whole number: H x - ref is one
// rounding (an fma), changes of ref and joins are exact, and ln sum e^x = ref / H + ln(sum) to
// within the 1.3e-8 (largest x - x) that H's rounding leaves, where x has its weight.  So
// an element costs an fma, an exponential and an add.  The threads' sums are joined in f64.
// The segment's K largest logits are collected on the way: the K-th largest of the threads'
// maxima so far (found by one warp, two of the upper 16 bits of its order at a time) is a value
// that at least K logits reach, and only 16-byte vectors with a logit that reaches it are put
// aside, whole.  It is taken after the first chunk and again after 8, 64, ... (each time the
// other warps wait for the one; from chunk to chunk some K more vectors reach it), and at the
// end (ranking four chunks' worth by counting took three times as long).  The logits put aside that reach the last one are ranked by
// counting.  A segment in which more are put aside, or reach it, than there
// is room for (rows of equal logits) is read again, once for each of the K places.
//
// Join kernel.  A CTA per group joins the segments' sums into f64 log-sums, turns list
// entries into 64-bit scores (beams are compared at 2^-53: two f32 roundings of a score of
// -12 already span what separates neighbours), and sorts those that reach the K-th best
// head of a list.  Order: score, then the lower w V + v; keys are integers, since f64
// comparisons are a sixty-fourth of their rate.
//
// Bound by the read of the logits in the end; now by instructions: 64 x 8 rows of 131072 bf16
// (134 MB, 20 us) take 43 us in the row kernel, at 62 % of the issue rate, and 55 a call.
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
constexpr int kAside = 768;     // vectors put aside
constexpr int kRanked = 1024;    // logits of them, ranked by counting
constexpr int kRoom = 2048;     // entries of the join's sorts
constexpr int kMaxSegs = 32;    // a lane each
constexpr float kH = 1.4426950408889634f;  // log2(e) in f32

// What a segment leaves: the count of its list's entries (value key, ~index), and its sum of
// 2^(H x - ref) (ref -inf: nothing is above that).
struct SegSum {
  float ref;
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
  __device__ void get(float2 (&x)[4]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)};
  }
  __device__ uint4 bits() const { return r; }
  __device__ void from(const uint4& b) { r = b; }
  __device__ float top() const {  // (a NaN counts only beside another)
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&r);
    const __nv_bfloat162 m = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  float4 r;
  __device__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ void get(float2 (&x)[2]) const {
    x[0] = {r.x, r.y};
    x[1] = {r.z, r.w};
  }
  __device__ uint4 bits() const { return *reinterpret_cast<const uint4*>(&r); }
  __device__ void from(const uint4& b) { r = *reinterpret_cast<const float4*>(&b); }
  __device__ float top() const { return fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w)); }
};

// The warp's largest value; a NaN is passed over.
__device__ __forceinline__ float warp_top(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// A value that at least `n` of the warp's values reach, -inf if fewer are above that: its
// n-th largest.
__device__ __forceinline__ float nth_top(float x, int n) {
  float y = warp_top(x);
  for (;;) {
    const unsigned equal = __ballot_sync(0xffffffffu, x == y);
    n -= __popc(equal);
    if (n <= 0 || y == -INFINITY) return y;
    if (x == y) x = -INFINITY;
    y = warp_top(x);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const __grid_constant__ BeamLaunch p,
                                                                int seg_len) {
  attn::start_next_kernel();
  attn::wait_for_previous_kernel();
  __shared__ uint4 aside[kAside];
  __shared__ int aside_at[kAside];
  __shared__ unsigned long long few[kRanked];
  __shared__ volatile float floors[kWarps];  // values that K / kWarps of a warp's threads have reached
  __shared__ float refs[kThreads], parts[kThreads];
  __shared__ unsigned long long best[kWarps];
  __shared__ int count, few_count;
  using V = Vec<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = blockIdx.x, segs = gridDim.x, K = p.K;
  const int row = blockIdx.z * p.W + blockIdx.y;
  const Ws ws = carve(p.ws, (int64_t)p.B * p.W * segs);
  SegSum* sum_out = ws.sums + (int64_t)row * segs + seg;
  unsigned long long* list = ws.list + ((int64_t)row * segs + seg) * K;
  const float score = p.scores[row];
  if (!(fabsf(score) <= 3.402823466e38f) || (p.finished != nullptr && p.finished[row] != 0)) {
    if (tid == 0) *sum_out = SegSum{-INFINITY, 0, 0.0};
    return;
  }
  const T* x = static_cast<const T*>(p.logits) + blockIdx.z * p.batch_stride + blockIdx.y * p.beam_stride;
  const int v0 = min((int64_t)p.V, (int64_t)seg * seg_len), v1 = (int)min((int64_t)p.V, (int64_t)v0 + seg_len);
  if (tid == 0) count = few_count = 0;
  if (lane == 0) floors[warp] = -INFINITY;
  // The row's 16-byte boundaries: logits before the first and behind the last go one by one.
  const int mis = (int)((reinterpret_cast<uintptr_t>(x + v0) & 15u) / sizeof(T));
  const int head = min(v1 - v0, mis ? V::N - mis : 0);
  const int vecs = (v1 - v0 - head) / V::N;
  const int tail0 = v0 + head + vecs * V::N;
  const T* body = x + v0 + head;
  float top = -INFINITY;  // this thread's largest logit
  float ref = -INFINITY;  // its sum of 2^(H x - ref), in two parts
  float2 sum = {0.0f, 0.0f};
  float use = 0.0f;          // -ref, or 0 while that is -inf
  float floor_ = -INFINITY;  // logits below it are not among the segment's K
  auto raise = [&](float y) {
    if (y > top) {
      top = y;
      const float r = ceilf(y * kH);
      if (r > ref) {
        if (ref != -INFINITY) {  // (a sum of NaN stays one)
          const float f = ex2(ref - r);
          sum.x *= f;
          sum.y *= f;
        }
        ref = r;
        use = -r;
      }
    }
  };
  // A logit that reaches the floor, to be ranked.
  auto put = [&](float y, int v) {
    if (y >= floor_ && y > -INFINITY) {
      const int at = atomicAdd(&few_count, 1);
      if (at < kRanked) few[at] = entry(y, (uint32_t)v);
    }
  };
  __syncthreads();
  constexpr int kChunk = kThreads * kUnroll;
  V r[kUnroll], ahead[kUnroll];
  auto load = [&](int base, bool whole) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kThreads + tid;
      if (whole || i < vecs) ahead[u].load(body + (int64_t)i * V::N);
    }
  };
  // The least of the warps' floors: a value that at least K logits have reached.
  auto read_floor = [&] {
    float f = floors[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) f = fminf(f, floors[w]);
    floor_ = f;
  };
  const int share = (K + kWarps - 1) / kWarps;
  auto work = [&](int base, bool whole) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = ahead[u];
    if (base + 2 * kChunk <= vecs) load(base + kChunk, true);
    else load(base + kChunk, false);
    float tops[kUnroll], most = -INFINITY;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      tops[u] = whole || base + u * kThreads + tid < vecs ? r[u].top() : -INFINITY;
      most = fmaxf(most, tops[u]);
    }
    raise(most);
    const float2 h2 = {kH, kH}, use2 = {use, use};
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!whole && base + u * kThreads + tid >= vecs) continue;
      float2 y[V::N / 2];
      r[u].get(y);
#pragma unroll
      for (int e = 0; e < V::N / 2; ++e) {
        const float2 t = __ffma2_rn(y[e], h2, use2);
        sum = __fadd2_rn(sum, float2{ex2(t.x), ex2(t.y)});
      }
    }
    // Only a warp with a logit that reaches the floor that it knows looks for a newer one.
    // (floors only rise: an old one lets more pass.)
    if (__any_sync(0xffffffffu, base == 0 || most >= floor_)) {
      const float mine = nth_top(top, share);
      if (lane == 0) floors[warp] = mine;
      if (base == 0) __syncthreads();  // (every warp is here, with nothing known yet)
      else __syncwarp();
      read_floor();
      if (most >= floor_ && most > -INFINITY) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (tops[u] >= floor_ && tops[u] > -INFINITY) {
            const int at = atomicAdd(&count, 1);
            if (at < kAside) {
              aside[at] = r[u].bits();
              aside_at[at] = base + u * kThreads + tid;
            }
          }
      }
    }
  };
  load(0, false);
  int base = 0;
  for (; base + kChunk <= vecs; base += kChunk) work(base, true);
  if (base < vecs) work(base, false);
  const bool ragged = tid < head + (v1 - tail0);  // fewer than 16 of them
  const int ragged_v = tid < head ? v0 + tid : tail0 + tid - head;
  const float ragged_y = ragged ? attn::to_f(x[ragged_v]) : -INFINITY;
  if (ragged) {
    raise(ragged_y);
    sum.x += ex2(fmaf(ragged_y, kH, use));
  }
  refs[tid] = ref;
  parts[tid] = sum.x + sum.y;
  __syncthreads();
  read_floor();
  const int n = count;
  for (int i = tid; i < min(n, kAside); i += kThreads) {
    V v;
    v.from(aside[i]);
    if (v.top() < floor_) continue;
    float2 y[V::N / 2];
    v.get(y);
#pragma unroll
    for (int e = 0; e < V::N / 2; ++e) {
      put(y[e].x, v0 + head + aside_at[i] * V::N + 2 * e);
      put(y[e].y, v0 + head + aside_at[i] * V::N + 2 * e + 1);
    }
  }
  if (ragged) put(ragged_y, ragged_v);
  // The threads' sums, by the last warp (f64 is slow: thirteen additions instead of a
  // tree in every warp).
  float most = -INFINITY;
  double d = 0.0;
  if (warp == kWarps - 1) {
    float rs[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      rs[w] = refs[32 * w + lane];
      most = fmaxf(most, rs[w]);
    }
    most = warp_top(most);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float s = parts[32 * w + lane];
      d += (double)(rs[w] == -INFINITY ? s : s * ex2(rs[w] - most));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  }
  const bool writer = tid == kThreads - 32;
  __syncthreads();
  const int c = few_count;
  const bool all_there = n <= kAside && c <= kRanked;  // then at least K, or all above -inf
  if (all_there) {
    if (writer) *sum_out = SegSum{most, min(c, K), d};
    for (int k = tid; k < c; k += kThreads) {
      const unsigned long long mine = few[k];
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < c; ++i) rank += few[i] > mine;
      if (rank < K) list[rank] = mine;
    }
    return;
  }
  // Too many: place after place, the largest entry below the last one.
  unsigned long long last = ~0ull;
  int places = 0;
  for (; places < K; ++places) {
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
    if (mine == 0) break;  // no more
    last = mine;
    if (tid == 0) list[places] = mine;
    __syncthreads();
  }
  if (writer) *sum_out = SegSum{most, places, d};
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
  __shared__ float base_f[kBeamMaxW];
  __shared__ int counts[kBeamMaxW * kMaxSegs];
  __shared__ float least;
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x, K = p.K;
  const int lists = p.W * segs;  // at most kRoom
  attn::start_next_kernel();
  attn::wait_for_previous_kernel();
  const Ws ws = carve(p.ws, (int64_t)p.B * lists);
  const SegSum* sums = ws.sums + (int64_t)b * lists;
  const unsigned long long* list = ws.list + (int64_t)b * lists * K;
  if (tid == 0) count = 0;
  // Few entries are on their way while the sums are joined: a warp's lists, a lane per entry
  // (no division in the way; each would be a sixth of the time of all else).
  const int all = lists * K, warp = tid >> 5;
  constexpr int kAhead = 4;
  const bool ahead = lists <= kAhead * kWarps && K <= 32;
  unsigned long long entries[kAhead];
  if (ahead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int l = warp * kAhead + u;
      entries[u] = l < lists && lane < K ? list[l * K + lane] : 0;
    }
  }
  for (int w = tid >> 5; w < p.W; w += kWarps) {  // a warp per beam, a lane per segment
    SegSum x{-INFINITY, 0, 0.0};
    if (lane < segs) {
      x = sums[w * segs + lane];
      counts[w * segs + lane] = x.count;
    }
    float most = x.ref;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    // 2^(ref - most) from its bits; 0 from 2^-1023 on.
    const float e = x.ref - most + 1023.0f;
    double total = x.ref == -INFINITY ? x.sum : x.sum * __longlong_as_double(e > 0.0f ? (long long)e << 52 : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) {
      base[w] = total;
      base_f[w] = most;
    }
  }
  __syncthreads();
  // A lane per beam: f64 instructions of a warp take as long for one lane as for 32.
  if (tid < p.W) {
    // Nothing in the row, an infinity or a NaN: no score of it is finite.
    const double x = (double)p.scores[(int64_t)b * p.W + tid] -
                     ((double)base_f[tid] * (1.0 / (double)kH) + log(base[tid]));
    base[tid] = x;
    base_f[tid] = (float)x;
  }
  __syncthreads();
  auto score_of = [&](int w, unsigned long long e) -> unsigned long long {
    const double s = base[w] + (double)value_of((uint32_t)(e >> 32));
    return s - s == 0.0 ? order_of(s) : 0ull;
  };
  // In f32, to within 2^-22 (|base| + |s|); NaN: none.
  auto near_score = [&](int w, unsigned long long e) {
    const float s = base_f[w] + value_of((uint32_t)(e >> 32));
    return s - s == 0.0f ? s : __int_as_float(0x7fffffff);
  };
  // The K-th best head of a list is a score that K entries reach.  It is found in f32, and
  // entries that do not come near it are left out before any f64 arithmetic.
  float floor_ = -INFINITY;
  if (lists >= K && lists <= kThreads) {
    float* heads = reinterpret_cast<float*>(key);
    const float none = __int_as_float(0x7fffffff);
    if (ahead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int l = warp * kAhead + u;
        if (lane == 0 && l < lists) heads[l] = counts[l] > 0 ? near_score(l / segs, entries[u]) : none;
      }
    } else if (tid < lists) {
      heads[tid] = counts[tid] > 0 ? near_score(tid / segs, list[(int64_t)tid * K]) : none;
    }
    if (tid == 0) least = -INFINITY;
    __syncthreads();
    if (tid < lists) {
      const float mine = heads[tid];
      int rank = 0;  // equal heads by their number
#pragma unroll 8
      for (int i = 0; i < lists; ++i) rank += heads[i] > mine || (heads[i] == mine && i < tid);
      if (rank == K - 1 && mine == mine) least = mine;
    }
    __syncthreads();
    floor_ = least;
    float big = fabsf(floor_);
    for (int w = 0; w < p.W; ++w) big = fmaxf(big, fabsf(base_f[w]));  // (a NaN is passed over)
    floor_ -= big * 0x1p-20f;  // -inf stays
    __syncthreads();  // `key` is written again
  }
  // Beams that ended come first: one entry each.
  for (int w = tid; w < p.W; w += kThreads) {
    const float s = p.scores[(int64_t)b * p.W + w];
    if (p.finished != nullptr && p.finished[(int64_t)b * p.W + w] != 0 && fabsf(s) <= 3.402823466e38f) {
      const int at = atomicAdd(&count, 1);
      key[at] = order_of((double)s);
      index[at] = (uint32_t)(w * p.V + p.pad);
    }
  }
  auto take = [&](int w, unsigned long long e) {
    if (!(near_score(w, e) >= floor_)) return;
    const unsigned long long s = score_of(w, e);
    if (s != 0) {
      const int at = atomicAdd(&count, 1);
      key[at] = s;
      index[at] = (uint32_t)(w * p.V) + ~(uint32_t)e;
    }
  };
  auto write = [&](int k, unsigned long long s, uint32_t at) {
    const int64_t to = (int64_t)b * K + k;
    p.parents[to] = (int32_t)(at / (uint32_t)p.V);
    p.tokens[to] = (int32_t)(at % (uint32_t)p.V);
    p.out_scores[to] = (float)value_of(s);
  };
  int kept;
  if (ahead) {  // at most 32 x 32 + W entries
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int l = warp * kAhead + u;
      if (l < lists && lane < counts[l]) take(l / segs, entries[u]);
    }
    __syncthreads();
    const int n = count;
    kept = min(n, K);
    if (n <= kThreads) {  // by counting
      if (tid < n) {
        const unsigned long long mine = key[tid];
        const uint32_t at = index[tid];
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) rank += key[i] > mine || (key[i] == mine && index[i] < at);
        if (rank < K) write(rank, mine, at);
      }
    } else {
      sort_scores(key, index, n);
      for (int k = tid; k < kept; k += kThreads) write(k, key[k], index[k]);
    }
  } else {
    __syncthreads();
    kept = count;
    const int room = kRoom - kBeamMaxK;  // new ones of a pass; W <= kBeamMaxW <= kBeamMaxK
    for (int at0 = 0; at0 < all; at0 += room) {
      for (int i = at0 + tid; i < min(all, at0 + room); i += kThreads) {
        const int l = i / K;
        if (i - l * K < counts[l]) take(l / segs, list[i]);
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
    for (int k = tid; k < kept; k += kThreads) write(k, key[k], index[k]);
  }
  for (int k = kept + tid; k < K; k += kThreads) {
    const int64_t to = (int64_t)b * K + k;
    p.parents[to] = p.tokens[to] = -1;
    p.out_scores[to] = -INFINITY;
  }
}

// Segments of a row.  Twelve CTAs for each SM (four at a time) even out, while a segment of
// fewer than 4096 logits spends its time on the selection; the sums depend on the sizes
// alone.
int segments(int64_t rows, int64_t V) {
  const int64_t want = (12 * 152 + rows - 1) / rows, most = (V + 4095) / 4096;
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
  const dim3 grid((unsigned)segs, (unsigned)p.W, (unsigned)p.B);
  // (Both launches are prepared while the kernel before them still runs.)
  const cudaError_t e =
      p.bf16 ? attn::launch_after(beam_rows_kernel<__nv_bfloat16>, grid, kThreads, st, 0, p, seg_len)
             : attn::launch_after(beam_rows_kernel<float>, grid, kThreads, st, 0, p, seg_len);
  if (e != cudaSuccess) return e;
  return attn::launch_after(beam_join_kernel, dim3((unsigned)p.B), kThreads, st, 0, p, segs);
}

}  // namespace gdn
