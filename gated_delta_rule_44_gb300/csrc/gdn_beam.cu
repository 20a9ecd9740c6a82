// gdn_beam.cu -- beam search's selection: the K best continuations (beam, token) of each
// group of W beams,
//   s[w, v] = score[w] + x[w, v] - ln sum_u e^{x[w, u]},
// in one pass over the logits.
//
// Row kernel.  The rows' chunks of 1024 vectors of 16 bytes, one row after another, are
// divided equally among two CTAs per SM, and a CTA's part of a row is a segment of it.  Each
// thread copies its vectors three chunks ahead into shared memory (asynchronously, past
// segments' ends, so that reading goes on while a segment is finished; rows that take no part
// are not read), and keeps a running sum of 2^(H x - ref) (f32), H = log2(e) rounded to f32 and
// ref a whole number: H x - ref is one rounding (an fma), changes of ref and joins are exact,
// and ln sum e^x = ref / H + ln(sum) to within the 1.3e-8 (largest x - x) that H's rounding
// leaves, where x has its weight.  So an element costs half of an fma, an exponential and
// half of an add.  A chunk's terms are added as a tree, and the chunks' sums with what each addition
// loses (Knuth's two-sum): one after another, 256 equal terms of a flat row of 131072 were off by
// 2.4e-6 together.  The threads' sums are joined in f64.  (Where a row is cut, and where its first
// 16-byte boundary lies, still decides which terms meet: equal rows may differ by some 2^-22.)
// Past 2^22 a whole number near H x is no longer near the product (from 2^32 on the fma's result may
// be in the hundreds).  So ref is -2^22 at least, where what is further down (a mask) has no
// weight beside anything else; and a segment whose largest logit itself is beyond 2^22 on
// either side sums 2^(H (x - top)), top its largest logit, by reading it once more ("far").
// The segment's K largest logits: while it reads, a thread notes only its largest logit of each
// chunk.  Then every warp gives the n-th largest of its threads' maxima, n warps' shares of
// K, and the least of these is a value that at least K logits reach; the some 3 K chunks of
// a thread that reach it are read again, and their logits that do are ranked by counting.
// (Putting vectors aside on the way took 13 us of 42 for K = 16: each time the warp waits.)
// A segment in which more reach it than there is room for (rows of equal logits; a finite mask over
// all but fewer than K tokens, the mask then being the floor) is read again, once for each of the K
// places: 64 x 8 rows of 131072 with 20 tokens above a mask of -1e9 take 1050 us, with 1000 of them 66.
//
// Join kernel.  A CTA per group joins the segments' sums into f64 log-sums, turns list
// entries into 64-bit scores (beams are compared at 2^-53: two f32 roundings of a score of
// -12 already span what separates neighbours), those that can be among the K, and ranks
// them.  Order: score, then the lower w V + v; keys are integers, since f64 comparisons
// are a sixty-fourth of their rate.
//
// Bound by the read of the logits in the end; now by the instructions and their latency: 64 x 8
// rows of 131072 bf16 (134 MB, 20 us) take 38.5 us with K = 16, some 9 of them the join's and
// what goes on around it, and 35 with K = 2; f32 (268 MB, 40 us) 55.  A stage more or less
// and chunks of 2048 vectors are within 2 %; chunks of 512 took 46.  (The care for far segments takes
// 0.9 of the 38.5, sums that keep what they lose 0.5.)
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
constexpr int kCells = 16;      // chunks between two looks at their maxima
constexpr int kRanked = 1024;   // logits ranked by counting
constexpr int kFound = 512;     // cells read again
constexpr int kRoom = 2048;     // entries of the join's sorts
constexpr int kMaxSegs = 32;    // a lane each
constexpr int kStages = 3;      // chunks of a CTA on their way
constexpr int kChunk = kThreads * kUnroll;  // vectors
constexpr int kCtasPerSm = 2;
constexpr float kH = 1.4426950408889634f;  // log2(e) in f32
constexpr float kFarRef = 4194304.0f;
constexpr int kFar = 1 << 30;

// What a segment leaves: the count of its list's entries (value key, ~index), and its sum of
// 2^(H x - ref) (ref -inf: nothing is above that).  A far segment, kFar in `count`: of
// 2^(H (x - ref)).
struct SegSum {
  float ref;
  int count;
  double sum;
};
struct Ws {
  SegSum* sums;               // [rows][segs]
  unsigned long long* list;   // [rows][segs][K]
};
// The rows' chunks, one row after another, in equal ranges for the CTAs.
struct Split {
  int64_t chunks;  // of all rows
  int per_row, ctas, segs;  // segs: a row's segments at most
};
__device__ __forceinline__ int64_t range_begin(const Split& s, int cta) {
  return (int64_t)((uint64_t)s.chunks * (uint32_t)cta / (uint32_t)s.ctas);
}
// The CTA whose range holds a chunk: the last one that begins at or before it.
__device__ __forceinline__ int cta_of(const Split& s, int64_t chunk) {
  return (int)(((uint64_t)(chunk + 1) * (uint32_t)s.ctas - 1) / (uint64_t)s.chunks);
}
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
  __device__ void from(const uint4& b) { r = b; }
  __device__ void fill() { r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }  // -inf
  __device__ __nv_bfloat162 tops() const {  // (a NaN counts only beside another)
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&r);
    return __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
  }
  static __device__ __nv_bfloat162 larger(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2(a, b); }
  static __device__ float top_of(__nv_bfloat162 m) {
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);  // (-inf of NaN)
  }
  __device__ float top() const { return top_of(tops()); }
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
  __device__ void from(const uint4& b) { r = *reinterpret_cast<const float4*>(&b); }
  __device__ void fill() { r = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ float tops() const { return fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w)); }
  static __device__ float larger(float a, float b) { return fmaxf(a, b); }
  static __device__ float top_of(float m) { return fmaxf(m, -INFINITY); }
  __device__ float top() const { return top_of(tops()); }
};
// The largest logit of vectors; -inf of NaN alone.
template <typename V, int N>
__device__ __forceinline__ float top_of(const V (&v)[N]) {
  auto m = v[0].tops();
#pragma unroll
  for (int i = 1; i < N; ++i) m = V::larger(m, v[i].tops());
  return V::top_of(m);
}

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
struct RowShared {
  uint4 ring[kStages][kUnroll][kThreads];
  unsigned long long few[2][kRanked];  // of every other segment
  unsigned long long best[kWarps];
  float refs[kThreads], parts[kThreads];
  float cells[kCells][kThreads];  // each thread's largest logit of a chunk
  float floors[kWarps];           // values that a warp's share of K logits has reached
  double far[kWarps];             // a far segment's sums
  float most;                     // the segment's largest ref
  int few_count[2], found_count;
  uint16_t found[kFound];  // cells that reach the floor
};

// A row as both cursors see it.
template <typename T>
struct Row {
  const T* x;
  int head, vecs;  // logits before the first 16-byte boundary, whole vectors behind it
  bool takes_part;
  __device__ void set(const BeamLaunch& p, int64_t row, float score, bool ended) {
    const int64_t b = row / p.W, w = row - b * p.W;
    x = static_cast<const T*>(p.logits) + b * p.batch_stride + w * p.beam_stride;
    const int mis = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    head = min(p.V, mis ? Vec<T>::N - mis : 0);
    vecs = (p.V - head) / Vec<T>::N;
    takes_part = fabsf(score) <= 3.402823466e38f && !ended;
  }
};

// 16 bytes that are read once: they leave L2 before others.
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from), "l"(policy)
               : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
beam_rows_kernel(const __grid_constant__ BeamLaunch p, const __grid_constant__ Split split) {
  extern __shared__ __align__(16) unsigned char smem[];
  RowShared<T>& sh = *reinterpret_cast<RowShared<T>*>(smem);
  attn::start_next_kernel();
  attn::wait_for_previous_kernel();
  using V = Vec<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = p.K, U = split.per_row;
  const int64_t rows = (int64_t)p.B * p.W;
  const Ws ws = carve(p.ws, rows * split.segs);
  const int64_t first = range_begin(split, blockIdx.x);
  int left = (int)(range_begin(split, blockIdx.x + 1) - first);  // chunks to work on
  int64_t row = first / U;
  int u0 = (int)(first - row * U);  // and where in the row

  // The copies run kStages chunks ahead, through the rows' ends: every thread copies the
  // vectors that it will read itself, so that they need no barrier.
  auto ended = [&](int64_t r) { return p.finished != nullptr && p.finished[r] != 0; };
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&sh.ring[0][0][tid]);
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  int64_t copy_row = row;
  int copy_u = u0, copy_left = left;
  Row<T> from;
  from.set(p, row, p.scores[row], ended(row));
  float next_score = row + 1 < rows ? p.scores[row + 1] : 0.0f;
  bool next_ended = row + 1 < rows && ended(row + 1);
  auto copy = [&](int stage) {
    if (copy_left > 0) {
      if (from.takes_part) {
        const int i = copy_u * kChunk + tid;
        const T* src = from.x + from.head + (int64_t)i * V::N;
        const uint32_t to = ring + stage * (kUnroll * kThreads * 16);
        if ((copy_u + 1) * kChunk <= from.vecs) {
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) copy_async(to + u * kThreads * 16, src + u * kThreads * V::N, policy);
        } else {
#pragma unroll
          for (int u = 0; u < kUnroll; ++u)
            if (i + u * kThreads < from.vecs) copy_async(to + u * kThreads * 16, src + u * kThreads * V::N, policy);
        }
      }
      --copy_left;
      if (++copy_u == U && copy_left > 0) {
        copy_u = 0;
        ++copy_row;
        from.set(p, copy_row, next_score, next_ended);
        if (copy_row + 1 < rows) {
          next_score = p.scores[copy_row + 1];
          next_ended = ended(copy_row + 1);
        }
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) copy(i);
  int stage = 0;

  int side = 0;
  for (; left > 0; ++row, u0 = 0) {
    const int u1 = min(U, u0 + left);
    left -= u1 - u0;
    Row<T> r;
    r.set(p, row, p.scores[row], ended(row));
    const int64_t at = row * split.segs + (u0 == 0 ? 0 : (int)blockIdx.x - cta_of(split, row * U));
    SegSum* sum_out = ws.sums + at;
    unsigned long long* list = ws.list + at * K;
    // A row's last segment also leaves the places behind it empty.
    if (u1 == U) {
      const int64_t end = (row + 1) * split.segs;
      for (int64_t i = at + 1 + tid; i < end; i += kThreads) ws.sums[i] = SegSum{-INFINITY, 0, 0.0};
    }
    if (!r.takes_part) {
      if (tid == 0) *sum_out = SegSum{-INFINITY, 0, 0.0};
      for (int u = u0; u < u1; ++u) {
        copy(stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }
      continue;
    }
    unsigned long long* few = sh.few[side];
    if (tid == 0) sh.few_count[side] = sh.found_count = 0;  // (counted behind the next barrier)
    bool crowded = false;   // more found than there is room for
    float top = -INFINITY;  // this thread's largest logit
    float ref = -INFINITY;  // its sum of 2^(H x - ref), and what the sum's additions lost
    float sum = 0.0f, lost = 0.0f;
    float use = 0.0f;          // -ref, or 0 while that is -inf
    float floor_ = -INFINITY;  // logits below it are not among the segment's K
    auto raise = [&](float y) {
      if (y > top) {
        top = y;
        const float up = fmaxf(ceilf(y * kH), -kFarRef);
        if (up > ref) {
          if (ref != -INFINITY) {  // (a sum of NaN stays one)
            const float f = ex2(ref - up);
            sum *= f;
            lost *= f;
          }
          ref = up;
          use = -up;
        }
      }
    };
    auto add = [&](float x) {
      const float s = sum + x, z = s - sum;
      lost += (sum - (s - z)) + (x - z);
      sum = s;
    };
    auto work = [&](int u, bool whole) {
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
      const int i = u * kChunk + tid;
      V v[kUnroll];
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        v[e].from(sh.ring[stage][e][tid]);
        if (!whole && i + e * kThreads >= r.vecs) v[e].fill();
      }
      const float most = top_of(v);
      sh.cells[(u - u0) % kCells][tid] = most;
      raise(most);
      copy(stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const float2 h2 = {kH, kH}, use2 = {use, use};
      float2 of[kUnroll];
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        float2 y[V::N / 2];
        v[e].get(y);
#pragma unroll
        for (int k = 0; k < V::N / 2; ++k) {
          const float2 t = __ffma2_rn(y[k], h2, use2);
          y[k] = float2{ex2(t.x), ex2(t.y)};
        }
#pragma unroll
        for (int n = V::N / 4; n > 0; n /= 2)
#pragma unroll
          for (int k = 0; k < n; ++k) y[k] = __fadd2_rn(y[k], y[k + n]);
        of[e] = y[0];
      }
      const float2 all = __fadd2_rn(__fadd2_rn(of[0], of[1]), __fadd2_rn(of[2], of[3]));
      add(all.x + all.y);
    };
    // A logit that reaches the floor, to be ranked.
    auto put = [&](float y, int v) {
      if (y >= floor_ && y > -INFINITY) {
        const int to = atomicAdd(&sh.few_count[side], 1);
        if (to < kRanked) few[to] = entry(y, (uint32_t)v);
      }
    };
    // The warps with a vector for every thread of theirs (one at least) take their shares of K.
    const int warps = max(1, min(kWarps, (min(r.vecs, u1 * kChunk) - u0 * kChunk) / 32));
    const int share = (K + warps - 1) / warps;
    // What the row has before its first vector and behind its last: fewer than 16 logits.
    const int heads = u0 == 0 ? r.head : 0, tail0 = r.head + r.vecs * V::N;
    const bool ragged = tid < heads + (u1 == U ? p.V - tail0 : 0);
    const int ragged_v = tid < heads ? tid : tail0 + tid - heads;
    const float ragged_y = ragged ? attn::to_f(r.x[ragged_v]) : -INFINITY;
    for (int u = u0; u < u1;) {
      const int c0 = u, c1 = min(u1, u + kCells);
      for (; u < c1; ++u) {
        if ((u + 1) * kChunk <= r.vecs) work(u, true);
        else work(u, false);
      }
      const bool end = u == u1;
      if (end) {
        if (ragged) {
          raise(ragged_y);
          add(ex2(fmaf(ragged_y, kH, use)));
        }
        sh.refs[tid] = ref;
        sh.parts[tid] = sum + lost;
      }
      const float mine = warp < warps ? nth_top(top, share) : INFINITY;
      if (lane == 0) sh.floors[warp] = mine;
      __syncthreads();
      floor_ = sh.floors[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) floor_ = fminf(floor_, sh.floors[w]);
      if (end && ragged) put(ragged_y, ragged_v);
      // The chunks' vectors with a logit that reaches the floor are listed, and come again from
      // L2, one to a thread.
      if (top >= floor_ && top > -INFINITY) {
#pragma unroll 4
        for (int c = 0; c < c1 - c0; ++c) {
          const float most = sh.cells[c][tid];
          if (most >= floor_ && most > -INFINITY) {
            const int to = atomicAdd(&sh.found_count, 1);
            if (to < kFound) sh.found[to] = (uint16_t)(c * kThreads + tid);
          }
        }
      }
      __syncthreads();
      const int found = sh.found_count;
      crowded |= found > kFound;
      for (int j = tid; j < min(found, kFound) * kUnroll; j += kThreads) {
        const int cell = sh.found[j / kUnroll];
        const int i = (c0 + cell / kThreads) * kChunk + j % kUnroll * kThreads + cell % kThreads;
        if (i >= r.vecs) continue;
        V v;
        v.load(r.x + r.head + (int64_t)i * V::N);
        if (!(v.top() >= floor_)) continue;
        float2 y[V::N / 2];
        v.get(y);
#pragma unroll
        for (int k = 0; k < V::N / 2; ++k) {
          put(y[k].x, r.head + i * V::N + 2 * k);
          put(y[k].y, r.head + i * V::N + 2 * k + 1);
        }
      }
      if (!end) {
        __syncthreads();
        if (tid == 0) sh.found_count = 0;  // (counted behind the next floors' barrier)
      }
    }
    // The threads' sums, by the last warp (f64 is slow: thirteen additions instead of a
    // tree in every warp).
    float most = -INFINITY;
    double d = 0.0;
    if (warp == kWarps - 1) {
      float rs[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        rs[w] = sh.refs[32 * w + lane];
        most = fmaxf(most, rs[w]);
      }
      most = warp_top(most);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float s = sh.parts[32 * w + lane];
        d += (double)(rs[w] == -INFINITY ? s : s * ex2(rs[w] - most));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    }
    const bool writer = tid == kThreads - 32;
    if (writer) sh.most = most;
    __syncthreads();
    const int v0 = u0 == 0 ? 0 : r.head + u0 * kChunk * V::N;
    const uint32_t v1 = u1 == U ? p.V : r.head + u1 * kChunk * V::N;
    const bool far = sh.most > kFarRef || sh.most == -kFarRef;
    if (far) {
      const float mine = warp_top(top);
      if (lane == 0) sh.floors[warp] = mine;
      __syncthreads();
      most = sh.floors[0];
      for (int w = 1; w < kWarps; ++w) most = fmaxf(most, sh.floors[w]);
      d = 0.0;
      for (uint32_t v = v0 + tid; v < v1; v += kThreads) d += (double)ex2((attn::to_f(r.x[v]) - most) * kH);
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (lane == 0) sh.far[warp] = d;
      __syncthreads();
      d = 0.0;
      for (int w = 0; w < kWarps; ++w) d += sh.far[w];
    }
    const int c = sh.few_count[side];
    int places = min(c, K);
    if (!crowded && c <= kRanked) {  // at least K, or all above -inf
      for (int k = tid; k < c; k += kThreads) {
        const unsigned long long mine = few[k];
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < c; ++i) rank += few[i] > mine;
        if (rank < K) list[rank] = mine;
      }
    } else {
      // Too many: place after place, the largest entry below the last one.
      unsigned long long last = ~0ull;
      for (places = 0; places < K; ++places) {
        unsigned long long mine = 0;
        for (uint32_t v = v0 + tid; v < v1; v += kThreads) {
          const float y = attn::to_f(r.x[v]);
          if (y > -INFINITY) {
            const unsigned long long e = entry(y, v);
            if (e < last && e > mine) mine = e;
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long other = __shfl_xor_sync(0xffffffffu, mine, o);
          mine = other > mine ? other : mine;
        }
        if (lane == 0) sh.best[warp] = mine;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) mine = sh.best[w] > mine ? sh.best[w] : mine;
        if (mine == 0) break;  // no more
        last = mine;
        if (tid == 0) list[places] = mine;
        __syncthreads();
      }
    }
    if (writer) *sum_out = SegSum{most, places | (far ? kFar : 0), d};
    // The warps that have none to rank go on: `few` is filled anew two segments on, and the rest
    // behind the barriers above.
    side ^= 1;
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

// A beam's segments with a far one among them: the logit that their joined sum refers to.
// By a warp, a lane per segment; `total`: the lane's part of the sum.
__device__ __noinline__ double far_join(const SegSum& x, double& total) {
  const double at = x.count & kFar ? (double)x.ref : (double)x.ref * (1.0 / (double)kH);
  double most = at;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
  total = at == -INFINITY ? x.sum : x.sum * exp2((at - most) * (double)kH);  // (NaN of an infinity)
  return most;
}

// What limits the join is fetching its own instructions, so loops are not unrolled.
struct JoinShared {
  unsigned long long list[kRoom];
  unsigned long long key[kRoom];
  uint32_t index[kRoom];
  float heads[8 * kThreads];  // [level][list]
  double base[kBeamMaxW];     // score - log of the sum of each beam; NaN: takes no part
  double at[kBeamMaxW];       // the logit that the sum refers to
  float base_f[kBeamMaxW], at_f[kBeamMaxW];
  int counts[kBeamMaxW * kMaxSegs];
  uint32_t least;
  int count;
};
__global__ void __launch_bounds__(kThreads)
beam_join_kernel(const __grid_constant__ BeamLaunch p, const __grid_constant__ Split split) {
  extern __shared__ __align__(16) unsigned char smem[];
  JoinShared& sh = *reinterpret_cast<JoinShared*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x, K = p.K, segs = split.segs;
  const int lists = p.W * segs, all = lists * K;  // at most kRoom lists
  attn::start_next_kernel();
  attn::wait_for_previous_kernel();
  const Ws ws = carve(p.ws, (int64_t)p.B * lists);
  const SegSum* sums = ws.sums + (int64_t)b * lists;
  const unsigned long long* list = ws.list + (int64_t)b * all;
  // The entries come while the sums are joined, if there is room for them.
  const bool here = all <= kRoom;
  if (here) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(sh.list);
#pragma unroll 1
    for (int i = tid; i < all; i += kThreads)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to + i * 8), "l"(list + i) : "memory");
    list = sh.list;
  }
  float score = 0.0f;
  bool ended = false;
  if (tid < p.W) {
    score = p.scores[(int64_t)b * p.W + tid];
    ended = p.finished != nullptr && p.finished[(int64_t)b * p.W + tid] != 0;
  }
  if (tid == 0) {
    sh.count = 0;
    sh.least = 0;
  }
#pragma unroll 1
  for (int w = warp; w < p.W; w += kWarps) {  // a warp per beam, a lane per segment
    SegSum x{-INFINITY, 0, 0.0};
    if (lane < segs) {
      x = sums[w * segs + lane];
      sh.counts[w * segs + lane] = x.count & ~kFar;
    }
    double total, at;
    if (!__any_sync(0xffffffffu, x.count & kFar)) {
      const float most = warp_top(x.ref);
      // 2^(ref - most) from its bits; 0 from 2^-1023 on.
      const float e = x.ref - most + 1023.0f;
      total = x.ref == -INFINITY ? x.sum : x.sum * __longlong_as_double(e > 0.0f ? (long long)e << 52 : 0);
      at = (double)most * (1.0 / (double)kH);
    } else {
      at = far_join(x, total);
    }
#pragma unroll 1
    for (int o = segs > 1 ? 1 << (31 - __clz(segs - 1)) : 0; o > 0; o >>= 1)
      total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) {
      sh.base[w] = total;
      sh.at[w] = at;
    }
  }
  __syncthreads();
  // A lane per beam: f64 instructions of a warp take as long for one lane as for 32.
  if (tid < p.W) {
    // Nothing in the row, an infinity or a NaN: no score of it is finite.
    const double x = (double)score - log(sh.base[tid]);
    sh.base[tid] = x;
    sh.base_f[tid] = (float)x;
    sh.at_f[tid] = (float)sh.at[tid];
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  __syncthreads();
  // base + (x - at) in f32, to within 2^-24 (|base| + |at| + |x - at| + |s|), of which the third is no
  // more than the first and the last; NaN or an infinity: none.
  auto near_score = [&](int l, unsigned long long e) {
    return sh.base_f[l / segs] + (value_of((uint32_t)(e >> 32)) - sh.at_f[l / segs]);
  };
  // If j entries of each of r lists reach a score, K = r j do: for j = 1, 2, 4, ..., the r-th
  // best of the lists' j-th entries is a floor, and the highest of these floors is taken.
  // It is found in f32, and entries that do not come near it are left out before any f64
  // arithmetic.
  float floor_ = -3.402823466e38f;
  if (lists <= kThreads) {
    const int heads = (32 - __clz(K)) * lists;  // 8 levels at most
#pragma unroll 1
    for (int i = tid; i < heads; i += kThreads) {
      const int level = i / lists, l = i - level * lists, k = (1 << level) - 1;
      sh.heads[i] = k < sh.counts[l] ? near_score(l, list[(int64_t)l * K + k]) : -INFINITY;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < heads; i += kThreads) {
      const int level = i / lists;
      const float mine = sh.heads[i];
      int reach = 0;
#pragma unroll 4
      for (int l = 0; l < lists; ++l) reach += sh.heads[level * lists + l] >= mine;
      if (fabsf(mine) <= 3.402823466e38f && reach << level >= K) atomicMax(&sh.least, order_of(mine));
    }
    __syncthreads();
    if (sh.least != 0) {
      floor_ = value_of(sh.least);
      float big = fabsf(floor_);
#pragma unroll 1
      for (int w = 0; w < p.W; ++w) {  // (a NaN is passed over; infinite ones have no entries)
        const float f = fabsf(sh.base_f[w]), at = fabsf(sh.at_f[w]);
        if (f <= 3.402823466e38f) big = fmaxf(big, f);
        if (at <= kFarRef) big = fmaxf(big, at);  // (a far segment's is an f32)
      }
      floor_ = fmaxf(floor_ - big * 0x1p-20f, -3.402823466e38f);
    }
  }
  // Beams that ended come first: one entry each.
  if (ended && fabsf(score) <= 3.402823466e38f) {
    const int at = atomicAdd(&sh.count, 1);
    sh.key[at] = order_of((double)score);
    sh.index[at] = (uint32_t)(tid * p.V + p.pad);
  }
  __syncthreads();
  int kept = sh.count;  // scored entries in front
  // Entries are put behind those with their beam in `index`, and then scored, a thread each.
  // A list holds at most K, and `key` the K best of what came before and kRoom / 2 more.
  int l0 = 0;
  do {
    __syncthreads();  // `count` is `kept`
    const int step = here ? lists : max(1, kRoom / 2 / K);
#pragma unroll 1
    for (int l = l0 + warp; l < min(lists, l0 + step); l += kWarps) {
#pragma unroll 1
      for (int k = lane; k < sh.counts[l]; k += 32) {
        const unsigned long long e = list[(int64_t)l * K + k];
        const float s = near_score(l, e);
        if (s >= floor_ && s <= 3.402823466e38f) {
          const int at = atomicAdd(&sh.count, 1);
          sh.key[at] = e;
          sh.index[at] = l / segs;
        }
      }
    }
    l0 += step;
    __syncthreads();
    const int n = sh.count;
#pragma unroll 1
    for (int i = kept + tid; i < n; i += kThreads) {
      const unsigned long long e = sh.key[i];
      const uint32_t w = sh.index[i];
      sh.key[i] = order_of(sh.base[w] + ((double)value_of((uint32_t)(e >> 32)) - sh.at[w]));
      sh.index[i] = w * p.V + ~(uint32_t)e;
    }
    __syncthreads();
    if (n > kThreads || l0 < lists) {
      if (n > kept || kept > K) sort_scores(sh.key, sh.index, n);
      kept = min(n, K);
      if (tid == 0) sh.count = kept;
    } else {
      kept = n;
    }
  } while (l0 < lists);
  __syncthreads();
  // (few are ranked by counting, more have been sorted)
  const int n = sh.count;
  auto write = [&](int k, unsigned long long s, uint32_t at) {
    const int64_t to = (int64_t)b * K + k;
    const uint32_t w = at / (uint32_t)p.V;
    p.parents[to] = (int32_t)w;
    p.tokens[to] = (int32_t)(at - w * (uint32_t)p.V);
    p.out_scores[to] = (float)value_of(s);
  };
  if (tid < n && n <= kThreads) {
    const unsigned long long mine = sh.key[tid];
    const uint32_t at = sh.index[tid];
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) rank += sh.key[i] > mine || (sh.key[i] == mine && sh.index[i] < at);
    if (rank < K) write(rank, mine, at);
  }
  for (int k = min(n, K) + tid; k < K; k += kThreads) {
    const int64_t to = (int64_t)b * K + k;
    p.parents[to] = p.tokens[to] = -1;
    p.out_scores[to] = -INFINITY;
  }
}

// The CTAs share the chunks equally, but a row has at most 30 of them (a lane each in the
// join).
Split split_rows(int64_t rows, int64_t V, bool bf16) {
  const int64_t chunk = kChunk * (bf16 ? 8 : 4);
  Split s;
  s.per_row = (int)((V + chunk - 1) / chunk);
  s.chunks = rows * s.per_row;
  s.ctas = (int)std::min<int64_t>({kCtasPerSm * 152, s.chunks, (kMaxSegs - 2) * rows});
  s.segs = (int)std::min<int64_t>(s.per_row, s.ctas / rows + (s.ctas % rows ? 2 : 0));
  return s;
}

template <typename T>
cudaError_t launch_rows(const BeamLaunch& p, const Split& s, cudaStream_t st) {
  constexpr size_t smem = sizeof(RowShared<T>);
  static_assert(kCtasPerSm * (smem + 1024) <= 228 * 1024, "CTAs of an SM");
  static std::atomic<uint64_t> devices{0};
  const cudaError_t e = attn::allow_shared(beam_rows_kernel<T>, smem, devices);
  if (e != cudaSuccess) return e;
  return attn::launch_after(beam_rows_kernel<T>, dim3((unsigned)s.ctas), kThreads, st, smem, p, s);
}

}  // namespace

size_t beam_workspace_bytes(int64_t B, int64_t W, int64_t V, int64_t K) {
  // Of both types (f32 has more chunks), and as much for any smaller sizes: segs <= per_row, and
  // rows * segs <= ctas + 2 rows.
  const int64_t rows = B * W;
  const int64_t lists = std::min<int64_t>(rows * split_rows(rows, V, false).per_row, kCtasPerSm * 152 + 2 * rows);
  return (size_t)(lists * ((int64_t)sizeof(SegSum) + 8 * K));
}

cudaError_t launch_beam(const BeamLaunch& p, cudaStream_t st) {
  const Split s = split_rows((int64_t)p.B * p.W, p.V, p.bf16);
  // (Both launches are prepared while the kernel before them still runs.)
  cudaError_t e =
      p.bf16 ? launch_rows<__nv_bfloat16>(p, s, st) : launch_rows<float>(p, s, st);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = sizeof(JoinShared);
  static std::atomic<uint64_t> devices{0};
  e = attn::allow_shared(beam_join_kernel, smem, devices);
  if (e != cudaSuccess) return e;
  return attn::launch_after(beam_join_kernel, dim3((unsigned)p.B), kThreads, st, smem, p, s);
}

}  // namespace gdn
