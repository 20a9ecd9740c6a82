// gdn_attn8_wide.cu -- attention over a cache in 8 bits for many rows per kv head: the
// contexts are widened to the activation type, and the kernels of the wide cache run on
// them.
//
//   value = code * scale, exact in bf16 for the powers of two that the library writes
//   (an e4m3 code has 4 significant bits), else rounded once.
//
// A chunk's attention is bound by its products, 4 D flops for each row and key; widening a
// key and value moves 2 D (1 + 2) bytes once, whatever the rows.  So from a few hundred
// rows on it is a small part of the call: 2048 tokens over 32768 keys, 32 + 4 heads of 128,
// take 0.75 ms, of which the widening is 0.028 (39 MB of codes read, 77 MB written, 4.1 TB/s).
// Inside the attention kernel it would be repeated for every 256 rows, by the warps whose
// softmax is what binds there.  The number of rows from which it pays is kMostRows in
// gdn_attn8_tc.cu, with both sides.
//
// The workspace holds the contexts of some sequences at a time, up to 1 GiB or one
// sequence, whichever is more; each group of them is one pass of the two kernels.  The host knows
// the table's width, not the lengths, so a wide table makes small groups: 64 chunks of 100 tokens
// over 1000, 64 + 8 heads of 128, take 310 us with a table for 1024 positions, 440 with 8192 (two
// groups) and 3100 with 131072 (64 groups of one).
//
// f32 comes here with more rows than the row kernel holds (gdn_attn_simt.cu), single tokens of wide
// groups among them: 8 tokens over 4096 keys each, 2 kv heads of 128, take 200 us with 16 query
// heads to a kv head where 8 take 41 on the codes (floor 2.5); 64 tokens 923 and 243 (floor 20).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

using namespace attn;

constexpr int kThreads = 256;
constexpr int64_t kGroupBytes = (int64_t)1 << 30;

// 16 codes of a row times f, in T.
__device__ __forceinline__ void widen16(const uint4& c, float f, __nv_bfloat16* to) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = e4x2_to_f((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x * f, x.y * f);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  reinterpret_cast<uint4*>(to)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(to)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void widen16(const uint4& c, float f, float* to) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4x2_to_f(w[i] & 0xffffu), b = e4x2_to_f(w[i] >> 16);
    reinterpret_cast<float4*>(to)[i] = make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
  }
}

// A head's page blockIdx.x of sequence s0 + blockIdx.y, of K or V (blockIdx.z), into page
// blockIdx.y * max_pages + blockIdx.x of the workspace; its entry of the table there.
template <typename T>
__global__ void __launch_bounds__(kThreads) widen_kernel(const __grid_constant__ AttnLaunch p, int s0,
                                                         int32_t* table, T* k, T* v) {
  start_next_kernel();
  wait_for_previous_kernel();
  const int s = s0 + blockIdx.y, pi = blockIdx.x;
  const SeqRange q = seq_range(p, s);
  if (q.bad && pi == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadSeqlens);
  const int64_t to = (int64_t)blockIdx.y * p.max_pages + pi;
  if (threadIdx.x == 0 && blockIdx.z == 0) table[to] = (int32_t)to;
  const int rows = min(p.page_size, q.kv - pi * p.page_size);
  if (q.b <= q.a || rows <= 0) return;
  const int64_t pg = page_of(p, s, pi);
  if (pg < 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
  const int vecs = p.D / 16, n = rows * vecs;  // 16-code pieces of a head's rows
  // Head blockIdx.z of K, or Hkv + head of V.  Loads four at a time: one at a time, all heads
  // of a page by a CTA, took 37 us where HBM takes 17 (a chunk of 2048 over 32768 tokens).
  for (int z = blockIdx.z; z < 2 * p.Hkv; z += gridDim.z) {
    const bool of_v = z >= p.Hkv;
    const int h = of_v ? z - p.Hkv : z;
    const AttnPages& src = of_v ? p.vc : p.kc;
    const unsigned char* from = static_cast<const unsigned char*>(src.p) + pg * src.ps + (int64_t)h * src.hs;
    const float* scales = (of_v ? p.vs : p.ks) + scale_at(p.Hkv, p.page_size, p.block, max(pg, (int64_t)0), h, 0);
    T* out = (of_v ? v : k) + (to * p.Hkv + h) * p.page_size * p.D;
    constexpr int kAhead = 4;
    for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * kThreads) {
      uint4 c[kAhead];
      float f[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads, r = i / vecs;
        c[u] = make_uint4(0u, 0u, 0u, 0u);
        f[u] = 0.0f;
        if (i < n && pg >= 0) {  // a bad page reads as zeros
          c[u] = *reinterpret_cast<const uint4*>(from + (int64_t)r * src.ts + (i - r * vecs) * 16);
          f[u] = scales[r / p.block];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads;
        if (i < n) widen16(c[u], f[u], out + (int64_t)i * 16);
      }
    }
  }
}

int64_t seq_bytes(int64_t Hkv, int64_t D, bool bf16, int64_t max_pages, int64_t page_size) {
  return 2 * max_pages * page_size * Hkv * D * (bf16 ? 2 : 4);
}
int64_t group_of(int64_t N, int64_t Hkv, int64_t D, bool bf16, int64_t max_pages, int64_t page_size) {
  const int64_t one = seq_bytes(Hkv, D, bf16, max_pages, page_size);
  // (65535: the grid's second dimension; page numbers of a group stay below 2^31.)
  return std::max<int64_t>(
      1, std::min<int64_t>({N, kGroupBytes / one, (int64_t)65535, (int64_t)INT32_MAX / max_pages}));
}
size_t table_bytes(int64_t seqs, int64_t max_pages) {
  return ((size_t)(seqs * max_pages) * 4 + 255) & ~(size_t)255;
}

template <typename T>
cudaError_t run(const AttnLaunch& p, cudaStream_t st) {
  const int64_t group = group_of(p.N, p.Hkv, p.D, p.bf16, p.max_pages, p.page_size);
  const int64_t half = seq_bytes(p.Hkv, p.D, p.bf16, p.max_pages, p.page_size) / 2 * group;
  char* ws = static_cast<char*>(p.ws);
  int32_t* table = reinterpret_cast<int32_t*>(ws);
  T* k = reinterpret_cast<T*>(ws + table_bytes(group, p.max_pages));
  T* v = reinterpret_cast<T*>(reinterpret_cast<char*>(k) + half);
  for (int64_t s0 = 0; s0 < p.N; s0 += group) {
    const int ns = (int)std::min<int64_t>(group, p.N - s0);
    cudaError_t e = launch_after(widen_kernel<T>, dim3((unsigned)p.max_pages, (unsigned)ns, (unsigned)std::min(2 * p.Hkv, 65535)), kThreads, st,
                                 0, p, (int)s0, table, k, v);
    if (e != cudaSuccess) return e;
    AttnLaunch w = p;
    w.N = ns;
    w.part = ns != p.N;
    w.kv_lens = p.kv_lens + s0;
    if (p.cu != nullptr) {
      w.cu = p.cu + s0;
    } else {  // a token per sequence
      w.T = ns;
      w.part = false;
      w.q.p = static_cast<const T*>(p.q.p) + s0 * p.q.ts;
      if (p.gate.p != nullptr) w.gate.p = static_cast<const T*>(p.gate.p) + s0 * p.gate.ts;
      w.out = static_cast<T*>(p.out) + s0 * p.Hq * p.D;
      if (p.lse != nullptr) w.lse = p.lse + s0 * p.Hq;
    }
    w.table = table;
    w.table_stride = p.max_pages;
    w.num_pages = (int64_t)ns * p.max_pages;
    w.kc = AttnPages{k, (int64_t)p.Hkv * p.page_size * p.D, (int64_t)p.page_size * p.D, p.D};
    w.vc = AttnPages{v, w.kc.ps, w.kc.hs, w.kc.ts};
    w.ks = w.vs = nullptr;
    w.block = 0;
    w.ws = reinterpret_cast<char*>(v) + half;
    e = attn_tc_supported(w) ? launch_attn_tc(w, st) : launch_attn_simt(w, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t attn8_wide_workspace_bytes(int64_t T, int64_t N, int64_t Hq, int64_t Hkv, int64_t D,
                                  int64_t max_q, bool bf16, int64_t max_pages, int64_t page_size) {
  const int64_t group = group_of(N, Hkv, D, bf16, max_pages, page_size);
  // Fewer sequences may be cut into more key ranges: the last group's need counts, too.
  size_t inner = 0;
  for (int64_t ns : {group, N % group})
    for (int64_t t : {T, ns}) {  // (ns tokens: of a call without offsets)
      if (ns == 0) continue;
      inner = std::max(inner, attn_simt_workspace_bytes(t, ns, Hq, Hkv, D, max_q));
      if (bf16) inner = std::max(inner, attn_tc_workspace_bytes(t, ns, Hq, Hkv, D, max_q));
    }
  return table_bytes(group, max_pages) +
         (size_t)(group * seq_bytes(Hkv, D, bf16, max_pages, page_size)) + inner;
}

cudaError_t launch_attn8_wide(const AttnLaunch& p, cudaStream_t st) {
  return p.bf16 ? run<__nv_bfloat16>(p, st) : run<float>(p, st);
}

}  // namespace gdn
