// gdn_attn_stream.cuh -- what the tensor-core attention kernels share: bounded waits of
// whole warps, elected issue, and the stream form's work, in which the key tiles of all
// (sequence, kv head) pairs, in order, are cut into equal consecutive ranges, one per CTA,
// whatever the lengths.  A pair cut between CTAs leaves its sums in a workspace, and a
// second kernel joins them in the order of their keys.  A sequence with more than tq new
// tokens makes a pair of its own for every tq of them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"
#include "tcgen05.cuh"

namespace gdn {
namespace attn {

using namespace umma;

constexpr long long kWaitBudget = 2000000000LL;  // ~1 s of SM clock per wait
constexpr int BK = 128;                          // keys per tile

// A range of key tiles of one (tile, kv head).
struct Seg {
  int s, hkv, t0, nt, pos0, hi, kt0, kt1;  // s < 0: no more
  int64_t slot;  // workspace block of its sums; -1: it has every key of its rows
};

__device__ __forceinline__ int key_tiles(const SeqRange& q) {
  return q.b > q.a ? (q.kv + BK - 1) / BK : 0;
}
// TILES: a sequence's tokens may be several tiles of tq; else they are one (and the rest is as it
// was without them, for the wide cache).
template <bool TILES>
__device__ __forceinline__ int row_tiles(const AttnLaunch& p, const SeqRange& q, int tq) {
  return !TILES ? 1 : (min(q.b - q.a, p.max_q) + tq - 1) / tq;
}

// The ranges of one CTA of the stream form.
template <bool TILES>
struct SegIter {
  int s, hkv, rt, u, cta, tq;
  int64_t left;
  __device__ bool next(const AttnLaunch& p, Seg& g) {
    if (left <= 0) return false;
    SeqRange q;
    int n;
    for (;; ++s) {
      if (s >= p.N) return false;
      q = seq_range(p, s);
      n = key_tiles(q);
      if (n > 0) break;
    }
    const int take = (int)min((int64_t)(n - u), left);
    g.s = s;
    g.hkv = hkv;
    const int t = TILES ? rt * tq : 0;
    g.t0 = q.a + t;
    g.nt = min(q.b - q.a, p.max_q) - t;
    if (TILES) g.nt = min(g.nt, tq);
    g.pos0 = q.kv - (q.b - q.a) + t;
    g.hi = q.kv;
    g.kt0 = u;
    g.kt1 = u + take;
    g.slot = take == n ? -1 : 2 * (int64_t)cta + (u == 0 ? 1 : 0);
    left -= take;
    u += take;
    if (u == n) {
      u = 0;
      if (!TILES || ++rt == row_tiles<TILES>(p, q, tq)) {
        rt = 0;
        if (++hkv == p.Hkv) {
          hkv = 0;
          ++s;
        }
      }
    }
    return true;
  }
};

// A wait that parks the warp until the phase completes or about 20 us have gone
// by.  Without a time limit of its own a try returns after a short one, and some
// ten waiting warps' retries then slow every other shared-memory access of the SM
// (a wait for a completed phase took 200 cycles instead of 30).
__device__ __forceinline__ bool parked_wait(uint32_t mb, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(mb), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// The long part of every role's bounded wait; false: leave.  It is kept out of
// line: the roles' hot loops share the instruction cache.  Sh holds `abort`, and `redone`:
// rows evaluated again so far, and parts of them.
template <typename Sh>
__device__ __noinline__ bool long_wait(uint32_t mb, uint32_t parity, Sh* sh, unsigned* status) {
  long long t0 = clock64();
  int redone = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (parked_wait(mb, parity)) return true;
    if (*(volatile int*)&sh->abort) return false;
    // Rows evaluated again take about 1 us a key: the time counts from the last sign of
    // one of them.
    const int now = *(volatile int*)&sh->redone;
    if (now != redone) {
      redone = now;
      t0 = clock64();
    }
    if (clock64() - t0 > kWaitBudget) {
      *(volatile int*)&sh->abort = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}
// By a whole warp, with one answer for it: near the limit the lanes' own answers may
// differ, and a warp that some of them leave may not go on with the rest.  (A vote in
// front of the branch: behind a branch per lane it cost the tile forms 1 %.)
template <typename Sh>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Sh* sh, unsigned* status) {
  const uint32_t mb = smem_u32(bar);
  const bool ok = parked_wait(mb, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  return __all_sync(0xffffffffu, ok || long_wait(mb, parity, sh, status));
}
// One lane of a converged warp.  The issuing roles run with all 32 lanes on
// values the compiler can see are the warp's (from lane 0 by a shuffle), and
// only the tcgen05 / TMA instruction itself is under this: operands then stay
// in uniform registers.  Issued by a lone lane of a diverged warp, each MMA
// cost some 100 cycles of register moves, more than its own 64.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e != 0;
}
template <typename T>
__device__ __forceinline__ T uni(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t mbar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(mbar)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Where CTA blockIdx.x of `ctas` begins, into sh->start_s, start_hkv, start_rt, start_u, and how many
// key tiles it has (sh->left); by the whole CTA, which synchronises before it reads them.
template <int kThreads, bool TILES, typename Sh>
__device__ __forceinline__ void stream_start(const AttnLaunch& p, int ctas, int tq, Sh* sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Prefix sum of the key tiles over the sequences, a run of them per thread.
  const int per = (p.N + kThreads - 1) / kThreads;
  const int s0 = min(p.N, tid * per), s1 = min(p.N, s0 + per);
  long long mine = 0;
  unsigned bad = 0;
  for (int s = s0; s < s1; ++s) {
    const SeqRange q = seq_range(p, s);
    mine += (long long)key_tiles(q) * row_tiles<TILES>(p, q, tq);
    bad |= q.bad;
  }
  if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadSeqlens);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh->scan[warp] = inc;
  if (tid == 0) sh->start_s = p.N;
  __syncthreads();
  long long before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh->scan[w];
    total += sh->scan[w];
  }
  total *= p.Hkv;
  const long long w0 = total * blockIdx.x / ctas, w1 = total * (blockIdx.x + 1) / ctas;
  if (tid == 0) {
    sh->left = w1 - w0;
    sh->total = total;
  }
  if (w1 > w0 && before * p.Hkv <= w0 && w0 < (before + mine) * p.Hkv) {
    long long at = before * p.Hkv;
    for (int s = s0; s < s1; ++s) {
      const SeqRange q = seq_range(p, s);
      const int n = key_tiles(q);
      const long long all = (long long)n * row_tiles<TILES>(p, q, tq);  // of a kv head
      if (w0 < at + all * p.Hkv) {
        sh->start_s = s;
        sh->start_hkv = (int)((w0 - at) / all);
        sh->start_rt = TILES ? (int)((w0 - at) % all / n) : 0;
        sh->start_u = (int)((w0 - at) % all % n);
        break;
      }
      at += all * p.Hkv;
    }
  }
}

// What the joining kernel needs of CTA blockIdx.x's ranges, by one thread:
// {s, kv head + 2^16 row tile of the pair it began and left open (s = -1: none), how its first
// range ends: 0 open, 1 the pair's end, 2 no range at all; the CTA that ends the pair it left open}.
template <bool TILES, typename Sh>
__device__ __forceinline__ int4 stream_info(const AttnLaunch& p, int ctas, int tq, const Sh* sh) {
  int4 r = make_int4(-1, 0, 2, 0);
  SegIter<TILES> every{sh->start_s, sh->start_hkv, sh->start_rt, sh->start_u, (int)blockIdx.x, tq, sh->left};
  long long at = sh->total * blockIdx.x / ctas;  // tiles before the range
  Seg g;
  for (bool first = true; every.next(p, g); first = false) {
    const SeqRange q = seq_range(p, g.s);
    const int n = key_tiles(q);
    if (first) r.z = g.kt1 == n ? 1 : 0;
    if (g.kt0 == 0 && g.kt1 < n) {
      r.x = g.s;
      r.y = g.hkv + (TILES ? (g.t0 - q.a) / tq << 16 : 0);
      // The CTA with the pair's last tile, total c / ctas <= last < total (c + 1) / ctas.
      const long long last = at + n - 1;
      long long c = last * ctas / sh->total;
      while (sh->total * (c + 1) / ctas <= last) ++c;
      r.w = (int)c;
    }
    at += g.kt1 - g.kt0;
  }
  return r;
}

// Joins the ranges of the pairs that the stream form cut: CTA c serves the pair
// that range c began and left open, a row of it per blockIdx.y and its multiples;
// its further sums are in the blocks of the CTAs after it, in the order of their
// keys.
// `a` has the grid of the streaming kernel (ctas), its int4 info per CTA, the sums (ws), the
// rows of a block of them and tq.
// FEW: pairs in few ranges are joined by a warp a row, eight rows to a CTA.  (Drafts of 128
// sequences, every one of 304 CTAs leaving a pair of 16 rows open: 15 us of 208 went into
// 4900 CTAs of eight warps for two ranges.)
template <typename T, int D, bool FEW, typename Args>
__device__ __forceinline__ void stream_join(const AttnLaunch& p, const Args& a) {
  start_next_kernel();
  wait_for_previous_kernel();
  const int c0 = blockIdx.x;
  const int4 mine = a.info[c0];
  if (mine.x < 0) return;
  const int G = p.Hq / p.Hkv;
  const SeqRange q = seq_range(p, mine.x);
  const int hkv = mine.y & 0xffff, first = (mine.y >> 16) * a.tq;  // tokens before the row tile's
  const int rows = min(a.tq, min(q.b - q.a, p.max_q) - first) * G;
  if ((int)blockIdx.y >= rows) return;
  const int c1 = mine.w;  // the last range's CTA
  const Partials part(a.ws, 2 * (int64_t)a.ctas, a.rows, D);
  // Block 2 c0 + 1 for the first range, 2 c for the rest; none for a CTA without one.
  auto slot_of = [&](int z) -> int64_t {
    return z == 0 ? 2 * (int64_t)c0 + 1 : a.info[c0 + z].z == 2 ? -1 : 2 * (int64_t)(c0 + z);
  };
  if (FEW && c1 - c0 < 8) {
    for (int r0 = 8 * blockIdx.y; r0 < rows; r0 += 8 * gridDim.y) {
      const int r = r0 + (threadIdx.x >> 5);
      join_row<T, D, 1>(p, part, c1 - c0 + 1, slot_of, r, r < rows, q.a + first + r / G, hkv * G + r % G);
    }
    return;
  }
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    join_row<T, D, 8, FEW ? 8 : 4>(p, part, c1 - c0 + 1, slot_of, r, true, q.a + first + r / G, hkv * G + r % G);
    __syncthreads();
  }
}

inline size_t info_bytes(int ctas) { return ((size_t)ctas * sizeof(int4) + 255) & ~(size_t)255; }

}  // namespace attn
}  // namespace gdn
