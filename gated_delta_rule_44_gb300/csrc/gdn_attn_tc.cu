// gdn_attn_tc.cu -- full attention on tcgen05 tensor cores: packed prompts,
// chunks and single tokens over a paged cache, in one kernel.
//
// A tile is 128 rows: consecutive tokens of one sequence times the G query
// heads of one kv head, so a key tile read once serves the whole group.  Keys
// come 128 at a time:
//   S = Q K^T                       (M = 128 rows, N = 128 keys, K = D)
//   P = 2^(c S - m),  c = scale log2(e);   l += row sum of P
//   O += P V                        (M = 128 rows, N = D, K = 128 keys)
//   out = O / l
// S and O are f32 in TMEM; P is bf16 and takes S's place there (an A operand
// in tensor memory), so nothing of a tile but K and V passes through shared
// memory.  m is a reference at or below the running maximum: it is raised,
// and O and l scaled, only when the maximum has outgrown it by 2^8, which
// after the first tiles is rare; P's values stay below 2^8 and its rounding
// (2^-9 relative) is the same for any reference.  l sums P before the rounding.
//
// Warps:  0, 3    TMA loads of Q and K, of V, in units of 128 keys x up to 128 dims
//                 (two warps, because a page of 16 rows makes 16 loads a unit)
//         1       every MMA
//         2       zeroes the rows of V past the last visible key (a stale or
//                 foreign NaN there would survive a weight of 0); the stream
//                 form's bookkeeping
//         4-11    softmax and output of row tile 0: two threads per row, each with
//                 half the keys (one warp per row would be as many instructions,
//                 but its dependent chain would outlast the other tile's MMAs)
//         12-19   the same for row tile 1 (two-tile form)
// Two-tile form (D <= 128, 256 rows): while one tile's softmax runs on the CUDA
// cores the other's MMAs run.  One-tile form (D = 256, whose O fills half the
// TMEM, and few rows): two S buffers, so that the next key tile's scores are
// computed during a softmax.
//
// Work.  The tile form has one CTA per (tile, kv head), the longest first, and
// with few of them cuts each into key ranges whose sums a second kernel joins.
// The stream form serves sequences whose new rows fit one tile (decode,
// drafts): the key tiles of all (sequence, kv head) pairs, in order, are cut
// into equal consecutive ranges, one per SM, whatever the lengths; a pair cut
// between SMs leaves its sums in the workspace, and a second kernel joins them
// in the order of their keys.
//
// A row whose result is not finite is evaluated again key by key (exact_row):
// the product above multiplies a masked key's weight 0 into its v.
//
// Every wait is bounded; once one gives up, every role leaves at its next
// wait, copies and MMAs in flight are waited for (bounded) and TMEM is freed.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_common.cuh"
#include "gdn_chunk_common.cuh"
#include "gdn_internal.h"
#include "tcgen05.cuh"

namespace gdn {
namespace {

using namespace attn;
using namespace umma;
using bf16 = __nv_bfloat16;

constexpr long long kWaitBudget = 2000000000LL;  // ~1 s of SM clock per wait
constexpr int BK = 128;                          // keys per tile
constexpr float kRaise = 8.0f;                   // log2 headroom of the reference m
constexpr int kMaxSplits = 64;

constexpr uint32_t kSmemMax = 232448;  // per CTA

struct Shared {
  uint64_t full[12], empty[12];
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv, o_full[2], o_empty, v_landed, v_fixed, end, pair[2][4];
  uint32_t tmem;
  int abort;
  uint32_t loads[12], q_loads;  // issued so far into each place, and of Q
  uint32_t v_at[2];  // places of the V units to clear
  int start_s, start_hkv, start_u;
  long long left;
  long long scan[20];
  union {  // what the two warps of 32 rows exchange
    uint16_t top[2][2][2][128];  // [tile & 1][row tile][half][row]: maxima, as bf16
    float val[2][2][128];        // [row tile][half][row]
  } swap;
};

template <int D, int NQ>
struct Cfg {
  static constexpr int DU = D < 128 ? D : 128;          // dims of a K / V unit
  static constexpr int NU = D / DU;                     // units per key tile
  static constexpr uint32_t kUnit = BK * DU * 2;        // bytes
  static constexpr uint32_t kQTile = 128 * D * 2;
  static constexpr uint32_t kQ = NQ * kQTile;
  static constexpr int kFit = (int)((kSmemMax - sizeof(Shared) - kQ) / kUnit);
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static constexpr uint32_t kBars = kQ + kStages * kUnit;
  static constexpr uint32_t kBytes = kBars + sizeof(Shared);
  static constexpr int kThreads = 128 + 256 * NQ;
};
static_assert(Cfg<128, 2>::kStages >= 5 && Cfg<256, 1>::kStages >= 5, "units in flight");

// TMEM columns (512 allocated): S buffers of 128, then O.
constexpr uint32_t kTO = 256;

struct TcArgs {
  int splits;   // key ranges per tile (tile form)
  int TQ;       // tokens per row tile: 128 / G
  int q_box;    // tokens of a Q load
  int pb;       // rows of a K / V load: 128 (packed), or a divisor of the page
  int ctas;     // stream form: the grid
  int rows;     // rows of a workspace block
  int4* info;   // stream form, per CTA: {s, kv head of the pair it began and left open (s = -1:
                // none), how its first range ends: 0 open, 1 the pair's end, 2 no range at all}
  float* ws;    // the sums
};

// A range of key tiles of one (tile, kv head).
struct Seg {
  int s, hkv, t0, nt, pos0, hi, kt0, kt1;
  int64_t slot;  // workspace block of its sums; -1: it has every key of its rows
};

__device__ __forceinline__ int key_tiles(const SeqRange& q) {
  return q.b > q.a ? (q.kv + BK - 1) / BK : 0;
}

// The ranges of one CTA of the stream form.
struct SegIter {
  int s, hkv, u, cta;
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
    g.t0 = q.a;
    g.nt = min(q.b - q.a, p.max_q);
    g.pos0 = q.kv - (q.b - q.a);
    g.hi = q.kv;
    g.kt0 = u;
    g.kt1 = u + take;
    g.slot = take == n ? -1 : 2 * (int64_t)cta + (u == 0 ? 1 : 0);
    left -= take;
    u += take;
    if (u == n) {
      u = 0;
      if (++hkv == p.Hkv) {
        hkv = 0;
        ++s;
      }
    }
    return true;
  }
};

// The bounded wait of every role; false: leave.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Shared* sh,
                                              unsigned* status) {
  const uint32_t mb = smem_u32(bar);
  if (mbar_try_wait(mb, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(mb, parity)) {
    if (*(volatile int*)&sh->abort) return false;
    if (clock64() - t0 > kWaitBudget) {
      *(volatile int*)&sh->abort = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}
// The same by a whole warp, with one answer for it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Shared* sh,
                                          unsigned* status) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, sh, status));
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
// Inside a role: the bounded wait, or leave the role.
#define WAIT(bar, parity) \
  if (!wait_or_abort(&(bar), (parity), sh, p.status)) return

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
// (a0, a1) * (c, c) + (b, b), two f32 lanes in one instruction.
__device__ __forceinline__ void fma2(float& x0, float& x1, float c, float b) {
  uint64_t x, cc, bb;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
  asm("mov.b64 %0, {%1, %1};" : "=l"(bb) : "f"(b));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(cc), "l"(bb));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(x));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
  uint64_t s, x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(s) : "f"(s0), "f"(s1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s) : "l"(x));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(s));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int NQ, bool PAGED, bool STREAM>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnLaunch p, const __grid_constant__ CUtensorMap mq,
                   const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ TcArgs a) {
  using C = Cfg<D, NQ>;
  constexpr int DU = C::DU, NU = C::NU, ST = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];  // the swizzle atoms' alignment
  Shared* sh = reinterpret_cast<Shared*>(smem + C::kBars);
  const uint32_t sq = smem_u32(smem), skv = sq + C::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;

  // ---- which work ----
  Seg seg0;
  if constexpr (!STREAM) {
    const int TT = NQ * a.TQ;
    const int id = (int)(gridDim.x / p.Hkv) - 1 - (int)(blockIdx.x / p.Hkv);
    const SeqTile t = find_tile(p, id, TT);
    if (t.bad && tid == 0) atomicOr(p.status, kStatusBadSeqlens);
    if (t.nt == 0) return;
    seg0.s = t.s;
    seg0.hkv = blockIdx.x % p.Hkv;
    seg0.t0 = t.t0;
    seg0.nt = t.nt;
    seg0.pos0 = t.pos0;
    seg0.hi = max(0, t.pos0 + t.nt);
    const int n = (seg0.hi + BK - 1) / BK;
    seg0.kt0 = (int)((int64_t)n * blockIdx.y / a.splits);
    seg0.kt1 = (int)((int64_t)n * (blockIdx.y + 1) / a.splits);
    seg0.slot = a.splits > 1 ? ((int64_t)id * p.Hkv + seg0.hkv) * a.splits + blockIdx.y : -1;
    if (seg0.kt0 == seg0.kt1) {  // no key here
      const Partials part(a.ws, (int64_t)gridDim.x * a.splits, a.rows, D);
      for (int r = warp; r < seg0.nt * G; r += C::kThreads / 32) {
        const float zero[D / 32] = {};
        if (seg0.slot >= 0) part.put<D / 32>(seg0.slot, r, lane, zero, -INFINITY, 0.0f);
        else finish_row<bf16, D>(p, seg0.t0 + r / G, seg0.hkv * G + r % G, lane, zero, -INFINITY, 0.0f);
      }
      return;
    }
  }

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < ST; ++i) {
        mbar_init(smem_u32(&sh->full[i]), 1);
        mbar_init(smem_u32(&sh->empty[i]), 1);
      }
      mbar_init(smem_u32(&sh->q_full), 1);
      mbar_init(smem_u32(&sh->q_empty), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&sh->s_full[i]), 1);
        mbar_init(smem_u32(&sh->p_full[i]), 8);
        mbar_init(smem_u32(&sh->o_full[i]), 1);
        for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&sh->pair[i][w]), 2);
      }
      mbar_init(smem_u32(&sh->pv), 1);
      mbar_init(smem_u32(&sh->o_empty), 8);
      mbar_init(smem_u32(&sh->v_landed), 1);
      mbar_init(smem_u32(&sh->v_fixed), 1);
      mbar_init(smem_u32(&sh->end), 1);
      sh->abort = 0;
      sh->q_loads = 0;
      for (int i = 0; i < ST; ++i) sh->loads[i] = 0;
      fence_mbar_init();
    }
  } else if (warp == 2) {
    tmem_alloc(smem_u32(&sh->tmem), 512);
  }
  if constexpr (STREAM) {
    // Prefix sum of the key tiles over the sequences, a run of them per thread.
    const int per = (p.N + C::kThreads - 1) / C::kThreads;
    const int s0 = min(p.N, tid * per), s1 = min(p.N, s0 + per);
    long long mine = 0;
    unsigned bad = 0;
    for (int s = s0; s < s1; ++s) {
      const SeqRange q = seq_range(p, s);
      mine += key_tiles(q);
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
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) before += sh->scan[w];
      total += sh->scan[w];
    }
    total *= p.Hkv;
    const long long w0 = total * blockIdx.x / a.ctas, w1 = total * (blockIdx.x + 1) / a.ctas;
    if (tid == 0) sh->left = w1 - w0;
    if (w1 > w0 && before * p.Hkv <= w0 && w0 < (before + mine) * p.Hkv) {
      long long at = before * p.Hkv;
      for (int s = s0; s < s1; ++s) {
        const int n = key_tiles(seq_range(p, s));
        if (w0 < at + (long long)n * p.Hkv) {
          sh->start_s = s;
          sh->start_hkv = (int)((w0 - at) / n);
          sh->start_u = (int)((w0 - at) % n);
          break;
        }
        at += (long long)n * p.Hkv;
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  // All 512 columns: their base is 0, which the addresses below use as such.
  if (sh->tmem != 0 && tid == 0) atomicOr(p.status, kStatusTimeout);
  constexpr uint32_t tmem = 0;
  SegIter iter{};
  if constexpr (STREAM)
    iter = SegIter{sh->start_s, sh->start_hkv, sh->start_u, (int)blockIdx.x, sh->left};

  // The next range into g; one of them in the tile form.
  bool once = true;
  auto next_seg = [&](Seg& g) -> bool {
    if constexpr (STREAM) {
      return iter.next(p, g);
    } else {
      g = seg0;
      const bool r = once;
      once = false;
      return r;
    }
  };

  if (warp == 0 || warp == 3) {
    // ---- loads: Q and K by warp 0, V by warp 3 ----
    // Units go round the ring in the order of their use: K 0 .. A-1, then V j and
    // K j+A in turn (A = key tiles whose scores run ahead of P V).  Each warp
    // waits for its own units' places; a place it waits for was freed after every
    // place it has filled before, so a phase cannot be mistaken for the one two
    // before it.
    constexpr int A = NQ == 1 ? 2 : 1;
    const bool is_k = warp == 0;
    uint32_t base = 0;           // units of the ranges before
    int seg_n = 0;
    auto role = [&] {
      Seg g;
      while (next_seg(g)) {
        const int kt0 = uni(g.kt0), n = uni(g.kt1) - kt0, hi = uni(g.hi), hkv = uni(g.hkv);
        if (is_k) {
          const int nq = uni((NQ == 2 && g.nt > a.TQ) ? 2 : 1), t0 = uni(g.t0);
          if (seg_n > 0)
            if (!warp_wait(&sh->q_empty, (seg_n - 1) & 1, sh, p.status)) return;
          if (elect_one()) {
            sh->q_loads = seg_n + 1;
            mbar_expect_tx(smem_u32(&sh->q_full), nq * (D / 64) * 128u * G * a.q_box);
            for (int q = 0; q < nq; ++q)
#pragma unroll
              for (int b = 0; b < D / 64; ++b)
                tma_load_4d(sq + q * C::kQTile + b * 16384, &mq, smem_u32(&sh->q_full), b * 64, 0, hkv,
                            t0 + q * a.TQ);
          }
          ++seg_n;
        }
        // Loads of 64 dims x pb keys; those past the last visible key are left out.
        constexpr int NB = DU / 64;
        const CUtensorMap* map = is_k ? &mk : &mv;
        const int per_tile = BK / a.pb;
        const int row0 = PAGED ? 0 : uni(cu_at(p.cu, g.s));
        // Lane i looks up the page of, and issues, the tile's i-th load: 64 dims of a
        // group of pb keys.  (A loop over the loads with one elected lane was slower:
        // 461 against 380 us for drafts over pages of 16 rows.)
        const int grp = lane / NB, blk = lane % NB;
        auto find_page = [&](int kt) -> int {
          const int jb = kt * BK + grp * a.pb;
          if (!PAGED || grp >= per_tile || kt >= kt0 + n || jb >= hi) return 0;
          const int64_t pg = page_of(p, g.s, jb / p.page_size);
          if (pg < 0 && is_k) atomicOr(p.status, kStatusBadIndex);
          return pg < 0 ? (int)p.num_pages : (int)pg;  // past the end: reads as zeros
        };
        int next_page = find_page(kt0);
        for (int j = 0; j < n; ++j) {
          const int j0 = (kt0 + j) * BK;
          const int page = next_page;
          next_page = find_page(kt0 + j + 1);  // its latency passes during this tile's waits
          const int groups = min(per_tile, (hi - j0 + a.pb - 1) / a.pb);
          const uint32_t at = base + NU * (j + (is_k ? max(0, j - A + 1) : min(n, j + A)));
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            const uint32_t it = at + u, st = it % ST;
            if (it >= (uint32_t)ST)
              if (!warp_wait(&sh->empty[st], (it / ST - 1) & 1, sh, p.status)) return;
            const uint32_t full = smem_u32(&sh->full[st]);
            const uint32_t dst = skv + st * C::kUnit;
            if (elect_one()) {
              sh->loads[st] = it / ST + 1;
              mbar_expect_tx(full, groups * NB * a.pb * 128u);
            }
            if constexpr (PAGED) {
              __syncwarp();
              if (grp < groups)
                tma_load_4d(dst + blk * 16384 + grp * a.pb * 128, map, full, u * DU + blk * 64,
                            (j0 + grp * a.pb) % p.page_size, hkv, page);
              __syncwarp();
            } else {
              if (elect_one()) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  tma_load_3d(dst + b * 16384, map, full, u * DU + b * 64, row0 + j0, hkv);
              }
            }
          }
        }
        base += 2 * n * NU;
      }
    };
    role();
  } else if (warp == 1) {
    // ---- MMAs ----
    constexpr uint32_t kIdQK = idesc_bf16_f32(128, BK, false, false);
    constexpr uint32_t kIdPV = idesc_bf16_f32(128, DU, false, true);
    auto role = [&] {
      uint32_t nk = 0;  // key tiles done (one-tile form: S buffer and its phases)
      uint32_t st = 0, round = 0;  // place of the next unit, parity of its round
      int seg_n = 0, fixes = 0;
      Seg g;
      auto wait = [&](uint64_t& bar, uint32_t parity) { return warp_wait(&bar, parity, sh, p.status); };
      // The next unit has landed; its place in at.
      auto take1 = [&](uint32_t& at) -> bool {
        at = st;
        if (!wait(sh->full[st], round)) return false;
        if (++st == ST) {
          st = 0;
          round ^= 1;
        }
        fence_after_sync();
        return true;
      };
      // One unit's MMAs, 8 at most: the pipe has about 280 cycles of work queued
      // when they have been issued, so that one wait between two such blocks is
      // hidden, and the waits below are spread accordingly.  `done`, if any, is
      // arrived on when all MMAs so far are complete, and so is the unit's place
      // if it is not needed again.
      // S[buf] (+)= Q[q] K^T over the dims of unit u.
      auto qk = [&](int q, uint32_t buf, int u, uint32_t at, bool last_use, uint64_t* done) {
        if (elect_one()) {
          const uint64_t kd = desc_sw128(skv + at * C::kUnit, 16, 1024);
          const uint64_t qd = desc_sw128(sq + q * C::kQTile + u * (DU / 64) * 16384, 16, 1024);
#pragma unroll
          for (int k = 0; k < DU / 16; ++k) {
            const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
            mma_bf16(buf * 128, qd + off, kd + off, kIdQK, u + k > 0);
          }
          if (last_use) mma_commit(smem_u32(&sh->empty[at]));
          if (done) mma_commit(smem_u32(done));
        }
      };
      // O[q] (+)= P[buf] V over the dims of unit u.
      auto pv = [&](int q, uint32_t buf, int u, uint32_t at, bool acc, bool last_use, uint64_t* done) {
        if (elect_one()) {
          const uint64_t vd = desc_sw128(skv + at * C::kUnit, 16384, 1024);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            mma_bf16_ta(kTO + q * 128 + u * DU, buf * 128 + (k >> 2) * 64 + (k & 3) * 8, vd + ((k * 2048) >> 4), kIdPV,
                        acc || k > 0);
          if (last_use) mma_commit(smem_u32(&sh->empty[at]));
          if (done) mma_commit(smem_u32(done));
        }
      };
      auto ask_fix = [&](const uint32_t(&at)[NU]) {  // V's units have landed: clear their tail
        if (lane == 0) {
#pragma unroll
          for (int u = 0; u < NU; ++u) sh->v_at[u] = at[u];
          mbar_arrive(smem_u32(&sh->v_landed));
        }
        __syncwarp();
      };
      while (next_seg(g)) {
        const int n = uni(g.kt1 - g.kt0);
        const int nq = uni((NQ == 2 && g.nt > a.TQ) ? 2 : 1);
        const bool partial = uni((int)(g.kt1 * BK > g.hi));  // the last tile ends inside
        if (!wait(sh->q_full, seg_n & 1)) return;
        fence_after_sync();
        uint32_t ak[NU], av[NU];
        if constexpr (NQ == 2) {
          // NU = 1.  PV 0 | QK 0 | PV 1 | QK 1, a wait before each.
          if (!take1(ak[0])) return;
          for (int q = 0; q < nq; ++q) qk(q, q, 0, ak[0], q == nq - 1, &sh->s_full[q]);
          if (!take1(av[0])) return;
          for (int j = 0; j < n; ++j) {
            const bool more = j + 1 < n;
            if (!more && partial) ask_fix(av);
            uint32_t next_v = 0;
            for (int q = 0; q < nq; ++q) {
              if (!wait(sh->p_full[q], j & 1)) return;
              if (!more && partial && q == 0)
                if (!wait(sh->v_fixed, fixes++ & 1)) return;
              fence_after_sync();
              pv(q, q, 0, av[0], j > 0, q == nq - 1, more ? nullptr : &sh->o_full[q]);
              if (more) {
                if (q == 0)
                  if (!take1(ak[0])) return;
                if (q == nq - 1)
                  if (!take1(next_v)) return;
                qk(q, q, 0, ak[0], q == nq - 1, &sh->s_full[q]);
              }
            }
            av[0] = next_v;
          }
        } else {
          // PV j | QK j+2, unit by unit; K j+2 and V j+1 are waited for on the way.
          for (int j = 0; j < min(n, 2); ++j)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              if (!take1(ak[u])) return;
              qk(0, (nk + j) & 1, u, ak[u], true, u == NU - 1 ? &sh->s_full[(nk + j) & 1] : nullptr);
            }
#pragma unroll
          for (int u = 0; u < NU; ++u)
            if (!take1(av[u])) return;
          for (int j = 0; j < n; ++j, ++nk) {
            const uint32_t buf = nk & 1;
            const bool more_v = j + 1 < n, more_k = j + 2 < n;
            if (!more_v && partial) ask_fix(av);
            if (j == 0 && seg_n > 0)  // the last range's O has been read
              if (!wait(sh->o_empty, (seg_n - 1) & 1)) return;
            if (!wait(sh->p_full[buf], (nk >> 1) & 1)) return;
            if (!more_v && partial)
              if (!wait(sh->v_fixed, fixes++ & 1)) return;
            fence_after_sync();
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              pv(0, buf, u, av[u], j > 0, true, u == NU - 1 ? &sh->pv : nullptr);
              if (more_k)
                if (!take1(ak[u])) return;
            }
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              if (more_k) qk(0, buf, u, ak[u], true, u == NU - 1 ? &sh->s_full[buf] : nullptr);
              if (more_v)
                if (!take1(av[u])) return;
            }
          }
          if (elect_one()) mma_commit(smem_u32(&sh->o_full[0]));
        }
        if (elect_one()) mma_commit(smem_u32(&sh->q_empty));
        ++seg_n;
      }
    };
    role();
    if (elect_one()) mma_commit(smem_u32(&sh->end));
    warp_wait(&sh->end, 0, sh, p.status);
  } else if (warp == 2) {
    if constexpr (STREAM) {
      // What the joining kernel needs of this CTA's ranges; the outputs of
      // sequences without a key.
      if (lane == 0) {
        int4 r = make_int4(-1, 0, 2, 0);
        SegIter every = iter;
        Seg g;
        for (bool first = true; every.next(p, g); first = false) {
          const int n = key_tiles(seq_range(p, g.s));
          if (first) r.z = g.kt1 == n ? 1 : 0;
          if (g.kt0 == 0 && g.kt1 < n) {
            r.x = g.s;
            r.y = g.hkv;
          }
        }
        a.info[blockIdx.x] = r;
      }
      for (int s = blockIdx.x; s < p.N; s += a.ctas) {
        const SeqRange q = seq_range(p, s);
        if (key_tiles(q) > 0) continue;
        const float zero[D / 32] = {};
        for (int t = q.a; t < q.b; ++t)
          for (int h = 0; h < p.Hq; ++h) finish_row<bf16, D>(p, t, h, lane, zero, -INFINITY, 0.0f);
      }
    }
    // ---- V's rows past the last visible key ----
    auto role = [&] {
      int fixes = 0;
      Seg g;
      while (next_seg(g)) {
        if (g.kt1 * BK <= g.hi) continue;
        WAIT(sh->v_landed, fixes & 1);
        ++fixes;
        const int r0 = g.hi - (g.kt1 - 1) * BK;  // first row to clear
        for (int u = 0; u < NU; ++u) {
          unsigned char* v = smem + C::kQ + sh->v_at[u] * C::kUnit;
          // Whole 128-byte rows: the swizzle permutes inside a row only.
          for (int i = lane; i < (BK - r0) * (DU / 8); i += 32) {
            const int r = r0 + i / (DU / 8), ch = i % (DU / 8);
            *reinterpret_cast<uint4*>(v + (ch >> 3) * 16384 + r * 128 + (ch & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->v_fixed));
      }
    };
    role();
  } else {
    // ---- softmax, output ----
    // Two warps share 32 rows: `half` is the half of the keys of a tile, and of
    // the dims of O, that this one handles.
    const int sw = warp - 4, half = (sw >> 2) & 1, qt = NQ == 2 ? sw >> 3 : 0;
    const int r = tid & 127;                            // row of the tile, lane of TMEM
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // (32 * (warp % 4)) << 16
    const float c = p.scale * kLog2e;
    const int tok = qt * a.TQ + r / G;                  // token of the tile
    auto role = [&] {
    uint32_t nk = 0, np = 0;
    // Meeting the pair's other warp (bounded; false: leave).
    uint64_t& pair = sh->pair[qt][warp & 3];
    auto pair_arrive = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&pair));
    };
    auto pair_wait = [&]() -> bool { return wait_or_abort(&pair, np++ & 1, sh, p.status); };
    // x becomes the row's value of it from the other warp (between two meetings
    // that keep `val` from being written early).
    auto swap = [&](float& x) -> bool {
      sh->swap.val[qt][half][r] = x;
      pair_arrive();
      const bool ok = pair_wait();
      x = sh->swap.val[qt][half ^ 1][r];
      return ok;
    };
    int seg_n = 0;
    Seg g;
    while (next_seg(g)) {
      if (NQ == 2 && qt == 1 && g.nt <= a.TQ) break;   // no second row tile
      const bool valid = r < a.TQ * G && tok < g.nt;
      // The row's last visible key; rows that do not exist see all (their
      // values are not used) so that they cost no masking.
      const int last = valid ? g.pos0 + tok : INT32_MAX;
      const bool idle = __all_sync(0xffffffffu, !valid);
      // m, the reference of P, is the same in both warps.  It follows the scores
      // one tile behind: the first tile's maximum is exchanged before its P, later
      // ones while the next tile's scores are computed, so that neither the
      // exchange nor the maximum itself delays a P.  P may thus exceed 2^8 (one
      // rounding relative to its size all the same); should it overflow, the row
      // is not finite and is evaluated again.
      float m = -INFINITY, l = 0.0f;
      uint32_t top_bits = 0;  // this warp's last published maximum
      const uint32_t to = tmem + lanes + kTO + qt * 128 + half * (D / 2);
      for (int kt = g.kt0; kt < g.kt1; ++kt, ++nk) {
        const int buf = NQ == 2 ? qt : (int)(nk & 1);
        const uint32_t ph = NQ == 2 ? (uint32_t)(kt - g.kt0) & 1 : (nk >> 1) & 1;
        const int jj = kt - g.kt0;
        WAIT(sh->s_full[buf], ph);
        fence_after_sync();
        if (!idle) {
          const uint32_t ts = tmem + lanes + buf * 128;
          float s[2][32];
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_ld32(ts + half * 64 + i * 32, s[i]);
          tmem_ld_wait();
          const int j0 = kt * BK + half * 64;
          if (__any_sync(0xffffffffu, j0 + 63 > last)) {
            const int lim = last - j0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 32; ++e) s[i][e] = i * 32 + e <= lim ? s[i][e] : -INFINITY;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto publish = [&] {
            const float t = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            top_bits = __float_as_uint(t) >> 16;  // cut to bf16: only the agreement matters
            sh->swap.top[jj & 1][qt][half][r] = (uint16_t)top_bits;
            pair_arrive();
          };
          if (jj == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 32; e += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mx[k] = fmaxf(mx[k], fmaxf(s[i][e + 2 * k], s[i][e + 2 * k + 1]));
            publish();
          }
          if (jj != 1) {
            if (!pair_wait()) return;
            const int slot = jj == 0 ? 0 : (jj - 1) & 1;
            const float top = fmaxf(__uint_as_float(top_bits << 16),
                                    __uint_as_float((uint32_t)sh->swap.top[slot][qt][half ^ 1][r] << 16));
            // Without a score above -inf so far the reference is 0.  (c may be 0,
            // and 0 * -inf must not count as a score.)
            const float tm = top == -INFINITY ? -INFINITY : top * c;
            float f = 1.0f;
            bool raise = false;
            if (tm > m + kRaise || (m == -INFINITY && tm > m)) {
              raise = valid && jj > 0;
              f = ex2(m - tm);
              m = tm;
            }
            if (m == -INFINITY) m = 0.0f;
            if (__any_sync(0xffffffffu, raise)) {
              // O is at rest: in the two-tile form S j follows P V j-1, in the
              // other that product is waited for.
              if constexpr (NQ == 1) {
                WAIT(sh->pv, (nk - 1) & 1);
                fence_after_sync();
              }
              l *= f;
#pragma unroll 1
              for (int i = 0; i < D / 32; ++i) {
                float o[16];
                tmem_ld16(to + i * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= f;
                tmem_st16(to + i * 16, o);
              }
              tmem_st_wait();
            }
          }
          const float ref = -m;
          float l0 = 0.0f, l1 = 0.0f, l2 = 0.0f, l3 = 0.0f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float(&x)[32] = s[i];
            float pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              mx[(e >> 1) & 2] = fmaxf(mx[(e >> 1) & 2], fmaxf(x[e], x[e + 1]));
              mx[((e >> 1) & 2) + 1] = fmaxf(mx[((e >> 1) & 2) + 1], fmaxf(x[e + 2], x[e + 3]));
              fma2(x[e], x[e + 1], c, ref);
              fma2(x[e + 2], x[e + 3], c, ref);
#pragma unroll
              for (int k = 0; k < 4; ++k) x[e + k] = ex2(x[e + k]);
              add2(l0, l1, x[e], x[e + 1]);
              add2(l2, l3, x[e + 2], x[e + 3]);
              pk[e / 2] = __uint_as_float(pack_bf16(x[e], x[e + 1]));
              pk[e / 2 + 1] = __uint_as_float(pack_bf16(x[e + 2], x[e + 3]));
            }
            tmem_st16(ts + half * 64 + i * 16, pk);
          }
          tmem_st_wait();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[buf]));
          l += (l0 + l1) + (l2 + l3);
          if (jj > 0 && kt + 1 < g.kt1) publish();
        } else if (lane == 0) {
          mbar_arrive(smem_u32(&sh->p_full[buf]));
        }
      }
      // ---- the row's sums out ----
      const int t = g.t0 + tok, h = g.hkv * G + r % G;
      const bool gated = p.gate.p != nullptr && g.slot < 0 && valid;
      const uint4* gate = reinterpret_cast<const uint4*>(
          static_cast<const bf16*>(p.gate.p) + (int64_t)t * p.gate.ts + (int64_t)h * p.gate.hs +
          half * (D / 2));
      // The gate's loads go out before the wait and a chunk of 32 dims ahead: one
      // at a time, just before use, they were half the time of a short row.
      uint4 gw[4];
      if (gated) {
#pragma unroll
        for (int e = 0; e < 4; ++e) gw[e] = gate[e];
      }
      WAIT(sh->o_full[qt], seg_n & 1);
      fence_after_sync();
      if (!idle) {
        float theirs = l;
        if (!swap(theirs)) return;
        l = half == 0 ? l + theirs : theirs + l;  // the same sum on both sides
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const Partials part(a.ws, STREAM ? 2 * (int64_t)a.ctas : (int64_t)gridDim.x * a.splits, a.rows, D);
        const int pr = tok * G + r % G;
        // A sum of 0 with a key in sight: every weight was lost beside a reference
        // of 0 that no score gave.
        bool finite = isfinite(l) && !(l == 0.0f && last >= g.kt0 * BK);
        bf16* out = static_cast<bf16*>(p.out) + ((int64_t)t * p.Hq + h) * D + half * (D / 2);
#pragma unroll 1
        for (int i = 0; i < D / 64; ++i) {
          float o[32];
          tmem_ld32(to + i * 32, o);
          tmem_ld_wait();
          float big = 0.0f;  // NaN and infinities survive a sum of x - x
#pragma unroll
          for (int e = 0; e < 32; ++e) big += o[e] - o[e];
          finite = finite && big == 0.0f;
          if (g.slot >= 0) {
            if (valid) {
              float4* d = reinterpret_cast<float4*>(part.o + (g.slot * a.rows + pr) * D +
                                                    half * (D / 2) + i * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
            continue;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (gated) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t gp[4] = {gw[e].x, gw[e].y, gw[e].z, gw[e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[e * 8 + 2 * k] *= sigmoid_gate(__uint_as_float(gp[k] << 16));
                o[e * 8 + 2 * k + 1] *= sigmoid_gate(__uint_as_float(gp[k] & 0xffff0000u));
              }
            }
            if (i + 1 < D / 64) {
#pragma unroll
              for (int e = 0; e < 4; ++e) gw[e] = gate[(i + 1) * 4 + e];
            }
          }
          if (valid) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = pack_bf16(o[e * 8 + 2 * k], o[e * 8 + 2 * k + 1]);
              *reinterpret_cast<uint4*>(out + i * 32 + e * 8) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (valid && half == 0) {
          if (g.slot >= 0) part.ml[g.slot * a.rows + pr] = make_float2(l == 0.0f ? -INFINITY : m, l);
          else if (p.lse != nullptr)
            p.lse[(int64_t)t * p.Hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        // Rows to evaluate again, by the pair's first warp once both have stored.
        pair_arrive();
        if (!pair_wait()) return;
        theirs = finite ? 1.0f : 0.0f;
        if (!swap(theirs)) return;
        unsigned redo = __ballot_sync(0xffffffffu, valid && !(finite && theirs == 1.0f));
        pair_arrive();  // `theirs` has been read: the next range may publish
        if (!pair_wait()) return;
        if (half == 1) redo = 0;
        while (redo) {
          const int src = __ffs(redo) - 1;
          redo &= redo - 1;
          const int rt = __shfl_sync(0xffffffffu, t, src), rh = __shfl_sync(0xffffffffu, h, src);
          const int rl = __shfl_sync(0xffffffffu, last, src), rp = __shfl_sync(0xffffffffu, pr, src);
          float acc[D / 32], em, el;
          exact_row<bf16, D>(p, g.s, cu_at(p.cu, g.s), rt, rh, g.kt0 * BK, min(g.kt1 * BK, rl + 1), acc,
                             em, el);
          if (g.slot >= 0) part.put<D / 32>(g.slot, rp, lane, acc, em, el);
          else finish_row<bf16, D>(p, rt, rh, lane, acc, em, el);
        }
      }
      ++seg_n;
      if constexpr (STREAM) {
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->o_empty));
      }
    }
    };
    role();
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (sh->abort) {
    // A wait gave up: copies may still be in flight (otherwise the MMA role has
    // waited for each).  They land before the CTA's memory is given up.
    if (tid == 0) {
      for (int i = 0; i < ST; ++i)
        if (sh->loads[i]) mbar_wait(smem_u32(&sh->full[i]), (sh->loads[i] - 1) & 1, kWaitBudget);
      if (sh->q_loads) mbar_wait(smem_u32(&sh->q_full), (sh->q_loads - 1) & 1, kWaitBudget);
    }
    __syncthreads();
  }
  if (warp == 2) tmem_dealloc(sh->tmem, 512);
}

// Joins the ranges of the pairs that the stream form cut: CTA c serves the pair
// that range c began and left open; its further sums are in the blocks of the
// CTAs after it, in the order of their keys.  A block takes 8 rows, a warp one
// row at a time: the ranges' (m, l) first, a lane each, then the weighted sum of
// their O, whose loads do not wait for one another.
template <int D>
__global__ void __launch_bounds__(256) attn_stream_join_kernel(const __grid_constant__ AttnLaunch p,
                                                               const __grid_constant__ TcArgs a) {
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 mine = a.info[c0];
  if (mine.x < 0) return;
  const int G = p.Hq / p.Hkv;
  const SeqRange q = seq_range(p, mine.x);
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  // The last range: the first after c0 that ends the pair.
  int c1 = c0;
  for (int c = c0 + 1; c1 == c0 && c < a.ctas; c += 32) {
    const unsigned ends = __ballot_sync(0xffffffffu, c + lane < a.ctas && a.info[c + lane].z == 1);
    c1 = ends ? c + __ffs(ends) - 1 : (c + 32 >= a.ctas ? a.ctas - 1 : c0);
  }
  if (r >= min(q.b - q.a, p.max_q) * G) return;
  const Partials part(a.ws, 2 * (int64_t)a.ctas, a.rows, D);
  constexpr int E = D / 32;
  float acc[E] = {}, m = -INFINITY, l = 0.0f;
  for (int c = c0; c <= c1; c += 32) {
    // Range c + lane: block 2 c0 + 1 for the first, 2 c' for the rest; CTAs
    // without a range (z = 2) hold nothing.
    const int cl = c + lane;
    const int64_t slot = 2 * (int64_t)cl + (cl == c0 ? 1 : 0);
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (cl <= c1 && (cl == c0 || a.info[cl].z != 2)) ml = part.ml[slot * a.rows + r];
    float mn = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mn = fmaxf(mn, m);
    if (mn == -INFINITY) continue;
    const float f = exp2f(m - mn);  // 0 for m = -inf
    const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - mn);
    float lw = ml.x == -INFINITY ? 0.0f : w * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    l = fmaf(l, f, lw);
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
    unsigned live = __ballot_sync(0xffffffffu, ml.x != -INFINITY);
    while (live) {  // four ranges' loads in flight
      float x[4][E], wk[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        wk[k] = 0.0f;
        if (live) {
          const int src = __ffs(live) - 1;
          live &= live - 1;
          wk[k] = __shfl_sync(0xffffffffu, w, src);
          const int ck = c + src;
          const float* o = part.o + ((2 * (int64_t)ck + (ck == c0 ? 1 : 0)) * a.rows + r) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) x[k][e] = o[e];
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) x[k][e] = 0.0f;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wk[k], x[k][e], acc[e]);
    }
  }
  finish_row<bf16, D>(p, q.a + r / G, mine.y * G + r % G, lane, acc, m, l);
}

// ---- host ------------------------------------------------------------------------

bool encode(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const int64_t* strides,
            const cuuint32_t* box) {
  auto enc = chunk::encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t st[4];
  for (int i = 0; i < rank - 1; ++i) st[i] = (cuuint64_t)strides[i] * 2;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, st,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool q_map(CUtensorMap* m, const AttnLaunch& p, int q_box) {
  const int G = p.Hq / p.Hkv;
  const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)G, (cuuint64_t)p.Hkv, (cuuint64_t)p.T};
  const int64_t st[3] = {p.q.hs, p.q.hs * G, p.q.ts};
  const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)q_box};
  return encode(m, p.q.p, 4, dims, st, box);
}
bool rows_map(CUtensorMap* m, const AttnRows& r, const AttnLaunch& p) {
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.T, (cuuint64_t)p.Hkv};
  const int64_t st[2] = {r.ts, r.hs};
  const cuuint32_t box[3] = {64, (cuuint32_t)BK, 1};
  return encode(m, r.p, 3, dims, st, box);
}
bool pages_map(CUtensorMap* m, const AttnPages& c, const AttnLaunch& p, int pb) {
  const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv,
                              (cuuint64_t)p.num_pages};
  const int64_t st[3] = {c.ts, c.hs, c.ps};
  const cuuint32_t box[4] = {64, (cuuint32_t)pb, 1, 1};
  return encode(m, c.p, 4, dims, st, box);
}

// Sequences whose new rows all fit one row tile take the stream form.
bool use_stream(int64_t max_q, int64_t G) { return max_q * G <= 128; }

int tile_splits(int64_t items, int64_t max_kv, int sms) {
  return (int)std::max<int64_t>(1, std::min<int64_t>({sms / items, max_kv / (4 * BK), kMaxSplits}));
}

template <int D>
constexpr int tiles_of() {
  return D <= 128 ? 2 : 1;
}

size_t info_bytes(int ctas) { return ((size_t)ctas * sizeof(int4) + 255) & ~(size_t)255; }

template <int D, int NQ, bool PAGED, bool STREAM>
cudaError_t run(const AttnLaunch& p, TcArgs a, dim3 grid, cudaStream_t st) {
  using C = Cfg<D, NQ>;
  CUtensorMap mq, mk, mv;
  if (!q_map(&mq, p, a.q_box) || !(PAGED ? pages_map(&mk, p.kc, p, a.pb) : rows_map(&mk, p.k, p)) ||
      !(PAGED ? pages_map(&mv, p.vc, p, a.pb) : rows_map(&mv, p.v, p)))
    return cudaErrorInvalidValue;
  static const cudaError_t attr =
      cudaFuncSetAttribute(attn_tc_kernel<D, NQ, PAGED, STREAM>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kBytes);
  if (attr != cudaSuccess) return attr;
  attn_tc_kernel<D, NQ, PAGED, STREAM><<<grid, C::kThreads, C::kBytes, st>>>(p, mq, mk, mv, a);
  note_launch();
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const AttnLaunch& p, cudaStream_t st) {
  constexpr int NQ = tiles_of<D>();
  const int G = p.Hq / p.Hkv, sms = chunk::sm_count();
  TcArgs a{};
  a.TQ = 128 / G;
  a.splits = 1;
  a.pb = BK;
  if (p.table != nullptr)
    while (p.page_size % a.pb != 0) a.pb >>= 1;
  if (p.table != nullptr && use_stream(p.max_q, G)) {
    a.q_box = std::min(a.TQ, p.max_q);
    a.ctas = sms;
    a.rows = p.max_q * G;
    a.info = static_cast<int4*>(p.ws);
    a.ws = reinterpret_cast<float*>(static_cast<char*>(p.ws) + info_bytes(sms));
    cudaError_t e = run<D, 1, true, true>(p, a, dim3(sms), st);
    if (e != cudaSuccess) return e;
    attn_stream_join_kernel<D><<<dim3(sms, (a.rows + 7) / 8), 256, 0, st>>>(p, a);
    note_launch();
    return cudaGetLastError();
  }
  a.q_box = a.TQ;
  const int TT = NQ * a.TQ;
  const int64_t items = tile_bound(p.T, p.N, TT) * p.Hkv;
  a.rows = 128 * NQ;
  if (p.table == nullptr) return run<D, NQ, false, false>(p, a, dim3((unsigned)items), st);
  a.splits = tile_splits(items, (int64_t)p.max_pages * p.page_size, sms);
  a.ws = static_cast<float*>(p.ws);
  cudaError_t e = run<D, NQ, true, false>(p, a, dim3((unsigned)items, a.splits), st);
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch_attn_join(p, a.splits, a.rows, TT, st);
}

// What a tensor map takes: strides below 2^40 bytes.
bool map_stride(int64_t s) { return s >= 0 && s < (int64_t)1 << 38; }

}  // namespace

bool attn_tc_supported(const AttnLaunch& p) {
  if (!p.bf16 || p.D < 64) return false;
  if (!map_stride(p.q.ts) || !map_stride(p.q.hs * (p.Hq / p.Hkv))) return false;
  if (p.table == nullptr)
    return map_stride(p.k.ts) && map_stride(p.k.hs) && map_stride(p.v.ts) && map_stride(p.v.hs);
  return p.page_size % 16 == 0 && map_stride(p.kc.ps) && map_stride(p.kc.hs) && map_stride(p.kc.ts) &&
         map_stride(p.vc.ps) && map_stride(p.vc.hs) && map_stride(p.vc.ts);
}

size_t attn_tc_workspace_bytes(int64_t T, int64_t N, int64_t Hq, int64_t Hkv, int64_t D,
                               int64_t max_q) {
  if (D < 64) return 0;
  const int sms = chunk::sm_count();
  const int64_t G = Hq / Hkv;
  if (use_stream(max_q, G))
    return info_bytes(sms) + Partials::bytes(2 * (int64_t)sms, (int)(max_q * G), D);
  const int64_t nq = D <= 128 ? 2 : 1, items = tile_bound(T, N, nq * (128 / G)) * Hkv;
  const int splits = tile_splits(items, INT64_MAX, sms);
  return splits > 1 ? Partials::bytes(items * splits, (int)(128 * nq), D) : 0;
}

cudaError_t launch_attn_tc(const AttnLaunch& p, cudaStream_t st) {
  switch (p.D) {
    case 64: return launch<64>(p, st);
    case 128: return launch<128>(p, st);
    default: return launch<256>(p, st);
  }
}

}  // namespace gdn
