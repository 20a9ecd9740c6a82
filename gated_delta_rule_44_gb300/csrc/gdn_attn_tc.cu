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
// memory.  m is a reference near the running maximum: the first tile's, then raised,
// and O and l scaled, only when the maximum of the tiles before has outgrown it by
// 2^8, which is rare.  It does not matter to P's rounding (2^-8 relative at any
// size); P overflows only where one tile's scores exceed all before by 2^120, and
// such a row is evaluated again (below).  l sums P before the rounding.
//
// Warps:  0       hands out the work; TMA loads of Q and K
//         1, 2    the MMAs: two-tile form, a row tile each, in turns; one-tile form,
//                 Q K^T and P V.  Issuing an MMA takes its warp as long as the pipe
//                 works on it (64 cycles), so that whatever a lone issuer does between
//                 two is a hole in the pipe; here the other warp fills it.  Without
//                 turns two row tiles fall into step and wait for their P together
//         3       TMA loads of V; clears the rows of V past the last visible key (a
//                 stale or foreign NaN there would survive a weight of 0); the
//                 stream form's bookkeeping
//         4-11    softmax and output of row tile 0, two threads per row, each with
//                 half the keys and half the dims of O
//         12-19   the same for row tile 1 (two-tile form)
// K and V each go through their own ring of 16 KB units (K: 128 keys x 64 dims;
// V: 64 keys x 128 dims, or 128 x 64 for D = 64).
// Two-tile form (D <= 128, 256 rows): while one tile's softmax runs on the CUDA
// cores the other's MMAs run.  One-tile form (D = 256, whose O fills half the
// TMEM, and few rows): two S buffers, so that the next key tile's scores are
// computed during a softmax.
// At D = 256 a key tile's K and V are 128 KB for 128 rows, and the SMs together ask
// 11 TB/s of L2 for them, which binds.  A wait costs 150 cycles even for what is there,
// so over prompts and chunks Q K^T has its four units' before that for the S buffer
// (the eight prompts below: 6 % slower with a wait in front of each unit).  Few rows have
// the waits unit by unit.
//
// Work.  The tile form has a grid of (tile, kv head) items, the longest first,
// and with few of them cuts each into key ranges whose sums a second kernel
// joins.  A CTA that nears the end of its item takes the next one off the grid
// (cluster launch control) and loads for it while the last one's rows are
// stored.  The stream form serves sequences whose new rows fit one tile (decode,
// drafts): the key tiles of all (sequence, kv head) pairs, in order, are cut
// into equal consecutive ranges, one per SM, whatever the lengths; a pair cut
// between SMs leaves its sums in the workspace, and a second kernel joins them
// in the order of their keys.
//
// A row whose result is not finite is evaluated again key by key (exact_row):
// the product above multiplies a masked key's weight 0 into its v.
//
// Every wait is bounded (counted from the last sign of a row evaluated again); once one
// gives up, every role leaves at its next wait, copies and MMAs in flight are waited for
// (bounded) and TMEM is freed.
//
// Measured on GB300 (1.93 GHz, hot loop of one key tile pair = 2048 cycles of MMA):
//   one 4096-token prompt, 32 + 4 heads of 128: 109 us, 1.26 PFLOP/s, 65 % of the
//     burst rate of a library product.  An iteration takes 3070 cycles: a tile's
//     chain of scores, softmax (1300), P V and Q K^T (1150) and their latencies is
//     longer than the two tiles' MMAs.
//   2048 tokens over 32768, the same heads, pages of 128: 720-760 us, 1.44-1.52 PFLOP/s,
//     84-88 % of the sustained rate.
//   eight prompts of 512 .. 8192, 16 + 2 heads of 256: 1100-1170 us (the latter call after
//     call, at the power limit), 1.31-1.40 PFLOP/s, 77-82 % of the sustained rate.
//   256 single tokens over 1 .. 16384 keys, 32 + 4 heads of 128, pages of 64: 660-670 us,
//     6.7 TB/s, 99 % of the copy rate.  128 x 1 .. 4 drafts, pages of 16: 352 us, 88 %.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_common.cuh"
#include "gdn_attn_stream.cuh"
#include "gdn_chunk_common.cuh"
#include "gdn_internal.h"
#include "tcgen05.cuh"

namespace gdn {
namespace {

using namespace attn;
using namespace umma;
using bf16 = __nv_bfloat16;

constexpr float kRaise = 8.0f;                   // log2 headroom of the reference m
constexpr int kMaxSplits = 64;

constexpr uint32_t kSmemMax = 232448;  // per CTA

constexpr int kMaxRing = 6;

struct Shared {
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t q_full, q_empty, s_full[2], p_full[2], turn[2], pv[2], o_full[2], o_empty[2], end[2];
  uint64_t v_land[kMaxRing];
  uint64_t pair[2][4];
  uint64_t seg_full[2], seg_empty[2], clc_full;
  alignas(16) uint4 clc;  // the next item's answer
  Seg seg[2];
  uint32_t tmem;
  int abort;
  int redone;  // rows evaluated again so far, and parts of them
  uint32_t k_loads[kMaxRing], v_loads[kMaxRing], v_lands[kMaxRing], q_loads, clc_asked;  // issued so far
  int start_s, start_hkv, start_rt, start_u;
  long long left, total;
  long long scan[20];
  // What the two warps of 32 rows exchange, 256 bytes twice for each of the four
  // pairs of the one-tile form, once for each of the eight of the other.
  alignas(16) unsigned char swap[2048];
};

template <int D, int NQ>
struct Cfg {
  static constexpr uint32_t kUnit = 16384;
  static constexpr int NU = D / 64;                       // units of a key tile, of K and of V
  static constexpr int VK = D == 64 ? 128 : 64;           // keys of a V unit
  static constexpr int VD = D == 64 ? 64 : 128;           // its dims
  static constexpr uint32_t kQTile = 128 * D * 2;
  static constexpr uint32_t kQ = NQ * kQTile;
  static constexpr int kFit = (int)((kSmemMax - sizeof(Shared) - kQ) / kUnit) / 2;
  static constexpr int ST = kFit > kMaxRing ? kMaxRing : kFit;  // units of either ring
  static constexpr uint32_t kBars = kQ + 2 * ST * kUnit;
  static constexpr uint32_t kBytes = kBars + sizeof(Shared);
  static constexpr int kThreads = 128 + 256 * NQ;
  static constexpr int kReaders = 3 + 8 * NQ;  // warps that read the handed-out work
};
static_assert(Cfg<128, 2>::ST >= 5 && Cfg<256, 1>::ST >= 5, "units in flight");

// TMEM columns (512 allocated): S buffers of 128, then O.
constexpr uint32_t kTO = 256;

struct TcArgs {
  int splits;   // key ranges per tile (tile form)
  int TQ;       // tokens per row tile: 128 / G
  int q_box;    // tokens of a Q load
  int pbk, pbv; // rows of a load of K, of V: a unit's keys, or a divisor of the page
  int ctas;     // stream form: the grid
  int rows;     // rows of a workspace block
  int tq;       // stream form: tokens of a pair (all of a sequence's)
  int4* info;   // stream form, per CTA: see stream_info
  float* ws;    // the sums
};

// Inside a role: the bounded wait, or leave the role.
#define WAIT(bar, parity) \
  if (!warp_wait(&(bar), (parity), sh, p.status)) return

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Asks for a further CTA of the grid in place of its launch.
__device__ __forceinline__ void clc_ask(Shared* sh) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];\n" ::"r"(smem_u32(&sh->clc)),
      "r"(smem_u32(&sh->clc_full))
      : "memory");
}
// The answer: false when no CTA was left.
__device__ __forceinline__ bool clc_answer(Shared* sh, uint32_t& x, uint32_t& y) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%3];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, _, _}, r;\n\t}\n"
      : "=r"(ok), "=&r"(x), "=&r"(y)
      : "r"(smem_u32(&sh->clc))
      : "memory");
  return ok != 0;
}

template <int D, int NQ, bool PAGED, bool STREAM>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnLaunch p, const __grid_constant__ CUtensorMap mq,
                   const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ TcArgs a) {
  using C = Cfg<D, NQ>;
  constexpr int NU = C::NU, ST = C::ST, VK = C::VK, VD = C::VD;
  extern __shared__ __align__(1024) unsigned char smem[];  // the swizzle atoms' alignment
  Shared* sh = reinterpret_cast<Shared*>(smem + C::kBars);
  const uint32_t sq = smem_u32(smem), sk = sq + C::kQ, sv = sk + ST * C::kUnit;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;

  start_next_kernel();
  if (warp == 0) {
    if (lane == 0) {
      constexpr int kReleases = NQ;  // MMA warps that use a unit
      for (int i = 0; i < ST; ++i) {
        mbar_init(smem_u32(&sh->k_full[i]), 1);
        mbar_init(smem_u32(&sh->k_empty[i]), kReleases);
        mbar_init(smem_u32(&sh->v_full[i]), 1);
        mbar_init(smem_u32(&sh->v_empty[i]), kReleases);
        mbar_init(smem_u32(&sh->v_land[i]), 1);
        sh->k_loads[i] = sh->v_loads[i] = sh->v_lands[i] = 0;
      }
      mbar_init(smem_u32(&sh->q_full), 1);
      mbar_init(smem_u32(&sh->q_empty), NQ);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&sh->s_full[i]), 1);
        mbar_init(smem_u32(&sh->p_full[i]), 8);
        mbar_init(smem_u32(&sh->turn[i]), 1);
        mbar_init(smem_u32(&sh->pv[i]), 1);
        mbar_init(smem_u32(&sh->o_full[i]), 1);
        mbar_init(smem_u32(&sh->o_empty[i]), 8);
        mbar_init(smem_u32(&sh->end[i]), 1);
        mbar_init(smem_u32(&sh->seg_full[i]), 1);
        mbar_init(smem_u32(&sh->seg_empty[i]), C::kReaders);
        for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&sh->pair[i][w]), 2);
      }
      mbar_init(smem_u32(&sh->clc_full), 1);
      sh->abort = sh->redone = 0;
      sh->q_loads = sh->clc_asked = 0;
      fence_mbar_init();
    }
  } else if (warp == 2) {
    tmem_alloc(smem_u32(&sh->tmem), 512);
  }
  if constexpr (STREAM) stream_start<C::kThreads, false>(p, a.ctas, a.tq, sh);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  // All 512 columns: their base is 0, which the addresses below use as such.
  if (sh->tmem != 0 && tid == 0) atomicOr(p.status, kStatusTimeout);
  constexpr uint32_t tmem = 0;

  // The ranges handed out by warp 0, through two places, to every other role.
  int seg_in = 0;
  auto next_seg = [&](Seg& g) -> bool {
    const int i = seg_in & 1;
    if (!warp_wait(&sh->seg_full[i], (seg_in >> 1) & 1, sh, p.status)) return false;
    g = sh->seg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->seg_empty[i]));
    ++seg_in;
    return g.s >= 0;
  };
  // A ring's position: place and parity of its round.
  struct Ring {
    uint32_t st = 0, round = 0;
    __device__ void step() {
      if (++st == ST) {
        st = 0;
        round ^= 1;
      }
    }
  };
  if (warp == 0) {
    // ---- work; loads of Q and K ----
    SegIter<false> iter{};
    if constexpr (STREAM)
      iter = SegIter<false>{sh->start_s, sh->start_hkv, sh->start_rt, sh->start_u, (int)blockIdx.x, a.tq, sh->left};
    auto role = [&] {
      Ring ring;
      uint32_t filled = 0;  // units so far
      int nseg = 0, loads = 0, asked = 0;
      bool more = true;     // the tile form's grid may have an item left
      uint32_t bx = blockIdx.x, by = blockIdx.y;
      for (;;) {
        // The next range, into g.
        Seg g;
        g.s = -1;
        if constexpr (STREAM) {
          if (!iter.next(p, g)) g.s = -1;
        } else {
          while (more) {
            const int item = (int)bx;
            const int id = (int)(gridDim.x / p.Hkv) - 1 - item / p.Hkv;
            const SeqTile t = find_tile(p, id, NQ * a.TQ);
            if ((lane == 0 && t.bad) ||
                (lane == 1 && by == 0 && item % p.Hkv == 0 && own_range_bad(p, id)))
              atomicOr(p.status, kStatusBadSeqlens);
            if (t.nt > 0) {
              g.s = t.s;
              g.hkv = item % p.Hkv;
              g.t0 = t.t0;
              g.nt = t.nt;
              g.pos0 = t.pos0;
              g.hi = max(0, t.pos0 + t.nt);
              const int n = (g.hi + BK - 1) / BK;
              g.kt0 = (int)((int64_t)n * by / a.splits);
              g.kt1 = (int)((int64_t)n * (by + 1) / a.splits);
              g.slot = a.splits > 1 ? ((int64_t)id * p.Hkv + g.hkv) * a.splits + by : -1;
            }
            // The item after this one is asked for now and taken when this one's
            // loads have been issued.
            if (asked > 0) fence_proxy_async();  // the last answer has been read
            __syncwarp();
            if (elect_one()) {
              sh->clc_asked = asked + 1;
              mbar_expect_tx(smem_u32(&sh->clc_full), 16);
              clc_ask(sh);
            }
            ++asked;
            if (g.s >= 0) break;
            if (!warp_wait(&sh->clc_full, (asked - 1) & 1, sh, p.status)) return;
            more = uni((int)clc_answer(sh, bx, by));
          }
        }
        {
          const int i = nseg & 1;
          if (nseg >= 2)
            if (!warp_wait(&sh->seg_empty[i], ((nseg >> 1) - 1) & 1, sh, p.status)) return;
          if (lane == 0) {
            sh->seg[i] = g;
            mbar_arrive(smem_u32(&sh->seg_full[i]));
          }
          __syncwarp();
          ++nseg;
        }
        if (g.s < 0) return;
        const int kt0 = uni(g.kt0), n = uni(g.kt1) - kt0, hi = uni(g.hi), hkv = uni(g.hkv);
        const int per_tile = BK / a.pbk;
        const int row0 = PAGED ? 0 : uni(cu_at(p.cu, g.s));
        // Lane i looks up the page of, and issues, the i-th group of pbk keys.  (A
        // loop over the groups with one elected lane was slower: 461 against
        // 380 us for drafts over pages of 16 rows.)
        auto find_page = [&](int kt) -> int {
          const int jb = kt * BK + lane * a.pbk;
          if (!PAGED || lane >= per_tile || kt >= kt0 + n || jb >= hi) return 0;
          const int64_t pg = page_of(p, g.s, jb / p.page_size);
          if (pg < 0) atomicOr(p.status, kStatusBadIndex);
          return pg < 0 ? (int)p.num_pages : (int)pg;  // past the end: reads as zeros
        };
        int next_page = find_page(kt0);
        for (int j = 0; j < n; ++j) {
          const int j0 = (kt0 + j) * BK;
          const int page = next_page;
          next_page = find_page(kt0 + j + 1);  // its latency passes during this tile's waits
          const int groups = min(per_tile, (hi - j0 + a.pbk - 1) / a.pbk);
#pragma unroll
          for (int u = 0; u < NU; ++u, ring.step(), ++filled) {
            if (filled >= ST)
              if (!warp_wait(&sh->k_empty[ring.st], ring.round ^ 1, sh, p.status)) return;
            const uint32_t full = smem_u32(&sh->k_full[ring.st]), dst = sk + ring.st * C::kUnit;
            if (elect_one()) {
              ++sh->k_loads[ring.st];
              mbar_expect_tx(full, groups * a.pbk * 128u);
              if constexpr (!PAGED) tma_load_3d(dst, &mk, full, u * 64, row0 + j0, hkv);
            }
            if constexpr (PAGED) {
              __syncwarp();
              const int row = (j0 + lane * a.pbk) % p.page_size;
              if (lane < groups) tma_load_4d(dst + lane * a.pbk * 128, &mk, full, u * 64, row, hkv, page);
              __syncwarp();
            }
          }
          if (j == 0) {  // Q, once the last range's scores are done
            const int nq = uni((NQ == 2 && g.nt > a.TQ) ? 2 : 1), t0 = uni(g.t0);
            if (loads > 0)
              if (!warp_wait(&sh->q_empty, (loads - 1) & 1, sh, p.status)) return;
            ++loads;
            if (elect_one()) {
              sh->q_loads = loads;
              mbar_expect_tx(smem_u32(&sh->q_full), nq * NU * 128u * G * a.q_box);
              for (int q = 0; q < nq; ++q)
#pragma unroll
                for (int b = 0; b < NU; ++b)
                  tma_load_4d(sq + q * C::kQTile + b * 16384, &mq, smem_u32(&sh->q_full), b * 64, 0, hkv,
                              t0 + q * a.TQ);
            }
          }
        }
        if constexpr (!STREAM) {
          if (!warp_wait(&sh->clc_full, (asked - 1) & 1, sh, p.status)) return;
          more = uni((int)clc_answer(sh, bx, by));
        }
      }
    };
    role();
  } else if (warp == 1 || warp == 2) {
    // ---- MMAs ----
    constexpr uint32_t kIdQK = idesc_bf16_f32(128, BK, false, false);
    constexpr uint32_t kIdPV = idesc_bf16_f32(128, VD, false, true);
    // Two-tile form: this warp's row tile; the warps take turns, and wait for what
    // a turn needs before it.  One-tile form: warp 1 has the scores, warp 2 P V.
    const int me = warp - 1, q = NQ == 2 ? me : 0;
    Ring kr, vr;
    int turns = 0;
    auto wait = [&](uint64_t& bar, uint32_t parity) { return warp_wait(&bar, parity, sh, p.status); };
    auto take_turn = [&]() -> bool {
      const int k = turns++ - (me == 0 ? 1 : 0);  // warp 1 begins
      return k < 0 || wait(sh->turn[me], k & 1);
    };
    auto pass_turn = [&] {
      if (elect_one()) mbar_arrive(smem_u32(&sh->turn[me ^ 1]));
    };
    // The next key tile's units of a ring have landed; their places.
    auto land = [&](Ring& ring, uint64_t* full, uint32_t(&at)[NU]) -> bool {
#pragma unroll
      for (int u = 0; u < NU; ++u, ring.step()) {
        at[u] = ring.st;
        if (!wait(full[ring.st], ring.round)) return false;
      }
      return true;
    };
    // The MMAs so far have read the unit.
    auto release = [&](uint64_t* empty) { mma_commit(smem_u32(empty)); };
    // S[buf] = Q[q] K^T of unit u.
    auto qk_unit = [&](uint32_t buf, int u, uint32_t at) {
      if (elect_one()) {
        const uint64_t kd = desc_sw128(sk + at * C::kUnit, 16, 1024);
        const uint64_t qd = desc_sw128(sq + q * C::kQTile + u * 16384, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(buf * 128, qd + k * 2, kd + k * 2, kIdQK, u + k > 0);
        release(&sh->k_empty[at]);
        if (u == NU - 1) mma_commit(smem_u32(&sh->s_full[buf]));
      }
    };
    // O[q] (+)= P[buf] V of the key tile's unit u (keys outermost).
    auto pv_unit = [&](uint32_t buf, bool acc, int u, uint32_t at) {
      constexpr int ND = D / VD;  // units side by side in the dims
      if (elect_one()) {
        const uint64_t vd = desc_sw128(sv + at * C::kUnit, VK * 128, 1024);
#pragma unroll
        for (int k = 0; k < VK / 16; ++k) {
          const int ks = (u / ND) * (VK / 16) + k;  // step of 16 keys in the tile
          mma_bf16_ta(kTO + q * 128 + (u % ND) * VD, buf * 128 + (ks >> 2) * 64 + (ks & 3) * 8,
                      vd + ((k * 2048) >> 4), kIdPV, acc || ks > 0);
        }
        release(&sh->v_empty[at]);
      }
    };
    auto role = [&] {
      uint32_t nk = 0;  // key tiles before this range (of this row tile)
      int nseg = 0, nact = 0;  // ranges, of them with rows of tile q
      uint32_t ak[NU], av[NU];
      Seg g;
      while (next_seg(g)) {
        const int n = uni(g.kt1 - g.kt0);
        if (n == 0) continue;
        if constexpr (NQ == 2) {
          const bool idle = uni((int)(q == 1 && g.nt <= a.TQ));  // no row of this tile
          if (!wait(sh->q_full, nseg & 1)) return;
          // Turn 0: the scores of key tile 0; turn j + 1: P V of tile j and the scores
          // of tile j + 1.
          for (int j = -1; j < n; ++j) {
            if (j >= 0)
              if (!land(vr, sh->v_full, av)) return;
            if (j + 1 < n)
              if (!land(kr, sh->k_full, ak)) return;
            if (j == 0 && nact > 0 && !idle)  // the last range's O has been read
              if (!wait(sh->o_empty[q], (nact - 1) & 1)) return;
            if (!take_turn()) return;
            if (j >= 0 && !idle)
              if (!wait(sh->p_full[q], nk & 1)) return;
            fence_after_sync();
            if (idle) {
              pass_turn();
              if (elect_one()) {
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                  if (j >= 0) mbar_arrive(smem_u32(&sh->v_empty[av[u]]));
                  if (j + 1 < n) mbar_arrive(smem_u32(&sh->k_empty[ak[u]]));
                }
              }
              continue;
            }
            if (j >= 0) {
#pragma unroll
              for (int u = 0; u < NU; ++u) pv_unit(q, j > 0, u, av[u]);
              if (j == n - 1 && elect_one()) mma_commit(smem_u32(&sh->o_full[q]));
              ++nk;
            }
            if (j + 1 < n) {
#pragma unroll
              for (int u = 0; u < NU; ++u) {
                if (u == NU - 1) pass_turn();
                qk_unit(q, u, ak[u]);
              }
            } else {
              pass_turn();
            }
          }
          nact += idle ? 0 : 1;
          if (elect_one()) mma_commit(smem_u32(&sh->q_empty));
        } else if (warp == 1) {
          if (!wait(sh->q_full, nseg & 1)) return;
          for (int j = 0; j < n; ++j, ++nk) {
            if constexpr (!STREAM)  // (for single tokens, bound by the reads of K, 1 % slower)
              if (!land(kr, sh->k_full, ak)) return;
            if (nk >= 2)  // P V has read the buffer's last P
              if (!wait(sh->pv[nk & 1], ((nk >> 1) - 1) & 1)) return;
            fence_after_sync();
            if constexpr (!STREAM) {
#pragma unroll
              for (int u = 0; u < NU; ++u) qk_unit(nk & 1, u, ak[u]);
            } else {
#pragma unroll
              for (int u = 0; u < NU; ++u, kr.step()) {
                if (!wait(sh->k_full[kr.st], kr.round)) return;
                fence_after_sync();
                qk_unit(nk & 1, u, kr.st);
              }
            }
          }
          if (elect_one()) mma_commit(smem_u32(&sh->q_empty));
        } else {
          for (int j = 0; j < n; ++j, ++nk) {
            if (!land(vr, sh->v_full, av)) return;
            if (j == 0 && nseg > 0)
              if (!wait(sh->o_empty[0], (nseg - 1) & 1)) return;
            if (!wait(sh->p_full[nk & 1], (nk >> 1) & 1)) return;
            fence_after_sync();
#pragma unroll
            for (int u = 0; u < NU; ++u) pv_unit(nk & 1, j > 0, u, av[u]);
            if (elect_one()) {
              mma_commit(smem_u32(&sh->pv[nk & 1]));
              if (j == n - 1) mma_commit(smem_u32(&sh->o_full[0]));
            }
          }
        }
        ++nseg;
      }
    };
    role();
    __syncwarp();
    if (elect_one()) mma_commit(smem_u32(&sh->end[warp - 1]));
    mbar_wait(smem_u32(&sh->end[warp - 1]), 0, kWaitBudget);
  } else if (warp == 3) {
    // ---- loads of V ----
    auto role = [&] {
      Ring ring;
      uint32_t filled = 0, landed = 0;  // bit i: phase of v_land[i]
      Seg g;
      while (next_seg(g)) {
        const int kt0 = uni(g.kt0), n = uni(g.kt1) - kt0, hi = uni(g.hi), hkv = uni(g.hkv);
        const int row0 = PAGED ? 0 : uni(cu_at(p.cu, g.s));
        constexpr int NB = VD / 64;
        const int per_unit = VK / a.pbv, per_tile = BK / a.pbv;
        const int grp = lane / NB, blk = lane % NB;  // this lane's load of a unit
        auto find_page = [&](int kt) -> int {  // lane i: of the tile's i-th group of pbv keys
          const int jb = kt * BK + lane * a.pbv;
          if (!PAGED || lane >= per_tile || kt >= kt0 + n || jb >= hi) return 0;
          const int64_t pg = page_of(p, g.s, jb / p.page_size);
          return pg < 0 ? (int)p.num_pages : (int)pg;
        };
        int next_page = find_page(kt0);
        for (int j = 0; j < n; ++j) {
          const int j0 = (kt0 + j) * BK;
          const int pages = next_page;
          next_page = find_page(kt0 + j + 1);
          const int r0 = hi - j0;  // the first row past the last visible key, if below 128
          const bool tail = r0 < BK;
          Ring first = ring;
#pragma unroll
          for (int u = 0; u < NU; ++u, ring.step(), ++filled) {
            constexpr int ND = D / VD;
            const int kh = u / ND, db = u % ND;
            if (filled >= ST)
              if (!warp_wait(&sh->v_empty[ring.st], ring.round ^ 1, sh, p.status)) return;
            // Units of a tile with a tail land on barriers of their own and are passed on
            // below.
            const uint32_t full = smem_u32(tail ? &sh->v_land[ring.st] : &sh->v_full[ring.st]);
            const uint32_t dst = sv + ring.st * C::kUnit;
            // Loads of groups with a visible key; none for a unit past the last one.
            const int groups = max(0, min(per_unit, (r0 - kh * VK + a.pbv - 1) / a.pbv));
            if (elect_one()) {
              ++(tail ? sh->v_lands : sh->v_loads)[ring.st];
              mbar_expect_tx(full, groups * NB * a.pbv * 128u);
              if constexpr (!PAGED) {
                if (groups > 0)
#pragma unroll
                  for (int b = 0; b < NB; ++b) {
                    const int d = db * VD + b * 64, row = row0 + j0 + kh * VK;
                    tma_load_3d(dst + b * VK * 128, &mv, full, d, row, hkv);
                  }
              }
            }
            if constexpr (PAGED) {
              const int page = __shfl_sync(0xffffffffu, pages, (kh * per_unit + grp) & 31);
              const uint32_t to = dst + blk * VK * 128 + grp * a.pbv * 128;
              const int d = db * VD + blk * 64, row = (j0 + kh * VK + grp * a.pbv) % p.page_size;
              if (grp < groups) tma_load_4d(to, &mv, full, d, row, hkv, page);
              __syncwarp();
            }
          }
          if (tail) {
            // Whole 128-byte rows: the swizzle permutes inside a row only.
            Ring at = first;
#pragma unroll
            for (int u = 0; u < NU; ++u, at.step()) {
              if (!warp_wait(&sh->v_land[at.st], (landed >> at.st) & 1, sh, p.status)) return;
              landed ^= 1u << at.st;
              constexpr int ND = D / VD;
              const int c0 = max(0, r0 - (u / ND) * VK);  // first row of the unit to clear
              unsigned char* v = smem + C::kQ + (ST + at.st) * C::kUnit;
              for (int i = lane; i < (VK - c0) * (VD / 8); i += 32) {
                const int r = c0 + i / (VD / 8), ch = i % (VD / 8);
                *reinterpret_cast<uint4*>(v + (ch >> 3) * (VK * 128) + r * 128 + (ch & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
              }
            }
            fence_proxy_async();
            __syncwarp();
#pragma unroll
            for (int u = 0; u < NU; ++u, first.step())
              if (elect_one()) {
                ++sh->v_loads[first.st];
                mbar_arrive(smem_u32(&sh->v_full[first.st]));
              }
          }
        }
      }
    };
    role();
    if constexpr (STREAM) {
      // What the joining kernel needs of this CTA's ranges; the outputs of
      // sequences without a key.
      if (lane == 0) {
        a.info[blockIdx.x] = stream_info<false>(p, a.ctas, a.tq, sh);
      }
      for (int s = blockIdx.x; s < p.N; s += a.ctas) {
        const SeqRange q = seq_range(p, s);
        if (key_tiles(q) > 0) continue;
        const float zero[D / 32] = {};
        for (int t = q.a; t < q.b; ++t)
          for (int h = 0; h < p.Hq; ++h) finish_row<bf16, D>(p, t, h, lane, zero, -INFINITY, 0.0f);
      }
    }
  } else {
    // ---- softmax, output ----
    // Two warps share 32 rows: `half` is the half of the keys of a tile, and of
    // the dims of O, that this one handles.
    const int sw = warp - 4, half = (sw >> 2) & 1, qt = NQ == 2 ? sw >> 3 : 0;
    const int r = tid & 127;                            // row of the tile, lane of TMEM
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // (32 * (warp % 4)) << 16
    const float c = p.scale * kLog2e;
    const float2 c2 = make_float2(c, c);
    const int tok = qt * a.TQ + r / G;                  // token of the tile
    auto role = [&] {
    uint32_t nk = 0, np = 0;
    // Meeting the pair's other warp (bounded; false: leave).
    uint64_t& pair = sh->pair[qt][warp & 3];
    // Values in f32 [half][row], and maxima in bf16 [key tile & 1][half][row].  In the
    // two-tile form they share their place: the scores of a tile wait for the P of
    // the one before of both warps, so that neither can write one kind while the
    // other warp still reads the other.
    unsigned char* mine = sh->swap + (NQ == 2 ? (qt * 4 + (warp & 3)) * 256 : (warp & 3) * 512);
    float* val = reinterpret_cast<float*>(mine) + lane;
    uint16_t* tops = reinterpret_cast<uint16_t*>(mine + (NQ == 2 ? 0 : 256)) + lane;
    auto pair_arrive = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&pair));
    };
    auto pair_wait = [&]() -> bool { return warp_wait(&pair, np++ & 1, sh, p.status); };
    // x becomes the row's value of it from the other warp (between two meetings
    // that keep `val` from being written early).
    auto swap = [&](float& x) -> bool {
      val[half * 32] = x;
      pair_arrive();
      const bool ok = pair_wait();
      x = val[(half ^ 1) * 32];
      return ok;
    };
    int seg_n = 0;
    Seg g;
    while (next_seg(g)) {
      if (NQ == 2 && qt == 1 && g.nt <= a.TQ) continue;   // no second row tile
      if (g.kt0 == g.kt1) {  // no key for any row
        const Partials part(a.ws, (int64_t)gridDim.x * a.splits, a.rows, D);
        const float zero[D / 32] = {};
        const int rows = (min(g.nt, (qt + 1) * a.TQ) - qt * a.TQ) * G;
        for (int i = (warp - 4) & 7; i < rows; i += 8) {
          const int in_tile = qt * a.TQ * G + i, t = g.t0 + in_tile / G, h = g.hkv * G + in_tile % G;
          if (g.slot >= 0) part.put<D / 32>(g.slot, in_tile, lane, zero, -INFINITY, 0.0f);
          else finish_row<bf16, D>(p, t, h, lane, zero, -INFINITY, 0.0f);
        }
        continue;
      }
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
      // A row with keys but no score in the first tile of the range (all of them -inf)
      // has no reference for the others, which may lie where a weight relative to 0 is 0
      // or infinite: it is evaluated again, too.
      float m = -INFINITY, l = 0.0f;
      bool scoreless = false;
      uint32_t top_bits = 0;  // this warp's last published maximum
      const uint32_t to = tmem + lanes + kTO + qt * 128 + half * (D / 2);
      for (int kt = g.kt0; kt < g.kt1; ++kt, ++nk) {
        const int buf = NQ == 2 ? qt : (int)(nk & 1);
        const uint32_t ph = NQ == 2 ? nk & 1 : (nk >> 1) & 1;
        const int jj = kt - g.kt0;
        // Takes a maximum of both halves (m of the first tile becomes it); raise: m grew.
        float f = 1.0f;
        bool raise = false;
        auto raise_to = [&](float top) {
          if (top > m + kRaise) {
            raise = valid && jj > 0;
            f = ex2(m - top);
            m = top;
          }
        };
        if (jj > 1 && !idle) {
          if (!pair_wait()) return;
          const uint32_t their_bits = tops[(((jj - 1) & 1) * 2 + (half ^ 1)) * 32];
          raise_to(fmaxf(__uint_as_float(top_bits << 16), __uint_as_float(their_bits << 16)));
        }
        const bool raising = __any_sync(0xffffffffu, raise);
        const int lim = last - kt * BK - half * 64;  // the row's last visible column
        const bool masked = __any_sync(0xffffffffu, lim < 63);
        WAIT(sh->s_full[buf], ph);
        fence_after_sync();
        if (!idle) {
          const uint32_t ts = tmem + lanes + buf * 128;
          auto scores = [&](float(&y)[32], int i) {
            tmem_ld32(ts + half * 64 + i * 32, y);
            tmem_ld_wait();
            if (masked) {
              const int li = lim - i * 32;
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = e <= li ? y[e] : -INFINITY;
            }
          };
          if (jj == 0) {
            float t = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              float y[32];
              scores(y, i);
#pragma unroll
              for (int e = 0; e < 32; e += 2) t = fmaxf(t, fmaxf(y[e], y[e + 1]));
            }
            // In full f32: a row whose largest weight is then exactly 1 loses nothing
            // of it to P's rounding.  (0 * -inf must not count as a score.)
            t = t == -INFINITY ? t : t * c;
            float theirs = t;
            if (!swap(theirs)) return;
            raise_to(fmaxf(t, theirs));
            if (m == -INFINITY) {  // no score above -inf: a reference that no score gave
              m = 0.0f;
              scoreless = last >= kt * BK;
            }
          }
          if (raising) {
            // O is at rest: in the two-tile form S j follows P V j-1, in the other
            // that product is waited for.
            if constexpr (NQ == 1) {
              WAIT(sh->pv[(nk - 1) & 1], ((nk - 1) >> 1) & 1);
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
          float2 sum01 = make_float2(0.0f, 0.0f), sum23 = sum01;
          __nv_bfloat162 big = __float2bfloat162_rn(0.0f);
          const float2 nm2 = make_float2(-m, -m);
          // 16 columns at a time in a rolled loop: unrolled, the roles' loops together
          // overflowed the instruction cache (95 % hits) and the registers, and an
          // iteration took 4800 cycles, most of them waiting for instructions and
          // spills.  P's 8 columns of a step go where scores have been read.  The
          // next reference comes from the largest P, two at a time in bf16.
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            float y[16];
            tmem_ld16(ts + half * 64 + i * 16, y);
            tmem_ld_wait();
            if (masked) {
              const int li = lim - i * 16;
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = e <= li ? y[e] : -INFINITY;
            }
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 w = __ffma2_rn(make_float2(y[e], y[e + 1]), c2, nm2);
              w.x = ex2(w.x);
              w.y = ex2(w.y);
              float2& sum = e & 2 ? sum23 : sum01;
              sum = __fadd2_rn(sum, w);
              const __nv_bfloat162 h = __floats2bfloat162_rn(w.x, w.y);
              big = __hmax2(big, h);
              pk[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
            }
            tmem_st8u(ts + half * 64 + i * 8, pk);
          }
          tmem_st_wait();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[buf]));
          sum01 = __fadd2_rn(sum01, sum23);
          l += sum01.x + sum01.y;
          if (jj > 0 && kt + 1 < g.kt1) {
            // Published in bf16, rounded towards -inf: a reference above the scores by as
            // much as a bf16 step of -20000 (128) would leave their weights out of f32's
            // range, while one below them makes a weight that overflows, which is seen.
            const float t = m + log2f(fmaxf(__low2float(big), __high2float(big)));
            top_bits = (__float_as_uint(t) + (t < 0.0f ? 0xffffu : 0u)) >> 16;
            tops[((jj & 1) * 2 + half) * 32] = (uint16_t)top_bits;
            pair_arrive();
          }
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
      // The gate's loads go out before the wait and a chunk of 16 dims ahead: one
      // at a time, just before use, they were half the time of a short row.
      uint4 gw[2];
      if (gated) {
#pragma unroll
        for (int e = 0; e < 2; ++e) gw[e] = gate[e];
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
        bool finite = isfinite(l) && !scoreless;
        bf16* out = static_cast<bf16*>(p.out) + ((int64_t)t * p.Hq + h) * D + half * (D / 2);
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[16];
          tmem_ld16(to + i * 16, o);
          tmem_ld_wait();
          float big = 0.0f;  // NaN and infinities survive a sum of x - x
#pragma unroll
          for (int e = 0; e < 16; ++e) big += o[e] - o[e];
          finite = finite && big == 0.0f;
          if (g.slot >= 0) {
            if (valid) {
              float4* d = reinterpret_cast<float4*>(part.o + (g.slot * a.rows + pr) * D +
                                                    half * (D / 2) + i * 16);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
            continue;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= inv;
          if (gated) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t gp[4] = {gw[e].x, gw[e].y, gw[e].z, gw[e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[e * 8 + 2 * k] *= sigmoid_gate(__uint_as_float(gp[k] << 16));
                o[e * 8 + 2 * k + 1] *= sigmoid_gate(__uint_as_float(gp[k] & 0xffff0000u));
              }
            }
            if (i + 1 < D / 32) {
#pragma unroll
              for (int e = 0; e < 2; ++e) gw[e] = gate[(i + 1) * 2 + e];
            }
          }
          if (valid) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = pack_bf16(o[e * 8 + 2 * k], o[e * 8 + 2 * k + 1]);
              *reinterpret_cast<uint4*>(out + i * 16 + e * 8) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (valid && half == 0) {
          if (g.slot >= 0) part.ml[g.slot * a.rows + pr] = make_float2(l == 0.0f ? -INFINITY : m, l);
          else if (p.lse != nullptr)
            p.lse[(int64_t)t * p.Hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        // Rows to evaluate again once both warps have stored, every other one by either.
        pair_arrive();
        if (!pair_wait()) return;
        theirs = finite ? 1.0f : 0.0f;
        if (!swap(theirs)) return;
        unsigned redo = __ballot_sync(0xffffffffu, valid && !(finite && theirs == 1.0f));
        pair_arrive();  // `theirs` has been read: the next range may publish
        if (!pair_wait()) return;
        redo &= half ? 0xaaaaaaaau : 0x55555555u;
        while (redo) {
          const int src = __ffs(redo) - 1;
          redo &= redo - 1;
          const int rt = __shfl_sync(0xffffffffu, t, src), rh = __shfl_sync(0xffffffffu, h, src);
          const int rl = __shfl_sync(0xffffffffu, last, src), rp = __shfl_sync(0xffffffffu, pr, src);
          float acc[D / 32], em, el;
          exact_row<bf16, D>(p, g.s, cu_at(p.cu, g.s), rt, rh, g.kt0 * BK, min(g.kt1 * BK, rl + 1), acc,
                             em, el, &sh->redone);
          if (g.slot >= 0) part.put<D / 32>(g.slot, rp, lane, acc, em, el);
          else finish_row<bf16, D>(p, rt, rh, lane, acc, em, el);
          if (lane == 0) atomicAdd(&sh->redone, 1);
        }
      }
      ++seg_n;
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh->o_empty[qt]));
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
      for (int i = 0; i < ST; ++i) {
        if (sh->k_loads[i]) mbar_wait(smem_u32(&sh->k_full[i]), (sh->k_loads[i] - 1) & 1, kWaitBudget);
        if (sh->v_lands[i]) mbar_wait(smem_u32(&sh->v_land[i]), (sh->v_lands[i] - 1) & 1, kWaitBudget);
        if (sh->v_loads[i]) mbar_wait(smem_u32(&sh->v_full[i]), (sh->v_loads[i] - 1) & 1, kWaitBudget);
      }
      if (sh->q_loads) mbar_wait(smem_u32(&sh->q_full), (sh->q_loads - 1) & 1, kWaitBudget);
      if (sh->clc_asked) mbar_wait(smem_u32(&sh->clc_full), (sh->clc_asked - 1) & 1, kWaitBudget);
    }
    __syncthreads();
  }
  if (warp == 2) tmem_dealloc(sh->tmem, 512);
}

template <int D>
__global__ void __launch_bounds__(256) attn_stream_join_kernel(const __grid_constant__ AttnLaunch p,
                                                               const __grid_constant__ TcArgs a) {
  stream_join<bf16, D, false>(p, a);
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
bool rows_map(CUtensorMap* m, const AttnRows& r, const AttnLaunch& p, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.T, (cuuint64_t)p.Hkv};
  const int64_t st[2] = {r.ts, r.hs};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
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

template <int D, int NQ, bool PAGED, bool STREAM>
cudaError_t run(const AttnLaunch& p, TcArgs a, dim3 grid, cudaStream_t st) {
  using C = Cfg<D, NQ>;
  CUtensorMap mq, mk, mv;
  if (!q_map(&mq, p, a.q_box) || !(PAGED ? pages_map(&mk, p.kc, p, a.pbk) : rows_map(&mk, p.k, p, a.pbk)) ||
      !(PAGED ? pages_map(&mv, p.vc, p, a.pbv) : rows_map(&mv, p.v, p, a.pbv)))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> devices{0};
  const cudaError_t attr = allow_shared(attn_tc_kernel<D, NQ, PAGED, STREAM>, C::kBytes, devices);
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
  a.pbk = BK;
  if (p.table != nullptr)
    while (p.page_size % a.pbk != 0) a.pbk >>= 1;
  a.pbv = std::min(a.pbk, Cfg<D, NQ>::VK);
  if (p.table != nullptr && use_stream(p.max_q, G)) {
    a.q_box = std::min(a.TQ, p.max_q);
    a.ctas = sms;
    a.rows = p.max_q * G;
    a.tq = p.max_q;
    a.info = static_cast<int4*>(p.ws);
    a.ws = reinterpret_cast<float*>(static_cast<char*>(p.ws) + info_bytes(sms));
    cudaError_t e = run<D, 1, true, true>(p, a, dim3(sms), st);
    if (e != cudaSuccess) return e;
    return launch_after(attn_stream_join_kernel<D>, dim3(sms, std::min(a.rows, 16)), 256, st, 0, p, a);
  }
  a.q_box = a.TQ;
  const int TT = NQ * a.TQ;
  const int64_t items = tile_bound(p.T, p.N, TT) * p.Hkv;
  a.rows = NQ * 128;
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
  const int NQ = D <= 128 ? tiles_of<128>() : tiles_of<256>();
  const int64_t items = tile_bound(T, N, NQ * (128 / G)) * Hkv;
  const int splits = tile_splits(items, INT64_MAX, sms);
  return splits > 1 ? Partials::bytes(items * splits, NQ * 128, D) : 0;
}

cudaError_t launch_attn_tc(const AttnLaunch& p, cudaStream_t st) {
  switch (p.D) {
    case 64: return launch<64>(p, st);
    case 128: return launch<128>(p, st);
    default: return launch<256>(p, st);
  }
}

}  // namespace gdn
