// gdn_attn8_tc.cu -- attention of up to 256 rows per kv head (decode, drafts, short chunks)
// over a cache in 8 bits, on tcgen05 tensor cores, without widening a code.
//
// The codes go from the cache to the tensor cores as they are; what is multiplied with
// them comes in e4m3 parts.  q, scaled by a power of two per row, in two, x ~ hi + lo / 32 with
// hi = e4m3(x), lo = e4m3(32 (x - hi)), which hold it exactly down to 2^-10 of the row's largest
// value (a bf16 has 8 significant bits, the parts 4 and a sign each).  The products are
// transposed, so that the 128 rows of an MMA are keys or dims, all in use, and the few rows
// of q are its columns, twice, for hi and lo:
//   S^T [128 keys x 2R] = K q^T          A = K as it lies in the cache, B = q
//   O^T [128 dims x 2R] += V^T p^T       A = V^T (keys outermost), B = p
// with  s = (S_hi + S_lo / 32) kscale qscale log2(e),
//       p = 2^(s - m) vscale,  l += 2^(s - m),  out = (O_1 + O_2 / 2^15) / l.
// m is a reference for p, which has to stay within e4m3's range: the maximum of s +
// log2(vscale) so far, raised (and O and l scaled) once a tile's maximum is 2^4 above it.
// So blocks of small values keep their precision beside blocks of large ones.
//
// p in four parts, two for each of O's accumulators: x = 16 p, rounded to f16, is
//   x ~ a + b + (c + d) / 2^15,  a = e4m3(x), b = e4m3(x - a), c = e4m3(y), d = e4m3(y - c),
//   y = 2^15 (x - a - b),
// a and c in one B operand of the MMAs, b and d in a second one that adds to the same two
// accumulators.  Two parts alone (a and e4m3(32 (x - a))) end at 2^-14: where one key has
// most of a row's weight, thousands of others are below that, and what they add up to was lost.
// Four hold every f16 to 2^-9 of itself, so that a weight is off by 2^-8 of it at most down to
// 2^-21 of the largest, and by 2^-29 of that below.
//
// Warps:  0       hands out the ranges of key tiles; TMA loads of K, a ring of tiles of 128 keys
//         1       the MMAs
//         2       TMA loads of V; the scales.  (One warp for both loads issued one of a 16-row
//                 page every 40 cycles.)
//         3       TMEM; the stream form's bookkeeping
//         4 ..    softmax and output: a group of 4 warps for each 16 rows of q (or the 8 of a
//                 kernel of its own).  A thread has one key of the tile, so that a row's
//                 maximum is one reduction over the warp and one exchange between the four.
// What a tile costs is the chain of its softmax, 2600 cycles for 16 rows at first and 1400
// now; a wait alone takes 150 to 250 even for what is there.  So there are three: for the
// scores (whose barrier says also that the scales are there, and, the MMAs being one warp's in
// order, that P's buffer is free again), for the maxima, and for the P V of the tile before
// where O is scaled.  More groups that took the tiles in turns were no faster (spills).
// Two S and two P buffers (one P for 64 rows of D = 256, where K and V leave room for no
// more): the scores of a tile are computed during the softmax of the one before.  Two CTAs
// share an SM where their memory allows it, and hide each other's chains.
// The work is that of the stream form (gdn_attn_stream.cuh).
//
// Bound by HBM where many sequences keep every SM's rings full: 256 single tokens over 1 to
// 16384 keys, 32 + 4 heads of 128, take 339 to 342 us (2.2 GB at 6.6 TB/s, 98 % of the copy rate); 128
// sequences with 1 to 4 drafts over up to 8192 keys, 32 + 8 heads, 16-row pages, 198 to 200 (1.06 GB
// at 5.3 TB/s: TMA loads of 2 KB, and the ranges' ends); one token over 200003 keys 48 (205 MB,
// 33 to 41 of it the main kernel, then the join of 76 ranges).  With 32 and 64 rows for each of the
// 256 single tokens, 128 and 256 query heads, the first call takes 474 and 730 (bound by the chain of
// the softmax and, at 64, the MMAs).  Against two parts of p, four cost 0.5 to 2 % with up to 16 rows,
// 5 and 12 % with 32 and 64.
//
// A row whose result is not finite, or whose l is too small to be trusted (value scales of 2^60 and
// more), is evaluated again key by key (exact_row).  Every wait is bounded.
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
using bf16 = __nv_bfloat16;

constexpr int kMaxRing = 8, kSegs = 4, kMaxGroups = 4;
constexpr float kHeadroom = 4.0f;       // log2: p reaches 2^4 before the reference follows
constexpr float kPScale = 16.0f;        // p 2^4 in the parts' units: at most 256 of 448
constexpr float kLoScale = 32.0f;       // of q's second part
constexpr float kLowScale = 32768.0f;   // 2^15: of p's third and fourth
// A sum l below 2^-60 is not trusted.  m goes down to log2 of the least value scale, 2^-64, below a
// row's scores and, where l may be that small, 60 above them: parts of a row are joined at 2^-124 at
// the least, short of where f32 loses bits.
constexpr float kLeastSum = 8.6e-19f;

struct Shared {
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t q_full, s_full[2], p_full[2], pv[2], o_full, o_empty, end;
  uint64_t meet[kMaxGroups];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Seg seg[kSegs];
  uint32_t tmem;
  int abort;
  int redone;  // rows evaluated again so far, and parts of them
  uint32_t k_loads[kMaxRing], v_loads[kMaxRing];  // issued so far
  int start_s, start_hkv, start_rt, start_u;
  long long left, total;
  long long scan[20];
  uint32_t redo[kMaxGroups][2];                      // rows to evaluate again, by range parity
  float2 scales[2][8];                               // of K and V, for each 16 keys of a tile
  alignas(16) float qscale[kMaxGroups][16];
  alignas(16) int last[kMaxGroups][16];              // a row's last visible key
  alignas(16) float top[kMaxGroups][2][4][16];       // the warps' maxima (sums at the end)
  alignas(16) float own[kMaxGroups][4][2][16];       // a warp's references and factors
};

template <int D, int R>
struct Cfg {
  static constexpr int RG = R < 16 ? R : 16;           // rows of a softmax group
  static constexpr int N = R < 16 ? 32 : 2 * R;        // columns: hi and lo of each row (R = 8:
                                                       // 16 more that nothing looks at)
  static constexpr int kRowBytes = D < 128 ? D : 128;  // of a swizzled row of K, V and q
  static constexpr int NB = D / kRowBytes;             // blocks of them
  static constexpr uint32_t kTile = 128 * D;           // of K, of V
  static constexpr uint32_t kQ = N * D, kHalfP = 128 * N, kP = 2 * kHalfP;
  static constexpr int kCtas = D <= 128 && R <= 16 ? 2 : 1;  // per SM
  static constexpr uint32_t kRoom = kCtas == 2 ? 115712 : 232448;
  // P buffers: two, but for the largest tiles, whose K and V would not be two each any more.
  static constexpr int kPBufs = kRoom - sizeof(Shared) - kQ - 2 * kP >= 4 * kTile ? 2 : 1;
  static constexpr int kFit = (int)((kRoom - sizeof(Shared) - kQ - kPBufs * kP) / (2 * kTile));
  static constexpr int ST = kFit > kMaxRing ? kMaxRing : kFit;
  static constexpr uint32_t kV = ST * kTile, kQAt = 2 * ST * kTile, kPAt = kQAt + kQ, kBars = kPAt + kPBufs * kP;
  static constexpr uint32_t kBytes = kBars + sizeof(Shared);
  static constexpr int kGroups = R / RG;
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int OB = D == 256 ? 2 : 1;          // blocks of 128 dims of O^T
  static constexpr uint32_t kTO = 2 * N;               // TMEM column of O^T
  static constexpr uint32_t kCols = kTO + OB * N <= 128 ? 128 : kTO + OB * N <= 256 ? 256 : 512;
  static_assert(ST >= 2, "tiles in flight");
  static_assert(kBars % 16 == 0 && kBytes <= kRoom, "shared memory");
};

struct Tc8Args {
  int pb;      // rows of a load: a tile's keys, or a divisor of the page
  int ctas;    // the grid
  int rows;    // rows of a workspace block
  int tq;      // tokens of a pair's row tile
  int4* info;  // per CTA, see stream_info
  float* ws;   // the sums
};

// Operand descriptor for rows (or keys) of 32, 64 or 128 swizzled bytes.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, uint32_t lbo, uint32_t sbo, int row_bytes) {
  const uint64_t mode = row_bytes == 128 ? 2u : row_bytes == 64 ? 4u : 6u;
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1u << 46 | mode << 61;
}
// The 16-byte chunk at which chunk c of row r lies.
template <int ROW>
__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t c) {
  return c ^ (ROW == 128 ? r & 7u : ROW == 64 ? (r >> 1) & 3u : (r >> 2) & 1u);
}
// kind::f8f6f4 with e4m3 operands and f32 accumulation, M = 128.
constexpr uint32_t idesc_e4m3(int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// The sum over the warp of each of RG values: lane i is left with that of value i % RG.
// Each step halves the values a lane keeps.
template <int RG>
__device__ __forceinline__ float sum_across(float (&v)[RG], int lane) {
#pragma unroll
  for (int w = RG / 2; w > 0; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
    }
  }
#pragma unroll
  for (int w = RG; w < 32; w <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
  return v[0];
}
// The maximum over the warp, of numbers only.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(y) : "f"(x));
  return y;
}
template <int RG>
__device__ __forceinline__ void read_rows(const float* from, float2 (&x)[RG / 2]) {
#pragma unroll
  for (int i = 0; i < RG / 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(from)[i];
    x[2 * i] = make_float2(v.x, v.y);
    x[2 * i + 1] = make_float2(v.z, v.w);
  }
}
template <int RG>
__device__ __forceinline__ void read_rows(const float* from, float (&x)[RG]) {
#pragma unroll
  for (int i = 0; i < RG / 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(from)[i];
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
// 2 RG columns of a lane: hi, then lo of each row.
template <int RG>
__device__ __forceinline__ void load_parts(uint32_t from, float (&y)[2 * RG]) {
  if constexpr (RG == 16) tmem_ld32(from, y);
  else tmem_ld16(from, y);
  tmem_ld_wait();
}
// The parts of a pair of values.  Between them in f16, whose 11 bits hold the two parts' 8
// (and all of a bf16's): six instructions, where f32 takes nine.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 x = __floats2half2_rn(a, b);
  uint32_t back;
  asm("{\n\t.reg .b16 c;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 c, %2;\n\t"
      "cvt.u32.u16 %0, c;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, c;\n\t}\n"
      : "=r"(hi), "=r"(back)
      : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  const __half2 rest =
      __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(kLoScale));
  asm("{\n\t.reg .b16 c;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 c, %1;\n\t"
      "cvt.u32.u16 %0, c;\n\t}\n"
      : "=r"(lo)
      : "r"(*reinterpret_cast<const uint32_t*>(&rest)));
}
// The four parts of a pair of weights: a and b, and 2^15 times what they leave in c and d.  (What
// is more than 448 becomes that: of weights that a and b hold to 2^-9 already.)
__device__ __forceinline__ void split4(float a, float b, uint32_t (&part)[4]) {
  __half2 x = __floats2half2_rn(a, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i == 2) x = __hmul2(x, __float2half2_rn(kLowScale));
    uint32_t back;
    asm("{\n\t.reg .b16 c;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 c, %2;\n\t"
        "cvt.u32.u16 %0, c;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, c;\n\t}\n"
        : "=r"(part[i]), "=r"(back)
        : "r"(*reinterpret_cast<const uint32_t*>(&x)));
    if (i < 3) x = __hsub2(x, *reinterpret_cast<const __half2*>(&back));
  }
}

#define WAIT(bar, parity) \
  if (!warp_wait(&(bar), (parity), sh, p.status)) return

template <int D, int R>
__global__ void __launch_bounds__(Cfg<D, R>::kThreads, Cfg<D, R>::kCtas)
    attn8_tc_kernel(const __grid_constant__ AttnLaunch p, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ Tc8Args a) {
  using C = Cfg<D, R>;
  constexpr int N = C::N, ST = C::ST, ROW = C::kRowBytes, NB = C::NB, RG = C::RG;
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared* sh = reinterpret_cast<Shared*>(smem + C::kBars);
  const uint32_t sk = smem_u32(smem), sv = sk + C::kV, sq = sk + C::kQAt, sp = sk + C::kPAt;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;

  // (Launched with programmatic dependence: up to the wait, beside the kernel before.)
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < ST; ++i) {
        mbar_init(smem_u32(&sh->k_full[i]), 1);
        mbar_init(smem_u32(&sh->k_empty[i]), 1);
        mbar_init(smem_u32(&sh->v_full[i]), 1);
        mbar_init(smem_u32(&sh->v_empty[i]), 1);
        sh->k_loads[i] = sh->v_loads[i] = 0;
      }
      mbar_init(smem_u32(&sh->q_full), 4 * C::kGroups);
      mbar_init(smem_u32(&sh->o_full), 1);
      mbar_init(smem_u32(&sh->o_empty), 4 * C::kGroups);
      mbar_init(smem_u32(&sh->end), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&sh->s_full[i]), 2);  // the scores, the scales
        mbar_init(smem_u32(&sh->p_full[i]), 4 * C::kGroups);
        mbar_init(smem_u32(&sh->pv[i]), 1);
      }
      for (int i = 0; i < C::kGroups; ++i) {
        mbar_init(smem_u32(&sh->meet[i]), 4);
        sh->redo[i][0] = sh->redo[i][1] = 0;
      }
      for (int i = 0; i < kSegs; ++i) {
        mbar_init(smem_u32(&sh->seg_full[i]), 1);
        mbar_init(smem_u32(&sh->seg_empty[i]), 2 + 4 * C::kGroups);
      }
      sh->abort = sh->redone = 0;
      fence_mbar_init();
    }
  }
  wait_for_previous_kernel();
  // Tensor memory is taken only now: had a CTA of this kernel taken it first, one of the kernel
  // before, beside it on the SM, could wait for it, and this one for that kernel's end.
  if (warp == 3) tmem_alloc(smem_u32(&sh->tmem), C::kCols);
  start_next_kernel();
  stream_start<C::kThreads, true>(p, a.ctas, a.tq, sh);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh->tmem;

  int seg_in = 0;
  auto next_seg = [&](Seg& g) -> bool {
    const int i = seg_in % kSegs;
    if (!warp_wait(&sh->seg_full[i], (seg_in / kSegs) & 1, sh, p.status)) return false;
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
  // The loads of a range's tiles, of K or V.  Pages are looked up four tiles at a time, a
  // batch ahead: lane 8 t + i has that of the i-th group of pb keys of the t-th tile.
  uint32_t loaded = 0;  // tiles before this range
  auto load_range = [&](const Seg& g, uint32_t to, const CUtensorMap* map, uint64_t* full, uint64_t* empty,
                        uint32_t* loads, bool raise, auto batch, auto after) -> bool {
    const int kt0 = uni(g.kt0), kt1 = uni(g.kt1), hi = uni(g.hi), hkv = uni(g.hkv);
    const int per_tile = BK / a.pb;
    auto find_pages = [&](int kt) -> int {
      const int i = lane & 7, jb = (kt + (lane >> 3)) * BK + i * a.pb;
      if (i >= per_tile || kt + (lane >> 3) >= kt1 || jb >= hi) return 0;
      const int64_t pg = page_of(p, g.s, jb / p.page_size);
      if (pg < 0 && raise) atomicOr(p.status, kStatusBadIndex);
      return pg < 0 ? (int)p.num_pages : (int)pg;  // past the end: reads as zeros
    };
    int next_pages = find_pages(kt0);
    for (int kt = kt0; kt < kt1; kt += 4) {
      const int pages = next_pages;
      next_pages = find_pages(kt + 4);
      batch(kt);
      for (int t = 0; t < 4 && kt + t < kt1; ++t, ++loaded) {
        const int j0 = (kt + t) * BK, page = __shfl_sync(0xffffffffu, pages, t * 8 + (lane & 7));
        const int groups = min(per_tile, (hi - j0 + a.pb - 1) / a.pb);
        const int row = (j0 + lane * a.pb) % p.page_size;
        const uint32_t at = loaded % ST, round = loaded / ST;
        if (round > 0)
          if (!warp_wait(&empty[at], (round - 1) & 1, sh, p.status)) return false;
        const uint32_t bar = smem_u32(&full[at]);
        if (elect_one()) {
          ++loads[at];
          mbar_expect_tx(bar, groups * a.pb * (uint32_t)D);
        }
        __syncwarp();
        if (lane < groups)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            tma_load_4d(to + at * C::kTile + b * 128 * ROW + lane * a.pb * ROW, map, bar, b * ROW, row, hkv,
                        page);
        __syncwarp();
        if (!after(t)) return false;
      }
    }
    return true;
  };
  if (warp == 0) {
    // ---- ranges, loads of K ----
    auto role = [&] {
      SegIter<true> iter{sh->start_s, sh->start_hkv, sh->start_rt, sh->start_u, (int)blockIdx.x, a.tq, sh->left};
      for (int n = 0;; ++n) {
        Seg g;
        if (!iter.next(p, g)) g.s = -1;
        const int i = n % kSegs;
        if (n >= kSegs) WAIT(sh->seg_empty[i], (n / kSegs - 1) & 1);
        if (lane == 0) {
          sh->seg[i] = g;
          mbar_arrive(smem_u32(&sh->seg_full[i]));
        }
        __syncwarp();
        if (g.s < 0) return;
        if (!load_range(g, sk, &mk, sh->k_full, sh->k_empty, sh->k_loads, true, [](int) {},
                        [](int) { return true; }))
          return;
      }
    };
    role();
  } else if (warp == 1) {
    // ---- MMAs ----
    auto role = [&] {
      constexpr uint32_t kIdQK = idesc_e4m3(N, false, false), kIdPV = idesc_e4m3(N, true, true);
      Ring kr, vr;
      uint32_t nk = 0;  // tiles whose P V has been issued
      int nseg = 0;
      auto scores = [&](uint32_t n) -> bool {  // of tile n, into S[n & 1]
        if (!warp_wait(&sh->k_full[kr.st], kr.round, sh, p.status)) return false;
        fence_after_sync();
        if (elect_one()) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint64_t kd = desc_of(sk + kr.st * C::kTile + b * 128 * ROW, 16, 8 * ROW, ROW);
            const uint64_t qd = desc_of(sq + b * N * ROW, 16, 8 * ROW, ROW);
#pragma unroll
            for (int k = 0; k < ROW / 32; ++k)
              mma_e4m3(tmem + (n & 1) * N, kd + k * 2, qd + k * 2, kIdQK, b + k > 0);
          }
          mma_commit(smem_u32(&sh->k_empty[kr.st]));
          mma_commit(smem_u32(&sh->s_full[n & 1]));
        }
        kr.step();
        return true;
      };
      Seg g;
      while (next_seg(g)) {
        const int n = uni(g.kt1 - g.kt0);
        WAIT(sh->q_full, nseg & 1);
        fence_after_sync();
        if (!scores(nk)) return;
        for (int j = 0; j < n; ++j, ++nk) {
          if (j + 1 < n)
            if (!scores(nk + 1)) return;
          WAIT(sh->v_full[vr.st], vr.round);
          WAIT(sh->p_full[nk & 1], (nk >> 1) & 1);
          if (j == 0 && nseg > 0) WAIT(sh->o_empty, (nseg - 1) & 1);
          fence_after_sync();
          if (elect_one()) {
            const uint64_t pd = desc_of(sp + (C::kPBufs == 2 ? (nk & 1) * C::kP : 0), 16, 8 * N, N);
#pragma unroll
            for (int b = 0; b < C::OB; ++b) {
              // (D = 64: dims 64 .. 127 of the product are not used; they read the tile's
              // second half.)
              const uint64_t vd = desc_of(sv + vr.st * C::kTile + b * 128 * ROW, 64 * ROW, 8 * ROW, ROW);
#pragma unroll
              for (int k = 0; k < 8; ++k)  // a and c, then b and d, of 32 keys
                mma_e4m3(tmem + C::kTO + b * N, vd + ((k / 2 * 32 * ROW) >> 4),
                         pd + ((k % 2 * C::kHalfP + k / 2 * 32 * N) >> 4), kIdPV, j + k > 0);
            }
            mma_commit(smem_u32(&sh->v_empty[vr.st]));
            mma_commit(smem_u32(&sh->pv[nk & 1]));
            if (j == n - 1) mma_commit(smem_u32(&sh->o_full));
          }
          vr.step();
        }
        ++nseg;
      }
    };
    role();
    __syncwarp();
    if (elect_one()) mma_commit(smem_u32(&sh->end));
    mbar_wait(smem_u32(&sh->end), 0, kWaitBudget);
  } else if (warp == 2) {
    // ---- loads of V, scales ----
    // Lane 8 t + i has the scales of keys 16 i .. 16 i + 15 of the t-th of four tiles.  Loaded
    // by the threads that use them, a tile ahead, they came too late under load and cost each
    // thread their addresses (decode of 256 sequences: 371 for 361 us).
    auto role = [&] {
      Seg g;
      float2 x, next;
      while (next_seg(g)) {
        auto find_scales = [&](int kt) -> float2 {
          const int t = kt + (lane >> 3), j = t * BK + (lane & 7) * 16;
          float2 s = make_float2(0.0f, 0.0f);
          if (t < g.kt1 && j < g.hi) {
            const int pi = j / p.page_size;
            const int64_t pg = page_of(p, g.s, pi);
            if (pg >= 0) {
              const int64_t at = scale_at(p.Hkv, p.page_size, p.block, pg, g.hkv, j - pi * p.page_size);
              s = make_float2(p.ks[at], p.vs[at]);
            }
          }
          return s;
        };
        next = find_scales(g.kt0);
        auto batch = [&](int kt) {
          x = next;
          next = find_scales(kt + 4);
        };
        auto after = [&](int t) -> bool {  // tile `loaded`'s V is on its way
          // The tile two before has used its scales.
          if (loaded >= 2)
            if (!warp_wait(&sh->p_full[loaded & 1], ((loaded >> 1) - 1) & 1, sh, p.status)) return false;
          if ((lane >> 3) == t) sh->scales[loaded & 1][lane & 7] = x;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->s_full[loaded & 1]));
          return true;
        };
        if (!load_range(g, sv, &mv, sh->v_full, sh->v_empty, sh->v_loads, false, batch, after)) return;
      }
    };
    role();
  } else if (warp == 3) {
    if (lane == 0) a.info[blockIdx.x] = stream_info<true>(p, a.ctas, a.tq, sh);
    // Sequences without a key.
    for (int s = blockIdx.x; s < p.N; s += a.ctas) {
      const SeqRange q = seq_range(p, s);
      if (key_tiles(q) > 0) continue;
      const float zero[D / 32] = {};
      for (int t = q.a; t < q.b; ++t)
        for (int h = 0; h < p.Hq; ++h) finish_row<bf16, D>(p, t, h, lane, zero, -INFINITY, 0.0f);
    }
  } else {
    // ---- softmax, output ----
    const int gr = (warp - 4) >> 2, w4 = warp & 3;
    const int r = tid & 127;                       // key of the tile, dim of O, lane of TMEM
    const uint32_t lanes = (uint32_t)w4 << 21;     // (32 * w4) << 16
    const uint32_t ts = tmem + lanes + 2 * RG * gr;
    auto role = [&] {
      uint32_t nk = 0, met = 0;
      int seg_n = 0;
      Ring vr;
      // Meeting the group's other warps (bounded).
      auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->meet[gr]));
        return warp_wait(&sh->meet[gr], met++ & 1, sh, p.status);
      };
      float* own = &sh->own[gr][w4][0][0];
      Seg g;
      while (next_seg(g)) {
        const int rows = g.nt * G;  // of q
        {
          // q of the group's rows.  All its products with the range before are done: their
          // scores have been read.
          constexpr int kPer = 128 / RG, E = D / kPer;  // threads of a row, dims of a thread
          const int i = r / kPer, part = r % kPer, row = gr * RG + i;
          float x[E];
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = 0.0f;
          if (row < rows) {
            const bf16* from = static_cast<const bf16*>(p.q.p) + (int64_t)(g.t0 + row / G) * p.q.ts +
                               (int64_t)(g.hkv * G + row % G) * p.q.hs + part * E;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              const uint2 v = *reinterpret_cast<const uint2*>(from + e);
              x[e] = __uint_as_float(v.x << 16);
              x[e + 1] = __uint_as_float(v.x & 0xffff0000u);
              x[e + 2] = __uint_as_float(v.y << 16);
              x[e + 3] = __uint_as_float(v.y & 0xffff0000u);
            }
          }
          float big = 0.0f;
#pragma unroll
          for (int e = 0; e < E; ++e) big = fmaxf(big, fabsf(x[e]));
#pragma unroll
          for (int o = kPer / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          // 2^e that brings the largest into [128, 256).
          const int ex = max(-126, min(126, 134 - (int)(__float_as_uint(big) >> 23)));
          const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
          if (part == 0) {
            sh->qscale[gr][i] = p.scale * kLog2e * __uint_as_float((uint32_t)(127 - ex) << 23);
            sh->last[gr][i] = row < rows ? g.pos0 + row / G : -1;
          }
          uint32_t hi[E / 4], lo[E / 4];
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            uint32_t h0, l0, h1, l1;
            // (x - x: what is not finite becomes NaN)
            split2(fmaf(x[e], up, x[e] - x[e]), fmaf(x[e + 1], up, x[e + 1] - x[e + 1]), h0, l0);
            split2(fmaf(x[e + 2], up, x[e + 2] - x[e + 2]), fmaf(x[e + 3], up, x[e + 3] - x[e + 3]), h1, l1);
            hi[e / 4] = h0 | h1 << 16;
            lo[e / 4] = l0 | l1 << 16;
          }
          auto put = [&](uint32_t n, const uint32_t(&c)[E / 4]) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              const int d = part * E + e, b = d / ROW, in = d % ROW;
              *reinterpret_cast<uint32_t*>(smem + C::kQAt + b * N * ROW + n * ROW + swz<ROW>(n, in >> 4) * 16 +
                                           (in & 15)) = c[e / 4];
            }
          };
          put(2 * RG * gr + i, hi);
          put(2 * RG * gr + RG + i, lo);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->q_full));
        }
        if (!meet()) return;  // qscale, last
        float2 l[RG / 2];     // of this thread's keys
        float m = -INFINITY;  // of row lane % RG
#pragma unroll
        for (int i = 0; i < RG / 2; ++i) l[i] = make_float2(0.0f, 0.0f);
        for (int kt = g.kt0; kt < g.kt1; ++kt, ++nk, vr.step()) {
          const uint32_t buf = nk & 1;
          const int j = kt * BK + r;
          const bool masked = kt * BK + BK - 1 > g.pos0;
          float2 s[RG / 2];  // of rows 2 i, 2 i + 1: f32 instructions take pairs
          float vsc, lv;
          {
            float2 qs[RG / 2];
            read_rows<RG>(sh->qscale[gr], qs);
            WAIT(sh->s_full[buf], (nk >> 1) & 1);
            fence_after_sync();
            const float2 scale = sh->scales[buf][r >> 4];
            vsc = scale.y;
            // (a scale of nothing, 0, has no logarithm: 2^-64 stands for smaller ones)
            lv = fmaxf(__log2f(fabsf(vsc)), -64.0f);
            float y[2 * RG];
            load_parts<RG>(ts + buf * N, y);
            const float2 ksc = make_float2(scale.x, scale.x);
            const float2 part = make_float2(1.0f / kLoScale, 1.0f / kLoScale);
#pragma unroll
            for (int i = 0; i < RG / 2; ++i)
              s[i] = __fmul2_rn(__ffma2_rn(make_float2(y[RG + 2 * i], y[RG + 2 * i + 1]), part,
                                           make_float2(y[2 * i], y[2 * i + 1])),
                                __fmul2_rn(ksc, qs[i]));
          }
          if (masked) {
            const int4* last = reinterpret_cast<const int4*>(sh->last[gr]);
#pragma unroll
            for (int i = 0; i < RG / 4; ++i) {
              const int4 v = last[i];
              s[2 * i].x = j <= v.x ? s[2 * i].x : -INFINITY;
              s[2 * i].y = j <= v.y ? s[2 * i].y : -INFINITY;
              s[2 * i + 1].x = j <= v.z ? s[2 * i + 1].x : -INFINITY;
              s[2 * i + 1].y = j <= v.w ? s[2 * i + 1].y : -INFINITY;
            }
          }
          {
            const float2 lv2 = make_float2(lv, lv);
            float t[RG];
#pragma unroll
            for (int i = 0; i < RG / 2; ++i) {
              const float2 x = __fadd2_rn(s[i], lv2);
              t[2 * i] = warp_max(x.x);
              t[2 * i + 1] = warp_max(x.y);
            }
            if (lane == 0) {
#pragma unroll
              for (int i = 0; i < RG / 4; ++i)
                reinterpret_cast<float4*>(sh->top[gr][buf][w4])[i] =
                    make_float4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
            }
          }
          if (!meet()) return;
          bool raise = false;
          {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) top = fmaxf(top, sh->top[gr][buf][w][lane & (RG - 1)]);
            float f = 1.0f;
            if (top > m + kHeadroom) {  // the same in the group's warps
              raise = true;
              f = ex2(m - top);
              m = top;
            }
            if (lane < RG) {
              own[lane] = m == -INFINITY ? 0.0f : -m;
              own[16 + lane] = f;
            }
            __syncwarp();
          }
          if (__any_sync(0xffffffffu, raise)) {
            float2 f[RG / 2];
            read_rows<RG>(own + 16, f);
#pragma unroll
            for (int i = 0; i < RG / 2; ++i) l[i] = __fmul2_rn(l[i], f[i]);
            if (kt > g.kt0) {
              WAIT(sh->pv[buf ^ 1], ((nk - 1) >> 1) & 1);
              fence_after_sync();
#pragma unroll 1
              for (int b = 0; b < (RG == 16 ? 2 : 1) * C::OB; ++b) {  // 16 columns at a time
                const uint32_t at = ts + C::kTO + (RG == 16 ? (b >> 1) * N + (b & 1) * 16 : b * N);
                float o[16];
                tmem_ld16(at, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= i % 2 ? f[i % RG / 2].y : f[i % RG / 2].x;
                tmem_st16(at, o);
              }
              tmem_st_wait();
            }
          }
          {
            float2 ref[RG / 2];
            read_rows<RG>(own, ref);
            const float2 vs = make_float2(vsc * kPScale, vsc * kPScale);
            uint32_t parts[4][RG / 4];
#pragma unroll
            for (int i = 0; i < RG / 4; ++i) {
              uint32_t of[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = 2 * i + e;
                float2 w = __fadd2_rn(s[k], ref[k]);  // (minus the reference)
                w.x = ex2(w.x);
                w.y = ex2(w.y);
                l[k] = __fadd2_rn(l[k], w);
                w = __fmul2_rn(w, vs);
                split4(w.x, w.y, of[e]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) parts[k][i] = of[0][k] | of[1][k] << 16;
            }
            // (P[buf] has been read: the scores' MMAs followed that product.  One buffer is read
            // by the product of the tile before.)
            if constexpr (C::kPBufs == 1)
              if (kt > g.kt0) WAIT(sh->pv[buf ^ 1], ((nk - 1) >> 1) & 1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const auto &first = parts[k], &second = parts[k + 2];
              unsigned char* to = smem + C::kPAt + (C::kPBufs == 2 ? buf * C::kP : 0) + k * C::kHalfP + r * N;
              if constexpr (RG == 16) {
                *reinterpret_cast<uint4*>(to + swz<N>(r, 2 * gr) * 16) = make_uint4(first[0], first[1], first[2], first[3]);
                *reinterpret_cast<uint4*>(to + swz<N>(r, 2 * gr + 1) * 16) = make_uint4(second[0], second[1], second[2], second[3]);
              } else {
                *reinterpret_cast<uint4*>(to + swz<N>(r, 0) * 16) = make_uint4(first[0], first[1], second[0], second[1]);
              }
            }
          }
          if (gr == 0 && (kt + 1) * BK > g.hi) {
            // Rows of V past the context's end: a stale NaN there would survive a weight of 0.
            WAIT(sh->v_full[vr.st], vr.round);
            if (j >= g.hi) {
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                uint4* to = reinterpret_cast<uint4*>(smem + C::kV + vr.st * C::kTile + b * 128 * ROW + r * ROW);
#pragma unroll
                for (int e = 0; e < ROW / 16; ++e) to[e] = make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
          fence_proxy_async();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[buf]));
        }
        // ---- the rows' sums out ----
        float ls[RG];
#pragma unroll
        for (int i = 0; i < RG / 2; ++i) {
          ls[2 * i] = l[i].x;
          ls[2 * i + 1] = l[i].y;
        }
        const float part_l = sum_across<RG>(ls, lane);
        if (lane < RG) sh->top[gr][nk & 1][w4][lane] = part_l;
        if (!meet()) return;
        if (r == 0) sh->redo[gr][(seg_n & 1) ^ 1] = 0;  // (the last range's has been read)
        float L = 0.0f;  // of row lane % RG, the same in every warp
#pragma unroll
        for (int w = 0; w < 4; ++w) L += sh->top[gr][nk & 1][w][lane & (RG - 1)];
        const int live = min(RG, rows - gr * RG);  // rows of this group
        if (lane < RG) own[lane] = g.slot >= 0 ? 1.0f / kPScale : L == 0.0f ? 0.0f : 1.0f / (L * kPScale);
        __syncwarp();
        const bool fine = (L - L == 0.0f && L >= kLeastSum) || (m == -INFINITY && L == 0.0f);
        uint32_t bad = __ballot_sync(0xffffffffu, !fine) & ((1u << RG) - 1u);
        const Partials part(a.ws, 2 * (int64_t)a.ctas, a.rows, D);
        WAIT(sh->o_full, seg_n & 1);
        fence_after_sync();
#pragma unroll 1
        for (int b = 0; b < C::OB; ++b) {
          float o[RG];
          {
            float y[2 * RG];
            load_parts<RG>(ts + C::kTO + b * N, y);
            float f[RG];
            read_rows<RG>(own, f);
#pragma unroll
            for (int i = 0; i < RG; ++i) o[i] = fmaf(y[RG + i], 1.0f / kLowScale, y[i]) * f[i];
          }
          const int dim = b * 128 + r;
          if (D >= 128 || r < D) {
            if (g.slot >= 0) {
              float* to = part.o + (g.slot * a.rows + gr * RG) * D + dim;
#pragma unroll
              for (int i = 0; i < RG; ++i) {
                if (i >= live) continue;
                if (!(o[i] - o[i] == 0.0f)) bad |= 1u << i;
                to[i * D] = o[i];
              }
            } else {
              // Row after row: the next head, or the next token's first of the group.
              int h = gr * RG % G;
              const int t = g.t0 + gr * RG / G;
              bf16* to = static_cast<bf16*>(p.out) + ((int64_t)t * p.Hq + g.hkv * G + h) * D + dim;
              const bf16* gate = static_cast<const bf16*>(p.gate.p) + (int64_t)t * p.gate.ts +
                                 (int64_t)(g.hkv * G + h) * p.gate.hs + dim;
              const int64_t out_wrap = (int64_t)(p.Hq - G) * D, gate_wrap = p.gate.ts - G * p.gate.hs;
#pragma unroll
              for (int i = 0; i < RG; ++i) {
                if (i >= live) continue;
                if (!(o[i] - o[i] == 0.0f)) bad |= 1u << i;
                float x = o[i];
                if (p.gate.p != nullptr) x *= sigmoid_gate(to_f(*gate));
                *to = __float2bfloat16_rn(x);
                to += D;
                gate += p.gate.hs;
                if (++h == G) {
                  h = 0;
                  to += out_wrap;
                  gate += gate_wrap;
                }
              }
            }
          }
        }
        fence_before_sync();
        if (w4 == 0 && lane < live) {
          const int row = gr * RG + lane;
          if (g.slot >= 0)
            part.ml[g.slot * a.rows + row] = make_float2(L == 0.0f ? -INFINITY : m, L);
          else if (p.lse != nullptr)
            p.lse[(int64_t)(g.t0 + row / G) * p.Hq + g.hkv * G + row % G] =
                L == 0.0f ? -INFINITY : (m + log2f(L)) * kLn2;
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (live < RG) bad &= live > 0 ? (1u << live) - 1u : 0u;
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh->o_empty));
          if (bad) atomicOr(&sh->redo[gr][seg_n & 1], bad);
        }
        if (!meet()) return;
        uint32_t redo = *(volatile uint32_t*)&sh->redo[gr][seg_n & 1] & (0x1111u << w4);
        while (redo) {
          const int i = __ffs(redo) - 1, row = gr * RG + i;
          redo &= redo - 1;
          const int t = g.t0 + row / G, h = g.hkv * G + row % G;
          float acc[D / 32], em, el;
          exact_row<bf16, D, E4>(p, g.s, cu_at(p.cu, g.s), t, h, g.kt0 * BK,
                                 min(g.kt1 * BK, g.pos0 + row / G + 1), acc, em, el, &sh->redone);
          if (g.slot >= 0) part.put<D / 32>(g.slot, row, lane, acc, em, el);
          else finish_row<bf16, D>(p, t, h, lane, acc, em, el);
          if (lane == 0) atomicAdd(&sh->redone, 1);
        }
        ++seg_n;
      }
    };
    role();
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (sh->abort) {
    // A wait gave up: copies may still be in flight (otherwise the MMA role has waited for
    // each).  They land before the CTA's memory is given up.
    if (tid == 0)
      for (int i = 0; i < ST; ++i) {
        if (sh->k_loads[i]) mbar_wait(smem_u32(&sh->k_full[i]), (sh->k_loads[i] - 1) & 1, kWaitBudget);
        if (sh->v_loads[i]) mbar_wait(smem_u32(&sh->v_full[i]), (sh->v_loads[i] - 1) & 1, kWaitBudget);
      }
    __syncthreads();
  }
  if (warp == 3) tmem_dealloc(tmem, C::kCols);
}

template <int D>
__global__ void __launch_bounds__(256) attn8_join_kernel(const __grid_constant__ AttnLaunch p,
                                                         const __grid_constant__ Tc8Args a) {
  stream_join<bf16, D, true>(p, a);
}

// ---- host ------------------------------------------------------------------------

template <int D, int R>
bool codes_map(CUtensorMap* m, const AttnPages& c, const AttnLaunch& p, int pb) {
  auto enc = chunk::encode_fn();
  if (enc == nullptr) return false;
  constexpr int ROW = Cfg<D, R>::kRowBytes;
  const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv,
                              (cuuint64_t)p.num_pages};
  const cuuint64_t st[3] = {(cuuint64_t)c.ts, (cuuint64_t)c.hs, (cuuint64_t)c.ps};
  const cuuint32_t box[4] = {ROW, (cuuint32_t)pb, 1, 1}, es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.p, dims, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             ROW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMostRows = 256;
constexpr int row_class(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int D, int R>
cudaError_t run(const AttnLaunch& p, cudaStream_t st) {
  using C = Cfg<D, R>;
  Tc8Args a{};
  a.pb = BK;
  while (p.page_size % a.pb != 0) a.pb >>= 1;
  a.ctas = C::kCtas * chunk::sm_count();
  const int G = p.Hq / p.Hkv;
  a.tq = std::min(p.max_q, R / G);  // (G <= R)
  a.rows = a.tq * G;
  a.info = static_cast<int4*>(p.ws);
  a.ws = reinterpret_cast<float*>(static_cast<char*>(p.ws) + info_bytes(a.ctas));
  CUtensorMap mk, mv;
  if (!codes_map<D, R>(&mk, p.kc, p, a.pb) || !codes_map<D, R>(&mv, p.vc, p, a.pb))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> devices{0};
  cudaError_t e = allow_shared(attn8_tc_kernel<D, R>, C::kBytes, devices);
  if (e != cudaSuccess) return e;
  e = launch_after(attn8_tc_kernel<D, R>, dim3(a.ctas), C::kThreads, st, C::kBytes, p, mk, mv, a);
  if (e != cudaSuccess) return e;
  return launch_after(attn8_join_kernel<D>, dim3(a.ctas, std::min(a.rows, 16)), 256, st, 0, p, a);
}

template <int D>
cudaError_t by_rows(const AttnLaunch& p, cudaStream_t st) {
  switch (row_class((int64_t)p.max_q * (p.Hq / p.Hkv))) {
    case 8: return run<D, 8>(p, st);
    case 16: return run<D, 16>(p, st);
    case 32: return run<D, 32>(p, st);
    default: return run<D, 64>(p, st);
  }
}

template <int D>
int ctas_per_sm(int64_t rows) {
  return row_class(rows) <= 16 ? Cfg<D, 16>::kCtas : 1;
}

}  // namespace

// More than 64 rows read their keys again for every 64.  Against widening first (4 kv heads; 128
// sequences of 4096 keys, one of 32768), us:
//   rows       64              128             192             256
//   D = 64     188/374 32/45   354/397 40/56   520/422 52/44   688/429 61/54
//   D = 128    191/541 32/55   357/570 42/68   524/547 53/55   693/556 63/68
//   D = 256    249/1025 46/96  465/1127 54/117 682/1136 69/96  909/1157 81/109
// Widening also takes a workspace as large as the contexts, so it begins where it gains in
// every shape of D = 128 and more.
bool attn8_tc_supported(int64_t rows, int64_t D, bool bf16) { return bf16 && D >= 64 && rows <= kMostRows; }

size_t attn8_tc_workspace_bytes(int64_t rows, int64_t D) {
  const int per = D == 64 ? ctas_per_sm<64>(rows) : D == 128 ? ctas_per_sm<128>(rows) : ctas_per_sm<256>(rows);
  const int ctas = per * chunk::sm_count();
  return info_bytes(ctas) + Partials::bytes(2 * (int64_t)ctas, (int)std::min<int64_t>(rows, 64), D);
}

cudaError_t launch_attn8_tc(const AttnLaunch& p, cudaStream_t st) {
  switch (p.D) {
    case 64: return by_rows<64>(p, st);
    case 128: return by_rows<128>(p, st);
    default: return by_rows<256>(p, st);
  }
}

}  // namespace gdn
