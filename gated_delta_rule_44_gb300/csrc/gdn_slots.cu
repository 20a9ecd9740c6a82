// gdn_slots.cu -- slots of any pools (recurrence states, conv tails, cache pages and their
// scales, block tables) copied by lists, or reordered within groups in place:
//   pool[dst[i]] = pool[src[i]]                          (lists)
//   pool[dst[g, i]] = old pool[dst[g, src[g, i]]]        (groups: src are places in the group)
//
// An item is a piece of a pool's slots, [offset, offset + bytes) of each, for some whole
// groups (a list's pairs are groups of one).  Its CTA brings the pieces that move into
// shared memory with bulk copies, waits for all of them, and only then sends them to their
// destinations.  As every CTA handles the same bytes of all the slots of its groups, a
// group is reordered in place whatever its cycles, without a second pool.  A source of
// several places is read once for every 32 pairs of an item (a warp's) that it is in; a slot that
// stays where it is is not touched.
//
// Bound by HBM: each moved byte is read and written once.  The copies need no registers and
// one thread per slot, so the number of bytes in flight is the shared memory's: 40 KB for
// each of five CTAs per SM.  16 groups of four beams' states and conv tails of three layers
// (541 MB moved) take 79 to 85 us, 6.4 to 6.8 TB/s; 1001 pages of two layers (214 MB) 36, of which
// 31.6 are the bytes.  The lists are checked by CTAs of their own beside the copies.
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn_common.cuh"
#include "gdn_internal.h"
#include "tcgen05.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kThreads = 128;
constexpr uint32_t kStage = 40960;
constexpr long long kWaitBudget = 2000000000LL;  // ~1 s of SM clock

__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint32_t mbar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(to),
               "l"(from), "r"(bytes), "r"(mbar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* to, uint32_t from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(to), "r"(from), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_stores_done() {
  asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group 0;\n" ::: "memory");
}

// Pair i's slots in a pool of `slots`; false: it moves nothing.
__device__ __forceinline__ bool pair_of(const SlotsLaunch& p, int64_t i, int64_t slots, int& from, int& to,
                                        bool& bad) {
  to = p.dst[i];
  from = p.src[i];
  if (to < 0 || from < 0) return false;
  if (p.W > 0) {
    if (from >= p.W) {
      bad = true;
      return false;
    }
    from = p.dst[i / p.W * p.W + from];
    if (from < 0) return false;
  }
  if (to >= slots || from >= slots) {
    bad = true;
    return false;
  }
  return from != to;
}

// Looks for a slot that is a destination twice, or, of lists, both a destination and
// another pair's source: of the slots from w0 on that the stage has bits for.  Every such
// window reads the whole lists, eight pairs of a thread at a time.
constexpr int kBits = kStage * 8;
__device__ void check_lists(const SlotsLaunch& p, int64_t w0, uint32_t* seen) {
  constexpr int kAhead = 8;
  bool bad = false;
  for (int i = threadIdx.x; i < kBits / 32; i += kThreads) seen[i] = 0;
  __syncthreads();
  for (int pass = 0; pass < (p.W > 0 ? 1 : 2); ++pass) {
    for (int64_t i0 = threadIdx.x; i0 < p.n; i0 += kThreads * kAhead) {
      int d[kAhead], s[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t i = i0 + u * kThreads;
        d[u] = i < p.n ? p.dst[i] : -1;
        s[u] = i < p.n && p.W == 0 ? p.src[i] : 0;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t at = (int64_t)(pass == 0 ? d[u] : s[u]) - w0;
        if (d[u] < 0 || s[u] < 0 || at < 0 || at >= kBits) continue;
        const uint32_t bit = 1u << (at & 31);
        if (pass == 0) bad |= (atomicOr(&seen[at >> 5], bit) & bit) != 0;
        else bad |= s[u] != d[u] && (seen[at >> 5] & bit) != 0;
      }
    }
    __syncthreads();
  }
  if (bad) atomicOr(p.status, kStatusBadIndex);
}

__global__ void __launch_bounds__(kThreads) slots_kernel(const __grid_constant__ SlotsLaunch p) {
  extern __shared__ __align__(128) unsigned char stage[];
  __shared__ uint64_t landed;
  attn::start_next_kernel();
  attn::wait_for_previous_kernel();
  const int tid = threadIdx.x, lane = tid & 31;
  // The pool whose items hold this number.
  int64_t item = blockIdx.x;
  int pool = 0;
  while (pool < p.pools && item >= p.pool[pool].items) item -= p.pool[pool++].items;
  if (pool == p.pools) {
    check_lists(p, item * kBits, reinterpret_cast<uint32_t*>(stage));
    return;
  }
  const SlotPool& q = p.pool[pool];
  const int64_t first = item / q.pieces * q.pairs;  // pair
  const int pairs = (int)min((int64_t)q.pairs, p.n - first);
  const int64_t offset = item % q.pieces * q.piece;
  const uint32_t bytes = (uint32_t)min((int64_t)q.piece, q.bytes - offset);
  unsigned char* base = static_cast<unsigned char*>(q.data) + offset;
  bool bad = false;
  if (q.words) {  // not in 16-byte units: by plain loads of 4 bytes
    uint32_t* words = reinterpret_cast<uint32_t*>(stage);
    const int n = (int)(bytes / 4), step = (int)(q.piece / 4);
    for (int i = 0; i < pairs; ++i) {
      int from, to;
      if (!pair_of(p, first + i, q.slots, from, to, bad)) continue;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(base + (int64_t)from * q.stride);
      for (int e = tid; e < n; e += kThreads) words[i * step + e] = src[e];
    }
    __syncthreads();
    for (int i = 0; i < pairs; ++i) {
      int from, to;
      if (!pair_of(p, first + i, q.slots, from, to, bad)) continue;
      uint32_t* dst = reinterpret_cast<uint32_t*>(base + (int64_t)to * q.stride);
      for (int e = tid; e < n; e += kThreads) dst[e] = words[i * step + e];
    }
    if (bad && tid == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  if (tid == 0) {
    mbar_init(smem_u32(&landed), kThreads / 32);
    fence_mbar_init();
  }
  __syncthreads();
  int from = -1, to = -1;
  const bool moves = tid < pairs && pair_of(p, first + tid, q.slots, from, to, bad);
  if (bad) atomicOr(p.status, kStatusBadIndex);
  // The first lane of a warp's with a source reads it for the others.
  const unsigned same = __match_any_sync(0xffffffffu, moves ? from : -1 - lane);
  const int reader = __ffs(same) - 1;
  const bool reads = moves && reader == lane;
  const uint32_t mb = smem_u32(&landed), at = smem_u32(stage) + (tid - lane + reader) * (uint32_t)q.piece;
  const unsigned readers = __ballot_sync(0xffffffffu, reads);
  if (lane == 0) mbar_expect_tx(mb, __popc(readers) * bytes);
  __syncwarp();
  if (reads) bulk_load(at, base + (int64_t)from * q.stride, bytes, mb);
  bool ok = mbar_wait(mb, 0, kWaitBudget);
  if (!ok) {  // give the copies in flight one more limit to land before the memory is given up
    atomicOr(p.status, kStatusTimeout);
    ok = false;
    mbar_wait(mb, 0, kWaitBudget);
  }
  if (ok && moves) bulk_store(base + (int64_t)to * q.stride, at, bytes);
  bulk_stores_done();
}

}  // namespace

cudaError_t launch_slots(SlotsLaunch& p, cudaStream_t st) {
  const int64_t W = std::max(p.W, 1);
  int64_t items = 0;
  for (int i = 0; i < p.pools; ++i) {
    SlotPool& q = p.pool[i];
    const int64_t unit = q.words ? 4 : 16;
    // Whole groups per item, a thread for each pair; the stage holds a piece of each.
    const int64_t fit = std::max<int64_t>(1, (int64_t)kStage / (W * q.bytes));
    const int64_t groups = std::max<int64_t>(1, std::min<int64_t>({kThreads / W, fit, p.n / W}));
    q.pairs = (int)(groups * W);
    q.piece = std::min<int64_t>(q.bytes, (int64_t)kStage / q.pairs / unit * unit);
    q.pieces = (q.bytes + q.piece - 1) / q.piece;
    q.items = (p.n + q.pairs - 1) / q.pairs * q.pieces;
    items += q.items;
  }
  items += (p.most_slots + kBits - 1) / kBits;  // the check's windows, a CTA each
  if (items > INT32_MAX) return cudaErrorInvalidConfiguration;
  return attn::launch_after(slots_kernel, dim3((unsigned)items), kThreads, st, kStage, p);
}

}  // namespace gdn
