// gdn_internal.h -- launch descriptors shared by the host API (gdn_api.cpp)
// and the kernel translation units.  Everything here is already validated:
// the launchers only choose a configuration and launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

// Bits of the per-device status word (see gdn_status.cu).
enum : unsigned {
  kStatusBadIndex = 1u,     // state index outside [-1, slots)
  kStatusBadSeqlens = 2u,   // cu_seqlens not 0..T, empty or decreasing range
  kStatusTimeout = 4u,      // a bounded device wait gave up
};

// Counts one kernel launch (gdn_launch_count()).
void note_launch();

// Device address of the current device's status word (cached per device);
// nullptr if the symbol could not be resolved.
unsigned* status_word();

// Records `msg` as the calling thread's gdn_last_error_message() and returns
// `code` (for sources outside the API translation unit).
int report_error(int code, const char* msg);

struct PrepareLaunch {
  int T, N, Hk, Hv, Dk, Dv, K;
  bool bf16, norm;
  const void* x;
  int64_t x_stride;  // elements
  const float* w;
  const void* a;
  int64_t a_stride;
  const void* b;
  int64_t b_stride;
  const float* A_log;
  const float* dt_bias;
  const int32_t* cu;
  const int32_t* sidx;      // may be null
  const uint8_t* has_init;  // may be null
  float* conv_pool;
  int64_t slots;
  int state_len;                // speculative prepare: conv row length per channel
  const int32_t* num_accepted;  // speculative prepare: [N]
  void* q;
  void* k;
  void* v;
  float* g;
  float* beta;
  unsigned* status;
};
cudaError_t launch_prepare(const PrepareLaunch& p, cudaStream_t s);
// The prepare of a speculative step: sequence s's conv row (slot sidx[s],
// state_len entries per channel) is read at offset num_accepted[s] - 1 and
// shifted by one tap; has_init is ignored.
cudaError_t launch_spec_prepare(const PrepareLaunch& p, cudaStream_t s);

// One token per row (decode) or token-sequential over sequences (recurrent
// prefill) -- the same register-resident row update.
struct RecurLaunch {
  int T, N, Hk, Hv, Dk, Dv;
  bool bf16, norm;
  float scale;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  float* pool;
  int64_t slots;
  const int32_t* cu;        // null for decode (row b = sequence b)
  const int32_t* sidx;      // may be null; [N, num_cols] for the speculative decode
  const uint8_t* has_init;  // may be null (prefill only)
  const int32_t* num_accepted;  // speculative decode only: [N]
  int num_cols;                 // speculative decode only
  void* out;
  unsigned* status;
  // Gated RMSNorm of the output rows (on when onorm_w != nullptr): out =
  // core / sqrt(mean(core^2) + eps) * w * act(z), core rounded to the
  // activation type first.
  const void* onorm_z;
  int64_t onorm_z_stride;  // elements between token rows of z
  const void* onorm_w;
  float onorm_eps;
  bool onorm_sigmoid;
  bool onorm_in_kernel;  // decode: inside the recurrence kernel where it fits
};
cudaError_t launch_decode(const RecurLaunch& p, cudaStream_t s);
cudaError_t launch_recurrent(const RecurLaunch& p, cudaStream_t s);
// KDA: the recurrent prefill with g [T, Hv, Dk], a log decay per key channel
// (p.norm must be false).
cudaError_t launch_kda(const RecurLaunch& p, cudaStream_t s);
// Speculative multi-token decode: sequence s's initial slot is
// sidx[s * num_cols + num_accepted[s] - 1] and the state after its token j is
// stored into sidx[s * num_cols + j] (negative: skipped); p.norm false.
cudaError_t launch_spec_decode(const RecurLaunch& p, cudaStream_t s);
bool recurrent_supported(int Dk);
// Whether gdn_decode applies the output norm inside the recurrence kernel
// (the row's value-dimension slices, 64 rows each at Dk = 128, fit one CTA
// of at most 4 x 128 threads).
bool decode_norm_in_kernel(int Dk, int Dv);

// Decode in one launch from the packed projections: conv update, SiLU, q/k
// norm, gates and the recurrence (one token per row b; the conv pool and the
// state pool share the slot sidx[b]).
struct PackedDecodeLaunch {
  int B, Hk, Hv, Dk, Dv, K;
  bool bf16, norm;
  float scale;
  const void* x;  // raw (pre-conv) rows: q, k, v channels first
  int64_t x_stride;
  const float* w;
  const void* a;
  int64_t a_stride;
  const void* b;
  int64_t b_stride;
  const float* A_log;
  const float* dt_bias;
  const int32_t* sidx;
  float* conv_pool;  // [slots, C_conv, K-1]
  float* pool;       // [slots, Hv, Dv, Dk]
  int64_t slots;
  void* out;
  unsigned* status;
};
bool packed_decode_supported(int Dk, int Dv, int K);
cudaError_t launch_packed_decode(const PackedDecodeLaunch& p, cudaStream_t s);

// Chunked (C = 64) tensor-core prefill.
struct ChunkedLaunch {
  RecurLaunch r;
  void* workspace;
  size_t workspace_bytes;
};
bool chunked_supported(int Dk, int Dv, bool bf16);

// The chunked form of the KDA recurrence (g [T, Hv, Dk]; p.norm false): two
// launches over a caller workspace of kda_chunked_workspace_bytes().
bool kda_chunked_supported(int Dk, int Dv, bool bf16);
size_t kda_chunked_workspace_bytes(int64_t T, int64_t N, int64_t Hv, int64_t Dk, int64_t Dv);
cudaError_t launch_kda_chunked(const ChunkedLaunch& c, cudaStream_t s);

// The same chunked form in one launch of one CTA per (sequence, value head);
// with a workspace of fused_workspace_bytes() and more chains than SMs, one
// CTA per SM over a wrap-around schedule of the chains' chunks (a small
// schedule launch first).
bool fused_supported(int Dk, int Dv, bool bf16);
size_t fused_workspace_bytes(int64_t N, int64_t Hv);
cudaError_t launch_fused(const RecurLaunch& p, void* workspace, size_t workspace_bytes,
                         cudaStream_t s);

// Gated RMSNorm of the recurrence output.
struct NormLaunch {
  int64_t rows;   // tokens * heads
  int heads, dim;
  bool bf16, sigmoid_gate;
  float eps;
  const void* core;
  const void* z;
  int64_t z_stride;  // elements between token rows of z
  const void* weight;
  void* out;
};
cudaError_t launch_gated_rmsnorm(const NormLaunch& p, cudaStream_t s);
size_t chunked_workspace_bytes(int64_t T, int64_t N, int64_t Hv, int64_t Dk, int64_t Dv);
cudaError_t launch_chunked(const ChunkedLaunch& p, cudaStream_t s);

// ---- full (softmax) attention layer ------------------------------------------

// One strided [tokens, heads, D] tensor (D contiguous; strides in elements).
struct AttnRows {
  const void* p;
  int64_t ts, hs;  // token, head stride
};

// One paged cache tensor [pages, heads, page_size, D] by strides (elements).
struct AttnPages {
  void* p;
  int64_t ps, hs, ts;  // page, head, token stride
};

struct AttnPrepareLaunch {
  int T, N, Hq, Hkv, D, rot;
  bool bf16;
  float eps;
  AttnRows q, k, v;
  const void* q_w;  // null: no norm
  const void* k_w;
  const float* cos_sin;  // [max_pos, rot]; null when rot == 0
  int64_t max_pos;
  const int32_t* positions;  // null: the token's place in its sequence
  const int32_t* cu;         // null: one token per sequence
  const int32_t* kv_lens;    // null: the number of new tokens
  const int32_t* table;      // null: no cache
  int64_t table_stride;
  int max_pages, page_size;
  int64_t num_pages;
  AttnPages kc, vc;
  void* q_out;  // [T, Hq, D]
  void* k_out;  // [T, Hkv, D] or null
  unsigned* status;
  // A cache in 8 bits: the scales of its blocks of `block` rows (see AttnLaunch).
  float* ks;
  float* vs;
  int block;
};
cudaError_t launch_attn_prepare(const AttnPrepareLaunch& p, cudaStream_t s);
cudaError_t launch_attn8_prepare(const AttnPrepareLaunch& p, cudaStream_t s);

// Causal attention of packed new tokens over packed keys (table == null: k, v
// are [T, Hkv, D] rows) or over a paged cache.
struct AttnLaunch {
  int T, N, Hq, Hkv, D, max_q;
  bool bf16;
  float scale;
  AttnRows q;
  AttnRows k, v;         // packed form
  const int32_t* cu;     // null: one token per sequence
  const int32_t* kv_lens;  // paged form
  const int32_t* table;
  int64_t table_stride;
  int max_pages, page_size;
  int64_t num_pages;
  AttnPages kc, vc;
  AttnRows gate;  // p null: none
  void* out;      // [T, Hq, D]
  float* lse;     // [T, Hq] or null
  void* ws;
  unsigned* status;
  bool part;      // the N sequences are some of a call's: their tokens need not span all T
  // A cache in 8 bits (kc, vc: e4m3 codes, strides in bytes): the scales of its blocks of
  // `block` rows, [num_pages, Hkv, page_size / block]; null otherwise.
  const float* ks;
  const float* vs;
  int block;
};
// CUDA-core form: any supported size (D in {32, 64, 128, 256}, Hq / Hkv <= 64).
cudaError_t launch_attn_simt(const AttnLaunch& p, cudaStream_t s);
// Joins the sums of `splits` key ranges per tile of TT tokens, left in p.ws in
// blocks of bm rows.
cudaError_t launch_attn_join(const AttnLaunch& p, int splits, int bm, int TT, cudaStream_t s);
size_t attn_simt_workspace_bytes(int64_t T, int64_t N, int64_t Hq, int64_t Hkv, int64_t D,
                                 int64_t max_q);
// Tensor-core form: bf16, D in {64, 128, 256}, pages of a multiple of 16 rows.
bool attn_tc_supported(const AttnLaunch& p);
cudaError_t launch_attn_tc(const AttnLaunch& p, cudaStream_t s);
size_t attn_tc_workspace_bytes(int64_t T, int64_t N, int64_t Hq, int64_t Hkv, int64_t D,
                               int64_t max_q);

// The same attention over a cache in 8 bits (p.ks, p.vs, p.block).
// Few rows per kv head on tensor cores, and on CUDA cores (attn8_..._supported() sizes).
bool attn8_tc_supported(int64_t rows, int64_t D, bool bf16);
cudaError_t launch_attn8_tc(const AttnLaunch& p, cudaStream_t s);
size_t attn8_tc_workspace_bytes(int64_t rows, int64_t D);
bool attn8_rows_supported(int64_t rows, int64_t D);
cudaError_t launch_attn8_rows(const AttnLaunch& p, cudaStream_t s);
// Any sizes: the contexts of some sequences at a time are widened into the workspace, and
// the kernels above run on them.
cudaError_t launch_attn8_wide(const AttnLaunch& p, cudaStream_t s);
size_t attn8_wide_workspace_bytes(int64_t T, int64_t N, int64_t Hq, int64_t Hkv, int64_t D,
                                  int64_t max_q, bool bf16, int64_t max_pages, int64_t page_size);

// ---- searches over several continuations ----------------------------------------------

constexpr int kBeamMaxW = 64, kBeamMaxK = 128;

// The K best (beam, token) of each of B groups of W beams.
struct BeamLaunch {
  int B, W, V, K, pad;
  bool bf16;
  const void* logits;  // rows of V, strides in elements
  int64_t batch_stride, beam_stride;
  const float* scores;      // [B, W]
  const uint8_t* finished;  // [B, W] or null
  int32_t* parents;         // [B, K]
  int32_t* tokens;
  float* out_scores;
  void* ws;
};
size_t beam_workspace_bytes(int64_t B, int64_t W, int64_t V, int64_t K);
cudaError_t launch_beam(const BeamLaunch& p, cudaStream_t s);

// Slots copied (W = 0) or reordered within groups of W.
struct SlotPool {
  void* data;
  int64_t stride, bytes, slots;  // of a slot
  bool words;                    // in units of 4 bytes, not 16
  // set by the launch
  int pairs;                     // of an item
  int64_t piece, pieces, items;
};
constexpr int kMaxSlotPools = 48;
struct SlotsLaunch {
  int pools, W;
  int64_t n, most_slots;
  const int32_t* dst;
  const int32_t* src;
  unsigned* status;
  SlotPool pool[kMaxSlotPools];
};
cudaError_t launch_slots(SlotsLaunch& p, cudaStream_t s);

}  // namespace gdn
