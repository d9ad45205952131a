// Internal interface between the C ABI (gqa_api.cu) and the kernels
// (gqa_decode_lsu.cu, gqa_decode_tma.cu, gqa_merge.cu). Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "gqa_plan.h"

namespace gqa {

// Bits of the sticky device error word.
constexpr int kErrTimeoutFull = 1;   // a consumer waited too long for a stage's data
constexpr int kErrTimeoutEmpty = 2;  // the producer waited too long for a free stage
constexpr int kErrBadPage = 4;       // a kv_indices entry outside [0, num_pages)
constexpr int kErrBadIndptr = 8;     // kv_indptr not starting at 0 / decreasing
constexpr int kErrTicket = 16;       // a split sequence's arrival ticket did not settle
constexpr int kErrMergeWait = 32;    // an in-kernel merge waited too long for a sequence's pieces
constexpr int kErrKvBound = 64;      // a prompt pass's sequences hold more tokens than the caller's bound

struct DecodeParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int* kv_indptr;
  const int* kv_indices;
  void* out;
  float* lse;
  float* part_o;    // [2 * (P1 + P2)][NG][128 dims][8 heads] fp32
  float* part_lse;  // [2 * (P1 + P2)][NG][8 heads] fp32
  const int* skip_if_set;  // optional: return without work if *skip_if_set != 0
  int* err;                // device error word (bit flags below)
  unsigned long long* tickets;  // [P1 + P2][NG] arrival tickets of split sequences
  unsigned long long epoch;     // this call's ticket epoch (never 0, < 2^40)
  int4* split_rec;              // [P1 + P2] per-CTA split records for the merge kernel
  PlanConfig plan;              // the grid is plan.tier1_ctas + plan.tier2_ctas CTAs
  int batch;                    // sequences (sparse mode: query rows)
  int sparse_topk;              // 0: paged mode (kv_indptr / kv_indices); > 0: every row has this many
                                // columns and kv_indices holds their resolved slots (-1: masked out)
  int sparse_total;             // sparse mode: rows * sparse_topk (kv_indptr is not read)
  float scale_log2;        // sm_scale * log2(e)
  int num_pages_check;     // > 0: page ids are range-checked against it
  int fuse_max_splits;     // split sequences of at most this many pieces are merged by the decode kernel
  unsigned long long wait_limit_ns;  // give-up limit of a bounded wait (TMA variant; in-kernel merge)
  int inline_merge;             // one-wave mode: grid = tier-1 CTAs, tier 2 taken from `grab`, merge in-kernel
  unsigned long long* grab;     // [NG] one-wave mode: tier-2 range counters (epoch-tagged)
  // forms for long and shared contexts (kForm*)
  int index_count;              // entries of kv_indices
  int64_t whole_base;           // kFormParts: partial slot of sequence 0 when it is whole
  float* scores;                // kFormScores: [4][index_count][8], base 2
};

// Forms of the decode kernel (gqa_decode_lsu.cu, where they are described).
enum : int { kFormPlain = 0, kFormParts = 1, kFormHeads = 2, kFormScores = 3 };

// One-wave mode: a warp walks at most this many ranges (its tier-1 range and
// tier-2 ranges); the host uses the mode only when P2 <= (this - 1) * P1.
constexpr int kMaxWarpRanges = 16;

// How a decode kernel is launched.
enum : int { kLaunchPlain = 0, kLaunchPdl = 1, kLaunchCooperative = 2 };

// Default give-up limit of a bounded mbarrier wait (the drain before exit keeps it).
constexpr unsigned long long kDefaultWaitLimitNs = 2000000000ull;

// Default: every split sequence goes to the merge kernel, whose CTAs share the
// work of one sequence; merging inside the decode kernel (the warp that brings
// a sequence's last piece combines its partials) is a tuning option for
// sequences cut into at most fuse_max_splits pieces.
constexpr int kDefaultFuseMaxSplits = 1;

// Merge CTAs per boundary between consecutive decode CTAs.
constexpr int kMergeCtasPerBoundary = 1;

struct MergeParams {
  const int* kv_indptr;
  const float* part_o;
  const float* part_lse;
  void* out;
  float* lse;
  const int* skip_if_set;
  const int4* split_rec;          // the decode CTAs' split records
  unsigned long long epoch;       // the call's epoch (tags the records)
  PlanConfig plan;  // the decode kernel's plan
  int batch;
  int sparse_topk;   // as in DecodeParams
  int sparse_total;
  int use_pdl;
  int fuse_max_splits;  // sequences of at most this many pieces were merged by the decode kernel
  int index_cap;        // kFormScores: offsets are cut to it; -1: they are not
};

// Decode with the split partials in a fixed caller scratch (gqa_api.cu): a plan
// whose partials do not fit uses fewer tier-2 CTAs, down to none. Returns a
// GQA_* code (GQA_ERR_WORKSPACE if even the tier-1 partials do not fit).
int decode_in_scratch(const void* q, const void* k_cache, const void* v_cache, const int* kv_indptr,
                      const int* kv_indices, float sm_scale, void* out, float* lse, int batch, cudaStream_t stream,
                      void* scratch, size_t scratch_bytes);

// What a call of a decode form needs besides its own arguments (gqa_api.cu): the plan of the default variant under the
// present tuning, and the call's epoch. Returns a GQA_* code.
struct DecodeSetup {
  PlanConfig plan;
  bool default_plan;  // no tuning of CTA counts, tiers or smallest shares: the forms' own rules apply
  int sm_count;
  unsigned long long epoch;
  unsigned long long wait_limit_ns;
  int* err;
};
int decode_setup(bool fp8, DecodeSetup* setup);

// Dense MLA decode (gqa_mla.cu): one latent KV head of 576 values per token,
// 512 of them also V; `rows` = s_q * h_q query rows per sequence, a multiple
// of 16. The prep kernels fill kv_indptr_mut / slots_mut (workspace) from
// cache_seqlens and the block table; the decode and merge read them.
struct MlaParams {
  const void* q;             // [B][rows][576] bf16
  const void* kv;            // [num_blocks * page_size][576] bf16 (the cache, slot-major)
  const int* kv_indptr;      // [B + 1]
  int* kv_indptr_mut;        // the same buffer, written by the scan
  const int* slots;          // [T] slot of every cached token, -1 outside the pool
  int* slots_mut;
  void* out;                 // [B][rows][512] bf16
  float* lse;                // [B][h_q][s_q] fp32 natural log, or NULL
  float* part_o;             // [2 * CTAs][16][512] fp32
  float* part_lse;           // [2 * CTAs][16] fp32 (base 2)
  int4* split_rec;           // [2 * CTAs]
  int* err;
  PlanConfig plan;
  unsigned long long epoch;
  int batch, rows, h_q, s_q;
  float scale_log2;
  const int* block_table;  // [batch][width]
  int width, page_size, num_blocks;
  int piece_rows;  // query rows per piece (row group): 16, or 32 / 64 for the tensor-memory kernel's wide tiles
  // tensor-memory kernel, one tier: the first unit of each of the P1 CTAs (and the unit count at
  // [P1]), placed by the scan so that every CTA carries the same tokens plus piece_cost per sequence
  // start; NULL: the plan's equal ranges
  int64_t* bounds;
  int* cost_ptr;   // [B + 1] scratch of the scan: prefix of (length + piece_cost) over non-empty sequences
  int piece_cost;  // tokens one extra piece costs a CTA of the tensor-memory kernel
};

// MLA decode kernels: the tensor-memory kernel (block sizes that are a
// multiple of 32) and the mma.sync kernel with a 3-stage (3 CTAs per SM) or
// 4-stage (2 CTAs per SM) ring.
enum : int { kMlaKernelDefault = 0, kMlaKernelTensorMemory = 1, kMlaKernelMma3 = 3, kMlaKernelMma4 = 4 };
int mla_smem_bytes(int stages);
int mla_ctas_per_sm(int kind);
struct MlaTcMaps {  // 2D tensor maps of the latent cache (boxes of 64 x 32) and of Q (64 x 16)
  CUtensorMap kv;
  CUtensorMap q;
};
bool mla_tc_supported(int page_size);
int mla_tc_piece_rows(int rows);  // 64 / 32 when the rows of a sequence come in multiples of 64 / 32, else 16
bool mla_tc_encode(const MlaParams& p, MlaTcMaps* maps);
cudaError_t launch_mla_tc_decode(const MlaParams& p, const MlaTcMaps& maps, int ctas, cudaStream_t stream);
cudaError_t launch_mla(const MlaParams& p, const int* cache_seqlens, int kind, const MlaTcMaps* maps,
                       cudaStream_t stream);

// Compile-time variant of the decode kernel.
// kGatherLsuF8: FP8 caches only; kGatherLsuCc: the default's gather with the
// contractions on the CUDA cores (a comparison variant)
enum : int { kGatherLsu = 0, kGatherTma = 1, kGatherLsuF8 = 2, kGatherLsuCc = 3 };

struct KernelChoice {
  int gather;         // kGatherLsu: self-loading warps with cp.async; kGatherTma: producer warp + bulk copies
  int heads_per_cta;  // NG: KV heads per CTA (4, 2 or 1)
  int tile;           // tokens per pipeline stage (16; 32 for the TMA variant)
  int stages;         // pipeline depth
};

int lsu_smem_bytes(int ng, int stages);
int lsu_f8_smem_bytes(int stages, int tile);
int lsu_cc_smem_bytes();
cudaError_t launch_decode_lsu_cc(const DecodeParams& p, int num_ctas, cudaStream_t stream);
cudaError_t launch_decode_lsu_f8(int stages, int tile, const DecodeParams& p, int num_ctas, cudaStream_t stream,
                                 int launch);
cudaError_t launch_decode_lsu(int ng, int stages, const DecodeParams& p, int num_ctas, cudaStream_t stream,
                              int launch);
// The selected-token variant (p.sparse_topk > 0): 4 KV heads per CTA, 2 stages.
cudaError_t launch_decode_lsu_sparse(const DecodeParams& p, int num_ctas, cudaStream_t stream, int launch);
// A form other than kFormPlain: 4 KV heads per CTA, 2 stages (kFormHeads: bf16 caches only).
cudaError_t launch_decode_lsu_form(int form, bool fp8, const DecodeParams& p, int num_ctas, cudaStream_t stream, int launch);
// CTAs of a cp.async variant (sparse: the selected-token one) that the current
// device holds at once; 0 for the TMA variant or if unknown.
int decode_coresident_ctas(const KernelChoice& k, bool sparse);
// Resolve the selected columns of a sparse batch to slots (-1: invalid column).
cudaError_t launch_sparse_resolve(const int* logical_indices, const int* block_table, const int* token_to_req,
                                  int* slots, int rows, int topk, int page_size, int page_table_width,
                                  int num_requests, int num_cache_blocks, int sm_count, cudaStream_t stream);
int tma_smem_bytes(int ng, int tile, int stages);
cudaError_t launch_decode_tma(int ng, int tile, int stages, const DecodeParams& p, int num_ctas, cudaStream_t stream);

// Shared memory of a variant, or -1 if it is not compiled in.
inline int decode_smem_bytes(const KernelChoice& k) {
  if (k.gather == kGatherLsu) return k.tile == 16 ? lsu_smem_bytes(k.heads_per_cta, k.stages) : -1;
  if (k.gather == kGatherTma) return tma_smem_bytes(k.heads_per_cta, k.tile, k.stages);
  if (k.gather == kGatherLsuF8) return k.heads_per_cta == 4 ? lsu_f8_smem_bytes(k.stages, k.tile) : -1;
  if (k.gather == kGatherLsuCc) return k.heads_per_cta == 4 && k.tile == 16 && k.stages == 2 ? lsu_cc_smem_bytes() : -1;
  return -1;
}

// Warps a variant runs per CTA and the most CTAs per SM worth launching.
inline int decode_max_ctas_per_sm(const KernelChoice& k) {
  // LSU: up to 16 gathering warps per SM; TMA: up to 4 consumer warps per SM; FP8 and the
  // CUDA-core variant: 3 CTAs (their launch bounds leave 170 registers per thread); FP8 with
  // 32-token stages: 2 (shared memory).
  if (k.gather == kGatherLsuF8) return k.tile == 32 ? 2 : 3;
  if (k.gather == kGatherLsuCc) return 3;
  return k.gather == kGatherLsu ? 16 / k.heads_per_cta : 4 / k.heads_per_cta;
}

inline cudaError_t launch_decode(const KernelChoice& k, const DecodeParams& p, int num_ctas, cudaStream_t stream,
                                 int launch) {
  if (k.gather == kGatherLsu) return launch_decode_lsu(k.heads_per_cta, k.stages, p, num_ctas, stream, launch);
  if (k.gather == kGatherTma) return launch_decode_tma(k.heads_per_cta, k.tile, k.stages, p, num_ctas, stream);
  if (k.gather == kGatherLsuF8) return launch_decode_lsu_f8(k.stages, k.tile, p, num_ctas, stream, launch);
  if (k.gather == kGatherLsuCc) return launch_decode_lsu_cc(p, num_ctas, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_merge(int heads_per_cta, const MergeParams& p, cudaStream_t stream);
cudaError_t launch_validate(const int* indptr, const int* indices, int batch, int num_pages, int* err,
                            cudaStream_t stream);
cudaError_t launch_kv_append(const void* k_new, const void* v_new, const int* slots, void* k_cache, void* v_cache,
                             int n, int num_pages, int sm_count, cudaStream_t stream);
// ------------------------------------------- serving operators around decode
// Element types of gqa_rope (GQA_TYPE_* of the public header).
enum : int { kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2 };

struct RopeParams {  // gqa_rope.cu; strides in elements
  const void* x;
  void* out;
  const int* positions;    // [num_tokens]
  const double* inv_freq;  // [rot_dim / 2]
  int64_t x_token_stride, x_head_stride, out_token_stride, out_head_stride;
  float scale;
  int num_tokens, num_heads, head_dim, rot_offset, rot_dim, layout, inverse;
  int copy_rest;           // copy the elements outside the window (0: in place)
  int heads_each;          // heads a thread walks
};
cudaError_t launch_rope(const RopeParams& p, int dtype, int sm_count, cudaStream_t stream);

struct AppendParams {  // gqa_rope_append.cu; token strides in elements
  const void* q;  // [n][32][128] or NULL
  const void* k;  // [n][4][128]
  const void* v;
  const int* positions;
  const int* slots;
  const double* inv_freq;  // NULL: no rotation
  void* q_out;             // [n][32][128] contiguous
  void* k_cache;
  void* v_cache;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  int num_tokens, num_pages, rot_offset, rot_dim, layout, fp8;
  int splits;  // warps a token
};
cudaError_t launch_rope_append(AppendParams p, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_read_fp8(const void* k_cache, const void* v_cache, const int* indices, void* k_out, void* v_out,
                               int n, int num_pages, int sm_count, cudaStream_t stream);

struct MlaAppendParams {  // gqa_rope_append.cu
  const void* latent;  // [n][512]
  const void* k_rope;  // [n][64]
  const int* positions;
  const int* slots;
  const double* inv_freq;  // [32] or NULL
  void* kv_cache;          // [num_slots][576]
  int64_t latent_stride, rope_stride;
  float scale;
  int num_tokens, num_slots, layout;
};
cudaError_t launch_mla_append(const MlaAppendParams& p, int sm_count, cudaStream_t stream);

struct MlaProjParams {  // gqa_mla_proj.cu
  const void* x;  // absorb_q: q [n][h][192]; expand_out: o_lat [n][h][512]
  const void* w;  // [h][256][512]
  const int* positions;
  const double* inv_freq;  // [32] or NULL (absorb_q)
  void* out;               // [n][h][out_width] contiguous
  int64_t x_token_stride, x_head_stride;
  float scale;
  int num_tokens, num_heads, out_width, layout;
  int* err;
  unsigned long long wait_limit_ns;  // give-up limit of the tensor-memory kernel's waits
};
cudaError_t launch_mla_absorb_q(const MlaProjParams& p, cudaStream_t stream);
cudaError_t launch_mla_expand_out(const MlaProjParams& p, cudaStream_t stream);

// Latent attention's prompt pass (gqa_mla_prefill.cu).
struct MlaPrefillParams {
  const void* q;             // [total_q][h][192]
  const void* w;             // [h][256][512]
  const void* kv;            // [num_blocks * page_size][576]
  const int* block_table;    // [batch][width]
  const int* cache_seqlens;  // [batch]
  const int* cu_q;           // [batch + 1]
  void* out;                 // [total_q][h][128]
  float* lse;                // [h][total_q] or NULL
  int64_t q_token_stride, q_head_stride;
  float scale_log2;
  int batch, total_q, num_heads, page_size, num_blocks, width, causal;
  int fill;       // rows of no sequence: 1: out becomes 0, 2: lse becomes -inf, 0: they stay
  int cap;        // packed key rows the workspace holds, a multiple of 128
  int q_tiles;    // query tiles that total_q rows of batch sequences make at most
  int heads_per_pass;
  // workspace
  int* kv_len;    // [batch] keys of each sequence that are read
  int* kv_start;  // [batch + 1] first packed row (multiples of 128)
  int* q_start;   // [batch][2] first query row and query count, cut to [0, total_q)
  int* qt_start;  // [batch + 1] first query tile
  unsigned* amax;      // largest finite |value| bits: key weights, value weights; from [4] on [batch][4] latent, rotary key, and
                       // those of the token with the smallest ones above 0, inverted
  int* units;          // [num_heads] units of the attention taken so far, a counter a pass
  int* steps;          // [256] first step of each query tile (see kSplitTiles), [255] the most steps of one; then
                       // [256] the steps of each, the most first
  float* part;         // outputs and statistics of pieces; both NULL below kSplitRows packed rows
  unsigned* valid;     // [cap / 32] packed rows that hold a token of the pool
  unsigned* bad;       // [cap / 32] packed rows whose latent is not all finite
  uint2* row_top;      // [cap] largest finite |value| bits of a row: latent, rotary key
  float2* row_scale;   // [cap] in sequences whose rows have their own exponents: factor of the scores, exponent of the values
  void* lat;           // [cap][512] bf16
  void* kr;            // [cap][64] rotary keys: bf16 from the gather, fp16 (scaled) after the expansion
  void* kn;            // [heads_per_pass][cap][128] fp16 keys (scaled)
  void* vv;            // [heads_per_pass][cap][128] fp16 values (scaled)
  int* err;
  int pass, head0, heads;  // this pass over the heads, and its heads
  int head_group;      // heads whose CTAs run together
  int split;           // units may be split over their keys
};
// ------------------------------- decode forms for long and shared contexts
struct SharedParams {  // gqa_shared.cu
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int* prefix_indptr;   // [groups + 1]
  const int* prefix_indices;  // [prefix_count]
  const int* group_indptr;    // [groups + 1]
  const int* kv_indptr;       // [batch + 1]
  void* out;
  float* lse;                 // or NULL
  int64_t* group_start;       // [groups + 1] first step of each group's prefix (written by the prefix pass)
  // parts of 1024 outputs and 8 LSEs: the prefixes' [batch][4] and [pre_ctas / 2][64], [8 heads][128 dims] each; from
  // own_base on the own tokens' (DecodeParams::part_o, part_lse), [128 dims][8 heads]
  float* part_o;
  float* part_lse;
  int64_t own_base;
  int64_t whole_base;
  PlanConfig plan;
  float scale_log2;
  int batch, groups, prefix_count, index_count, num_pages, fp8;
  int pre_ctas;               // an even number; 0: no prefix has a token
  unsigned long long wait_limit_ns;
  int* err;
};
int shared_prefix_blocks(int batch, int ctas);
cudaError_t launch_shared(const SharedParams& p, const DecodeParams& own, cudaStream_t stream);

struct BoundsParams {  // gqa_blocks.cu
  const void* k_cache;     // [num_blocks][page_size][4][128]
  void* bounds;            // [num_blocks][2][4][128]
  const int* block_table;  // [requests][width]
  const int* lens;         // [requests]
  const int* first;        // [requests] or NULL: 0
  int requests, page_size, num_blocks, width;
};
cudaError_t launch_block_bounds(const BoundsParams& p, int sm_count, cudaStream_t stream);

struct BlockParams {  // gqa_blocks.cu
  const void* q;            // [rows][32][128]
  const void* bounds;
  const int* block_table;   // [requests][width]
  const int* token_to_req;  // [rows]
  const int* lens;          // [rows]
  int* blocks;              // [rows][4][top]
  float* scores;            // workspace: [rows][4][width] scores, NaN of bits kNoBlock where there is none
  float* errors;            // [rows][4][ceil(width / 16)] error bounds of 16 scores
  float2* again;            // [rows][4][width] scores formed again
  int* slots;               // [4][rows * top * page_size]
  int rows, requests, page_size, num_blocks, width, top, keep_first, keep_last;
};
cudaError_t launch_block_select(const BlockParams& p, cudaStream_t stream);
cudaError_t launch_block_slots(const BlockParams& p, int sm_count, cudaStream_t stream);

struct WeighParams {  // gqa_weights.cu
  const float* scores;  // [4][index_count][8]
  const float* lse;     // [batch][32]
  const float* weights; // [batch][width]
  float* out;           // the same, or `weights` itself
  const int* kv_indptr;
  float decay;
  int batch, width, index_count;
};
cudaError_t launch_weigh(const WeighParams& p, cudaStream_t stream);

struct EvictParams {  // gqa_weights.cu
  const float* weights;  // [batch][width]
  const int* kv_indptr;
  const int* kv_indices;
  float* weights_out;
  int* new_indptr;   // [batch + 1]
  int* new_indices;  // [index_count]
  int* freed_indptr;
  int* freed;
  int budget, keep_first, keep_last, batch, width, index_count;
  int cluster, held;  // blocks a sequence, words that one holds in shared memory (set by the launch)
  int sums;           // a kernel ahead forms new_indptr and freed_indptr (set by the launch)
};
cudaError_t launch_evict(EvictParams p, int sm_count, cudaStream_t stream);
void set_evict_cluster_limit(int blocks);  // test hook; 0: none

// Launches a kernel that begins with pdl_wait() so that it may start while the one before it on the stream ends, over
// clusters of `cluster` blocks.
template <typename Params>
inline cudaError_t launch_chained(void (*kernel)(Params), dim3 grid, int threads, int smem, cudaStream_t stream, int cluster,
                                  const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// A tensor map of 2 or 3 dimensions (sizes and boxes from the contiguous one on, `pitch` bytes between steps of the
// others, 128-byte swizzle). False if the driver call is missing or refuses.
bool tc_encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const int64_t* size,
               const int64_t* pitch, const int* box);
// Rows of `width` values, `pitch` bytes apart, as boxes of box_w x box_rows.
bool tc_encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t width, int64_t rows,
                  int64_t pitch, int box_w, int box_rows);
// Bytes of the workspace; with base != NULL also points the params' fields into it.
size_t mla_prefill_workspace(MlaPrefillParams* p, char* base);
cudaError_t launch_mla_prefill(MlaPrefillParams p, int sm_count, cudaStream_t stream);

cudaError_t read_and_clear_device_error(int* out);
cudaError_t device_error_word(int** ptr);  // device address of the error word (current device)
// GQA_OK, the SM count and the give-up limit of bounded waits when the current device is supported
int current_device_sms(int* sm_count, unsigned long long* wait_limit_ns = nullptr);

// Raises a kernel's dynamic shared-memory limit to `bytes` once per device
// (`done` is the kernel's own flag table, zero-initialised static storage).
// Safe to call from several host threads at once: the attribute call is
// idempotent and the flags are atomic. Devices past the table set it on
// every call.
constexpr int kMaxDevices = 64;
inline cudaError_t set_attribute_once(std::atomic<int> (&done)[kMaxDevices], const void* fn, cudaFuncAttribute what, int value) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < kMaxDevices;
  if (tracked && done[dev].load(std::memory_order_acquire) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, what, value);
  if (e == cudaSuccess && tracked) done[dev].store(1, std::memory_order_release);
  return e;
}
inline cudaError_t set_smem_limit_once(std::atomic<int> (&done)[kMaxDevices], const void* fn, int bytes) {
  return set_attribute_once(done, fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace gqa
