// C ABI of the decode's forms for long and shared contexts: shared prefixes, selected blocks, accumulated weights and the
// eviction by them. Argument checks and launches only; no call synchronises, allocates or keeps state.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_paged_decode.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kPartBytes = gqa::kHeadDim * gqa::kGroup * sizeof(float);  // outputs of one part and KV head

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
int launched(cudaError_t e) { return e == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH; }
bool scale_ok(float s) { return std::isfinite(s) && std::isfinite(s * kLog2e); }
bool format_ok(int f) { return f == GQA_CACHE_BF16 || f == GQA_CACHE_FP8; }
// Sizes that kernels walk in steps of up to 8192: no index of theirs passes 31 bits.
constexpr int kMostItems = 1 << 30;
bool items_ok(int n) { return n >= 0 && n <= kMostItems; }
bool table_ok(int page_size, int num_blocks, int width) {
  return page_size > 0 && num_blocks > 0 && width > 0 && width <= kMostItems && static_cast<int64_t>(num_blocks) * page_size <= INT_MAX &&
         static_cast<int64_t>(width) * page_size <= INT_MAX;
}

// The split decode's share of a workspace: outputs and LSEs of 2 parts a CTA, and the split records.
struct DecodeSpace {
  size_t o, lse, rec, end;
  DecodeSpace(const gqa::PlanConfig& plan, size_t at) {
    const size_t ctas = static_cast<size_t>(plan.tier1_ctas) + plan.tier2_ctas, parts = 2 * ctas * gqa::kKvHeads;
    o = at;
    lse = o + parts * kPartBytes;
    rec = lse + round256(parts * gqa::kGroup * sizeof(float));
    end = rec + round256(ctas * 16);
  }
};

// The plan for `tokens` at most. The second tier evens out long ranges; where a CTA of the first has few tokens, its ranges of 64
// tokens begin when the first's, as short, are done. Two tiers and one, us a call, by tokens a CTA: blocks of bf16 caches 9: 15.5
// and 16.7, 21: 17.6 both, 36: 28 and 20, 72: 34 and 25, 287: 61 and 55, 449: 84 and 82, 575: 101 and 105; accumulated weights, FP8
// caches 35: 24 and 19, 283: 52 and 47, 555: 84 and 77, 1169: 157 and 153, 2278: 289 and 307.
// Short sequences: a CTA takes them one after another (2 us each), so its smallest share is two of them where they are shorter than
// 16 tokens, and no second tier (100 sequences of a token each: 78 us with shares of 32 tokens, 13 of 2).
void share_for(gqa::PlanConfig& plan, int64_t tokens, int64_t sequences) {
  const int64_t two = 2 * tokens / sequences;
  if (two >= plan.min_units) return;
  plan.min_units = static_cast<int>(two < 2 ? 2 : two);
  plan.tier2_ctas = 0;
}

gqa::PlanConfig plan_for(const gqa::DecodeSetup& setup, int64_t tokens, int64_t sequences, bool fp8) {
  gqa::PlanConfig plan = setup.plan;
  if (!setup.default_plan) return plan;
  share_for(plan, tokens, sequences);
  if (tokens >= int64_t{20} * plan.tier1_ctas && tokens < int64_t{fp8 ? 1536 : 512} * plan.tier1_ctas) plan.tier2_ctas = 0;
  return plan;
}

gqa::DecodeParams decode_params(const gqa::DecodeSetup& setup, void* part_o, void* part_lse, void* split_rec, float sm_scale) {
  gqa::DecodeParams d{};
  d.part_o = static_cast<float*>(part_o);
  d.part_lse = static_cast<float*>(part_lse);
  d.split_rec = static_cast<int4*>(split_rec);
  d.err = setup.err;
  d.epoch = setup.epoch;
  d.plan = setup.plan;
  d.scale_log2 = sm_scale * kLog2e;
  d.fuse_max_splits = 1;  // parts are joined by the kernel behind
  d.wait_limit_ns = setup.wait_limit_ns;
  return d;
}

gqa::MergeParams merge_params(const gqa::DecodeParams& d) {
  gqa::MergeParams m{};
  m.kv_indptr = d.kv_indptr;
  m.part_o = d.part_o;
  m.part_lse = d.part_lse;
  m.out = d.out;
  m.lse = d.lse;
  m.split_rec = d.split_rec;
  m.epoch = d.epoch;
  m.plan = d.plan;
  m.batch = d.batch;
  m.sparse_topk = d.sparse_topk;
  m.sparse_total = d.sparse_total;
  m.use_pdl = 1;
  m.fuse_max_splits = 1;
  m.index_cap = d.sparse_topk > 0 ? -1 : d.index_count;
  return m;
}

// Parts of the prefixes, then of the own tokens: one array of outputs, one of LSEs.
struct SharedSpace {
  int64_t own_base, whole_base;
  size_t start, o, lse, rec, end;
  SharedSpace(const gqa::DecodeSetup& setup, int batch, int groups) {
    const int64_t ctas = static_cast<int64_t>(setup.plan.tier1_ctas) + setup.plan.tier2_ctas;
    own_base = gqa::shared_prefix_blocks(batch, setup.sm_count);
    whole_base = 2 * ctas;
    const size_t parts = static_cast<size_t>(own_base + (whole_base + batch) * gqa::kKvHeads);
    start = 0;
    o = round256((static_cast<size_t>(groups) + 1) * sizeof(int64_t));
    lse = o + parts * kPartBytes;
    rec = lse + round256(parts * gqa::kGroup * sizeof(float));
    end = rec + round256(static_cast<size_t>(ctas) * 16);
  }
};

struct SelectSpaceLayout {
  size_t scores, errors, again, end;
  SelectSpaceLayout(int rows, int width) {
    const size_t n = static_cast<size_t>(rows) * gqa::kKvHeads * static_cast<size_t>(width);
    scores = 0;
    errors = round256(n * sizeof(float));
    again = errors + round256(static_cast<size_t>(rows) * gqa::kKvHeads * ((static_cast<size_t>(width) + 15) / 16) * sizeof(float));
    end = again + round256(n * sizeof(float2));
  }
};

// How the SMs are shared between the prefix pass, a pair of CTAs on two, and the own tokens' decode, which runs beside it on the
// others: the number of pairs whose estimate, as far as the sizes tell (groups alike, offsets that use all of the indices), has
// both done soonest. In us, measured with 4 to 72 pairs of 76: the pass 20 and 1.6 a step of its run (FP8 2.6; 1.3 and 2.1 where
// the sequences of a group fill one tile), 0.3 a part that is joined, and 7 where a run ends inside a unit, or for each unit more that it holds; the decode 16
// and 0.031 a token and SM, at least what HBM takes. Against shares in proportion and the decode's whole grid: 16384 tokens x 128
// sequences with 64 to 1024 own tokens 68 -> 62, 4000 x 64 with 500 to 4000 87 -> 60, 500 x 64 with 2000 to 8000 170 -> 115, four
// groups of 1000 x 32 with 100 to 1500 66 -> 47.
int prefix_pairs(int sms, int batch, int groups, int prefix_count, int index_count, bool fp8) {
  const int pairs = sms / 2;
  if (groups <= 0 || prefix_count <= 0 || pairs == 0) return 0;
  const int64_t members = (batch - 1) / groups + 1, units = gqa::kKvHeads * ((members - 1) / 64 + 1) * groups;
  const int64_t tiles = (prefix_count - 1) / (int64_t{128} * groups) + 1, steps = units * tiles;
  const double step = members <= 32 ? (fp8 ? 2.1 : 1.3) : (fp8 ? 2.6 : 1.6), least = index_count * (fp8 ? 1056 / 6.3e6 : 2048 / 6.3e6);
  int best = 1;
  double best_us = 1e30;
  int64_t last = 0;
  for (int n = 1; n <= pairs - (index_count > 0 && pairs > 1); ++n) {
    const int64_t run = (steps - 1) / n + 1;
    if (run == last) continue;  // more pairs, none of them done sooner
    last = run;
    const double pass = 20 + step * run + 0.3 * tiles / run + (run > tiles ? 7.0 * ((run - 1) / tiles) : (tiles % run != 0 ? 7.0 : 0.0));
    const double alone = index_count * 0.031 / (sms - 2 * n), r = std::fmin(alone, least) / std::fmax(std::fmax(alone, least), 1e-9), r3 = r * r * r;
    const double own = 16 + std::fmax(alone, least) * (1 + 0.15 * r3 * r3);  // both near the end of what they have
    const double us = std::fmax(pass, own) + 0.1 * std::fmin(pass, own);
    if (us < best_us) best_us = us, best = n;
  }
  return best;
}

// The decode's plan beside `pairs` pairs: one tier that fills the other SMs, three CTAs each, or two where they have few tokens
// (2048 tokens x 64 sequences with 200 to 1000 own tokens 28 us with two, 32 with three; groups of 1000 x 32 with 100 to 1500
// 50 and 47; FP8 caches always three: 61 and 54 for 4000 x 64).
gqa::PlanConfig plan_beside(const gqa::DecodeSetup& setup, int pairs, int index_count, int batch, bool fp8) {
  gqa::PlanConfig plan = setup.plan;
  const int left = setup.sm_count - 2 * pairs;
  if (!setup.default_plan || left <= 0) return plan;
  share_for(plan, index_count, batch);
  const int ctas = left * (!fp8 && index_count < 512 * left ? 2 : 3);
  if (index_count < 20 * ctas) return plan;  // (8 sequences of 148 tokens behind 2048: 19.4 us with the whole grid, 21.0)
  if (ctas < plan.tier1_ctas) plan.tier1_ctas = ctas;
  plan.tier2_ctas = 0;
  return plan;
}

bool select_sizes_ok(int rows, int width) { return rows > 0 && width > 0 && width <= kMostItems && static_cast<int64_t>(rows) * width <= (int64_t{1} << 34); }
bool sparse_sizes_ok(int rows, int top, int page_size) {
  return rows > 0 && top > 0 && page_size > 0 && static_cast<int64_t>(top) * page_size <= INT_MAX &&
         static_cast<int64_t>(rows) * (static_cast<int64_t>(top) * page_size) <= INT_MAX;
}

}  // namespace

extern "C" {

size_t gqa_shared_paged_decode_ws_size(int batch, int groups, int cache_format) {
  gqa::DecodeSetup setup;
  if (batch <= 0 || batch > (1 << 20) || groups < 0 || groups > (1 << 20) || !format_ok(cache_format) || gqa::decode_setup(cache_format == GQA_CACHE_FP8, &setup) != GQA_OK) return 0;
  return SharedSpace(setup, batch, groups).end;
}

int gqa_shared_paged_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* prefix_indptr,
                            const int32_t* prefix_indices, const int32_t* group_indptr, const int32_t* kv_indptr,
                            const int32_t* kv_indices, float sm_scale, void* out, float* lse, int batch, int groups,
                            int prefix_count, int index_count, int num_pages, int cache_format, void* workspace,
                            size_t workspace_bytes, struct CUstream_st* stream) {
  if (batch < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (batch == 0) return GQA_OK;
  if (batch > (1 << 20) || groups < 0 || groups > (1 << 20) || !items_ok(prefix_count) || !items_ok(index_count) || num_pages < 0 ||
      !format_ok(cache_format) || !scale_ok(sm_scale))
    return GQA_ERR_INVALID_ARGUMENT;
  if (q == nullptr || kv_indptr == nullptr || out == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (groups > 0 && (prefix_indptr == nullptr || group_indptr == nullptr)) return GQA_ERR_INVALID_ARGUMENT;
  if (prefix_count > 0 && prefix_indices == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (index_count > 0 && kv_indices == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 8) ||
      !aligned(prefix_indptr, 4) || !aligned(prefix_indices, 4) || !aligned(group_indptr, 4) || !aligned(kv_indptr, 4) ||
      !aligned(kv_indices, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  if (workspace == nullptr || !aligned(workspace, 256)) return GQA_ERR_WORKSPACE;
  const bool fp8 = cache_format == GQA_CACHE_FP8;
  gqa::DecodeSetup setup;
  const int rc = gqa::decode_setup(fp8, &setup);
  if (rc != GQA_OK) return rc;
  const SharedSpace at(setup, batch, groups);
  if (workspace_bytes < at.end) return GQA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  float* part_o = reinterpret_cast<float*>(ws + at.o);
  float* part_lse = reinterpret_cast<float*>(ws + at.lse);
  gqa::DecodeParams d = decode_params(setup, part_o + at.own_base * (gqa::kHeadDim * gqa::kGroup),
                                      part_lse + at.own_base * gqa::kGroup, ws + at.rec, sm_scale);
  d.q = q;
  d.k_cache = k_cache;
  d.v_cache = v_cache;
  d.kv_indptr = kv_indptr;
  d.kv_indices = kv_indices;
  d.out = out;
  d.lse = lse;
  d.batch = batch;
  d.num_pages_check = num_pages;
  d.index_count = index_count;
  d.whole_base = at.whole_base;
  gqa::SharedParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.prefix_indptr = prefix_indptr;
  p.prefix_indices = prefix_indices;
  p.group_indptr = group_indptr;
  p.kv_indptr = kv_indptr;
  p.out = out;
  p.lse = lse;
  p.group_start = reinterpret_cast<int64_t*>(ws + at.start);
  const int pairs = prefix_pairs(setup.sm_count, batch, groups, prefix_count, index_count, fp8);
  p.pre_ctas = 2 * pairs;
  p.wait_limit_ns = setup.wait_limit_ns;
  p.part_o = part_o;
  p.part_lse = part_lse;
  p.own_base = at.own_base;
  p.whole_base = d.whole_base;
  d.plan = pairs > 0 ? plan_beside(setup, pairs, index_count, batch, fp8) : plan_for(setup, index_count, batch, fp8);
  p.plan = d.plan;
  p.scale_log2 = d.scale_log2;
  p.batch = batch;
  p.groups = groups;
  p.prefix_count = prefix_count;
  p.index_count = index_count;
  p.num_pages = num_pages;
  p.fp8 = fp8 ? 1 : 0;
  p.err = setup.err;
  return launched(gqa::launch_shared(p, d, stream));
}

int gqa_block_bounds(const void* k_cache, void* bounds, const int32_t* block_table, const int32_t* lens,
                     const int32_t* first, int requests, int page_size, int num_blocks, int page_table_width,
                     struct CUstream_st* stream) {
  if (requests < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (requests == 0) return GQA_OK;
  if (!items_ok(requests) || !items_ok(page_size) || !table_ok(page_size, num_blocks, page_table_width)) return GQA_ERR_INVALID_ARGUMENT;
  if (k_cache == nullptr || bounds == nullptr || block_table == nullptr || lens == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(first, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  const gqa::BoundsParams p{k_cache, bounds, block_table, lens, first, requests, page_size, num_blocks, page_table_width};
  return launched(gqa::launch_block_bounds(p, sms, stream));
}

size_t gqa_block_select_ws_size(int rows, int page_table_width) {
  return select_sizes_ok(rows, page_table_width) ? SelectSpaceLayout(rows, page_table_width).end : 0;
}

int gqa_block_select(const void* q, const void* bounds, const int32_t* block_table, const int32_t* token_to_req,
                     const int32_t* lens, int32_t* blocks, int rows, int requests, int page_size, int num_blocks,
                     int page_table_width, int top, int keep_first, int keep_last, void* workspace, size_t workspace_bytes,
                     struct CUstream_st* stream) {
  if (rows < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return GQA_OK;
  if (!table_ok(page_size, num_blocks, page_table_width) || requests <= 0 || !select_sizes_ok(rows, page_table_width))
    return GQA_ERR_INVALID_ARGUMENT;
  if (top <= 0 || keep_first < 0 || keep_last < 0 || keep_first > top || keep_last > top - keep_first ||
      static_cast<int64_t>(rows) * top > INT_MAX)
    return GQA_ERR_INVALID_ARGUMENT;
  if (q == nullptr || bounds == nullptr || block_table == nullptr || token_to_req == nullptr || lens == nullptr || blocks == nullptr)
    return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) || !aligned(token_to_req, 4) || !aligned(lens, 4) ||
      !aligned(blocks, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  const SelectSpaceLayout at(rows, page_table_width);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < at.end) return GQA_ERR_WORKSPACE;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  gqa::BlockParams p{};
  p.q = q;
  p.bounds = bounds;
  p.block_table = block_table;
  p.token_to_req = token_to_req;
  p.lens = lens;
  p.blocks = blocks;
  p.scores = reinterpret_cast<float*>(ws + at.scores);
  p.errors = reinterpret_cast<float*>(ws + at.errors);
  p.again = reinterpret_cast<float2*>(ws + at.again);
  p.rows = rows;
  p.requests = requests;
  p.page_size = page_size;
  p.num_blocks = num_blocks;
  p.width = page_table_width;
  p.top = top;
  p.keep_first = keep_first;
  p.keep_last = keep_last;
  return launched(gqa::launch_block_select(p, stream));
}

size_t gqa_block_sparse_decode_ws_size(int rows, int top, int page_size) {
  gqa::DecodeSetup setup;
  if (!sparse_sizes_ok(rows, top, page_size) || gqa::decode_setup(false, &setup) != GQA_OK) return 0;
  return DecodeSpace(setup.plan, round256(sizeof(int32_t) * gqa::kKvHeads * static_cast<size_t>(rows) * top * page_size)).end;
}

int gqa_block_sparse_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* blocks,
                            const int32_t* block_table, const int32_t* token_to_req, const int32_t* lens, float sm_scale,
                            void* out, float* lse, int rows, int requests, int top, int page_size, int num_blocks,
                            int page_table_width, void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  if (rows < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return GQA_OK;
  if (!table_ok(page_size, num_blocks, page_table_width) || requests <= 0 || !sparse_sizes_ok(rows, top, page_size) || !scale_ok(sm_scale))
    return GQA_ERR_INVALID_ARGUMENT;
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || blocks == nullptr || block_table == nullptr ||
      token_to_req == nullptr || lens == nullptr || out == nullptr)
    return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 8) ||
      !aligned(blocks, 4) || !aligned(block_table, 4) || !aligned(token_to_req, 4) || !aligned(lens, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  if (workspace == nullptr || !aligned(workspace, 256)) return GQA_ERR_WORKSPACE;
  gqa::DecodeSetup setup;
  const int rc = gqa::decode_setup(false, &setup);
  if (rc != GQA_OK) return rc;
  const int total = rows * (top * page_size);
  const DecodeSpace at(setup.plan, round256(sizeof(int32_t) * gqa::kKvHeads * static_cast<size_t>(total)));
  if (workspace_bytes < at.end) return GQA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  gqa::BlockParams p{};
  p.block_table = block_table;
  p.token_to_req = token_to_req;
  p.lens = lens;
  p.blocks = const_cast<int32_t*>(blocks);
  p.slots = reinterpret_cast<int32_t*>(ws);
  p.rows = rows;
  p.requests = requests;
  p.page_size = page_size;
  p.num_blocks = num_blocks;
  p.width = page_table_width;
  p.top = top;
  if (gqa::launch_block_slots(p, setup.sm_count, stream) != cudaSuccess) return GQA_ERR_LAUNCH;
  gqa::DecodeParams d = decode_params(setup, ws + at.o, ws + at.lse, ws + at.rec, sm_scale);
  d.q = q;
  d.k_cache = k_cache;
  d.v_cache = v_cache;
  d.kv_indices = p.slots;
  d.out = out;
  d.lse = lse;
  d.batch = rows;
  d.sparse_topk = top * page_size;
  d.sparse_total = total;
  d.plan = plan_for(setup, total, rows, false);
  if (gqa::launch_decode_lsu_form(gqa::kFormHeads, false, d, d.plan.tier1_ctas + d.plan.tier2_ctas, stream,
                                  gqa::kLaunchPdl) != cudaSuccess)
    return GQA_ERR_LAUNCH;
  return launched(gqa::launch_merge(gqa::kKvHeads, merge_params(d), stream));
}

size_t gqa_paged_decode_weighted_ws_size(int index_count, int cache_format) {
  gqa::DecodeSetup setup;
  if (!items_ok(index_count) || !format_ok(cache_format) || gqa::decode_setup(cache_format == GQA_CACHE_FP8, &setup) != GQA_OK) return 0;
  return DecodeSpace(setup.plan, round256(static_cast<size_t>(index_count) * gqa::kQoHeads * sizeof(float))).end;
}

int gqa_paged_decode_weighted(const void* q, const void* k_cache, const void* v_cache, const int32_t* kv_indptr,
                              const int32_t* kv_indices, float sm_scale, const float* weights, float decay,
                              float* weights_out, void* out, float* lse, int batch, int width, int index_count,
                              int num_pages, int cache_format, void* workspace, size_t workspace_bytes,
                              struct CUstream_st* stream) {
  if (batch < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (batch == 0) return GQA_OK;
  if (!items_ok(batch) || !items_ok(width) || !items_ok(index_count) || num_pages < 0 || !format_ok(cache_format) || !scale_ok(sm_scale) || !std::isfinite(decay))
    return GQA_ERR_INVALID_ARGUMENT;
  if (q == nullptr || kv_indptr == nullptr || out == nullptr || lse == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (width > 0 && (weights == nullptr || weights_out == nullptr)) return GQA_ERR_INVALID_ARGUMENT;
  if (index_count > 0 && kv_indices == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 8) ||
      !aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(kv_indptr, 4) || !aligned(kv_indices, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  if (workspace == nullptr || !aligned(workspace, 256)) return GQA_ERR_WORKSPACE;
  const bool fp8 = cache_format == GQA_CACHE_FP8;
  gqa::DecodeSetup setup;
  const int rc = gqa::decode_setup(fp8, &setup);
  if (rc != GQA_OK) return rc;
  const DecodeSpace at(setup.plan, round256(static_cast<size_t>(index_count) * gqa::kQoHeads * sizeof(float)));
  if (workspace_bytes < at.end) return GQA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  gqa::DecodeParams d = decode_params(setup, ws + at.o, ws + at.lse, ws + at.rec, sm_scale);
  d.q = q;
  d.k_cache = k_cache;
  d.v_cache = v_cache;
  d.kv_indptr = kv_indptr;
  d.kv_indices = kv_indices;
  d.out = out;
  d.lse = lse;
  d.batch = batch;
  d.num_pages_check = num_pages;
  d.index_count = index_count;
  d.scores = reinterpret_cast<float*>(ws);
  d.plan = plan_for(setup, index_count, batch, fp8);
  if (gqa::launch_decode_lsu_form(gqa::kFormScores, fp8, d, d.plan.tier1_ctas + d.plan.tier2_ctas, stream,
                                  gqa::kLaunchPlain) != cudaSuccess)
    return GQA_ERR_LAUNCH;
  if (gqa::launch_merge(gqa::kKvHeads, merge_params(d), stream) != cudaSuccess) return GQA_ERR_LAUNCH;
  const gqa::WeighParams w{d.scores, lse, weights, weights_out, kv_indptr, decay, batch, width, index_count};
  return launched(gqa::launch_weigh(w, stream));
}

int gqa_kv_evict(const float* weights, const int32_t* kv_indptr, const int32_t* kv_indices, int budget, int keep_first,
                 int keep_last, float* weights_out, int32_t* new_indptr, int32_t* new_indices, int32_t* freed_indptr,
                 int32_t* freed, int batch, int width, int index_count, struct CUstream_st* stream) {
  if (batch < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (batch == 0) return GQA_OK;
  if (!items_ok(batch) || !items_ok(width) || !items_ok(index_count) || budget < 0 || keep_first < 0 || keep_last < 0 || keep_first > budget ||
      keep_last > budget - keep_first)
    return GQA_ERR_INVALID_ARGUMENT;
  if (kv_indptr == nullptr || new_indptr == nullptr || freed_indptr == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (width > 0 && (weights == nullptr || weights_out == nullptr || weights == weights_out)) return GQA_ERR_INVALID_ARGUMENT;
  if (index_count > 0 && (kv_indices == nullptr || new_indices == nullptr || freed == nullptr || new_indices == kv_indices ||
                          freed == kv_indices || freed == new_indices))
    return GQA_ERR_INVALID_ARGUMENT;
  if (new_indptr == kv_indptr || freed_indptr == kv_indptr || freed_indptr == new_indptr) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(kv_indptr, 4) || !aligned(kv_indices, 4) ||
      !aligned(new_indptr, 4) || !aligned(new_indices, 4) || !aligned(freed_indptr, 4) || !aligned(freed, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  const gqa::EvictParams p{weights, kv_indptr, kv_indices, weights_out, new_indptr, new_indices, freed_indptr, freed,
                           budget, keep_first, keep_last, batch, width, index_count, 1, 0, 0};
  return launched(gqa::launch_evict(p, sms, stream));
}

int gqa_paged_decode_test_cluster_limit(int blocks) {
  if (blocks < 0 || blocks > 16 || (blocks & (blocks - 1)) != 0) return GQA_ERR_INVALID_ARGUMENT;
  gqa::set_evict_cluster_limit(blocks);
  return GQA_OK;
}

}  // extern "C"
