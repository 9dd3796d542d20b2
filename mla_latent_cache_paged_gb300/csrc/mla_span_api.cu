// C ABI of the decodes over parts of a batch's cached tokens: the plan and the
// argument checks of mla_decode_shared and mla_decode_window (declared in
// include/mla_decode.h).
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>

#include "mla_span.cuh"

namespace mla {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Where the workspace's arrays lie.
struct SpanLayout {
    uint64_t tile_row, own_item, items, lse_part, o_part, bytes;
};

SpanLayout layout_of(int64_t batch, int64_t heads, int64_t groups, int64_t pairs) {
    auto up = [](uint64_t n) { return (n + 255) & ~uint64_t(255); };
    // A group's last tile may be part full; only groups of two requests or
    // more have tiles.
    const int64_t shared = groups < batch / 2 ? groups : batch / 2;
    const int64_t tiles = groups > 0 ? batch * heads / kSpanRows + shared : 0;
    const int64_t rows = tiles * kSpanRows + batch * heads + pairs * kSpanRows;
    SpanLayout s{};
    s.tile_row = kStatusBytes;
    s.own_item = s.tile_row + up(uint64_t(batch) * 4);
    s.items = s.own_item + up(uint64_t(batch) * 4);
    s.lse_part = s.items + up(uint64_t(tiles + batch) * sizeof(SpanItem));
    s.o_part = s.lse_part + up(uint64_t(rows) * 4);
    s.bytes = s.o_part + uint64_t(rows) * kLkv * 4;
    return s;
}

int check_plan(const mla_span_plan_t* plan) {
    if (!plan) return MLA_ERR_INVALID_ARG;
    mla_span_plan_t want;
    const int rc = mla_span_plan(plan->batch, plan->num_heads, plan->max_blocks_per_seq,
                                 plan->max_groups, plan->num_sms, plan->flags, &want);
    if (rc != MLA_OK) return rc;
    return std::memcmp(plan, &want, sizeof(want)) == 0 ? MLA_OK : MLA_ERR_INVALID_ARG;
}

// What both decodes check, and their launches. p: groups or window set.
int decode_spans(const mla_span_plan_t* plan, SpanParams p, bool fp8, const void* q,
                 const void* cache, int64_t num_blocks, const int32_t* block_table,
                 const int32_t* seq_lens, float softmax_scale, float k_scale, void* out, float* lse,
                 void* workspace, size_t workspace_bytes, void* stream) {
    if (num_blocks < 1 || !std::isfinite(softmax_scale)) return MLA_ERR_INVALID_ARG;
    if (fp8 && (!std::isfinite(k_scale) || !(k_scale > 0.f))) return MLA_ERR_INVALID_ARG;
    p.scale_log2 = softmax_scale * (fp8 ? k_scale : 1.f) * 1.4426950408889634f;
    if (!std::isfinite(p.scale_log2)) return MLA_ERR_INVALID_ARG;
    // A scale of zero weighs every token 1; so does the smallest normal one in
    // fp32, and a masked score of -inf stays -inf.
    if (std::fabs(p.scale_log2) < FLT_MIN) p.scale_log2 = FLT_MIN;
    p.v_scale = fp8 ? k_scale : 1.f;
    if (num_blocks > tc_max_blocks()) return MLA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < plan->workspace_bytes || !aligned(workspace, 256))
        return MLA_ERR_WORKSPACE;
    if (plan->batch == 0) return MLA_OK;
    if (!q || !cache || !block_table || !seq_lens || !out) return MLA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || (lse && !aligned(lse, 4)))
        return MLA_ERR_INVALID_ARG;
    p.q = static_cast<const uint16_t*>(q);
    p.cache = cache;
    p.num_blocks = num_blocks;
    p.table = block_table;
    p.seq_lens = seq_lens;
    p.batch = plan->batch;
    p.heads = plan->num_heads;
    p.max_blocks = plan->max_blocks_per_seq;
    p.pairs = plan->pairs;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    const SpanLayout s = layout_of(plan->batch, plan->num_heads, plan->max_groups, plan->pairs);
    char* ws = static_cast<char*>(workspace);
    p.status = reinterpret_cast<int32_t*>(ws);
    p.items = reinterpret_cast<SpanItem*>(ws + s.items);
    p.tile_row = reinterpret_cast<int32_t*>(ws + s.tile_row);
    p.own_item = reinterpret_cast<int32_t*>(ws + s.own_item);
    p.o_part = reinterpret_cast<float*>(ws + s.o_part);
    p.lse_part = reinterpret_cast<float*>(ws + s.lse_part);
    p.timeout_ns = kDefaultTimeoutNs;
    if (plan->flags & MLA_PLAN_DEBUG_WITHHOLD_LOAD) {
        p.debug = kDebugWithholdLoad;
        p.timeout_ns = kDebugTimeoutNs;
    }
    if (launch_span_attention(p, fp8, stream) != 0 || launch_span_merge(p, stream) != 0)
        return MLA_ERR_CUDA;
    return MLA_OK;
}

int decode_shared(const mla_span_plan_t* plan, bool fp8, const void* q, const void* cache,
                  int64_t num_blocks, const int32_t* block_table, const int32_t* seq_lens,
                  const int32_t* group_starts, const int32_t* shared_lens, int num_groups,
                  float softmax_scale, float k_scale, void* out, float* lse, void* workspace,
                  size_t workspace_bytes, void* stream) {
    const int rc = check_plan(plan);
    if (rc != MLA_OK) return rc;
    if (num_groups < 0 || num_groups > plan->max_groups) return MLA_ERR_INVALID_ARG;
    if (num_groups > 0 && (!group_starts || !shared_lens || !aligned(group_starts, 4) ||
                           !aligned(shared_lens, 4)))
        return MLA_ERR_INVALID_ARG;
    SpanParams p{};
    p.group_starts = group_starts;
    p.shared_lens = shared_lens;
    p.groups = num_groups;
    return decode_spans(plan, p, fp8, q, cache, num_blocks, block_table, seq_lens, softmax_scale,
                        k_scale, out, lse, workspace, workspace_bytes, stream);
}

int decode_window(const mla_span_plan_t* plan, bool fp8, const void* q, const void* cache,
                  int64_t num_blocks, const int32_t* block_table, const int32_t* seq_lens,
                  int window, int sinks, float softmax_scale, float k_scale, void* out, float* lse,
                  void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_plan(plan);
    if (rc != MLA_OK) return rc;
    if (window < 1 || sinks < 0) return MLA_ERR_INVALID_ARG;
    SpanParams p{};
    p.window = window;
    p.sinks = sinks;
    return decode_spans(plan, p, fp8, q, cache, num_blocks, block_table, seq_lens, softmax_scale,
                        k_scale, out, lse, workspace, workspace_bytes, stream);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_span_plan(int batch, int num_heads, int max_blocks_per_seq, int max_groups,
                             int num_sms, uint32_t flags, mla_span_plan_t* plan) {
    if (!plan || batch < 0 || num_heads < 1 || max_blocks_per_seq < 1 || max_groups < 0 ||
        num_sms < 1)
        return MLA_ERR_INVALID_ARG;
    if (flags & ~MLA_PLAN_DEBUG_WITHHOLD_LOAD) return MLA_ERR_INVALID_ARG;
    if (num_heads > kMaxHeads || batch > kSpanMaxBatch || max_groups > kSpanMaxBatch ||
        max_blocks_per_seq > tc_max_blocks() ||
        // (the schedule counts units, at most a page of each table row and six
        // for its two items, in 32 bits)
        int64_t(batch) * (int64_t(max_blocks_per_seq) + 6) > INT_MAX)
        return MLA_ERR_UNSUPPORTED;
    std::memset(plan, 0, sizeof(*plan));
    plan->batch = batch;
    plan->num_heads = num_heads;
    plan->max_blocks_per_seq = max_blocks_per_seq;
    plan->max_groups = max_groups;
    plan->num_sms = num_sms;
    plan->flags = flags;
    const int pairs = num_sms / 2 > 1 ? num_sms / 2 : 1;
    plan->pairs = pairs < kMaxBalancedPairs ? pairs : kMaxBalancedPairs;
    plan->workspace_bytes = layout_of(batch, num_heads, max_groups, plan->pairs).bytes;
    return MLA_OK;
}

extern "C" int mla_decode_shared(const mla_span_plan_t* plan, const void* q,
                                 const void* latent_cache, int64_t num_blocks,
                                 const int32_t* block_table, const int32_t* seq_lens,
                                 const int32_t* group_starts, const int32_t* shared_lens,
                                 int num_groups, float softmax_scale, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    return decode_shared(plan, false, q, latent_cache, num_blocks, block_table, seq_lens,
                         group_starts, shared_lens, num_groups, softmax_scale, 1.f, out, lse,
                         workspace, workspace_bytes, stream);
}

extern "C" int mla_decode_shared_fp8(const mla_span_plan_t* plan, const void* q,
                                     const void* latent_cache_fp8, int64_t num_blocks,
                                     const int32_t* block_table, const int32_t* seq_lens,
                                     const int32_t* group_starts, const int32_t* shared_lens,
                                     int num_groups, float softmax_scale, float k_scale, void* out,
                                     float* lse, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    return decode_shared(plan, true, q, latent_cache_fp8, num_blocks, block_table, seq_lens,
                         group_starts, shared_lens, num_groups, softmax_scale, k_scale, out, lse,
                         workspace, workspace_bytes, stream);
}

extern "C" int mla_decode_window(const mla_span_plan_t* plan, const void* q,
                                 const void* latent_cache, int64_t num_blocks,
                                 const int32_t* block_table, const int32_t* seq_lens, int window,
                                 int sinks, float softmax_scale, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    return decode_window(plan, false, q, latent_cache, num_blocks, block_table, seq_lens, window,
                         sinks, softmax_scale, 1.f, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int mla_decode_window_fp8(const mla_span_plan_t* plan, const void* q,
                                     const void* latent_cache_fp8, int64_t num_blocks,
                                     const int32_t* block_table, const int32_t* seq_lens,
                                     int window, int sinks, float softmax_scale, float k_scale,
                                     void* out, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    return decode_window(plan, true, q, latent_cache_fp8, num_blocks, block_table, seq_lens, window,
                         sinks, softmax_scale, k_scale, out, lse, workspace, workspace_bytes,
                         stream);
}
