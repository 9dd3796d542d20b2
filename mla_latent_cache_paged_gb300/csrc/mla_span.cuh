// Decode over parts of a batch's cached tokens (mla_decode_shared,
// mla_decode_window): what the schedule, the attention kernel and the merge
// share.
//
// An item is up to 128 query rows that see the same tokens: the pages
// 0 .. head_pages - 1 of a block-table row and, `page_shift` pages further on,
// the pages after them (virtual pages 0 .. pages - 1 in all), of whose tokens
// t those with t < end and (t < sink_end or t >= tail_lo). Items are
//   - 128 rows (several requests' heads) of a group that shares a prefix, over
//     the prefix,
//   - one request's heads over the tokens that it does not share, or over its
//     sinks and window.
// An item's work is its steps of two pages; kSpanItemCost steps of fixed cost
// (query staging, epilogue) stand before them. The items' units, one after
// another, are cut into contiguous ranges, one per CTA pair, of about equal
// length. The part of an item that lies in one pair's range is a piece. An item that is the only
// one of its rows and is not cut writes the results; every other piece leaves
// its rows (fp32, normalised) and their LSEs in the workspace, piece of pair c
// from row part_row + 128 c on, which no other piece uses: from one piece to the
// next either c grows by one or part_row by the item's rows (at most 128).
#pragma once

#include "mla_device.cuh"

namespace mla {

constexpr int kSpanRows = 128;
constexpr int kSpanStepPages = 2;
// An item's fixed cost. 64 requests of 32 heads over two fp8 prefixes of 8,000 to
// 12,000 tokens take 72.8 us with 2, 79.4 with 1, 72.6 with 3, a window of 4,000
// over 96 of them 63.7, 70.7 and 64.5; in bf16 48 requests of 16 heads over five
// prefixes 27.7, 28.6 and 28.7, a prefix of 16,384 under 64 requests of 128 heads
// 203, 208 and 204.
constexpr int kSpanItemCost = 2;
// All cuts move to items' edges if no pair's share grows by more than this: the
// pieces of an item that is cut are merged from fp32 rows. 128 requests of 64 heads
// over 640 tokens take 30.8 us with 4, 2 or 6 and 34.8 with 0; a window of 1,024 over
// 128 requests of 128 heads 56 to 59 with 4 or 6, 60 with 0 or 2.
constexpr int kSpanCutCost = 4;
// Prefixes are shared if that saves as many steps for every pair: items of their
// own come with pieces to merge for every row. With 4 groups of 8 requests of 16
// heads, 1,024 tokens together and 128 each, it saves 2.84 and takes 18.8 us
// (22.6 apart); 32 groups of 4 requests of 64 heads, 512 together, would save
// 1.68 and take 37.1 (30.8 apart). Between 1.1 and 2.9 the two are mostly within
// 1 us of each other (fp8 cache: the same, 22.6 against 27.5, 44.7 against 39.5).
constexpr int kSpanShareGain = 2;
constexpr int kSpanMaxBatch = 4096;

struct alignas(16) SpanItem {       // 64 bytes
    int32_t unit0;      // units [unit0, unit1) of the call's work
    int32_t unit1;
    int32_t row0;       // its rows of q, out and lse: row0 .. row0 + rows - 1
    int32_t rows;
    int32_t table_row;
    int32_t pages;
    int32_t head_pages;
    int32_t page_shift;
    int32_t sink_end;
    int32_t tail_lo;
    int32_t end;
    int32_t part_row;
    int32_t alone;      // the only item of its rows
    int16_t first_pair; // the pairs that work on it
    int16_t last_pair;
};
static_assert(sizeof(SpanItem) == 64, "four 16-byte loads");

struct SpanParams {
    const uint16_t* q;             // bf16 [B, N, 576]
    const void* cache;             // bf16 or E4M3 [num_blocks, 64, 576]
    int64_t num_blocks;
    const int32_t* table;          // [B, max_blocks]
    const int32_t* seq_lens;       // [B]
    const int32_t* group_starts;   // [groups + 1]
    const int32_t* shared_lens;    // [groups]
    int32_t groups;
    int32_t window, sinks;         // window = 0: none
    int32_t batch, heads, max_blocks;
    int32_t pairs;                 // CTA pairs of the grid
    float scale_log2, v_scale;
    uint16_t* out;
    float* lse;
    // In the workspace.
    int32_t* status;
    SpanItem* items;               // tiles of shared prefixes first; none without units
    int32_t* tile_row;             // [B]: 128 * the first of the request's tiles + the row in it, or -1
    int32_t* own_item;             // [B]: the request's other item, or -1
    float* o_part;                 // [rows, 512]
    float* lse_part;               // [rows]
    uint64_t timeout_ns;
    uint32_t debug;
};

int launch_span_attention(const SpanParams& p, bool fp8, void* stream);
int launch_span_merge(const SpanParams& p, void* stream);

}  // namespace mla
