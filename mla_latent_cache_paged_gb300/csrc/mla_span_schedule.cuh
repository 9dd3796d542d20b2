// The schedule of mla_decode_shared and mla_decode_window, made by every CTA of
// the attention kernel for itself, from the lengths on the device (so that a
// captured call can be replayed with others): a kernel of its own in front
// cost 4 to 5 us a call, which is when its dependent's CTAs start. The items'
// numbers and units follow from a scan over groups and requests; each pair
// writes the records of the items that it works on (those that several pairs
// work on come out the same), the first CTA what the merge needs of each
// request. Bound by latency: of 3,400 cycles for 4 requests without groups (5,600
// for 8 requests in one) 900 are the lengths' way from L2, 900 the scan, 900 the
// cuts; the pair's CTAs wait for each other's barriers meanwhile.
#pragma once

#include <climits>

#include "mla_span.cuh"

namespace mla {

// What a CTA keeps of the schedule while it works.
constexpr int kSpanKept = 14;
struct SpanRange {
    int32_t g0, g1;      // the pair's units
    int32_t first, end;  // the items that they belong to
    SpanItem kept[kSpanKept];
};

// Shared memory that making the schedule takes. Requests' items and units are
// counted from the first of their own (the tiles' come before them).
struct SpanScratch {
    int4 warps[32];
    // Where the pairs' ranges may begin (equal ones, ranges of whole items): the
    // unit, and twice its item's number, plus one if it is not the item's first.
    int2 cuts[kMaxBalancedPairs + 1], edges[kMaxBalancedPairs + 1];
    int32_t lens[kSpanMaxBatch];
    int32_t req_unit0[kSpanMaxBatch + 1];     // requests' own items: where their units begin
    int32_t req_item[kSpanMaxBatch + 1];      // the items before the request's own
    int32_t req_group[kSpanMaxBatch];         // the request's group if that has tiles, or -1
    int32_t starts[kSpanMaxBatch + 1];
    int32_t pages[kSpanMaxBatch];             // shortest member's length, then the prefix's pages
    int32_t tile0[kSpanMaxBatch];             // the tiles before the group's
    int32_t group_unit0[kSpanMaxBatch];       // where their units begin
    int32_t leader[kSpanMaxBatch];            // its first member with tokens
    int32_t shared[kSpanMaxBatch];
    int32_t saved;                            // the units that sharing saves
};

__device__ __forceinline__ int4 operator+(int4 a, int4 b) {
    return make_int4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Exclusive prefix sums over the CTA's threads, of which the first n have
// something to add; *total: the sums.
__device__ __forceinline__ int4 span_scan(int4 v, int n, int4* warps, int4* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int count = (min(n, int(blockDim.x)) + 31) >> 5;
    int4 incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int4 up = make_int4(__shfl_up_sync(0xffffffffu, incl.x, o),
                                  __shfl_up_sync(0xffffffffu, incl.y, o),
                                  __shfl_up_sync(0xffffffffu, incl.z, o),
                                  __shfl_up_sync(0xffffffffu, incl.w, o));
        if (lane >= o) incl = incl + up;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    int4 before = make_int4(0, 0, 0, 0), all = before;
#pragma unroll 4
    for (int w = 0; w < count; ++w) {
        const int4 sum = warps[w];
        if (w < warp) before = before + sum;
        all = all + sum;
    }
    *total = all;
    return make_int4(before.x + incl.x - v.x, before.y + incl.y - v.y, before.z + incl.z - v.z,
                     before.w + incl.w - v.w);
}

__device__ __forceinline__ int span_steps(int pages) {
    return (pages + kSpanStepPages - 1) / kSpanStepPages;
}

// A length, or 0 (recorded) for one that no table row can have.
__device__ __forceinline__ int span_length(const SpanParams& p, int L) {
    if (L < 0 || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
        record_error(p.status, MLA_ERR_BAD_SEQ_LEN, L);
        return 0;
    }
    return L;
}

// The last i < n with a[i] <= v (a[0] <= v, a not decreasing).
template <typename T>
__device__ __forceinline__ int span_find(const T* a, int n, T v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
}

// Called by all threads of the CTA. (The plan sees to it that a call's units
// are fewer than 2^31.)
__device__ __forceinline__ void span_schedule(const SpanParams& p, SpanScratch& s, int pair,
                                              bool first_cta, SpanRange* range) {
    const int tid = threadIdx.x, threads = blockDim.x;
    const int B = p.batch;
    int G = p.groups;
    if (tid == 0) {
        range->first = range->end = 0;
        range->g0 = range->g1 = 0;
        s.saved = 0;
    }
    // Lengths and groups, read together; groups only if their starts make sense:
    // not decreasing, within the batch.
    bool bad = false;
    const int top = G > 0 && G >= B ? G + 1 : B;
    for (int i = tid; i < top; i += threads) {
        const bool start = G > 0 && i <= G;
        const int L = i < B ? p.seq_lens[i] : 0;
        const int a = start ? p.group_starts[i] : 0;
        const int before = start && i > 0 ? p.group_starts[i - 1] : 0;
        const int S = i < G ? p.shared_lens[i] : 0;
        if (i < B) {
            s.lens[i] = span_length(p, L);
            s.req_group[i] = -1;
        }
        if (start) {
            s.starts[i] = a;
            bad = bad || a < 0 || a > B || before > a;
        }
        if (i < G) {
            s.shared[i] = span_length(p, S);
            s.pages[i] = s.leader[i] = INT_MAX;
        }
    }
    if (__syncthreads_or(bad ? 1 : 0)) {
        if (tid == 0) record_error(p.status, MLA_ERR_BAD_ROW, 0);
        G = 0;
    }
    if (G > 0) {
        const int begin = s.starts[0], end = s.starts[G];
        for (int b = begin + tid; b < end; b += threads) {
            const int g = span_find(s.starts, G, b);
            s.req_group[b] = g;
            if (s.lens[b] > 0) {
                atomicMin(&s.pages[g], s.lens[b]);
                atomicMin(&s.leader[g], b);
            }
        }
        __syncthreads();
        for (int g = tid; g < G; g += threads) {
            const int members = s.starts[g + 1] - s.starts[g];
            const int shortest = s.pages[g] == INT_MAX ? 0 : s.pages[g];
            const int pg = min(s.shared[g], shortest) / kPageSize;
            const int tiles = (members * p.heads + kSpanRows - 1) / kSpanRows;
            // Worth it where a tile holds the rows of several requests: the
            // steps that this saves against the tiles' fixed cost.
            const int saved = (members - tiles) * span_steps(pg) - tiles * kSpanItemCost;
            s.pages[g] = saved > 0 ? pg : 0;
            if (saved > 0) atomicAdd(&s.saved, saved);
        }
        __syncthreads();
        if (s.saved < kSpanShareGain * p.pairs) G = 0;
    }

    // A request's own item, but for its place.
    auto own_item = [&](int b) {
        SpanItem it{};
        const int L = s.lens[b], g = s.req_group[b];
        const int shared = G > 0 && g >= 0 && L > 0 ? s.pages[g] : 0;
        it.row0 = b * p.heads;
        it.rows = p.heads;
        it.table_row = b;
        it.end = L;
        it.alone = shared == 0;
        it.page_shift = shared;
        if (p.window > 0) {
            const int lo = L > p.window ? L - p.window : 0;
            const int head = int((int64_t(p.sinks) + kPageSize - 1) / kPageSize);
            it.sink_end = p.sinks;
            it.tail_lo = lo;
            if (lo / kPageSize > head) {
                it.head_pages = head;
                it.page_shift = lo / kPageSize - head;
            }
        }
        it.pages = pages_of(L) - it.page_shift;
        return it;
    };
    // Tiles and their units (x, y), requests' items and theirs (z, w).
    int4 done = make_int4(0, 0, 0, 0);
    for (int i0 = 0; i0 < B || i0 < G; i0 += threads) {
        const int i = i0 + tid;
        int4 v = make_int4(0, 0, 0, 0), total;
        if (i < G && s.pages[i] > 0) {
            v.x = ((s.starts[i + 1] - s.starts[i]) * p.heads + kSpanRows - 1) / kSpanRows;
            v.y = v.x * (kSpanItemCost + span_steps(s.pages[i]));
        }
        const int steps = i < B ? span_steps(own_item(i).pages) : 0;
        if (steps > 0) {
            v.z = 1;
            v.w = kSpanItemCost + steps;
        }
        if (i0 > 0) __syncthreads();       // (the scan before has been read)
        const int4 at = done + span_scan(v, max(B, G) - i0, s.warps, &total);
        done = done + total;
        if (i < G) {
            s.tile0[i] = at.x;
            s.group_unit0[i] = at.y;
        }
        if (i < B) {
            s.req_item[i] = at.z;
            s.req_unit0[i] = at.w;
        }
    }
    const int tiles = done.x, tile_units = done.y, T = done.y + done.w;
    const int C = T < p.pairs ? T : p.pairs;
    if (tid == 0) {
        s.req_item[B] = done.z;
        s.req_unit0[B] = done.w;
        s.cuts[C] = s.edges[C] = make_int2(T, 2 * (done.x + done.z));
    }
    __syncthreads();

    // The cuts between the pairs' ranges: equal ones, or all moved to an item's
    // edge if that costs no pair much (then no item leaves pieces).
    auto tile_units_of = [&](int g) { return kSpanItemCost + span_steps(s.pages[g]); };
    const int share = C > 0 ? int(unsigned(T) / unsigned(C)) : 0, rest = T - share * C;
    for (int c = tid; c < C; c += threads) {
        const int u = c * share + min(c, rest);
        int u0, u1, index;
        if (u < tile_units) {
            const int g = span_find(s.group_unit0, G, u), each = tile_units_of(g);
            const int k = int(unsigned(u - s.group_unit0[g]) / unsigned(each));
            index = s.tile0[g] + k;
            u0 = s.group_unit0[g] + k * each;
            u1 = u0 + each;
        } else {
            const int b = span_find(s.req_unit0, B, u - tile_units);
            index = tiles + s.req_item[b];
            u0 = tile_units + s.req_unit0[b];
            u1 = tile_units + s.req_unit0[b + 1];
        }
        s.cuts[c] = make_int2(u, 2 * index + (u > u0 ? 1 : 0));
        s.edges[c] = u - u0 <= u1 - u ? make_int2(u0, 2 * index) : make_int2(u1, 2 * index + 2);
    }
    __syncthreads();
    const int most = share + (rest > 0 ? 1 : 0) + kSpanCutCost;
    bool far = false;
    for (int c = tid; c < C; c += threads) far = far || s.edges[c + 1].x - s.edges[c].x > most;
    const bool whole = __syncthreads_or(far ? 1 : 0) == 0;

    // The pair's items, and the pairs that work on each.
    const int2* cuts = whole ? s.edges : s.cuts;
    const int2 from = pair < C ? cuts[pair] : make_int2(0, 0);
    const int2 to = pair < C ? cuts[pair + 1] : from;
    const int g0 = from.x, g1 = to.x;
    if (g0 < g1) {
        auto pair_of = [&](int u) {
            const int longer = rest * (share + 1);       // units of the pairs with one more
            return u < longer ? int(unsigned(u) / unsigned(share + 1))
                              : rest + int(unsigned(u - longer) / unsigned(share));
        };
        const int first = from.y >> 1, end = (to.y + 1) >> 1;
        for (int i = first + tid; i < end; i += threads) {
            SpanItem it{};
            if (i < tiles) {
                const int g = span_find(s.tile0, G, i), k = i - s.tile0[g], each = tile_units_of(g);
                it.unit0 = s.group_unit0[g] + k * each;
                it.unit1 = it.unit0 + each;
                it.row0 = s.starts[g] * p.heads + k * kSpanRows;
                it.rows = min(kSpanRows, s.starts[g + 1] * p.heads - it.row0);
                it.table_row = s.leader[g];
                it.pages = s.pages[g];
                it.end = s.pages[g] * kPageSize;
                it.part_row = i * kSpanRows;
            } else {
                const int b = span_find(s.req_item, B, i - tiles);
                it = own_item(b);
                it.unit0 = tile_units + s.req_unit0[b];
                it.unit1 = tile_units + s.req_unit0[b + 1];
                it.part_row = tiles * kSpanRows + (i - tiles) * p.heads;
            }
            it.first_pair = int16_t(whole ? pair : pair_of(it.unit0 + kSpanItemCost));
            it.last_pair = int16_t(whole ? pair : pair_of(it.unit1 - 1));
            p.items[i] = it;
            if (i - first < kSpanKept) range->kept[i - first] = it;
        }
        if (tid == 0) {
            range->first = first;
            range->end = end;
            range->g0 = g0;
            range->g1 = g1;
        }
    }
    if (first_cta)
        for (int b = tid; b < B; b += threads) {
            const int g = s.req_group[b];
            p.tile_row[b] = G > 0 && g >= 0 && s.pages[g] > 0 && s.lens[b] > 0
                                ? s.tile0[g] * kSpanRows + (b - s.starts[g]) * p.heads
                                : -1;
            p.own_item[b] =
                s.req_unit0[b + 1] > s.req_unit0[b] ? tiles + s.req_item[b] : -1;
        }
}

}  // namespace mla
