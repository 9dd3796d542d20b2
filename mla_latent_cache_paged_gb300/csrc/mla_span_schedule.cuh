// The schedule of mla_decode_shared and mla_decode_window, made by every CTA of
// the attention kernel for itself, from the lengths on the device (so that a
// captured call can be replayed with others): a kernel of its own in front
// cost 4 to 5 us a call, which is when its dependent's CTAs start. The items'
// numbers and units follow from a scan over groups and requests; each pair
// writes the records of the items that it works on (those that several pairs
// work on come out the same), the first CTA what the merge needs of each
// request. Bound by the latency of a few dependent loads and barriers.
#pragma once

#include <climits>

#include "mla_span.cuh"

namespace mla {

// What a CTA keeps of the schedule while it works.
constexpr int kSpanKept = 14;
struct SpanRange {
    int64_t g0, g1;      // the pair's units
    int32_t first, end;  // the items that they belong to
    SpanItem kept[kSpanKept];
};

// Shared memory that making the schedule takes.
struct SpanScratch {
    int64_t cuts[kMaxBalancedPairs + 1], edges[kMaxBalancedPairs + 1];
    int64_t req_unit0[kSpanMaxBatch + 1];     // requests' own items: where their units begin
    int64_t group_unit0[kSpanMaxBatch + 1];   // groups' tiles: likewise
    uint64_t warps[32];
    int32_t lens[kSpanMaxBatch];
    int32_t req_item[kSpanMaxBatch + 1];      // the items before the request's own
    int32_t req_group[kSpanMaxBatch];         // the request's group if that has tiles, or -1
    int32_t starts[kSpanMaxBatch + 1];
    int32_t pages[kSpanMaxBatch];             // shortest member's length, then the prefix's pages
    int32_t tile0[kSpanMaxBatch + 1];         // the tiles before the group's
    int32_t leader[kSpanMaxBatch];            // its first member with tokens
    int32_t shared[kSpanMaxBatch];
};

// Exclusive prefix sum over the CTA's threads; *total: the sum.
__device__ __forceinline__ uint64_t span_scan(uint64_t v, uint64_t* warps, uint64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, count = blockDim.x >> 5;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    // (every warp sums the warps for itself)
    uint64_t s = lane < count ? warps[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t n = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += n;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const uint64_t before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + incl - v;
}

// A number of items (high 20 bits) and of units, added together.
constexpr int kUnitBits = 44;
__device__ __forceinline__ uint64_t span_packed(int items, int64_t units) {
    return (uint64_t(items) << kUnitBits) | uint64_t(units);
}
__device__ __forceinline__ int span_items(uint64_t v) { return int(v >> kUnitBits); }
__device__ __forceinline__ int64_t span_units(uint64_t v) {
    return int64_t(v & ((uint64_t(1) << kUnitBits) - 1));
}

__device__ __forceinline__ int span_steps(int pages) {
    return (pages + kSpanStepPages - 1) / kSpanStepPages;
}

__device__ __forceinline__ int span_length(const SpanParams& p, int b) {
    const int L = p.seq_lens[b];
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

// a / b, in 32 bits where that does (a division in 64 takes some 400 cycles).
__device__ __forceinline__ int64_t span_div(int64_t a, int b) {
    return (a >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// Called by all threads of the CTA.
__device__ __forceinline__ void span_schedule(const SpanParams& p, SpanScratch& s, int pair,
                                              bool first_cta, SpanRange* range) {
    const int tid = threadIdx.x, threads = blockDim.x;
    const int B = p.batch;
    int G = p.groups;
    if (tid == 0) {
        range->first = range->end = 0;
        range->g0 = range->g1 = 0;
    }
    for (int b = tid; b < B; b += threads) {
        s.lens[b] = span_length(p, b);
        s.req_group[b] = -1;
    }
    uint64_t done = 0, total;                    // items and units so far
    if (G > 0) {
        // Groups, if their starts make sense: not decreasing, within the batch.
        bool bad = false;
        for (int g = tid; g <= G; g += threads) {
            const int a = p.group_starts[g], before = g > 0 ? p.group_starts[g - 1] : 0;
            s.starts[g] = a;
            bad = bad || a < 0 || a > B || before > a;
            if (g < G) {
                const int S = p.shared_lens[g];
                const bool past = S < 0 || int64_t(S) > int64_t(p.max_blocks) * kPageSize;
                if (past) record_error(p.status, MLA_ERR_BAD_SEQ_LEN, S);
                s.shared[g] = past ? 0 : S;
                s.pages[g] = s.leader[g] = INT_MAX;
            }
        }
        if (__syncthreads_or(bad ? 1 : 0)) {
            if (tid == 0) record_error(p.status, MLA_ERR_BAD_ROW, 0);
            G = 0;
        }
    }
    if (G > 0) {
        for (int b = tid; b < B; b += threads) {
            if (b < s.starts[0] || b >= s.starts[G]) continue;
            const int g = span_find(s.starts, G, b);
            s.req_group[b] = g;
            if (s.lens[b] > 0) {
                atomicMin(&s.pages[g], s.lens[b]);
                atomicMin(&s.leader[g], b);
            }
        }
        __syncthreads();
        // The prefixes and their tiles.
        for (int g0 = 0; g0 < G; g0 += threads) {
            const int g = g0 + tid;
            int n = 0, steps = 0;
            if (g < G) {
                const int members = s.starts[g + 1] - s.starts[g];
                const int shortest = s.pages[g] == INT_MAX ? 0 : s.pages[g];
                const int pg = min(s.shared[g], shortest) / kPageSize;
                const int tiles = (members * p.heads + kSpanRows - 1) / kSpanRows;
                steps = span_steps(pg);
                // Worth it where a tile holds the rows of several requests: the
                // steps that this saves against the tiles' fixed cost.
                n = int64_t(members - tiles) * steps > int64_t(tiles) * kSpanItemCost ? tiles : 0;
                s.pages[g] = n > 0 ? pg : 0;
            }
            const int64_t units = int64_t(n) * (kSpanItemCost + steps);
            const uint64_t at = done + span_scan(span_packed(n, units), s.warps, &total);
            done += total;
            if (g < G) {
                s.tile0[g] = span_items(at);
                s.group_unit0[g] = span_units(at);
            }
        }
        __syncthreads();
    }
    const int tiles = span_items(done);
    const int64_t tile_units = span_units(done);

    // A request's own item, but for its place.
    auto own_item = [&](int b) {
        SpanItem it{};
        const int L = s.lens[b], g = s.req_group[b];
        const int shared = g >= 0 && L > 0 ? s.pages[g] : 0;
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
    for (int b0 = 0; b0 < B; b0 += threads) {
        const int b = b0 + tid;
        const int steps = b < B ? span_steps(own_item(b).pages) : 0;
        const int n = steps > 0 ? 1 : 0;
        const uint64_t at =
            done + span_scan(span_packed(n, n > 0 ? kSpanItemCost + steps : 0), s.warps, &total);
        done += total;
        if (b < B) {
            s.req_item[b] = span_items(at);
            s.req_unit0[b] = span_units(at);
        }
    }
    const int items = span_items(done);
    const int64_t T = span_units(done);
    const int C = int(T < p.pairs ? T : p.pairs);
    if (tid == 0) {
        s.req_item[B] = items;
        s.req_unit0[B] = T;
        s.cuts[C] = s.edges[C] = T;
    }
    __syncthreads();

    // The item that holds unit u: of a request (its number), or a tile.
    auto tile_units_of = [&](int g) { return kSpanItemCost + span_steps(s.pages[g]); };
    auto find_request = [&](int64_t u) { return span_find(s.req_unit0, B, u); };
    auto find_tile = [&](int64_t u, int* g) {
        *g = span_find(s.group_unit0, G, u);
        return int(span_div(u - s.group_unit0[*g], tile_units_of(*g)));
    };
    // The cuts between the pairs' ranges: equal ones, or all moved to an item's
    // edge if that costs no pair much (then no item leaves pieces).
    for (int c = tid; c < C; c += threads) {
        const int64_t u = span_div(c * T, C);
        int64_t u0, u1;
        if (u < tile_units) {
            int g;
            const int k = find_tile(u, &g);
            u0 = s.group_unit0[g] + int64_t(k) * tile_units_of(g);
            u1 = u0 + tile_units_of(g);
        } else {
            const int b = find_request(u);
            u0 = s.req_unit0[b];
            u1 = s.req_unit0[b + 1];
        }
        s.cuts[c] = u;
        s.edges[c] = u - u0 <= u1 - u ? u0 : u1;
    }
    __syncthreads();
    if (tid < 32) {
        int64_t most = 0;
        for (int c = tid; c < C; c += 32) most = max(most, s.edges[c + 1] - s.edges[c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        const bool whole = C > 0 && most <= span_div(T + C - 1, C) + kSpanCutCost;
        for (int c = tid; c < C; c += 32)
            if (whole) s.cuts[c] = s.edges[c];
    }
    __syncthreads();

    // The pair's items, and the pairs that work on each.
    const int64_t g0 = pair < C ? s.cuts[pair] : 0, g1 = pair < C ? s.cuts[pair + 1] : 0;
    if (g0 < g1) {
        auto place = [&](SpanItem it, int index, int first) {
            it.first_pair = int16_t(span_find(s.cuts, C, it.unit0 + kSpanItemCost));
            it.last_pair = int16_t(span_find(s.cuts, C, it.unit1 - 1));
            p.items[index] = it;
            if (index - first < kSpanKept) range->kept[index - first] = it;
        };
        int first = -1, end = 0, g = 0, k = 0;
        if (g0 < tile_units) {
            k = find_tile(g0, &g);
            first = s.tile0[g] + k;
            end = tiles;
            if (g1 <= tile_units) {
                int ge;
                const int ke = find_tile(g1 - 1, &ge);
                end = s.tile0[ge] + ke + 1;
            }
            for (int i = first + tid; i < end; i += threads) {
                const int gi = span_find(s.tile0, G, i), ki = i - s.tile0[gi];
                SpanItem it{};
                it.unit0 = s.group_unit0[gi] + int64_t(ki) * tile_units_of(gi);
                it.unit1 = it.unit0 + tile_units_of(gi);
                it.row0 = s.starts[gi] * p.heads + ki * kSpanRows;
                it.rows = min(kSpanRows, s.starts[gi + 1] * p.heads - it.row0);
                it.table_row = s.leader[gi];
                it.pages = s.pages[gi];
                it.end = s.pages[gi] * kPageSize;
                it.part_row = i * kSpanRows;
                place(it, i, first);
            }
        }
        if (g1 > tile_units) {
            const int b0 = find_request(g0 > tile_units ? g0 : tile_units);
            const int b1 = find_request(g1 - 1);
            if (first < 0) first = s.req_item[b0];
            end = s.req_item[b1] + 1;
            for (int b = b0 + tid; b <= b1; b += threads) {
                if (s.req_unit0[b + 1] == s.req_unit0[b]) continue;      // (nothing to do)
                SpanItem it = own_item(b);
                it.unit0 = s.req_unit0[b];
                it.unit1 = s.req_unit0[b + 1];
                it.part_row = tiles * kSpanRows + (s.req_item[b] - tiles) * p.heads;
                place(it, s.req_item[b], first);
            }
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
            p.tile_row[b] = g >= 0 && s.pages[g] > 0 && s.lens[b] > 0
                                ? s.tile0[g] * kSpanRows + (b - s.starts[g]) * p.heads
                                : -1;
            p.own_item[b] = s.req_unit0[b + 1] > s.req_unit0[b] ? s.req_item[b] : -1;
        }
}

}  // namespace mla
