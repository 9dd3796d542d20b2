// The schedule of mla_decode_shared and mla_decode_window, and the merge of
// their pieces (mla_span.cuh says what items, units and pieces are).
//
// Schedule: one CTA, from the lengths on the device, so that a captured call
// can be replayed with other lengths. A request's group is found by a search
// in the starts; the prefix that a group shares is cut to its shortest member
// (rows of a tile then all see the same tokens); a block-wide scan numbers the
// items and their units. Bound by the latency of a few dependent loads and
// barriers: it is launched ahead of the attention kernel, whose set-up runs
// meanwhile.
//
// Merge: out = sum_p w_p o_p with w_p = exp(lse_p - lse), lse the log of the
// sum of exp(lse_p), over the pieces of a row's one or two items. The pieces of
// an item lie a constant distance apart, so their loads do not wait for one
// another. A warp per row; where there are few rows, which then have many
// pieces, a CTA per row, its warps taking the pieces in turn.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "mla_span.cuh"
#include "tensor_map.cuh"

namespace mla {
namespace {

constexpr int kScheduleThreads = 1024;

// Exclusive prefix sum over the CTA's threads; *total: the sum.
__device__ __forceinline__ uint64_t scan_exclusive(uint64_t v, uint64_t* warps, uint64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const uint64_t w = warps[lane];
        uint64_t s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t n = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += n;
        }
        warps[lane] = s;
    }
    __syncthreads();
    *total = warps[31];
    return (warp > 0 ? warps[warp - 1] : 0) + incl - v;
}

// A number of items (high 20 bits) and of units, added together.
constexpr int kUnitBits = 44;
__device__ __forceinline__ uint64_t packed(int items, int64_t units) {
    return (uint64_t(items) << kUnitBits) | uint64_t(units);
}
__device__ __forceinline__ int items_of(uint64_t v) { return int(v >> kUnitBits); }
__device__ __forceinline__ int64_t units_of(uint64_t v) {
    return int64_t(v & ((uint64_t(1) << kUnitBits) - 1));
}

__device__ __forceinline__ int span_steps(int pages) {
    return (pages + kSpanStepPages - 1) / kSpanStepPages;
}

__device__ __forceinline__ int span_length(const SpanParams& p, int b, bool record) {
    const int L = p.seq_lens[b];
    if (L < 0 || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
        if (record) record_error(p.status, MLA_ERR_BAD_SEQ_LEN, L);
        return 0;
    }
    return L;
}

__global__ void __launch_bounds__(kScheduleThreads) mla_span_schedule_kernel(const SpanParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ int64_t group_smem[];
    __shared__ uint64_t warps[32];
    __shared__ int64_t cuts[kMaxBalancedPairs + 1], edges[kMaxBalancedPairs + 1];
    const int tid = threadIdx.x;
    int G = p.groups;
    int64_t* unit0 = group_smem;                 // the group's first unit
    int32_t* starts = reinterpret_cast<int32_t*>(unit0 + G);
    int32_t* pages = starts + G + 1;             // the shortest member's length, then the prefix's pages
    int32_t* tile0 = pages + G;                  // the group's first tile, or -1
    int32_t* leader = tile0 + G;                 // its first member with tokens

    // Groups, if their starts make sense: not decreasing, within the batch.
    bool bad = false;
    for (int g = tid; G > 0 && g <= G; g += kScheduleThreads) {
        const int a = p.group_starts[g];
        starts[g] = a;
        bad = bad || a < 0 || a > p.batch || (g > 0 && p.group_starts[g - 1] > a);
        if (g < G) pages[g] = leader[g] = INT_MAX;
    }
    if (__syncthreads_or(bad ? 1 : 0)) {
        if (tid == 0) record_error(p.status, MLA_ERR_BAD_ROW, 0);
        G = 0;
    }
    // The group of a request: the last one that starts at it or before and
    // does not end before it.
    auto group_of = [&](int b) {
        int lo = 0, hi = G;                      // the first group that ends behind b
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid + 1] > b) hi = mid; else lo = mid + 1;
        }
        return lo < G && starts[lo] <= b ? lo : -1;
    };
    for (int b = tid; G > 0 && b < p.batch; b += kScheduleThreads) {
        const int g = group_of(b);
        const int L = span_length(p, b, false);
        if (g >= 0 && L > 0) {
            atomicMin(&pages[g], L);
            atomicMin(&leader[g], b);
        }
    }
    __syncthreads();

    // The prefixes and their tiles.
    uint64_t done = 0, total;                    // items and units so far
    for (int g0 = 0; g0 < G; g0 += kScheduleThreads) {
        const int g = g0 + tid;
        int n = 0, steps = 0;
        if (g < G) {
            const int members = starts[g + 1] - starts[g];
            int S = p.shared_lens[g];
            if (S < 0 || int64_t(S) > int64_t(p.max_blocks) * kPageSize) {
                record_error(p.status, MLA_ERR_BAD_SEQ_LEN, S);
                S = 0;
            }
            const int shortest = pages[g] == INT_MAX ? 0 : pages[g];
            const int pg = (S < shortest ? S : shortest) / kPageSize;
            const int tiles = int((int64_t(members) * p.heads + kSpanRows - 1) / kSpanRows);
            steps = span_steps(pg);
            // Worth it where a tile holds the rows of several requests: the
            // steps that this saves against the tiles' fixed cost.
            n = int64_t(members - tiles) * steps > int64_t(tiles) * kSpanItemCost ? tiles : 0;
            pages[g] = n > 0 ? pg : 0;
        }
        const int64_t units = int64_t(n) * (kSpanItemCost + steps);
        const uint64_t at = done + scan_exclusive(packed(n, units), warps, &total);
        done += total;
        if (g < G) {
            tile0[g] = n > 0 ? items_of(at) : -1;
            unit0[g] = units_of(at);
        }
    }
    const int tiles = items_of(done);
    __syncthreads();

    // The requests' own items.
    for (int b0 = 0; b0 < p.batch; b0 += kScheduleThreads) {
        const int b = b0 + tid;
        SpanItem it{};
        if (b < p.batch) {
            const int L = span_length(p, b, true);
            const int g = G > 0 ? group_of(b) : -1;
            const bool tiled = g >= 0 && tile0[g] >= 0;
            const bool shares = tiled && L > 0;
            const int held = pages_of(L);
            p.tile_row[b] = shares ? tile0[g] * kSpanRows + (b - starts[g]) * p.heads : -1;
            if (tiled) {
                // The tile whose first row is one of this request's.
                const int r0 = (b - starts[g]) * p.heads;
                const int k = (r0 + kSpanRows - 1) / kSpanRows;
                if (k * kSpanRows < r0 + p.heads) {
                    const int steps = span_steps(pages[g]);
                    SpanItem t{};
                    t.unit0 = unit0[g] + int64_t(k) * (kSpanItemCost + steps);
                    t.unit1 = t.unit0 + kSpanItemCost + steps;
                    t.row0 = starts[g] * p.heads + k * kSpanRows;
                    t.rows = min(kSpanRows, starts[g + 1] * p.heads - t.row0);
                    t.table_row = leader[g];
                    t.pages = pages[g];
                    t.end = pages[g] * kPageSize;
                    t.part_row = (tile0[g] + k) * kSpanRows;
                    p.items[tile0[g] + k] = t;
                }
            }
            it.row0 = b * p.heads;
            it.rows = p.heads;
            it.table_row = b;
            it.end = L;
            it.alone = shares ? 0 : 1;
            if (shares) {
                it.page_shift = pages[g];
                it.pages = held - pages[g];
            } else if (p.window > 0) {
                const int lo = L > p.window ? L - p.window : 0;
                const int head = int((int64_t(p.sinks) + kPageSize - 1) / kPageSize);
                it.sink_end = p.sinks;
                it.tail_lo = lo;
                if (lo / kPageSize > head) {
                    it.head_pages = head;
                    it.page_shift = lo / kPageSize - head;
                }
                it.pages = held - it.page_shift;
            } else {
                it.pages = held;
            }
        }
        const int steps = span_steps(it.pages);
        const int n = steps > 0 ? 1 : 0;
        const int units = n * (kSpanItemCost + steps);
        const uint64_t at = done + scan_exclusive(packed(n, units), warps, &total);
        done += total;
        if (b < p.batch) {
            p.own_item[b] = n > 0 ? items_of(at) : -1;
            if (n > 0) {
                it.unit0 = units_of(at);
                it.unit1 = it.unit0 + units;
                it.part_row = tiles * kSpanRows + (items_of(at) - tiles) * p.heads;
                p.items[items_of(at)] = it;
            }
        }
    }
    // The cuts between the pairs' ranges: equal ones, moved to an item's edge
    // where that is near, or all of them if that costs no pair much.
    const int items = items_of(done);
    const int64_t T = units_of(done);
    const int C = int(T < p.pairs ? T : p.pairs);
    __syncthreads();
    for (int i = tid; i < items; i += kScheduleThreads) {
        const int64_t u0 = p.items[i].unit0, u1 = p.items[i].unit1;
        for (int64_t c = (u0 * C + T - 1) / T; c < C && pair_begin(int(c), C, T) < u1; ++c) {
            const int64_t g = pair_begin(int(c), C, T);
            const int64_t edge = g - u0 <= u1 - g ? u0 : u1;
            cuts[c] = g;
            edges[c] = edge;
        }
    }
    if (tid == 0) cuts[C] = edges[C] = T;
    __syncthreads();
    if (tid < 32 && C > 0) {
        int64_t most = 0;
        for (int c = tid; c < C; c += 32) most = max(most, edges[c + 1] - edges[c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        const bool whole = most <= (T + C - 1) / C + kSpanCutCost;
        for (int c = tid; c < C; c += 32) {
            const int64_t d = edges[c] - cuts[c];
            if (whole || (d <= kSpanSnap && d >= -kSpanSnap)) cuts[c] = edges[c];
        }
    }
    if (tid == 0) *p.header = SpanHeader{T, C, items};
    __syncthreads();
    // The pairs that work on each item, and the item that each pair begins
    // with: the one that holds its first unit.
    for (int i = tid; i < items; i += kScheduleThreads) {
        const int64_t u0 = p.items[i].unit0, u1 = p.items[i].unit1;
        auto pair_of = [&](int64_t u) {          // the last pair that begins at u or before
            int lo = 0, hi = C;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cuts[mid] <= u) lo = mid; else hi = mid;
            }
            return lo;
        };
        const int c0 = pair_of(u0 + kSpanItemCost), c1 = pair_of(u1 - 1);
        p.items[i].first_pair = int16_t(c0);
        p.items[i].last_pair = int16_t(c1);
        for (int c = pair_of(u0); c <= c1; ++c)
            if (cuts[c] >= u0) p.pair_item[c] = i;
    }
    for (int c = tid; c <= C; c += kScheduleThreads) p.cuts[c] = cuts[c];
}

// ------------------------------------------------------------------ merge

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMaxPieces = 2 * kMaxBalancedPairs;
constexpr int kMergeFewRows = 1024;

// The weight of a part with LSE `l` among parts whose greatest is m. (A NaN
// comes through; -inf has none.)
__device__ __forceinline__ float part_weight(float l, float m) {
    return l == -INFINITY ? 0.f : __expf(l - m);
}

// kWarps warps per row: 1, or all of a CTA's, which take its pieces in turn.
template <int kWarps>
__global__ void __launch_bounds__(kMergeThreads) mla_span_merge_kernel(const SpanParams p) {
    __shared__ float weights[kMergeWarps / kWarps][kMaxPieces];
    __shared__ float4 sums[kWarps > 1 ? kMergeWarps : 1][kLkv / 4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * (kMergeWarps / kWarps) + warp / kWarps;
    const int sub = warp % kWarps;
    if (row >= p.batch * p.heads) return;
    const int b = row / p.heads, h = row - b * p.heads;
    const int tr = p.tile_row[b], own = p.own_item[b];
    // The pieces of the row's one or two items: n[k] of them, 128 rows apart.
    int64_t at[2] = {0, 0};
    int n[2] = {0, 0};
    if (own >= 0) {
        const SpanItem it = p.items[own];
        if (it.alone && it.first_pair == it.last_pair) return;    // its results are written
        at[0] = int64_t(it.part_row) + h + int64_t(it.first_pair) * kSpanRows;
        n[0] = it.last_pair - it.first_pair + 1;
    }
    if (tr >= 0) {
        const SpanItem it = p.items[(tr + h) / kSpanRows];
        at[1] = int64_t(it.part_row) + (tr + h) % kSpanRows + int64_t(it.first_pair) * kSpanRows;
        n[1] = it.last_pair - it.first_pair + 1;
    }
    const int pieces = n[0] + n[1];
    float* weight = weights[warp / kWarps];
    float m = -INFINITY;
    for (int i = lane; i < pieces; i += 32) {
        const float l = i < n[0] ? p.lse_part[at[0] + int64_t(i) * kSpanRows]
                                 : p.lse_part[at[1] + int64_t(i - n[0]) * kSpanRows];
        if (sub == 0) weight[i] = l;
        m = fmaxf(m, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (kWarps > 1) __syncthreads(); else __syncwarp();
    float z = 0.f;
    for (int i = lane; i < pieces; i += 32) z += part_weight(weight[i], m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);

    // 512 columns: a lane has four of each 128.
    float4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int begin = (sub + kWarps - (k == 0 ? 0 : n[0] % kWarps)) % kWarps;
        const float* src = p.o_part + at[k] * kLkv + 4 * lane;
#pragma unroll 2
        for (int i = begin; i < n[k]; i += kWarps) {
            const float w = part_weight(weight[(k == 0 ? 0 : n[0]) + i], m);
            const float* piece = src + int64_t(i) * kSpanRows * kLkv;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(piece + 128 * c);
                acc[c].x += w * v.x;
                acc[c].y += w * v.y;
                acc[c].z += w * v.z;
                acc[c].w += w * v.w;
            }
        }
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
    uint16_t* out = p.out + int64_t(row) * kLkv;
    if constexpr (kWarps == 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint2*>(out + 128 * c + 4 * lane) =
                make_uint2(pack_bf16(acc[c].x * inv, acc[c].y * inv),
                           pack_bf16(acc[c].z * inv, acc[c].w * inv));
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) sums[warp][32 * c + lane] = acc[c];
        __syncthreads();
        const int tid = threadIdx.x;
        if (tid < kLkv / 4) {
            float4 s = sums[0][tid];
#pragma unroll
            for (int w = 1; w < kMergeWarps; ++w) {
                const float4 v = sums[w][tid];
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            *reinterpret_cast<uint2*>(out + 4 * tid) =
                make_uint2(pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv));
        }
    }
    if (sub == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = z == 0.f ? -INFINITY : m + logf(z);
}

}  // namespace

int launch_span_schedule(const SpanParams& p, void* stream) {
    const auto bytes = [](int groups) { return groups * 24 + 4; };
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared_memory(mla_span_schedule_kernel,
                                              bytes(kSpanMaxBatch), &allowed);
    if (e != cudaSuccess) return int(e);
    mla_span_schedule_kernel<<<1, kScheduleThreads, bytes(p.groups), static_cast<cudaStream_t>(stream)>>>(p);
    return int(cudaGetLastError());
}

int launch_span_merge(const SpanParams& p, void* stream) {
    const int rows = p.batch * p.heads;
    const bool few = rows <= kMergeFewRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(few ? rows : (rows + kMergeWarps - 1) / kMergeWarps), 1, 1);
    cfg.blockDim = dim3(kMergeThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return int(cudaLaunchKernelEx(&cfg, few ? mla_span_merge_kernel<kMergeWarps>
                                            : mla_span_merge_kernel<1>, p));
}

}  // namespace mla
