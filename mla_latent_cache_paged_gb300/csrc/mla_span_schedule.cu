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
// sum of exp(lse_p), over the pieces of a row's one or two items. One CTA per
// row, a thread per four columns: the pieces of an item lie a constant
// distance apart, so their loads do not wait for one another.
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
    const int items = items_of(done);
    const int64_t T = units_of(done);
    const int C = int(T < p.pairs ? T : p.pairs);
    if (tid == 0) *p.header = SpanHeader{T, C, items};
    __syncthreads();
    // The item that holds each pair's first unit.
    for (int i = tid; i < items; i += kScheduleThreads) {
        const int64_t u0 = p.items[i].unit0, u1 = p.items[i].unit1;
        for (int64_t c = (u0 * C + T - 1) / T; c < C && pair_begin(int(c), C, T) < u1; ++c)
            p.pair_item[c] = i;
    }
}

// ------------------------------------------------------------------ merge

constexpr int kMergeThreads = 128;           // 4 columns each
constexpr int kMaxPieces = 2 * kMaxBalancedPairs;

// The weight of a part with LSE `l` among parts whose greatest is m. (A NaN
// comes through; -inf has none.)
__device__ __forceinline__ float part_weight(float l, float m) {
    return l == -INFINITY ? 0.f : __expf(l - m);
}

__global__ void __launch_bounds__(kMergeThreads) mla_span_merge_kernel(const SpanParams p) {
    __shared__ float weight[kMaxPieces];
    __shared__ float red[2 * kMergeThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = blockIdx.x, tid = threadIdx.x;
    const int b = row / p.heads, h = row - b * p.heads;
    const SpanHeader head = *p.header;
    const int tr = p.tile_row[b], own = p.own_item[b];
    const float* part[2] = {nullptr, nullptr};     // first piece's row of each item
    const float* lses[2] = {nullptr, nullptr};
    int n[2] = {0, 0};
    auto add = [&](int k, int item, int r) {
        const SpanItem it = p.items[item];
        int c0, c1;
        span_pairs(it, head, &c0, &c1);
        if (it.alone && c0 == c1) return false;    // its results are written
        const int64_t at = int64_t(it.part_row) + r + int64_t(c0) * kSpanRows;
        part[k] = p.o_part + at * kLkv;
        lses[k] = p.lse_part + at;
        n[k] = c1 - c0 + 1;
        return true;
    };
    if (own >= 0 && !add(0, own, h)) return;
    if (tr >= 0) add(1, (tr + h) / kSpanRows, (tr + h) % kSpanRows);

    const int pieces = n[0] + n[1];
    auto lse_at = [&](int i) {
        return i < n[0] ? lses[0][int64_t(i) * kSpanRows] : lses[1][int64_t(i - n[0]) * kSpanRows];
    };
    float m = -INFINITY;
    for (int i = tid; i < pieces; i += kMergeThreads) {
        const float l = lse_at(i);
        weight[i] = l;
        m = fmaxf(m, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float z = 0.f;
    for (int i = tid; i < pieces; i += kMergeThreads) {
        weight[i] = part_weight(weight[i], m);
        z += weight[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if ((tid & 31) == 0) red[4 + (tid >> 5)] = z;
    __syncthreads();
    z = (red[4] + red[5]) + (red[6] + red[7]);

    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    int w0 = 0;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const float* src = part[k] + 4 * tid;
#pragma unroll 4
        for (int i = 0; i < n[k]; ++i) {
            const float w = weight[w0 + i];
            const float4 v = *reinterpret_cast<const float4*>(src + int64_t(i) * kSpanRows * kLkv);
            acc.x += w * v.x;
            acc.y += w * v.y;
            acc.z += w * v.z;
            acc.w += w * v.w;
        }
        w0 += n[k];
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
    uint2 o;
    o.x = pack_bf16(acc.x * inv, acc.y * inv);
    o.y = pack_bf16(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(p.out + int64_t(row) * kLkv + 4 * tid) = o;
    if (tid == 0 && p.lse != nullptr) p.lse[row] = z == 0.f ? -INFINITY : m + logf(z);
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.batch) * unsigned(p.heads), 1, 1);
    cfg.blockDim = dim3(kMergeThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return int(cudaLaunchKernelEx(&cfg, mla_span_merge_kernel, p));
}

}  // namespace mla
