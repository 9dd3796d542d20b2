// The merge of the pieces that mla_decode_shared and mla_decode_window leave
// (mla_span.cuh says what items and pieces are):
//
//   out = sum_p w_p o_p, w_p = exp(lse_p - lse), lse = log sum_p exp(lse_p)
//
// over the pieces of a row's one or two items. The pieces of an item lie a
// constant distance apart, so their loads do not wait for one another. A warp
// per row; where there are few rows, which then have many pieces, a CTA per
// row, its warps taking the pieces in turn. Bound by HBM (or L2, where the
// pieces still are): 2,052 bytes a piece's row and 1,028 a result's; with few
// rows by four dependent loads.
#include <cuda_runtime.h>

#include <cmath>

#include "mla_span.cuh"

namespace mla {
namespace {

constexpr int kMaxPieces = 2 * kMaxBalancedPairs;
// Eight warps a row, four, or one: a row's pieces are read one behind the other
// by each warp, so few rows (two, then eight, for each of 152 SMs: the merge's
// CTAs spread over the GPU, whatever number of SMs the plan is for) get more of
// them. 8 requests of 16 heads (128 rows) take 16.6 us a call with eight, 17.1 with
// four and 18.0 with one; 48 of 16 (768 rows, some 10 pieces each) 28.0 with four,
// 28.9 with eight, 30.7 with one; 128 of 128 (mostly one piece) 57 to 59 with one, 64
// with four, 71 with eight. (With four and eight the compiler spills 24 bytes, at 48
// registers a thread.)
constexpr int kMergeRows8 = 304, kMergeRows4 = 1216;

// The weight of a part with LSE `l` among parts whose greatest is m. (A NaN
// comes through; -inf has none.)
__device__ __forceinline__ float part_weight(float l, float m) {
    return l == -INFINITY ? 0.f : __expf(l - m);
}

// One row, by kWarps warps: 1, or all of a CTA's, which take its pieces in turn.
template <int kWarps>
__device__ __forceinline__ void merge_row(const SpanParams& p, int row, int lane, int sub,
                                          float* weight, float4 (*sums)[kLkv / 4]) {
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
        for (int c = 0; c < 4; ++c) sums[sub][32 * c + lane] = acc[c];
        __syncthreads();
        const int tid = threadIdx.x;
        if (tid < kLkv / 4) {                    // (128 threads or more)
            float4 s = sums[0][tid];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
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

// Warps of a CTA, and rows that they merge at once.
template <int kWarps>
constexpr int kCtaWarps = kWarps == 1 ? 8 : kWarps;

template <int kWarps>
__global__ void __launch_bounds__(32 * kCtaWarps<kWarps>)
mla_span_merge_kernel(const SpanParams p) {
    constexpr int kRows = kCtaWarps<kWarps> / kWarps;
    __shared__ float weights[kRows][kMaxPieces];
    __shared__ float4 sums[kWarps][kLkv / 4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * kRows + warp / kWarps;
    if (row < p.batch * p.heads)
        merge_row<kWarps>(p, row, lane, warp % kWarps, weights[warp / kWarps], sums);
}

template <int kWarps>
int launch(const SpanParams& p, void* stream) {
    constexpr int kRows = kCtaWarps<kWarps> / kWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((p.batch * p.heads + kRows - 1) / kRows), 1, 1);
    cfg.blockDim = dim3(32 * kCtaWarps<kWarps>, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return int(cudaLaunchKernelEx(&cfg, mla_span_merge_kernel<kWarps>, p));
}

}  // namespace

int launch_span_merge(const SpanParams& p, void* stream) {
    const int rows = p.batch * p.heads;
    return rows <= kMergeRows8 ? launch<8>(p, stream)
           : rows <= kMergeRows4 ? launch<4>(p, stream) : launch<1>(p, stream);
}

}  // namespace mla
