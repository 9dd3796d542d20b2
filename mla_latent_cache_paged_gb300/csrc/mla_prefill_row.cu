// Expanded-form latent attention for single query rows (one new token a
// sequence): the mathematics of mla_prefill.cu on the CUDA cores.
//
// With one query row a sequence every key and value of a head is used for 320
// multiply-adds, and the bound is HBM: 512 bytes a token and head (k_nope and
// v, side by side) and 128 a token for k_pe. The tensor kernel's 128-row tiles
// make a chain of score product, softmax and value product per 128 keys of
// that, about 1.6 us a step, on one CTA per SM.
//
// An item is one query row, one head and one split of its keys; a CTA works
// on it in groups of 8 lanes. A group takes every kGroups-th key, kKeys of them
// in flight: a lane reads 16 columns of k_nope and of v and 8 of k_pe, three
// shuffles sum a score over the group, and the group keeps its own running
// maximum, sum and 128-wide result (16 columns a lane). The groups are joined
// at the end, in the warp and then through shared memory; the splits of an
// item are the CTAs of a cluster and are joined in the first one's shared
// memory. Weights stay in fp32, and keys that a row does not see are not read.
//
// Measured with the keys in HBM (3 keys a group in flight: 128 registers, 512
// threads an SM; 2 and 4 keys were 6-17% slower where there are many items): 8
// sequences of 186 to 1,400 keys, 16 heads, 16.6 us (54 MB: 8.0 us at the
// measured HBM rate; the longest ones' chain of reads is what takes the time);
// 64 x 2,048 keys, 16 heads, 165 us (6.6 TB/s); 4 x 2,048 keys, 128 heads, 83 us
// (6.5 TB/s). Where there are fewer CTAs than the SMs hold, each has more
// threads: 8,000 keys, 16 heads, in 8 splits 30.3 us with 128 threads, 20.9 with
// 256 and 26.5 with 512 (clusters of 8 such CTAs do not all find room at once);
// 4,000 and 300 keys 17.7 and 13.8 with 128 and 256.
#include <cooperative_groups.h>

#include <cmath>
#include <cstdint>

#include "mla_prefill.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace {

constexpr int kSmThreads = 512;       // at 128 registers
constexpr int kKeys = 3;              // keys of a group in flight

// 8 bf16 values of 16 bytes.
__device__ __forceinline__ void widen8(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// What a part with maximum m and sum l is scaled by when it is joined to
// others with maximum `top`. (m = -inf: it saw no key, or only NaN scores,
// which must come through.)
__device__ __forceinline__ float join_factor(float m, float l, float top) {
    return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ptx::ex2(m - top);
}

// n parts of one column joined.
__device__ __forceinline__ void join(const float* m, const float* l, const float* o, int n,
                                     float* top, float* sum, float* x) {
    *top = -INFINITY;
    *sum = *x = 0.f;
    for (int i = 0; i < n; ++i) *top = fmaxf(*top, m[i]);
    for (int i = 0; i < n; ++i) {
        const float f = join_factor(m[i], l[i], *top);
        *sum = fmaf(f, l[i], *sum);
        *x = fmaf(f, o[i * kPrefillV], *x);
    }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, kSmThreads / kThreads)
prefill_row_kernel(const PrefillParams p) {
    constexpr int kWarps = kThreads / 32;
    constexpr int kGroups = kThreads / 8;
    __shared__ float part_m[kWarps], part_l[kWarps], part_o[kWarps][kPrefillV];
    // (read in the cluster's first CTA only)
    __shared__ float split_m[kMaxRowSplits], split_l[kMaxRowSplits];
    __shared__ float split_o[kMaxRowSplits][kPrefillV];
    auto cluster = cooperative_groups::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = threadIdx.x >> 3, part = threadIdx.x & 7;
    const int head = blockIdx.y, split = blockIdx.z;

    // The row's sequence: the last b with cu_q[b] <= row (every thread looks
    // for itself; empty sequences share their successor's start).
    const int row = blockIdx.x;
    int at = 0, end = p.batch;
    while (end - at > 1) {
        const int mid = (at + end) >> 1;
        if (__ldg(p.cu_q + mid) <= row) at = mid; else end = mid;
    }
    int q0, lq, k0, lk;
    sequence(p, at, &q0, &lq, &k0, &lk);
    if (row < q0 || row >= q0 + lq) return;
    // It sees keys 0..lk - lq + i (causal) or all; this split's are [lo, hi).
    const int keys = p.causal ? max(0, min(lk - lq + (row - q0) + 1, lk)) : lk;
    const int chunk = (keys + p.splits - 1) / p.splits;
    const int lo = min(keys, split * chunk), hi = min(keys, lo + chunk);

    // The row's query: this lane's 16 + 8 columns.
    float qn[16], qp[8];
    const uint4* q = reinterpret_cast<const uint4*>(
        p.q + (int64_t(row) * p.heads + head) * kPrefillQk);
    widen8(__ldg(q + 2 * part), qn);
    widen8(__ldg(q + 2 * part + 1), qn + 8);
    widen8(__ldg(q + 16 + part), qp);
    float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    for (int k = lo + group; k < hi; k += kGroups * kKeys) {
        uint4 kn[kKeys][2], kp[kKeys], v[kKeys][2];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int key = k + u * kGroups;
            if (key < hi) {
                const uint4* e = reinterpret_cast<const uint4*>(
                    p.kv + (int64_t(k0 + key) * p.heads + head) * kPrefillKv);
                kn[u][0] = __ldg(e + 2 * part);
                kn[u][1] = __ldg(e + 2 * part + 1);
                v[u][0] = __ldg(e + 16 + 2 * part);
                v[u][1] = __ldg(e + 16 + 2 * part + 1);
                kp[u] = __ldg(reinterpret_cast<const uint4*>(p.k_pe + int64_t(k0 + key) * kRope) +
                              part);
            }
        }
        float s[kKeys];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            s[u] = 0.f;
            if (k + u * kGroups < hi) {
                float a[16], b[8];
                widen8(kn[u][0], a);
                widen8(kn[u][1], a + 8);
                widen8(kp[u], b);
#pragma unroll
                for (int i = 0; i < 16; ++i) s[u] = fmaf(qn[i], a[i], s[u]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[u] = fmaf(qp[i], b[i], s[u]);
            }
        }
        // (the lanes of a group share its keys, so they come here together)
        const uint32_t mine = 0xffu << (lane & 24);
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) s[u] += __shfl_xor_sync(mine, s[u], d);
            s[u] = k + u * kGroups < hi ? s[u] * p.scale_log2 : -INFINITY;
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < kKeys; ++u) top = fmaxf(top, s[u]);
        // (nothing but -inf and NaN so far: the sums stay as they are)
        const float base = top == -INFINITY ? 0.f : top;
        const float alpha = m == -INFINITY ? 1.f : ptx::ex2(m - base);
        m = top;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] *= alpha;
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            if (k + u * kGroups < hi) {
                const float w = ptx::ex2(s[u] - base);
                l += w;
                float x[16];
                widen8(v[u][0], x);
                widen8(v[u][1], x + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = fmaf(w, x[i], o[i]);
            }
        }
    }
    __syncwarp();

    // The warp's four groups, then the warps, then the splits.
    float top = m;
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float f = join_factor(m, l, top);
    l *= f;
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        o[i] *= f;
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) o[i] += __shfl_xor_sync(0xffffffffu, o[i], d);
    }
    if (lane == 0) {
        part_m[warp] = top;
        part_l[warp] = l;
    }
    if (lane < 8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) part_o[warp][16 * part + i] = o[i];
    }
    // (the cluster's first CTA has begun before its shared memory is written)
    if (p.splits > 1) cluster.sync();
    else __syncthreads();
    const int col = threadIdx.x;
    float sum = 0.f, x = 0.f;
    if (col < kPrefillV) {
        join(part_m, part_l, &part_o[0][col], kWarps, &top, &sum, &x);
        if (p.splits > 1) {
            cluster.map_shared_rank(&split_o[0][0], 0)[split * kPrefillV + col] = x;
            if (col == 0) {
                cluster.map_shared_rank(split_m, 0)[split] = top;
                cluster.map_shared_rank(split_l, 0)[split] = sum;
            }
        }
    }
    if (p.splits > 1) {
        cluster.sync();
        if (split != 0) return;
        if (col < kPrefillV) join(split_m, split_l, &split_o[0][col], p.splits, &top, &sum, &x);
    }
    if (col < kPrefillV) {
        const int64_t out_row = int64_t(row) * p.heads + head;
        const float inv = sum != 0.f ? 1.f / sum : 0.f;   // (a NaN sum stays NaN)
        p.out[out_row * kPrefillV + col] = f32_to_bf16_bits_rn(x * inv);
        if (col == 0 && p.lse != nullptr)
            p.lse[out_row] = sum == 0.f ? -INFINITY : 0.693147180559945309f * top + logf(sum);
    }
}

}  // namespace

int launch_prefill_row(const PrefillParams& p, int num_sms, void* stream) {
    // As many threads a CTA as the SMs have room for (half of it with the
    // largest: a cluster's CTAs want SMs of one cluster region).
    const int64_t ctas = int64_t(p.total_q) * p.heads * p.splits;
    const int threads = 2 * ctas <= num_sms ? 512 : ctas <= 2 * int64_t(num_sms) ? 256 : 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.total_q), unsigned(p.heads), unsigned(p.splits));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = unsigned(p.splits);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return int(cudaLaunchKernelEx(&cfg,
                                  threads == 512   ? prefill_row_kernel<512>
                                  : threads == 256 ? prefill_row_kernel<256>
                                                   : prefill_row_kernel<128>,
                                  p));
}

}  // namespace mla
