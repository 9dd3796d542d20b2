// Rows of the latent cache, written and read back (mla_cache_write,
// mla_cache_gather and their fp8 forms, declared in include/mla_decode.h).
//
//   write:  entry slot_mapping[t] = [kv_c[t] | k_pe[t]], or its E4M3 codes
//           e4m3(x / k_scale)
//   gather: rows[t] = the entry of packed token t, or k_scale times its codes
//
// Both move a row as 72 pieces of 8 values, one per thread, so that a row's
// loads and stores are whole lines, with several rows in flight per thread.
// Bound by HBM for many rows: 65,536 rows take 24.3 us written in bf16 (151 MB,
// 6.2 TB/s), 18.6 us in fp8 (113 MB), 23.8 and 17.4 us gathered; by the launch
// and one load's latency (two in a gather: the table's first) for a step's few:
// 32 rows take 1.4 and 1.9 us a call, one behind the other in a graph.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "mla_device.cuh"

namespace mla {
namespace {

constexpr int kPieces = kD / 8;              // of 8 values
constexpr int kLatentPieces = kLkv / 8;
constexpr int kRowsAtOnce = 4;
constexpr int kThreads = kRowsAtOnce * kPieces;   // 288

// ------------------------------------------------------------------ write

struct WriteParams {
    const uint16_t* kv_c;        // rows kv_stride apart
    const uint16_t* k_pe;        // rows pe_stride apart
    int64_t kv_stride, pe_stride;
    const int64_t* slots;        // [T]
    int tokens;
    void* cache;
    int64_t num_slots;
    float down0, down1;          // fp8: x * down0 * down1 is about x / k_scale (code_scale)
    int32_t* status;
};

// The borders between two codes (where the next code begins, or a tie) have at
// most five significant bits, a bf16 value x has eight: x / k_scale can only lie
// on a border, or nearer to one than 2^-14 of it, if k_scale is that near to a
// ratio a / b with a < 256 and b < 32, times a power of two. Two such ratios are
// further apart than 2^-13, so there is one at most, and one answer for all the
// values that meet a border through it: above it, below it, or the tie itself.
// code_scale finds the ratio and makes a factor f = down0 * down1 of it,
//   1 / k_scale               if there is none
//   b / a * (1 - 2^-16)       if k_scale is above it: quotients just below a border
//   b / a * (1 + 2^-16)       if k_scale is below it
//   b / a * (1 + 2^-21)       if k_scale is the ratio: ties
// With it the fp32 product x * f, its last four bits cut off (at most 2^-19 of
// it; they hold the tie's 2^-21 and the product's rounding), has the code of the
// exact quotient for every x. A remainder taken for each value, with a rounding
// to odd, took 10.2 us for 16,384 rows.
__device__ __forceinline__ float quotient(float x, const WriteParams& p) {
    return __uint_as_float(__float_as_uint(x * p.down0 * p.down1) & ~15u);
}

// (down0 is a power of two and takes half of the exponent, so that both factors
// are normal numbers for every k_scale; x * down0 is exact unless the quotient
// is far above 448 or rounds to 0.)
void code_scale(float k_scale, WriteParams& p) {
    int e = 0;
    const double m = 2. * std::frexp(double(k_scale), &e);      // k_scale = m * 2^(e - 1)
    double f = 1. / m;
    for (int b = 1; b < 32; b += 2) {
        double v = m * b, power = 1.;        // (exact: 24 bits and 5)
        while (v < 128.) v *= 2., power *= 2.;
        const double a = std::nearbyint(v);
        if (std::fabs(v - a) >= a * 0x1p-14) continue;
        f = b * power / a * (v > a ? 1. - 0x1p-16 : v < a ? 1. + 0x1p-16 : 1. + 0x1p-21);
        break;
    }
    const int k = 1 - e, half = k / 2;
    p.down0 = float(std::ldexp(1., half));
    p.down1 = float(std::ldexp(f, k - half));
}

// Two quotients as E4M3 codes: to nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

template <bool kFp8, int kRounds>
__global__ void __launch_bounds__(kThreads) mla_cache_write_kernel(const WriteParams p) {
    const int c = threadIdx.x % kPieces;
    const int64_t t0 = int64_t(blockIdx.x) * (kRowsAtOnce * kRounds) + threadIdx.x / kPieces;
    uint4 v[kRounds];
    int64_t slot[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int64_t t = t0 + k * kRowsAtOnce;
        slot[k] = -1;
        if (t < p.tokens) {
            slot[k] = p.slots[t];
            const uint16_t* src = c < kLatentPieces
                                      ? p.kv_c + t * p.kv_stride + 8 * c
                                      : p.k_pe + t * p.pe_stride + 8 * (c - kLatentPieces);
            v[k] = __ldg(reinterpret_cast<const uint4*>(src));
        }
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (slot[k] < 0) continue;
        if (slot[k] >= p.num_slots) {
            if (c == 0) {
                const int64_t page = slot[k] / kPageSize;
                record_error(p.status, MLA_ERR_BAD_BLOCK_ID,
                             int32_t(page < INT_MAX ? page : INT_MAX));
            }
            continue;
        }
        if constexpr (kFp8) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = codes2(quotient(__uint_as_float(w[i] << 16), p),
                              quotient(__uint_as_float(w[i] & 0xffff0000u), p));
            *reinterpret_cast<uint2*>(static_cast<unsigned char*>(p.cache) + slot[k] * kD + 8 * c) =
                make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.cache) + slot[k] * kD + 8 * c) =
                v[k];
        }
    }
}

// ------------------------------------------------------------------ gather

struct GatherParams {
    const void* cache;
    int64_t num_blocks;
    const int32_t* table;        // [B, max_blocks]
    int max_blocks;
    const int32_t* first;        // [B] or null
    const int32_t* cu;           // [B + 1]
    int batch, total;
    float scale, power;          // fp8: a code's value * scale * power (gather_scale)
    uint16_t* rows;              // bf16 [total, 576]
    int32_t* status;
};

constexpr int64_t kNoRow = -2;   // the packed row belongs to no request
constexpr int64_t kNoPage = -1;  // its page is not there: zeros

// The cache slot of packed row t.
__device__ __forceinline__ int64_t find_slot(const GatherParams& p, int t) {
    // (the last row speaks for the sequences that the rows have no room for)
    if (t == p.total - 1 && p.cu[p.batch] > p.total)
        record_error(p.status, MLA_ERR_BAD_SEQ_LEN, p.cu[p.batch]);
    int lo = 0, hi = p.batch;       // the last b with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int begin = p.cu[lo], end = p.cu[lo + 1];
    if (begin < 0 || t < begin || t >= end) return kNoRow;
    const int64_t pos = int64_t(p.first != nullptr ? p.first[lo] : 0) + (t - begin);
    if (pos < 0 || pos >= int64_t(p.max_blocks) * kPageSize) {
        record_error(p.status, MLA_ERR_BAD_SEQ_LEN, int32_t(pos < INT_MAX ? pos : INT_MAX));
        return kNoPage;
    }
    const int page = p.table[int64_t(lo) * p.max_blocks + pos / kPageSize];
    if (page < 0 || int64_t(page) >= p.num_blocks) {
        record_error(p.status, MLA_ERR_BAD_BLOCK_ID, page);
        return kNoPage;
    }
    return int64_t(page) * kPageSize + pos % kPageSize;
}

// A code's value has four significant bits, k_scale 24: their product does not
// fit fp32, and rounded there it may become a tie between two bf16 numbers that
// it was next to. A tie has at most nine significant bits, so this takes a
// k_scale next to a ratio t / f with t <= 512 and f < 16, times a power of two.
// Two such ratios are further apart than 2^-13 of them (512 * 15 < 2^13), so
// k_scale is within 2^-15 of one at most, and all of its products that are that
// near to a tie lie on the same side of theirs: above, below, or on it. So
// gather_scale splits k_scale = scale * power, power = 2^k, and moves a scale
// that is within 2^-15 of a ratio, but not the ratio itself, to 2^-14 beyond it
// on its side, which takes no product past a tie. A product is then a tie (in
// fp32 too) or at least 2^-15 of it away from one, and neither its rounding to
// fp32 (2^-24) nor, for a result below 2^-126, that of its product with the
// power (2^-150, where the least tie is 2^-134) brings it there: the rounding to
// bf16 is that of the exact product.
void gather_scale(float k_scale, GatherParams& p) {
    int e = 0;
    double m = 2. * std::frexp(double(k_scale), &e);      // k_scale = m * 2^(e - 1)
    for (int f = 1; f < 16; f += 2) {
        double v = m * f, power = 1.;        // (exact: 24 bits and 4)
        while (v < 256.) v *= 2., power *= 2.;
        const double t = std::nearbyint(v);
        if (std::fabs(v - t) >= t * 0x1p-15) continue;
        if (v != t) m = t / (f * power) * (v > t ? 1. + 0x1p-14 : 1. - 0x1p-14);
        break;
    }
    p.scale = float(m);
    p.power = float(std::ldexp(1., e - 1));
}

// Two codes times k_scale as bf16, rounded once.
__device__ __forceinline__ uint32_t scaled2(uint32_t codes16, const GatherParams& p) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes16), __NV_E4M3);
    const float2 f = __fmul2_rn(
        __fmul2_rn(__half22float2(__half2(h)), make_float2(p.scale, p.scale)),
        make_float2(p.power, p.power));
    return pack_bf16(f.x, f.y);
}

template <bool kFp8, int kRounds>
__global__ void __launch_bounds__(kThreads) mla_cache_gather_kernel(const GatherParams p) {
    constexpr int kRows = kRowsAtOnce * kRounds;
    __shared__ int64_t slots[kRows];
    const int64_t t0 = int64_t(blockIdx.x) * kRows;
    if (threadIdx.x < kRows) {
        const int64_t t = t0 + threadIdx.x;
        slots[threadIdx.x] = t < p.total ? find_slot(p, int(t)) : kNoRow;
    }
    __syncthreads();
    const int c = threadIdx.x % kPieces, r = threadIdx.x / kPieces;
    uint4 v[kRounds];
    int64_t slot[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        slot[k] = slots[r + k * kRowsAtOnce];
        v[k] = make_uint4(0, 0, 0, 0);
        if (slot[k] < 0) continue;
        if constexpr (kFp8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(
                static_cast<const unsigned char*>(p.cache) + slot[k] * kD + 8 * c));
            v[k].x = u.x;
            v[k].y = u.y;
        } else {
            v[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.cache) +
                                                        slot[k] * kD + 8 * c));
        }
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (slot[k] == kNoRow) continue;
        if constexpr (kFp8)
            v[k] = make_uint4(scaled2(v[k].x & 0xffffu, p), scaled2(v[k].x >> 16, p),
                              scaled2(v[k].y & 0xffffu, p), scaled2(v[k].y >> 16, p));
        *reinterpret_cast<uint4*>(p.rows + (t0 + r + k * kRowsAtOnce) * kD + 8 * c) = v[k];
    }
}

// Rows per thread: one while the rows are few, where every SM's share of them
// counts (32 rows written: 1.4 us against 1.9 with four), and four beyond, where
// loads in flight count (65,536 rows written in bf16: 24.3 us against 26.9 with
// one; gathered from fp8: 17.4 against 27.1). At 4,096 rows they meet (written
// 2.4 and 2.6, gathered 2.9 and 2.8). Two and eight are between or worse.
constexpr int kFewRounds = 1, kManyRounds = 4;
constexpr int kFewRows = 4096;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <bool kFp8>
int write(WriteParams p, float k_scale, int64_t num_blocks, void* workspace,
          size_t workspace_bytes, void* stream) {
    if (p.tokens < 0 || num_blocks < 1 || p.kv_stride < 0 || p.pe_stride < 0 ||
        p.kv_stride % 8 != 0 || p.pe_stride % 8 != 0)
        return MLA_ERR_INVALID_ARG;
    if (kFp8 && (!std::isfinite(k_scale) || !(k_scale > 0.f))) return MLA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kStatusBytes || !aligned(workspace, 256))
        return MLA_ERR_WORKSPACE;
    if (num_blocks > INT64_MAX / (kPageSize * kD * 2)) return MLA_ERR_UNSUPPORTED;
    if (p.tokens == 0) return MLA_OK;
    if (!p.kv_c || !p.k_pe || !p.slots || !p.cache) return MLA_ERR_INVALID_ARG;
    if (!aligned(p.kv_c, 16) || !aligned(p.k_pe, 16) || !aligned(p.slots, 8) ||
        !aligned(p.cache, 16))
        return MLA_ERR_INVALID_ARG;
    p.num_slots = num_blocks * kPageSize;
    p.status = static_cast<int32_t*>(workspace);
    if (kFp8) code_scale(k_scale, p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rounds = p.tokens <= kFewRows ? kFewRounds : kManyRounds;
    const int per_cta = kRowsAtOnce * rounds;
    const unsigned grid = unsigned((int64_t(p.tokens) + per_cta - 1) / per_cta);
    if (rounds == kFewRounds)
        mla_cache_write_kernel<kFp8, kFewRounds><<<grid, kThreads, 0, st>>>(p);
    else
        mla_cache_write_kernel<kFp8, kManyRounds><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

template <bool kFp8>
int gather(GatherParams p, float k_scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (p.batch < 0 || p.total < 0 || p.num_blocks < 1 || p.max_blocks < 1)
        return MLA_ERR_INVALID_ARG;
    if (kFp8 && (!std::isfinite(k_scale) || !(k_scale > 0.f))) return MLA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kStatusBytes || !aligned(workspace, 256))
        return MLA_ERR_WORKSPACE;
    if (p.batch == 0 || p.total == 0) return MLA_OK;
    if (!p.cache || !p.table || !p.cu || !p.rows) return MLA_ERR_INVALID_ARG;
    if (!aligned(p.cache, 16) || !aligned(p.rows, 16) || !aligned(p.table, 4) ||
        !aligned(p.cu, 4) || (p.first && !aligned(p.first, 4)))
        return MLA_ERR_INVALID_ARG;
    p.status = static_cast<int32_t*>(workspace);
    if (kFp8) gather_scale(k_scale, p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rounds = p.total <= kFewRows ? kFewRounds : kManyRounds;
    const int per_cta = kRowsAtOnce * rounds;
    const unsigned grid = unsigned((int64_t(p.total) + per_cta - 1) / per_cta);
    if (rounds == kFewRounds)
        mla_cache_gather_kernel<kFp8, kFewRounds><<<grid, kThreads, 0, st>>>(p);
    else
        mla_cache_gather_kernel<kFp8, kManyRounds><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

WriteParams write_params(const void* kv_c, int64_t kv_stride, const void* k_pe, int64_t pe_stride,
                         const int64_t* slots, int tokens, void* cache) {
    WriteParams p{};
    p.kv_c = static_cast<const uint16_t*>(kv_c);
    p.k_pe = static_cast<const uint16_t*>(k_pe);
    p.kv_stride = kv_stride;
    p.pe_stride = pe_stride;
    p.slots = slots;
    p.tokens = tokens;
    p.cache = cache;
    return p;
}

GatherParams gather_params(const void* cache, int64_t num_blocks, const int32_t* table,
                           int max_blocks, const int32_t* first, const int32_t* cu, int batch,
                           int total, void* rows) {
    GatherParams p{};
    p.cache = cache;
    p.num_blocks = num_blocks;
    p.table = table;
    p.max_blocks = max_blocks;
    p.first = first;
    p.cu = cu;
    p.batch = batch;
    p.total = total;
    p.rows = static_cast<uint16_t*>(rows);
    return p;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_cache_write(const void* kv_c, int64_t kv_c_stride, const void* k_pe,
                               int64_t k_pe_stride, const int64_t* slot_mapping, int num_tokens,
                               void* latent_cache, int64_t num_blocks, void* workspace,
                               size_t workspace_bytes, void* stream) {
    return write<false>(write_params(kv_c, kv_c_stride, k_pe, k_pe_stride, slot_mapping, num_tokens,
                                     latent_cache), 1.f, num_blocks, workspace, workspace_bytes,
                        stream);
}

extern "C" int mla_cache_write_fp8(const void* kv_c, int64_t kv_c_stride, const void* k_pe,
                                   int64_t k_pe_stride, const int64_t* slot_mapping,
                                   int num_tokens, float k_scale, void* latent_cache_fp8,
                                   int64_t num_blocks, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    return write<true>(write_params(kv_c, kv_c_stride, k_pe, k_pe_stride, slot_mapping, num_tokens,
                                    latent_cache_fp8), k_scale, num_blocks, workspace,
                       workspace_bytes, stream);
}

extern "C" int mla_cache_gather(const void* latent_cache, int64_t num_blocks,
                                const int32_t* block_table, int max_blocks_per_seq,
                                const int32_t* first_token, const int32_t* cu_seqlens_k, int batch,
                                int total_k, void* rows, void* workspace, size_t workspace_bytes,
                                void* stream) {
    return gather<false>(gather_params(latent_cache, num_blocks, block_table, max_blocks_per_seq,
                                       first_token, cu_seqlens_k, batch, total_k, rows),
                         1.f, workspace, workspace_bytes, stream);
}

extern "C" int mla_cache_gather_fp8(const void* latent_cache_fp8, float k_scale,
                                    int64_t num_blocks, const int32_t* block_table,
                                    int max_blocks_per_seq, const int32_t* first_token,
                                    const int32_t* cu_seqlens_k, int batch, int total_k,
                                    void* rows, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    return gather<true>(gather_params(latent_cache_fp8, num_blocks, block_table,
                                      max_blocks_per_seq, first_token, cu_seqlens_k, batch,
                                      total_k, rows),
                        k_scale, workspace, workspace_bytes, stream);
}
