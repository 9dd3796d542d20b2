// Expansion of paged latent rows into per-head keys and values
// (mla_expand_kv, mla_expand_kv_fp8): what lies between the latent cache and
// the attention in its expanded form.
//
//   kv[t, n, 0:128]   = c_t . W_UK_T[n]^T     W_UK_T bf16 [N, 128, 512]
//   kv[t, n, 128:256] = c_t . W_UV[n]         W_UV   bf16 [N, 512, 128]
//   k_pe[t, 0:64]     = the entry's last 64 columns
// where c_t is the 512-wide latent part of packed token t's cache entry, read
// through the block table. The weights are the ones the decode's front end
// and up-projection use, in their layouts: W_UK_T tiles are K-major operands
// and W_UV tiles MN-major ones, so neither is laid out a second time.
//
// A matrix product with T rows, N * 256 columns and K = 512. Its bound at
// N = 128 is the tensor pipe (2 * 512 flops per output element against 2
// bytes written). A CTA works on 256 tokens and walks the (head, half) column
// tiles of 128: a weight tile streamed from L2 then serves 256 rows, 32 bytes
// per clock per SM at the tensor pipe's full rate (with 128 rows it would be
// 64). Both halves of the 256 x 512 latent tile stay on chip for all of a
// CTA's columns: rows 0..127 as the A operand in TMEM (256 columns of bf16
// pairs), rows 128..255 in shared memory (128 KB), which leaves 96 KB for the
// ring of weight chunks (6 x 128 columns x 64 k) and 2 x 128 TMEM columns for
// the two accumulators. The accumulators are single; the second half's MMAs
// run kSkew chunks behind the first's, so one accumulator is read out while
// the tensor pipe works on the other.
//
// What bounds it now: the shared-memory pipe. Per weight chunk and 256 rows the
// MMAs read 48 KB (the chunk twice, the second half's rows once) and the loads
// write 16 KB, 512 clocks at 128 bytes a clock and as many as the MMAs take;
// the result's stores pass through the same pipe. 7,865 tokens, N = 128: 204 us
// (1,290 TFLOP/s, 2.5 TB/s written), 165 us with the stores left out; 500
// tokens, N = 16: 14 us (bf16 cache), 15 us (fp8).
//
// Work: the (token tile, head, half) items in that order, cut into one
// contiguous range per CTA, so each CTA gathers one or two token tiles.
// Warps: 0 = weight loads (TMA), 1 = MMAs, 2-5 and 6-9 = gather and epilogue
// of the first and second 128 rows (thread = row = TMEM lane). Every wait is
// bounded (MLA_ERR_TIMEOUT).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "mla_device.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"

namespace mla {
namespace {

constexpr int kThreads = 320;
constexpr int kRows = 256;                    // tokens per CTA tile
constexpr int kChunk = 64;                    // K per ring stage
constexpr int kChunks = kLkv / kChunk;        // 8 per column tile
constexpr int kStages = 6;
constexpr int kSkew = 2;                      // chunks the second half runs behind
constexpr int kStageBytes = 128 * kChunk * 2; // 16 KB
constexpr int kHalf = 128;                    // columns of a tile: k_nope or v of one head
constexpr int kOffA = 0;                      // second half's rows: 8 x [128 x 64] bf16, SW128
constexpr int kOffRing = kChunks * 16384;
constexpr int kOffBar = kOffRing + kStages * kStageBytes;
constexpr int kSmemBytes = kOffBar + 256;     // base is 1 KB aligned
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
constexpr uint32_t kTmemA = 0;                // 256 columns: first half's rows, bf16 pairs
constexpr uint32_t kTmemAcc = 256;            // 2 x 128 fp32 columns
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr uint32_t kSuspendNs = 20000;

enum ExpandSite : int32_t { kSiteEmpty = 50, kSiteFull, kSiteA, kSiteAccEmpty, kSiteAccFull,
                            kSiteDrain };

struct Bars {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t a_ready[2];      // 128 arrivals: this half's rows are staged
    uint64_t acc_full[2];
    uint64_t acc_empty[2];    // 4 warps: accumulator read out
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct ExpandParams {
    const void* cache;              // bf16 or E4M3 [num_blocks, 64, 576]
    int64_t num_blocks;
    const int32_t* table;           // [B, max_blocks]
    int max_blocks;
    const int32_t* first;           // [B] or null
    const int32_t* cu;              // [B + 1]
    int batch, heads;
    int total;                      // packed rows of kv
    uint16_t* kv;                   // bf16 [total, N, 256]
    uint16_t* k_pe;                 // bf16 [total, 64]
    float scale;                    // 1, or the fp8 cache's
    int64_t items;                  // token tiles * N * 2
    int32_t* status;
};

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Bars* bars, int32_t* status,
                                     int32_t site, bool ignore_abort = false) {
    if (ptx::mbar_test_wait(bar, parity)) return true;
    volatile int32_t* abort = &bars->abort;
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        for (int i = 0; i < 4; ++i)
            if (ptx::mbar_try_wait_sleep(bar, parity, kSuspendNs)) return true;
        if (!ignore_abort && *abort != 0) return false;
        if (ptx::globaltimer() - t0 > kTimeoutNs) {
            *abort = 1;
            record_error(status, MLA_ERR_TIMEOUT, site);
            return false;
        }
    }
}

// Where packed row t comes from: its cache entry, and whether the row exists
// (t in [cu[0], cu[B]); a row that exists but whose page does not is zeros).
struct RowSource {
    const char* entry;
    bool exists;
};

template <int kEntryBytes>
__device__ __forceinline__ RowSource find_row(const ExpandParams& p, int t) {
    RowSource r{nullptr, false};
    if (t >= p.total) return r;
    // (the last row speaks for the sequences that the rows have no room for)
    if (t == p.total - 1 && p.cu[p.batch] > p.total)
        record_error(p.status, MLA_ERR_BAD_SEQ_LEN, p.cu[p.batch]);
    int lo = 0, hi = p.batch;       // the last b with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int begin = p.cu[lo], end = p.cu[lo + 1];
    if (begin < 0 || t < begin || t >= end) return r;
    r.exists = true;
    const int64_t pos = int64_t(p.first != nullptr ? p.first[lo] : 0) + (t - begin);
    if (pos < 0 || pos >= int64_t(p.max_blocks) * kPageSize) {
        record_error(p.status, MLA_ERR_BAD_SEQ_LEN, int32_t(pos < INT_MAX ? pos : INT_MAX));
        return r;
    }
    const int page = p.table[int64_t(lo) * p.max_blocks + pos / kPageSize];
    if (page < 0 || int64_t(page) >= p.num_blocks) {
        record_error(p.status, MLA_ERR_BAD_BLOCK_ID, page);
        return r;
    }
    r.entry = static_cast<const char*>(p.cache) +
              (int64_t(page) * kPageSize + pos % kPageSize) * (kD * kEntryBytes);
    return r;
}

// Two E4M3 codes as bf16 (exact: 4 exponent and 3 mantissa bits).
__device__ __forceinline__ uint32_t widen2(uint32_t codes16) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes16), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return uint32_t(f32_to_bf16_bits_rn(f.x)) | (uint32_t(f32_to_bf16_bits_rn(f.y)) << 16);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t* w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}
// 32 bytes (32-byte aligned).
__device__ __forceinline__ void load32(const char* p, uint32_t* r) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}

// 64 entries (32 words of bf16 pairs) from column 64 g of a row; zeros
// without one.
template <int kEntryBytes>
__device__ __forceinline__ void load64(const char* entry, int g, uint32_t* w) {
    uint32_t c[16 * kEntryBytes];
#pragma unroll
    for (int k = 0; k < 16 * kEntryBytes; ++k) c[k] = 0;
    if (entry != nullptr) {
#pragma unroll
        for (int k = 0; k < 2 * kEntryBytes; ++k)
            load32(entry + g * 64 * kEntryBytes + k * 32, c + 8 * k);
    }
    if constexpr (kEntryBytes == 2) {
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = c[k];
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            w[2 * k] = widen2(c[k] & 0xffffu);
            w[2 * k + 1] = widen2(c[k] >> 16);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return uint32_t(f32_to_bf16_bits_rn(a)) | (uint32_t(f32_to_bf16_bits_rn(b)) << 16);
}

template <int kEntryBytes>
__global__ void __launch_bounds__(kThreads, 1)
mla_expand_kernel(const ExpandParams p, const __grid_constant__ CUtensorMap map_uk,
                  const __grid_constant__ CUtensorMap map_uv) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
    const uint32_t b0 = sbase + kOffBar;
    auto full = [&](int s) { return b0 + uint32_t(offsetof(Bars, full)) + 8 * s; };
    auto empty = [&](int s) { return b0 + uint32_t(offsetof(Bars, empty)) + 8 * s; };
    auto a_ready = [&](int h) { return b0 + uint32_t(offsetof(Bars, a_ready)) + 8 * h; };
    auto acc_full = [&](int h) { return b0 + uint32_t(offsetof(Bars, acc_full)) + 8 * h; };
    auto acc_empty = [&](int h) { return b0 + uint32_t(offsetof(Bars, acc_empty)) + 8 * h; };
    const uint32_t drain = b0 + uint32_t(offsetof(Bars, drain));
    const int warp = threadIdx.x >> 5;

    if ((sbase & 1023u) != 0) {   // the swizzled tiles need it
        if (threadIdx.x == 0) record_error(p.status, MLA_ERR_UNSUPPORTED, 0);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int h = 0; h < 2; ++h) {
            ptx::mbar_init(a_ready(h), 128);
            ptx::mbar_init(acc_full(h), 1);
            ptx::mbar_init(acc_empty(h), 4);
        }
        ptx::mbar_init(drain, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&bars->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    // This CTA's items, and their token tiles. A token tile's rows past
    // `total` are zeros; a second half without rows does not run.
    const int per_tile = p.heads * 2;
    const int64_t begin = int64_t(blockIdx.x) * p.items / gridDim.x;
    const int64_t end = int64_t(blockIdx.x + 1) * p.items / gridDim.x;
    auto tile_end = [&](int64_t it) {
        const int64_t e = (it / per_tile + 1) * per_tile;
        return e < end ? e : end;
    };
    auto two_halves = [&](int64_t it) { return int64_t(p.total) - (it / per_tile) * kRows > 128; };

    if (warp == 0) {
        if (ptx::elect_one()) {
            uint32_t chunk = 0;
            const uint32_t chunks = uint32_t(end - begin) * kChunks;
            int item = int(begin % per_tile);
            for (; chunk < chunks; ++chunk) {
                const int s = int(chunk % kStages);
                const uint32_t turn = chunk / kStages;
                if (turn > 0 && !wait(empty(s), (turn - 1) & 1, bars, p.status, kSiteEmpty)) break;
                const int n = item >> 1, c = int(chunk % kChunks);
                const bool is_k = (item & 1) == 0;
                if (c == kChunks - 1 && ++item == per_tile) item = 0;
                const uint32_t st = sbase + uint32_t(kOffRing + s * kStageBytes);
                ptx::mbar_arrive_expect_tx(full(s), kStageBytes);
                if (is_k) {
                    ptx::tma_load_2d(st, &map_uk, c * kChunk, n * kHalf, full(s));
                } else {
                    ptx::tma_load_2d(st, &map_uv, 0, n * kLkv + c * kChunk, full(s));
                    ptx::tma_load_2d(st + 8192, &map_uv, 64, n * kLkv + c * kChunk, full(s));
                }
            }
            // Loads still in flight (after an abort) land before the CTA exits.
            for (uint32_t i = chunk > kStages ? chunk - kStages : 0; i < chunk; ++i)
                wait(full(int(i % kStages)), (i / kStages) & 1, bars, p.status, kSiteDrain,
                     true);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (ptx::elect_one()) {
            constexpr uint32_t idesc_k = ptx::idesc_bf16_f32(kHalf, false);
            constexpr uint32_t idesc_v = ptx::idesc_bf16_f32(kHalf, true);
            // (The thread that issues MMAs waits for the tensor pipe to take
            // each; what it does in between should be little. A descriptor is
            // the layout's constant bits plus the address, and only the first
            // half waits for a weight chunk.)
            const uint64_t desc_k = ptx::desc_sw128(0, 16, 1024);
            const uint64_t desc_v = ptx::desc_sw128(0, 8192, 1024);
            const uint32_t ring = (sbase + uint32_t(kOffRing)) >> 4;
            const uint64_t a_base = desc_k + ((sbase + uint32_t(kOffA)) >> 4);
            bool ok = true;
            uint32_t slot0 = 0, slot1 = 0, turn = 0;   // ring slot per half, parity of the first's
            uint32_t tiles[2] = {0, 0};                // column tiles begun per half
            uint32_t seg[2] = {0, 0};                  // token tiles begun per half
            for (int64_t it = begin; it < end && ok;) {
                const int64_t e = tile_end(it);
                const bool two = two_halves(it);
                ok = wait(a_ready(0), seg[0]++ & 1, bars, p.status, kSiteA);
                if (two) ok = ok && wait(a_ready(1), seg[1]++ & 1, bars, p.status, kSiteA);
                for (; it < e && ok; ++it) {
                    // W_UK_T: 16 k = 32 bytes per step; W_UV: 16 k-rows = 2 KB
                    // per step, its two 64-column blocks 8 KB apart.
                    const bool is_v = (it & 1) != 0;
                    const uint64_t w_base = (is_v ? desc_v : desc_k) + ring;
                    const uint32_t st = is_v ? 128 : 2;
                    const uint32_t idesc = is_v ? idesc_v : idesc_k;
                    // First half's chunk k, second half's chunk k - kSkew; the
                    // tile's last chunks of the second half go out before the
                    // next tile's first of the first half, so that three
                    // chunks' MMAs cover the readout of each accumulator.
#pragma unroll
                    for (int k = 0; k < kChunks + kSkew; ++k) {
                        if (k < kChunks) {
                            if (k == 0 && tiles[0]++ > 0)
                                ok = wait(acc_empty(0), tiles[0] & 1, bars, p.status,
                                          kSiteAccEmpty);
                            ok = ok && wait(full(slot0), turn, bars, p.status, kSiteFull);
                            if (!ok) break;
                            ptx::tc_fence_after();
                            const uint64_t w = w_base + slot0 * (kStageBytes / 16);
                            const uint32_t a = tmem + kTmemA + uint32_t(k * 32);
                            ptx::mma4_ts(tmem + kTmemAcc, a, a + 8, a + 16, a + 24, w, w + st,
                                         w + 2 * st, w + 3 * st, idesc, k > 0 ? 1u : 0u);
                            if (!two) ptx::mma_commit(empty(slot0));
                            if (k == kChunks - 1) ptx::mma_commit(acc_full(0));
                            if (++slot0 == kStages) {
                                slot0 = 0;
                                turn ^= 1;
                            }
                        }
                        if (two && k >= kSkew) {
                            if (k == kSkew && tiles[1]++ > 0) {
                                ok = wait(acc_empty(1), tiles[1] & 1, bars, p.status,
                                          kSiteAccEmpty);
                                if (!ok) break;
                                ptx::tc_fence_after();
                            }
                            const uint64_t w = w_base + slot1 * (kStageBytes / 16);
                            const uint64_t a = a_base + uint32_t((k - kSkew) * 1024);
                            ptx::mma4_ss(tmem + kTmemAcc + uint32_t(kHalf), a, a + 2, a + 4, a + 6,
                                         w, w + st, w + 2 * st, w + 3 * st, idesc,
                                         k > kSkew ? 1u : 0u);
                            ptx::mma_commit(empty(slot1));
                            if (k == kChunks + kSkew - 1) ptx::mma_commit(acc_full(1));
                            if (++slot1 == kStages) slot1 = 0;
                        }
                    }
                }
                if (!two) slot1 = slot0;
            }
            // Every MMA issued above has completed before TMEM is freed.
            ptx::mma_commit(drain);
            wait(drain, 0, bars, p.status, kSiteDrain, true);
        }
        __syncwarp();
    } else {
        const int h = warp >= 6 ? 1 : 0;
        const int lanes = (warp & 3) * 32;                 // TMEM lanes this warp reads
        const int lane = threadIdx.x & 31;
        const int r = lanes + lane;                        // row of the half
        const uint32_t lane_addr = uint32_t(lanes) << 16;
        bool ok = true;
        uint32_t done = 0;
        for (int64_t it = begin; it < end && ok;) {
            const int64_t e = tile_end(it);
            const int64_t t = (it / per_tile) * kRows + h * 128 + r;
            if (h == 1 && !two_halves(it)) { it = e; continue; }
            // Gather: this thread's row of the latent tile. Every MMA that
            // read the half's previous rows is done: its last accumulator was
            // waited for below.
            const RowSource src = find_row<kEntryBytes>(p, t < INT_MAX ? int(t) : INT_MAX);
            __syncwarp();
            if (h == 0) {
                // (TMEM takes a row per lane; whole 32-byte sectors at a time.)
#pragma unroll 1
                for (int g = 0; g < kLkv / 64; ++g) {
                    uint32_t w[32];
                    load64<kEntryBytes>(src.entry, g, w);
                    __syncwarp();
                    ptx::tmem_st32(tmem + kTmemA + lane_addr + uint32_t(g * 32), w);
                }
                ptx::tc_fence_before();
            } else {
                // A warp takes its 32 rows one after the other, eight in
                // flight, each lane a piece of the row: a lane per row reads
                // 32 lines a load (it took 20,000 clocks a token tile). Column
                // 8 j is 16-byte piece j % 8 of chunk j / 8.
                constexpr int kLoads = kEntryBytes;     // 16-byte loads per lane and row
#pragma unroll 1
                for (int i0 = 0; i0 < 32; i0 += 8) {
                    uint4 v[8][kLoads];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint64_t entry = __shfl_sync(
                            0xffffffffu, reinterpret_cast<uint64_t>(src.entry), i0 + i);
#pragma unroll
                        for (int k = 0; k < kLoads; ++k) {
                            v[i][k] = make_uint4(0, 0, 0, 0);
                            if (entry != 0)
                                v[i][k] = __ldg(reinterpret_cast<const uint4*>(entry) + k * 32 + lane);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int q = lanes + i0 + i;
                        const uint32_t row = sbase + uint32_t(kOffA + q * 128);
                        auto put = [&](int j, const uint32_t* w) {
                            st_shared16(row + uint32_t((j >> 3) * 16384 + (((j & 7) ^ (q & 7)) * 16)), w);
                        };
                        if constexpr (kEntryBytes == 2) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t w[4] = {v[i][k].x, v[i][k].y, v[i][k].z, v[i][k].w};
                                put(k * 32 + lane, w);
                            }
                        } else {
                            const uint32_t c[4] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w};
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                w[2 * k] = widen2(c[k] & 0xffffu);
                                w[2 * k + 1] = widen2(c[k] >> 16);
                            }
                            put(2 * lane, w);
                            put(2 * lane + 1, w + 4);
                        }
                    }
                }
                ptx::fence_proxy_async_smem();
            }
            ptx::mbar_arrive(a_ready(h));
            // The CTA with a token tile's first item writes its rows' k_pe.
            if (it % per_tile == 0 && src.exists) {
                uint4* dst = reinterpret_cast<uint4*>(p.k_pe + t * kRope);
                uint32_t w[32];
                load64<kEntryBytes>(src.entry, kLkv / 64, w);
                if constexpr (kEntryBytes == 1) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)   // one rounding of scale * code
                        w[i] = pack2(p.scale * bf16_bits_to_f32(w[i] & 0xffffu),
                                     p.scale * bf16_bits_to_f32(w[i] >> 16));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
            int item = int(it % per_tile);
            for (; it < e; ++it, ++item) {
                ok = wait(acc_full(h), done & 1, bars, p.status, kSiteAccFull);
                // (one answer for the warp: the TMEM loads are warp-wide)
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++done;
                ptx::tc_fence_after();
                uint32_t lo[64], hi[64];
                ptx::tmem_ld64(tmem + kTmemAcc + lane_addr + uint32_t(h * kHalf), lo);
                ptx::tmem_ld64(tmem + kTmemAcc + lane_addr + uint32_t(h * kHalf + 64), hi);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(acc_empty(h));
                uint32_t o[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    float a = __uint_as_float(i < 32 ? lo[2 * i] : hi[2 * i - 64]);
                    float b = __uint_as_float(i < 32 ? lo[2 * i + 1] : hi[2 * i - 63]);
                    if constexpr (kEntryBytes == 1) {
                        a *= p.scale;
                        b *= p.scale;
                    }
                    o[i] = pack2(a, b);
                }
                // 32 bytes of a row per lane and store. (Swapping pieces between
                // lanes so that a store fills whole 128-byte lines was 18%
                // slower at N = 128: shuffles share the shared-memory pipe
                // that feeds the MMAs, which is this kernel's bound.)
                if (src.exists) {
                    uint16_t* dst = p.kv + (t * p.heads + (item >> 1)) * 256 + (item & 1) * kHalf;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = o[i * 8 + k];
                        ptx::st_global_v8(dst + i * 16, w);
                    }
                }
                __syncwarp();
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

template <int kEntryBytes>
int launch_expand(const ExpandParams& p, const void* w_uk_t, const void* w_uv, int num_sms,
                  cudaStream_t st) {
    CUtensorMap uk, uv;
    if (!encode_2d(&uk, w_uk_t, kLkv, uint64_t(p.heads) * kHalf, 128) ||
        !encode_2d(&uv, w_uv, kHalf, uint64_t(p.heads) * kLkv, kChunk))
        return int(cudaErrorInvalidValue);
    auto kernel = mla_expand_kernel<kEntryBytes>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared_memory(kernel, kSmemBytes, &allowed);
    if (e != cudaSuccess) return int(e);
    const unsigned grid = unsigned(p.items < num_sms ? p.items : num_sms);
    kernel<<<grid, kThreads, kSmemBytes, st>>>(p, uk, uv);
    return int(cudaGetLastError());
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int expand(const void* cache, int entry_bytes, float scale, int64_t num_blocks,
           const int32_t* block_table, int max_blocks_per_seq, const int32_t* first_token,
           const int32_t* cu_seqlens_k, int batch, int total_k, int num_heads, const void* w_uk_t,
           const void* w_uv, void* kv, void* k_pe, void* workspace, size_t workspace_bytes,
           void* stream) {
    if (batch < 0 || total_k < 0 || num_blocks < 1 || max_blocks_per_seq < 1 || num_heads < 1)
        return MLA_ERR_INVALID_ARG;
    if (num_heads > kMaxHeads) return MLA_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || !(scale > 0.f)) return MLA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kStatusBytes || !aligned(workspace, 256))
        return MLA_ERR_WORKSPACE;
    if (batch == 0 || total_k == 0) return MLA_OK;
    if (!cache || !block_table || !cu_seqlens_k || !w_uk_t || !w_uv || !kv || !k_pe)
        return MLA_ERR_INVALID_ARG;
    if (!aligned(cache, 32) || !aligned(w_uk_t, 16) || !aligned(w_uv, 16) || !aligned(kv, 32) ||
        !aligned(k_pe, 16) || !aligned(block_table, 4) || !aligned(cu_seqlens_k, 4) ||
        (first_token && !aligned(first_token, 4)))
        return MLA_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return MLA_ERR_CUDA;
    ExpandParams p{};
    p.cache = cache;
    p.num_blocks = num_blocks;
    p.table = block_table;
    p.max_blocks = max_blocks_per_seq;
    p.first = first_token;
    p.cu = cu_seqlens_k;
    p.batch = batch;
    p.heads = num_heads;
    p.total = total_k;
    p.kv = static_cast<uint16_t*>(kv);
    p.k_pe = static_cast<uint16_t*>(k_pe);
    p.scale = scale;
    p.items = (int64_t(total_k) + kRows - 1) / kRows * num_heads * 2;
    p.status = static_cast<int32_t*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int e = entry_bytes == 2 ? launch_expand<2>(p, w_uk_t, w_uv, sms, st)
                                   : launch_expand<1>(p, w_uk_t, w_uv, sms, st);
    return e == 0 ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_expand_kv(const void* latent_cache, int64_t num_blocks,
                             const int32_t* block_table, int max_blocks_per_seq,
                             const int32_t* first_token, const int32_t* cu_seqlens_k, int batch,
                             int total_k, int num_heads, const void* w_uk_t, const void* w_uv,
                             void* kv, void* k_pe, void* workspace, size_t workspace_bytes,
                             void* stream) {
    return expand(latent_cache, 2, 1.f, num_blocks, block_table, max_blocks_per_seq, first_token,
                  cu_seqlens_k, batch, total_k, num_heads, w_uk_t, w_uv, kv, k_pe, workspace,
                  workspace_bytes, stream);
}

extern "C" int mla_expand_kv_fp8(const void* latent_cache_fp8, float k_scale, int64_t num_blocks,
                                 const int32_t* block_table, int max_blocks_per_seq,
                                 const int32_t* first_token, const int32_t* cu_seqlens_k,
                                 int batch, int total_k, int num_heads, const void* w_uk_t,
                                 const void* w_uv, void* kv, void* k_pe, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    return expand(latent_cache_fp8, 1, k_scale, num_blocks, block_table, max_blocks_per_seq,
                  first_token, cu_seqlens_k, batch, total_k, num_heads, w_uk_t, w_uv, kv, k_pe,
                  workspace, workspace_bytes, stream);
}
