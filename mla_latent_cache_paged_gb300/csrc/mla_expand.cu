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
// bytes written). A pair of CTAs works on 256 tokens and walks the (head,
// half) column tiles of 128 with M = 256 MMAs (cta_group::2): each CTA holds
// 128 of the rows, as the A operand in TMEM (256 columns of bf16 pairs) for all
// of the pair's columns, and half of each weight chunk in shared memory, 32
// bytes per clock per SM from L2 at the tensor pipe's full rate. The other 2 x
// 128 TMEM columns are two accumulators: one is read out while the tensor pipe
// fills the other. (One CTA on 256 rows, half of them in shared memory, was
// bound by that pipe: 205 us where this takes 153-157.)
//
// 7,865 tokens, N = 128: 153-157 us (1,670-1,725 TFLOP/s, 3.3 TB/s written);
// with the stores left out 137 us (1,920 TFLOP/s). What is between is the
// weights' way from L2 under the result's writes: a ring of 6 chunks instead
// of 8 costs 11 us, and 9 and 10 (which leave less of the SM's memory to L1)
// 4 to 7. 7,865 tokens, N = 16: 30 us; 500 tokens, N = 16: 9.5 us (bf16 cache)
// and 8.7 us (fp8). Arrivals on the other CTA's barriers carry no writes of
// memory (what they announce lies in TMEM, ordered by the tcgen05 fences), so
// they release at CTA scope: at cluster scope each waited for the thread's
// earlier stores (183 us).
//
// Work: the (token tile, head, half) items in that order, cut into one
// contiguous range per pair, so each pair gathers one or two token tiles.
// Warps: 0 = weight loads (TMA; each CTA its half), 1 = MMAs (the first CTA's),
// 2-5 and 6-9 = gather and epilogue (thread = row = TMEM lane), each of the
// two groups half of a row's columns, then every other column tile. Every wait
// is bounded (MLA_ERR_TIMEOUT).
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
constexpr int kRows = 256;                    // tokens per tile of a CTA pair
constexpr int kCtaRows = 128;                 // of which a CTA holds half
constexpr int kChunk = 128;                   // K per ring stage
constexpr int kChunks = kLkv / kChunk;        // 4 per column tile
constexpr int kStages = 8;
constexpr int kHalf = 128;                    // columns of a tile: k_nope or v of one head
constexpr int kCtaCols = kHalf / 2;           // of whose weights a CTA holds half
constexpr int kStageBytes = kCtaCols * kChunk * 2;   // 16 KB
constexpr int kWarpOut = 32 * kHalf * 2;      // a warp's part of a column tile: 2 boxes of 32 x 64
constexpr int kOffOut = kStages * kStageBytes;
constexpr int kOffBar = kOffOut + 8 * kWarpOut;
constexpr int kSmemBytes = kOffBar + 512;     // base is 1 KB aligned
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
// (Two pairs on the same SMs could each hold one SM's TMEM and wait for the other's.)
static_assert(2 * kSmemBytes > 233472, "one CTA per SM");
constexpr uint32_t kTmemA = 0;                // 256 columns: the CTA's rows, bf16 pairs
constexpr uint32_t kTmemAcc = 256;            // 2 x 128 fp32 columns
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr uint32_t kSuspendNs = 20000;
constexpr uint16_t kBoth = 3;                 // the pair's CTAs

enum ExpandSite : int32_t { kSiteEmpty = 50, kSiteFull, kSiteA, kSiteAFree, kSiteAccEmpty,
                            kSiteAccFull, kSiteDrain };

// In both CTAs; those marked L are used in the pair's first CTA only, the one
// that issues the MMAs.
struct Bars {
    uint64_t full[kStages];   // L: both CTAs' halves of the weight chunk
    uint64_t empty[kStages];
    uint64_t a_ready;         // L: 2 x 8 warps: the rows of a token tile are staged
    uint64_t a_free;          // the MMAs that read them are done
    uint64_t acc_full[2];
    uint64_t acc_empty[2];    // L: 2 x 4 warps: accumulator read out
    uint64_t drain;           // L
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

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
    return pack_bf16(f.x, f.y);
}

// 32 bytes (32-byte aligned).
__device__ __forceinline__ void load32(const char* p, uint32_t* r) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}

// 64 entries from column 64 g of a row, as they lie; zeros without one.
template <int kEntryBytes>
__device__ __forceinline__ void load64(const char* entry, int g, uint32_t (&c)[16 * kEntryBytes]) {
#pragma unroll
    for (int k = 0; k < 16 * kEntryBytes; ++k) c[k] = 0;
    if (entry != nullptr) {
#pragma unroll
        for (int k = 0; k < 2 * kEntryBytes; ++k)
            load32(entry + g * 64 * kEntryBytes + k * 32, c + 8 * k);
    }
}
// The same as bf16 pairs.
template <int kEntryBytes>
__device__ __forceinline__ void widen64(const uint32_t (&c)[16 * kEntryBytes], uint32_t (&w)[32]) {
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

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t* w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}
template <int kEntryBytes>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mla_expand_kernel(const ExpandParams p, const __grid_constant__ CUtensorMap map_uk,
                  const __grid_constant__ CUtensorMap map_uv,
                  const __grid_constant__ CUtensorMap map_kv) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
    const uint32_t b0 = sbase + kOffBar;
    auto full = [&](int s) { return b0 + uint32_t(offsetof(Bars, full)) + 8 * s; };
    auto empty = [&](int s) { return b0 + uint32_t(offsetof(Bars, empty)) + 8 * s; };
    auto acc_full = [&](int a) { return b0 + uint32_t(offsetof(Bars, acc_full)) + 8 * a; };
    auto acc_empty = [&](int a) { return b0 + uint32_t(offsetof(Bars, acc_empty)) + 8 * a; };
    const uint32_t a_ready = b0 + uint32_t(offsetof(Bars, a_ready));
    const uint32_t a_free = b0 + uint32_t(offsetof(Bars, a_free));
    const uint32_t drain = b0 + uint32_t(offsetof(Bars, drain));
    const int warp = threadIdx.x >> 5;
    const int rank = int(ptx::cluster_ctarank());

    if ((sbase & 1023u) != 0) {   // the swizzled tiles need it (the same in both CTAs)
        if (threadIdx.x == 0) record_error(p.status, MLA_ERR_UNSUPPORTED, 0);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(acc_full(a), 1);
            ptx::mbar_init(acc_empty(a), 2 * 4);
        }
        ptx::mbar_init(a_ready, 2 * 8);
        ptx::mbar_init(a_free, 1);
        ptx::mbar_init(drain, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(&bars->tmem_base), 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();          // (the pair's barriers exist before either uses the other's)
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    // The pair's items, and their token tiles. A token tile's rows past
    // `total` are zeros.
    const int per_tile = p.heads * 2;
    const int64_t pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int64_t begin = pair * p.items / pairs;
    const int64_t end = (pair + 1) * p.items / pairs;
    auto tile_end = [&](int64_t it) {
        const int64_t e = (it / per_tile + 1) * per_tile;
        return e < end ? e : end;
    };

    if (warp == 0) {
        if (ptx::elect_one()) {
            // This CTA's half of each weight chunk; the first CTA's barrier
            // counts the bytes of both.
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
                const uint32_t st = sbase + uint32_t(s * kStageBytes);
                const uint32_t bar = ptx::map_to_rank(full(s), 0);
                if (rank == 0) ptx::mbar_arrive_expect_tx(full(s), 2 * kStageBytes);
                if (is_k) {
                    const int y = n * kHalf + rank * kCtaCols;
                    ptx::tma_load_2d_pair(st, &map_uk, c * kChunk, y, bar);
                    ptx::tma_load_2d_pair(st + kStageBytes / 2, &map_uk, c * kChunk + 64, y, bar);
                } else {
                    ptx::tma_load_2d_pair(st, &map_uv, rank * kCtaCols, n * kLkv + c * kChunk, bar);
                }
            }
            // Loads still in flight (after an abort) land before the CTA
            // exits; the second CTA exits after the first.
            if (rank == 0)
                for (uint32_t i = chunk > kStages ? chunk - kStages : 0; i < chunk; ++i)
                    wait(full(int(i % kStages)), (i / kStages) & 1, bars, p.status, kSiteDrain,
                         true);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && ptx::elect_one()) {
            constexpr uint32_t idesc_k = ptx::idesc_bf16_f32_pair(kHalf, false);
            constexpr uint32_t idesc_v = ptx::idesc_bf16_f32_pair(kHalf, true);
            // (The thread that issues MMAs waits for the tensor pipe to take
            // each; what it does in between should be little. A descriptor is
            // the layout's constant bits plus the address.)
            const uint64_t desc_k = ptx::desc_sw128(0, 16, 1024) + (sbase >> 4);
            const uint64_t desc_v = ptx::desc_sw128(0, 8192, 1024) + (sbase >> 4);
            bool ok = true;
            uint32_t slot = 0, turn = 0;               // ring slot and its parity
            uint32_t n = 0, seg = 0;                   // column and token tiles begun
            for (int64_t it = begin; it < end && ok; ++seg) {
                const int64_t e = tile_end(it);
                ok = wait(a_ready, seg & 1, bars, p.status, kSiteA);
                for (; it < e && ok; ++it, ++n) {
                    // W_UK_T: 16 k = 32 bytes per step, 64 k = 8 KB; W_UV: 16
                    // k-rows = 2 KB per step.
                    const bool is_v = (it & 1) != 0;
                    const uint64_t desc = is_v ? desc_v : desc_k;
                    const uint32_t st = is_v ? 128 : 2;
                    const uint32_t idesc = is_v ? idesc_v : idesc_k;
                    const uint32_t acc = tmem + kTmemAcc + (n & 1) * kHalf;
                    if (n >= 2)
                        ok = wait(acc_empty(n & 1), ((n >> 1) - 1) & 1, bars, p.status,
                                  kSiteAccEmpty);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        ok = ok && wait(full(slot), turn, bars, p.status, kSiteFull);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint64_t w = desc + slot * (kStageBytes / 16);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a = tmem + kTmemA + uint32_t(c * 64 + h * 32);
                            const uint64_t b = w + uint32_t(h * 512);
                            ptx::mma4_ts_pair(acc, a, a + 8, a + 16, a + 24, b, b + st, b + 2 * st,
                                              b + 3 * st, idesc, c + h > 0 ? 1u : 0u);
                        }
                        ptx::mma_commit_pair(empty(slot), kBoth);
                        if (++slot == kStages) {
                            slot = 0;
                            turn ^= 1;
                        }
                    }
                    if (ok) ptx::mma_commit_pair(acc_full(n & 1), kBoth);
                }
                if (ok) ptx::mma_commit_pair(a_free, kBoth);
            }
            // Every MMA issued above has completed before TMEM is freed.
            ptx::mma_commit_pair(drain, 1);
            wait(drain, 0, bars, p.status, kSiteDrain, true);
        }
        __syncwarp();
    } else {
        // Gather and epilogue. Group g takes columns 256 g.. of the latent
        // rows into TMEM, and every other column tile out of it.
        const int g = warp >= 6 ? 1 : 0;
        const int lanes = (warp & 3) * 32;                 // TMEM lanes this warp reads
        const int lane = threadIdx.x & 31;
        const int r = lanes + lane;                        // row of the CTA
        const uint32_t lane_addr = uint32_t(lanes) << 16;
        const uint32_t acc = tmem + kTmemAcc + lane_addr + uint32_t(g * kHalf);
        const uint32_t to_ready = ptx::map_to_rank(a_ready, 0);
        const uint32_t to_empty = ptx::map_to_rank(acc_empty(g), 0);
        const uint32_t out = sbase + uint32_t(kOffOut + (warp - 2) * kWarpOut);
        bool ok = true;
        uint32_t n = 0, seg = 0;
        for (int64_t it = begin; it < end && ok; ++seg) {
            const int64_t e = tile_end(it);
            const int64_t t = (it / per_tile) * kRows + rank * kCtaRows + r;
            const RowSource src = find_row<kEntryBytes>(p, t < INT_MAX ? int(t) : INT_MAX);
            __syncwarp();
            const bool whole = __all_sync(0xffffffffu, src.exists);
            // A row per lane, as TMEM takes it; whole 32-byte sectors at a time.
            uint32_t c[4][16 * kEntryBytes];
#pragma unroll
            for (int k = 0; k < 4; ++k) load64<kEntryBytes>(src.entry, 4 * g + k, c[k]);
            if (seg > 0) {
                ok = __all_sync(0xffffffffu,
                                wait(a_free, (seg - 1) & 1, bars, p.status, kSiteAFree));
                if (!ok) break;
                ptx::tc_fence_after();
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t w[32];
                widen64<kEntryBytes>(c[k], w);
                __syncwarp();
                ptx::tmem_st32(tmem + kTmemA + lane_addr + uint32_t(g * 128 + k * 32), w);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster(to_ready);
            // The pair with a token tile's first item writes its rows' k_pe.
            if (g == 0 && it % per_tile == 0 && src.exists) {
                uint4* dst = reinterpret_cast<uint4*>(p.k_pe + t * kRope);
                uint32_t pe[16 * kEntryBytes], w[32];
                load64<kEntryBytes>(src.entry, kLkv / 64, pe);
                widen64<kEntryBytes>(pe, w);
                if constexpr (kEntryBytes == 1) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)   // one rounding of scale * code
                        w[i] = pack_bf16(p.scale * bf16_bits_to_f32(w[i] & 0xffffu),
                                     p.scale * bf16_bits_to_f32(w[i] >> 16));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
            __syncwarp();
            int item = int(it % per_tile);
            for (; it < e; ++it, ++item, ++n) {
                if (int(n & 1) != g) continue;
                ok = wait(acc_full(g), (n >> 1) & 1, bars, p.status, kSiteAccFull);
                // (one answer for the warp: the TMEM loads are warp-wide)
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                uint32_t lo[64], hi[64];
                ptx::tmem_ld64(acc, lo);
                ptx::tmem_ld64(acc + 64, hi);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(to_empty);
                uint32_t o[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    float a = __uint_as_float(i < 32 ? lo[2 * i] : hi[2 * i - 64]);
                    float b = __uint_as_float(i < 32 ? lo[2 * i + 1] : hi[2 * i - 63]);
                    if constexpr (kEntryBytes == 1) {
                        a *= p.scale;
                        b *= p.scale;
                    }
                    o[i] = pack_bf16(a, b);
                }
                if (whole) {
                    // Through shared memory (16-byte piece k of a row of a box
                    // at k ^ row % 8), so that whole lines are written: 153 us
                    // against 159 by the stores below.
                    if (lane == 0) ptx::bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        st_shared16(out + uint32_t((i >> 3) * (kWarpOut / 2) + lane * 128 +
                                                   (((i & 7) ^ (lane & 7)) * 16)), o + 4 * i);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        const int x = (item >> 1) * 256 + (item & 1) * kHalf;
                        ptx::tma_store_2d(&map_kv, x, int(t), out);
                        ptx::tma_store_2d(&map_kv, x + 64, int(t), out + kWarpOut / 2);
                        ptx::bulk_commit();
                    }
                } else if (src.exists) {
                    // 32 bytes of a row per lane and store.
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
        if (lane == 0) ptx::bulk_wait();
        __syncwarp();
    }
    // Neither CTA leaves while the other's MMAs, loads or arrivals may reach it.
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
}

template <int kEntryBytes>
int launch_expand(const ExpandParams& p, const void* w_uk_t, const void* w_uv, int num_sms,
                  cudaStream_t st) {
    CUtensorMap uk, uv, kv;
    if (!encode_2d(&uk, w_uk_t, kLkv, uint64_t(p.heads) * kHalf, kCtaCols) ||
        !encode_2d(&uv, w_uv, kHalf, uint64_t(p.heads) * kLkv, kChunk) ||
        !encode_2d(&kv, p.kv, uint64_t(p.heads) * 256, uint64_t(p.total), 32))
        return int(cudaErrorInvalidValue);
    auto kernel = mla_expand_kernel<kEntryBytes>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared_memory(kernel, kSmemBytes, &allowed);
    if (e != cudaSuccess) return int(e);
    const int64_t most = num_sms / 2 > 1 ? num_sms / 2 : 1;
    const unsigned pairs = unsigned(p.items < most ? p.items : most);
    kernel<<<2 * pairs, kThreads, kSmemBytes, st>>>(p, uk, uv, kv);
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
