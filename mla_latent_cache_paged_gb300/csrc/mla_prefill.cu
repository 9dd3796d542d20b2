// Expanded-form latent attention for many query tokens (mla_prefill): ragged
// sequences, causal or not, head dims 192 (keys: 128 of the token's own head
// and 64 shared by all heads) and 128 (values).
//
//   s_ij  = scale * (q_i[0:128] . k_nope_j + q_i[128:192] . k_pe_j)
//   lse_i = ln sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j
// over the keys that query i sees: j <= Lk - Lq + i (causal) or all Lk. k_pe
// is read where it lies, once per key tile; no per-head copy of it exists.
//
// A work item is 256 query rows (two tiles of 128) of one head of one
// sequence (and one split of its keys). Persistent CTAs, one per SM, draw
// items as they finish. Per 128-key step and tile:
//   S = Q K^T      tcgen05.mma 128 x 128 x 192, Q and K in shared memory
//   P = 2^(S c - m c)   128 threads, one query row each (= TMEM lane), fp32;
//                  P as bf16 over S in TMEM. The reference maximum m moves
//                  only when it would grow by more than 2^8, so rescaling O
//                  (a TMEM read-modify-write) is rare; the sum is kept in
//                  fp32 of the unrounded weights. P's rounding to bf16 is
//                  what the tensor cores' operand type costs.
//   O += P V       128 x 128 x 128, P the A operand in TMEM, V in shared memory
// The two tiles share every key and value block and run half a step apart:
// the tensor pipe works on one while the softmax works on the other. TMEM:
// S/P 2 x 128 columns, O 2 x 128 columns.
//
// Bound: the tensor pipe, 2 * 320 flops per visible (query, key, head) pair;
// per 128-key step of a 256-row item 2,560 clocks of it, against 1,024-2,048
// clocks of exponentials (32,768 of them) and 80 KB of loads (32 bytes per
// clock per SM, from L2: the items of a group of heads run together, so that
// their keys and values stay there).
// Measured, 4,096 causal tokens x 128 heads (344 us at cuBLAS's burst rate, 394
// at its rate under the power cap): 442-462 us replayed, 520 in calls back to
// back under the power cap. Copies of the kernel for timing took 405 us with the
// softmax left out and 379 us with the key and value loads left out too (468 as
// it was then): the score MMAs take both operands from shared memory, 128 bytes
// a clock, which is its rate, and the loads write there as well. 24 prompts of
// 2 to 886 tokens x 16 heads 64-65 us; four chunks of ~480 rows over 3,589 to
// 5,711 keys x 32 heads 141-147 us.
//
// Keys and values of a 128-key step that lie past the sequence's end belong to
// the next sequence, and those past a row's causal limit are its own future:
// scores there are replaced by -inf, but a weight of 0 does not keep a NaN or
// infinity of V out of the product. So, in the steps where some row's limit
// falls, a helper warp clears V's rows past the end and replaces non-finite
// values by 0 before the tensor pipe reads them; if it replaced any, the
// epilogue adds them, times their weights, to the rows that do see them.
//
// Warps: 0-3 and 4-7 = softmax and epilogue of the tiles, 8 = loads (TMA), 9 =
// MMAs, 10 = helper, 11 = item scheduler. Every wait is bounded
// (MLA_ERR_TIMEOUT).
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "mla_prefill.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"

namespace mla {
namespace {

constexpr int kThreads = 384;
constexpr int kTileRows = 128;
constexpr int kItemRows = 2 * kTileRows;
constexpr int kStep = 128;                    // keys per step
constexpr int kQk = kPrefillQk, kV = kPrefillV, kKvHead = kPrefillKv;
constexpr int kBlock = 16384;                 // 128 x 64 (Q, K) or 64 x 128 (V) bf16
constexpr int kQBlocks = 3;                   // per tile
constexpr int kRing = 8;                      // blocks: K of a step takes 3, V takes 2
constexpr int kOffRing = 2 * kQBlocks * kBlock;
constexpr int kOffBar = kOffRing + kRing * kBlock;
constexpr int kItemSlots = 2;
// The next item is drawn when the loads come to an item's last steps, so that
// a CTA with a long item does not hold another that an idle one could take:
// 2,048 causal tokens x 32 heads 48 -> 40 us, sequences of 700 and 300 rows over
// 6,000 and 3,000 keys x 32 heads 130 -> 93 us. (The draw takes 3,000 clocks. With
// 1 to 3 steps the long prompt takes 1-2% more, with 5 to 8 0.5%.)
constexpr int kNearSteps = 5;
constexpr int kSmemBytes = kOffBar + 1024;    // base is 1 KB aligned
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
constexpr uint32_t kTmemS = 0;                // 2 x 128 columns; P overwrites the first 64 of each
constexpr uint32_t kTmemO = 256;              // 2 x 128 columns
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr uint32_t kSuspendNs = 20000;
constexpr int kMaxSplits = 64;
// Keys and values of the heads that run together (a third of the L2).
constexpr int64_t kGroupBytes = int64_t(40) << 20;

enum PrefillSite : int32_t { kSiteItem = 70, kSiteItemFree, kSiteQ, kSiteQFree, kSiteRing,
                             kSiteRingFree, kSiteS, kSiteP, kSitePv, kSiteRaw, kSiteDrain };

struct Item {
    int32_t head;         // -1: no more items
    int32_t q_row;        // packed row of the item's first query
    int32_t q_rows;       // its queries (1..256)
    int32_t k_row;        // packed row of the sequence's first key
    int32_t lk;           // the sequence's keys
    int32_t limit0;       // last key that the item's first query sees (causal: row i sees limit0 + i)
    int32_t step_lo;      // steps of this split, per tile [step_lo, step_hi[t])
    int32_t step_hi[2];
    int32_t fix_from;     // first step whose values need the helper
    int32_t part_stride;  // 0: all of the item's keys. Else this is a part of them, and query i's
    int64_t part_row;     // result is partial row part_row + i * part_stride
};

struct Bars {
    // Steps alternate between the two of a pair: a waiter tells a phase from
    // its predecessor only, and the loads may be two releases behind the MMAs
    // (they wait for an item between two steps), but never a whole pair.
    uint64_t k_full[2], v_full[2];
    uint64_t k_empty[2], v_empty[2];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2];       // scores of the step complete
    uint64_t p_ready[2];      // 4 arrivals, one per softmax warp: weights in TMEM, O rescaled
    uint64_t pv_done[2];      // P.V of the step complete
    // A step whose values the helper works on: its V blocks land here, and the
    // helper completes v_full.
    uint64_t raw_full[2];
    uint64_t item_full[kItemSlots], item_empty[kItemSlots];
    uint64_t item_near;       // the loads have come to an item's last steps
    uint64_t drain;
    Item items[kItemSlots];
    int32_t bad_item[kItemSlots];   // sequence number of an item with replaced values
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier block");
constexpr int kItemConsumers = 8 + 3;   // softmax warps, loads, MMAs, helper

// Bounded wait. A waiting thread sleeps in mbarrier.try_wait: threads that
// poll take issue slots from the softmax warps (256 polls before the first
// sleep made the whole kernel 1.7 times slower).
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

// 32 lanes x 128 columns.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
    uint32_t lo[64], hi[64];
    ptx::tmem_ld64(taddr, lo);
    ptx::tmem_ld64(taddr + 64, hi);
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        v[i] = __uint_as_float(lo[i]);
        v[64 + i] = __uint_as_float(hi[i]);
    }
}

// sum += 0 * x for a pair of bf16 values.
__device__ __forceinline__ void add_zero_times(uint32_t x, uint32_t* sum) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(*sum) : "r"(x), "r"(0));
}

// q . k of one row (of q [total_q, N]) and one key, not scaled. For the few
// that need it outside the tensor pipe: rolled loops, little code.
__device__ __forceinline__ float score(const PrefillParams& p, int64_t q_row, int k_row, int head) {
    const uint4* q = reinterpret_cast<const uint4*>(p.q + q_row * kQk);
    const uint4* k = reinterpret_cast<const uint4*>(
        p.kv + (int64_t(k_row) * p.heads + head) * kKvHead);
    const uint4* pe = reinterpret_cast<const uint4*>(p.k_pe + int64_t(k_row) * kRope);
    float s = 0.f;
#pragma unroll 1
    for (int i = 0; i < kQk / 8; ++i) {
        const uint4 a = __ldg(q + i), b = __ldg(i < 16 ? k + i : pe + (i - 16));
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), s);
            s = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), s);
        }
    }
    return s;
}

// Pairs of floats: one instruction for two (round to nearest, as the single ones).
__device__ __forceinline__ uint64_t pack_f32(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack_f32(uint64_t d, float* a, float* b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ int item_tiles(int lq) { return lq / kItemRows + (lq % kItemRows != 0); }

// The order of the items. CTAs draw items as they finish, so the long ones
// should come first and the short ones fill the end; but the items of one head
// should also run together, so that its keys and values are read from HBM
// once. So the row tiles are taken in four classes by the keys their last row
// sees (more than 3/4, 1/2, 1/4 of the longest, the rest), in a class heads in
// groups, in a group tile after tile, then heads, then splits. In the lower two
// classes all heads are one group: what comes last is short then (long prompt
// 472 -> 464 us, 24 prompts 67.9 -> 66.5).
// (4,096 causal tokens x 128 heads: within 1% of the mean load, against 29%
// above it for a fixed deal by groups; four 480-row chunks over 3,589 to 5,711
// keys x 32 heads: 168 -> 148 us against an order by position.)
constexpr int kClasses = 4;

// The first row tile of a sequence whose last row sees more than `keys` keys.
__device__ __forceinline__ int first_tile(const PrefillParams& p, int lq, int lk, int keys) {
    const int tiles = item_tiles(lq);
    if (lk <= keys) return tiles;
    if (!p.causal) return 0;
    const int64_t d = int64_t(keys) - lk + lq;     // tile i's last row sees min(lk, lk - lq + 256 (i + 1))
    return d < 0 ? 0 : int(min(d / kItemRows, int64_t(tiles)));
}

struct Order {
    int64_t tiles[kClasses];
    int longest;          // most keys of a sequence with queries

    __device__ __forceinline__ int above(int c) const {   // class c: more keys than this
        return int(int64_t(longest) * (kClasses - 1 - c) / kClasses);
    }
    // The tiles [*lo, *hi) of a sequence that are in class c.
    __device__ __forceinline__ void range(const PrefillParams& p, int lq, int lk, int c, int* lo,
                                          int* hi) const {
        *hi = c == 0 ? item_tiles(lq) : first_tile(p, lq, lk, above(c - 1));
        *lo = c == kClasses - 1 ? 0 : first_tile(p, lq, lk, above(c));
    }
};

__device__ __forceinline__ Order count_tiles(const PrefillParams& p) {
    const int lane = threadIdx.x & 31;
    Order o;
    o.longest = 0;
    int q0, lq, k0, lk;
    for (int b = lane; b < p.batch; b += 32) {
        sequence(p, b, &q0, &lq, &k0, &lk);
        if (lq > 0) o.longest = max(o.longest, lk);
    }
    __syncwarp();
    o.longest = __reduce_max_sync(0xffffffffu, o.longest);
    int n[kClasses] = {0, 0, 0, 0};
    for (int b = lane; b < p.batch; b += 32) {
        sequence(p, b, &q0, &lq, &k0, &lk);
#pragma unroll
        for (int c = 0; c < kClasses; ++c) {
            int lo, hi;
            o.range(p, lq, lk, c, &lo, &hi);
            n[c] += hi - lo;
        }
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kClasses; ++c) o.tiles[c] = __reduce_add_sync(0xffffffffu, n[c]);
    return o;
}

// Which items are split, and how often: all of them p.splits times, or
// (split_rest) those of the last, partly filled wave, [whole, total), which
// would leave SMs without work for its whole length. Of that wave each CTA gets
// one part at most, so a wave that is more than half full is not split: a
// part's fp32 rows and its share of the merge cost about as much as three steps.
struct Units {
    int64_t whole, total;      // items not split, items
    int splits;
    __device__ __forceinline__ Units(const PrefillParams& p, const Order& o) {
        total = 0;
#pragma unroll
        for (int c = 0; c < kClasses; ++c) total += o.tiles[c] * p.heads;
        whole = 0;
        splits = p.splits;
        if (p.split_rest) {
            const int rest = int(total % gridDim.x);
            if (rest > 0) splits = min(splits, int(gridDim.x) / rest);
            whole = rest > 0 && splits > 1 ? total - rest : total;
        }
    }
    __device__ __forceinline__ int64_t count() const { return whole + (total - whole) * splits; }
};

// Everything an item's roles need, from the unit's place in the order. The
// whole warp works on it.
__device__ __forceinline__ Item find_item(const PrefillParams& p, int64_t index, const Order& o,
                                          const Units& units) {
    const int lane = threadIdx.x & 31;
    Item it;
    int splits = 1, split = 0;
    int64_t part = 0;
    if (index >= units.whole) {
        part = index - units.whole;
        splits = units.splits;
        split = int(part % splits);
        index = units.whole + part / splits;
    }
    int cls = 0;
    int64_t tiles = o.tiles[0];
#pragma unroll
    for (int c = 1; c < kClasses; ++c) {
        if (cls == c - 1 && index >= tiles * p.heads) {
            index -= tiles * p.heads;
            cls = c;
            tiles = o.tiles[c];
        }
    }
    const int group = cls >= kClasses / 2 ? p.heads : p.group;
    const int64_t per_group = tiles * group;
    const int head0 = int(index / per_group) * group;
    const int64_t rem = index % per_group;
    const int per_tile = min(group, p.heads - head0);
    int64_t tile = rem / per_tile;
    it.head = head0 + int(rem % per_tile);
    // The sequence that holds the class's tile of this number.
    int q0 = 0, lq = 0, k0 = 0, lk = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        int lo = 0, hi = 0;
        if (b0 + lane < p.batch) {
            sequence(p, b0 + lane, &q0, &lq, &k0, &lk);
            o.range(p, lq, lk, cls, &lo, &hi);
        }
        __syncwarp();
        int inc = hi - lo;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += u;
        }
        const int all = __shfl_sync(0xffffffffu, inc, 31);
        if (tile < all) {
            const int src = __ffs(__ballot_sync(0xffffffffu, inc > tile)) - 1;
            // (the last of the sequence's tiles first)
            tile = __shfl_sync(0xffffffffu, lo + inc - 1, src) - tile;
            q0 = __shfl_sync(0xffffffffu, q0, src);
            lq = __shfl_sync(0xffffffffu, lq, src);
            k0 = __shfl_sync(0xffffffffu, k0, src);
            lk = __shfl_sync(0xffffffffu, lk, src);
            break;
        }
        tile -= all;
    }
    const int first = int(tile) * kItemRows;
    it.q_row = q0 + first;
    it.q_rows = min(kItemRows, lq - first);
    it.k_row = k0;
    it.lk = lk;
    it.limit0 = p.causal ? lk - lq + first : lk - 1;
    // Keys that the last row of each tile sees, then this split's steps.
    int steps[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int rows = min(kTileRows, it.q_rows - t * kTileRows);
        int keys = 0;
        if (rows > 0) {
            keys = p.causal ? it.limit0 + t * kTileRows + rows : lk;
            keys = max(0, min(keys, lk));
        }
        steps[t] = keys / kStep + (keys % kStep != 0);
    }
    const int most = max(steps[0], steps[1]);
    const int chunk = (most + splits - 1) / splits;
    it.step_lo = min(most, split * chunk);
    const int hi = min(most, it.step_lo + chunk);
    it.step_hi[0] = max(it.step_lo, min(hi, steps[0]));
    it.step_hi[1] = max(it.step_lo, min(hi, steps[1]));
    // Steps before this one lie wholly within every row's limit.
    const int whole = p.causal ? max(0, min(it.limit0 + 1, lk)) : lk;
    it.fix_from = max(it.step_lo, whole / kStep);
    // (parts of the last wave: one per CTA at most)
    it.part_stride = splits == 1 ? 0 : p.split_rest ? 1 : p.heads * splits;
    it.part_row = p.split_rest ? part * kItemRows
                               : (int64_t(it.q_row) * p.heads + it.head) * splits + split;
    return it;
}

// The item consumers' side of the item ring.
struct ItemReader {
    uint32_t full, empty;
    uint32_t n = 0;
    __device__ __forceinline__ bool next(Bars* bars, int32_t* status, Item* out) {
        const uint32_t s = n % kItemSlots;
        if (!wait(full + 8 * s, (n / kItemSlots) & 1, bars, status, kSiteItem)) return false;
        *out = bars->items[s];
        return true;
    }
    __device__ __forceinline__ void release() {
        ptx::mbar_arrive(empty + 8 * (n % kItemSlots));
        ++n;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
mla_prefill_kernel(const PrefillParams p, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_kv,
                   const __grid_constant__ CUtensorMap map_pe) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
    const uint32_t b0 = sbase + kOffBar;
#define MLA_BAR(field) (b0 + uint32_t(offsetof(Bars, field)))
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if ((sbase & 1023u) != 0) {   // the swizzled tiles need it
        if (threadIdx.x == 0) record_error(p.status, MLA_ERR_UNSUPPORTED, 0);
        return;
    }
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(MLA_BAR(k_full) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(v_full) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(k_empty) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(v_empty) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(raw_full) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(q_full) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(q_empty) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(s_full) + 8 * t, 1);
            ptx::mbar_init(MLA_BAR(p_ready) + 8 * t, 4);
            ptx::mbar_init(MLA_BAR(pv_done) + 8 * t, 1);
        }
        for (int s = 0; s < kItemSlots; ++s) {
            ptx::mbar_init(MLA_BAR(item_full) + 8 * s, 1);
            ptx::mbar_init(MLA_BAR(item_empty) + 8 * s, kItemConsumers);
            bars->bad_item[s] = -1;
        }
        ptx::mbar_init(MLA_BAR(item_near), 1);
        ptx::mbar_init(MLA_BAR(drain), 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        ptx::tmem_alloc(ptx::smem_addr(&bars->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    ItemReader items{MLA_BAR(item_full), MLA_BAR(item_empty)};
    Item it;

    // Registers: 384 threads x 168 at launch = 64,512; the softmax warps take
    // 200 (a row's 128 scores stay in registers), the others 104:
    // 256 x 200 + 128 x 104 = 64,512.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == 8) {
            // ------------------------------------------------------- loads
            if (ptx::elect_one()) {
                // Ring blocks in order: step g's keys at 5g..5g+2, its values at
                // 5g+3 and 5g+4. Eight blocks back from keys 1 and 2 lie the
                // values of step g-2, from the values the keys of step g-1
                // (and from key 0 those of step g-2, waited for by then).
                uint32_t step = 0, q_loads[2] = {0, 0}, raws = 0;
                bool ok = true, raw_last[2] = {false, false};
                auto addr = [&](uint32_t i) {
                    return sbase + uint32_t(kOffRing) + (i % kRing) * kBlock;
                };
                while (ok && items.next(bars, p.status, &it)) {
                    if (it.head < 0) break;
                    const int steps = max(it.step_hi[0], it.step_hi[1]);
                    const int near = max(it.step_lo, steps - kNearSteps);
                    if (near >= steps) ptx::mbar_arrive(MLA_BAR(item_near));
                    for (int j = it.step_lo; j < steps && ok; ++j, ++step) {
                        if (j == near) ptx::mbar_arrive(MLA_BAR(item_near));
                        const int row = it.k_row + j * kStep;
                        const uint32_t bar = MLA_BAR(k_full) + 8 * (step & 1);
                        ptx::mbar_arrive_expect_tx(bar, 3 * kBlock);
                        // (boxes of 64 rows; a block of keys takes two)
                        auto load_keys = [&](uint32_t dst, int x) {
                            ptx::tma_load_2d(dst, &map_kv, x, row, bar);
                            ptx::tma_load_2d(dst + kBlock / 2, &map_kv, x, row + kStep / 2, bar);
                        };
                        load_keys(addr(5 * step), it.head * kKvHead);
                        if (step >= 2)
                            ok = wait(MLA_BAR(v_empty) + 8 * (step & 1), ((step - 2) >> 1) & 1,
                                      bars, p.status, kSiteRingFree);
                        // (after an abort the phase's other bytes still come, so
                        // that the drain below ends)
                        load_keys(addr(5 * step + (ok ? 1 : 0)), it.head * kKvHead + 64);
                        ptx::tma_load_2d(addr(5 * step + (ok ? 2 : 0)), &map_pe, 0, row, bar);
                        if (j == it.step_lo) {
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                if (!ok || it.step_hi[t] <= it.step_lo) continue;
                                if (q_loads[t] > 0)
                                    ok = wait(MLA_BAR(q_empty) + 8 * t, (q_loads[t] - 1) & 1, bars,
                                              p.status, kSiteQFree);
                                if (!ok) continue;
                                const uint32_t q_bar = MLA_BAR(q_full) + 8 * t;
                                ptx::mbar_arrive_expect_tx(q_bar, kQBlocks * kBlock);
                                for (int c = 0; c < kQBlocks; ++c)
                                    ptx::tma_load_2d(sbase + uint32_t((t * kQBlocks + c) * kBlock),
                                                     &map_q, it.head * kQk + 64 * c,
                                                     it.q_row + t * kTileRows, q_bar);
                                ++q_loads[t];
                            }
                        }
                        if (step >= 1)
                            ok = ok && wait(MLA_BAR(k_empty) + 8 * ((step - 1) & 1),
                                            ((step - 1) >> 1) & 1, bars, p.status, kSiteRingFree);
                        if (!ok) {
                            ++step;
                            raw_last[(step - 1) & 1] = true;   // no values were asked for
                            break;
                        }
                        const bool raw = j >= it.fix_from;
                        const uint32_t v_bar = raw ? MLA_BAR(raw_full) + 8 * (raws & 1)
                                                   : MLA_BAR(v_full) + 8 * (step & 1);
                        raw_last[step & 1] = raw;
                        raws += raw ? 1 : 0;
                        ptx::mbar_arrive_expect_tx(v_bar, 2 * kBlock);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int x = it.head * kKvHead + 128, y = row + 64 * c;
                            const uint32_t dst = addr(5 * step + 3 + c);
                            ptx::tma_load_2d(dst, &map_kv, x, y, v_bar);
                            ptx::tma_load_2d(dst + 8192, &map_kv, x + 64, y, v_bar);
                        }
                    }
                    items.release();
                }
                // Loads still in flight (after an abort) land before the CTA exits.
                for (uint32_t g = step > 2 ? step - 2 : 0; g < step; ++g) {
                    wait(MLA_BAR(k_full) + 8 * (g & 1), (g >> 1) & 1, bars, p.status, kSiteDrain,
                         true);
                    if (!raw_last[g & 1])
                        wait(MLA_BAR(v_full) + 8 * (g & 1), (g >> 1) & 1, bars, p.status,
                             kSiteDrain, true);
                }
                for (uint32_t i = raws > 2 ? raws - 2 : 0; i < raws; ++i)
                    wait(MLA_BAR(raw_full) + 8 * (i & 1), (i >> 1) & 1, bars, p.status, kSiteDrain,
                         true);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (q_loads[t] > 0)
                        wait(MLA_BAR(q_full) + 8 * t, (q_loads[t] - 1) & 1, bars, p.status,
                             kSiteDrain, true);
            }
            __syncwarp();
        } else if (warp == 9) {
            // -------------------------------------------------------- MMAs
            if (ptx::elect_one()) {
                constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(kStep, false);
                constexpr uint32_t idesc_o = ptx::idesc_bf16_f32(kV, true);
                // An operand's descriptor: the layout's constant bits and the
                // block's address. (A thread that issues MMAs waits for the
                // tensor pipe to take each; what it does in between is time
                // that the pipe may run dry, so descriptors cost two adds,
                // barriers are tested before they are slept on, and a step has
                // one release for its keys and one for its values.)
                const uint64_t desc_k = ptx::desc_sw128(0, 16, 1024);
                const uint64_t desc_v = ptx::desc_sw128(0, 8192, 1024);
                uint32_t step = 0;
                uint32_t q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
                bool ok = true;
                auto ring = [&](uint32_t i) {      // address >> 4
                    return (sbase + uint32_t(kOffRing) + (i % kRing) * kBlock) >> 4;
                };
                // Scores of tile t for step g.
                auto scores = [&](int t, uint32_t g) {
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        const uint64_t a =
                            desc_k + ((sbase + uint32_t((t * kQBlocks + c) * kBlock)) >> 4);
                        const uint64_t b = desc_k + ring(5 * g + c);
                        ptx::mma4_ss(tmem + kTmemS + 128 * t, a, a + 2, a + 4, a + 6, b, b + 2,
                                     b + 4, b + 6, idesc_s, c > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(MLA_BAR(s_full) + 8 * t);
                };
                // O of tile t += P V of step g.
                auto values = [&](int t, uint32_t g, bool first) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t a = tmem + kTmemS + 128 * t + 32 * c;
                        const uint64_t b = desc_v + ring(5 * g + 3 + c);
                        ptx::mma4_ts(tmem + kTmemO + 128 * t, a, a + 8, a + 16, a + 24, b, b + 128,
                                     b + 256, b + 384, idesc_o, c > 0 || !first ? 1u : 0u);
                    }
                    ptx::mma_commit(MLA_BAR(pv_done) + 8 * t);
                };
                while (ok && items.next(bars, p.status, &it)) {
                    if (it.head < 0) break;
                    const int steps = max(it.step_hi[0], it.step_hi[1]);
                    if (steps > it.step_lo) {
                        // The scores of the first step.
                        ok = wait(MLA_BAR(k_full) + 8 * (step & 1), (step >> 1) & 1, bars, p.status,
                                  kSiteRing);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!ok || it.step_hi[t] <= it.step_lo) continue;
                            ok = wait(MLA_BAR(q_full) + 8 * t, q_uses[t] & 1, bars, p.status,
                                      kSiteQ);
                            ++q_uses[t];
                            if (!ok) continue;
                            ptx::tc_fence_after();
                            scores(t, step);
                            if (it.step_hi[t] == it.step_lo + 1)
                                ptx::mma_commit(MLA_BAR(q_empty) + 8 * t);
                        }
                        if (ok) ptx::mma_commit(MLA_BAR(k_empty) + 8 * (step & 1));
                    }
                    // Per step: P.V of the step and the scores of the next,
                    // tile after tile.
                    for (int j = it.step_lo; j < steps && ok; ++j, ++step) {
                        bool have_v = false, have_k = false;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!ok) continue;
                            if (j < it.step_hi[t]) {
                                ok = wait(MLA_BAR(p_ready) + 8 * t, p_uses[t] & 1, bars, p.status,
                                          kSiteP);
                                if (!have_v)
                                    ok = ok && wait(MLA_BAR(v_full) + 8 * (step & 1),
                                                    (step >> 1) & 1, bars, p.status, kSiteRing);
                                if (!ok) continue;
                                have_v = true;
                                ++p_uses[t];
                                ptx::tc_fence_after();
                                values(t, step, j == it.step_lo);
                            }
                            if (t == 1) ptx::mma_commit(MLA_BAR(v_empty) + 8 * (step & 1));
                            if (j + 1 < it.step_hi[t]) {
                                if (!have_k)
                                    ok = wait(MLA_BAR(k_full) + 8 * ((step + 1) & 1),
                                              ((step + 1) >> 1) & 1, bars, p.status, kSiteRing);
                                if (!ok) continue;
                                have_k = true;
                                ptx::tc_fence_after();
                                scores(t, step + 1);
                                if (j + 2 == it.step_hi[t])
                                    ptx::mma_commit(MLA_BAR(q_empty) + 8 * t);
                            }
                        }
                        if (ok && j + 1 < steps)
                            ptx::mma_commit(MLA_BAR(k_empty) + 8 * ((step + 1) & 1));
                    }
                    items.release();
                }
                // Every MMA issued above has completed before TMEM is freed.
                ptx::mma_commit(MLA_BAR(drain));
                wait(MLA_BAR(drain), 0, bars, p.status, kSiteDrain, true);
            }
            __syncwarp();
        } else if (warp == 10) {
            // ------------------------------------------------------ helper
            uint32_t step = 0, raws = 0;
            bool ok = true;
            while (ok) {
                ok = __all_sync(0xffffffffu, items.next(bars, p.status, &it));
                if (!ok || it.head < 0) break;
                const int steps = max(it.step_hi[0], it.step_hi[1]);
                step += uint32_t(min(it.fix_from, steps) - it.step_lo);
                for (int j = it.fix_from; j < steps; ++j, ++step, ++raws) {
                    ok = __all_sync(0xffffffffu,
                                    wait(MLA_BAR(raw_full) + 8 * (raws & 1), (raws >> 1) & 1, bars,
                                         p.status, kSiteRaw));
                    if (!ok) break;
                    const int end = it.lk - j * kStep;      // rows of the step that exist
                    // 0 x + sum: NaN as soon as one x is a NaN or an infinity.
                    uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        // Two 64 x 64 boxes of 128-byte rows; a row is 8 pieces of 16 bytes.
                        uint4* v = reinterpret_cast<uint4*>(
                            smem + kOffRing + ((5 * step + 3 + c) % kRing) * kBlock);
                        const bool cut = end < 64 * (c + 1);
#pragma unroll 1
                        for (int k0 = lane; k0 < kBlock / 16; k0 += 8 * 32) {
                            uint4 x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = v[k0 + 32 * i];
                            if (cut) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (64 * c + (((k0 + 32 * i) >> 3) & 63) >= end)
                                        v[k0 + 32 * i] = x[i] = make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                add_zero_times(x[i].x, &sum[0]);
                                add_zero_times(x[i].y, &sum[1]);
                                add_zero_times(x[i].z, &sum[2]);
                                add_zero_times(x[i].w, &sum[3]);
                            }
                        }
                    }
                    // (the sums are +-0 or NaN)
                    const uint32_t any = (sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu;
                    const bool bad = any != 0;
                    if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t* v = reinterpret_cast<uint32_t*>(
                                smem + kOffRing + ((5 * step + 3 + c) % kRing) * kBlock);
#pragma unroll 1
                            for (int k = lane; k < kBlock / 4; k += 32) {
                                uint32_t x = v[k];
                                if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                                if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
                                v[k] = x;
                            }
                        }
                        if (lane == 0) bars->bad_item[items.n % kItemSlots] = int32_t(items.n);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(MLA_BAR(v_full) + 8 * (step & 1));
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(MLA_BAR(item_empty) + 8 * (items.n % kItemSlots));
                ++items.n;
            }
        } else {
            // --------------------------------------------------- scheduler
            const Order order = count_tiles(p);
            const Units units(p, order);
            const int64_t total = units.count();
            if (p.split_rest && blockIdx.x == 0 && lane == 0) {   // for the merge
                p.rest[0] = int(units.total - units.whole);
                p.rest[1] = units.splits;
            }
            uint32_t n = 0;
            while (true) {
                // The next item of all CTAs. A CTA holds two at most, the one
                // it works on and the one its loads run ahead to. The first
                // ones need no ticket.
                const uint32_t s = n % kItemSlots, turn = n / kItemSlots;
                const bool ok = (n == 0 || wait(MLA_BAR(item_near), (n - 1) & 1, bars, p.status,
                                                kSiteItemFree)) &&
                                (turn == 0 || wait(MLA_BAR(item_empty) + 8 * s, (turn - 1) & 1,
                                                   bars, p.status, kSiteItemFree));
                if (!__all_sync(0xffffffffu, ok)) break;
                unsigned long long drawn = blockIdx.x;
                if (n > 0) {
                    if (lane == 0) drawn = gridDim.x + atomicAdd(p.ticket, 1ull);
                    drawn = __shfl_sync(0xffffffffu, drawn, 0);
                }
                const int64_t index = int64_t(drawn);
                const bool more = index < total;
                Item next;
                next.head = -1;
                if (more) next = find_item(p, index, order, units);
                if (lane == 0) {
                    bars->items[s] = next;
                    ptx::mbar_arrive(MLA_BAR(item_full) + 8 * s);
                }
                __syncwarp();
                ++n;
                if (!more) break;
            }
        }
    } else {
        // ------------------------------------------------ softmax, epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int t = warp >> 2;
        const int row = (warp & 3) * 32 + lane;            // of the tile, = TMEM lane
        const uint32_t ts = tmem + kTmemS + 128 * t + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t to = tmem + kTmemO + 128 * t + (uint32_t((warp & 3) * 32) << 16);
        uint32_t s_uses = 0;
        bool ok = true;
        while (ok) {
            ok = __all_sync(0xffffffffu, items.next(bars, p.status, &it));
            if (!ok || it.head < 0) break;
            const int in_item = t * kTileRows + row;
            const int limit = p.causal ? min(it.limit0 + in_item, it.lk - 1) : it.lk - 1;
            float m = -INFINITY, sum = 0.f;
            const int hi = t == 0 ? it.step_hi[0] : it.step_hi[1];
            for (int j = it.step_lo; j < hi; ++j) {
                ok = __all_sync(0xffffffffu, wait(MLA_BAR(s_full) + 8 * t, s_uses & 1, bars,
                                                  p.status, kSiteS));
                if (!ok) break;
                ++s_uses;
                ptx::tc_fence_after();
                const int seen = limit - j * kStep + 1;     // keys of the step this row sees
                if (__any_sync(0xffffffffu, seen < kStep)) {
                    // Scores of other keys become -inf in TMEM, in a rolled
                    // loop over the columns that need it. (Compares and
                    // selects of all 128 in registers are 4 KB of code that is
                    // run once or twice an item, and not in the instruction
                    // cache by then: 1,400-3,400 clocks against 300-1,400. 24
                    // prompts of 2 to 886 tokens, 16 heads: 73.3 -> 69.9 us.)
                    const int least = __reduce_min_sync(0xffffffffu, max(seen, 0));
#pragma unroll 1
                    for (int c = least & ~31; c < kStep; c += 32) {
                        uint32_t x[32];
                        ptx::tmem_ld32(ts + c, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = i < seen - c ? x[i] : 0xff800000u;
                        ptx::tmem_st32(ts + c, x);
                    }
                }
                float v[128];
                tmem_ld128(ts, v);
                float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int c = 4; c < 124; c += 8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m4[i] = ptx::fmax3(m4[i], v[c + i], v[c + 4 + i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], v[124 + i]);
                const float m_new = fmaxf(fmaxf(m, ptx::fmax3(m4[0], m4[1], m4[2])), m4[3]);
                // (what a row does follows from its own scores alone, so that its
                // result does not depend on the other rows of the warp)
                const bool grown = (m_new - m) * p.scale_log2 > kRescaleThreshold;
                if (j == it.step_lo) {
                    m = m_new;
                } else if (__any_sync(0xffffffffu, grown)) {
                    // (m = -inf: no key seen so far, O and the sum are 0)
                    const float alpha =
                        grown && m != -INFINITY ? ptx::ex2((m - m_new) * p.scale_log2) : 1.f;
                    if (grown) m = m_new;
                    sum *= alpha;
                    ok = __all_sync(0xffffffffu, wait(MLA_BAR(pv_done) + 8 * t, s_uses & 1, bars,
                                                      p.status, kSitePv));
                    if (!ok) break;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kV; c += 32) {
                        uint32_t o[32];
                        ptx::tmem_ld32(to + c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        ptx::tmem_st32(to + c, o);
                    }
                }
                // One FMA per weight, 2^(v c - fl(m c)); its exponent is off by
                // the rounding of m c, |m c| 2^-24 at most. Where that could
                // count (2^-14 at 1024; an overflow at 2^31) m is taken off
                // the scores first (rare, so it is a small loop as well).
                float shift = m == -INFINITY ? 0.f : -m * p.scale_log2;
                const bool far = fabsf(shift) > 1024.f;
                if (__any_sync(0xffffffffu, far)) {
                    const float base = far ? m : 0.f;
#pragma unroll 1
                    for (int c = 0; c < kStep; c += 32) {
                        uint32_t x[32];
                        ptx::tmem_ld32(ts + c, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) - base);
                        ptx::tmem_st32(ts + c, x);
                    }
                    tmem_ld128(ts, v);
                    if (far) shift = 0.f;
                }
                const uint64_t scale2 = pack_f32(p.scale_log2, p.scale_log2);
                const uint64_t shift2 = pack_f32(shift, shift);
                uint64_t part[2] = {0, 0};                  // two pairs of sums
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float a, b;
                        unpack_f32(fma_f32x2(pack_f32(v[g * 64 + 2 * i], v[g * 64 + 2 * i + 1]),
                                             scale2, shift2), &a, &b);
                        a = ptx::ex2(a);
                        b = ptx::ex2(b);
                        part[i & 1] = add_f32x2(part[i & 1], pack_f32(a, b));
                        w[i] = pack_bf16(a, b);
                    }
                    ptx::tmem_st32(ts + 32 * g, w);
                }
                float part_a, part_b;
                unpack_f32(add_f32x2(part[0], part[1]), &part_a, &part_b);
                sum += part_a + part_b;
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(MLA_BAR(p_ready) + 8 * t);
            }
            if (!ok) break;
            // Epilogue.
            bool repair = false;
            if (hi > it.step_lo) {
                ok = __all_sync(0xffffffffu, wait(MLA_BAR(pv_done) + 8 * t, (s_uses - 1) & 1, bars,
                                                  p.status, kSitePv));
                if (!ok) break;
                ptx::tc_fence_after();
                // (the last P.V waited for the helper, so its word is there)
                if (hi > it.fix_from)
                    repair = *reinterpret_cast<volatile int32_t*>(
                                 &bars->bad_item[items.n % kItemSlots]) == int32_t(items.n);
            }
            const bool mine = in_item < it.q_rows;
            const float inv = sum != 0.f ? 1.f / sum : 0.f;   // (a NaN sum stays NaN)
            const int64_t out_row = int64_t(it.q_row + in_item) * p.heads + it.head;
            const int64_t part_row = it.part_row + int64_t(in_item) * it.part_stride;
            if (mine) {
                const float lse =
                    sum == 0.f ? -INFINITY : m * (p.scale_log2 * kLn2) + logf(sum);
                if (it.part_stride != 0)
                    p.lse_part[part_row] = lse;
                else if (p.lse != nullptr)
                    p.lse[out_row] = lse;
            }
            if (it.part_stride != 0 && p.split_rest) p.rest_rows[part_row] = mine ? out_row : -1;
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < kV; c += 32) {
                uint32_t o[32];
                if (hi > it.step_lo) {
                    ptx::tmem_ld32(to + c, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0;
                }
                if (mine) {
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
                    if (repair) {
                        // The values the helper took out of the product, for
                        // the keys this row sees, times their weight: an
                        // infinity whose weight is 0 in fp32 gives NaN, as it
                        // does in the product.
                        const int last = min(limit, hi * kStep - 1);
#pragma unroll 1
                        for (int k = it.fix_from * kStep; k <= last; ++k) {
                            const uint4* vr = reinterpret_cast<const uint4*>(
                                p.kv + (int64_t(it.k_row + k) * p.heads + it.head) * kKvHead +
                                128 + c);
                            uint32_t u[16];
                            bool any = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint4 x = __ldg(vr + i);
                                u[4 * i] = x.x;
                                u[4 * i + 1] = x.y;
                                u[4 * i + 2] = x.z;
                                u[4 * i + 3] = x.w;
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                any = any || (u[i] & 0x7f80u) == 0x7f80u ||
                                      (u[i] & 0x7f800000u) == 0x7f800000u;
                            if (!any) continue;
                            const float w = ptx::ex2((score(p, out_row, it.k_row + k, it.head) - m) *
                                                     p.scale_log2);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if ((u[i] & 0x7f80u) == 0x7f80u)
                                    f[2 * i] += w * __uint_as_float(u[i] << 16);
                                if ((u[i] & 0x7f800000u) == 0x7f800000u)
                                    f[2 * i + 1] += w * __uint_as_float(u[i] & 0xffff0000u);
                            }
                        }
                    }
                    if (it.part_stride != 0) {
                        float* dst = p.o_part + part_row * kV + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(f[i + k]);
                            ptx::st_global_v8(dst + i, w);
                        }
                    } else {
                        uint16_t* dst = p.out + out_row * kV + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                w[k] = pack_bf16(f[i + 2 * k], f[i + 2 * k + 1]);
                            ptx::st_global_v8(dst + i, w);
                        }
                    }
                }
                __syncwarp();
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(MLA_BAR(item_empty) + 8 * (items.n % kItemSlots));
            ++items.n;
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 9) ptx::tmem_dealloc(tmem, 512);
    // The last CTA leaves the ticket at 0 for the next call.
    if (threadIdx.x == 0 && atomicAdd(p.done, 1u) == gridDim.x - 1) {
        *p.ticket = 0;
        *p.done = 0;
    }
#undef MLA_BAR
}

// One row's n partial rows, `stride` rows apart, into the result, with the
// identity of mla_merge_splits. A warp, four columns per lane.
__device__ __forceinline__ void merge_row(const PrefillParams& p, int64_t row, int64_t first,
                                          int64_t stride, int n) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int s = 0; s < n; ++s) m = fmaxf(m, p.lse_part[first + s * stride]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float z = 0.f;
    for (int s = 0; s < n; ++s) {
        const float l = p.lse_part[first + s * stride];
        if (l == -INFINITY) continue;
        const float w = expf(l - m);   // (NaN where a partial is NaN)
        const float4 v = *reinterpret_cast<const float4*>(
            p.o_part + (first + s * stride) * kV + lane * 4);
        z += w;
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
    }
    const float inv = z != 0.f ? 1.f / z : 0.f;
    uint2 o;
    o.x = pack_bf16(acc.x * inv, acc.y * inv);
    o.y = pack_bf16(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(p.out + row * kV + lane * 4) = o;
    if (lane == 0 && p.lse != nullptr) p.lse[row] = z == 0.f ? -INFINITY : m + logf(z);
}

// Every item was split: one warp per (row, head); only rows that a sequence
// holds are written.
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillParams p) {
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= int64_t(p.total_q) * p.heads) return;
    // The row's sequence: the last b with cu_q[b] <= q.
    const int q = int(row / p.heads);
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_q[mid] <= q) lo = mid; else hi = mid;
    }
    const int begin = p.cu_q[lo], end = p.cu_q[lo + 1];
    if (begin < 0 || q < begin || q >= end || end > p.total_q) return;
    merge_row(p, row, row * p.splits, 1, p.splits);
}

// The items of the last wave were split: one warp per row of the most items
// there can be. (What the tensor kernel left is checked against what there is
// room for: after an expired wait it may be an earlier call's.)
__global__ void __launch_bounds__(256) prefill_merge_rest_kernel(const PrefillParams p) {
    const int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int item = int(i / kItemRows), splits = p.rest[1];
    if (item >= p.rest[0] || splits < 1 || int64_t(p.rest[0]) * splits > p.rest_parts) return;
    const int64_t first = int64_t(item) * splits * kItemRows + i % kItemRows;
    const int64_t row = p.rest_rows[first];
    if (row < 0 || row >= int64_t(p.total_q) * p.heads) return;
    merge_row(p, row, first, kItemRows, splits);
}

// The tensor kernel.
int launch_prefill_tiles(PrefillParams p, int num_sms, cudaStream_t st) {
    const int64_t head_bytes = int64_t(p.total_k) * kKvHead * 2;
    const int64_t group = head_bytes > 0 ? kGroupBytes / head_bytes : p.heads;
    p.group = group < 1 ? 1 : group > p.heads ? p.heads : int(group);
    // (Without keys the maps over them are never read through; the queries
    // stand in.)
    CUtensorMap mq, mkv, mpe;
    const void* kv_base = p.total_k > 0 ? p.kv : p.q;
    const void* pe_base = p.total_k > 0 ? p.k_pe : p.q;
    const uint64_t k_rows = p.total_k > 0 ? uint64_t(p.total_k) : 1;
    const uint64_t kv_cols = p.total_k > 0 ? uint64_t(p.heads) * kKvHead : 64;
    if (!encode_2d(&mq, p.q, uint64_t(p.heads) * kQk, uint64_t(p.total_q), kTileRows) ||
        !encode_2d(&mkv, kv_base, kv_cols, k_rows, kStep / 2) ||
        !encode_2d(&mpe, pe_base, kRope, k_rows, kStep))
        return int(cudaErrorInvalidValue);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared_memory(mla_prefill_kernel, kSmemBytes, &allowed);
    if (e != cudaSuccess) return int(e);
    const int64_t most = (int64_t(p.total_q) / kItemRows + p.batch) * p.heads * p.splits;
    const unsigned grid = unsigned(most < num_sms ? most : num_sms);
    mla_prefill_kernel<<<grid, kThreads, kSmemBytes, st>>>(p, mq, mkv, mpe);
    return int(cudaGetLastError());
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

uint64_t round256(uint64_t x) { return (x + 255) / 256 * 256; }

// A split should have at least this many key steps: fewer cost more in items
// and merging than the extra CTAs bring.
constexpr int kMinSplitSteps = 4;
// Parts of the items of a last, partly filled wave, and the waves up to which
// they are planned: with more of them the wave counts for less (3 sequences of
// 512 rows over 8,000 keys, 128 heads, 5.1 waves: 675 -> 608 us; 6 over 3,000
// keys, 10.1 waves: 500 -> 478 us; 4 of 1,024 rows over 4,000 keys, 118 heads,
// 12.4 waves: 721 and 725 us).
constexpr int kRestSplits = 4;
constexpr int kRestWaves = 6;
// The single-row kernel: CTAs an SM that its splits aim at, and the fewest
// keys of a split.
constexpr int kRowCtasPerSm = 4;
constexpr int kMinSplitKeys = 128;

// What a split call keeps in its workspace, by byte offset: fp32 rows of
// partial results, their LSEs and (split_rest) the result rows they belong to.
struct Partials {
    uint64_t rows, lse, rest_rows, end;
    int64_t rest_parts;
};

// All items split: S partial rows per (query, head). Only those of the last
// wave split: 256 rows for each of its parts, of which there is one per CTA at
// most, whatever the number of queries (512 rows of 3 sequences, 128 heads: 20
// MB, where S rows for every query are 406).
Partials partials(const mla_prefill_plan_t& p, bool rest) {
    Partials l{};
    l.rows = l.lse = l.rest_rows = l.end = kStatusBytes;
    if (p.num_kv_splits <= 1 || p.single_rows) return l;
    uint64_t rows = uint64_t(p.total_q) * p.num_heads * p.num_kv_splits;
    if (rest) {
        const int64_t most =
            (int64_t(p.total_q) / kItemRows + p.batch) * p.num_heads * p.num_kv_splits;
        l.rest_parts = most < p.num_sms ? most : p.num_sms;
        rows = uint64_t(l.rest_parts) * kItemRows;
    }
    l.lse = l.rows + round256(rows * kV * 4);
    l.rest_rows = l.lse + round256(rows * 4);
    l.end = l.rest_rows + (rest ? round256(rows * 8) : 0);
    return l;
}

// The workspace of a plan. One that splits all items has room for the other
// way too, so that a caller may set split_rest on it.
void layout(mla_prefill_plan_t* p) {
    const Partials l = partials(*p, p->split_rest != 0), other = partials(*p, true);
    p->partial_offset = l.rows;
    p->lse_partial_offset = l.lse;
    p->workspace_bytes = l.end > other.end ? l.end : other.end;
}

bool same_layout(const mla_prefill_plan_t& a, const mla_prefill_plan_t& b) {
    return a.partial_offset == b.partial_offset && a.lse_partial_offset == b.lse_partial_offset &&
           a.workspace_bytes == b.workspace_bytes;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_prefill_plan(int batch, int num_heads, int total_q, int max_q_len,
                                int max_k_len, int num_kv_splits, int num_sms,
                                mla_prefill_plan_t* plan) {
    if (!plan || batch < 0 || num_heads < 1 || total_q < 0 || max_q_len < 0 || max_k_len < 0 ||
        num_kv_splits < 0 || num_sms < 1)
        return MLA_ERR_INVALID_ARG;
    if (num_heads > kMaxHeads || num_kv_splits > kMaxSplits) return MLA_ERR_UNSUPPORTED;
    mla_prefill_plan_t p;
    std::memset(&p, 0, sizeof(p));
    p.batch = batch;
    p.num_heads = num_heads;
    p.total_q = total_q;
    p.num_sms = num_sms;
    p.num_kv_splits = num_kv_splits;
    // One query row a sequence: HBM is the bound. (Measured with the keys in
    // HBM, tensor kernel against single-row kernel: 8 sequences of 816 keys, 16
    // heads, one row each 21.5 and 14.2 us, two 21.8 and 21.2, three 20.4 and
    // 28.9; 64 of 2,048 keys, 16 heads, one row 203 and 166 us, two 205 and 246;
    // 4 of 2,048 keys, 128 heads, one row 106 and 83 us, two 106 and 125.)
    p.single_rows = max_q_len <= 1 ? 1 : 0;
    if (num_kv_splits == 0) {
        const int rows = p.single_rows ? 1 : kItemRows;
        const int64_t per_seq = (int64_t(max_q_len) + rows - 1) / rows;
        int64_t tiles = batch * per_seq;
        const int64_t bound = int64_t(total_q) / rows + batch;
        if (tiles > bound) tiles = bound;
        const int64_t items = tiles * num_heads;
        // Split while every item finds room for S parts: of the tensor
        // kernel's one CTA per SM, of the other's kRowCtasPerSm. (So items for
        // more than half of the SMs are not split, and the other SMs are idle:
        // 1,280 rows over 30,000 keys, 16 heads, 80 items, 404 us, where a
        // caller's S = 3, in one and a half waves, takes 288.)
        const int64_t slots = p.single_rows ? int64_t(num_sms) * kRowCtasPerSm : num_sms;
        const int64_t most =
            p.single_rows ? max_k_len / kMinSplitKeys : max_k_len / (kStep * kMinSplitSteps);
        int64_t s = items > 0 ? slots / items : 1;
        if (s > most) s = most;
        if (s > kMaxSplits) s = kMaxSplits;
        p.num_kv_splits = s < 1 ? 1 : int(s);
        // Few waves of long items, the last one not half full: it is split.
        // (80 heads, 512 rows over 8,000 keys, 160 items: 224 -> 150 us; 90 heads
        // over 3,000 keys 92 -> 73 us. Where shorter items fill the wave anyway
        // it costs up to 5%, 101.7 -> 104.9 us for 160 items of 700 and 300 rows.)
        const int64_t rest = items % slots;
        if (!p.single_rows && items > slots && items < slots * kRestWaves &&
            most >= kRestSplits && rest > 0 && rest * 2 <= slots) {
            p.num_kv_splits = kRestSplits;
            p.split_rest = 1;
        }
    }
    if (p.single_rows) {
        // The splits are a cluster: 1, 2, 4 or 8.
        int s = 1;
        while (2 * s <= p.num_kv_splits && s < kMaxRowSplits) s *= 2;
        p.num_kv_splits = s;
    }
    layout(&p);
    *plan = p;
    return MLA_OK;
}

extern "C" int mla_prefill(const mla_prefill_plan_t* plan, const void* q, const void* kv,
                           const void* k_pe, int total_k, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, int causal, float softmax_scale, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (!plan) return MLA_ERR_INVALID_ARG;
    if (plan->batch < 0 || plan->num_heads < 1 || plan->num_heads > kMaxHeads ||
        plan->total_q < 0 || plan->num_kv_splits < 1 || plan->num_kv_splits > kMaxSplits ||
        plan->num_sms < 1 || (plan->single_rows & ~1) != 0 || (plan->split_rest & ~1) != 0 ||
        (plan->split_rest != 0 && plan->single_rows != 0) || total_k < 0)
        return MLA_ERR_INVALID_ARG;
    if (plan->single_rows &&
        (plan->num_kv_splits > kMaxRowSplits || (plan->num_kv_splits & (plan->num_kv_splits - 1))))
        return MLA_ERR_INVALID_ARG;
    mla_prefill_plan_t check = *plan;
    layout(&check);
    const bool as_planned = same_layout(*plan, check);
    if (!as_planned) {               // split_rest may have been changed since
        check.split_rest = 1 - plan->split_rest;
        layout(&check);
        if (!same_layout(*plan, check)) return MLA_ERR_INVALID_ARG;
    }
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (!(scale_log2 > 0.f) || !std::isfinite(scale_log2)) return MLA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < plan->workspace_bytes || !aligned(workspace, 256))
        return MLA_ERR_WORKSPACE;
    if (plan->batch == 0 || plan->total_q == 0) return MLA_OK;
    if (!q || !out || !cu_seqlens_q || !cu_seqlens_k || (total_k > 0 && (!kv || !k_pe)))
        return MLA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(k_pe, 16) || !aligned(out, 32) ||
        (lse && !aligned(lse, 4)) || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
        return MLA_ERR_INVALID_ARG;
    PrefillParams p{};
    char* ws = static_cast<char*>(workspace);
    p.q = static_cast<const uint16_t*>(q);
    p.kv = static_cast<const uint16_t*>(kv);
    p.k_pe = static_cast<const uint16_t*>(k_pe);
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.batch = plan->batch;
    p.heads = plan->num_heads;
    p.total_q = plan->total_q;
    p.total_k = total_k;
    p.causal = causal ? 1 : 0;
    // (split_rest cleared: there is room for the last wave's parts only, so no
    // keys are cut)
    p.splits = as_planned || plan->split_rest ? plan->num_kv_splits : 1;
    p.split_rest = p.splits > 1 ? plan->split_rest : 0;
    const Partials parts = partials(*plan, p.split_rest != 0);
    p.scale_log2 = scale_log2;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.o_part = reinterpret_cast<float*>(ws + parts.rows);
    p.lse_part = reinterpret_cast<float*>(ws + parts.lse);
    p.rest_rows = reinterpret_cast<int64_t*>(ws + parts.rest_rows);
    p.rest = reinterpret_cast<int32_t*>(ws + 4 * kRestWord);
    p.rest_parts = int(parts.rest_parts);
    p.status = reinterpret_cast<int32_t*>(ws);
    p.ticket = reinterpret_cast<unsigned long long*>(ws + 4 * kTicketWord);
    p.done = reinterpret_cast<uint32_t*>(ws + 4 * kDoneCtasWord);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int e = plan->single_rows ? launch_prefill_row(p, plan->num_sms, stream)
                                    : launch_prefill_tiles(p, plan->num_sms, st);
    if (e != 0) return MLA_ERR_CUDA;
    if (p.splits > 1 && !plan->single_rows) {
        // (an item that is split has two parts or more)
        const int64_t rows = p.split_rest ? int64_t(p.rest_parts / 2) * kItemRows
                                          : int64_t(p.total_q) * p.heads;
        if (rows == 0) return MLA_OK;     // (one part in all: nothing can be split)
        (p.split_rest ? prefill_merge_rest_kernel
                      : prefill_merge_kernel)<<<unsigned((rows + 7) / 8), 256, 0, st>>>(p);
        if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
    }
    return MLA_OK;
}
