// Attention of the items of mla_decode_shared and mla_decode_window
// (mla_span.cuh): rows of absorbed queries over the pages of a latent cache.
//
//   s[t] = softmax_scale q . K[t], out = sum_t exp(s[t] - lse) V[t],
//   K[t] the 576-wide entry, V[t] its first 512 columns.
//
// 128 rows against a page pair are 2 * 128 * 128 * (576 + 512) flops for 147 KB
// of cache: the tensor pipe and HBM take about the same time, and a prefix
// that many tiles share is in L2, so the tensor pipe is the bound. 128 rows
// of 512 fp32 results are all of one SM's TMEM. So a pair of CTAs works on an
// item with cta_group::2 MMAs of M = 128: each CTA holds 64 of the rows, and
// TMEM lanes 0..63 and 64..127 of a CTA hold those rows' first and second half
// of an MMA's columns. Nothing is computed twice:
//   * Scores: N = 128, the two pages of a step, one from each CTA's shared
//     memory; lanes 64 f + r get row r's scores of page f. Two buffers.
//   * P V: K = 128 tokens; CTA f holds value columns 256 f .. 256 f + 255 of
//     both pages, so lanes 64 f + r get those columns of row r (256 TMEM
//     columns).
// A CTA's own page arrives whole (nine 64-column blocks). Of its blocks the
// four of the other CTA's value columns are done with after the scores, and
// the other page's blocks of its own value columns take their slots: slots
// 0..3 hold the first page's values in both CTAs then, slots 4..7 the second
// page's, at the same addresses in both, as the MMAs need it. Two such stages
// of eight slots, one slot for the RoPE block, the queries (72 KB) and the
// weights (16 KB) fill an SM. Each pair of slots is loaded again as soon as
// the P V MMAs that read it are done.
//
// Softmax: a thread has 64 scores of a row; the two threads of a row exchange
// their maxima through shared memory. fp32, base 2; the reference maximum moves
// only when a step raises it by more than 8, so that results are seldom
// rescaled. Weights are rounded to bf16 for the tensor cores, or to f16 with an
// fp8 cache: by half a step, 2^-8 or 2^-11, of each weight, in f16 by up to 2^-32 of
// the row's greatest. Results are normalised by the sum of the rounded weights,
// the LSE keeps the sum of the others.
//
// What the weights' barrier announces to the first CTA's MMA thread lies in the
// announcing SM: shared memory, written before a proxy fence and read by that
// SM's tensor core, and TMEM. So its arrivals release at CTA scope (at cluster
// scope each took 1,400 cycles, and a step 3,850).
//
// An fp8 cache: thirteen warps load the codes into registers and widen them into
// the slots (exact).
//
// Measured, calls one behind the other in a graph: 64 requests of 128 heads over
// a prefix of 16,384 tokens and 100 to 1,500 of their own (308 GFLOP) 205 us,
// 1,500 TFLOP/s; a step takes 2,900 cycles in a short call and 3,100 to 3,600 in a
// long one, of which the MMAs need 2,176; the operands that they read and the
// tiles that TMA writes take shared memory for 2,750 (128 bytes a cycle). With an
// fp8 cache a step takes some 4,000: the same port, with 1,886 for the operands and
// 1,900 for the codes' way through L1 and registers and the weights; 64 requests
// of 32 heads over two prefixes of 8,000 to 12,000 tokens 73 us. 128 requests of
// 128 heads through a window of 1,024 tokens (177 MB) 57 to 59 us; small batches
// take 15 to 16 us: the schedule (2 to 3), the first page (2), a step or two,
// results (2), the merge (3).
//
// Registers: 201 a thread; 96 with an fp8 cache (19 warps), which spills 28 bytes.
//
// Warps: 1 = MMAs (first CTA), 2-5 = softmax and epilogue, 0 and 6 = loads (fp8
// cache: 0 = queries, 6-18 = codes). Every wait is bounded (MLA_ERR_TIMEOUT).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstddef>

#include "mla_span_schedule.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"

namespace mla {
namespace {

constexpr int kThreads = 224;
constexpr int kThreadsFp8 = 608;
constexpr int kCtaRows = 64;
constexpr int kBlock = 64 * 128;                  // 64 rows x 64 16-bit columns
constexpr int kStages = 2;
constexpr int kSlots = 8;
constexpr int kStageBytes = kSlots * kBlock;
constexpr int kOffQ = 0;                          // 9 blocks
constexpr int kOffStage = 9 * kBlock;
constexpr int kOffRope = kOffStage + kStages * kStageBytes;
constexpr int kOffP = kOffRope + kBlock;          // a block per page of the step
constexpr int kOffBar = kOffP + 2 * kBlock;       // 229,376
constexpr int kOffSwap = kOffBar + 512;           // 2 x 128 floats that rows' halves exchange
constexpr int kOffRange = kOffSwap + 2 * 128 * 4;
constexpr int kOffScale = kOffRange + int(sizeof(SpanRange));   // fp8 cache: 2 x 64 rows' scales
constexpr int kSmemBytes = kOffScale + 2 * kCtaRows * 4;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
static_assert(sizeof(SpanScratch) <= kOffBar, "the schedule is made where the operands go");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;                    // 2 x 64 columns
constexpr uint32_t kTmemO = 128;                  // 256 columns

constexpr uint32_t kSuspendNs = 20000;
constexpr uint16_t kBoth = 3;                     // the pair's CTAs
constexpr float kRescaleThreshold = 8.f;          // log2 units
// The weight of the reference (log2): f16 has no more than 2^-25 of a weight, 2^-32
// of the greatest with this, and up to 2^15 of it. bf16 has fp32's range.
template <bool kFp8>
constexpr float kLift = kFp8 ? 7.f : 0.f;
constexpr float kLn2 = 0.693147180559945309f;

enum SpanSite : int32_t { kSiteQ = 70, kSiteK, kSiteRope, kSiteV, kSiteSlot, kSiteQkDone,
                          kSiteP, kSitePv, kSiteStaged, kSiteDrain };

// Step j of a pair uses stage j & 1. Those marked L are used in the pair's
// first CTA only, the one that issues the MMAs.
struct Bars {
    uint64_t q_full;              // L: both CTAs' rows
    uint64_t k_full[2][4];        // L: slots 2g, 2g + 1 of both CTAs
    uint64_t rope_full;           // L
    uint64_t v_full[2];           // this CTA's value blocks of the other page
    uint64_t qk_part[2];          // the MMAs of slots 0..3 and of the RoPE block are done
    uint64_t s_full[2];           // all score MMAs of the step
    uint64_t pv_done[2][4];       // the P V MMAs that read slots 2g, 2g + 1; [3]: all of the step
    uint64_t p_ready;             // L: 2 x 4 warps: weights written, results rescaled
    uint64_t drain;               // L
    uint64_t q_staged;            // fp8 cache: the queries have landed as bf16
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, Bars* bars, int32_t* status,
                                       int32_t site, uint64_t limit_ns, bool ignore_abort) {
    volatile int32_t* abort = &bars->abort;
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        for (int i = 0; i < 4; ++i)
            if (ptx::mbar_try_wait_sleep(bar, parity, kSuspendNs)) return true;
        if (!ignore_abort && *abort != 0) return false;
        if (ptx::globaltimer() - t0 > limit_ns) {
            *abort = 1;
            record_error(status, MLA_ERR_TIMEOUT, site);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Bars* bars, int32_t* status,
                                     int32_t site, uint64_t limit_ns, bool ignore_abort = false) {
    if (ptx::mbar_test_wait(bar, parity)) return true;
    return wait_slow(bar, parity, bars, status, site, limit_ns, ignore_abort);
}

// Four MMAs of a pair of CTAs (M = 128: 64 rows of A and D in each, half of
// B's columns in each CTA's shared memory), K steps `sa` and `sb` apart.
__device__ __forceinline__ void mma4_pair(uint32_t d, uint64_t a, uint64_t sa, uint64_t b,
                                          uint64_t sb, uint32_t idesc, uint32_t acc0) {
    asm volatile(
        "{\n .reg .pred p;\n"
        " setp.ne.b32 p, %10, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %5, %9, p;\n"
        " setp.eq.b32 p, %10, %10;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %2, %6, %9, p;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %3, %7, %9, p;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %4, %8, %9, p;\n}\n"
        ::"r"(d), "l"(a), "l"(a + sa), "l"(a + 2 * sa), "l"(a + 3 * sa), "l"(b), "l"(b + sb),
          "l"(b + 2 * sb), "l"(b + 3 * sb), "r"(idesc), "r"(acc0)
        : "memory");
}

// ------------------------------------------------------------ a pair's work

struct Piece {
    SpanItem it;
    int first, steps;      // steps [first, first + steps) of the item
    int64_t part_row;      // -1: it writes the results
};

struct Walk {
    const SpanRange* range;
    int item, pair;
};

__device__ __forceinline__ bool walk_next(const SpanParams& p, Walk& w, Piece& pc) {
    const SpanRange& r = *w.range;
    while (w.item < r.end) {
        const int i = w.item++ - r.first;
        const int4* src = reinterpret_cast<const int4*>(i < kSpanKept ? r.kept + i
                                                                      : p.items + r.first + i);
        int4* dst = reinterpret_cast<int4*>(&pc.it);
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k] = src[k];
        // Its steps [first, first + steps) in the pair's units.
        const int s0 = pc.it.unit0 + kSpanItemCost;
        const int lo = max(s0, r.g0), hi = min(pc.it.unit1, r.g1);
        if (lo >= hi) continue;      // (of its units only the fixed cost)
        pc.first = lo - s0;
        pc.steps = hi - lo;
        pc.part_row = pc.it.alone && pc.it.first_pair == pc.it.last_pair
                          ? -1
                          : int64_t(pc.it.part_row) + int64_t(w.pair) * kSpanRows;
        return true;
    }
    return false;
}

__device__ __forceinline__ int real_page(const SpanItem& it, int v) {
    return v < it.head_pages ? v : v + it.page_shift;
}

// The tokens of virtual page v that are seen: rows [0, a) and [b, e).
struct PageMask {
    int a, b, e;
    __device__ __forceinline__ bool all() const {
        return e == kPageSize && (b <= 0 || a >= kPageSize || b <= a);
    }
    __device__ __forceinline__ bool sees(int i) const { return i < e && (i < a || i >= b); }
};
__device__ __forceinline__ PageMask page_mask(const SpanItem& it, int v) {
    if (v >= it.pages) return PageMask{0, 0, 0};
    const int t0 = real_page(it, v) * kPageSize;
    return PageMask{it.sink_end - t0, it.tail_lo - t0, min(it.end - t0, kPageSize)};
}

// The y coordinate of a page in the cache's tensor map; rows before the first
// one (which TMA fills with zeros) for one that is not there.
__device__ __forceinline__ int32_t page_row(const SpanParams& p, const SpanItem& it, int v,
                                            bool record) {
    if (v >= it.pages) return -kPageSize;
    const int page = p.table[int64_t(it.table_row) * p.max_blocks + real_page(it, v)];
    if (page < 0 || int64_t(page) >= p.num_blocks) {
        if (record) record_error(p.status, MLA_ERR_BAD_BLOCK_ID, page);
        return -kPageSize;
    }
    return page * kPageSize;
}

// A pair's steps, one after another over its pieces.
struct Steps {
    Walk w;
    Piece pc;
    int k;               // the step's number in its piece
    __device__ __forceinline__ Steps(const SpanRange* range, int pair)
        : w{range, range->first, pair} {
        pc.steps = 0;
        k = -1;
    }
    __device__ __forceinline__ bool next(const SpanParams& p) {
        if (++k < pc.steps) return true;
        k = 0;
        return walk_next(p, w, pc);
    }
    __device__ __forceinline__ bool first() const { return k == 0; }
    __device__ __forceinline__ int page() const { return kSpanStepPages * (pc.first + k); }
};

// ------------------------------------------------------------ loads
// Two threads: one loads queries and pages, the other RoPE blocks and the
// other page's value blocks, so that neither waits for what the other one
// waits for (with one thread for all, a page's slots, free in the middle of
// the P V MMAs, waited for the score MMAs: a step took 2,970 cycles).
struct Loader {
    const SpanParams& p;
    const CUtensorMap* map_q;
    const CUtensorMap* map_c;
    Bars* bars;
    uint32_t sbase, b0;
    int rank;
    uint64_t limit;

    __device__ __forceinline__ uint32_t bar(size_t off) const { return b0 + uint32_t(off); }
    __device__ __forceinline__ bool until(uint32_t b, uint32_t parity, int32_t site) const {
        return wait(b, parity, bars, p.status, site, limit);
    }
    // Phase n of a barrier that counts loads: they have landed.
    __device__ __forceinline__ void landed(uint32_t b, int n) const {
        wait(b, uint32_t(n) & 1, bars, p.status, kSiteDrain, limit, true);
    }
    // A box of 64 rows x 64 columns, an operand of the pair's MMAs: it counts on
    // a barrier of the first CTA, which alone announces both CTAs' bytes.
    __device__ __forceinline__ void box(const CUtensorMap* map, int to, int x, int32_t y,
                                        uint32_t bar) const {
        ptx::tma_load_2d_pair(sbase + uint32_t(to), map, x, y, ptx::map_to_rank(bar, 0));
    }
    __device__ __forceinline__ void expect(uint32_t bar, int blocks) const {
        if (rank == 0) ptx::mbar_arrive_expect_tx(bar, uint32_t(2 * blocks * kBlock));
    }

    __device__ __forceinline__ void pages(const SpanRange* range, int pair) const {
        const uint32_t q_full = bar(offsetof(Bars, q_full)), k_full = bar(offsetof(Bars, k_full));
        Steps s(range, pair);
        int pieces = 0, j = 0, part = 0;       // part: pairs of slots of step j asked for
        bool ok = true;
        for (; s.next(p); ++j) {
            const int32_t y = page_row(p, s.pc.it, s.page() + rank, true);
            if (s.first()) {
                // (the last scores of the piece before have been formed)
                ok = j == 0 || until(bar(offsetof(Bars, s_full)) + 8 * ((j - 1) & 1),
                                     ((j - 1) >> 1) & 1, kSiteQkDone);
                if (!ok) break;
                expect(q_full, 9);
                for (int k = 0; k < 9; ++k)
                    box(map_q, kOffQ + k * kBlock, 64 * k, s.pc.it.row0 + rank * kCtaRows, q_full);
                ++pieces;
            }
            const int st = j & 1;
            for (part = 0; part < 4; ++part) {
                const uint32_t off = uint32_t(8 * (4 * st + part));
                ok = j < 2 ||
                     until(bar(offsetof(Bars, pv_done)) + off, ((j >> 1) - 1) & 1, kSiteSlot);
                if (!ok) break;
                expect(k_full + off, 2);
                for (int i = 2 * part; i < 2 * part + 2; ++i)
                    box(map_c, kOffStage + st * kStageBytes + i * kBlock, 64 * i, y, k_full + off);
            }
            if (!ok) break;
        }
        // Every load asked for lands before the CTAs leave (the second CTA
        // leaves after the first, whose barriers count for both).
        if (rank != 0) return;
        if (pieces > 0) landed(q_full, pieces - 1);
        for (int i = j > 2 ? j - 2 : 0; i <= j; ++i)
            for (int g = 0; g < (i < j ? 4 : ok ? 0 : part); ++g)
                landed(k_full + 8 * (4 * (i & 1) + g), i >> 1);
    }

    // The first CTA: the second page's blocks 0..3 into slots 4..7; the second:
    // the first page's blocks 4..7 into slots 0..3.
    __device__ __forceinline__ void values(const SpanRange* range, int pair) const {
        const uint32_t r_full = bar(offsetof(Bars, rope_full)), v_full = bar(offsetof(Bars, v_full));
        const uint32_t v_free =
            rank == 0 ? bar(offsetof(Bars, s_full)) : bar(offsetof(Bars, qk_part));
        Steps s(range, pair);
        int ropes = 0, j = 0;
        int32_t other = 0, y[2] = {0, 0};
        auto rope = [&]() {
            if (ropes == 0 && (p.debug & kDebugWithholdLoad) != 0 && blockIdx.x == 0) return;
            expect(r_full, 1);
            box(map_c, kOffRope, kLkv, y[rank], r_full);
            ++ropes;
        };
        auto take = [&]() {
            const bool more = s.next(p);
            if (more) {
                y[0] = page_row(p, s.pc.it, s.page(), false);
                y[1] = page_row(p, s.pc.it, s.page() + 1, false);
            }
            return more;
        };
        // A window's pages come from HBM, whose answer takes longer than the two
        // stages cover: a step's page is pulled into L2 a step before its slots
        // are free (128 requests x 128 heads, window 1,024: 64 -> 58 us; two
        // steps before: 61; pages that requests share are in L2).
        Steps ahead(range, pair);
        bool far = p.window > 0;
        auto pull = [&]() {
            far = far && ahead.next(p);
            if (!far) return;
            const int32_t page = page_row(p, ahead.pc.it, ahead.page() + rank, false);
            if (page >= 0)
                ptx::prefetch_l2(static_cast<const uint16_t*>(p.cache) + int64_t(page) * kD,
                                 kPageSize * kD * 2);
        };
        far = far && ahead.next(p);
        bool more = take();
        if (more) rope();
        for (; more; ++j) {
            const int st = j & 1;
            const uint32_t ph = (j >> 1) & 1;
            other = y[1 - rank];
            pull();
            more = take();
            if (more) {
                if (!until(bar(offsetof(Bars, qk_part)) + 8 * st, ph, kSiteRope)) break;
                rope();
            }
            if (!until(v_free + 8 * st, ph, kSiteV)) break;
            ptx::mbar_arrive_expect_tx(v_full + 8 * st, uint32_t(4 * kBlock));
            for (int k = 0; k < 4; ++k)
                ptx::tma_load_2d(sbase + uint32_t(kOffStage + st * kStageBytes +
                                                  ((rank == 0 ? 4 : 0) + k) * kBlock),
                                 map_c, 256 * rank + 64 * k, other, v_full + 8 * st);
        }
        if (ropes > 0 && rank == 0) landed(r_full, ropes - 1);
        for (int i = j > 2 ? j - 2 : 0; i < j; ++i) landed(v_full + 8 * (i & 1), i >> 1);
    }
};

// ------------------------------------------------------------ fp8 widening

// Four codes as two pairs of f16 (exact).
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    uint2 h;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n"
        " cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
        : "=r"(h.x), "=r"(h.y)
        : "r"(w));
    return h;
}

// Two bf16 times a power of two as two f16.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float up = 1.f) {
    const __half2 v = __floats2half2_rn(__uint_as_float(w << 16) * up,
                                        __uint_as_float(w & 0xffff0000u) * up);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 bf16_to_f16(const uint4& v, float up = 1.f) {
    return make_uint4(bf16x2_to_f16x2(v.x, up), bf16x2_to_f16x2(v.y, up),
                      bf16x2_to_f16x2(v.z, up), bf16x2_to_f16x2(v.w, up));
}

// The greater magnitudes of two pairs of bf16 (a NaN is the greatest; signs mean
// nothing).
__device__ __forceinline__ uint32_t greater2(uint32_t m, uint32_t w) {
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
    return m;
}

// bf16 magnitudes: the greatest that f16 holds (65280), and 2^-4.
constexpr uint32_t kGreatestF16 = 0x477f, kSmallRow = (127 - 4) << 7;

// A query of that row is beyond f16. (A tile has its rows of requests without
// tokens too: nothing is computed for them, and they may hold anything.)
__device__ __noinline__ void range_error(const SpanParams& p, int row) {
    const int b = row / p.heads, L = p.seq_lens[b];
    if (L > 0 && int64_t(L) <= int64_t(p.max_blocks) * kPageSize)
        record_error(p.status, MLA_ERR_RANGE, b);
}

// Each of thirteen warps has a part as large as a 64-column block of every step (a
// page's eight, the RoPE block, four of the other page's value blocks): it holds
// the part's codes in registers, loaded while the slot was still in use, and
// widens them into the slot when that is free, so that between one use of a
// slot and the next there is no load, only the conversion. (Six warps that
// loaded codes into the slot by TMA and widened them in place: 6,500 cycles a
// step.)
struct Widener {
    const SpanParams& p;
    const CUtensorMap* map_q;
    Bars* bars;
    unsigned char* smem;
    uint32_t sbase, b0;
    int rank, lane;
    uint64_t limit;

    __device__ __forceinline__ uint32_t bar(size_t off) const { return b0 + uint32_t(off); }
    // One answer for the warp.
    __device__ __forceinline__ bool until(uint32_t b, uint32_t parity, int32_t site) const {
        return __all_sync(0xffffffffu, wait(b, parity, bars, p.status, site, limit));
    }
    // The writes before this are the tensor cores' to read.
    __device__ __forceinline__ void done(uint32_t to) const {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(to);
    }
    // A warp's codes of a page: 32 rows of 128 (two blocks), or 64 rows of 64
    // (the RoPE block). 16 codes a lane and load: a load of two blocks touches six
    // lines of 128 bytes; one of a block's rows, 576 bytes apart, eight (96 requests
    // of 32 heads through a window of 4,000 tokens: 63.7 us against 66.4).
    struct Part {
        int row, step;       // the lane's first row, and rows from one load to the next
        int column;          // and its first column
        int to;              // bytes from the first slot to the row's in its block
        int first, second;   // its two 16-byte pieces there (swizzled)
        int flip;            // what the swizzle does to them in every second load
        bool swapped;        // it stores the second one first (no bank conflicts)
    };
    __device__ __forceinline__ Part part(bool two, int half, int column) const {
        Part q;
        const int c = two ? lane & 7 : lane & 3;
        q.row = two ? 32 * half + (lane >> 3) : lane >> 2;
        q.step = two ? 4 : 8;
        q.column = column + 16 * c;
        q.to = (c >> 2) * kBlock + q.row * 128;
        q.swapped = c >= 4;
        const int piece = 2 * (c & 3) + (q.swapped ? 1 : 0);
        q.first = (piece ^ (q.row & 7)) * 16;
        q.second = q.first ^ 16;
        q.flip = two ? 64 : 0;
        return q;
    }
    // From row y of the cache; zeros for a page that is not there (y < 0). (Not
    // through the read-only path: this kernel starts while the one that writes the
    // cache may still run.)
    __device__ __forceinline__ void load(int32_t y, const Part& q, uint4 (&v)[8]) const {
        const unsigned char* src = static_cast<const unsigned char*>(p.cache) +
                                   (int64_t(y) + q.row) * kD + q.column;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = y >= 0 ? *reinterpret_cast<const uint4*>(src + k * q.step * kD)
                          : make_uint4(0, 0, 0, 0);
    }
    // Them as f16 in the swizzled layout.
    __device__ __forceinline__ void store(const uint4 (&v)[8], const Part& q, int at) const {
        unsigned char* row = smem + at + q.to;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t u0 = q.swapped ? v[k].z : v[k].x, u1 = q.swapped ? v[k].w : v[k].y;
            const uint32_t u2 = q.swapped ? v[k].x : v[k].z, u3 = q.swapped ? v[k].y : v[k].w;
            const uint2 a = widen4(u0), b = widen4(u1), d = widen4(u2), e = widen4(u3);
            unsigned char* to = row + k * q.step * 128;
            const int flip = (k & 1) ? q.flip : 0;
            *reinterpret_cast<uint4*>(to + (q.first ^ flip)) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4*>(to + (q.second ^ flip)) = make_uint4(d.x, d.y, e.x, e.y);
        }
    }

    // Warps 2 g and 2 g + 1: half of the rows of blocks 2 g and 2 g + 1 (0 .. 7) of
    // this CTA's page, 8: its RoPE block, 9 .. 12: likewise this CTA's value
    // columns of the other page.
    __device__ __forceinline__ void blocks(const SpanRange* range, int pair, int w) const {
        const bool own = w <= 8;
        const int two = own ? w >> 1 : (w - 9) >> 1;         // which two blocks
        const int slot = 2 * two + (own || rank != 0 ? 0 : 4);
        const Part q = part(w != 8, own ? w & 1 : (w - 9) & 1,
                            own ? 128 * two : 256 * rank + 128 * two);
        const int side = own ? rank : 1 - rank;
        Steps s(range, pair);
        uint4 v[8];
        bool more = s.next(p), first = true;
        int rows = 0, row0 = 0;
        uint32_t pieces = 0;
        int32_t y = -1;
        if (more) load(page_row(p, s.pc.it, s.page() + side, w == 0), q, v);
        for (int j = 0; more; ++j) {
            const int st = j & 1;
            const uint32_t ph = (j >> 1) & 1;
            if (first) {
                rows = s.pc.it.rows;
                row0 = s.pc.it.row0;
            }
            const bool begins = first;
            // The next step's page is looked up now, its codes are loaded below.
            more = s.next(p);
            first = more && s.first();
            if (more) y = page_row(p, s.pc.it, s.page() + side, w == 0);
            // (The stores are there once: the warps' code has to fit the
            // instruction caches.)
            uint32_t free_at = 0, free_ph = ph, to;
            int32_t site = kSiteV;
            int at = kOffStage + st * kStageBytes + slot * kBlock;
            if (w < 8) {
                const uint32_t off = uint32_t(8 * (4 * st + (w >> 1)));
                if (j >= 2) free_at = bar(offsetof(Bars, pv_done)) + off;
                free_ph = ph ^ 1;
                site = kSiteSlot;
                to = ptx::map_to_rank(bar(offsetof(Bars, k_full)) + off, 0);
            } else if (w == 8) {
                if (j > 0) free_at = bar(offsetof(Bars, qk_part)) + 8 * (st ^ 1);
                free_ph = ((j - 1) >> 1) & 1;
                site = kSiteRope;
                at = kOffRope;
                to = ptx::map_to_rank(bar(offsetof(Bars, rope_full)), 0);
                if (j == 0 && (p.debug & kDebugWithholdLoad) != 0 && blockIdx.x == 0) return;
            } else {
                free_at = (rank == 0 ? bar(offsetof(Bars, s_full)) : bar(offsetof(Bars, qk_part))) +
                          8 * st;
                to = ptx::map_to_rank(bar(offsetof(Bars, v_full)) + 8 * st, uint32_t(rank));
            }
            if (free_at != 0 && !until(free_at, free_ph, site)) return;
            store(v, q, at);
            done(to);
            if (more) load(y, q, v);
            // (The queries land after the codes, but for the first piece's.)
            if (w < 8 && begins) {
                if (!until(bar(offsetof(Bars, q_staged)), pieces & 1, kSiteStaged)) return;
                // (A range's pieces are of items one after another.)
                widen_queries(w, rows - rank * kCtaRows, row0 + rank * kCtaRows,
                              range->first + int(pieces++));
            }
        }
    }
    // An eighth of the queries, from bf16, in place: 16-byte pieces of rows 4 w + lane / 8
    // and 32 more, of each of the nine blocks. f16 has all of a bf16 number's bits
    // from 2^-17 to 65504 and loses 2^-25 at most of a smaller one, 2^-21 of a
    // row's greatest if that is 2^-4 or more. A row of smaller ones is read
    // again (the conversion above has rounded them) and multiplied by the power
    // of two that brings its greatest to [2^14, 2^15), 2^126 at most; its scores are
    // divided by that power (exactly, or to 2^-150, which the softmax scale makes
    // 2^-22 of at most). Looking for such rows costs nothing here, asking for
    // them in the softmax 0.7 us (64 requests of 32 heads over two prefixes 73.4 us
    // against 72.7, a window of 4,000 over 96 of them 64.6 against 64.0).
    __device__ __forceinline__ void widen_queries(int w, int live, int row0, int item) const {
        float* scales = reinterpret_cast<float*>(smem + kOffScale) + (item & 1) * kCtaRows;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            const int r = 32 * half + 4 * w + (lane >> 3);
            uint4* a = reinterpret_cast<uint4*>(smem + kOffQ) + 8 * r + (lane & 7);
            uint32_t m2 = 0;
#pragma unroll 3
            for (int k = 0; k < 9; ++k) {
                const uint4 v = a[k * (kBlock / 16)];
                m2 = greater2(greater2(greater2(greater2(m2, v.x), v.y), v.z), v.w);
                a[k * (kBlock / 16)] = bf16_to_f16(v);
            }
            uint32_t m = max(m2 & 0x7fffu, (m2 >> 16) & 0x7fffu);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            int up = 0;
            if (m != 0 && m < kSmallRow && r < live) {
                up = min(127 + 14 - int(m >> 7), 126);
                const uint16_t* q = p.q + int64_t(row0 + r) * kD + 8 * ((lane ^ r) & 7);
#pragma unroll 1
                for (int k = 0; k < 9; ++k)
                    a[k * (kBlock / 16)] = bf16_to_f16(*reinterpret_cast<const uint4*>(q + 64 * k),
                                                       __uint_as_float(uint32_t(127 + up) << 23));
            }
            if ((lane & 7) == 0) {
                scales[r] = copysignf(__uint_as_float(uint32_t(127 - up) << 23), p.scale_log2);
                if (m > kGreatestF16 && r < live) range_error(p, row0 + r);
            }
        }
        done(ptx::map_to_rank(bar(offsetof(Bars, q_full)), 0));
    }
    // One thread: a piece's queries, when the scores of the piece before it have
    // been formed. (It waits for every step in turn: a phase is told from the one
    // before the last by nothing.)
    __device__ __forceinline__ void queries(const SpanRange* range, int pair) const {
        const uint32_t staged = bar(offsetof(Bars, q_staged));
        Steps s(range, pair);
        int pieces = 0;
        for (int j = 0; s.next(p); ++j) {
            if (s.first()) {
                ptx::mbar_arrive_expect_tx(staged, 9 * kBlock);
                for (int k = 0; k < 9; ++k)
                    ptx::tma_load_2d(sbase + uint32_t(kOffQ + k * kBlock), map_q, 64 * k,
                                     s.pc.it.row0 + rank * kCtaRows, staged);
                ++pieces;
            }
            if (!wait(bar(offsetof(Bars, s_full)) + 8 * (j & 1), (j >> 1) & 1, bars, p.status,
                      kSiteQkDone, limit))
                break;
        }
        if (pieces > 0)
            wait(staged, uint32_t(pieces - 1) & 1, bars, p.status, kSiteDrain, limit, true);
    }
};

// A row's scores of a step times a factor, in TMEM. (Few calls come here: it is kept
// out of the softmax's code.)
__device__ __noinline__ void scale_scores(uint32_t at, float by) {
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        uint32_t o[32];
        ptx::tmem_ld32(at + uint32_t(c), o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
        ptx::tmem_st32(at + uint32_t(c), o);
    }
}

// ------------------------------------------------------------ the kernel

// The cache's tensor map. (An fp8 cache's codes are loaded by threads.)
template <bool kFp8>
struct CacheMap {
    CUtensorMap map;
};
template <>
struct CacheMap<true> {};

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFp8 ? kThreadsFp8 : kThreads, 1)
mla_span_kernel(const SpanParams p, const __grid_constant__ CUtensorMap map_q,
                const __grid_constant__ CacheMap<kFp8> cache) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
    const uint32_t b0 = sbase + kOffBar;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(ptx::cluster_ctarank());
    const int pair = blockIdx.x >> 1;
    auto bar = [&](size_t off) { return b0 + uint32_t(off); };

    if ((sbase & 1023u) != 0) {   // the swizzled tiles need it (the same in both CTAs)
        if (threadIdx.x == 0) record_error(p.status, MLA_ERR_UNSUPPORTED, 0);
        return;
    }
    if (threadIdx.x == 0) {
        // With an fp8 cache the widening warps of both CTAs announce operands.
        ptx::mbar_init(bar(offsetof(Bars, q_full)), kFp8 ? 2 * 8 : 1);
        ptx::mbar_init(bar(offsetof(Bars, rope_full)), kFp8 ? 2 : 1);
        ptx::mbar_init(bar(offsetof(Bars, p_ready)), 2 * 4);
        ptx::mbar_init(bar(offsetof(Bars, drain)), 1);
        ptx::mbar_init(bar(offsetof(Bars, q_staged)), 1);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(bar(offsetof(Bars, v_full)) + 8 * s, kFp8 ? 4 : 1);
            ptx::mbar_init(bar(offsetof(Bars, qk_part)) + 8 * s, 1);
            ptx::mbar_init(bar(offsetof(Bars, s_full)) + 8 * s, 1);
            for (int g = 0; g < 4; ++g) {
                const uint32_t off = uint32_t(8 * (4 * s + g));
                ptx::mbar_init(bar(offsetof(Bars, k_full)) + off, kFp8 ? 2 * 2 : 1);
                ptx::mbar_init(bar(offsetof(Bars, pv_done)) + off, 1);
            }
        }
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(&bars->tmem_base), kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    // The pair's barriers exist, and its TMEM, before either uses the other's:
    // the wait for that is over when the schedule is made.
    ptx::tc_fence_before();
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // What this call reads is there, and what it writes is no longer read.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // The merge's CTAs may be placed while this grid works; they wait for its end.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    SpanRange* range = reinterpret_cast<SpanRange*>(smem + kOffRange);
    span_schedule(p, *reinterpret_cast<SpanScratch*>(smem), pair, blockIdx.x == 0, range);
    ptx::fence_proxy_async_smem();     // (loads go where that was)
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const uint64_t lim_mma = p.timeout_ns, lim_dep = 2 * p.timeout_ns;

    if (warp == 0 || warp >= 6) {
        if constexpr (kFp8) {
            const Widener l{p, &map_q, bars, smem, sbase, b0, rank, lane, lim_dep};
            if (warp >= 6)
                l.blocks(range, pair, warp - 6);
            else if (ptx::elect_one())
                l.queries(range, pair);
        } else if (ptx::elect_one()) {
            const Loader l{p, &map_q, &cache.map, bars, sbase, b0, rank, lim_dep};
            if (warp == 0)
                l.pages(range, pair);
            else
                l.values(range, pair);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && ptx::elect_one()) {
            constexpr uint32_t idesc_qk =
                kFp8 ? ptx::idesc_f16_f32(128, false) : ptx::idesc_bf16_f32(128, false);
            constexpr uint32_t idesc_pv =
                kFp8 ? ptx::idesc_f16_f32(256, true) : ptx::idesc_bf16_f32(256, true);
            // K-major blocks: 16 k are 32 bytes. Value blocks (MN-major): 16
            // tokens are 2 KB, 64 columns a block.
            const uint64_t desc_k = ptx::desc_sw128(0, 16, 1024) + (sbase >> 4);
            const uint64_t desc_v = ptx::desc_sw128(0, kBlock, 1024) + (sbase >> 4);
            auto at = [](int off) { return uint64_t(off >> 4); };
            auto until = [&](uint32_t b, uint32_t parity, int32_t site) {
                return wait(b, parity, bars, p.status, site, lim_mma);
            };
            // Scores of step j.
            auto scores = [&](int j) {
                const int st = j & 1;
                const uint32_t ph = (j >> 1) & 1;
                const uint32_t d = tmem + kTmemS + uint32_t(st * 64);
                const uint32_t kf = bar(offsetof(Bars, k_full)) + 32 * st;
                const uint64_t q = desc_k + at(kOffQ);
                const uint64_t k = desc_k + at(kOffStage) + uint64_t(st) * at(kStageBytes);
                auto slots = [&](int g) {
#pragma unroll
                    for (int i = 2 * g; i < 2 * g + 2; ++i)
                        mma4_pair(d, q + at(i * kBlock), 2, k + at(i * kBlock), 2, idesc_qk,
                                  i > 0 ? 1u : 0u);
                };
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g == 2) {
                        if (!until(bar(offsetof(Bars, rope_full)), j & 1, kSiteRope)) return false;
                        ptx::tc_fence_after();
                        mma4_pair(d, q + at(8 * kBlock), 2, desc_k + at(kOffRope), 2, idesc_qk, 1u);
                        ptx::mma_commit_pair(bar(offsetof(Bars, qk_part)) + 8 * st, kBoth);
                    }
                    if (!until(kf + 8 * g, ph, kSiteK)) return false;
                    ptx::tc_fence_after();
                    slots(g);
                }
                ptx::mma_commit_pair(bar(offsetof(Bars, s_full)) + 8 * st, kBoth);
                return true;
            };
            // P V of step j, the first of its piece or not.
            auto values = [&](int j, bool first) {
                const int st = j & 1;
                if (!until(bar(offsetof(Bars, p_ready)), j & 1, kSiteP)) return false;
                ptx::tc_fence_after();
                const uint64_t v = desc_v + at(kOffStage) + uint64_t(st) * at(kStageBytes);
#pragma unroll
                for (int g = 0; g < 4; ++g) {        // page g / 2, value columns g % 2
                    mma4_pair(tmem + kTmemO + uint32_t((g & 1) * 128),
                              desc_k + at(kOffP + (g >> 1) * kBlock), 2, v + at(2 * g * kBlock),
                              at(16 * 128), idesc_pv, first && g < 2 ? 0u : 1u);
                    ptx::mma_commit_pair(bar(offsetof(Bars, pv_done)) + 8 * (4 * st + g), kBoth);
                }
                return true;
            };
            Walk w{range, range->first, pair};
            Piece pc;
            bool ok = true;
            int j = 0;
            for (uint32_t n = 0; ok && walk_next(p, w, pc); ++n) {
                ok = until(bar(offsetof(Bars, q_full)), n & 1, kSiteQ);
                for (int k = 0; ok && k < pc.steps; ++k, ++j) {
                    ok = scores(j);
                    if (ok && k > 0) ok = values(j - 1, k == 1);
                }
                if (ok) ok = values(j - 1, pc.steps == 1);
            }
            // Every MMA issued above has completed before TMEM is freed.
            ptx::mma_commit_pair(bar(offsetof(Bars, drain)), 1);
            wait(bar(offsetof(Bars, drain)), 0, bars, p.status, kSiteDrain, lim_mma, true);
        }
        __syncwarp();
    } else {
        // Softmax and epilogue: lane 64 f + r of TMEM holds row r's page f of a
        // step, and its value columns 256 f .. 256 f + 255.
        const int l = (warp & 3) * 32 + lane;
        const int f = l >> 6, r = l & 63;
        const uint32_t trow = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t swap_bar = 1 + (warp & 1);          // the two warps with these rows
        float* swap = reinterpret_cast<float*>(smem + kOffSwap);
        const uint32_t to_ready = ptx::map_to_rank(bar(offsetof(Bars, p_ready)), 0);
        const float scale = fabsf(p.scale_log2);
        Walk w{range, range->first, pair};
        Piece pc;
        bool ok = true;
        int j = 0;
        // Both threads' answer, and the other one's value.
        int turn = 0;
        auto exchange = [&](float v, float* other) {
            float* at = swap + (turn & 1) * 128;
            ++turn;
            at[l] = v;
            ok = !ptx::named_barrier_or(swap_bar, 64, !ok);
            *other = at[l ^ 64];
        };
        auto until = [&](uint32_t b, uint32_t parity, int32_t site) {
            return __all_sync(0xffffffffu, wait(b, parity, bars, p.status, site, lim_dep));
        };
        while (ok && walk_next(p, w, pc)) {
            float x_ref = -INFINITY;   // a score, before the scale
            float l_sum = 0.f;         // of the weights (for the LSE)
            float l_mma = 0.f;         // of the rounded ones (for the results)
            // fp8 cache: what a row's scores are multiplied by first (widen_queries;
            // negative with a negative softmax scale). (Written before the queries
            // were announced, which the scores waited for, and again with those of
            // the second item after this one, whose queries land when this one's
            // last weights have been announced.)
            const float* row_scale = reinterpret_cast<const float*>(smem + kOffScale) +
                                     ((w.item - 1) & 1) * kCtaRows + r;
            for (int k = 0; k < pc.steps; ++k, ++j) {
                const int st = j & 1;
                const int v = kSpanStepPages * (pc.first + k);
                const PageMask mine = page_mask(pc.it, v + f);
                ok = ok && until(bar(offsetof(Bars, s_full)) + 8 * st, (j >> 1) & 1, kSiteQkDone);
                // (Asked at each step: an answer kept from the item's first one, or the
                // product where the scores are read below, took 1 to 2 us of 73.)
                if (kFp8 && ok && __any_sync(0xffffffffu, *row_scale != 1.f)) {
                    ptx::tc_fence_after();
                    scale_scores(trow + kTmemS + uint32_t(st * 64), *row_scale);
                }
                // With an fp8 cache the scores are read twice, half of them at a
                // time: its many warps leave 96 registers a thread.
                constexpr int kPart = kFp8 ? 32 : 64;
                float x[kPart];
                auto read_scores = [&](int first) {
                    uint32_t raw[kPart];
                    if constexpr (kFp8)
                        ptx::tmem_ld32(trow + kTmemS + uint32_t(st * 64 + first), raw);
                    else
                        ptx::tmem_ld64(trow + kTmemS + uint32_t(st * 64), raw);
#pragma unroll
                    for (int i = 0; i < kPart; ++i) x[i] = __uint_as_float(raw[i]);
                    if (!kFp8 && p.scale_log2 < 0.f) {
#pragma unroll
                        for (int i = 0; i < kPart; ++i) x[i] = -x[i];
                    }
                    if (!mine.all()) {
#pragma unroll
                        for (int i = 0; i < kPart; ++i)
                            x[i] = mine.sees(first + i) ? x[i] : -INFINITY;
                    }
                };
                float mx = -INFINITY;
                if (ok) {
                    ptx::tc_fence_after();
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int first = 0; first < 64; first += kPart) {
                        read_scores(first);
#pragma unroll
                        for (int i = 0; i < kPart; i += 2)
                            m4[(i >> 1) & 3] = ptx::fmax3(m4[(i >> 1) & 3], x[i], x[i + 1]);
                    }
                    mx = ptx::fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
                }
                float other;
                exchange(mx, &other);
                if (!ok) break;
                mx = fmaxf(mx, other);
                float alpha = 1.f;
                if ((mx - x_ref) * scale > kRescaleThreshold) {
                    alpha = ptx::ex2((x_ref - mx) * scale);
                    x_ref = mx;
                }
                // The reference is taken off the scores, not off their products
                // with the scale: beyond 2^27 a product's rounding is more than the
                // exponents of the weights' type. A row that has seen no token
                // yet keeps x_ref = -inf: its weights are 2^-inf = 0, not NaN.
                const float neg = x_ref == -INFINITY ? 0.f : -x_ref;
                uint32_t pk[32];
                float2 ls = make_float2(0.f, 0.f), lm = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int at = (2 * i) % kPart;
                    if (kFp8 && at == 0) read_scores(2 * i);
                    const float2 a =
                        __fadd2_rn(make_float2(x[at], x[at + 1]), make_float2(neg, neg));
                    const float2 d = __ffma2_rn(a, make_float2(scale, scale),
                                                make_float2(kLift<kFp8>, kLift<kFp8>));
                    const float2 e = make_float2(ptx::ex2(d.x), ptx::ex2(d.y));
                    ls = __fadd2_rn(ls, e);
                    if constexpr (kFp8) {
                        const __half2 h = __floats2half2_rn(e.x, e.y);
                        pk[i] = *reinterpret_cast<const uint32_t*>(&h);
                        lm = __fadd2_rn(lm, __half22float2(h));
                    } else {
                        pk[i] = pack_bf16(e.x, e.y);
                        lm = __fadd2_rn(lm, make_float2(__uint_as_float(pk[i] << 16),
                                                        __uint_as_float(pk[i] & 0xffff0000u)));
                    }
                }
                l_sum = l_sum * alpha + (ls.x + ls.y);
                l_mma = l_mma * alpha + (lm.x + lm.y);
                // The step before has read the weights and added to the results.
                // (A piece's first step: the epilogue has waited for it.)
                if (k > 0) {
                    ok = until(bar(offsetof(Bars, pv_done)) + 8 * (4 * (st ^ 1) + 3),
                               ((j - 1) >> 1) & 1, kSitePv);
                    if (ok && __any_sync(0xffffffffu, alpha != 1.f)) {
                        ptx::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 256; c += 32) {
                            uint32_t o[32];
                            ptx::tmem_ld32(trow + kTmemO + uint32_t(c), o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            ptx::tmem_st32(trow + kTmemO + uint32_t(c), o);
                        }
                    }
                }
                if (ok) {
                    unsigned char* row = smem + kOffP + f * kBlock + r * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4*>(row + ((c ^ (r & 7)) * 16)) =
                            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                }
                // The other page's value blocks are there. Rows that are not
                // seen may hold anything (even NaN), and 0 times that is to
                // be 0.
                ok = ok && until(bar(offsetof(Bars, v_full)) + 8 * st, (j >> 1) & 1, kSiteV);
                if (ok) {
#pragma unroll 1
                    for (int g = 0; g < 2; ++g) {
                        const PageMask mask = page_mask(pc.it, v + g);
                        if (v + g >= pc.it.pages || mask.all()) continue;   // (no page: zeros)
                        unsigned char* vs = smem + kOffStage + st * kStageBytes + 4 * g * kBlock;
                        for (int i = l; i < 64 * 32; i += 128) {
                            const int t = i >> 5;
                            if (!mask.sees(t))
                                *reinterpret_cast<uint4*>(vs + ((i >> 3) & 3) * kBlock + t * 128 +
                                                          (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    ptx::fence_proxy_async_smem();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(to_ready);
                }
                // (a thread that failed says so at the next exchange)
            }
            // Results: normalised, to the output or to the piece's rows.
            if (ok)
                ok = until(bar(offsetof(Bars, pv_done)) + 8 * (4 * ((j - 1) & 1) + 3),
                           ((j - 1) >> 1) & 1, kSitePv);
            float other_sum, other_mma;
            exchange(l_sum, &other_sum);
            exchange(l_mma, &other_mma);
            if (!ok) break;
            ptx::tc_fence_after();
            l_sum += other_sum;
            l_mma += other_mma;
            const float inv = l_mma == 0.f ? 0.f : p.v_scale / l_mma;
            // (a NaN comes through)
            const float lse = l_sum == 0.f ? -INFINITY : (x_ref * scale + (log2f(l_sum) - kLift<kFp8>)) * kLn2;
            const int row = rank * kCtaRows + r;           // of the item
            const int64_t row0 = pc.part_row < 0 ? int64_t(pc.it.row0) : pc.part_row;
            // 128 bytes of a warp's 32 rows at a time, through the weights' place
            // (these rows' own, which the last P V has read), 16-byte piece c of
            // row i at c ^ i % 8: a lane reads TMEM by rows and writes whole lines
            // (rows from registers, 32 bytes of each a store, took 7,000 cycles).
            unsigned char* tile = smem + kOffP + (warp & 3) * (32 * 128);
            const int first_row = rank * kCtaRows + (r & 32);   // of the warp's rows
            auto put = [&](int c, const uint32_t* w) {
                *reinterpret_cast<uint4*>(tile + lane * 128 + ((c ^ (lane & 7)) * 16)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            };
            auto flush = [&](char* base, int64_t row_bytes) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = 4 * k + (lane >> 3), c = lane & 7;
                    const uint4 v = *reinterpret_cast<const uint4*>(tile + i * 128 +
                                                                    ((c ^ (i & 7)) * 16));
                    if (first_row + i < pc.it.rows)
                        *reinterpret_cast<uint4*>(base + (row0 + first_row + i) * row_bytes +
                                                  c * 16) = v;
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
                uint32_t o[32];
                ptx::tmem_ld32(trow + kTmemO + uint32_t(c), o);
                float y[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    y[i] = l_mma == 0.f ? 0.f : __uint_as_float(o[i]) * inv;
                if (pc.part_row < 0) {
                    // (64 columns are a line)
                    uint32_t h[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) h[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) put(((c & 32) >> 3) + i, h + 4 * i);
                    if ((c & 32) != 0)
                        flush(reinterpret_cast<char*>(p.out + 256 * f + c - 32), kLkv * 2);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        put(i, reinterpret_cast<const uint32_t*>(y) + 4 * i);
                    flush(reinterpret_cast<char*>(p.o_part + 256 * f + c), kLkv * 4);
                }
            }
            if (row < pc.it.rows && f == 0) {
                if (pc.part_row >= 0)
                    p.lse_part[row0 + row] = lse;
                else if (p.lse != nullptr)
                    p.lse[row0 + row] = lse;
            }
            // (The next piece's first P V overwrites the results: it waits for
            // all of these warps.)
            ptx::tc_fence_before();
        }
    }
    // Neither CTA leaves while the other's MMAs, loads or arrivals may reach it.
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc_pair(tmem, kTmemCols);
}

template <bool kFp8>
int launch(const SpanParams& p, cudaStream_t st) {
    CUtensorMap map_q;
    CacheMap<kFp8> cache;
    if (!encode_2d(&map_q, p.q, kD, uint64_t(p.batch) * p.heads, kCtaRows))
        return int(cudaErrorInvalidValue);
    if constexpr (!kFp8) {
        if (!encode_2d(&cache.map, p.cache, kD, uint64_t(p.num_blocks) * kPageSize, kPageSize))
            return int(cudaErrorInvalidValue);
    }
    auto kernel = mla_span_kernel<kFp8>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared_memory(kernel, kSmemBytes, &allowed);
    if (e != cudaSuccess) return int(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * p.pairs), 1, 1);
    cfg.blockDim = dim3(kFp8 ? kThreadsFp8 : kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return int(cudaLaunchKernelEx(&cfg, kernel, p, map_q, cache));
}

}  // namespace

int launch_span_attention(const SpanParams& p, bool fp8, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return fp8 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace mla
