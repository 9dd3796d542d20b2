// Page bookkeeping of the latent cache: fork, free and compact.
//
// State: one count per page (how many block-table entries name it; 0 = free)
// and the block tables. There is no free list: the free pages are those with
// count 0, and they are always handed out in ascending order, so a call's
// result follows from its arguments alone (no result depends on the order of
// atomics: counts are sums of integers, ranks come from prefix sums).
//
//   fork     child c: shares pages 0..F-1 of its parent (F = S / 64 whole
//            pages of the S shared tokens), copies the S % 64 rows of page F
//            into a page of its own in every layer, and gets fresh pages up
//            to ceil(L / 64).   count | assign | share + copy
//   free     counts - 1 for each entry of the named rows.
//   compact  M live pages. The k-th live page with id >= M goes to the k-th
//            free id below M: the fewest moves that leave the live pages in
//            [0, M), and no destination is another move's source, so the
//            copies run in any order.   count | list | move
//
// A grid-wide prefix sum needs all counts before the first rank, and the
// copies need the ranks. Each operation is one cooperative launch with a
// barrier (|) between its passes. Each CTA of the second pass sums the chunk
// counts below its own itself (num_blocks / 1024 values). The grid is at most
// kCtasPerSm CTAs per SM (all resident, as the barrier needs), and no more
// than the work has use for.
#include <climits>
#include <cstdint>

#include "mla_device.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace {

constexpr int kPageThreads = 256;
constexpr int kWarps = kPageThreads / 32;
constexpr int kChunkIters = 4;
constexpr int kChunk = kPageThreads * kChunkIters;   // pages whose counts one CTA reads
constexpr int kMaxChildren = 8192;                   // their page offsets fit shared memory
constexpr int kPieceBytes = 8192;                    // bytes of a page that one CTA copies at once

constexpr int kCtasPerSm = 4;                        // at most 64 registers a thread
constexpr uint64_t kBarrierTimeoutNs = 1000000000ull;
constexpr int32_t kSiteGrid = 90;

// Barriers of a cooperative grid on a word that is 0 between calls;
// arrive_last ends a CTA's part, and the last one of the grid clears the word.
// A wait that expires marks the word, if the arrivals are still short then: so
// either every CTA passes a barrier or none does, and the calls that find the
// mark (until the workspace is initialised again) stop at their first barrier,
// before they rely on what an abandoned call left in the workspace.
constexpr uint32_t kAbandoned = 0x80000000u;

struct GridBarrier {
    uint32_t* word;
    int32_t* status;
    uint32_t passed = 0;

    __device__ __forceinline__ bool wait(int* ok) {
        __syncthreads();
        ++passed;
        if (threadIdx.x == 0) {
            __threadfence();
            *ok = 1;
            atomicAdd(word, 1u);
            const uint64_t t0 = ptx::globaltimer();
            while (true) {
                const uint32_t v = arrivals();
                if (v < kAbandoned && v >= passed * gridDim.x) break;
                if (v >= kAbandoned ||
                    (ptx::globaltimer() - t0 > kBarrierTimeoutNs &&
                     atomicCAS(word, v, v | kAbandoned) == v)) {
                    record_error(status, MLA_ERR_TIMEOUT, kSiteGrid);
                    *ok = 0;
                    break;
                }
            }
            __threadfence();
        }
        __syncthreads();
        return *ok != 0;
    }
    __device__ __forceinline__ void arrive_last() {
        __syncthreads();
        if (threadIdx.x == 0 && atomicAdd(word, 1u) == (passed + 1) * gridDim.x - 1) *word = 0;
    }
    __device__ __forceinline__ uint32_t arrivals() const {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
        return v;
    }
};

struct CacheView {
    char* base;
    int64_t layer_stride;   // bytes
    int64_t page_bytes;
    int layers;
};

// Where the passes of one call leave what the next ones need (in the
// caller's workspace, behind the status header). What another CTA wrote is
// read from L2 (__ldcg).
struct PageScratch {
    int32_t* status;
    uint32_t* barrier;
    int32_t* go;            // fork: 1 if the call goes ahead
                            // compact: [0] live pages M, [1] pages to move
    int32_t* chunk_count;   // [chunks] free (fork) or live (compact) pages of each chunk
    uint32_t* live_bits;    // compact: one bit per page
    int32_t* need;          // fork: [children] fresh pages, -1 for a child that cannot be made
    int32_t* src;           // compact: [moves] ascending; fork: [children] page to copy from
    int32_t* dst;           // compact: [moves] ascending; fork: [children] first fresh page
    int32_t* moved_ref;     // compact: [moves] count of src[k]; fork: [children] rows to copy
};

// Pages of L >= 0 tokens, up to the largest int.
__device__ __forceinline__ int pages_in(int L) {
    return int((uint32_t(L) + kPageSize - 1) / kPageSize);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the CTA (every thread gets it); `tmp` has kWarps words.
__device__ __forceinline__ int block_sum(int v, int* tmp) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += tmp[w];
    return s;
}

// Exclusive prefix sum over the CTA in thread order; *total gets the sum.
__device__ __forceinline__ int block_exclusive(int v, int* tmp, int* total) {
    const int lane = threadIdx.x & 31;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) tmp[threadIdx.x >> 5] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < int(threadIdx.x >> 5)) before += tmp[w];
        all += tmp[w];
    }
    *total = all;
    return before + inc - v;
}

// counts[0..n) summed over the CTA.
__device__ __forceinline__ int sum_below(const int32_t* counts, int n, int* tmp) {
    int s = 0;
    for (int i = threadIdx.x; i < n; i += kPageThreads) s += __ldcg(counts + i);
    return block_sum(s, tmp);
}

// Copy the first `bytes` (a multiple of 16) of page src to page dst in one
// layer: the 8 KB pieces part, part + parts, ..., two pieces (four 16-byte
// loads a thread) in flight before their stores.
__device__ __forceinline__ void copy_page(const CacheView& cache, int layer, int src, int dst,
                                          int bytes, int part, int parts) {
    const char* s = cache.base + layer * cache.layer_stride + src * cache.page_bytes;
    char* d = cache.base + layer * cache.layer_stride + dst * cache.page_bytes;
    const int step = parts * kPieceBytes;
    for (int o = part * kPieceBytes + int(threadIdx.x) * 16; o < bytes; o += 2 * step) {
        uint4 v[4];
        const int at[4] = {o, o + kPieceBytes / 2, o + step, o + step + kPieceBytes / 2};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at[i] < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(s + at[i]));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at[i] < bytes) __stcs(reinterpret_cast<uint4*>(d + at[i]), v[i]);
    }
}
static_assert(kPieceBytes == 2 * 16 * kPageThreads, "a piece is two loads per thread");

// Parts that one page's copy is cut into, so that few pages still use the
// whole grid.
__device__ __forceinline__ uint32_t parts_of(const CacheView& cache, uint32_t pages) {
    const uint32_t most = uint32_t((cache.page_bytes + kPieceBytes - 1) / kPieceBytes);
    const uint32_t want = (2 * gridDim.x + pages - 1) / pages;
    return want < most ? want : most;
}

// ------------------------------------------------------------------- fork

struct ForkParams {
    CacheView cache;
    PageScratch ws;
    int64_t num_blocks;
    const int32_t* ref_in;
    int32_t* ref_out;
    const int32_t* table;
    int rows, max_blocks;
    const int32_t* parents;
    const int32_t* shared_lens;
    const int32_t* child_lens;
    int children;
    int32_t* child_table;
    int chunks;
};

// One warp checks one child and writes how many fresh pages it needs.
__device__ __forceinline__ void check_child(const ForkParams& p, int c) {
    const int lane = threadIdx.x & 31;
    const int parent = p.parents[c], S = p.shared_lens[c], L = p.child_lens[c];
    int bad = MLA_OK, detail = 0, from = 0;
    if (S < 0 || L < S || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
        bad = MLA_ERR_BAD_SEQ_LEN;
        detail = S < 0 ? S : L;
    } else if (parent >= p.rows || (parent < 0 && S > 0)) {
        bad = MLA_ERR_BAD_ROW;
        detail = parent;
    } else {
        // Every page that the child shares or copies from is in use.
        const int32_t* row = p.table + int64_t(parent) * p.max_blocks;
        for (int j = lane; j < pages_in(S); j += 32) {
            const int page = row[j];
            if (page < 0 || int64_t(page) >= p.num_blocks) {
                bad = MLA_ERR_BAD_BLOCK_ID;
                detail = page;
            } else if (p.ref_in[page] == 0) {
                bad = MLA_ERR_PAGE_STATE;
                detail = page;
            } else if (j == S / kPageSize) {
                from = page;                  // (in one lane at most)
            }
        }
    }
    if (bad != MLA_OK) record_error(p.ws.status, bad, detail);
    __syncwarp();
    const bool any = __any_sync(0xffffffffu, bad != MLA_OK);
    from = int(__reduce_add_sync(0xffffffffu, uint32_t(from)));
    if (lane == 0) {
        p.ws.need[c] = any ? -1 : pages_in(L) - S / kPageSize;
        p.ws.src[c] = from;
        p.ws.moved_ref[c] = S % kPageSize;
    }
}

__global__ void __launch_bounds__(kPageThreads, kCtasPerSm) fork_kernel(const ForkParams p) {
    __shared__ int tmp[kWarps];
    __shared__ int barrier_ok;
    __shared__ int warp_free[kChunkIters * kWarps];
    extern __shared__ int off[];      // [children + 1]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    GridBarrier grid{p.ws.barrier, p.ws.status};

    // Free pages of each chunk; then one warp per child.
    const int checkers = (p.children + kWarps - 1) / kWarps;
    for (int u = blockIdx.x; u < p.chunks + checkers; u += gridDim.x) {
        if (u < p.chunks) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < kChunkIters; ++i) {
                const int64_t page = int64_t(u) * kChunk + i * kPageThreads + threadIdx.x;
                if (page < p.num_blocks) n += p.ref_in[page] == 0;
            }
            n = block_sum(n, tmp);
            if (threadIdx.x == 0) p.ws.chunk_count[u] = n;
        } else {
            const int c = (u - p.chunks) * kWarps + warp;
            if (c < p.children) check_child(p, c);
        }
    }
    if (!grid.wait(&barrier_ok)) return;

    // CTAs with a chunk: the children's page offsets, then the chunk's free
    // pages to their owners and the chunk's counts.
    if (int(blockIdx.x) < p.chunks) {
        int total = 0, invalid = 0;
        bool over = false;
        for (int c0 = 0; c0 < p.children; c0 += kPageThreads) {
            const int c = c0 + threadIdx.x;
            const int n = c < p.children ? __ldcg(p.ws.need + c) : 0;
            if (n < 0) invalid = 1;
            // (one child alone may ask for more than the pool; no sum here wraps)
            int sum;
            const int before = block_exclusive(
                n < 0 ? 0 : int(min(int64_t(n), p.num_blocks + 1)), tmp, &sum);
            if (c < p.children) off[c] = total + before;
            over = over || int64_t(total) + sum > p.num_blocks;
            total = over ? 0 : total + sum;
        }
        if (threadIdx.x == 0) off[p.children] = total;
        invalid = block_sum(invalid, tmp);
        const int free_all = sum_below(p.ws.chunk_count, p.chunks, tmp);
        const bool go = invalid == 0 && !over && total <= free_all;
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            p.ws.go[0] = go ? 1 : 0;
            if (invalid == 0 && !go)
                record_error(p.ws.status, MLA_ERR_NO_PAGES, over ? INT_MAX : total - free_all);
        }
        for (int u = blockIdx.x; u < p.chunks; u += gridDim.x) {
            const int free_below = sum_below(p.ws.chunk_count, u, tmp);
            int ref[kChunkIters];
            uint32_t free_mask[kChunkIters];
#pragma unroll
            for (int i = 0; i < kChunkIters; ++i) {
                const int64_t page = int64_t(u) * kChunk + i * kPageThreads + threadIdx.x;
                ref[i] = page < p.num_blocks ? p.ref_in[page] : 1;
                free_mask[i] = __ballot_sync(0xffffffffu, ref[i] == 0);
                if (lane == 0) warp_free[i * kWarps + warp] = __popc(free_mask[i]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kChunkIters; ++i) {
                const int64_t page = int64_t(u) * kChunk + i * kPageThreads + threadIdx.x;
                if (page >= p.num_blocks) continue;
                if (ref[i] == 0 && go) {
                    int rank = free_below + __popc(free_mask[i] & ((1u << lane) - 1u));
                    for (int w = 0; w < i * kWarps + warp; ++w) rank += warp_free[w];
                    if (rank < total) {
                        // The child that owns rank: the last c with off[c] <=
                        // rank (children without fresh pages share their
                        // successor's offset).
                        int lo = 0, hi = p.children;
                        while (hi - lo > 1) {
                            const int mid = (lo + hi) >> 1;
                            if (off[mid] <= rank) lo = mid; else hi = mid;
                        }
                        const int j = rank - off[lo];
                        p.child_table[int64_t(lo) * p.max_blocks + p.shared_lens[lo] / kPageSize +
                                      j] = int32_t(page);
                        if (j == 0) p.ws.dst[lo] = int32_t(page);
                        ref[i] = 1;
                    }
                }
                p.ref_out[page] = ref[i];
            }
        }
    }
    if (!grid.wait(&barrier_ok)) return;

    // One warp per child for its shared pages; the whole grid copies the
    // partly filled pages.
    if (__ldcg(p.ws.go) != 0) {
        for (int c = blockIdx.x * kWarps + warp; c < p.children; c += gridDim.x * kWarps) {
            const int full = p.shared_lens[c] / kPageSize;
            const int32_t* row = p.table + int64_t(p.parents[c]) * p.max_blocks;
            for (int j = lane; j < full; j += 32) {
                const int page = row[j];
                p.child_table[int64_t(c) * p.max_blocks + j] = page;
                atomicAdd(p.ref_out + page, 1);
            }
        }
        const uint32_t layers = uint32_t(p.cache.layers);
        const uint32_t parts = p.children > 0 ? parts_of(p.cache, p.children * layers) : 1;
        const uint32_t per_child = layers * parts;
        const int row_bytes = int(p.cache.page_bytes / kPageSize);
        for (int64_t i = blockIdx.x; i < int64_t(p.children) * per_child; i += gridDim.x) {
            const int c = int(i / per_child);
            const uint32_t r = uint32_t(i - int64_t(c) * per_child);
            const int bytes = __ldcg(p.ws.moved_ref + c) * row_bytes;
            const int src = __ldcg(p.ws.src + c), dst = __ldcg(p.ws.dst + c);
            if (bytes > 0)
                copy_page(p.cache, int(r / parts), src, dst, bytes, int(r % parts), int(parts));
        }
    }
    grid.arrive_last();
}

// ------------------------------------------------------------------- free

struct FreeParams {
    int32_t* status;
    uint32_t* barrier;
    int64_t num_blocks;
    const int32_t* ref_in;
    int32_t* ref_out;
    const int32_t* table;
    int rows, max_blocks;
    const int32_t* seq_lens;
    const int32_t* free_rows;
    int count;
    int32_t* num_freed;
};

// The counts copied (unless in place), then 256 entries of a row at a time.
// Lanes of a warp that name the same page take it off with one atomic.
__global__ void __launch_bounds__(kPageThreads, kCtasPerSm) free_kernel(const FreeParams p) {
    __shared__ int barrier_ok;
    const int lane = threadIdx.x & 31;
    GridBarrier grid{p.barrier, p.status};
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.num_freed = 0;
    if (p.ref_in != p.ref_out)
        for (int64_t i = int64_t(blockIdx.x) * kPageThreads + threadIdx.x; i < p.num_blocks;
             i += int64_t(gridDim.x) * kPageThreads)
            p.ref_out[i] = p.ref_in[i];
    if (!grid.wait(&barrier_ok)) return;
    const int per_row = (p.max_blocks + kPageThreads - 1) / kPageThreads;
    for (int64_t u = blockIdx.x; u < int64_t(p.count) * per_row; u += gridDim.x) {
        const int r = int(u / per_row), j0 = int(u - int64_t(r) * per_row) * kPageThreads;
        const int row = p.free_rows[r];
        if (row < 0 || row >= p.rows) {
            if (j0 == 0 && threadIdx.x == 0) record_error(p.status, MLA_ERR_BAD_ROW, row);
            continue;
        }
        const int L = p.seq_lens[row];
        if (L < 0 || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
            if (j0 == 0 && threadIdx.x == 0) record_error(p.status, MLA_ERR_BAD_SEQ_LEN, L);
            continue;
        }
        const int n = pages_in(L);
        if (j0 >= n) continue;
        const int j = j0 + threadIdx.x;
        int page = j < n ? p.table[int64_t(row) * p.max_blocks + j] : -1;
        if (j < n && (page < 0 || int64_t(page) >= p.num_blocks)) {
            record_error(p.status, MLA_ERR_BAD_BLOCK_ID, page);
            page = -1;
        }
        __syncwarp();
        const uint32_t same = __match_any_sync(0xffffffffu, page);
        bool freed = false;
        if (page >= 0 && lane == __ffs(same) - 1) {
            const int off = __popc(same);
            const int old = atomicSub(p.ref_out + page, off);
            freed = old > 0 && old <= off;
            if (old < off) {
                // More entries than counts: the count stays at 0. What was
                // taken too much is put back, so whatever the order, the sum
                // of the atomics on this page is -(what it had).
                atomicAdd(p.ref_out + page, off - (old > 0 ? old : 0));
                record_error(p.status, MLA_ERR_PAGE_STATE, page);
            }
        }
        __syncwarp();
        const uint32_t f = __ballot_sync(0xffffffffu, freed);
        if (lane == 0 && f != 0) atomicAdd(p.num_freed, __popc(f));
    }
    grid.arrive_last();
}

// ---------------------------------------------------------------- compact

struct CompactParams {
    CacheView cache;
    PageScratch ws;
    int64_t num_blocks;
    const int32_t* ref_in;
    int32_t* ref_out;
    const int32_t* table;
    int32_t* table_out;
    int rows, max_blocks;
    const int32_t* seq_lens;
    int32_t* page_map;
    int32_t* num_live;
    int chunks;
};

// Index of `v` in the ascending list a[0..n), or -1.
__device__ __forceinline__ int find(const int32_t* a, int n, int v) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(a + mid) < v) lo = mid + 1; else hi = mid;
    }
    return lo < n && __ldcg(a + lo) == v ? lo : -1;
}

__global__ void __launch_bounds__(kPageThreads, kCtasPerSm) compact_kernel(const CompactParams p) {
    __shared__ int tmp[kWarps];
    __shared__ int barrier_ok;
    __shared__ uint32_t live_bits[kChunk / 32];
    GridBarrier grid{p.ws.barrier, p.ws.status};

    // Live pages of each chunk, and one bit per page: the next pass writes
    // the counts in place, so what it needs of other chunks it reads from the
    // bits.
    for (int u = blockIdx.x; u < p.chunks; u += gridDim.x) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kChunkIters; ++i) {
            const int64_t page = int64_t(u) * kChunk + i * kPageThreads + threadIdx.x;
            const bool live = page < p.num_blocks && p.ref_in[page] != 0;
            const uint32_t bits = __ballot_sync(0xffffffffu, live);
            if ((threadIdx.x & 31) == 0) p.ws.live_bits[page >> 5] = bits;
            n += live;
        }
        n = block_sum(n, tmp);
        if (threadIdx.x == 0) p.ws.chunk_count[u] = n;
    }
    if (!grid.wait(&barrier_ok)) return;

    if (int(blockIdx.x) < p.chunks) {
        const int M = sum_below(p.ws.chunk_count, p.chunks, tmp);
        // Live pages below M: those of the whole chunks before M's and of the
        // words of M's chunk up to M.
        const int m_chunk = M / kChunk;
        int part = 0;
        if (m_chunk < p.chunks && threadIdx.x < kChunk / 32) {
            const int first = m_chunk * kChunk + threadIdx.x * 32;
            const uint32_t bits = __ldcg(p.ws.live_bits + (first >> 5));
            const int take = M - first;   // bits of this word below M
            part = __popc(take >= 32 ? bits : take > 0 ? bits & ((1u << take) - 1u) : 0u);
        }
        const int live_low = sum_below(p.ws.chunk_count, m_chunk, tmp) + block_sum(part, tmp);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            p.ws.go[0] = M;
            p.ws.go[1] = M - live_low;
            if (p.num_live != nullptr) *p.num_live = M;
        }
        for (int u = blockIdx.x; u < p.chunks; u += gridDim.x) {
            const int live_before = sum_below(p.ws.chunk_count, u, tmp);
            if (threadIdx.x < kChunk / 32)
                live_bits[threadIdx.x] = __ldcg(p.ws.live_bits + u * (kChunk / 32) + threadIdx.x);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kChunkIters; ++i) {
                const int in = i * kPageThreads + threadIdx.x;
                const int64_t page = int64_t(u) * kChunk + in;
                if (page >= p.num_blocks) continue;
                const uint32_t bits = live_bits[in >> 5];
                int before = live_before + __popc(bits & ((1u << (in & 31)) - 1u));
                for (int w = 0; w < (in >> 5); ++w) before += __popc(live_bits[w]);
                const bool live = (bits >> (in & 31)) & 1u;
                const int ref = p.ref_in[page];
                if (live && page >= M) {
                    const int k = before - live_low;
                    p.ws.src[k] = int(page);
                    p.ws.moved_ref[k] = ref;
                    p.ref_out[page] = 0;
                    continue;                      // its map entry is the move pass's
                }
                if (!live && page < M) {
                    p.ws.dst[int(page) - before] = int(page);   // its count is the move pass's
                } else {
                    p.ref_out[page] = ref;
                }
                if (p.page_map != nullptr) p.page_map[page] = live ? int(page) : -1;
            }
            __syncthreads();
        }
    }
    if (!grid.wait(&barrier_ok)) return;

    const int M = __ldcg(p.ws.go), moves = __ldcg(p.ws.go + 1);
    const int64_t tid = int64_t(blockIdx.x) * kPageThreads + threadIdx.x;
    const int64_t threads = int64_t(gridDim.x) * kPageThreads;
    for (int64_t k = tid; k < moves; k += threads) {
        const int dst = __ldcg(p.ws.dst + k);
        p.ref_out[dst] = __ldcg(p.ws.moved_ref + k);
        if (p.page_map != nullptr) p.page_map[__ldcg(p.ws.src + k)] = dst;
    }
    const int64_t entries = int64_t(p.rows) * p.max_blocks;
    for (int64_t e = tid; e < entries; e += threads) {
        const int row = int(e / p.max_blocks), j = int(e - int64_t(row) * p.max_blocks);
        const int L = p.seq_lens[row];
        if (L < 0 || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
            if (j == 0) record_error(p.ws.status, MLA_ERR_BAD_SEQ_LEN, L);
            continue;
        }
        if (j >= pages_in(L)) continue;
        int page = p.table[e];
        if (page < 0 || int64_t(page) >= p.num_blocks) {
            record_error(p.ws.status, MLA_ERR_BAD_BLOCK_ID, page);
        } else if (page >= M) {
            const int k = find(p.ws.src, moves, page);
            if (k < 0) record_error(p.ws.status, MLA_ERR_PAGE_STATE, page);
            else page = __ldcg(p.ws.dst + k);
        } else if (find(p.ws.dst, moves, page) >= 0) {
            record_error(p.ws.status, MLA_ERR_PAGE_STATE, page);   // it was free
        }
        p.table_out[e] = page;
    }
    const int64_t pages = int64_t(moves) * p.cache.layers;
    const uint32_t parts =
        pages > 0 ? parts_of(p.cache, uint32_t(min(pages, int64_t(1) << 30))) : 1;
    const int64_t per_move = int64_t(p.cache.layers) * parts;
    for (int64_t i = blockIdx.x; i < moves * per_move; i += gridDim.x) {
        const int k = int(i / per_move);
        const uint32_t r = uint32_t(i - k * per_move);
        copy_page(p.cache, int(r / parts), __ldcg(p.ws.src + k), __ldcg(p.ws.dst + k),
                  int(p.cache.page_bytes), int(r % parts), int(parts));
    }
    grid.arrive_last();
}

// ------------------------------------------------------------------- host

constexpr int kMaxCacheBlocks = (1 << 23) - 2;   // 256 of these still sum below 2^31

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int chunks_of(int64_t num_blocks) { return int((num_blocks + kChunk - 1) / kChunk); }

// Scratch layout; returns its size behind the status header.
size_t page_scratch(char* ws, int64_t num_blocks, int children, PageScratch* s) {
    const size_t chunks = size_t(chunks_of(num_blocks));
    // moves <= half the pages
    const size_t lists = size_t(num_blocks) / 2 + 1 > size_t(children)
                             ? size_t(num_blocks) / 2 + 1 : size_t(children);
    size_t at = kStatusBytes;
    auto take = [&](size_t bytes) {
        char* p = ws + at;
        at += round256(bytes);
        return reinterpret_cast<int32_t*>(p);
    };
    PageScratch t{};
    t.status = reinterpret_cast<int32_t*>(ws);
    t.barrier = reinterpret_cast<uint32_t*>(ws + 4 * kPageBarrierWord);
    t.go = take(8);
    t.chunk_count = take(chunks * 4);
    t.live_bits = reinterpret_cast<uint32_t*>(take(chunks * (kChunk / 8)));
    t.need = take(size_t(children) * 4);
    t.src = take(lists * 4);
    t.dst = take(lists * 4);
    t.moved_ref = take(lists * 4);
    if (s != nullptr) *s = t;
    return at;
}

// A cooperative launch of as many CTAs as the work has use for, at most
// kCtasPerSm per SM.
template <typename Kernel, typename Params>
int launch(Kernel kernel, int64_t want, size_t smem, void* stream, const Params& p) {
    int device = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return int(e);
    const int64_t most = int64_t(sms) * kCtasPerSm;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(want < 1 ? 1 : want < most ? want : most));
    cfg.blockDim = dim3(kPageThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return int(cudaLaunchKernelEx(&cfg, kernel, p));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, const void* b, size_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y ? y - x < bytes : x - y < bytes;
}

// Either the same array or none of its bytes.
bool same_or_apart(const void* a, const void* b, size_t bytes) {
    return a == b || !overlap(a, b, bytes);
}

int check_cache(const void* cache, int num_layers, int64_t layer_stride_bytes, int64_t num_blocks,
                int entry_bytes, CacheView* v) {
    if (num_layers < 1 || num_blocks < 1) return MLA_ERR_INVALID_ARG;
    if (entry_bytes != 1 && entry_bytes != 2) return MLA_ERR_UNSUPPORTED;
    if (num_blocks > kMaxCacheBlocks) return MLA_ERR_UNSUPPORTED;
    if (!cache || !aligned(cache, 16)) return MLA_ERR_INVALID_ARG;
    v->page_bytes = int64_t(kPageSize) * kD * entry_bytes;
    if (num_layers > 1 && (layer_stride_bytes % 16 != 0 ||
                           layer_stride_bytes < num_blocks * v->page_bytes))
        return MLA_ERR_INVALID_ARG;
    v->base = const_cast<char*>(static_cast<const char*>(cache));
    v->layer_stride = layer_stride_bytes;
    v->layers = num_layers;
    return MLA_OK;
}

int check_counts(const int32_t* in, const int32_t* out, int64_t num_blocks) {
    if (!in || !out || !aligned(in, 4) || !aligned(out, 4)) return MLA_ERR_INVALID_ARG;
    return same_or_apart(in, out, size_t(num_blocks) * 4) ? MLA_OK : MLA_ERR_INVALID_ARG;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
    return ws && aligned(ws, 256) && bytes >= need ? MLA_OK : MLA_ERR_WORKSPACE;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_cache_workspace_bytes(int64_t num_blocks, int children) {
    if (num_blocks < 1 || num_blocks > kMaxCacheBlocks || children < 0 || children > kMaxChildren)
        return 0;
    return page_scratch(nullptr, num_blocks, children, nullptr);
}

extern "C" int mla_cache_fork(void* latent_cache, int num_layers, int64_t layer_stride_bytes,
                              int64_t num_blocks, int entry_bytes, const int32_t* ref_counts,
                              int32_t* ref_counts_out, const int32_t* block_table, int rows,
                              int max_blocks_per_seq, const int32_t* parents,
                              const int32_t* shared_lens, const int32_t* child_lens, int children,
                              int32_t* child_table, void* workspace, size_t workspace_bytes,
                              void* stream) {
    ForkParams p{};
    int rc = check_cache(latent_cache, num_layers, layer_stride_bytes, num_blocks, entry_bytes,
                         &p.cache);
    if (rc != MLA_OK) return rc;
    if (rows < 0 || children < 0 || max_blocks_per_seq < 1) return MLA_ERR_INVALID_ARG;
    if (children > kMaxChildren) return MLA_ERR_UNSUPPORTED;
    rc = check_counts(ref_counts, ref_counts_out, num_blocks);
    if (rc != MLA_OK) return rc;
    if (children > 0 && (!parents || !shared_lens || !child_lens || !child_table ||
                         !aligned(parents, 4) || !aligned(shared_lens, 4) ||
                         !aligned(child_lens, 4) || !aligned(child_table, 4)))
        return MLA_ERR_INVALID_ARG;
    if (rows > 0 && (!block_table || !aligned(block_table, 4))) return MLA_ERR_INVALID_ARG;
    if (rows > 0 && children > 0) {
        // The children's table is written while the parents' is read.
        const uintptr_t a = reinterpret_cast<uintptr_t>(block_table);
        const uintptr_t b = reinterpret_cast<uintptr_t>(child_table);
        const uintptr_t row = uintptr_t(max_blocks_per_seq) * 4;
        if (a < b + row * children && b < a + row * rows) return MLA_ERR_INVALID_ARG;
    }
    rc = check_workspace(workspace, workspace_bytes,
                         mla_cache_workspace_bytes(num_blocks, children));
    if (rc != MLA_OK) return rc;
    page_scratch(static_cast<char*>(workspace), num_blocks, children, &p.ws);
    p.num_blocks = num_blocks;
    p.ref_in = ref_counts;
    p.ref_out = ref_counts_out;
    p.table = block_table;
    p.rows = rows;
    p.max_blocks = max_blocks_per_seq;
    p.parents = parents;
    p.shared_lens = shared_lens;
    p.child_lens = child_lens;
    p.children = children;
    p.child_table = child_table;
    p.chunks = chunks_of(num_blocks);
    const int64_t checks = p.chunks + (children + kWarps - 1) / kWarps;
    const int64_t copies =
        int64_t(children) * num_layers * ((p.cache.page_bytes + kPieceBytes - 1) / kPieceBytes);
    const int e = launch(fork_kernel, copies > checks ? copies : checks,
                         size_t(children + 1) * 4, stream, p);
    return e == 0 ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" int mla_cache_free(const int32_t* ref_counts, int32_t* ref_counts_out,
                              int64_t num_blocks, const int32_t* block_table, int rows,
                              int max_blocks_per_seq, const int32_t* seq_lens,
                              const int32_t* free_rows, int count, int32_t* num_freed,
                              void* workspace, size_t workspace_bytes, void* stream) {
    if (num_blocks < 1 || rows < 0 || count < 0 || max_blocks_per_seq < 1)
        return MLA_ERR_INVALID_ARG;
    if (num_blocks > kMaxCacheBlocks) return MLA_ERR_UNSUPPORTED;
    int rc = check_counts(ref_counts, ref_counts_out, num_blocks);
    if (rc != MLA_OK) return rc;
    if (!num_freed || !aligned(num_freed, 4)) return MLA_ERR_INVALID_ARG;
    if (count > 0 && (!free_rows || !aligned(free_rows, 4))) return MLA_ERR_INVALID_ARG;
    if (rows > 0 && (!block_table || !seq_lens || !aligned(block_table, 4) ||
                     !aligned(seq_lens, 4)))
        return MLA_ERR_INVALID_ARG;
    rc = check_workspace(workspace, workspace_bytes, kStatusBytes);
    if (rc != MLA_OK) return rc;
    FreeParams p{};
    p.status = static_cast<int32_t*>(workspace);
    p.num_blocks = num_blocks;
    p.ref_in = ref_counts;
    p.ref_out = ref_counts_out;
    p.table = block_table;
    p.rows = rows;
    p.max_blocks = max_blocks_per_seq;
    p.seq_lens = seq_lens;
    p.free_rows = free_rows;
    p.count = count;
    p.num_freed = num_freed;
    p.barrier = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + 4 * kPageBarrierWord);
    // (a thread copies four counts)
    const int64_t copy_ctas =
        ref_counts == ref_counts_out ? 0 : (num_blocks + 4 * kPageThreads - 1) / (4 * kPageThreads);
    const int64_t row_ctas =
        int64_t(count) * ((max_blocks_per_seq + kPageThreads - 1) / kPageThreads);
    const int e = launch(free_kernel, copy_ctas > row_ctas ? copy_ctas : row_ctas, 0, stream, p);
    return e == 0 ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" int mla_cache_compact(void* latent_cache, int num_layers, int64_t layer_stride_bytes,
                                 int64_t num_blocks, int entry_bytes, const int32_t* ref_counts,
                                 int32_t* ref_counts_out, const int32_t* block_table,
                                 int32_t* block_table_out, int rows, int max_blocks_per_seq,
                                 const int32_t* seq_lens, int32_t* page_map, int32_t* num_live,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    CompactParams p{};
    int rc = check_cache(latent_cache, num_layers, layer_stride_bytes, num_blocks, entry_bytes,
                         &p.cache);
    if (rc != MLA_OK) return rc;
    if (rows < 0 || max_blocks_per_seq < 1) return MLA_ERR_INVALID_ARG;
    rc = check_counts(ref_counts, ref_counts_out, num_blocks);
    if (rc != MLA_OK) return rc;
    if (rows > 0 && (!block_table || !block_table_out || !seq_lens || !aligned(block_table, 4) ||
                     !aligned(block_table_out, 4) || !aligned(seq_lens, 4) ||
                     !same_or_apart(block_table, block_table_out,
                                    size_t(rows) * size_t(max_blocks_per_seq) * 4)))
        return MLA_ERR_INVALID_ARG;
    if ((page_map && !aligned(page_map, 4)) || (num_live && !aligned(num_live, 4)))
        return MLA_ERR_INVALID_ARG;
    rc = check_workspace(workspace, workspace_bytes, mla_cache_workspace_bytes(num_blocks, 0));
    if (rc != MLA_OK) return rc;
    page_scratch(static_cast<char*>(workspace), num_blocks, 0, &p.ws);
    p.num_blocks = num_blocks;
    p.ref_in = ref_counts;
    p.ref_out = ref_counts_out;
    p.table = block_table;
    p.table_out = block_table_out;
    p.rows = rows;
    p.max_blocks = max_blocks_per_seq;
    p.seq_lens = seq_lens;
    p.page_map = page_map;
    p.num_live = num_live;
    p.chunks = chunks_of(num_blocks);
    const int64_t pieces = (p.cache.page_bytes + kPieceBytes - 1) / kPieceBytes;
    const int64_t entry_ctas =
        (int64_t(rows) * max_blocks_per_seq + kPageThreads - 1) / kPageThreads;
    const int64_t copy_ctas = num_blocks / 2 * num_layers * pieces;   // the most there can be
    const int64_t want = copy_ctas > entry_ctas ? copy_ctas : entry_ctas;
    const int e = launch(compact_kernel, want > p.chunks ? want : p.chunks, 0, stream, p);
    return e == 0 ? MLA_OK : MLA_ERR_CUDA;
}
