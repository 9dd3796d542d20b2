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
//            to ceil(L / 64).   count pass -> assign pass -> share + copy pass
//   free     counts - 1 for each entry of the named rows.
//   compact  M live pages. The k-th live page with id >= M goes to the k-th
//            free id below M: the fewest moves that leave the live pages in
//            [0, M), and no destination is another move's source, so the
//            copies run in any order.   count pass -> list pass -> move pass
//
// The passes are separate launches chained by programmatic dependent launch:
// a grid-wide prefix sum needs all counts before the first rank. Each CTA of
// the second pass sums the chunk counts below its own itself (num_blocks /
// 1024 values), which costs less than a third launch for a scan.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "mla_device.cuh"

namespace mla {
namespace {

constexpr int kPageThreads = 256;
constexpr int kWarps = kPageThreads / 32;
constexpr int kChunkIters = 4;
constexpr int kChunk = kPageThreads * kChunkIters;   // pages whose counts one CTA reads
constexpr int kMaxChildren = 8192;                   // their page offsets fit shared memory
constexpr int kPieceBytes = 8192;                    // bytes of a page that one CTA copies at once

__device__ __forceinline__ void grid_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

struct CacheView {
    char* base;
    int64_t layer_stride;   // bytes
    int64_t page_bytes;
    int layers;
};

// Where the passes of one call leave what the next ones need (in the
// caller's workspace, behind the status header).
struct PageScratch {
    int32_t* status;
    int32_t* go;            // fork: 1 if the call goes ahead
                            // compact: [0] live pages M, [1] pages to move
    int32_t* chunk_count;   // [chunks] free (fork) or live (compact) pages of each chunk
    uint32_t* live_bits;    // compact: one bit per page
    int32_t* need;          // fork: [children] fresh pages, -1 for a child that cannot be made
    int32_t* src;           // compact: [moves] ascending
    int32_t* dst;           //          [moves] ascending
    int32_t* moved_ref;     //          [moves] count of src[k]
};

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
    for (int i = threadIdx.x; i < n; i += kPageThreads) s += counts[i];
    return block_sum(s, tmp);
}

// Pages of this CTA's chunk whose count is zero (or not).
__device__ __forceinline__ int count_chunk(const int32_t* ref, int64_t num_blocks, bool zero,
                                           int* tmp) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kChunkIters; ++i) {
        const int64_t page = int64_t(blockIdx.x) * kChunk + i * kPageThreads + threadIdx.x;
        if (page < num_blocks) n += (ref[page] == 0) == zero;
    }
    return block_sum(n, tmp);
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

// CTAs [0, chunks): free pages of a chunk. The others: one warp per child
// checks it and writes how many fresh pages it needs.
__global__ void __launch_bounds__(kPageThreads) fork_count_kernel(const ForkParams p) {
    __shared__ int tmp[kWarps];
    grid_launch_dependents();
    if (int(blockIdx.x) < p.chunks) {
        const int n = count_chunk(p.ref_in, p.num_blocks, true, tmp);
        if (threadIdx.x == 0) p.ws.chunk_count[blockIdx.x] = n;
        return;
    }
    const int c = (blockIdx.x - p.chunks) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (c >= p.children) return;
    const int parent = p.parents[c], S = p.shared_lens[c], L = p.child_lens[c];
    int bad = MLA_OK, detail = 0;
    if (S < 0 || L < S || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
        bad = MLA_ERR_BAD_SEQ_LEN;
        detail = S < 0 ? S : L;
    } else if (parent >= p.rows || (parent < 0 && S > 0)) {
        bad = MLA_ERR_BAD_ROW;
        detail = parent;
    } else {
        // Every page that the child shares or copies from is in use.
        const int32_t* row = p.table + int64_t(parent) * p.max_blocks;
        for (int j = lane; j < pages_of(S); j += 32) {
            const int page = row[j];
            if (page < 0 || int64_t(page) >= p.num_blocks) {
                bad = MLA_ERR_BAD_BLOCK_ID;
                detail = page;
            } else if (p.ref_in[page] == 0) {
                bad = MLA_ERR_PAGE_STATE;
                detail = page;
            }
        }
    }
    if (bad != MLA_OK) record_error(p.ws.status, bad, detail);
    const bool any = __any_sync(0xffffffffu, bad != MLA_OK);
    if (lane == 0) p.ws.need[c] = any ? -1 : pages_of(L) - S / kPageSize;
}

// Every CTA: the children's page offsets, then its chunk's free pages to
// their owners and the chunk's counts.
__global__ void __launch_bounds__(kPageThreads) fork_assign_kernel(const ForkParams p) {
    __shared__ int tmp[kWarps];
    __shared__ int warp_free[kChunkIters * kWarps];
    extern __shared__ int off[];      // [children + 1]
    grid_launch_dependents();
    grid_wait();
    int total = 0, invalid = 0;
    bool over = false;
    for (int c0 = 0; c0 < p.children; c0 += kPageThreads) {
        const int c = c0 + threadIdx.x;
        const int n = c < p.children ? p.ws.need[c] : 0;
        if (n < 0) invalid = 1;
        // (one child alone may ask for more than the pool; no sum here wraps)
        int sum;
        const int before = block_exclusive(n < 0 ? 0 : int(min(int64_t(n), p.num_blocks + 1)), tmp,
                                           &sum);
        if (c < p.children) off[c] = total + before;
        over = over || int64_t(total) + sum > p.num_blocks;
        total = over ? 0 : total + sum;
    }
    if (threadIdx.x == 0) off[p.children] = total;
    invalid = block_sum(invalid, tmp);
    const int free_below = sum_below(p.ws.chunk_count, int(blockIdx.x), tmp);
    const int free_all = free_below + [&] {
        int s = 0;
        for (int i = blockIdx.x + threadIdx.x; i < p.chunks; i += kPageThreads)
            s += p.ws.chunk_count[i];
        return block_sum(s, tmp);
    }();
    const bool go = invalid == 0 && !over && total <= free_all;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.ws.go[0] = go ? 1 : 0;
        if (invalid == 0 && !go)
            record_error(p.ws.status, MLA_ERR_NO_PAGES, over ? INT_MAX : total - free_all);
    }

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ref[kChunkIters];
    uint32_t free_mask[kChunkIters];
#pragma unroll
    for (int i = 0; i < kChunkIters; ++i) {
        const int64_t page = int64_t(blockIdx.x) * kChunk + i * kPageThreads + threadIdx.x;
        ref[i] = page < p.num_blocks ? p.ref_in[page] : 1;
        free_mask[i] = __ballot_sync(0xffffffffu, ref[i] == 0);
        if (lane == 0) warp_free[i * kWarps + warp] = __popc(free_mask[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kChunkIters; ++i) {
        const int64_t page = int64_t(blockIdx.x) * kChunk + i * kPageThreads + threadIdx.x;
        if (page >= p.num_blocks) continue;
        if (ref[i] == 0 && go) {
            int rank = free_below + __popc(free_mask[i] & ((1u << lane) - 1u));
            for (int w = 0; w < i * kWarps + warp; ++w) rank += warp_free[w];
            if (rank < total) {
                // The child that owns rank: the last c with off[c] <= rank
                // (children without fresh pages share their successor's offset).
                int lo = 0, hi = p.children;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (off[mid] <= rank) lo = mid; else hi = mid;
                }
                const int j = p.shared_lens[lo] / kPageSize + (rank - off[lo]);
                p.child_table[int64_t(lo) * p.max_blocks + j] = int32_t(page);
                ref[i] = 1;
            }
        }
        p.ref_out[page] = ref[i];
    }
}

// Copy `bytes` (a multiple of 16) of one piece of a page, two 16-byte loads
// in flight per thread before their stores.
__device__ __forceinline__ void copy_piece(const CacheView& cache, int layer, int src, int dst,
                                           int piece, int64_t bytes) {
    const char* s = cache.base + layer * cache.layer_stride + src * cache.page_bytes;
    char* d = cache.base + layer * cache.layer_stride + dst * cache.page_bytes;
    const int64_t o0 = int64_t(piece) * kPieceBytes + threadIdx.x * 16;
    const int64_t o1 = o0 + kPieceBytes / 2;
    uint4 a, b;
    if (o0 < bytes) a = __ldcs(reinterpret_cast<const uint4*>(s + o0));
    if (o1 < bytes) b = __ldcs(reinterpret_cast<const uint4*>(s + o1));
    if (o0 < bytes) __stcs(reinterpret_cast<uint4*>(d + o0), a);
    if (o1 < bytes) __stcs(reinterpret_cast<uint4*>(d + o1), b);
}
static_assert(kPieceBytes == 2 * 16 * kPageThreads, "a piece is two loads per thread");

// One warp per child for its shared pages, then the whole grid copies the
// partly filled pages piece by piece.
__global__ void __launch_bounds__(kPageThreads) fork_copy_kernel(const ForkParams p) {
    grid_wait();
    if (p.ws.go[0] == 0) return;
    const int lane = threadIdx.x & 31;
    for (int c = blockIdx.x * kWarps + (threadIdx.x >> 5); c < p.children;
         c += gridDim.x * kWarps) {
        const int full = p.shared_lens[c] / kPageSize;
        const int32_t* row = p.table + int64_t(p.parents[c]) * p.max_blocks;
        for (int j = lane; j < full; j += 32) {
            const int page = row[j];
            p.child_table[int64_t(c) * p.max_blocks + j] = page;
            atomicAdd(p.ref_out + page, 1);
        }
    }
    const int pieces = int((p.cache.page_bytes + kPieceBytes - 1) / kPieceBytes);
    const int64_t items = int64_t(p.children) * p.cache.layers * pieces;
    const int64_t row_bytes = p.cache.page_bytes / kPageSize;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int c = int(i / (int64_t(p.cache.layers) * pieces));
        const int r = int(i - int64_t(c) * p.cache.layers * pieces);
        const int S = p.shared_lens[c];
        const int64_t bytes = (S % kPageSize) * row_bytes;
        const int piece = r % pieces;
        if (int64_t(piece) * kPieceBytes >= bytes) continue;
        copy_piece(p.cache, r / pieces,
                   p.table[int64_t(p.parents[c]) * p.max_blocks + S / kPageSize],
                   p.child_table[int64_t(c) * p.max_blocks + S / kPageSize], piece, bytes);
    }
}

// ------------------------------------------------------------------- free

struct FreeParams {
    int32_t* status;
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

__global__ void __launch_bounds__(kPageThreads) free_copy_kernel(const FreeParams p) {
    grid_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.num_freed = 0;
    if (p.ref_in == p.ref_out) return;
    for (int64_t i = int64_t(blockIdx.x) * kPageThreads + threadIdx.x; i < p.num_blocks;
         i += int64_t(gridDim.x) * kPageThreads)
        p.ref_out[i] = p.ref_in[i];
}

// CTA (x, r): entries 256x.. of row free_rows[r]. Lanes of a warp that name
// the same page (a prompt that many rows share) take it off with one atomic.
__global__ void __launch_bounds__(kPageThreads) free_rows_kernel(const FreeParams p) {
    grid_wait();
    const int lane = threadIdx.x & 31;
    for (int r = blockIdx.y; r < p.count; r += gridDim.y) {
        const int row = p.free_rows[r];
        if (row < 0 || row >= p.rows) {
            if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.status, MLA_ERR_BAD_ROW, row);
            continue;
        }
        const int L = p.seq_lens[row];
        if (L < 0 || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
            if (blockIdx.x == 0 && threadIdx.x == 0)
                record_error(p.status, MLA_ERR_BAD_SEQ_LEN, L);
            continue;
        }
        const int n = pages_of(L);
        for (int j0 = blockIdx.x * kPageThreads; j0 < n; j0 += gridDim.x * kPageThreads) {
            const int j = j0 + threadIdx.x;
            int page = j < n ? p.table[int64_t(row) * p.max_blocks + j] : -1;
            if (j < n && (page < 0 || int64_t(page) >= p.num_blocks)) {
                record_error(p.status, MLA_ERR_BAD_BLOCK_ID, page);
                page = -1;
            }
            const uint32_t same = __match_any_sync(0xffffffffu, page);
            bool freed = false;
            if (page >= 0 && lane == __ffs(same) - 1) {
                const int off = __popc(same);
                const int old = atomicSub(p.ref_out + page, off);
                freed = old > 0 && old <= off;
                if (old < off) {
                    // More entries than counts: the count stays at 0. What was
                    // taken too much is put back, so whatever the order, the
                    // sum of the atomics on this page is -(what it had).
                    atomicAdd(p.ref_out + page, off - (old > 0 ? old : 0));
                    record_error(p.status, MLA_ERR_PAGE_STATE, page);
                }
            }
            const uint32_t f = __ballot_sync(0xffffffffu, freed);
            if (lane == 0 && f != 0) atomicAdd(p.num_freed, __popc(f));
        }
    }
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

// Live pages of each chunk, and one bit per page: the list pass writes the
// counts in place, so what it needs of other chunks it reads from the bits.
__global__ void __launch_bounds__(kPageThreads) compact_count_kernel(const CompactParams p) {
    __shared__ int tmp[kWarps];
    grid_launch_dependents();
    int n = 0;
#pragma unroll
    for (int i = 0; i < kChunkIters; ++i) {
        const int64_t page = int64_t(blockIdx.x) * kChunk + i * kPageThreads + threadIdx.x;
        const bool live = page < p.num_blocks && p.ref_in[page] != 0;
        const uint32_t bits = __ballot_sync(0xffffffffu, live);
        if ((threadIdx.x & 31) == 0) p.ws.live_bits[page >> 5] = bits;
        n += live;
    }
    n = block_sum(n, tmp);
    if (threadIdx.x == 0) p.ws.chunk_count[blockIdx.x] = n;
}

__global__ void __launch_bounds__(kPageThreads) compact_list_kernel(const CompactParams p) {
    __shared__ int tmp[kWarps];
    __shared__ uint32_t live_bits[kChunk / 32];
    grid_launch_dependents();
    grid_wait();
    const int live_before = sum_below(p.ws.chunk_count, int(blockIdx.x), tmp);
    int rest = 0;
    for (int i = blockIdx.x + threadIdx.x; i < p.chunks; i += kPageThreads)
        rest += p.ws.chunk_count[i];
    const int M = live_before + block_sum(rest, tmp);
    // Live pages below M: those of the whole chunks before M's and of the
    // words of M's chunk up to M.
    const int m_chunk = M / kChunk;
    int part = 0;
    if (m_chunk < p.chunks && threadIdx.x < kChunk / 32) {
        const int first = m_chunk * kChunk + threadIdx.x * 32;
        const uint32_t bits = p.ws.live_bits[first >> 5];
        const int take = M - first;   // bits of this word below M
        part = __popc(take >= 32 ? bits : take > 0 ? bits & ((1u << take) - 1u) : 0u);
    }
    const int live_low = sum_below(p.ws.chunk_count, m_chunk, tmp) + block_sum(part, tmp);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.ws.go[0] = M;
        p.ws.go[1] = M - live_low;
        if (p.num_live != nullptr) *p.num_live = M;
    }
    if (threadIdx.x < kChunk / 32)
        live_bits[threadIdx.x] = p.ws.live_bits[blockIdx.x * (kChunk / 32) + threadIdx.x];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kChunkIters; ++i) {
        const int in = i * kPageThreads + threadIdx.x;
        const int64_t page = int64_t(blockIdx.x) * kChunk + in;
        if (page >= p.num_blocks) continue;
        const uint32_t bits = live_bits[in >> 5];
        int before = live_before + __popc(bits & ((1u << (in & 31)) - 1u));
        for (int w = 0; w < (in >> 5); ++w) before += __popc(live_bits[w]);
        const bool live = (bits >> (in & 31)) & 1u;
        const int ref = p.ref_in[page];
        int to = live ? int(page) : -1;
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
        if (p.page_map != nullptr) p.page_map[page] = to;
    }
}

// Index of `v` in the ascending list a[0..n), or -1.
__device__ __forceinline__ int find(const int32_t* a, int n, int v) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] < v) lo = mid + 1; else hi = mid;
    }
    return lo < n && a[lo] == v ? lo : -1;
}

__global__ void __launch_bounds__(kPageThreads) compact_move_kernel(const CompactParams p) {
    grid_wait();
    const int M = p.ws.go[0], moves = p.ws.go[1];
    const int64_t tid = int64_t(blockIdx.x) * kPageThreads + threadIdx.x;
    const int64_t threads = int64_t(gridDim.x) * kPageThreads;
    for (int64_t k = tid; k < moves; k += threads) {
        const int dst = p.ws.dst[k];
        p.ref_out[dst] = p.ws.moved_ref[k];
        if (p.page_map != nullptr) p.page_map[p.ws.src[k]] = dst;
    }
    const int64_t entries = int64_t(p.rows) * p.max_blocks;
    for (int64_t e = tid; e < entries; e += threads) {
        const int row = int(e / p.max_blocks), j = int(e - int64_t(row) * p.max_blocks);
        const int L = p.seq_lens[row];
        if (L < 0 || int64_t(L) > int64_t(p.max_blocks) * kPageSize) {
            if (j == 0) record_error(p.ws.status, MLA_ERR_BAD_SEQ_LEN, L);
            continue;
        }
        if (j >= pages_of(L)) continue;
        int page = p.table[e];
        if (page < 0 || int64_t(page) >= p.num_blocks) {
            record_error(p.ws.status, MLA_ERR_BAD_BLOCK_ID, page);
        } else if (page >= M) {
            const int k = find(p.ws.src, moves, page);
            if (k < 0) record_error(p.ws.status, MLA_ERR_PAGE_STATE, page);
            else page = p.ws.dst[k];
        } else if (find(p.ws.dst, moves, page) >= 0) {
            record_error(p.ws.status, MLA_ERR_PAGE_STATE, page);   // it was free
        }
        p.table_out[e] = page;
    }
    const int pieces = int((p.cache.page_bytes + kPieceBytes - 1) / kPieceBytes);
    const int64_t per_move = int64_t(p.cache.layers) * pieces;
    const int64_t items = moves * per_move;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int k = int(i / per_move);
        const int r = int(i - k * per_move);
        copy_piece(p.cache, r / pieces, p.ws.src[k], p.ws.dst[k], r % pieces, p.cache.page_bytes);
    }
}

// ------------------------------------------------------------------- host

constexpr int kMaxCacheBlocks = (1 << 23) - 2;   // 256 of these still sum below 2^31
constexpr int kCopyCtas = 152 * 8;               // eight CTAs fill an SM's threads

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int chunks_of(int64_t num_blocks) { return int((num_blocks + kChunk - 1) / kChunk); }

// Scratch layout; returns its size behind the status header.
size_t page_scratch(char* ws, int64_t num_blocks, int children, PageScratch* s) {
    const size_t chunks = size_t(chunks_of(num_blocks));
    const size_t half = round256((size_t(num_blocks) / 2 + 1) * 4);   // moves <= half the pages
    size_t at = kStatusBytes;
    auto take = [&](size_t bytes) {
        char* p = ws + at;
        at += round256(bytes);
        return reinterpret_cast<int32_t*>(p);
    };
    PageScratch t{};
    t.status = reinterpret_cast<int32_t*>(ws);
    t.go = take(8);
    t.chunk_count = take(chunks * 4);
    t.live_bits = reinterpret_cast<uint32_t*>(take(chunks * (kChunk / 8)));
    t.need = take(size_t(children) * 4);
    t.src = take(half);
    t.dst = take(half);
    t.moved_ref = take(half);
    if (s != nullptr) *s = t;
    return at;
}

template <typename Kernel, typename Params>
int launch(Kernel kernel, dim3 grid, size_t smem, void* stream, const Params& p, bool dependent) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kPageThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
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

int min_int(int64_t a, int64_t b) { return int(a < b ? a : b); }

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
    const int checkers = (children + kWarps - 1) / kWarps;
    int e = launch(fork_count_kernel, dim3(unsigned(p.chunks + checkers)), 0, stream, p, false);
    if (e == 0)
        e = launch(fork_assign_kernel, dim3(unsigned(p.chunks)), size_t(children + 1) * 4, stream,
                   p, true);
    if (e == 0 && children > 0) {
        const int64_t pieces = (p.cache.page_bytes + kPieceBytes - 1) / kPieceBytes;
        e = launch(fork_copy_kernel,
                   dim3(unsigned(min_int(int64_t(children) * num_layers * pieces, kCopyCtas))), 0,
                   stream, p, true);
    }
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
    const int64_t copy_ctas =
        ref_counts == ref_counts_out ? 1 : (num_blocks + kPageThreads - 1) / kPageThreads;
    int e = launch(free_copy_kernel, dim3(unsigned(min_int(copy_ctas, kCopyCtas))), 0, stream, p,
                   false);
    if (e == 0 && count > 0) {
        const dim3 grid(unsigned(min_int((max_blocks_per_seq + kPageThreads - 1) / kPageThreads, 64)),
                        unsigned(min_int(count, 32768)));
        e = launch(free_rows_kernel, grid, 0, stream, p, true);
    }
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
    const int64_t most_moves = num_blocks / 2;
    const int64_t entry_ctas =
        (int64_t(rows) * max_blocks_per_seq + kPageThreads - 1) / kPageThreads;
    const int64_t copy_ctas = most_moves * num_layers * pieces;
    int e = launch(compact_count_kernel, dim3(unsigned(p.chunks)), 0, stream, p, false);
    if (e == 0) e = launch(compact_list_kernel, dim3(unsigned(p.chunks)), 0, stream, p, true);
    const int64_t want = copy_ctas > entry_ctas ? copy_ctas : entry_ctas;
    if (e == 0 && want > 0)
        e = launch(compact_move_kernel, dim3(unsigned(min_int(want, kCopyCtas))), 0, stream, p,
                   true);
    return e == 0 ? MLA_OK : MLA_ERR_CUDA;
}
