// pages.cuh -- the pages of a cache: copied, freed, forked and compacted.
//
// A page is block i of a cache [num_blocks, ...]: `bytes` contiguous bytes at
// base + i * stride.  Several caches (keys, values, their scales, several
// layers) share page numbers, so every move is made in all of them at once.
//
// What bounds these kernels is memory: each moved byte is read and written
// once (2 x bytes at the card's copy rate).  The bookkeeping (page numbers,
// reference counts, table rows) is a few words per page.
#pragma once

#include "kvq_device.cuh"
#include "tma_pipe.cuh"

namespace kvq {

constexpr unsigned FAULT_NO_PAGE = 0x4u;
constexpr int PG_MAX_CACHES = 64;

struct PageCache {
    uint8_t* base;
    int64_t stride;          // bytes between pages
    uint32_t bytes;          // of one page
    uint32_t unit0;          // first copy unit of this cache within a page pair
};

// where the (source, destination) pairs of a copy come from
enum { PG_LIST = 0, PG_FORK = 1, PG_COMPACT = 2 };

struct PageCopyArgs {
    PageCache cache[PG_MAX_CACHES];
    int32_t n_caches;
    uint32_t units;          // copy units of one pair, over all caches
    uint32_t chunk;          // bytes of a unit (the last one of a page may be shorter)
    int64_t n_pairs;
    int64_t num_pages;
    const void* src;         // PG_LIST: source pages; PG_FORK: parent rows
    const void* dst;         // PG_LIST: destination pages; PG_FORK: child rows
    int32_t src_i64, dst_i64;
    const int32_t* pair_page;   // PG_FORK: fresh page of each child (-1, -2: none); PG_COMPACT: page_map
    int32_t* table;             // PG_FORK: the block table; PG_COMPACT: the new table
    const int32_t* old_table;   // PG_COMPACT
    int64_t table_stride, old_table_stride, table_rows, table_cols;
    int32_t* seq_lens;          // PG_FORK
    int32_t* ref_count;         // PG_FORK
    int64_t block_size;         // PG_FORK
};

__device__ __forceinline__ int64_t load_index(const void* p, int i64, int64_t i) {
    return i64 ? static_cast<const int64_t*>(p)[i] : (int64_t)static_cast<const int32_t*>(p)[i];
}

// The pages of pair i; false when there is nothing to copy.  Page numbers
// outside the pool set FAULT_SLOT_RANGE once per pair (`report`).
template <int MODE>
__device__ __forceinline__ bool page_pair(const PageCopyArgs& a, int64_t i, bool report, int64_t& s, int64_t& d) {
    if (MODE == PG_LIST) {
        s = load_index(a.src, a.src_i64, i);
        d = load_index(a.dst, a.dst_i64, i);
        if (s == -1 || d == -1) return false;
    } else if (MODE == PG_FORK) {
        d = a.pair_page[i];
        if (d < 0) return false;
        // the plan has checked the row and its length (partly filled last page)
        const int64_t row = load_index(a.src, a.src_i64, i);
        s = a.table[row * a.table_stride + (a.seq_lens[row] - 1) / a.block_size];
    } else {
        s = i;
        d = a.pair_page[i];
        if (d < 0 || d == s) return false;
    }
    if ((uint64_t)s >= (uint64_t)a.num_pages || (uint64_t)d >= (uint64_t)a.num_pages) {
        if (report) raise_fault(FAULT_SLOT_RANGE);
        return false;
    }
    return s != d;
}

// The addresses and size of copy unit u (0 bytes: nothing to copy).
template <int MODE>
__device__ __forceinline__ uint32_t page_unit(const PageCopyArgs& a, int64_t u, const uint8_t*& src, uint8_t*& dst) {
    const int64_t i = u / a.units;
    const uint32_t r = (uint32_t)(u - i * a.units);
    int64_t s, d;
    if (!page_pair<MODE>(a, i, r == 0, s, d)) return 0u;
    int c = 0;
    while (c + 1 < a.n_caches && r >= a.cache[c + 1].unit0) ++c;
    const uint32_t off = (r - a.cache[c].unit0) * a.chunk;
    src = a.cache[c].base + s * a.cache[c].stride + off;
    dst = a.cache[c].base + d * a.cache[c].stride + off;
    const uint32_t left = a.cache[c].bytes - off;
    return left < a.chunk ? left : a.chunk;
}

// What goes with the pages, before them: the children's rows (PG_FORK: the
// parent's full pages shared and counted, the fresh page, -1 behind them), or
// the renumbered table (PG_COMPACT, in place or not).
template <int MODE>
__device__ __forceinline__ void page_tables(const PageCopyArgs& a) {
    const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, nthr = (int64_t)gridDim.x * blockDim.x;
    if (MODE == PG_FORK) {
        const int lane = threadIdx.x & 31;
        for (int64_t i = tid >> 5; i < a.n_pairs; i += nthr >> 5) {
            const int32_t fresh = a.pair_page[i];
            if (fresh == -2) continue;                        // refused by the plan
            const int64_t p = load_index(a.src, a.src_i64, i), c = load_index(a.dst, a.dst_i64, i);
            const int32_t len = a.seq_lens[p];
            const int64_t full = len / a.block_size;
            for (int64_t e = lane; e < a.table_cols; e += 32) {
                int32_t page = -1;
                if (e < full) {
                    page = a.table[p * a.table_stride + e];
                    if ((uint64_t)page < (uint64_t)a.num_pages) {
                        atomicAdd(a.ref_count + page, 1);
                    } else {
                        raise_fault(FAULT_SLOT_RANGE);
                        page = -1;
                    }
                } else if (e == full && fresh >= 0) {
                    page = fresh;
                    a.ref_count[page] = 1;                    // free until now: no other writer
                }
                a.table[c * a.table_stride + e] = page;
            }
            if (lane == 0) a.seq_lens[c] = len;
        }
    }
    if (MODE == PG_COMPACT) {
        const int64_t n = a.table_rows * a.table_cols;
        for (int64_t k = tid; k < n; k += nthr) {
            const int64_t r = k / a.table_cols, e = k - r * a.table_cols;
            const int32_t page = a.old_table[r * a.old_table_stride + e];
            int32_t to = -1;
            if (page >= 0 && page < a.num_pages) to = a.pair_page[page];
            else if (page != -1) raise_fault(FAULT_SLOT_RANGE);
            a.table[r * a.table_stride + e] = to;
        }
    }
}

// The copies, bound by memory.  W is the widest word that all addresses,
// strides and sizes allow.
// A list's units are looked up one by one, each a load away: 4001 pairs of
// 2 x 32 KB pages in 85 us, 6.2 TB/s, 0.94 of the copy peak (in batches, as
// below, 94 us: more registers, fewer CTAs on an SM).
// Forks and compactions: every warp of a CTA looks up the CTA's next 32 units,
// a lane each (the same loads in all warps, so they need no barrier), and
// drops those with nothing to move; the CTA's threads then move two units at a
// time, all loads before the stores.  A fork's lookup is a chain of four loads
// whose latency is paid once for 32 units that way (480 children, 8 caches:
// 48 -> 34 us), and a compaction, most of whose pages stay, only visits the
// ones that move (1800 of 8192 pages: 82 -> 54 us).
constexpr int PG_THREADS = 256;

template <int MODE, typename W>
__global__ void __launch_bounds__(PG_THREADS) page_copy_words_kernel(const __grid_constant__ PageCopyArgs a) {
    constexpr int PER = 8192 / sizeof(W) / PG_THREADS < 2 ? 2 : 8192 / sizeof(W) / PG_THREADS;   // words of a thread
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    page_tables<MODE>(a);
    const int64_t total = a.n_pairs * a.units;
    if constexpr (MODE == PG_LIST) {
        for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
            const uint8_t* src;
            uint8_t* dst;
            const uint32_t n = page_unit<MODE>(a, u, src, dst) / sizeof(W);
            for (uint32_t k = threadIdx.x; k < n; k += PG_THREADS)
                reinterpret_cast<W*>(dst)[k] = reinterpret_cast<const W*>(src)[k];
        }
    } else {
        for (int64_t base = blockIdx.x; base < total; base += 32 * (int64_t)gridDim.x) {
            const int64_t u = base + lane * (int64_t)gridDim.x;
            const uint8_t* src = nullptr;
            uint8_t* dst = nullptr;
            uint32_t bytes = 0;
            if (u < total) bytes = page_unit<MODE>(a, u, src, dst);
            unsigned todo = __ballot_sync(FULL_MASK, bytes != 0);
            while (todo) {
                const W* from[2];
                W* to[2];
                uint32_t n[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = todo ? __ffs(todo) - 1 : 0;
                    from[k] = reinterpret_cast<const W*>(__shfl_sync(FULL_MASK, reinterpret_cast<uint64_t>(src), at));
                    to[k] = reinterpret_cast<W*>(__shfl_sync(FULL_MASK, reinterpret_cast<uint64_t>(dst), at));
                    n[k] = __shfl_sync(FULL_MASK, bytes, at) / sizeof(W);
                    if (!todo) n[k] = 0;
                    todo &= todo - 1;
                }
                if (sizeof(W) == 16) {
                    W x[2][PER];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int q = 0; q < PER; ++q)
                            if (threadIdx.x + q * PG_THREADS < n[k]) x[k][q] = from[k][threadIdx.x + q * PG_THREADS];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int q = 0; q < PER; ++q)
                            if (threadIdx.x + q * PG_THREADS < n[k]) to[k][threadIdx.x + q * PG_THREADS] = x[k][q];
                } else {
                    for (int k = 0; k < 2; ++k)
                        for (uint32_t i = threadIdx.x; i < n[k]; i += PG_THREADS) to[k][i] = from[k][i];
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// free: one warp per row.  The row's length is taken by one exchange, so a row
// named twice is freed once.
// ---------------------------------------------------------------------------
struct FreeArgs {
    int32_t* table;
    int64_t table_stride, table_rows, table_cols;
    int32_t* seq_lens;
    int32_t* ref_count;
    int64_t num_pages;
    const void* rows;
    int32_t rows_i64;
    int64_t n_rows;
    int64_t block_size;
};

__global__ void __launch_bounds__(128) free_pages_kernel(const FreeArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < a.n_rows; i += nwarps) {
        const int64_t row = load_index(a.rows, a.rows_i64, i);
        if (row == -1) continue;
        if (row < 0 || row >= a.table_rows) {
            if (lane == 0) raise_fault(FAULT_SLOT_RANGE);
            continue;
        }
        int32_t len = 0;
        if (lane == 0) len = atomicExch(a.seq_lens + row, 0);
        len = __shfl_sync(FULL_MASK, len, 0);
        if (len == 0) continue;
        int64_t held = ((int64_t)len + a.block_size - 1) / a.block_size;
        if (len < 0 || held > a.table_cols) {
            if (lane == 0) raise_fault(FAULT_SLOT_RANGE);
            held = len < 0 ? 0 : a.table_cols;
        }
        for (int64_t e = lane; e < a.table_cols; e += 32) {
            int32_t* t = a.table + row * a.table_stride + e;
            if (e < held) {
                const int32_t page = *t;
                if (page < 0 || page >= a.num_pages) {
                    raise_fault(FAULT_SLOT_RANGE);
                } else if (atomicSub(a.ref_count + page, 1) <= 0) {
                    atomicAdd(a.ref_count + page, 1);         // it was free already
                    raise_fault(FAULT_SLOT_RANGE);
                }
            }
            *t = -1;
        }
    }
}

// ---------------------------------------------------------------------------
// block-wide exclusive scan of one int per thread of 1024; total in *sum
// ---------------------------------------------------------------------------
constexpr int PL_THREADS = 1024;

__device__ __forceinline__ int block_scan(int v, int* sum, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                                          // warp_sums of the previous scan are read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, w, d);
        if (lane >= d) w += y;
    }
    *sum = __shfl_sync(FULL_MASK, w, 31);
    const int before = __shfl_sync(FULL_MASK, w, warp > 0 ? warp - 1 : 0);
    return x - v + (warp > 0 ? before : 0);
}

// ---------------------------------------------------------------------------
// fork, the plan: which children are valid and which fresh page each gets.
// One CTA: the lowest free pages go to the children in the order given, which
// is a scan over both.  A child row must be empty; of two entries that name
// the same child the first is taken (a minimum over claims left in the row's
// length, so the answer does not depend on timing), and a row may not be a
// parent and a child of one call.
// A few microseconds: chains of dependent loads, not work.
// fresh[i]: the page to copy the parent's last page into, -1 (whole pages
// only: nothing to copy), or -2 (refused).
// ---------------------------------------------------------------------------
struct ForkArgs {
    const int32_t* ref_count;
    int64_t num_pages;
    int32_t* seq_lens;
    int64_t table_rows, table_cols, block_size;
    const void* parents;
    const void* children;
    int32_t parents_i64, children_i64;
    int32_t n;
    int32_t* fresh;
};

__global__ void __launch_bounds__(PL_THREADS) fork_plan_kernel(const ForkArgs a) {
    constexpr int RING = 8192;
    __shared__ int32_t ring[RING];                            // free pages found and not given yet
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    // the rows and lengths themselves
    for (int i = tid; i < a.n; i += PL_THREADS) {
        const int64_t p = load_index(a.parents, a.parents_i64, i), c = load_index(a.children, a.children_i64, i);
        bool ok = p >= 0 && p < a.table_rows && c >= 0 && c < a.table_rows && p != c;
        if (ok) {
            const int32_t len = a.seq_lens[p];
            ok = len >= 0 && len <= a.table_cols * a.block_size && a.seq_lens[c] == 0;
        }
        a.fresh[i] = ok ? -1 : -2;
        if (!ok && !(p == -1 && c == -1)) raise_fault(FAULT_SLOT_RANGE);
    }
    __syncthreads();
    // claims: -(n - i), the smallest for the first entry
    for (int i = tid; i < a.n; i += PL_THREADS)
        if (a.fresh[i] == -1) atomicMin(a.seq_lens + load_index(a.children, a.children_i64, i), -(a.n - i));
    __syncthreads();
    // fresh pages, in order
    int64_t cursor = 0;
    int head = 0, avail = 0;
    for (int i0 = 0; i0 < a.n; i0 += PL_THREADS) {
        const int i = i0 + tid;
        bool mine = false, need = false, held = false;
        if (i < a.n && a.fresh[i] == -1) {
            const int64_t p = load_index(a.parents, a.parents_i64, i), c = load_index(a.children, a.children_i64, i);
            const int32_t len = __ldcg(a.seq_lens + p);
            held = __ldcg(a.seq_lens + c) == -(a.n - i);
            mine = held && len >= 0;
            need = mine && len % a.block_size != 0;
            if (!mine) raise_fault(FAULT_SLOT_RANGE);
        }
        int cnt, found;
        const int rank = block_scan(need ? 1 : 0, &cnt, warp_sums);
        while (avail < cnt && cursor < a.num_pages) {
            int f[4], k = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t page = cursor + 4 * tid + j;
                f[j] = page < a.num_pages && a.ref_count[page] <= 0;
                k += f[j];
            }
            int at = block_scan(k, &found, warp_sums);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (f[j]) ring[(head + avail + at++) % RING] = (int32_t)(cursor + 4 * tid + j);
            avail += found;
            cursor += 4 * PL_THREADS;
            __syncthreads();
        }
        if (i < a.n && a.fresh[i] == -1) {
            int32_t to = mine ? -1 : -2;
            if (need) {
                to = rank < avail ? ring[(head + rank) % RING] : -2;
                if (to == -2) raise_fault(FAULT_NO_PAGE);
            }
            a.fresh[i] = to;
        }
        const int given = cnt < avail ? cnt : avail;
        head = (head + given) % RING;
        avail -= given;
        __syncthreads();
    }
    // a claim that came to nothing leaves the row empty (the winners' lengths
    // are written with their tables)
    for (int i = tid; i < a.n; i += PL_THREADS) {
        if (a.fresh[i] != -2) continue;
        const int64_t c = load_index(a.children, a.children_i64, i);
        if (c >= 0 && c < a.table_rows && __ldcg(a.seq_lens + c) == -(a.n - i)) a.seq_lens[c] = 0;
    }
}

// ---------------------------------------------------------------------------
// compact, the plan: the U pages in use get the numbers 0 .. U-1.  Those below
// U stay; the others, in ascending order, take the holes below U, in ascending
// order, so that as few pages as possible move and no page is both a source
// and a destination.
// One CTA (8192 pages in 10 us, latency); a thread takes a stretch of consecutive pages, so that three scans
// over the threads' counts order everything.  The list of holes stands at
// page_map[U + i] until the page that takes hole i, which is at U + i or
// above, overwrites it: the pages above U go through the list from the last
// one down, PL_THREADS at a time, each round's reads before its writes.
// ---------------------------------------------------------------------------
struct CompactArgs {
    const int32_t* ref_count;
    int32_t* new_ref;          // may be ref_count
    int32_t* page_map;
    int32_t num_pages;
};

__global__ void __launch_bounds__(PL_THREADS) compact_plan_kernel(const CompactArgs a) {
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, n = a.num_pages;
    pdl_wait();
    pdl_trigger();
    const int len = (n + PL_THREADS - 1) / PL_THREADS, p0 = min(tid * len, n), p1 = min(p0 + len, n);
    int mine = 0, used, unused;
    // (the count of all does not care who reads which page: neighbours for neighbours, loads ahead)
#pragma unroll 8
    for (int p = tid; p < n; p += PL_THREADS) mine += a.ref_count[p] > 0;
    block_scan(mine, &used, warp_sums);
    // the holes below U, and the pages that stay
    const int q1 = min(p1, used);
    mine = 0;
    for (int p = p0; p < q1; ++p) mine += a.ref_count[p] <= 0;
    int at = used + block_scan(mine, &unused, warp_sums);
    for (int p = p0; p < q1; ++p) {
        const bool hole = a.ref_count[p] <= 0;
        if (hole) a.page_map[at++] = p;
        a.page_map[p] = hole ? -1 : p;
    }
    __syncthreads();
    int below = unused;                                       // pages to move that are not visited yet: as many as holes
    for (int top = n; top > used; top -= PL_THREADS) {
        const int p = top - 1 - tid;                          // descending over the threads
        const bool in = p >= used, moved = in && a.ref_count[p] > 0;
        int cnt;
        const int rank = block_scan(moved ? 1 : 0, &cnt, warp_sums);
        int to = -1;
        if (moved) to = __ldcg(a.page_map + used + (below - 1 - rank));
        __syncthreads();
        if (in) a.page_map[p] = to;
        below -= cnt;
    }
    __syncthreads();
    for (int q = tid; q < n; q += 4 * PL_THREADS) {
        int to[4], r[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int p = q + z * PL_THREADS;
            to[z] = p < n ? __ldcg(a.page_map + p) : -1;
            r[z] = p < n ? a.ref_count[p] : 0;
        }
        // in place: a page's new place below U was a hole, or the page itself, so no count that is still
        // to be read is written here
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int p = q + z * PL_THREADS;
            if (to[z] >= 0) a.new_ref[to[z]] = r[z];
            if (p < n && p >= used) a.new_ref[p] = 0;
        }
    }
}

}  // namespace kvq
