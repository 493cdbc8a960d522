// attention_shared.cuh -- attention of one token per request over a paged
// cache, for a batch that shares a prefix.
//
// The prefix is one product for the whole batch: the rows of a query tile are
// 128 / G requests x the G query heads of a key head, and every key of the
// prefix is read once for all of them (compute bound from some hundred rows
// on).  A request's own keys are read for its G rows alone (memory bound).
// Both run on the tensor cores in one persistent kernel (tcgen05, as the
// prompt kernel), and a second one joins the partial results.
//
// Work is a row of steps of 128 keys: the prefix of each group of requests and
// key head, then each request's own keys for each key head.  The row is cut
// into equal parts by cost, one for each CTA, wherever the cuts fall, so all
// CTAs end together whatever the lengths are.  A piece of a group on a CTA
// leaves its unnormalised output, maximum and sum in the workspace, at slot
// (group + CTA): that number grows along the row, so no two pieces share it.
//
// Two query tiles are in flight per CTA, one in its softmax while the tensor
// core works on the other.  A group of up to 128 rows has only one tile of
// rows: both tiles then hold the same rows and take the steps in turn.
// A group of up to 32 rows (a request's own keys, a small batch) would leave
// one warp of each tile to go through 128 keys alone, some 2600 cycles: its
// rows stand four times in the tile, at lanes 0, 32, 64 and 96, and the warp of
// each copy takes 32 of the step's keys, its weights of the others being zero.
// The four are pieces of their own for the join.  Zero times an infinite value
// is NaN: a copy whose output holds NaN puts those channels right at its end
// from the values themselves (16-bit caches; int8 codes are finite).
//
// Q has two buffers.  A piece of two tiles of rows fills both; others use them
// in turn, one for both tiles, so that the next piece's Q is in place before
// its turn (f16 queries over int8 pages take both, for two values each).
//
//   warps 0-3, 4-7   softmax of tile 0 and 1, a thread per row;
//   warps 8-11       int8 codes to f16 (exactly), from raw tiles into the
//                    product's; over 16-bit caches, zeros in V's last rows
//                    behind the keys;
//   warp 12          issues tcgen05.mma;
//   warp 13          cuts the work, and loads Q where it needs no scaling;
//   warp 14          scales Q over int8 caches, for the next piece while the
//                    tiles' last steps run (pieces of up to 32 rows; the
//                    softmax warps do it for larger ones: one warp alone took
//                    29000 cycles for 128 rows);
//   warp 15          keys and values by TMA.
//
// What bounds it (one B200; times of both kernels): over a long prefix the
// chain of a tile's softmax and products, as in the prompt kernel, with the
// scores read twice from TMEM for want of registers -- 256 requests over 32768
// bf16 keys 90 us (0.46 of the measured peak), over int8 ones 105 us, with f16
// queries 116; over own keys, int8, shared memory: 224 KB pass through it for a
// step of 128 keys (raw codes in and out, f16 tiles in, operands of the
// products), 1750 cycles -- 256 requests of 512 own keys 64 us, 134 MB (2.1
// TB/s; 69 us from a cold L2), f16 queries 72; bf16 66 us, 268 MB (4.0 TB/s;
// cold 79).  One step of one request takes 12 us, two launches among it.
//
// Pages of 8, 16, 32 .. tokens come by TMA, a box of up to 128 tokens of one
// page.  Other page sizes come
// by 16-byte asynchronous copies of warps 8-11, which cost those warps 790
// cycles for a tile of 128 int8 keys, as much again as the conversion.
//
// int8 caches: value = (code - offset) * scale per channel.  q is multiplied
// by the key scale in fp32, scaled by a power of two per row to f16's range
// and rounded to f16 -- one value for bf16 queries (2^-11, an eighth of their
// own half step), a sum of two for f16 queries (2^-22).  The key offset adds
// the same to all scores of a row and only enters lse; the value scale and
// offset are applied to the joined output.
#pragma once

#include "attention_common.cuh"
#include "tcgen05.cuh"

namespace kvq {

constexpr int SA_THREADS = 512;
constexpr int SA_KEYS = 128;
constexpr int SA_ITEMS = 3;
constexpr int SA_MAX_CTAS = 148;
constexpr int SA_BAD = 8;                          // steps whose missing keys are remembered
constexpr int SA_PAGES = 3;                        // steps whose page numbers are kept
constexpr float SA_SLACK = 7.0f;
constexpr uint64_t SA_WAIT_NS = 2000000000ull;

// tiles of the ring of keys and values (f16 or bf16), raw int8 tiles behind
// it, and copies in flight; 224 KB with the two query tiles at D = 128
__host__ __device__ constexpr int sa_ring(bool i8) { return i8 ? 3 : 5; }
__host__ __device__ constexpr int sa_lag(bool i8) { return i8 ? 3 : 2; }
__host__ __device__ constexpr uint32_t sa_tile_bytes(int D) { return 128u * (uint32_t)D * 2u; }
__host__ __device__ constexpr uint32_t sa_smem_bytes(int D, bool i8) {
    return (2u + (uint32_t)sa_ring(i8)) * sa_tile_bytes(D) + (i8 ? (uint32_t)(sa_lag(i8) + 1) * sa_tile_bytes(D) / 2u : 0u) +
           768u + SA_PAGES * 512u + 512u;          // + barriers and items, places of keys, exponents
}

// The cost of a step, by which the work is cut: two tiles of rows, one tile
// (prefix), a request's own keys over int8 and over 16-bit pages.  Measured
// with own steps at 3 (as two tiles) and at 2: 40 requests, prefix 2000, own 1
// to 1500, bf16: 41 and 32 us; 256 requests, prefix 32768, own 1 to 1024, int8:
// 235 and 220 us.  A piece's own start and end are not in it: the CTAs that get
// the pieces of 256 lists of one step have 48 of them each and end last (prefix
// 32768 bf16: 90 us without own keys, 168 with 16 of each request).
constexpr int SA_COST2 = 3, SA_COST1 = 2, SA_COST_OWN8 = 2, SA_COST_OWN16 = 2;

struct SharedPlan {
    int32_t group;           // requests of a prefix group
    int32_t n_groups;        // groups of requests
    int32_t blocks;          // prefix steps of a group
    int32_t cost_own;
    int32_t last_alt;        // the last group of requests has one tile of rows
    int32_t tile_rows;       // rows of a tile in a prefix slot
    int32_t own_rows;        // and in an own slot
    int32_t own_slot;        // rows of an own slot: of one tile, or two
    int64_t own_area;        // floats before the own slots
    int64_t stats_area;      // floats before the (maximum, sum) pairs of the prefix slots; own_stats behind
    int64_t own_stats;
    int64_t before;          // floats before the int32 counts of own steps ahead of each request, and of all
    int32_t hilo;
};

struct SharedItem {
    int32_t steps;           // -1: no more work
    int32_t alt;             // both tiles hold the same rows and take the steps in turn
    int32_t own;             // a request's own keys
    int32_t narrow;          // up to 32 rows, four times in each tile
    int32_t b0, nreq;        // requests
    int32_t kh;
    int32_t key0, keys;      // first key of the list, keys in all
    int32_t slot;
};

// ceil(x / k) for x >= 0 and one of the costs
__device__ __forceinline__ int64_t ceil_div(int64_t x, int k) {
    static_assert(SA_COST2 == 3 && SA_COST1 == 2 && SA_COST_OWN8 == 2 && SA_COST_OWN16 == 2, "divisions by constants");
    return k == 2 ? (x + 1) / 2 : (x + 2) / 3;
}

__device__ __forceinline__ int32_t own_blocks(const SharedArgs& a, int b) {
    const int32_t n = a.seq_lens[b];
    return n > 0 && n <= (int64_t)a.cols * a.block ? (n + SA_KEYS - 1) / SA_KEYS : 0;
}

// where prefix group (pt, kh) starts in the row of work, and a step's cost
__device__ __forceinline__ int64_t prefix_start(const SharedArgs& a, const SharedPlan& p, int pt, int kh, int* k) {
    const bool last = pt == p.n_groups - 1;
    const int full = p.hilo ? SA_COST1 : SA_COST2;
    *k = last && p.last_alt ? SA_COST1 : full;
    return ((int64_t)pt * a.Nkv * full + (int64_t)kh * *k) * p.blocks;
}
__device__ __forceinline__ int64_t prefix_cost(const SharedArgs& a, const SharedPlan& p) {
    if (p.blocks == 0) return 0;
    int k;
    const int64_t s = prefix_start(a, p, p.n_groups - 1, a.Nkv - 1, &k);
    return s + (int64_t)k * p.blocks;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// four int8 codes -> four f16 values: 1024 + (code + 128) is an f16 whose low
// byte is the code with its sign bit flipped
__device__ __forceinline__ void i8x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t x = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t l = __byte_perm(x, 0x64646464u, 0x4140), h = __byte_perm(x, 0x64646464u, 0x4342);
    __half2 a = __hsub2(*reinterpret_cast<__half2*>(&l), bias), b = __hsub2(*reinterpret_cast<__half2*>(&h), bias);
    lo = *reinterpret_cast<uint32_t*>(&a);
    hi = *reinterpret_cast<uint32_t*>(&b);
}

// The order in which a piece's tiles are loaded, which is that of their use:
// K0 K1 V0 K2 V1 .. V(n-1) where the tiles of rows take the steps in turn, else
// K0 V0 K1 V1 ..  Tile q of 2 n: whether it holds values, and its step.
__device__ __forceinline__ bool tile_of(int q, int n, bool alt, int* step) {
    if (!alt) {
        *step = q >> 1;
        return q & 1;
    }
    const bool is_v = q > 0 && ((q & 1) == 0 || q == 2 * n - 1);
    *step = q == 0 ? 0 : is_v ? (q == 2 * n - 1 ? n - 1 : (q - 2) / 2) : (q + 1) / 2;
    return is_v;
}

// TMA load of box {x, y, z, w} of a cache [pages, block, Nkv, D]
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t head, int32_t token,
                                              int32_t page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

template <int T, int C, int D, bool TM>
__global__ void __launch_bounds__(SA_THREADS, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q1,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ SharedArgs a, const __grid_constant__ SharedPlan plan) {
    constexpr bool I8 = C == ATT_I8;
    constexpr int MT = I8 ? ATT_F16 : T;                     // type of the products
    constexpr bool HILO = I8 && T == ATT_F16;
    constexpr int NS = sa_ring(I8), LAG = sa_lag(I8), NR = LAG + 1;
    constexpr int PANELS = D / 64;
    constexpr uint32_t TILE = sa_tile_bytes(D), PANEL = 128 * 128, O_COL = 256;
    extern __shared__ __align__(1024) uint8_t smem[];        // no room for slack: the swizzle needs the alignment
    uint8_t* q_s = smem;
    uint8_t* kv_s = smem + 2 * TILE;
    uint8_t* raw_s = smem + (2 + NS) * TILE;
    uint8_t* after = raw_s + (I8 ? NR * (TILE / 2) : 0);
    volatile uint32_t* row_at = reinterpret_cast<volatile uint32_t*>(after);             // [SA_PAGES][128]
    volatile uint8_t* q_exp = after + SA_PAGES * 512;                                    // [2][2][128]
    uint64_t* q_full = reinterpret_cast<uint64_t*>(after + SA_PAGES * 512 + 512);
    uint64_t* q_empty = q_full + 2;
    uint64_t* s_full = q_empty + 2;
    uint64_t* p_ready = s_full + 2;
    uint64_t* o_full = p_ready + 2;
    uint64_t* item_full = o_full + 2;
    uint64_t* item_empty = item_full + SA_ITEMS;
    uint64_t* kv_full = item_empty + SA_ITEMS;
    uint64_t* kv_empty = kv_full + NS;
    // raw_full: int8 tiles by TMA; over 16-bit caches the last V tiles of pieces, before their
    // zeros, in turn (at most 3 of them are in a ring of 5)
    uint64_t* raw_full = kv_empty + NS;
    uint64_t* raw_empty = raw_full + 4;
    uint64_t* page_bar = raw_empty + 4;
    uint64_t* drain = page_bar + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* bad = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);      // [SA_BAD]
    volatile uint32_t* key_ok = bad + SA_BAD;                                          // [SA_BAD][4]: a bit per key
    volatile SharedItem* items = reinterpret_cast<volatile SharedItem*>(tmem_slot + 2 + SA_BAD + 4 * SA_BAD);
    int* s_blocks = reinterpret_cast<int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a bounded wait of a whole warp
    auto all_wait = [](uint64_t* bar, uint32_t parity, uint64_t ns) {
        return __all_sync(FULL_MASK, mbar_wait_ns(bar, parity, ns)) != 0;
    };
    const int TOK = 128 / a.G;

    if (smem_u32(smem) & 1023u) {                            // uniform over the grid; never on this hardware
        if (threadIdx.x == 0) raise_fault(FAULT_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], I8 ? 4 : 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 128);
            mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < SA_ITEMS; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 13 + (I8 ? 1 : 0) + (TM ? 1 : 0));       // 8 softmax warps, 8-11, 12, and those of 14, 15 in use
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], !I8 && TM ? 5 : 128);         // by TMA: the issuer and warps 8-11
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        mbar_init(page_bar, 128);
        mbar_init(drain, 1);
        mbar_init_fence();
        *s_blocks = 0;
        for (int i = 0; i < SA_BAD; ++i) bad[i] = 0u;
    }
    if (TM && warp == 15 && lane < 2) tma_prefetch_map(lane ? &tm_v : &tm_k);
    if (!I8 && warp == 13 && lane < 2) tma_prefetch_map(lane ? &tm_q1 : &tm_q);
    if (warp == 12) tm_alloc(tmem_slot, 512);
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    // all requests' own steps
    {
        int n = 0;
        for (int b = threadIdx.x; b < a.B; b += SA_THREADS) n += own_blocks(a, b);
        n = __reduce_add_sync(FULL_MASK, n);
        if (lane == 0 && n) atomicAdd(s_blocks, n);
    }
    __syncthreads();
    const int64_t pre_cost = prefix_cost(a, plan);
    const int64_t total = pre_cost + (int64_t)*s_blocks * a.Nkv * plan.cost_own;
    const int64_t width = (total + gridDim.x - 1) / gridDim.x;

    // The K and V tiles of a piece by TMA, all lanes of one warp: a lane for
    // each stretch of `box` tokens that lies in one page.  `tile_no` and
    // `step_no` count over all pieces.
    auto load_tiles = [&](int n, bool alt, int own, int b0, int kh, int key0, int keys, uint32_t& tile_no, uint32_t& step_no,
                          uint32_t& tails) -> bool {
        constexpr int EB = I8 ? 1 : 2;
        const int32_t* list = own ? a.table + (int64_t)b0 * a.table_stride : a.prefix_table;
        const int box = min(a.block, SA_KEYS), pieces = SA_KEYS / box;
        for (int q = 0; q < 2 * n; ++q, ++tile_no) {
            int s;
            const bool is_v = tile_of(q, n, alt, &s);
            const int t = s * SA_KEYS + lane * box;
            const bool wanted = lane < pieces && t < keys;
            int32_t page = -1;
            if (wanted) page = list[(key0 + t) >> a.block_shift];
            const bool there = (uint32_t)page < (uint32_t)a.num_pages;
            const unsigned got = __ballot_sync(FULL_MASK, there), lost = __ballot_sync(FULL_MASK, wanted && !there);
            const uint32_t st = I8 ? tile_no % NR : tile_no % NS, turn = I8 ? tile_no / NR : tile_no / NS;
            if (!__all_sync(FULL_MASK, mbar_wait_ns(I8 ? &raw_empty[st] : &kv_empty[st], (turn & 1u) ^ 1u, SA_WAIT_NS))) return false;
            uint8_t* tile = I8 ? raw_s + st * (TILE / 2) : kv_s + st * TILE;
            if (lost) {
                // pages that are not there: their keys are marked, and their rows of V hold zeros
                if (!is_v) {
                    if (lane < 4) {
                        uint32_t have = 0;
                        for (int k = 0; k < 32; ++k) have |= ((got >> ((32 * lane + k) / box)) & 1u) << k;
                        key_ok[(step_no % SA_BAD) * 4 + lane] = have;
                    }
                    if (lane == 0) {
                        bad[step_no % SA_BAD] = step_no + 1;
                        raise_fault(FAULT_SLOT_RANGE);
                    }
                } else if (!I8) {
                    for (int k = lane; k < SA_KEYS * 8 * PANELS; k += 32)
                        if ((lost >> ((k >> 3) % SA_KEYS / box)) & 1u)
                            *reinterpret_cast<uint4*>(tile + (k >> 3) / SA_KEYS * PANEL + (k >> 3) % SA_KEYS * 128 + (k & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                __syncwarp();
            }
            if (!is_v) ++step_no;
            const bool tail = !I8 && is_v && s == n - 1 && keys < n * SA_KEYS;
            uint64_t* bar = I8 ? &raw_full[st] : tail ? &raw_full[tails++ % 4] : &kv_full[st];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, (uint32_t)__popc(got) * box * D * EB);
                if (tail) mbar_arrive(&kv_full[st]);
            }
            __syncwarp();
            if (there) {
                const CUtensorMap* map = is_v ? &tm_v : &tm_k;
                const int32_t in = (key0 + t) & (a.block - 1);
                if (I8) {
                    tma_load_page(smem_u32(tile) + lane * box * D, map, 0, kh, in, page, bar);
                } else {
                    for (int p = 0; p < PANELS; ++p)
                        tma_load_page(smem_u32(tile) + p * PANEL + lane * box * 128, map, 64 * p, kh, in, page, bar);
                }
            }
        }
        return true;
    };
    // no load may still be in flight when the CTA exits
    auto drain_tiles = [&](uint32_t tile_no) {
        constexpr uint32_t R = I8 ? NR : NS;
        for (uint32_t k = tile_no > R ? tile_no - R : 0; k < tile_no; ++k)
            mbar_wait_ns(I8 ? &raw_full[k % R] : &kv_full[k % R], (k / R) & 1u, SA_WAIT_NS);
    };

    // Rows [begin, end) of Q (requests from b0 on) times the key scale into buffer i,
    // by one warp: LPR lanes share a row, 16 channels each.
    auto scale_rows = [&](int i, int begin, int end, int b0, int kh, int own, bool copies, uint32_t parity) {
        constexpr int LPR = D / 16, RPP = 32 / LPR;          // rows of a pass
        const int sub = lane % LPR, c16 = sub * 16;
        float sc[16];
        const float4* sk = reinterpret_cast<const float4*>(a.scale_k + kh * D + c16);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const float4 e = __ldg(sk + z);
            sc[4 * z] = e.x;
            sc[4 * z + 1] = e.y;
            sc[4 * z + 2] = e.z;
            sc[4 * z + 3] = e.w;
        }
        uint4 e[4][2];
#pragma unroll 1
        for (int r0 = begin; r0 < end; r0 += 4 * RPP) {
            // four passes' loads are in flight together
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int lr = r0 + z * RPP + lane / LPR;
                const int b = b0 + (own ? 0 : lr / a.G), h = kh * a.G + (own ? lr : lr % a.G);
                const uint4* q = reinterpret_cast<const uint4*>(a.q.base + ((int64_t)b * a.q.tok + h * a.q.head + c16) * 2);
                e[z][0] = lr < end ? q[0] : make_uint4(0u, 0u, 0u, 0u);
                e[z][1] = lr < end ? q[1] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (r0 + u * RPP >= end) break;
                const int lr = r0 + u * RPP + lane / LPR;
                const bool live = lr < end;
                const uint4 e0 = e[u][0], e1 = e[u][1];
                const uint32_t ew[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
                float x[16], top = 0.0f;
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    float lo, hi;
                    unpack2<T>(ew[z], lo, hi);
                    x[2 * z] = __fmul_rn(lo, sc[2 * z]);
                    x[2 * z + 1] = __fmul_rn(hi, sc[2 * z + 1]);
                    top = fmaxf(top, fmaxf(fabsf(x[2 * z]), fabsf(x[2 * z + 1])));
                }
#pragma unroll
                for (int d = 1; d < LPR; d <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, d));
                // the power of two below the row's largest; 127 (times one) where there is none
                uint32_t ex = __float_as_uint(top) >> 23;
                if (ex == 0 || ex >= 254) ex = 127;
                const float down = __uint_as_float((254u - ex) << 23);
                if (live) {
                    if (sub == 0) q_exp[(parity * 2 + i) * 128 + lr] = (uint8_t)ex;
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int z = 0; z < 8; ++z) {
                        const float a0 = __fmul_rn(x[2 * z], down), a1 = __fmul_rn(x[2 * z + 1], down);
                        hi[z] = pack2<ATT_F16>(a0, a1);
                        if (HILO) {
                            float h0, h1;
                            unpack2<ATT_F16>(hi[z], h0, h1);
                            lo[z] = pack2<ATT_F16>(__fsub_rn(a0, h0), __fsub_rn(a1, h1));
                        }
                    }
                    for (int r = lr; r < (copies ? 128 : lr + 1); r += 32) {
                        uint8_t* row = q_s + i * TILE + (sub / 4) * PANEL + r * 128;
                        const int p0 = ((2 * (sub & 3)) ^ (r & 7)) << 4, p1 = ((2 * (sub & 3) + 1) ^ (r & 7)) << 4;
                        *reinterpret_cast<uint4*>(row + p0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(row + p1) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                        if (HILO) {
                            *reinterpret_cast<uint4*>(row + TILE + p0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                            *reinterpret_cast<uint4*>(row + TILE + p1) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                        }
                    }
                }
            }
        }
    };

    // 512 threads x 128 registers at launch, split 256 x 160 + 128 x 120 + 128 x 72
    if (warp == 13) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // ---------------- work, and Q where TMA can bring it ----------------
        uint32_t n_item = 0, q_n[2] = {0, 0};
        int q_next = 0;                                      // buffer of Q of the next piece that uses one
        const int64_t hi = min((int64_t)(blockIdx.x + 1) * width, total);
        int64_t at = (int64_t)blockIdx.x * width;
        // where the last piece was: a prefix group, or a request among the 32 whose steps the
        // lanes hold (cb: the first one, not loaded yet at -32; cstart: where their steps start)
        int pt = 0, cb = -32;
        int64_t cstart = pre_cost;
        int32_t nb = 0, incl = 0;
        bool dead = false;
        while (!dead) {
            SharedItem w;
            w.steps = -1;
            while (at < hi && w.steps <= 0) {
                int64_t gs;
                int32_t blocks, len;
                int k;
                if (at < pre_cost) {
                    int next;
                    while (pt + 1 < plan.n_groups && prefix_start(a, plan, pt + 1, 0, &next) <= at) ++pt;
                    gs = prefix_start(a, plan, pt, 0, &k);
                    w.own = 0;
                    w.b0 = pt * plan.group;
                    w.nreq = min(plan.group, a.B - w.b0);
                    w.alt = HILO || w.nreq <= TOK;
                    blocks = plan.blocks;
                    len = a.prefix_len;
                    w.slot = pt * a.Nkv;
                } else {
                    k = plan.cost_own;
                    unsigned past = 0;
                    for (;;) {
                        past = __ballot_sync(FULL_MASK, cb >= 0 && cstart + (int64_t)incl * a.Nkv * k > at);
                        if (past) break;
                        cstart += (int64_t)__shfl_sync(FULL_MASK, incl, 31) * a.Nkv * k;
                        cb += 32;
                        if (cb >= a.B) break;
                        nb = cb + lane < a.B ? own_blocks(a, cb + lane) : 0;
                        incl = nb;
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1) {
                            const int32_t y = __shfl_up_sync(FULL_MASK, incl, d);
                            if (lane >= d) incl += y;
                        }
                    }
                    if (!past) break;
                    const int src = __ffs(past) - 1;
                    w.b0 = cb + src;
                    blocks = __shfl_sync(FULL_MASK, nb, src);
                    gs = cstart + (int64_t)(__shfl_sync(FULL_MASK, incl, src) - blocks) * a.Nkv * k;
                    w.own = 1;
                    w.nreq = 1;
                    w.alt = 1;
                    len = a.seq_lens[w.b0];
                    w.slot = w.b0 * a.Nkv;
                }
                const int64_t cost = (int64_t)k * blocks;
                w.kh = 0;
                while (gs + cost <= at) {
                    gs += cost;
                    ++w.kh;
                }
                // the steps that start in this CTA's part (divisions only at its ends)
                const int32_t s0 = at > gs ? (int32_t)ceil_div(at - gs, k) : 0;
                const int32_t s1 = gs + cost <= hi ? blocks : (int32_t)min(ceil_div(hi - gs, k), (int64_t)blocks);
                at = gs + cost;
                if (s1 > s0) {
                    w.steps = s1 - s0;
                    w.key0 = s0 * SA_KEYS;
                    w.keys = min(len - w.key0, w.steps * SA_KEYS);
                    w.narrow = w.alt && w.nreq * a.G <= 32;
                    w.slot += w.kh + (int)blockIdx.x;
                }
            }
            const uint32_t slot = n_item % SA_ITEMS;
            if (!__all_sync(FULL_MASK, mbar_wait_ns(&item_empty[slot], ((n_item / SA_ITEMS) & 1u) ^ 1u, SA_WAIT_NS))) break;
            if (lane == 0) {
                volatile SharedItem& o = items[slot];
                o.steps = w.steps;
                o.alt = w.alt;
                o.own = w.own;
                o.narrow = w.narrow;
                o.b0 = w.b0;
                o.nreq = w.nreq;
                o.kh = w.kh;
                o.key0 = w.key0;
                o.keys = w.keys;
                o.slot = w.slot;
                mbar_arrive(&item_full[slot]);
            }
            __syncwarp();
            ++n_item;
            if (w.steps < 0) break;
            if (!I8 && lane == 0) {
                for (int i = w.alt ? q_next : 0; i < (w.alt ? q_next + 1 : 2) && !dead; ++i) {
                    if (!mbar_wait_ns(&q_empty[i], (q_n[i] & 1u) ^ 1u, SA_WAIT_NS)) {
                        dead = true;
                        break;
                    }
                    ++q_n[i];
                    // tm_q: a whole tile of requests; tm_q1: as many as 32 rows hold, or one
                    const int few = a.G <= 32 ? 32 / a.G : 1;
                    const bool one = w.narrow || w.own;
                    const int copies = w.narrow ? 4 : 1;
                    mbar_arrive_expect_tx(&q_full[i], (uint32_t)(one ? few * copies : TOK) * a.G * 128u * PANELS);
                    for (int p = 0; p < PANELS; ++p) {
                        uint8_t* dst = q_s + i * TILE + p * PANEL;
                        if (!one) tma_load_3d(dst, &tm_q, 64 * p, w.kh * a.G, w.b0 + (w.alt ? 0 : i * TOK), &q_full[i]);
                        for (int z = 0; one && z < copies; ++z)
                            tma_load_3d(dst + z * 32 * 128, &tm_q1, 64 * p, w.kh * a.G, w.b0, &q_full[i]);
                    }
                }
            }
            if (w.alt) q_next ^= 1;
            dead = __shfl_sync(FULL_MASK, dead, 0);
        }
        if (!I8 && lane == 0)
            for (int i = 0; i < 2; ++i)
                if (q_n[i] > 0) mbar_wait_ns(&q_full[i], (q_n[i] - 1) & 1u, SA_WAIT_NS);
    } else if (warp == 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // ---------------- tensor-core products ----------------
        const uint32_t lead = lane == 0;
        {
            constexpr bool BF = MT == ATT_BF16;
            constexpr uint32_t ID_S = umma_idesc(BF, false, 128, SA_KEYS), ID_O = umma_idesc(BF, true, 128, D);
            // tiles are used in the order of the ring: one stage and parity to follow
            uint32_t st = 0, turn = 0, q_turn = 0, p_turn = 0;                            // q_turn, p_turn: a bit per tile
            auto wait_kv = [&]() { return all_wait(&kv_full[st], turn, SA_WAIT_NS); };
            auto next_kv = [&]() {
                if (++st == NS) {
                    st = 0;
                    turn ^= 1u;
                }
            };
            const uint32_t q0 = umma_desc_k(smem_u32(q_s)), k0 = umma_desc_k(smem_u32(kv_s)),
                           v0 = umma_desc_mn(smem_u32(kv_s), PANEL);
            auto scores = [&](int i, int buffer) {
                const uint32_t qd = q0 + buffer * (TILE >> 4), kd = k0 + st * (TILE >> 4);
                tm_fence_after();
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const uint32_t off = ((d / 4) * PANEL + (d % 4) * 32) >> 4;
                    umma_ss(tmem + 128 * i, qd + off, kd + off, ID_S, d != 0, lead);
                    if (HILO) umma_ss(tmem + 128 * i, qd + (TILE >> 4) + off, kd + off, ID_S, true, lead);
                }
                umma_done(&s_full[i], lead);
            };
            auto values = [&](int i, bool first) {
                const uint32_t vd = v0 + st * (TILE >> 4), d_at = tmem + O_COL + D * i, p_at = tmem + 128 * i;
                tm_fence_after();
#pragma unroll
                for (int d = 0; d < SA_KEYS / 16; ++d) umma_ts(d_at, p_at + 8 * d, vd + 128 * d, ID_O, !first || d != 0, lead);
            };
            auto wait_q = [&](int i) {
                const uint32_t parity = q_turn >> i & 1u;
                q_turn ^= 1u << i;
                return all_wait(&q_full[i], parity, SA_WAIT_NS);
            };
            auto wait_p = [&](int i) {
                const uint32_t parity = p_turn >> i & 1u;
                p_turn ^= 1u << i;
                return all_wait(&p_ready[i], parity, SA_WAIT_NS);
            };
            bool ok = true;
            int q_next = 0;
            for (uint32_t n_item = 0; ok; ++n_item) {
                const uint32_t slot = n_item % SA_ITEMS;
                if (!all_wait(&item_full[slot], (n_item / SA_ITEMS) & 1u, SA_WAIT_NS)) break;
                const int n = __shfl_sync(FULL_MASK, items[slot].steps, 0);
                const bool alt = __shfl_sync(FULL_MASK, items[slot].alt, 0) != 0;
                if (lead) mbar_arrive(&item_empty[slot]);
                if (n < 0) break;
                // the first scores of each tile
                const int buffer = q_next;
                for (int i = 0; i < 2 && ok; ++i) {
                    if (alt && i >= n) break;
                    if (!alt || i == 0) ok = wait_q(alt ? buffer : i);
                    ok = ok && (i == 1 && !alt ? true : wait_kv());
                    if (!ok) break;
                    scores(i, alt ? buffer : i);
                    if (alt ? i + 1 == n : n == 1) umma_done(&q_empty[alt ? buffer : i], lead);
                    if (alt || i == 1) {
                        umma_done(&kv_empty[st], lead);
                        next_kv();
                    }
                }
                if (alt && !HILO) q_next ^= 1;
                if (alt) {
                    for (int s = 0; s < n && ok; ++s) {
                        const int i = s & 1;
                        ok = wait_kv() && wait_p(i);
                        if (!ok) break;
                        values(i, s < 2);
                        umma_done(&kv_empty[st], lead);
                        next_kv();
                        if (s + 2 >= n) {
                            umma_done(&o_full[i], lead);
                        } else {
                            ok = wait_kv();
                            if (!ok) break;
                            scores(i, buffer);
                            umma_done(&kv_empty[st], lead);
                            next_kv();
                            if (s + 3 == n) umma_done(&q_empty[buffer], lead);
                        }
                    }
                } else {
                    for (int s = 0; s < n && ok; ++s) {
                        const uint32_t vs = st, vt = turn;
                        ok = wait_kv();
                        next_kv();
                        const bool more = s + 1 < n;
                        const uint32_t ks = st, kt = turn;
                        for (int i = 0; i < 2 && ok; ++i) {
                            ok = wait_p(i);
                            if (!ok) break;
                            st = vs;
                            turn = vt;
                            values(i, s == 0);
                            st = ks;
                            turn = kt;
                            if (!more) {
                                umma_done(&o_full[i], lead);
                            } else {
                                ok = wait_kv();
                                if (!ok) break;
                                scores(i, i);
                                if (s + 2 == n) umma_done(&q_empty[i], lead);
                            }
                        }
                        if (!ok) break;
                        umma_done(&kv_empty[vs], lead);
                        if (more) {
                            umma_done(&kv_empty[ks], lead);
                            next_kv();
                        }
                    }
                }
            }
            umma_done(drain, lead);
            all_wait(drain, 0u, SA_WAIT_NS);
        }
    } else if (warp >= 14) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (TM && warp == 15) {
            // ---------------- K and V tiles ----------------
            uint32_t tile_no = 0, step_no = 0, tails = 0;
            for (uint32_t n_item = 0;; ++n_item) {
                const uint32_t slot = n_item % SA_ITEMS;
                if (!__all_sync(FULL_MASK, mbar_wait_ns(&item_full[slot], (n_item / SA_ITEMS) & 1u, SA_WAIT_NS))) break;
                const int n = items[slot].steps, own = items[slot].own, b0 = items[slot].b0, kh = items[slot].kh;
                const bool alt = items[slot].alt != 0;
                const int key0 = items[slot].key0, keys = items[slot].keys;
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[slot]);
                if (n < 0 || !load_tiles(n, alt, own, b0, kh, key0, keys, tile_no, step_no, tails)) break;
            }
            drain_tiles(tile_no);
        }
        if (blockIdx.x == 0 && warp == 14) {
            // ---------------- for the join: the own steps of the requests before each one ----------------
            int32_t* before = reinterpret_cast<int32_t*>(reinterpret_cast<float*>(a.workspace) + plan.before);
            int32_t sum = 0;
            for (int b0 = 0; b0 < a.B; b0 += 32) {
                const int32_t nb = b0 + lane < a.B ? own_blocks(a, b0 + lane) : 0;
                int32_t incl = nb;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int32_t y = __shfl_up_sync(FULL_MASK, incl, d);
                    if (lane >= d) incl += y;
                }
                if (b0 + lane < a.B) before[b0 + lane] = sum + incl - nb;
                sum += __shfl_sync(FULL_MASK, incl, 31);
            }
            if (lane == 0) before[a.B] = sum;
        }
        if (I8 && warp == 14) {
            // ---------------- Q times the key scale ----------------
            uint32_t used[2] = {0, 0};
            int q_next = 0;
            bool ok = true;
            for (uint32_t n_item = 0; ok; ++n_item) {
                const uint32_t slot = n_item % SA_ITEMS;
                if (!__all_sync(FULL_MASK, mbar_wait_ns(&item_full[slot], (n_item / SA_ITEMS) & 1u, SA_WAIT_NS))) break;
                const int steps = items[slot].steps, alt = items[slot].alt, own = items[slot].own;
                const int nreq = items[slot].nreq, kh = items[slot].kh, narrow = items[slot].narrow;
                const int b0 = items[slot].b0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[slot]);
                if (steps < 0) break;
                for (int i = alt ? q_next : 0; i < (alt ? q_next + 1 : 2); ++i) {
                    ok = __all_sync(FULL_MASK, mbar_wait_ns(&q_empty[i], (used[i] & 1u) ^ 1u, SA_WAIT_NS));
                    if (!ok) break;
                    if (narrow) {
                        scale_rows(i, 0, nreq * a.G, b0, kh, own, true, used[i] & 1u);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane < 4) mbar_arrive(&q_full[i]);
                    }
                    ++used[i];
                }
                if (alt && !HILO) q_next ^= 1;
            }
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        // ---------------- keys and values ----------------
        const int p = threadIdx.x - 256;
        constexpr int EB = I8 ? 1 : 2;
        constexpr int CH = D * EB / 16;                      // 16-byte pieces of a row
        constexpr int RP = 128 / CH;                         // rows of a pass
        constexpr int PASSES = 128 / RP;
        const int ch = p % CH, r0 = p / CH;
        const uint32_t row_units = (uint32_t)(a.Nkv * (D * EB / 64)), page_units = (uint32_t)(a.page_bytes / 64);
        uint32_t issued = 0, done = 0, block_no = 0, tails_seen = 0;
        bool ok = true;
        auto finish = [&]() {
            if (I8) {
                // this thread's own copies have arrived: codes to f16
                if (TM) ok = __all_sync(FULL_MASK, mbar_wait_ns(&raw_full[done % NR], (done / NR) & 1u, SA_WAIT_NS));
                if (!ok) return;
                ok = __all_sync(FULL_MASK, mbar_wait_ns(&kv_empty[done % NS], ((done / NS) & 1u) ^ 1u, SA_WAIT_NS));
                if (!ok) return;
                const uint8_t* src = raw_s + (done % NR) * (TILE / 2) + p * 16;
                uint8_t* dst = kv_s + (done % NS) * TILE + (ch / 4) * PANEL;
                const int c0 = 2 * (ch & 3);
                const int first = (ch >> 2) & 1;             // panel 1 starts with the other half: no bank conflict
                uint4 raw[PASSES];
#pragma unroll
                for (int k = 0; k < PASSES; ++k) raw[k] = *reinterpret_cast<const uint4*>(src + k * 2048);
                if (TM) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&raw_empty[done % NR]);
                }
#pragma unroll
                for (int k = 0; k < PASSES; ++k) {
                    const uint4 w = raw[k];
                    const int r = r0 + k * RP;
                    uint4 h[2];
                    i8x4_f16(w.x, h[0].x, h[0].y);
                    i8x4_f16(w.y, h[0].z, h[0].w);
                    i8x4_f16(w.z, h[1].x, h[1].y);
                    i8x4_f16(w.w, h[1].z, h[1].w);
                    uint8_t* row = dst + r * 128;
                    const uint4 e0 = first ? h[1] : h[0], e1 = first ? h[0] : h[1];
                    *reinterpret_cast<uint4*>(row + (((c0 + first) ^ (r & 7)) << 4)) = e0;
                    *reinterpret_cast<uint4*>(row + (((c0 + (first ^ 1)) ^ (r & 7)) << 4)) = e1;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&kv_full[done % NS]);
            ++done;
        };
        for (uint32_t n_item = 0; ok; ++n_item) {
            const uint32_t slot = n_item % SA_ITEMS;
            if (!__all_sync(FULL_MASK, mbar_wait_ns(&item_full[slot], (n_item / SA_ITEMS) & 1u, SA_WAIT_NS))) break;
            const int n = items[slot].steps, own = items[slot].own, b0 = items[slot].b0, kh = items[slot].kh;
            const bool alt = items[slot].alt != 0;
            const int key0 = items[slot].key0, keys = items[slot].keys;
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (n < 0) break;
            if (TM) {
                uint32_t tails = tails_seen;
                for (int q = 0; q < 2 * n && ok; ++q) {
                    if (I8) {
                        finish();
                        continue;
                    }
                    const uint32_t st = done % NS;
                    ok = __all_sync(FULL_MASK, mbar_wait_ns(&kv_empty[st], ((done / NS) & 1u) ^ 1u, SA_WAIT_NS));
                    if (!ok) break;
                    if (q == 2 * n - 1 && keys < n * SA_KEYS) {
                        // V's rows behind the last key, once they are there
                        ok = __all_sync(FULL_MASK, mbar_wait_ns(&raw_full[tails % 4], (tails / 4) & 1u, SA_WAIT_NS));
                        ++tails;
                        if (!ok) break;
                        const int first = keys - (n - 1) * SA_KEYS;
                        for (int k = first * 8 + p; k < SA_KEYS * 8; k += 128)
#pragma unroll
                            for (int z = 0; z < PANELS; ++z)
                                *reinterpret_cast<uint4*>(kv_s + st * TILE + z * PANEL + k * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kv_full[st]);
                    ++done;
                }
                tails_seen = tails;
                continue;
            }
            const int32_t* list = own ? a.table + (int64_t)b0 * a.table_stride : a.prefix_table;
            const int64_t head = (int64_t)kh * D * EB + ch * 16;
            // thread p looks up the place of key p of each step, one step ahead, in units of 64 bytes from the
            // cache's start (a token's values are a multiple of that)
            auto lookup = [&](int s) {
                const int t = s * SA_KEYS + p;
                if (t >= keys) return 0xFFFFFFFFu;
                const uint32_t tok = (uint32_t)(key0 + t);
                const uint32_t e = a.block_shift >= 0 ? tok >> a.block_shift : tok / (uint32_t)a.block;
                const int32_t page = list[e];
                const uint32_t in = (tok - e * (uint32_t)a.block) * row_units;
                return (uint32_t)page < (uint32_t)a.num_pages ? (uint32_t)page * page_units + in : 0xFFFFFFFFu;
            };
            const uint32_t block0 = block_no;
            uint32_t next = lookup(0);
            for (int q = 0; q < 2 * n && ok; ++q) {
                int s;
                const bool is_v = tile_of(q, n, alt, &s);
                if (!I8) {
                    ok = __all_sync(FULL_MASK, mbar_wait_ns(&kv_empty[issued % NS], ((issued / NS) & 1u) ^ 1u, SA_WAIT_NS));
                    if (!ok) break;
                }
                volatile uint32_t* place = row_at + ((block0 + s) % SA_PAGES) * 128;
                if (!is_v) {
                    const bool there = next != 0xFFFFFFFFu;
                    place[p] = next;
                    const unsigned word = __ballot_sync(FULL_MASK, there);
                    if (lane == 0) key_ok[(block_no % SA_BAD) * 4 + (p >> 5)] = word;
                    if (!there && s * SA_KEYS + p < keys) {
                        bad[block_no % SA_BAD] = block_no + 1;
                        raise_fault(FAULT_SLOT_RANGE);
                    }
                    ++block_no;
                    mbar_arrive(page_bar);
                    ok = __all_sync(FULL_MASK, mbar_wait_ns(page_bar, (block_no & 1u) ^ 1u, SA_WAIT_NS));
                    if (!ok) break;
                    if (s + 1 < n) next = lookup(s + 1);
                }
                const uint8_t* base = (is_v ? a.v_cache : a.k_cache) + head;
                const uint32_t dst = I8 ? smem_u32(raw_s + (issued % NR) * (TILE / 2) + p * 16)
                                        : smem_u32(kv_s + (issued % NS) * TILE + (ch / 8) * PANEL);
                uint32_t at[PASSES];
#pragma unroll
                for (int k = 0; k < PASSES; ++k) at[k] = place[r0 + k * RP];
#pragma unroll
                for (int k = 0; k < PASSES; ++k) {
                    const int r = r0 + k * RP;
                    const bool there = at[k] != 0xFFFFFFFFu;
                    cp_async16(I8 ? dst + k * 2048 : dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                               base + (there ? (uint64_t)at[k] * 64u : 0u), there ? 16u : 0u);
                }
                cp_async_commit();
                ++issued;
                if (issued - done > LAG) {
                    cp_async_wait<LAG>();
                    finish();
                }
            }
        }
        cp_async_wait<0>();
        while (!TM && ok && done < issued) finish();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        // ---------------- softmax and partial results ----------------
        const int i = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_t = tmem + lanes + 128 * i, o_t = tmem + lanes + O_COL + D * i;
        const float c0 = fmaxf(fabsf(a.scale) * ATT_LOG2E, 1.17549435e-38f);          // not 0: -inf stays -inf
        const uint32_t flip = a.scale < 0.0f ? 0x80000000u : 0u;
        constexpr float SHIFT = MT == ATT_F16 ? ATT_F16_SHIFT : 0.0f;
        float* ws = reinterpret_cast<float*>(a.workspace);
        uint32_t s_n = 0, o_n = 0, q_n[2] = {0, 0}, block_no = 0;        // q_n: uses of the buffers of Q
        int q_next = 0;
        bool ok = true;
        for (uint32_t n_item = 0; ok; ++n_item) {
            const uint32_t slot = n_item % SA_ITEMS;
            if (!__all_sync(FULL_MASK, mbar_wait_ns(&item_full[slot], (n_item / SA_ITEMS) & 1u, SA_WAIT_NS))) break;
            SharedItem w;
            w.steps = items[slot].steps;
            w.alt = items[slot].alt;
            w.own = items[slot].own;
            w.narrow = items[slot].narrow;
            w.b0 = items[slot].b0;
            w.nreq = items[slot].nreq;
            w.kh = items[slot].kh;
            w.key0 = items[slot].key0;
            w.keys = items[slot].keys;
            w.slot = items[slot].slot;
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
            if (w.steps < 0) break;
            const int first = w.alt ? i : 0, stride = w.alt ? 2 : 1;
            const int rows = (w.alt ? w.nreq : min(max(w.nreq - i * TOK, 0), TOK)) * a.G;
            const int lr = w.narrow ? lane : r;
            const bool live = lr < rows;
            const bool work = __any_sync(FULL_MASK, live);
            const int buffer = w.alt ? q_next : i;
            const uint32_t use = buffer ? q_n[1] : q_n[0];
            if (!w.alt || buffer == 0) ++q_n[0];
            if (!w.alt || buffer == 1) ++q_n[1];
            if (w.alt && !HILO) q_next ^= 1;
            if (I8 && !w.narrow && (!w.alt || i == 0)) {
                // Q of this piece: a quarter of the rows each warp, once the products that read the
                // buffer before are done
                ok = __all_sync(FULL_MASK, mbar_wait_ns(&q_empty[buffer], (use & 1u) ^ 1u, SA_WAIT_NS));
                if (!ok) break;
                const int begin = (warp & 3) * 32;
                scale_rows(buffer, begin, min(begin + 32, rows), w.b0 + (w.alt ? 0 : i * TOK), w.kh, w.own, false, use & 1u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[buffer]);
            }
            float c = c0;
            float m = -INFINITY, l = 0.0f;
            for (int s = first; s < w.steps; s += stride) {
                ok = __all_sync(FULL_MASK, mbar_wait_ns(&s_full[i], s_n++ & 1u, SA_WAIT_NS));
                if (!ok) break;
                tm_fence_after();
                if (I8 && s == first) {
                    // the row's power of two (Q of this piece is in place: S came from it)
                    const uint32_t ex = q_exp[((use & 1u) * 2 + buffer) * 128 + lr];
                    c = fmaxf(__fmul_rn(c0, __uint_as_float(ex << 23)), 1.17549435e-38f);
                }
                const int see = w.keys - s * SA_KEYS;
                const uint32_t blk = block_no + s;
                const bool gaps = bad[blk % SA_BAD] == blk + 1;
                // a new maximum: the reference m, the sum and O move to it; false if a wait ran out
                auto refer = [&](float bm) {
                    const bool grow = live && !(__fmul_rn(__fsub_rn(bm, m), c) <= SA_SLACK) && bm != -INFINITY;
                    if (s == first) {
                        m = bm;
                    } else if (__any_sync(FULL_MASK, grow)) {
                        const float f = !grow ? 1.0f : m == -INFINITY ? 0.0f : ex2(__fmul_rn(__fsub_rn(m, bm), c));
                        if (grow) m = bm;
                        l = __fmul_rn(l, f);
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            uint32_t o[32];
                            tm_ld32(o_t + k, o);
#pragma unroll
                            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__fmul_rn(__uint_as_float(o[q]), f));
                            tm_st32(o_t + k, o);
                        }
                    }
                };
                if (w.narrow) {
                    // this warp's 32 keys
                    const int k0 = 32 * (warp & 3);
                    uint32_t have = see - k0 >= 32 ? 0xFFFFFFFFu : see > k0 ? (1u << (see - k0)) - 1u : 0u;
                    if (gaps) have &= key_ok[(blk % SA_BAD) * 4 + (warp & 3)];
                    uint32_t x[32];
                    tm_ld32(s_t + k0, x);
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) x[k + q] = (have >> (k + q)) & 1u ? x[k + q] ^ flip : 0xFF800000u;
                        mx[0] = max3(mx[0], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                        mx[1] = max3(mx[1], __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
                    }
                    refer(max3(mx[0], mx[1], mx[1]));
                    const float ms = m == -INFINITY ? 0.0f : __fmaf_rn(m, c, -SHIFT);
                    const uint64_t c2 = f32x2(c, c), ms2 = f32x2(-ms, -ms);
                    uint64_t sum = 0ull;
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float lo, hi;
                        f32x2_split(fma2(f32x2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), c2, ms2), lo, hi);
                        lo = ex2(lo);
                        hi = ex2(hi);
                        sum = add2(sum, f32x2(lo, hi));
                        pk[k] = pack2<MT>(lo, hi);
                    }
                    float s0, s1;
                    f32x2_split(sum, s0, s1);
                    l = __fadd_rn(l, __fadd_rn(s0, s1));
                    tm_st16(s_t + 16 * (warp & 3), pk);
#pragma unroll
                    for (int k = 0; k < 16; ++k) pk[k] = 0u;
#pragma unroll 1
                    for (int z = 1; z < 4; ++z) tm_st16(s_t + 16 * ((warp + z) & 3), pk);
                    tm_wait_st();
                } else if (work) {
                    if (flip | (see < SA_KEYS) | gaps) {
                        // the uncommon cases are put right in TMEM, to keep the common code short:
                        // a negative scale, keys that are not there
#pragma unroll 1
                        for (int k0 = 0; k0 < SA_KEYS; k0 += 32) {
                            uint32_t have = see - k0 >= 32 ? 0xFFFFFFFFu : see > k0 ? (1u << (see - k0)) - 1u : 0u;
                            if (gaps) have &= key_ok[(blk % SA_BAD) * 4 + k0 / 32];
                            uint32_t x[32];
                            tm_ld32(s_t + k0, x);
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] = (have >> k) & 1u ? x[k] ^ flip : 0xFF800000u;
                            tm_st32(s_t + k0, x);
                        }
                        tm_wait_st();
                    }
                    // the scores are read twice, 64 at a time: for the maximum and for the weights
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        uint32_t x[64];
                        tm_ld64(s_t + 64 * half, x);
#pragma unroll
                        for (int k = 0; k < 64; k += 8) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mx[q] = max3(mx[q], __uint_as_float(x[k + 2 * q]), __uint_as_float(x[k + 2 * q + 1]));
                        }
                    }
                    const float bm = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
                    refer(bm);
                    const float ms = m == -INFINITY ? 0.0f : __fmaf_rn(m, c, -SHIFT);
                    const uint64_t c2 = f32x2(c, c), ms2 = f32x2(-ms, -ms);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        // the weights go over scores that have been read: keys 0 .. 127 into columns 0 .. 63
                        uint32_t x[64];
                        tm_ld64(s_t + 64 * half, x);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t pk[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const uint64_t xx = fma2(f32x2(__uint_as_float(x[32 * g + 2 * k]), __uint_as_float(x[32 * g + 2 * k + 1])), c2, ms2);
                                float lo, hi;
                                f32x2_split(xx, lo, hi);
                                lo = ex2(lo);
                                hi = ex2(hi);
                                sum[k & 1] = add2(sum[k & 1], f32x2(lo, hi));
                                pk[k] = pack2<MT>(lo, hi);
                            }
                            tm_st16(s_t + 32 * half + 16 * g, pk);
                        }
                    }
                    float s0, s1, s2, s3;
                    f32x2_split(sum[0], s0, s1);
                    f32x2_split(sum[1], s2, s3);
                    l = __fadd_rn(l, __fadd_rn(__fadd_rn(s0, s1), __fadd_rn(s2, s3)));
                    tm_wait_st();
                }
                tm_fence_before();
                mbar_arrive(&p_ready[i]);
            }
            if (!ok) break;
            block_no += w.steps;
            if (first >= w.steps) continue;
            ok = __all_sync(FULL_MASK, mbar_wait_ns(&o_full[i], o_n++ & 1u, SA_WAIT_NS));
            if (!ok) break;
            tm_fence_after();
            if (work) {
                const int tile_rows = w.own ? plan.own_rows : plan.tile_rows;
                const int64_t row = (int64_t)w.slot * (w.own ? plan.own_slot : 2 * tile_rows) + i * tile_rows + (w.narrow ? (warp & 3) * rows : 0) + lr;
                float* o_out = ws + (w.own ? plan.own_area : 0) + row * D;
                float any_nan = 0.0f;                        // NaN once a value is
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    uint32_t o[32];
                    tm_ld32(o_t + k, o);
                    if (!I8) {
#pragma unroll
                        for (int q = 0; q < 32; q += 2) any_nan = max3(any_nan, __uint_as_float(o[q]), __uint_as_float(o[q + 1]));
                    }
                    if (live) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            reinterpret_cast<uint4*>(o_out + k)[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    }
                }
                // (a row whose sum is NaN stays NaN whatever is done here)
                if (!I8 && w.narrow && __any_sync(FULL_MASK, live && any_nan != any_nan && l == l)) {
                    // The copies' zero weights met values of V that are not finite (0 * Inf is NaN).  Every row of
                    // the piece sees those values, so where one stands the joined channel is the sum of such
                    // values alone: this copy's part of it is the sum over its own 32 keys of each step, 0 if
                    // they hold none.  A lane looks at one channel of all keys.
                    const int32_t* list = w.own ? a.table + (int64_t)w.b0 * a.table_stride : a.prefix_table;
#pragma unroll 1
                    for (int k = 0; k < D; k += 32) {
                        float own = 0.0f;
                        bool odd = false;
#pragma unroll 1
                        for (int s = first; s < w.steps; s += stride) {
                            const int n = min(w.keys - s * SA_KEYS, SA_KEYS);
#pragma unroll 4
                            for (int t = 0; t < n; ++t) {
                                const uint32_t tok = (uint32_t)(w.key0 + s * SA_KEYS + t);
                                const uint32_t e = a.block_shift >= 0 ? tok >> a.block_shift : tok / (uint32_t)a.block;
                                const int32_t page = list[e];
                                if ((uint32_t)page >= (uint32_t)a.num_pages) continue;
                                const int64_t v = ((int64_t)(tok - e * (uint32_t)a.block) * a.Nkv + w.kh) * D + k + lane;
                                const float x = att_load<T>(a.v_cache + (int64_t)page * a.page_bytes, v);
                                if (fabsf(x) < INFINITY) continue;
                                odd = true;
                                if ((t >> 5) == (warp & 3)) own = __fadd_rn(own, x);
                            }
                        }
                        const unsigned odds = __ballot_sync(FULL_MASK, odd);
                        uint32_t o[32];
                        __syncwarp();
                        tm_ld32(o_t + k, o);
#pragma unroll
                        for (int q = 0; q < 32; ++q) {
                            const float x = __shfl_sync(FULL_MASK, own, q), y = __uint_as_float(o[q]);
                            if (live && (odds >> q & 1u) && y != y) o_out[k + q] = x;
                        }
                    }
                }
                if (live) {
                    float2* st = reinterpret_cast<float2*>(ws + (w.own ? plan.own_stats : plan.stats_area)) + row;
                    // a row with a NaN score has no maximum, but its sum, NaN, must count
                    *st = make_float2(l != l ? 0.0f : m == -INFINITY ? m : __fmaf_rn(m, c, -SHIFT), l);
                }
            }
            tm_fence_before();
        }
    }
    tm_fence_before();
    __syncthreads();
    if (warp == 12) {
        tm_fence_after();
        tm_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Join the pieces: one warp per request and head, a lane finding each piece and
// four rows in flight; 256 requests x 16 heads of 8 to 20 pieces in about 10 us
// (latency: a chain of counts, sums and rows, each a trip to L2).  Piece i: O_i, l_i relative
// to 2^M_i; out = sum 2^(M_i - M) O_i / sum 2^(M_i - M) l_i, then the value
// scale and offset.
// ---------------------------------------------------------------------------
constexpr int SJ_THREADS = 256;

template <int T, int C, int D>
__global__ void __launch_bounds__(SJ_THREADS, 4) shared_join_kernel(const __grid_constant__ SharedArgs a,
                                                                const __grid_constant__ SharedPlan plan, int ctas,
                                                                int hblocks) {
    constexpr bool HILO = C == ATT_I8 && T == ATT_F16;
    constexpr int E = D / 32;
    __shared__ int64_t s_at[SJ_THREADS / 32][32];            // the pieces found: where and how much
    __shared__ float s_w[SJ_THREADS / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / hblocks, h = (int)(blockIdx.x % hblocks) * (SJ_THREADS / 32) + warp;
    const int TOK = 128 / a.G;
    const float* ws = reinterpret_cast<const float*>(a.workspace);
    const int32_t* counts = reinterpret_cast<const int32_t*>(ws + plan.before);
    pdl_wait();
    pdl_trigger();
    if (h >= a.Nq || own_length(a, b) < 0) return;
    const int nb = own_blocks(a, b);
    const int64_t pre_cost = prefix_cost(a, plan);
    int64_t own_before = 0, own_all = 0;
    if (ctas > 0) {
        own_before = counts[b];
        own_all = counts[a.B];
    }
    const int64_t total = pre_cost + own_all * a.Nkv * plan.cost_own;
    const bool small = total < 0x7fffffff;                    // 32-bit divisions take a fraction of the time
    const int64_t width = ctas == 0 ? 1 : small ? (uint32_t)(total + ctas - 1) / (uint32_t)ctas : (total + ctas - 1) / ctas;
    auto cta_of = [&](int64_t x) { return (int)(small ? (uint32_t)x / (uint32_t)width : x / width); };
    const int kh = h / a.G, g = h - kh * a.G;

    // The pieces of the row: those of its prefix group, then those of its own
    // keys.  A group's steps of cost k start at gs and are cut at multiples of
    // width; it has a piece for each CTA from c0 on, tile (both, where they take
    // the steps in turn) and copy.
    struct Group {
        int64_t gs, base, stats;                              // base: floats before the slots
        int32_t k, blocks, first, count, per, copies, narrow, tile, slot, row;
    };
    auto group_of = [&](int64_t gs, int k, int blocks, bool alt, int narrow, int slot, int tile, int row, int64_t base,
                        int64_t stats) {
        Group x;
        x.gs = gs;
        x.k = k;
        x.blocks = blocks;
        x.copies = narrow ? 4 : 1;
        x.per = alt ? 2 * x.copies : 1;
        x.first = blocks > 0 ? cta_of(gs) : 0;
        x.count = blocks > 0 ? (cta_of(gs + (int64_t)k * blocks - 1) - x.first + 1) * x.per : 0;
        x.narrow = narrow;
        x.tile = alt ? -1 : tile;
        x.slot = slot;
        x.row = row;
        x.base = base;
        x.stats = stats;
        return x;
    };
    Group pre, mine;
    {
        const int pt = b / plan.group, q = b - pt * plan.group;
        const int nreq = min(plan.group, a.B - pt * plan.group);
        const bool alt = HILO || nreq <= TOK;
        int k = 2;
        int64_t gs = 0;
        if (plan.blocks > 0) gs = prefix_start(a, plan, pt, kh, &k);
        const int tile = alt ? 0 : q / TOK;
        pre = group_of(gs, k, plan.blocks, alt, alt && nreq * a.G <= 32 ? nreq * a.G : 0, pt * a.Nkv + kh, tile,
                         (q - tile * TOK) * a.G + g, 0, plan.stats_area);
        mine = group_of(pre_cost + (own_before * a.Nkv + (int64_t)kh * nb) * plan.cost_own, plan.cost_own, nb, true,
                         a.G <= 32 ? a.G : 0, b * a.Nkv + kh, 0, g, plan.own_area, plan.own_stats);
    }
    float M = -INFINITY, L = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int n0 = 0; n0 < pre.count + mine.count; n0 += 32) {
        // a lane looks at one piece
        int n = n0 + lane;
        const bool own = n >= pre.count;
        if (own) n -= pre.count;
        Group x;                                              // chosen field by field: no array in local memory
        x.gs = own ? mine.gs : pre.gs;
        x.base = own ? mine.base : pre.base;
        x.stats = own ? mine.stats : pre.stats;
        x.k = own ? mine.k : pre.k;
        x.blocks = own ? mine.blocks : pre.blocks;
        x.first = own ? mine.first : pre.first;
        x.count = own ? mine.count : pre.count;
        x.per = own ? mine.per : pre.per;
        x.copies = own ? mine.copies : pre.copies;
        x.narrow = own ? mine.narrow : pre.narrow;
        x.tile = own ? mine.tile : pre.tile;
        x.slot = own ? mine.slot : pre.slot;
        x.row = own ? mine.row : pre.row;
        float2 st = make_float2(-INFINITY, 0.0f);
        int64_t at = 0;
        if (n < x.count) {
            const int c = x.first + n / x.per, z = n % x.per, i = x.tile < 0 ? z / x.copies : x.tile;
            const int64_t lo = (int64_t)c * width - x.gs, hi = lo + width;
            const int64_t s0 = lo > 0 ? ceil_div(lo, x.k) : 0;
            const int64_t s1 = min(ceil_div(hi, x.k), (int64_t)x.blocks);
            if (s1 - s0 > (x.tile < 0 ? i : 0)) {
                const int64_t r = (int64_t)(x.slot + c) * (own ? plan.own_slot : 2 * plan.tile_rows) +
                                  i * (own ? plan.own_rows : plan.tile_rows) + z % x.copies * x.narrow + x.row;
                st = reinterpret_cast<const float2*>(ws + x.stats)[r];
                at = x.base + r * D;
            }
        }
        float top = st.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, d));
        const float mn = fmaxf(M, top);
        if (mn == -INFINITY) continue;                        // nothing visible so far
        const float f = exp2f(__fsub_rn(M, mn));
        const bool has = st.x != -INFINITY;
        const float w = has ? exp2f(__fsub_rn(st.x, mn)) : 0.0f;
        float sum = has ? __fmul_rn(st.y, w) : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(FULL_MASK, sum, d));
        L = __fmaf_rn(L, f, sum);
        M = mn;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = __fmul_rn(acc[e], f);
        const unsigned mask = __ballot_sync(FULL_MASK, has);
        const int count = __popc(mask);
        __syncwarp();
        if (has) {
            const int to = __popc(mask & ((1u << lane) - 1u));
            s_at[warp][to] = at;
            s_w[warp][to] = w;
        }
        __syncwarp();
        // 4 rows in flight: one after the other they cost a memory latency each
        for (int r0 = 0; r0 < count; r0 += 4) {
            float v[4][E];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (r0 + r < count) {
                    const float* o = ws + s_at[warp][r0 + r] + lane * E;
                    if (E == 4) *reinterpret_cast<float4*>(v[r]) = *reinterpret_cast<const float4*>(o);
                    else *reinterpret_cast<float2*>(v[r]) = *reinterpret_cast<const float2*>(o);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (r0 + r < count) {
                    const float wr = s_w[warp][r0 + r];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = __fmaf_rn(v[r][e], wr, acc[e]);
                }
            }
        }
    }
    const bool any = M != -INFINITY;
    const float inv = any ? __frcp_rn(L) : 0.0f;
    const int d0 = lane * E;
    uint32_t packed[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        float v[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            v[z] = any ? __fmul_rn(acc[e + z], inv) : 0.0f;
            if (C == ATT_I8 && any) {
                if (a.offset_v) v[z] = __fsub_rn(v[z], __ldg(a.offset_v + kh * D + d0 + e + z));
                v[z] = __fmul_rn(v[z], __ldg(a.scale_v + kh * D + d0 + e + z));
            }
        }
        packed[e / 2] = pack2<T>(v[0], v[1]);
    }
    // the key offset's share of every score of the row; before the store, since out may be q
    float off = 0.0f;
    if (C == ATT_I8 && a.lse && a.offset_k) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            off = __fmaf_rn(__fmul_rn(att_load<T>(a.q.base, (int64_t)b * a.q.tok + h * a.q.head + d0 + e),
                                      __ldg(a.scale_k + kh * D + d0 + e)), __ldg(a.offset_k + kh * D + d0 + e), off);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) off = __fadd_rn(off, __shfl_xor_sync(FULL_MASK, off, d));
    }
    uint8_t* out = a.out.base + ((int64_t)b * a.out.tok + h * a.out.head + d0) * 2;
    if (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(packed[0], packed[E / 2 - 1]);
    else *reinterpret_cast<uint32_t*>(out) = packed[0];
    if (a.lse && lane == 0)
        a.lse[(int64_t)b * a.Nq + h] =
            any ? __fsub_rn(__fmul_rn(__fadd_rn(M, log2f(L)), ATT_LN2), __fmul_rn(off, a.scale)) : -INFINITY;
}

}  // namespace kvq
