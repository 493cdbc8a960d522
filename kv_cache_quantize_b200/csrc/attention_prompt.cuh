// attention_prompt.cuh -- attention over whole prompts on the tensor cores.
//
//   S = Q K^T,  P = exp2(c S - m),  O = sum P V,  out = O / sum P
// with c = softmax_scale * log2(e) and one pass over the keys: m is a running
// reference for each row that only has to be near the row's maximum, so O and
// the sum are rescaled only when the maximum has grown by more than a factor
// of 2^PA_SLACK -- a handful of times per row instead of once per key block.
//
// A query tile holds 128 rows: 128 / G consecutive tokens x the G query heads
// that read one key head, so a short prompt fills its tiles with heads and K
// and V are read once for all of them.  One CTA per SM works on two such tiles
// at a time (columns of TMEM: S0, S1, O0, O1 take all 512 columns at D = 128), so
// that the tensor core multiplies for one tile while the other one's softmax
// runs:
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread owns a row; S from
//                   TMEM, P back into the same columns as 16-bit values (the A
//                   operand of P V is read from TMEM), and the epilogue;
//   warp 8          issues tcgen05.mma: P V of block j, then Q K^T of
//                   block j + 1, tile 0 and tile 1 in turn;
//   warp 9          work items and TMA: the grid has a CTA for every item, but a
//                   running CTA takes over items whose CTAs have not started
//                   (cluster launch control; against a fixed assignment 243 ->
//                   215 us for 24 prompts of 1 to 2048 tokens): sequences in
//                   the order given, the heavy items of each first (longest
//                   sequence last instead of first: 197 instead of 194 us);
//                   Q tiles, and a ring of K and V tiles of 128
//                   keys (128-byte swizzle; 5 stages, 4 cost 4 %).
// The tensor pipe executes a CTA's products in order, so Q K^T of block j + 1
// may overwrite the columns that P V of block j reads.
//
// What bounds it: a tile's softmax (about 1980 cycles for 128 keys) and its two
// products (1030 and their latencies) take turns, and two tiles cover each other
// only in part: 3400 cycles for 128 keys of both, where the products alone take
// 2160 (tensor pipe 56 % active).  One prompt of 16384 tokens, 16 / 4 heads of
// 128, bf16: 862 us, 1278 TFLOP/s, 0.78 of the measured peak on a cold card;
// 0.68 in a loop, where the power cap lowers the clock.  An item's start and end
// cost about three blocks, so short prompts are slower: 24 of 1 to 2048 tokens
// 205 us, 660 TFLOP/s.  At D = 64 the products halve and the softmax does not:
// 16384 tokens 768 us, 716 TFLOP/s.  Keys are not split: few queries behind
// many keys fill few SMs (16 tokens behind 100000: 4 items, 1370 us).
//
// A row's weights are rounded to the 16-bit type of V for the product (half a
// step, the rounding that the output itself gets); their sum is taken before.
// f16 weights are scaled up by 2^ATT_F16_SHIFT so that small ones stay normal.
//
// A masked key has weight 0, but 0 * NaN is NaN: V rows behind the sequence's
// last key are zeroed in shared memory, and in blocks that some row of the
// tiles sees only in part, values that are not finite are taken out and given
// back, in the epilogue, to exactly the rows that see them.
#pragma once

#include "attention_common.cuh"
#include "tcgen05.cuh"

namespace kvq {

constexpr int PA_THREADS = 384;                    // 8 softmax warps, MMA, loads, 2 idle (register groups)
constexpr int PA_KEYS = 128;                       // keys of a block
constexpr int PA_ITEMS = 2;                        // work item slots
constexpr float PA_SLACK = 7.0f;                   // log2 of how far above the reference a weight may get
constexpr uint64_t PA_WAIT_NS = 2000000000ull;     // every wait gives up after 2 s

__host__ __device__ constexpr int pa_stages(int D) { return D == 128 ? 5 : 8; }
__host__ __device__ constexpr uint32_t pa_tile_bytes(int D) { return 128u * (uint32_t)D * 2u; }
__host__ __device__ constexpr uint32_t pa_smem_bytes(int D) {
    return (2u + (uint32_t)pa_stages(D)) * pa_tile_bytes(D) + 512u + 1024u;    // + barriers and items + alignment
}

struct PromptItem {
    int32_t n0, n1;          // key blocks of tile 0 and 1; n0 = -1: no more work
    int32_t tok0;            // first query row
    int32_t ntok;            // tokens of the sequence from there on
    int32_t lim0;            // keys that the first token sees (may be <= 0)
    int32_t lk, k0;          // keys of the sequence, first key row
    int32_t kh;              // key head
    int32_t dirty;           // values that are not finite were taken out of V
};

template <int T, int D>
__global__ void __launch_bounds__(PA_THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PromptArgs a) {
    constexpr int NS = pa_stages(D);
    constexpr int PANELS = D / 64;
    constexpr uint32_t TILE = pa_tile_bytes(D);
    constexpr uint32_t PANEL = 128 * 128;
    constexpr uint32_t O_COL = 256;                          // S0 0, S1 128, O0 256, O1 256 + D
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* q_s = smem;
    uint8_t* kv_s = smem + 2 * TILE;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + (2 + NS) * TILE);
    uint64_t* q_empty = q_full + 2;
    uint64_t* s_full = q_empty + 2;
    uint64_t* p_ready = s_full + 2;
    uint64_t* o_full = p_ready + 2;
    uint64_t* item_full = o_full + 2;
    uint64_t* item_empty = item_full + PA_ITEMS;
    uint64_t* kv_full = item_empty + PA_ITEMS;
    uint64_t* kv_empty = kv_full + NS;
    uint64_t* next_item = kv_empty + NS;
    uint64_t* drain = next_item + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile PromptItem* items = reinterpret_cast<volatile PromptItem*>(tmem_slot + 2);
    uint8_t* taken = smem + (2 + NS) * TILE + 496;           // 16 bytes: which CTA's work was taken over
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a bounded wait of a whole warp
    auto all_wait = [](uint64_t* bar, uint32_t parity, uint64_t ns) {
        return __all_sync(FULL_MASK, mbar_wait_ns(bar, parity, ns)) != 0;
    };
    const int TOK = 128 / a.G;                               // tokens of a query tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 128);
            mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < PA_ITEMS; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 9);                    // 8 softmax warps and the MMA lane
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(next_item, 1);
        mbar_init(drain, 1);
        mbar_init_fence();
    }
    if (warp == 9 && lane < 3) tma_prefetch_map(lane == 0 ? &tm_q : lane == 1 ? &tm_k : &tm_v);
    if (warp == 8) tm_alloc(tmem_slot, 512);
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    // 384 threads x 168 registers at launch, split 256 x 216 + 128 x 72
    if (warp == 9) {
        // ---------------- work items and loads ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t q_bytes = (uint32_t)(TOK * a.G) * 128u * PANELS;
        uint32_t pos = 0, n_item = 0, n_asked = 0, n_answered = 0, q_n[2] = {0, 0};
        int cb = 0;
        int64_t cbase = 0;                                   // tiles of the sequences before cb
        bool dead = false;
        int64_t it = blockIdx.x;
        while (!dead) {
            const int64_t x = it / a.Nkv;
            if (x < cbase) {                                 // items come in ascending order; if not, start over
                cb = 0;
                cbase = 0;
            }
            // the sequence and tile of item x: the cursor only moves forward
            bool found = false;
            SeqSpan sp = {0, 0, 0, 0};
            int32_t local = 0, ntiles = 0;
            while (it >= 0 && !found && cb < a.B) {
                const int b = cb + lane;
                int32_t nt = 0;
                SeqSpan s = {0, 0, 0, 0};
                if (b < a.B) {
                    s = prompt_span(a, b);
                    nt = (s.lq + 2 * TOK - 1) / (2 * TOK);
                }
                int32_t incl = nt;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int32_t y = __shfl_up_sync(FULL_MASK, incl, d);
                    if (lane >= d) incl += y;
                }
                const unsigned past = __ballot_sync(FULL_MASK, cbase + incl > x);
                if (past) {
                    const int src = __ffs(past) - 1;
                    found = true;
                    sp.q0 = __shfl_sync(FULL_MASK, s.q0, src);
                    sp.k0 = __shfl_sync(FULL_MASK, s.k0, src);
                    sp.lq = __shfl_sync(FULL_MASK, s.lq, src);
                    sp.lk = __shfl_sync(FULL_MASK, s.lk, src);
                    ntiles = __shfl_sync(FULL_MASK, nt, src);
                    local = (int32_t)(x - cbase - (__shfl_sync(FULL_MASK, incl, src) - ntiles));
                } else {
                    cbase += __shfl_sync(FULL_MASK, incl, 31);
                    cb += 32;
                }
            }
            if (it >= 0) {
                if (lane == 0) take_over(taken, next_item);
                ++n_asked;
            }
            PromptItem w;
            w.n0 = -1;
            w.n1 = 0;
            if (found) {
                const int32_t t0 = (ntiles - 1 - local) * 2 * TOK;       // the longest rows first
                w.tok0 = (int32_t)sp.q0 + t0;
                w.ntok = sp.lq - t0;
                w.lk = sp.lk;
                w.k0 = (int32_t)sp.k0;
                w.kh = (int32_t)(it - x * a.Nkv);
                w.lim0 = a.causal ? t0 + 1 + sp.lk - sp.lq : sp.lk;
                const int32_t nt0 = min(w.ntok, TOK), nt1 = min(w.ntok - TOK, TOK);
                const int32_t m0 = a.causal ? w.lim0 + nt0 - 1 : sp.lk, m1 = a.causal ? w.lim0 + TOK + nt1 - 1 : sp.lk;
                w.n0 = m0 > 0 ? (m0 + PA_KEYS - 1) / PA_KEYS : 0;
                w.n1 = nt1 > 0 && m1 > 0 ? (m1 + PA_KEYS - 1) / PA_KEYS : 0;
            }
            // (the grid may have a few CTAs more than there are items)
            if (found || it < 0) {
                const uint32_t slot = n_item % PA_ITEMS;
                if (!__all_sync(FULL_MASK, mbar_wait_ns(&item_empty[slot], ((n_item / PA_ITEMS) & 1u) ^ 1u, PA_WAIT_NS))) break;
                if (lane == 0) {
                    volatile PromptItem& o = items[slot];
                    o.n0 = w.n0;
                    o.n1 = w.n1;
                    o.tok0 = w.tok0;
                    o.ntok = w.ntok;
                    o.lim0 = w.lim0;
                    o.lk = w.lk;
                    o.k0 = w.k0;
                    o.kh = w.kh;
                    o.dirty = 0;
                    mbar_arrive(&item_full[slot]);
                }
                ++n_item;
                if (it < 0) break;
            }
            if (found && lane == 0) {
                const int n = max(w.n0, w.n1);
                auto load_q = [&](int i) {
                    if ((i ? w.n1 : w.n0) == 0) return true;
                    if (!mbar_wait_ns(&q_empty[i], (q_n[i] & 1u) ^ 1u, PA_WAIT_NS)) return false;
                    ++q_n[i];
                    mbar_arrive_expect_tx(&q_full[i], q_bytes);
                    for (int p = 0; p < PANELS; ++p)
                        tma_load_3d(q_s + i * TILE + p * PANEL, &tm_q, 64 * p, w.kh * a.G, w.tok0 + i * TOK, &q_full[i]);
                    return true;
                };
                auto load_kv = [&](const CUtensorMap* map, int j) {
                    const uint32_t st = pos % NS;
                    if (!mbar_wait_ns(&kv_empty[st], ((pos / NS) & 1u) ^ 1u, PA_WAIT_NS)) return false;
                    mbar_arrive_expect_tx(&kv_full[st], TILE);
                    for (int p = 0; p < PANELS; ++p)
                        tma_load_3d(kv_s + st * TILE + p * PANEL, map, 64 * p, w.kh, w.k0 + j * PA_KEYS, &kv_full[st]);
                    ++pos;
                    return true;
                };
                // the first keys and values need only room in the ring; Q waits for the item before
                dead = (n > 0 && (!load_kv(&tm_k, 0) || !load_kv(&tm_v, 0))) || !load_q(0) || !load_q(1);
                for (int j = 1; j < n && !dead; ++j) dead = !load_kv(&tm_k, j) || !load_kv(&tm_v, j);
            }
            dead = __shfl_sync(FULL_MASK, dead, 0);
            // the answer to the request is there by now
            if (!__all_sync(FULL_MASK, mbar_wait_ns(next_item, n_answered++ & 1u, PA_WAIT_NS))) break;
            it = taken_over(taken);
            __syncwarp();
            fence_proxy_async_smem();                        // read before the next answer is written
        }
        // no load, and no answer, may still be in flight when the CTA exits
        if (lane == 0) {
            if (n_answered < n_asked) mbar_wait_ns(next_item, n_answered & 1u, PA_WAIT_NS);
            for (int i = 0; i < 2; ++i)
                if (q_n[i] > 0) mbar_wait_ns(&q_full[i], (q_n[i] - 1) & 1u, PA_WAIT_NS);
            for (uint32_t k = pos > NS ? pos - NS : 0; k < pos; ++k)
                mbar_wait_ns(&kv_full[k % NS], (k / NS) & 1u, PA_WAIT_NS);
        }
    } else if (warp == 8) {
        // ---------------- tensor-core products ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t lead = lane == 0;
        {
            constexpr bool BF = T == ATT_BF16;
            constexpr uint32_t ID_S = umma_idesc(BF, false, 128, PA_KEYS), ID_O = umma_idesc(BF, true, 128, D);
            uint32_t pos = 0, q_n[2] = {0, 0}, p_n[2] = {0, 0};
            auto wait_kv = [&](uint32_t k) { return all_wait(&kv_full[k % NS], (k / NS) & 1u, PA_WAIT_NS); };
            auto scores = [&](int i, uint32_t k) {
                const uint32_t qd = umma_desc_k(smem_u32(q_s + i * TILE)), kd = umma_desc_k(smem_u32(kv_s + (k % NS) * TILE));
                tm_fence_after();
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const uint32_t off = ((d / 4) * PANEL + (d % 4) * 32) >> 4;
                    umma_ss(tmem + 128 * i, qd + off, kd + off, ID_S, d != 0, lead);
                }
                umma_done(&s_full[i], lead);
            };
            auto values = [&](int i, uint32_t k, bool first) {
                const uint32_t vd = umma_desc_mn(smem_u32(kv_s + (k % NS) * TILE), PANEL);
                tm_fence_after();
#pragma unroll
                for (int d = 0; d < PA_KEYS / 16; ++d)
                    umma_ts(tmem + O_COL + D * i, tmem + 128 * i + 8 * d, vd + 128 * d, ID_O, !first || d != 0, lead);
            };
            bool ok = true;
            for (uint32_t n_item = 0; ok; ++n_item) {
                const uint32_t slot = n_item % PA_ITEMS;
                if (!all_wait(&item_full[slot], (n_item / PA_ITEMS) & 1u, PA_WAIT_NS)) break;
                const int nb[2] = {__shfl_sync(FULL_MASK, items[slot].n0, 0), __shfl_sync(FULL_MASK, items[slot].n1, 0)};
                if (lead) mbar_arrive(&item_empty[slot]);
                if (nb[0] < 0) break;
                const int n = max(nb[0], nb[1]);
                if (n == 0) continue;
                ok = wait_kv(pos);
                for (int i = 0; i < 2 && ok; ++i) {
                    if (nb[i] == 0) continue;
                    ok = all_wait(&q_full[i], q_n[i]++ & 1u, PA_WAIT_NS);
                    if (!ok) break;
                    scores(i, pos);
                    if (nb[i] == 1) umma_done(&q_empty[i], lead);
                }
                if (!ok) break;
                umma_done(&kv_empty[pos % NS], lead);
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t kv = pos + 2 * j + 1;                 // V of block j; K of block j + 1 follows
                    ok = wait_kv(kv);
                    for (int i = 0; i < 2 && ok; ++i) {
                        if (j >= nb[i]) continue;
                        ok = all_wait(&p_ready[i], p_n[i]++ & 1u, PA_WAIT_NS);
                        if (!ok) break;
                        values(i, kv, j == 0);
                        if (j + 1 == nb[i]) umma_done(&o_full[i], lead);
                        if (j + 1 < nb[i]) {
                            ok = wait_kv(kv + 1);
                            if (!ok) break;
                            scores(i, kv + 1);
                            if (j + 2 == nb[i]) umma_done(&q_empty[i], lead);
                        }
                    }
                    if (!ok) break;
                    umma_done(&kv_empty[kv % NS], lead);
                    if (j + 1 < n) umma_done(&kv_empty[(kv + 1) % NS], lead);
                }
                pos += 2 * n;
            }
            // every product has completed before TMEM is released
            umma_done(drain, lead);
            all_wait(drain, 0u, PA_WAIT_NS);
        }
    } else if (warp < 8) {
        // ---------------- softmax and epilogue ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int i = warp >> 2;                             // tile
        const int r = (warp & 3) * 32 + lane;                // row
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_t = tmem + lanes + 128 * i, o_t = tmem + lanes + O_COL + D * i;
        const int rt = r / a.G, g = r - rt * a.G;
        const float c = fmaxf(fabsf(a.scale) * ATT_LOG2E, 1.17549435e-38f);          // not 0: -inf stays -inf
        const uint32_t flip = a.scale < 0.0f ? 0x80000000u : 0u;
        constexpr float SHIFT = T == ATT_F16 ? ATT_F16_SHIFT : 0.0f;
        uint32_t pos = 0, s_n = 0, o_n = 0;
        bool ok = true;
        for (uint32_t n_item = 0; ok; ++n_item) {
            const uint32_t slot = n_item % PA_ITEMS;
            if (!__all_sync(FULL_MASK, mbar_wait_ns(&item_full[slot], (n_item / PA_ITEMS) & 1u, PA_WAIT_NS))) break;
            PromptItem w;
            w.n0 = items[slot].n0;
            w.n1 = items[slot].n1;
            w.tok0 = items[slot].tok0;
            w.ntok = items[slot].ntok;
            w.lim0 = items[slot].lim0;
            w.lk = items[slot].lk;
            w.k0 = items[slot].k0;
            w.kh = items[slot].kh;
            if (w.n0 < 0) break;
            const int nb = i ? w.n1 : w.n0;
            const int dt = rt + i * TOK;                     // token within the item
            const bool live = rt < TOK && dt < w.ntok;
            const int lim = a.causal ? min(w.lim0 + dt, w.lk) : w.lk;                // keys this row sees
            const int low = a.causal ? max(w.lim0 + i * TOK, 0) : w.lk;              // keys all rows of the tile see
            float m = -INFINITY, l = 0.0f;                   // reference (in units of S) and sum
            for (int j = 0; j < nb; ++j) {
                ok = __all_sync(FULL_MASK, mbar_wait_ns(&s_full[i], s_n++ & 1u, PA_WAIT_NS));
                if (!ok) break;
                tm_fence_after();
                const int key0 = j * PA_KEYS;
                if (key0 + PA_KEYS > low || flip) {
                    // the less common cases are put right in TMEM, to keep the common code short:
                    // keys that the row does not see, a negative scale
                    const int see = lim - key0;
#pragma unroll 1
                    for (int k0 = 0; k0 < PA_KEYS; k0 += 32) {
                        const uint32_t have = see - k0 >= 32 ? 0xFFFFFFFFu : see > k0 ? (1u << (see - k0)) - 1u : 0u;
                        uint32_t x[32];
                        tm_ld32(s_t + k0, x);
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = (have >> k) & 1u ? x[k] ^ flip : 0xFF800000u;
                        tm_st32(s_t + k0, x);
                    }
                    tm_wait_st();
                }
                uint32_t s[128];
                tm_ld128(s_t, s);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 128; k += 8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mx[q] = max3(mx[q], __uint_as_float(s[k + 2 * q]), __uint_as_float(s[k + 2 * q + 1]));
                }
                const float bm = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
                // the row's own reference moves only when its maximum has outgrown it
                // (or is NaN, which then stays)
                const bool grow = live && !(__fmul_rn(__fsub_rn(bm, m), c) <= PA_SLACK) && bm != -INFINITY;
                if (j == 0) {
                    m = bm;
                } else if (__any_sync(FULL_MASK, grow)) {
                    // the P V products of the earlier blocks are complete: S of
                    // this block came after them
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
                const float ms = m == -INFINITY ? 0.0f : __fmaf_rn(m, c, -SHIFT);
                const uint64_t c2 = f32x2(c, c), ms2 = f32x2(-ms, -ms);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint64_t xx = fma2(f32x2(__uint_as_float(s[32 * h + 2 * k]), __uint_as_float(s[32 * h + 2 * k + 1])), c2, ms2);
                        float lo, hi;
                        f32x2_split(xx, lo, hi);
                        lo = ex2(lo);
                        hi = ex2(hi);
                        sum[k & 1] = add2(sum[k & 1], f32x2(lo, hi));
                        p[k] = pack2<T>(lo, hi);
                    }
                    tm_st16(s_t + 16 * h, p);
                }
                float s0, s1, s2, s3;
                f32x2_split(sum[0], s0, s1);
                f32x2_split(sum[1], s2, s3);
                l = __fadd_rn(l, __fadd_rn(__fadd_rn(s0, s1), __fadd_rn(s2, s3)));
                // V rows that not every row of the tiles sees (tile 0 covers tile 1, which sees more)
                if (key0 + PA_KEYS > low && (i == 0 || j >= w.n0)) {
                    const uint32_t vp = pos + 2 * j + 1;
                    ok = __all_sync(FULL_MASK, mbar_wait_ns(&kv_full[vp % NS], (vp / NS) & 1u, PA_WAIT_NS));
                    if (!ok) break;
                    uint8_t* vs = kv_s + (vp % NS) * TILE;
                    const int r0 = max(low - key0, 0), end = w.lk - key0;
                    uint32_t bad = 0;
#pragma unroll 2
                    for (int k = r0 * 8 + r; k < PA_KEYS * 8; k += 128) {
#pragma unroll
                        for (int p = 0; p < PANELS; ++p) {
                            uint4* e = reinterpret_cast<uint4*>(vs + p * PANEL + k * 16);
                            if ((k >> 3) >= end) *e = make_uint4(0u, 0u, 0u, 0u);
                            else bad |= any_not_finite<T>(*e);
                        }
                    }
                    if (bad) {
                        // take them out (this thread's pieces of V)
                        items[slot].dirty = 1;
#pragma unroll 1
                        for (int k = r0 * 8 + r; k < PA_KEYS * 8; k += 128) {
#pragma unroll 1
                            for (int q = 0; q < 4 * PANELS; ++q) {
                                uint32_t* e = reinterpret_cast<uint32_t*>(vs + (q >> 2) * PANEL + k * 16) + (q & 3);
                                *e &= ~not_finite2<T>(*e);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                tm_wait_st();
                tm_fence_before();
                mbar_arrive(&p_ready[i]);
            }
            if (!ok) break;
            bool dirty = false;
            if (nb > 0) {
                ok = __all_sync(FULL_MASK, mbar_wait_ns(&o_full[i], o_n++ & 1u, PA_WAIT_NS));
                if (!ok) break;
                tm_fence_after();
                dirty = items[slot].dirty != 0;
            }
            const int64_t tok = (int64_t)w.tok0 + dt;
            const int h = w.kh * a.G + g;
            const float inv = lim > 0 ? __frcp_rn(l) : 0.0f;
            uint8_t* out = a.out.base + (tok * a.out.tok + h * a.out.head) * 2;
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
                uint32_t o[32];
                if (nb > 0) tm_ld32(o_t + k, o);
                float v[32];
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = lim > 0 ? __fmul_rn(__uint_as_float(o[q]), inv) : 0.0f;
                uint32_t x[16];
#pragma unroll
                for (int z = 0; z < 16; ++z) x[z] = pack2<T>(v[2 * z], v[2 * z + 1]);
                if (live) {
                    if (a.out32) {
                        store32(out + 2 * k, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
                        store32(out + 2 * k + 32, x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            reinterpret_cast<uint4*>(out + 2 * k)[q] = make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                    }
                }
            }
            if (dirty && live) {
                // give back to this row what was taken out of V and the row sees
                for (int key = a.causal ? max(w.lim0, 0) : w.lk; key < lim; ++key) {
                    const uint8_t* vr = a.v.base + ((w.k0 + (int64_t)key) * a.v.tok + w.kh * a.v.head) * 2;
#pragma unroll 1
                    for (int d = 0; d < D; d += 2) {
                        const uint32_t b = not_finite2<T>(*reinterpret_cast<const uint32_t*>(vr + 2 * d));
                        if (b & 0xFFFFu) att_store<T>(out, d, __fadd_rn(att_load<T>(out, d), att_load<T>(vr, d)));
                        if (b >> 16) att_store<T>(out, d + 1, __fadd_rn(att_load<T>(out, d + 1), att_load<T>(vr, d + 1)));
                    }
                }
            }
            if (a.lse && live)
                a.lse[tok * a.Nq + h] = lim > 0 ? __fmul_rn(__fadd_rn(__fmaf_rn(m, c, -SHIFT), log2f(l)), ATT_LN2) : -INFINITY;
            pos += 2 * max(w.n0, w.n1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }
    tm_fence_before();
    __syncthreads();
    if (warp == 8) {
        tm_fence_after();
        tm_dealloc(tmem, 512);
    }
}

}  // namespace kvq
