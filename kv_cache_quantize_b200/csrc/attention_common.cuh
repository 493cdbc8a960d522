// attention_common.cuh -- what the attention kernels share: the arguments of
// the two calls, where a sequence's tokens lie, and small numeric helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "tma_pipe.cuh"

namespace kvq {

constexpr float ATT_LOG2E = 1.4426950408889634f;
// f16 weights are scaled up by 2^8, so that weights down to 2^-22 of the
// largest stay normal numbers; with a slack of 2^7 they stay below 65504
constexpr float ATT_F16_SHIFT = 8.0f;
constexpr float ATT_LN2 = 0.6931471805599453f;

// What a kernel of this library may have written just before (queries, tables,
// lengths, offsets of sequences, caches) is read by plain loads: the kernels
// start while the one before them may still run (pdl_wait), and the read-only
// path (__ldg) is for data that nobody writes meanwhile, the caches' scales and
// offsets.

// element types of queries, outputs and 16-bit caches; ATT_I8: int8 caches
enum { ATT_BF16 = 0, ATT_F16 = 1, ATT_I8 = 2 };

// strides in elements; the last dimension is contiguous
struct AttnRows {
    uint8_t* base;
    int64_t tok, head;
};

struct PromptArgs {
    AttnRows q, k, v, out;
    float* lse;                    // [T, Nq] or null
    const int32_t* cu_q;           // [B + 1], or null: B sequences of S (Sk) tokens
    const int32_t* cu_k;
    int64_t T, Tk;                 // rows of q and k in all
    int32_t S, Sk;
    int32_t B;
    int32_t Nq, Nkv, G, D;
    int32_t causal;
    int32_t out32;                 // rows of out are 32-byte aligned
    float scale;                   // softmax scale
};

struct SeqSpan {
    int64_t q0, k0;
    int32_t lq, lk;
};

// Sequence b's rows; an offset outside [0, T] or a negative length sets
// FAULT_SLOT_RANGE and the sequence counts as empty.
__device__ __forceinline__ SeqSpan prompt_span(const PromptArgs& a, int b) {
    SeqSpan s;
    if (a.cu_q == nullptr) {
        s.q0 = (int64_t)b * a.S;
        s.lq = a.S;
    } else {
        const int32_t lo = a.cu_q[b], hi = a.cu_q[b + 1];
        const bool ok = lo >= 0 && hi >= lo && hi <= a.T;
        if (!ok) raise_fault(FAULT_SLOT_RANGE);
        s.q0 = ok ? lo : 0;
        s.lq = ok ? hi - lo : 0;
    }
    if (a.cu_k == nullptr) {
        s.k0 = (int64_t)b * a.Sk;
        s.lk = a.Sk;
    } else {
        const int32_t lo = a.cu_k[b], hi = a.cu_k[b + 1];
        const bool ok = lo >= 0 && hi >= lo && hi <= a.Tk;
        if (!ok) raise_fault(FAULT_SLOT_RANGE);
        s.k0 = ok ? lo : 0;
        s.lk = ok ? hi - lo : 0;
        if (!ok) s.lq = 0;
    }
    return s;
}

struct SharedArgs {
    AttnRows q, out;               // [B, Nq, D]
    float* lse;                    // [B, Nq] or null
    const uint8_t* k_cache;        // [pages, block, Nkv, D]
    const uint8_t* v_cache;
    int64_t page_bytes;            // from page to page, a multiple of 64
    int64_t num_pages;
    int32_t block;                 // tokens per page
    int32_t block_shift;           // log2(block) when a power of two, else -1
    const int32_t* table;          // [B, cols]: the requests' own pages
    int64_t table_stride;
    int32_t cols;
    const int32_t* seq_lens;       // [B]: own tokens, -1: the row takes no part
    const int32_t* prefix_table;
    int32_t prefix_len;
    const float *scale_k, *scale_v, *offset_k, *offset_v;   // [Nkv * D], int8 caches only
    int32_t B, Nq, Nkv, G, D;
    float scale;
    uint8_t* workspace;
};

// Request b's own length: -1 for a row that takes no part; a length that its
// table row cannot hold sets FAULT_SLOT_RANGE and counts as -1.
__device__ __forceinline__ int32_t own_length(const SharedArgs& a, int b) {
    const int32_t n = a.seq_lens[b];
    if (n < -1 || n > (int64_t)a.cols * a.block) {
        raise_fault(FAULT_SLOT_RANGE);
        return -1;
    }
    return n;
}

template <int T>
__device__ __forceinline__ float att_load(const uint8_t* p, int64_t i) {
    if (T == ATT_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(reinterpret_cast<const __half*>(p)[i]);
}

template <int T>
__device__ __forceinline__ void att_store(uint8_t* p, int64_t i, float v) {
    if (T == ATT_BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}

// nonzero if one of eight packed 16-bit values is not finite: adding one to an
// exponent of ones carries into the sign bit, and no further
template <int T>
__device__ __forceinline__ uint32_t any_not_finite(uint4 v) {
    constexpr uint32_t E = T == ATT_BF16 ? 0x7F807F80u : 0x7C007C00u, ONE = T == ATT_BF16 ? 0x00800080u : 0x04000400u;
    return (((v.x & E) + ONE) | ((v.y & E) + ONE) | ((v.z & E) + ONE) | ((v.w & E) + ONE)) & 0x80008000u;
}

// all bits of those of two packed 16-bit values that are not finite
template <int T>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
    constexpr uint32_t E = T == ATT_BF16 ? 0x7F807F80u : 0x7C007C00u;
    const uint32_t x = (w & E) ^ E;
    return ((x & 0xFFFFu) == 0u ? 0xFFFFu : 0u) | ((x >> 16) == 0u ? 0xFFFF0000u : 0u);
}

template <int T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (T == ATT_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int T>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
    if (T == ATT_BF16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    }
}

// 32 bytes in one store (32-byte aligned): a lane that writes a row of its own
// takes the store unit a cycle for each store, whatever its width
__device__ __forceinline__ void store32(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d),
                 "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}

// the largest of three; NaN if one is
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

}  // namespace kvq
