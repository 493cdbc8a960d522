// attention_common.cuh -- what the attention kernels share: the arguments of
// the two calls, where a sequence's tokens lie, and small numeric helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "tma_pipe.cuh"

namespace kvq {

constexpr float ATT_LOG2E = 1.4426950408889634f;
constexpr float ATT_LN2 = 0.6931471805599453f;

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
    float scale;                   // softmax scale
};

struct SeqSpan {
    int64_t q0, k0;
    int32_t lq, lk;
};

// Sequence b's rows; an offset outside [0, T] or a negative length sets
// FAULT_SLOT_RANGE (if `report`) and the sequence counts as empty.
__device__ __forceinline__ SeqSpan prompt_span(const PromptArgs& a, int b, bool report) {
    SeqSpan s;
    if (a.cu_q == nullptr) {
        s.q0 = (int64_t)b * a.S;
        s.lq = a.S;
    } else {
        const int32_t lo = __ldg(a.cu_q + b), hi = __ldg(a.cu_q + b + 1);
        const bool ok = lo >= 0 && hi >= lo && hi <= a.T;
        if (!ok && report) raise_fault(FAULT_SLOT_RANGE);
        s.q0 = ok ? lo : 0;
        s.lq = ok ? hi - lo : 0;
    }
    if (a.cu_k == nullptr) {
        s.k0 = (int64_t)b * a.Sk;
        s.lk = a.Sk;
    } else {
        const int32_t lo = __ldg(a.cu_k + b), hi = __ldg(a.cu_k + b + 1);
        const bool ok = lo >= 0 && hi >= lo && hi <= a.Tk;
        if (!ok && report) raise_fault(FAULT_SLOT_RANGE);
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
    int64_t k_page, v_page;        // page strides in bytes
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

// The page that holds token t of a page list, or -1 (FAULT_SLOT_RANGE) when
// the entry is not a page; *in_page receives the token's place in it.
__device__ __forceinline__ int32_t page_of(const SharedArgs& a, const int32_t* list, int32_t t, int32_t* in_page) {
    const int32_t e = a.block_shift >= 0 ? t >> a.block_shift : t / a.block;
    *in_page = t - e * a.block;
    const int32_t p = __ldg(list + e);
    if (p < 0 || p >= a.num_pages) {
        raise_fault(FAULT_SLOT_RANGE);
        return -1;
    }
    return p;
}

// Request b's own length: -1 for a row that takes no part; a length that its
// table row cannot hold sets FAULT_SLOT_RANGE and counts as -1.
__device__ __forceinline__ int32_t own_length(const SharedArgs& a, int b) {
    const int32_t n = __ldg(a.seq_lens + b);
    if (n < -1 || n > (int64_t)a.cols * a.block) {
        raise_fault(FAULT_SLOT_RANGE);
        return -1;
    }
    return n;
}

template <int T>
__device__ __forceinline__ float att_load(const uint8_t* p, int64_t i) {
    if (T == ATT_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    if (T == ATT_F16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    return (float)reinterpret_cast<const int8_t*>(p)[i];
}

template <int T>
__device__ __forceinline__ void att_store(uint8_t* p, int64_t i, float v) {
    if (T == ATT_BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(FULL_MASK, v, d));
    return v;
}

}  // namespace kvq
