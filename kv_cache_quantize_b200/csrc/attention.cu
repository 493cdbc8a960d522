// attention.cu -- host side of the attention calls of include/kvq.h:
// prompt_attention and shared_prefix_attention.
#include "kvq_host.cuh"
#include "attention_common.cuh"
#include "attention_prompt.cuh"
#include "attention_shared.cuh"

namespace kvq {
unsigned int* attention_fault_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_fault_word) == cudaSuccess ? static_cast<unsigned int*>(p) : nullptr;
}
}  // namespace kvq

namespace {

// tokens of one tensor and rows of one launch: 32-bit row numbers with room for a tile
constexpr int64_t ATT_MAX_TOKENS = 0x40000000;
constexpr int64_t ATT_MAX_STRIDE = int64_t(1) << 38;      // elements: a tensor map holds 40-bit byte strides

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// q, k, v or out: [T, heads, D] or [B, S, heads, D], D contiguous, rows that
// flatten to one token stride; 16-byte aligned rows.
kvq_status attn_rows(const kvq_tensor* t, int64_t* tokens, int64_t* heads, int64_t* dim, AttnRows* r) {
    const int n = t->ndim;
    *dim = t->shape[n - 1];
    *heads = t->shape[n - 2];
    *tokens = n == 3 ? t->shape[0] : t->shape[0] * t->shape[1];
    r->base = static_cast<uint8_t*>(t->data);
    r->head = t->stride[n - 2];
    r->tok = t->stride[n - 3];
    if (numel(t) == 0) return KVQ_OK;
    if (*dim > 1 && t->stride[n - 1] != 1) return KVQ_ERR_LAYOUT;
    if (*heads == 1) r->head = *dim;
    if (n == 4) {
        if (t->shape[1] == 1) r->tok = t->stride[0];
        else if (t->shape[0] > 1 && t->stride[0] != t->shape[1] * t->stride[1]) return KVQ_ERR_LAYOUT;
    }
    if (*tokens == 1) r->tok = *heads * *dim;
    if (r->head % 8 != 0 || r->tok % 8 != 0) return KVQ_ERR_LAYOUT;
    if (r->head < *dim || r->tok < *dim || r->head >= ATT_MAX_STRIDE || r->tok >= ATT_MAX_STRIDE) return KVQ_ERR_LAYOUT;
    return KVQ_OK;
}

// an output's rows must not overlap: either dimension may be the outer one
bool disjoint_rows(const AttnRows& r, int64_t tokens, int64_t heads, int64_t dim) {
    if (heads == 1) return tokens == 1 || r.tok >= dim;
    if (tokens == 1) return r.head >= dim;
    return (r.head >= dim && r.tok >= (heads - 1) * r.head + dim) ||
           (r.tok >= dim && r.head >= (tokens - 1) * r.tok + dim);
}

int att_type(int32_t dt) { return dt == KVQ_BF16 ? ATT_BF16 : (dt == KVQ_F16 ? ATT_F16 : (dt == KVQ_I8 ? ATT_I8 : -1)); }

// [tokens, heads, D] rows of a 16-bit type in boxes of box_tok x box_heads x 64
// values with the 128-byte swizzle; tokens past the end read as zero.
bool rows_map(CUtensorMap* m, int type, const AttnRows& r, int64_t tokens, int64_t heads, int64_t D, int box_heads,
              int box_tok) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)(r.head * 2), (cuuint64_t)(r.tok * 2)};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tok};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, type == ATT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, r.base, dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// at least the number of work items: pairs of tiles of each sequence and key head
int64_t prompt_items(const PromptArgs& a) { return (a.T / (2 * (128 / a.G)) + a.B) * a.Nkv; }

template <int T, int D>
kvq_status run_prompt(const PromptArgs& a, cudaStream_t s) {
    const int tok = 128 / a.G;
    CUtensorMap mq, mk, mv;
    // without keys nothing is loaded; the maps still need memory to point at
    const AttnRows& k = a.Tk > 0 ? a.k : a.q;
    const AttnRows& v = a.Tk > 0 ? a.v : a.q;
    const int64_t tk = a.Tk > 0 ? a.Tk : a.T, nkv = a.Tk > 0 ? a.Nkv : a.Nq;
    if (!rows_map(&mq, T, a.q, a.T, a.Nq, D, a.G, tok) || !rows_map(&mk, T, k, tk, nkv, D, 1, PA_KEYS) ||
        !rows_map(&mv, T, v, tk, nkv, D, 1, PA_KEYS))
        return KVQ_ERR_CUDA;
    auto kernel = prompt_kernel<T, D>;
    constexpr uint32_t smem = pa_smem_bytes(D);
    resident_blocks(reinterpret_cast<const void*>(kernel), PA_THREADS, smem);    // raises the shared-memory limit once
    return launched(launch(kernel, (unsigned)prompt_items(a), PA_THREADS, smem, s, mq, mk, mv, a));
}

// the own steps of a batch are counted in 32 bits
bool too_many_own_steps(int64_t batch, int64_t max_own) {
    return batch * ((max_own + SA_KEYS - 1) / SA_KEYS) > INT32_MAX;
}

// How the work is laid out, and the workspace in bytes.  The size is that of
// two-tile groups in either form (a one-tile group needs half the rows, twice
// the groups), for as many CTAs as the kernel ever has, and for requests of up
// to max_own own tokens: a list of one step only ever uses the first tile.
int64_t shared_plan(int64_t B, int64_t Nq, int64_t Nkv, int64_t D, int64_t prefix_len, int64_t max_own, bool hilo,
                    SharedPlan* p) {
    const int64_t G = Nq / Nkv, tok = 128 / G;
    auto area = [&](int64_t group, int64_t* slots, int64_t* rows) {
        *slots = prefix_len > 0 ? ((B + group - 1) / group) * Nkv + SA_MAX_CTAS : 0;
        // several groups: whole tiles; one group: its rows, four times where they are few
        *rows = B > tok ? 128 : B * G <= 32 ? 4 * B * G : B * G;
        return *slots * 2 * *rows;
    };
    int64_t slots, rows;
    const int64_t group = hilo ? tok : 2 * tok;
    const int64_t pre = area(tok, &slots, &rows);                   // rows of the prefix slots, the larger form
    area(group, &slots, &rows);
    p->own_rows = (int32_t)(G <= 32 ? 4 * G : G);
    p->own_slot = max_own == 0 ? 0 : max_own <= SA_KEYS ? p->own_rows : 2 * p->own_rows;
    const int64_t own = (B * Nkv + SA_MAX_CTAS) * p->own_slot;
    p->group = (int32_t)group;
    p->n_groups = (int32_t)((B + group - 1) / group);
    p->blocks = (int32_t)((prefix_len + SA_KEYS - 1) / SA_KEYS);
    p->last_alt = hilo || B - (p->n_groups - 1) * group <= tok;
    p->tile_rows = (int32_t)rows;
    p->own_area = pre * D;
    p->stats_area = (pre + own) * D;
    p->own_stats = p->stats_area + 2 * pre;
    p->before = p->own_stats + 2 * own;
    p->hilo = hilo;
    return (p->before + B + 1) * 4;
}

// A cache [pages, block, Nkv, D] in boxes of up to 128 tokens of one page and
// head: int8 rows as they are, 16-bit ones 64 values at a time with the 128-byte
// swizzle.
bool pages_map(CUtensorMap* m, int type, const void* base, const SharedArgs& a) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const bool i8 = type == ATT_I8;
    const int64_t eb = i8 ? 1 : 2, row = (int64_t)a.Nkv * a.D * eb;
    const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.Nkv, (cuuint64_t)a.block, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)(a.D * eb), (cuuint64_t)row,
                                   (cuuint64_t)(a.num_pages > 1 ? a.page_bytes : row * a.block)};
    const cuuint32_t box[4] = {(cuuint32_t)(i8 ? a.D : 64), 1, (cuuint32_t)(a.block < SA_KEYS ? a.block : SA_KEYS), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                     : type == ATT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               i8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int T, int C, int D>
kvq_status run_shared(const SharedArgs& a, cudaStream_t s) {
    constexpr bool I8 = C == ATT_I8;
    SharedPlan p;
    shared_plan(a.B, a.Nq, a.Nkv, D, a.prefix_len, (int64_t)a.cols * a.block, I8 && T == ATT_F16, &p);
    p.cost_own = I8 ? SA_COST_OWN8 : SA_COST_OWN16;
    CUtensorMap mq = {}, mq1 = {};
    if (!I8 && (!rows_map(&mq, T, a.q, a.B, a.Nq, D, a.G, 128 / a.G) || !rows_map(&mq1, T, a.q, a.B, a.Nq, D, a.G, a.G <= 32 ? 32 / a.G : 1)))
        return KVQ_ERR_CUDA;
    // at most one CTA per step that the lengths can ask for
    const int64_t steps = (int64_t)p.n_groups * a.Nkv * p.blocks +
                          (int64_t)a.B * a.Nkv * (((int64_t)a.cols * a.block + SA_KEYS - 1) / SA_KEYS);
    // TMA where a page holds 8, 16, 32 .. tokens: a swizzle repeats after 8 rows
    const bool tma = a.block_shift >= 3 && a.num_pages > 0;
    CUtensorMap mk = {}, mv = {};
    if (tma && (!pages_map(&mk, C, a.k_cache, a) || !pages_map(&mv, C, a.v_cache, a))) return KVQ_ERR_CUDA;
    auto kernel = tma ? shared_kernel<T, C, D, true> : shared_kernel<T, C, D, false>;
    constexpr uint32_t smem = sa_smem_bytes(D, I8);
    const int64_t ctas = persistent_grid(kernel, SA_THREADS, steps < SA_MAX_CTAS ? steps : SA_MAX_CTAS, smem);
    const int parts = steps > 0 ? (int)ctas : 0;
    if (steps > 0 && launch(kernel, (unsigned)ctas, SA_THREADS, smem, s, mq, mq1, mk, mv, a, p) != cudaSuccess) return KVQ_ERR_CUDA;
    const int hblocks = (a.Nq + SJ_THREADS / 32 - 1) / (SJ_THREADS / 32);
    return launched(launch(shared_join_kernel<T, C, D>, (unsigned)(a.B * hblocks), SJ_THREADS, 0, s, a, p, parts,
                           hblocks));
}

}  // namespace

extern "C" {

kvq_status kvq_prompt_attention(const kvq_tensor* q, const kvq_tensor* k, const kvq_tensor* v,
                                const kvq_tensor* cu_seqlens_q, const kvq_tensor* cu_seqlens_k, kvq_tensor* out,
                                kvq_tensor* lse, int32_t causal, float softmax_scale, kvq_stream stream) {
    Trace trace("kvq_prompt_attention");
    if (!q || !k || !v || !out) return KVQ_ERR_NULL;
    if (!valid_desc(q) || !valid_desc(k) || !valid_desc(v) || !valid_desc(out)) return KVQ_ERR_DTYPE;
    const int type = att_type(q->dtype);
    if (type != ATT_BF16 && type != ATT_F16) return KVQ_ERR_DTYPE;
    if (k->dtype != q->dtype || v->dtype != q->dtype || out->dtype != q->dtype) return KVQ_ERR_DTYPE;
    const int nd = cu_seqlens_q ? 3 : 4;
    if (q->ndim != nd || k->ndim != nd || v->ndim != nd || out->ndim != nd) return KVQ_ERR_NDIM;
    if (!cu_seqlens_q && cu_seqlens_k) return KVQ_ERR_NULL;
    if (!std::isfinite(softmax_scale)) return KVQ_ERR_ATTR;
    PromptArgs a = {};
    int64_t D, Nkv, Nq, n, h, d;
    kvq_status st;
    if ((st = attn_rows(q, &a.T, &Nq, &D, &a.q)) != KVQ_OK) return st;
    if ((st = attn_rows(k, &a.Tk, &Nkv, &d, &a.k)) != KVQ_OK) return st;
    if (d != D) return KVQ_ERR_SHAPE;
    if ((st = attn_rows(v, &n, &h, &d, &a.v)) != KVQ_OK) return st;
    if (n != a.Tk || h != Nkv || d != D) return KVQ_ERR_SHAPE;
    if ((st = attn_rows(out, &n, &h, &d, &a.out)) != KVQ_OK) return st;
    if (n != a.T || h != Nq || d != D) return KVQ_ERR_SHAPE;
    if (D != 64 && D != 128) return KVQ_ERR_UNSUPPORTED;
    if (Nkv < 1 || Nq < 1 || Nq % Nkv != 0) return KVQ_ERR_SHAPE;
    if (Nq / Nkv > 128) return KVQ_ERR_UNSUPPORTED;
    if (a.T > ATT_MAX_TOKENS || a.Tk > ATT_MAX_TOKENS || Nq > ATT_MAX_TOKENS) return KVQ_ERR_SHAPE;
    if (nd == 4) {
        if (k->shape[0] != q->shape[0] || v->shape[0] != q->shape[0] || v->shape[1] != k->shape[1] ||
            out->shape[0] != q->shape[0])
            return KVQ_ERR_SHAPE;
        a.B = (int32_t)q->shape[0];
        a.S = (int32_t)q->shape[1];
        a.Sk = (int32_t)k->shape[1];
    } else {
        const kvq_tensor* cu[2] = {cu_seqlens_q, cu_seqlens_k ? cu_seqlens_k : cu_seqlens_q};
        for (const kvq_tensor* c : cu) {
            if (!valid_desc(c) || c->dtype != KVQ_I32) return KVQ_ERR_DTYPE;
            if (c->ndim != 1) return KVQ_ERR_NDIM;
            if (c->shape[0] < 1 || c->shape[0] != cu_seqlens_q->shape[0] || c->shape[0] > ATT_MAX_TOKENS)
                return KVQ_ERR_SHAPE;
            if (!contiguous(c)) return KVQ_ERR_LAYOUT;
        }
        a.B = (int32_t)(cu_seqlens_q->shape[0] - 1);
        a.cu_q = static_cast<const int32_t*>(cu[0]->data);
        a.cu_k = static_cast<const int32_t*>(cu[1]->data);
    }
    if (!disjoint_rows(a.out, a.T, Nq, D)) return KVQ_ERR_LAYOUT;
    if (lse) {
        if (!valid_desc(lse) || lse->dtype != KVQ_F32) return KVQ_ERR_DTYPE;
        if (lse->ndim != nd - 1) return KVQ_ERR_NDIM;
        for (int i = 0; i + 1 < nd; ++i)
            if (lse->shape[i] != q->shape[i]) return KVQ_ERR_SHAPE;
        if (!contiguous(lse)) return KVQ_ERR_LAYOUT;
        a.lse = static_cast<float*>(lse->data);
    }
    if (a.T == 0 || a.B == 0) return KVQ_OK;
    a.Nq = (int32_t)Nq;
    a.Nkv = (int32_t)Nkv;
    a.G = (int32_t)(Nq / Nkv);
    if (prompt_items(a) > INT32_MAX) return KVQ_ERR_SHAPE;      // a grid's CTAs
    if (!q->data || !out->data || (a.Tk > 0 && (!k->data || !v->data)) || (nd == 3 && (!a.cu_q || !a.cu_k)) ||
        (lse && !a.lse))
        return KVQ_ERR_NULL;
    if (!aligned16(q->data) || !aligned16(k->data) || !aligned16(v->data) || !aligned16(out->data))
        return KVQ_ERR_LAYOUT;
    a.D = (int32_t)D;
    a.causal = causal != 0;
    a.out32 = reinterpret_cast<uintptr_t>(out->data) % 32 == 0 && a.out.tok % 16 == 0 && a.out.head % 16 == 0;
    a.scale = softmax_scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (type == ATT_BF16) return D == 64 ? run_prompt<ATT_BF16, 64>(a, s) : run_prompt<ATT_BF16, 128>(a, s);
    return D == 64 ? run_prompt<ATT_F16, 64>(a, s) : run_prompt<ATT_F16, 128>(a, s);
}

int64_t kvq_shared_prefix_attention_workspace(int64_t batch, int64_t n_q, int64_t n_kv, int64_t dim,
                                              int64_t prefix_len, int64_t max_own) {
    if (batch < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || n_q / n_kv > 128 || (dim != 64 && dim != 128) ||
        prefix_len < 0 || max_own < 0 || batch > ATT_MAX_TOKENS / n_q || max_own > ATT_MAX_TOKENS ||
        prefix_len > ATT_MAX_TOKENS || max_own + prefix_len > ATT_MAX_TOKENS || too_many_own_steps(batch, max_own))
        return -1;
    SharedPlan p;
    return shared_plan(batch, n_q, n_kv, dim, prefix_len, max_own, false, &p);
}

kvq_status kvq_shared_prefix_attention(const kvq_tensor* q, const kvq_tensor* k_cache, const kvq_tensor* v_cache,
                                       const kvq_tensor* block_table, const kvq_tensor* seq_lens,
                                       const kvq_tensor* prefix_table, int64_t prefix_len, const kvq_tensor* scale_k,
                                       const kvq_tensor* scale_v, const kvq_tensor* offset_k,
                                       const kvq_tensor* offset_v, kvq_tensor* out, kvq_tensor* lse,
                                       float softmax_scale, kvq_tensor* workspace, kvq_stream stream) {
    Trace trace("kvq_shared_prefix_attention");
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out) return KVQ_ERR_NULL;
    if (!valid_desc(q) || !valid_desc(k_cache) || !valid_desc(v_cache) || !valid_desc(out)) return KVQ_ERR_DTYPE;
    const int type = att_type(q->dtype);
    if (type != ATT_BF16 && type != ATT_F16) return KVQ_ERR_DTYPE;
    if (out->dtype != q->dtype || k_cache->dtype != v_cache->dtype) return KVQ_ERR_DTYPE;
    const int ctype = att_type(k_cache->dtype);
    if (ctype != ATT_I8 && ctype != type) return KVQ_ERR_DTYPE;
    if (q->ndim != 3 || out->ndim != 3 || k_cache->ndim != 4 || v_cache->ndim != 4) return KVQ_ERR_NDIM;
    if (!std::isfinite(softmax_scale)) return KVQ_ERR_ATTR;
    SharedArgs a = {};
    int64_t B, Nq, D, n, h, d;
    kvq_status st;
    if ((st = attn_rows(q, &B, &Nq, &D, &a.q)) != KVQ_OK) return st;
    if ((st = attn_rows(out, &n, &h, &d, &a.out)) != KVQ_OK) return st;
    if (n != B || h != Nq || d != D) return KVQ_ERR_SHAPE;
    if (D != 64 && D != 128) return KVQ_ERR_UNSUPPORTED;
    const int64_t Nkv = k_cache->shape[2], pages = k_cache->shape[0], block = k_cache->shape[1];
    if (k_cache->shape[3] != D || Nkv < 1 || Nq < 1 || Nq % Nkv != 0 || block < 1) return KVQ_ERR_SHAPE;
    if (Nq / Nkv > 128) return KVQ_ERR_UNSUPPORTED;
    for (int i = 0; i < 4; ++i)
        if (v_cache->shape[i] != k_cache->shape[i]) return KVQ_ERR_SHAPE;
    if (B > ATT_MAX_TOKENS / Nq || pages > INT32_MAX || block > ATT_MAX_TOKENS) return KVQ_ERR_SHAPE;
    const int64_t eb = elem_bytes(k_cache->dtype);
    for (const kvq_tensor* c : {k_cache, v_cache}) {
        if (numel(c) == 0) continue;
        if (c->stride[3] != 1 || (Nkv > 1 && c->stride[2] != D) || (block > 1 && c->stride[1] != Nkv * D) ||
            (pages > 1 && (c->stride[0] < block * Nkv * D || c->stride[0] * eb % 64 != 0 ||
                           c->stride[0] != k_cache->stride[0])))
            return KVQ_ERR_LAYOUT;
    }
    if (pages > 0 && pages * (pages > 1 ? k_cache->stride[0] : block * Nkv * D) * eb / 64 >= 0xFFFFFFFFll)
        return KVQ_ERR_SHAPE;                                    // 256 GB: places are 32-bit units of 64 bytes
    const bool i8 = ctype == ATT_I8;
    const kvq_tensor* par[4] = {scale_k, scale_v, offset_k, offset_v};
    const float* pp[4] = {nullptr, nullptr, nullptr, nullptr};
    for (int i = 0; i < 4; ++i) {
        if (!par[i]) {
            if (i8 && i < 2) return KVQ_ERR_NULL;
            continue;
        }
        if (!i8) return KVQ_ERR_ATTR;
        if (!valid_desc(par[i]) || par[i]->dtype != KVQ_F32) return KVQ_ERR_DTYPE;
        if (numel(par[i]) != Nkv * D) return KVQ_ERR_SHAPE;
        if (!contiguous(par[i])) return KVQ_ERR_LAYOUT;
        pp[i] = static_cast<const float*>(par[i]->data);
    }
    if (!valid_desc(block_table) || block_table->dtype != KVQ_I32) return KVQ_ERR_DTYPE;
    if (block_table->ndim != 2) return KVQ_ERR_NDIM;
    if (block_table->shape[0] != B) return KVQ_ERR_SHAPE;
    const int64_t cols = block_table->shape[1];
    if (cols > 1 && block_table->stride[1] != 1) return KVQ_ERR_LAYOUT;
    if (!valid_desc(seq_lens) || seq_lens->dtype != KVQ_I32) return KVQ_ERR_DTYPE;
    if (seq_lens->ndim != 1) return KVQ_ERR_NDIM;
    if (seq_lens->shape[0] != B) return KVQ_ERR_SHAPE;
    if (!contiguous(seq_lens)) return KVQ_ERR_LAYOUT;
    if (prefix_len < 0) return KVQ_ERR_ATTR;
    if (prefix_len > ATT_MAX_TOKENS) return KVQ_ERR_SHAPE;
    if (prefix_len > 0) {
        if (!prefix_table) return KVQ_ERR_NULL;
        if (!valid_desc(prefix_table) || prefix_table->dtype != KVQ_I32) return KVQ_ERR_DTYPE;
        if (prefix_table->ndim != 1) return KVQ_ERR_NDIM;
        if ((prefix_len + block - 1) / block > prefix_table->shape[0]) return KVQ_ERR_SHAPE;
        if (!contiguous(prefix_table)) return KVQ_ERR_LAYOUT;
        a.prefix_table = static_cast<const int32_t*>(prefix_table->data);
    }
    if (cols > ATT_MAX_TOKENS / block || cols * block + prefix_len > ATT_MAX_TOKENS ||
        too_many_own_steps(B, cols * block))
        return KVQ_ERR_SHAPE;
    if (!disjoint_rows(a.out, B, Nq, D)) return KVQ_ERR_LAYOUT;
    if (lse) {
        if (!valid_desc(lse) || lse->dtype != KVQ_F32) return KVQ_ERR_DTYPE;
        if (lse->ndim != 2) return KVQ_ERR_NDIM;
        if (lse->shape[0] != B || lse->shape[1] != Nq) return KVQ_ERR_SHAPE;
        if (!contiguous(lse)) return KVQ_ERR_LAYOUT;
        a.lse = static_cast<float*>(lse->data);
    }
    const int64_t need = kvq_shared_prefix_attention_workspace(B, Nq, Nkv, D, prefix_len, cols * block);
    if (need > 0 && !workspace) return KVQ_ERR_NULL;
    if (workspace) {
        if (!valid_desc(workspace) || workspace->dtype != KVQ_U8) return KVQ_ERR_DTYPE;
        if (!contiguous(workspace)) return KVQ_ERR_LAYOUT;
        if (numel(workspace) < need) return KVQ_ERR_CAPACITY;
        a.workspace = static_cast<uint8_t*>(workspace->data);
    }
    if (B == 0) return KVQ_OK;
    if (!q->data || !out->data || !seq_lens->data || (cols > 0 && !block_table->data) ||
        (prefix_len > 0 && !a.prefix_table) || (pages > 0 && (!k_cache->data || !v_cache->data)) ||
        (lse && !a.lse) || (need > 0 && !a.workspace))
        return KVQ_ERR_NULL;
    for (int i = 0; i < 4; ++i)
        if (par[i] && !pp[i]) return KVQ_ERR_NULL;
    if (!aligned16(q->data) || !aligned16(out->data) || !aligned16(k_cache->data) || !aligned16(v_cache->data) ||
        !aligned16(pp[0]) || !aligned16(a.workspace))
        return KVQ_ERR_LAYOUT;
    a.k_cache = static_cast<const uint8_t*>(k_cache->data);
    a.v_cache = static_cast<const uint8_t*>(v_cache->data);
    a.page_bytes = (pages > 1 ? k_cache->stride[0] : 0) * eb;
    a.num_pages = pages;
    a.block = (int32_t)block;
    a.block_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (block == (int64_t(1) << i)) a.block_shift = i;
    a.table = static_cast<const int32_t*>(block_table->data);
    a.table_stride = B > 1 ? block_table->stride[0] : 0;
    a.cols = (int32_t)cols;
    a.seq_lens = static_cast<const int32_t*>(seq_lens->data);
    a.prefix_len = (int32_t)prefix_len;
    a.scale_k = pp[0];
    a.scale_v = pp[1];
    a.offset_k = pp[2];
    a.offset_v = pp[3];
    a.B = (int32_t)B;
    a.Nq = (int32_t)Nq;
    a.Nkv = (int32_t)Nkv;
    a.G = (int32_t)(Nq / Nkv);
    a.D = (int32_t)D;
    a.scale = softmax_scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define KVQ_SHARED(T, C) (D == 64 ? run_shared<T, C, 64>(a, s) : run_shared<T, C, 128>(a, s))
    if (type == ATT_BF16) return i8 ? KVQ_SHARED(ATT_BF16, ATT_I8) : KVQ_SHARED(ATT_BF16, ATT_BF16);
    return i8 ? KVQ_SHARED(ATT_F16, ATT_I8) : KVQ_SHARED(ATT_F16, ATT_F16);
#undef KVQ_SHARED
}

}  // extern "C"
