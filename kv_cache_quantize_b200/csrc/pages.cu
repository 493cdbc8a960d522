// pages.cu -- host side of the page operations of include/kvq.h: copy_pages,
// free_pages, fork_pages and compact_pages.
#include "kvq_host.cuh"
#include "pages.cuh"

namespace kvq {
unsigned int* pages_fault_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_fault_word) == cudaSuccess ? static_cast<unsigned int*>(p) : nullptr;
}
}  // namespace kvq

namespace {

// The caches of a call: each [num_pages, ...] with the page contiguous and
// only the page dimension strided.
kvq_status page_caches(const kvq_tensor* caches, int32_t n, int64_t* num_pages, PageCopyArgs* a) {
    if (n < 0 || n > PG_MAX_CACHES) return KVQ_ERR_ATTR;
    if (n > 0 && !caches) return KVQ_ERR_NULL;
    a->n_caches = 0;
    for (int i = 0; i < n; ++i) {
        const kvq_tensor* c = caches + i;
        if (!valid_desc(c)) return KVQ_ERR_DTYPE;
        if (c->ndim < 2) return KVQ_ERR_NDIM;
        if (*num_pages < 0) *num_pages = c->shape[0];
        if (c->shape[0] != *num_pages) return KVQ_ERR_SHAPE;
        int64_t elems = 1;
        for (int k = c->ndim - 1; k >= 1; --k) {
            if (c->shape[k] > 1 && c->stride[k] != elems && numel(c) > 0) return KVQ_ERR_LAYOUT;
            elems *= c->shape[k];
            if (elems > INT32_MAX) return KVQ_ERR_SHAPE;
        }
        const int64_t eb = elem_bytes(c->dtype);
        if (elems * eb > INT32_MAX) return KVQ_ERR_SHAPE;
        if (elems == 0 || c->shape[0] == 0) continue;         // nothing to move in this cache
        if (c->shape[0] > 1 && c->stride[0] < elems) return KVQ_ERR_LAYOUT;
        PageCache& pc = a->cache[a->n_caches++];
        pc.base = static_cast<uint8_t*>(c->data);
        pc.bytes = (uint32_t)(elems * eb);
        pc.stride = (c->shape[0] > 1 ? c->stride[0] : elems) * eb;
    }
    return KVQ_OK;
}

kvq_status cache_pointers(const PageCopyArgs& a) {
    for (int i = 0; i < a.n_caches; ++i)
        if (!a.cache[i].base) return KVQ_ERR_NULL;
    return KVQ_OK;
}

// int32 [rows, cols] with the last dimension contiguous and rows apart
kvq_status table_desc(const kvq_tensor* t, int64_t* rows, int64_t* cols, int64_t* stride) {
    if (!valid_desc(t) || t->dtype != KVQ_I32) return KVQ_ERR_DTYPE;
    if (t->ndim != 2) return KVQ_ERR_NDIM;
    *rows = t->shape[0];
    *cols = t->shape[1];
    *stride = *rows > 1 ? t->stride[0] : *cols;
    if (*cols > 1 && t->stride[1] != 1) return KVQ_ERR_LAYOUT;
    if (*rows > 1 && *cols > 0 && *stride < *cols) return KVQ_ERR_LAYOUT;
    return KVQ_OK;
}

kvq_status vector_desc(const kvq_tensor* t, bool any_index, int64_t* n) {
    if (!valid_desc(t) || (any_index ? !is_index_dtype(t->dtype) : t->dtype != KVQ_I32)) return KVQ_ERR_DTYPE;
    if (t->ndim != 1) return KVQ_ERR_NDIM;
    if (!contiguous(t)) return KVQ_ERR_LAYOUT;
    *n = t->shape[0];
    return KVQ_OK;
}

template <int MODE>
kvq_status run_copy(PageCopyArgs& a, cudaStream_t s) {
    a.chunk = 8192;
    uint64_t align = 0;
    a.units = 0;
    for (int i = 0; i < a.n_caches; ++i) {
        PageCache& c = a.cache[i];
        align |= reinterpret_cast<uintptr_t>(c.base) | (uint64_t)c.stride | c.bytes;
        c.unit0 = a.units;
        a.units += (c.bytes + a.chunk - 1) / a.chunk;
    }
    if (a.units == 0) a.units = 1, a.n_caches = 0;
    const int64_t need = a.n_pairs * a.units;                   // units; a CTA takes every grid-th one
    auto go = [&](auto kernel) {
        return launched(launch(kernel, (unsigned)persistent_grid(kernel, PG_THREADS, need), PG_THREADS, 0, s, a));
    };
    if (align % 16 == 0) return go(page_copy_words_kernel<MODE, uint4>);
    if (align % 4 == 0) return go(page_copy_words_kernel<MODE, uint32_t>);
    return go(page_copy_words_kernel<MODE, uint8_t>);
}

}  // namespace

extern "C" {

kvq_status kvq_copy_pages(const kvq_tensor* caches, int32_t n_caches, const kvq_tensor* src, const kvq_tensor* dst,
                          kvq_stream stream) {
    Trace trace("kvq_copy_pages");
    if (!src || !dst) return KVQ_ERR_NULL;
    PageCopyArgs a = {};
    int64_t pages = -1, n, m;
    if (n_caches < 1) return KVQ_ERR_ATTR;
    kvq_status st = page_caches(caches, n_caches, &pages, &a);
    if (st != KVQ_OK) return st;
    if ((st = vector_desc(src, true, &n)) != KVQ_OK) return st;
    if ((st = vector_desc(dst, true, &m)) != KVQ_OK) return st;
    if (n != m || n > INT32_MAX) return KVQ_ERR_SHAPE;
    if (n == 0 || a.n_caches == 0) return KVQ_OK;
    if (!src->data || !dst->data) return KVQ_ERR_NULL;
    if ((st = cache_pointers(a)) != KVQ_OK) return st;
    a.n_pairs = n;
    a.num_pages = pages;
    a.src = src->data;
    a.dst = dst->data;
    a.src_i64 = src->dtype == KVQ_I64;
    a.dst_i64 = dst->dtype == KVQ_I64;
    return run_copy<PG_LIST>(a, reinterpret_cast<cudaStream_t>(stream));
}

kvq_status kvq_free_pages(kvq_tensor* block_table, kvq_tensor* seq_lens, kvq_tensor* ref_count,
                          const kvq_tensor* rows, int64_t block_size, kvq_stream stream) {
    Trace trace("kvq_free_pages");
    if (!block_table || !seq_lens || !ref_count || !rows) return KVQ_ERR_NULL;
    FreeArgs a = {};
    int64_t n;
    kvq_status st = table_desc(block_table, &a.table_rows, &a.table_cols, &a.table_stride);
    if (st != KVQ_OK) return st;
    if ((st = vector_desc(seq_lens, false, &n)) != KVQ_OK) return st;
    if (n != a.table_rows) return KVQ_ERR_SHAPE;
    if ((st = vector_desc(ref_count, false, &a.num_pages)) != KVQ_OK) return st;
    if ((st = vector_desc(rows, true, &a.n_rows)) != KVQ_OK) return st;
    if (block_size < 1 || block_size > INT32_MAX) return KVQ_ERR_ATTR;
    if (a.n_rows > INT32_MAX || a.num_pages > INT32_MAX - 8 * PL_THREADS) return KVQ_ERR_SHAPE;
    if (a.n_rows == 0 || a.table_rows == 0 || a.table_cols == 0) return KVQ_OK;
    if (!block_table->data || !seq_lens->data || !rows->data || (a.num_pages > 0 && !ref_count->data))
        return KVQ_ERR_NULL;
    a.table = static_cast<int32_t*>(block_table->data);
    a.seq_lens = static_cast<int32_t*>(seq_lens->data);
    a.ref_count = static_cast<int32_t*>(ref_count->data);
    a.rows = rows->data;
    a.rows_i64 = rows->dtype == KVQ_I64;
    a.block_size = block_size;
    return launched(launch(free_pages_kernel, (unsigned)persistent_grid(free_pages_kernel, 128, (a.n_rows + 3) / 4),
                           128, 0, reinterpret_cast<cudaStream_t>(stream), a));
}

kvq_status kvq_fork_pages(const kvq_tensor* caches, int32_t n_caches, kvq_tensor* block_table, kvq_tensor* seq_lens,
                          kvq_tensor* ref_count, const kvq_tensor* parents, const kvq_tensor* children,
                          int64_t block_size, kvq_tensor* fresh, kvq_stream stream) {
    Trace trace("kvq_fork_pages");
    if (!block_table || !seq_lens || !ref_count || !parents || !children || !fresh) return KVQ_ERR_NULL;
    PageCopyArgs a = {};
    ForkArgs f = {};
    int64_t n, pages, m;
    kvq_status st = table_desc(block_table, &a.table_rows, &a.table_cols, &a.table_stride);
    if (st != KVQ_OK) return st;
    if ((st = vector_desc(seq_lens, false, &n)) != KVQ_OK) return st;
    if (n != a.table_rows) return KVQ_ERR_SHAPE;
    if ((st = vector_desc(ref_count, false, &pages)) != KVQ_OK) return st;
    if ((st = page_caches(caches, n_caches, &pages, &a)) != KVQ_OK) return st;
    if ((st = vector_desc(parents, true, &n)) != KVQ_OK) return st;
    if ((st = vector_desc(children, true, &m)) != KVQ_OK) return st;
    if (n != m) return KVQ_ERR_SHAPE;
    if ((st = vector_desc(fresh, false, &m)) != KVQ_OK) return st;
    if (n != m || n > INT32_MAX - PL_THREADS || pages > INT32_MAX - 8 * PL_THREADS) return KVQ_ERR_SHAPE;
    if (block_size < 1 || block_size > INT32_MAX) return KVQ_ERR_ATTR;
    if (n == 0) return KVQ_OK;
    if (a.table_rows == 0 || a.table_cols == 0) return KVQ_ERR_SHAPE;
    if (!block_table->data || !seq_lens->data || !parents->data || !children->data || !fresh->data ||
        (pages > 0 && !ref_count->data))
        return KVQ_ERR_NULL;
    if ((st = cache_pointers(a)) != KVQ_OK) return st;
    f.ref_count = static_cast<const int32_t*>(ref_count->data);
    f.num_pages = pages;
    f.seq_lens = static_cast<int32_t*>(seq_lens->data);
    f.table_rows = a.table_rows;
    f.table_cols = a.table_cols;
    f.block_size = block_size;
    f.parents = parents->data;
    f.children = children->data;
    f.parents_i64 = parents->dtype == KVQ_I64;
    f.children_i64 = children->dtype == KVQ_I64;
    f.n = (int32_t)n;
    f.fresh = static_cast<int32_t*>(fresh->data);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch(fork_plan_kernel, 1, PL_THREADS, 0, s, f) != cudaSuccess) return KVQ_ERR_CUDA;
    a.n_pairs = n;
    a.num_pages = pages;
    a.src = parents->data;
    a.dst = children->data;
    a.src_i64 = f.parents_i64;
    a.dst_i64 = f.children_i64;
    a.pair_page = f.fresh;
    a.table = static_cast<int32_t*>(block_table->data);
    a.seq_lens = f.seq_lens;
    a.ref_count = static_cast<int32_t*>(ref_count->data);
    a.block_size = block_size;
    return run_copy<PG_FORK>(a, s);
}

kvq_status kvq_compact_pages(const kvq_tensor* caches, int32_t n_caches, const kvq_tensor* block_table,
                             const kvq_tensor* ref_count, kvq_tensor* new_table, kvq_tensor* new_ref_count,
                             kvq_tensor* page_map, kvq_stream stream) {
    Trace trace("kvq_compact_pages");
    if (!block_table || !ref_count || !new_table || !new_ref_count || !page_map) return KVQ_ERR_NULL;
    PageCopyArgs a = {};
    CompactArgs p = {};
    int64_t rows, cols, pages, n;
    kvq_status st = table_desc(block_table, &a.table_rows, &a.table_cols, &a.old_table_stride);
    if (st != KVQ_OK) return st;
    if ((st = table_desc(new_table, &rows, &cols, &a.table_stride)) != KVQ_OK) return st;
    if (rows != a.table_rows || cols != a.table_cols) return KVQ_ERR_SHAPE;
    if ((st = vector_desc(ref_count, false, &pages)) != KVQ_OK) return st;
    if ((st = vector_desc(new_ref_count, false, &n)) != KVQ_OK) return st;
    if (n != pages) return KVQ_ERR_SHAPE;
    if ((st = vector_desc(page_map, false, &n)) != KVQ_OK) return st;
    if (n != pages || pages > INT32_MAX - 8 * PL_THREADS) return KVQ_ERR_SHAPE;
    if ((st = page_caches(caches, n_caches, &pages, &a)) != KVQ_OK) return st;
    const bool has_table = a.table_rows > 0 && a.table_cols > 0;
    if ((pages > 0 && (!ref_count->data || !new_ref_count->data || !page_map->data)) ||
        (has_table && (!block_table->data || !new_table->data)))
        return KVQ_ERR_NULL;
    if (pages == 0 && !has_table) return KVQ_OK;
    if ((st = cache_pointers(a)) != KVQ_OK) return st;
    p.ref_count = static_cast<const int32_t*>(ref_count->data);
    p.new_ref = static_cast<int32_t*>(new_ref_count->data);
    p.page_map = static_cast<int32_t*>(page_map->data);
    p.num_pages = (int32_t)pages;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch(compact_plan_kernel, 1, PL_THREADS, 0, s, p) != cudaSuccess) return KVQ_ERR_CUDA;
    a.n_pairs = pages;
    a.num_pages = pages;
    a.pair_page = p.page_map;
    a.old_table = static_cast<const int32_t*>(block_table->data);
    a.table = static_cast<int32_t*>(new_table->data);
    return run_copy<PG_COMPACT>(a, s);
}

}  // extern "C"
