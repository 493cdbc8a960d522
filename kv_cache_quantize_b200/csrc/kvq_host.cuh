// kvq_host.cuh -- what the C ABI's translation units share on the host:
// descriptor checks, launch sizing, launches and the tensor-map encoder.
// Everything is internal to the unit that includes it.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <atomic>
#include <mutex>
#include <utility>

#include <nvtx3/nvToolsExt.h>

#include "kvq.h"
#include "kvq_device.cuh"

namespace kvq {
// The other units' fault words on the current device (each unit's kernels
// raise their bits in a word of its own; kvq_get_error reads them all).
unsigned int* attention_fault_word();
unsigned int* pages_fault_word();
}  // namespace kvq

namespace {

using namespace kvq;

// ---------------------------------------------------------------------------
// descriptor helpers
// ---------------------------------------------------------------------------
int64_t elem_bytes(int32_t dt) {
    switch (dt) {
        case KVQ_BF16: case KVQ_F16: return 2;
        case KVQ_F32: case KVQ_I32: return 4;
        case KVQ_I64: return 8;
        case KVQ_I8: case KVQ_U8: case KVQ_F8E4M3: case KVQ_F8E5M2: case KVQ_E8M0: return 1;
        default: return 0;
    }
}

bool valid_desc(const kvq_tensor* t) {
    if (!t || t->ndim < 0 || t->ndim > KVQ_MAX_DIMS || elem_bytes(t->dtype) == 0) return false;
    for (int i = 0; i < t->ndim; ++i)
        if (t->shape[i] < 0) return false;
    return true;
}

int64_t numel(const kvq_tensor* t) {
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
    return n;
}

int64_t numel_leading(const kvq_tensor* t) {
    int64_t n = 1;
    for (int i = 0; i + 1 < t->ndim; ++i) n *= t->shape[i];
    return n;
}

// Row-major contiguous (dimensions of size 1 may carry any stride).
bool contiguous(const kvq_tensor* t) {
    if (numel(t) == 0) return true;   // no elements: any strides describe it
    int64_t expect = 1;
    for (int i = t->ndim - 1; i >= 0; --i) {
        if (t->shape[i] == 1) continue;
        if (t->stride[i] != expect) return false;
        expect *= t->shape[i];
    }
    return true;
}

// Last dimension contiguous and the leading dimensions flattenable into rows
// with one row stride (in elements).
bool flatten_rows(const kvq_tensor* t, int64_t* rows, int64_t* row_stride) {
    if (t->ndim < 1) return false;
    const int64_t d = t->shape[t->ndim - 1];
    if (numel(t) == 0) {             // no elements: any strides describe it
        *rows = d == 0 ? 0 : numel_leading(t);
        *row_stride = d;
        return true;
    }
    if (d > 1 && t->stride[t->ndim - 1] != 1) return false;
    int64_t r = 1, rs = -1, expect = -1;
    for (int i = t->ndim - 2; i >= 0; --i) {
        r *= t->shape[i];
        if (t->shape[i] == 1) continue;
        if (rs < 0) {
            rs = t->stride[i];
        } else if (t->stride[i] != expect) {
            return false;
        }
        expect = t->stride[i] * t->shape[i];
    }
    if (rs < 0) rs = d;
    if (r > 1 && rs < d) return false;
    *rows = r;
    *row_stride = rs;
    return true;
}

// A cache [blockNum, a, b, headDim] with one of a/b equal to 1 (the other is
// blockSize) -- or, when inner > 1, [blockNum, blockSize, inner, headDim].
// Rows of inner*headDim elements are contiguous inside a block; only the
// block dimension may be strided.
kvq_status paged_from(const kvq_tensor* c, int64_t inner, PagedRows* out, int64_t* head_dim) {
    if (c->ndim != 4) return KVQ_ERR_NDIM;
    const int64_t eb = elem_bytes(c->dtype);
    const int64_t hd = c->shape[3];
    int64_t bs;
    int bs_dim;
    if (inner > 1) {
        if (c->shape[2] != inner) return KVQ_ERR_SHAPE;
        bs = c->shape[1];
        bs_dim = 1;
        if (hd > 1 && c->stride[3] != 1) return KVQ_ERR_LAYOUT;
        if (inner > 1 && c->stride[2] != hd) return KVQ_ERR_LAYOUT;
        if (bs > 1 && c->stride[1] != inner * hd) return KVQ_ERR_LAYOUT;
    } else {
        if (c->shape[2] == 1) { bs = c->shape[1]; bs_dim = 1; }
        else if (c->shape[1] == 1) { bs = c->shape[2]; bs_dim = 2; }
        else return KVQ_ERR_SHAPE;
        if (hd > 1 && c->stride[3] != 1) return KVQ_ERR_LAYOUT;
        if (bs > 1 && c->stride[bs_dim] != hd) return KVQ_ERR_LAYOUT;
    }
    const int64_t nb = c->shape[0];
    const int64_t row = inner * hd;
    if (nb > 1 && c->stride[0] < bs * row) return KVQ_ERR_LAYOUT;
    out->base = static_cast<uint8_t*>(c->data);
    out->num_slots = nb * bs;
    out->block_size = bs;
    out->row_bytes = row * eb;
    out->block_stride = (nb > 1 ? c->stride[0] : bs * row) * eb;
    out->bs_shift = -1;
    for (int k = 0; k < 62; ++k)
        if (bs == (int64_t(1) << k)) out->bs_shift = k;
    *head_dim = hd;
    return KVQ_OK;
}

bool is_index_dtype(int32_t dt) { return dt == KVQ_I32 || dt == KVQ_I64; }

// A named NVTX range over one C-ABI call (visible in profilers; a no-op
// unless a tool is attached).
struct Trace {
    explicit Trace(const char* name) { nvtxRangePushA(name); }
    ~Trace() { nvtxRangePop(); }
};

// ---------------------------------------------------------------------------
// launch sizing: a grid of (SMs x resident blocks) persistent blocks at most
// ---------------------------------------------------------------------------
int sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    if (!cached[dev]) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        cached[dev] = n > 0 ? n : 148;
    }
    return cached[dev];
}

// Resident blocks per SM of a kernel at a launch shape, asked of the runtime
// once per (kernel, device, threads, shared memory) and remembered: the
// query costs host time on every call otherwise.  Kernels with dynamic shared
// memory get their opt-in limit raised to the device maximum on first use.
int resident_blocks(const void* fn, int threads, size_t smem) {
    struct Entry { const void* fn; int dev, threads; size_t smem; int occ; };
    static std::mutex mu;
    static Entry table[512];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (table[i].fn == fn && table[i].dev == dev && table[i].threads == threads && table[i].smem == smem)
            return table[i].occ;
    bool attr_set = false;          // the shared-memory limit was raised by an earlier entry
    for (int i = 0; i < used; ++i)
        if (table[i].fn == fn && table[i].dev == dev && table[i].smem > 0) attr_set = true;
    if (smem > 0 && !attr_set) {
        int optin = 0;
        if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess || optin <= 0)
            optin = 227 * 1024;
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
    }
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem) != cudaSuccess || occ < 1) occ = 1;
    if (used < 512) table[used++] = Entry{fn, dev, threads, smem, occ};
    return occ;
}

template <typename K>
int64_t persistent_grid(K kernel, int threads, int64_t needed_blocks, size_t smem = 0) {
    const int occ = resident_blocks(reinterpret_cast<const void*>(kernel), threads, smem);
    const int64_t cap = (int64_t)sm_count() * occ;
    int64_t g = needed_blocks < cap ? needed_blocks : cap;
    return g < 1 ? 1 : g;
}

// Launch with programmatic stream serialization (see pdl_wait in
// kvq_device.cuh): the kernel may be scheduled before the previous kernel of
// the stream completes and waits for it on the device.
// Returns the launch's own status (not cudaGetLastError, which would also
// report -- and clear -- errors left by unrelated earlier CUDA work).
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

kvq_status launched(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

// cuTensorMapEncodeTiled through the runtime's driver entry point (the
// library links the CUDA runtime statically and never links the driver
// library itself)
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

}  // namespace
