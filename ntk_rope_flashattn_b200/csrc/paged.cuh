// paged.cuh -- the page cache as the kernels see it, and the checks its entry
// points share (lcx_paged_cache).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "lcx_internal.h"

namespace lcx {

struct PagedParams {
    char *k, *v;                                  // pools
    int *table, *lens, *ref, *free_pages, *n_free, *scratch;
    int es;                                       // bytes per element
    int ps, ps_log2;                              // page size
    int layers, P, H, D, S, MP;                   // pages, kv heads, dim, sequences, pages each
    long long ks[4], vs[4];                       // element strides: layer, page, slot, head
};

// Scratch (int32): the page pairs of a data copy, the number of pairs, and what
// one kernel of a call leaves for the next.  `mark` is zero between calls.
struct PagedScratch {
    int *n_pairs, *src, *dst, *remap, *mark, *ent_full, *ent_page;
};
__host__ __device__ inline PagedScratch paged_scratch(int *s, long long P) {
    PagedScratch x;
    x.n_pairs = s;
    x.ent_full = s + 4;
    x.ent_page = x.ent_full + LCX_PAGES_MAX_ENTRIES;
    x.src = x.ent_page + LCX_PAGES_MAX_ENTRIES;
    x.dst = x.src + P + LCX_PAGES_MAX_ENTRIES;
    x.remap = x.dst + P + LCX_PAGES_MAX_ENTRIES;
    x.mark = x.remap + P;
    return x;
}
inline long long paged_scratch_ints(long long P) {
    return 4 + 4ll * LCX_PAGES_MAX_ENTRIES + 4 * P;
}

// A status stays unless a larger code follows; LCX_ERR_TIMEOUT (results undefined)
// replaces every other one and stays.  (`code` is a constant: one branch is left.)
__device__ __forceinline__ void raise_status(int *status, int code) {
    if (!status) return;
    if (code == LCX_ERR_TIMEOUT) {
        atomicExch(status, code);
    } else if (code < LCX_ERR_TIMEOUT) {
        atomicMax(status, code);
    } else {
        for (int was = 0;;) {               // (every other writer raises it: a few turns)
            const int now = atomicCAS(status, was, code);
            if (now == was || now >= code || now == LCX_ERR_TIMEOUT) break;
            was = now;
        }
    }
}

// Validate `c` and fill `x`.
lcx_status paged_prepare(const lcx_paged_cache *c, PagedParams &x);

// Shared argument checks: a tensor of (token, head, dim) strides in elements.
lcx_status check_tokens(const void *ptr, const int64_t *st, int es, const char *name);
// Refuses a tensor whose tokens or heads share memory (stride 0).
lcx_status check_distinct(const int64_t *st, int64_t tokens, int64_t heads, const char *name);

// Launch `kern` as a programmatic dependent of the stream's previous kernel: it
// may be scheduled while that one ends and waits (griddepcontrol.wait) for its
// results.  A call's first kernel waits before all else and in every CTA, so that
// what it lets start early (pdl_launch_dependents) and what follows it find the
// stream's earlier work done.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

__device__ __forceinline__ void wait_previous_kernel() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The current device's SM count (148 when it cannot be asked).
inline int device_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    return sms;
}

}  // namespace lcx
