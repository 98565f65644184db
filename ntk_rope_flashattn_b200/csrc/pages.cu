// pages.cu -- the bookkeeping of the page cache on the device: sequences grow
// (extend), are copied (fork), end (free), and the used pages move together
// (compact).  See lcx_paged_cache in lcx.h for the state and its invariants.
//
// Each call decides in one small kernel what happens to every entry (ranks by
// prefix sums, so results do not depend on thread order), and a second kernel,
// a programmatic dependent, moves the data: page copies are the only traffic
// that counts, 2 x layers x page bytes read and written per page, bound by HBM.
// Measured: a fork of 32 sequences (free, fork and three small kernels) that moves
// 0.27 GB: 49 us, 5.5 TB/s; a compaction that moves 0.46 GB: 81 us, 5.6 TB/s (of 6.5 TB/s
// for a plain copy; 10 to 12 us are the deciding kernels and the launches).
#include <algorithm>
#include <climits>

#include "paged.cuh"

namespace lcx {
namespace {

constexpr int kT = 1024;  // threads of a deciding CTA, at most: one entry each
static_assert(kT == LCX_PAGES_MAX_ENTRIES, "one thread per entry");

// Inclusive prefix sum of x over the CTA's threads; *total = the whole sum.  Safe to
// call repeatedly.
__device__ int block_scan(int x, int *total) {
    __shared__ int warp_sum[kT / 32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x / 32;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) warp_sum[w] = v;
    __syncthreads();
    if (w == 0) {
        int s = lane < warps ? warp_sum[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    v += w > 0 ? warp_sum[w - 1] : 0;
    *total = warp_sum[warps - 1];
    __syncthreads();
    return v;
}

// Whether an entry before `i` names the same sequence (ids in shared memory).
__device__ bool seen_before(const int *ids, int i, int id) {
    for (int j = 0; j < i; ++j)
        if (ids[j] == id) return true;
    return false;
}

// The free stack's depth, kept inside the array whatever the word holds.
__device__ int free_depth(const PagedParams &p) { return min(max(*p.n_free, 0), p.P); }

// ------------------------------------------------------------------ extend
__global__ void __launch_bounds__(kT)
    extend_kernel(const __grid_constant__ PagedParams p, const int *ids, const int *n_new, int n,
                  int *start, int *status) {
    wait_previous_kernel();
    __shared__ int s_id[kT], s_end[kT], s_first[kT];
    const int i = threadIdx.x;
    const int id = i < n ? ids[i] : -1;
    s_id[i] = id;
    __syncthreads();
    const int avail = free_depth(p);
    long long need = 0;
    int old = -1, first = 0;
    long long grown = 0;
    if (id >= 0) {
        const int cnt = n_new ? n_new[i] : 1;
        if (id >= p.S || cnt < 0 || seen_before(s_id, i, id)) {
            raise_status(status, LCX_ERR_INVALID_ARG);
        } else {
            const int len = p.lens[id];
            grown = (long long)len + cnt;
            if (len < 0 || grown > (long long)p.MP * p.ps) {
                raise_status(status, LCX_ERR_INVALID_ARG);
            } else {
                old = len;
                first = (len + p.ps - 1) >> p.ps_log2;
                need = ((grown + p.ps - 1) >> p.ps_log2) - first;
            }
        }
    }
    // A need beyond the pool counts as num_pages + 1 (at most 2^20 + 1): still too
    // much, and 1024 of them stay inside 32 bits.
    const int need_c = int(min(need, (long long)p.P + 1));
    int total;
    const int incl = block_scan(need_c, &total);
    const bool granted = old >= 0 && (need == 0 || incl <= avail);
    if (old >= 0 && !granted) raise_status(status, LCX_ERR_NO_PAGES);
    // Granted entries with pages are the first ones: their sum is the largest
    // granted prefix, found as a sum of their own needs.
    int taken;
    const int end = block_scan(granted ? need_c : 0, &taken);
    s_end[i] = end;
    s_first[i] = first;
    if (granted) p.lens[id] = int(grown);
    if (i < n) start[i] = granted ? old : -1;
    __syncthreads();
    // Every page taken by its own thread: page t of the block belongs to the
    // first entry whose running end lies beyond t.
    for (int t = i; t < taken; t += blockDim.x) {
        int lo = 0, hi = int(blockDim.x) - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > t) hi = mid; else lo = mid + 1;
        }
        const int k = t - (lo > 0 ? s_end[lo - 1] : 0);
        const int at = avail - taken + t;
        const int page = p.free_pages[at];
        p.free_pages[at] = -1;
        const bool ok = page >= 0 && page < p.P;
        if (ok) p.ref[page] = 1; else raise_status(status, LCX_ERR_INVALID_ARG);
        p.table[(long long)s_id[lo] * p.MP + s_first[lo] + k] = ok ? page : -1;
    }
    if (i == 0) *p.n_free = avail - taken;
}

// ------------------------------------------------------------------ fork
__global__ void __launch_bounds__(kT)
    fork_kernel(const __grid_constant__ PagedParams p, const int *src, const int *dst, int n,
                int *status) {
    wait_previous_kernel();
    __shared__ int s_dst[kT], s_free[kT];
    const PagedScratch x = paged_scratch(p.scratch, p.P);
    const int i = threadIdx.x;
    const int a = i < n ? src[i] : -1, b = i < n ? dst[i] : -1;
    s_dst[i] = b;
    // (loads that need not wait for one another go out together: the kernel's time is
    // a chain of them)
    const int avail = free_depth(p);
    const bool named = a >= 0 && b >= 0, in = named && a < p.S && b < p.S;
    const int len_a = in ? p.lens[a] : 0, len_b = in ? p.lens[b] : 0;
    if (i < avail) s_free[i] = p.free_pages[avail - 1 - i];
    __syncthreads();
    int len = -1, need = 0, old_page = -1;
    if (named) {
        if (!in || len_b != 0 || seen_before(s_dst, i, b)) {
            raise_status(status, LCX_ERR_INVALID_ARG);
        } else {
            len = len_a;
            if (len < 0 || len > (long long)p.MP * p.ps) {
                raise_status(status, LCX_ERR_INVALID_ARG);
                len = -1;
            } else if (len & (p.ps - 1)) {
                old_page = p.table[(long long)a * p.MP + (len >> p.ps_log2)];
                if (old_page < 0 || old_page >= p.P) {
                    raise_status(status, LCX_ERR_INVALID_ARG);
                    len = -1;
                } else {
                    need = 1;
                }
            }
        }
    }
    int total;
    const int incl = block_scan(need, &total);   // (its barriers: every length read by now)
    const bool granted = len >= 0 && (need == 0 || incl <= avail);
    if (len >= 0 && !granted) raise_status(status, LCX_ERR_NO_PAGES);
    const int taken = min(total, avail);
    int page = -1;
    if (granted && need) {
        const int at = avail - taken + incl - 1;   // taken <= n: among the staged ones
        page = s_free[avail - 1 - at];
        p.free_pages[at] = -1;
        if (page < 0 || page >= p.P) {
            raise_status(status, LCX_ERR_INVALID_ARG);
            page = -1;
        } else {
            p.ref[page] = 1;
        }
        x.src[incl - 1] = page >= 0 ? old_page : -1;
        x.dst[incl - 1] = page;
    }
    if (granted) p.lens[b] = len;
    x.ent_full[i] = granted ? len >> p.ps_log2 : -1;
    x.ent_page[i] = granted && need ? page : -2;
    if (i == 0) {
        *x.n_pairs = taken;
        *p.n_free = avail - taken;
    }
}

// ------------------------------------------------------------------ page data
// How one page's bytes lie in a pool: dense (one run of ps H D elements), or
// rows of D elements per (slot, head).
struct PageShape {
    int vecs;        // 16-byte vectors of a page
    int vpr;         // vectors per row
    int H;
    bool dense_k, dense_v;
};

__device__ __forceinline__ long long page_vec(const PageShape &g, bool dense, int es,
                                              const long long *st, int v) {
    if (dense) return 16ll * v;
    const int row = v / g.vpr, c = v - row * g.vpr;
    const int slot = row / g.H, h = row - slot * g.H;
    return (slot * st[2] + h * st[3]) * es + 16ll * c;
}

constexpr int kCopyThreads = 256, kCopyVecs = 4;  // a CTA step copies 16 KB
constexpr int kCopyCtas = 8;                      // CTAs per SM

// Copy the n_pairs page pairs of the scratch list, every layer, K and V.
__device__ void copy_pairs(const PagedParams &p, const PageShape &g, const PagedScratch &x) {
    constexpr int kChunk = kCopyThreads * kCopyVecs;
    const int n = *x.n_pairs;
    const int cpp = (g.vecs + kChunk - 1) / kChunk;           // chunks per page
    const long long per_pair = 2ll * p.layers * cpp;
    for (long long u = blockIdx.x; u < n * per_pair; u += gridDim.x) {
        const int pair = int(u / per_pair);
        int r = int(u % per_pair);
        const int layer = r / (2 * cpp);
        r -= layer * 2 * cpp;
        const bool is_v = r >= cpp;
        const int c0 = (is_v ? r - cpp : r) * kChunk;
        const int a = x.src[pair], b = x.dst[pair];
        if (a < 0 || b < 0 || a >= p.P || b >= p.P) continue;
        const long long *st = is_v ? p.vs : p.ks;
        const bool dense = is_v ? g.dense_v : g.dense_k;
        char *pool = is_v ? p.v : p.k;
        const char *from = pool + (layer * st[0] + a * st[1]) * p.es;
        char *to = pool + (layer * st[0] + b * st[1]) * p.es;
        uint4 w[kCopyVecs];
#pragma unroll
        for (int k = 0; k < kCopyVecs; ++k) {
            const int v = c0 + k * kCopyThreads + threadIdx.x;
            if (v < g.vecs)
                w[k] = __ldcs(reinterpret_cast<const uint4 *>(from + page_vec(g, dense, p.es, st, v)));
        }
#pragma unroll
        for (int k = 0; k < kCopyVecs; ++k) {
            const int v = c0 + k * kCopyThreads + threadIdx.x;
            if (v < g.vecs)
                __stcs(reinterpret_cast<uint4 *>(to + page_vec(g, dense, p.es, st, v)), w[k]);
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ PagedParams p, PageShape g) {
    wait_previous_kernel();
    copy_pairs(p, g, paged_scratch(p.scratch, p.P));
}

// Second kernel of a fork: table rows and counts of the shared pages (one warp
// per entry and stretch of 32 pages), then the partial pages' data.
__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(const __grid_constant__ PagedParams p, PageShape g, const int *src,
                      const int *dst, int n, int *status) {
    wait_previous_kernel();
    const PagedScratch x = paged_scratch(p.scratch, p.P);
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kCopyThreads / 32);
    const int w0 = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const int per = (p.MP + 31) / 32;                 // stretches per entry
    for (long long u = w0; u < (long long)n * per; u += warps) {
        const int i = int(u / per), j = int(u % per) * 32 + lane;
        const int full = x.ent_full[i];
        if (full < 0) continue;
        const long long a = (long long)src[i] * p.MP, b = (long long)dst[i] * p.MP;
        if (j < full) {
            const int page = p.table[a + j];
            p.table[b + j] = page;
            if (page >= 0 && page < p.P) atomicAdd(&p.ref[page], 1);
            else raise_status(status, LCX_ERR_INVALID_ARG);
        } else if (j == full && j < p.MP && x.ent_page[i] != -2) {
            p.table[b + j] = x.ent_page[i];
        }
    }
    copy_pairs(p, g, x);
}

// ------------------------------------------------------------------ free
// One warp per (entry, stretch of 32 pages): the page's last holder marks it.
__global__ void __launch_bounds__(256)
    release_kernel(const __grid_constant__ PagedParams p, const int *ids, int n, int *status) {
    wait_previous_kernel();
    const PagedScratch x = paged_scratch(p.scratch, p.P);
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * 8, w0 = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int per = (p.MP + 31) / 32;
    for (long long u = w0; u < (long long)n * per; u += warps) {
        const int i = int(u / per), stretch = int(u % per), j = stretch * 32 + lane;
        const int id = ids[i];
        if (id < 0) continue;
        bool bad = id >= p.S;
        for (int e = lane; e < i && !bad; e += 32) bad = ids[e] == id;
        if (__any_sync(0xffffffffu, bad)) {
            if (lane == 0) raise_status(status, LCX_ERR_INVALID_ARG);
            continue;
        }
        if (j >= p.MP) continue;
        int *row = p.table + (long long)id * p.MP;
        const int page = row[j];
        if (page < 0) continue;
        row[j] = -1;
        if (page >= p.P) {
            raise_status(status, LCX_ERR_INVALID_ARG);
            continue;
        }
        const int had = atomicSub(&p.ref[page], 1);
        if (had == 1) {
            x.mark[page] = 1;
        } else if (had <= 0) {          // not held: the counts were wrong already
            atomicAdd(&p.ref[page], 1);
            raise_status(status, LCX_ERR_INVALID_ARG);
        }
    }
}

// Marked pages go back to the stack in ascending order; lengths become 0.
__global__ void __launch_bounds__(kT)
    collect_kernel(const __grid_constant__ PagedParams p, const int *ids, int n, int *status) {
    wait_previous_kernel();
    const PagedScratch x = paged_scratch(p.scratch, p.P);
    const int i = threadIdx.x;
    if (i < n && ids[i] >= 0 && ids[i] < p.S) p.lens[ids[i]] = 0;
    int depth = free_depth(p);
    for (int base = 0; base < p.P; base += 4 * kT) {
        const int q0 = base + 4 * i;
        int m[4], c = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m[k] = q0 + k < p.P ? x.mark[q0 + k] : 0;
            c += m[k] != 0;
        }
        int total;
        int at = depth + block_scan(c, &total) - c;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (m[k]) {
                x.mark[q0 + k] = 0;
                if (at < p.P) p.free_pages[at] = q0 + k;
                else raise_status(status, LCX_ERR_INVALID_ARG);
                ++at;
            }
        depth += total;
    }
    if (i == 0) *p.n_free = min(depth, p.P);
}

// ------------------------------------------------------------------ compact
__global__ void __launch_bounds__(kT) compact_kernel(const __grid_constant__ PagedParams p) {
    wait_previous_kernel();
    const PagedScratch x = paged_scratch(p.scratch, p.P);
    const int i = threadIdx.x;
    int used = 0;
    for (int q = i; q < p.P; q += kT) used += p.ref[q] > 0;
    int U;
    block_scan(used, &U);
    // Below U the free pages are ranked (holes), from U on the used ones
    // (movers); there are as many of each.
    int holes = 0, movers = 0;
    for (int base = 0; base < p.P; base += 4 * kT) {
        const int q0 = base + 4 * i;
        bool h[4], m[4];
        int ch = 0, cm = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int q = q0 + k;
            const bool in = q < p.P, u = in && p.ref[q] > 0;
            h[k] = in && !u && q < U;
            m[k] = u && q >= U;
            ch += h[k];
            cm += m[k];
            if (in) x.remap[q] = q;
        }
        int th, tm;
        int ah = holes + block_scan(ch, &th) - ch;
        int am = movers + block_scan(cm, &tm) - cm;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (h[k]) x.dst[ah++] = q0 + k;
            if (m[k]) x.src[am++] = q0 + k;
        }
        holes += th;
        movers += tm;
    }
    __syncthreads();
    for (int k = i; k < movers; k += kT) {
        const int a = x.src[k], b = x.dst[k];
        x.remap[a] = b;
        p.ref[b] = p.ref[a];
        p.ref[a] = 0;
    }
    for (int q = i; q < p.P; q += kT) p.free_pages[q] = q < p.P - U ? p.P - 1 - q : -1;
    if (i == 0) {
        *x.n_pairs = movers;
        *p.n_free = p.P - U;
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_apply_kernel(const __grid_constant__ PagedParams p, PageShape g, int *status) {
    wait_previous_kernel();
    const PagedScratch x = paged_scratch(p.scratch, p.P);
    const long long total = (long long)p.S * p.MP;
    for (long long u = blockIdx.x * (long long)kCopyThreads + threadIdx.x; u < total;
         u += (long long)gridDim.x * kCopyThreads) {
        const int page = p.table[u];
        if (page < 0) continue;
        if (page >= p.P) raise_status(status, LCX_ERR_INVALID_ARG);
        else p.table[u] = x.remap[page];
    }
    copy_pairs(p, g, x);
}

// ------------------------------------------------------------------ copy
__global__ void __launch_bounds__(kT)
    copy_list_kernel(const __grid_constant__ PagedParams p, const int *src, const int *dst, int n,
                     int *status) {
    wait_previous_kernel();
    __shared__ int s_src[kT], s_dst[kT];
    const PagedScratch x = paged_scratch(p.scratch, p.P);
    const int i = threadIdx.x;
    const int a = i < n ? src[i] : -1, b = i < n ? dst[i] : -1;
    s_src[i] = a;
    s_dst[i] = b;
    __syncthreads();
    bool go = a >= 0 && b >= 0 && a != b;
    if (go) {
        bool bad = a >= p.P || b >= p.P || seen_before(s_dst, i, b);
        for (int j = 0; j < n && !bad; ++j) bad = s_src[j] == b;
        if (bad) {
            raise_status(status, LCX_ERR_INVALID_ARG);
            go = false;
        }
    }
    if (i < n) {
        x.src[i] = go ? a : -1;
        x.dst[i] = go ? b : -1;
    }
    if (i == 0) *x.n_pairs = n;
}

PageShape page_shape(const PagedParams &p) {
    PageShape g;
    g.vpr = p.D * p.es / 16;
    g.H = p.H;
    g.vecs = p.ps * p.H * g.vpr;
    auto dense = [&](const long long *st) {
        // [slot][head][dim] or [head][slot][dim] without gaps
        const bool nhd = (p.H == 1 || st[3] == p.D) && (p.ps == 1 || st[2] == (long long)p.H * p.D);
        const bool hnd = (p.ps == 1 || st[2] == p.D) && (p.H == 1 || st[3] == (long long)p.ps * p.D);
        return nhd || hnd;
    };
    g.dense_k = dense(p.ks);
    g.dense_v = dense(p.vs);
    return g;
}

lcx_status entries_ok(const void *a, const void *b, int64_t n, const char *what) {
    if (n < 0) return fail(LCX_ERR_INVALID_ARG, "%s: negative entry count", what);
    if (n > LCX_PAGES_MAX_ENTRIES)
        return fail(LCX_ERR_UNSUPPORTED, "%s: more than %d entries in one call", what,
                    LCX_PAGES_MAX_ENTRIES);
    if (n > 0 && (!a || !b)) return fail(LCX_ERR_INVALID_ARG, "%s: NULL index array", what);
    return LCX_OK;
}

// Threads of a CTA that decides about n entries (more than n take pages in extend).
unsigned deciding(int64_t n) { return unsigned(std::max<int64_t>(256, (n + 31) / 32 * 32)); }

lcx_status launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
    return LCX_OK;
}

}  // namespace

lcx_status check_tokens(const void *ptr, const int64_t *st, int es, const char *name) {
    if (!ptr) return fail(LCX_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned16(ptr)) return fail(LCX_ERR_UNSUPPORTED, "%s must be 16-byte aligned", name);
    if (st[2] != 1) return fail(LCX_ERR_UNSUPPORTED, "%s: head_dim stride must be 1", name);
    for (int d = 0; d < 2; ++d) {
        if (st[d] < 0) return fail(LCX_ERR_UNSUPPORTED, "%s: negative stride", name);
        if ((st[d] * es) % 16 != 0)
            return fail(LCX_ERR_UNSUPPORTED, "%s: strides must be multiples of 16 bytes", name);
    }
    return LCX_OK;
}

lcx_status check_distinct(const int64_t *st, int64_t tokens, int64_t heads, const char *name) {
    if ((st[0] == 0 && tokens > 1) || (st[1] == 0 && heads > 1))
        return fail(LCX_ERR_UNSUPPORTED, "%s: stride 0", name);
    return LCX_OK;
}

lcx_status paged_prepare(const lcx_paged_cache *c, PagedParams &x) {
    if (!c) return fail(LCX_ERR_INVALID_ARG, "cache is NULL");
    if (c->dtype != LCX_BF16 && c->dtype != LCX_F32)
        return fail(LCX_ERR_INVALID_ARG, "unknown dtype %d", c->dtype);
    if (c->num_layers <= 0 || c->num_pages <= 0 || c->Hkv <= 0 || c->max_seqs <= 0 ||
        c->max_pages <= 0)
        return fail(LCX_ERR_INVALID_ARG, "cache: sizes must be positive");
    if (c->D != 64 && c->D != 128)
        return fail(LCX_ERR_UNSUPPORTED, "cache: head_dim %lld: only 64 and 128", (long long)c->D);
    if (c->page_size < 1 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return fail(LCX_ERR_UNSUPPORTED, "cache: page_size %d must be a power of two up to 1024",
                    c->page_size);
    if (c->num_pages > (1 << 20) || c->max_seqs > (1 << 20) || c->Hkv > 4096 ||
        c->num_layers > 4096 || c->max_pages * c->page_size > (int64_t(1) << 30) ||
        c->max_pages > (1 << 30))
        return fail(LCX_ERR_UNSUPPORTED, "cache: sizes too large");
    if (!c->k_pages || !c->v_pages || !c->block_table || !c->seq_lens || !c->ref_counts ||
        !c->free_pages || !c->n_free || !c->scratch)
        return fail(LCX_ERR_INVALID_ARG, "cache: NULL buffer");
    if (!aligned16(c->k_pages) || !aligned16(c->v_pages))
        return fail(LCX_ERR_UNSUPPORTED, "cache: pools must be 16-byte aligned");
    const int es = c->dtype == LCX_BF16 ? 2 : 4;
    const int64_t dims[4] = {c->num_layers, c->num_pages, c->page_size, c->Hkv};
    for (int t = 0; t < 2; ++t) {
        const int64_t *st = t ? c->v_strides : c->k_strides;
        if (st[4] != 1) return fail(LCX_ERR_UNSUPPORTED, "cache: head_dim stride must be 1");
        for (int d = 0; d < 4; ++d) {
            if (st[d] < 0 || (st[d] == 0 && dims[d] > 1))
                return fail(LCX_ERR_UNSUPPORTED, "cache: pool strides must be positive");
            if ((st[d] * es) % 16 != 0)
                return fail(LCX_ERR_UNSUPPORTED, "cache: strides must be multiples of 16 bytes");
        }
    }
    x.k = static_cast<char *>(c->k_pages);
    x.v = static_cast<char *>(c->v_pages);
    x.table = c->block_table;
    x.lens = c->seq_lens;
    x.ref = c->ref_counts;
    x.free_pages = c->free_pages;
    x.n_free = c->n_free;
    x.scratch = c->scratch;
    x.es = es;
    x.ps = c->page_size;
    x.ps_log2 = 0;
    while ((1 << x.ps_log2) < x.ps) ++x.ps_log2;
    x.layers = int(c->num_layers);
    x.P = int(c->num_pages);
    x.H = int(c->Hkv);
    x.D = int(c->D);
    x.S = int(c->max_seqs);
    x.MP = int(c->max_pages);
    for (int d = 0; d < 4; ++d) {
        x.ks[d] = c->k_strides[d];
        x.vs[d] = c->v_strides[d];
    }
    return LCX_OK;
}

}  // namespace lcx

using namespace lcx;

extern "C" int64_t lcx_paged_scratch_ints(int64_t num_pages) {
    if (num_pages <= 0 || num_pages > (1 << 20)) return -1;
    return paged_scratch_ints(num_pages);
}

extern "C" lcx_status lcx_pages_extend(const lcx_paged_cache *cache, const int32_t *seq_ids,
                                       const int32_t *n_new, int64_t n, int32_t *start,
                                       int32_t *dev_status, void *stream) {
    clear_error();
    PagedParams p;
    lcx_status st = paged_prepare(cache, p);
    if (st != LCX_OK) return st;
    if ((st = entries_ok(seq_ids, start, n, "extend")) != LCX_OK || n == 0) return st;
    return launched(launch_dependent(extend_kernel, dim3(1), dim3(deciding(n)), 0,
                                     static_cast<cudaStream_t>(stream), p, seq_ids, n_new, int(n),
                                     start, dev_status),
                    "pages_extend");
}

extern "C" lcx_status lcx_pages_fork(const lcx_paged_cache *cache, const int32_t *src,
                                     const int32_t *dst, int64_t n, int32_t *dev_status,
                                     void *stream) {
    clear_error();
    PagedParams p;
    lcx_status st = paged_prepare(cache, p);
    if (st != LCX_OK) return st;
    if ((st = entries_ok(src, dst, n, "fork")) != LCX_OK || n == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = launched(launch_dependent(fork_kernel, dim3(1), dim3(deciding(n)), 0, s, p, src, dst,
                                        int(n), dev_status),
                       "pages_fork")) != LCX_OK)
        return st;
    return launched(launch_dependent(fork_apply_kernel, dim3(device_sms() * kCopyCtas),
                                     dim3(kCopyThreads), 0, s, p, page_shape(p), src, dst, int(n),
                                     dev_status),
                    "pages_fork");
}

extern "C" lcx_status lcx_pages_free(const lcx_paged_cache *cache, const int32_t *seq_ids,
                                     int64_t n, int32_t *dev_status, void *stream) {
    clear_error();
    PagedParams p;
    lcx_status st = paged_prepare(cache, p);
    if (st != LCX_OK) return st;
    if ((st = entries_ok(seq_ids, seq_ids, n, "free")) != LCX_OK || n == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long warps = n * ((p.MP + 31) / 32);
    const unsigned grid = unsigned(std::min<long long>((warps + 7) / 8, device_sms() * kCopyCtas));
    if ((st = launched(launch_dependent(release_kernel, dim3(grid), dim3(256), 0, s, p, seq_ids,
                                        int(n), dev_status),
                       "pages_free")) != LCX_OK)
        return st;
    return launched(launch_dependent(collect_kernel, dim3(1), dim3(kT), 0, s, p, seq_ids, int(n),
                                     dev_status),
                    "pages_free");
}

extern "C" lcx_status lcx_pages_compact(const lcx_paged_cache *cache, int32_t *dev_status,
                                        void *stream) {
    clear_error();
    PagedParams p;
    lcx_status st = paged_prepare(cache, p);
    if (st != LCX_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = launched(launch_dependent(compact_kernel, dim3(1), dim3(kT), 0, s, p),
                       "pages_compact")) != LCX_OK)
        return st;
    return launched(launch_dependent(compact_apply_kernel, dim3(device_sms() * kCopyCtas),
                                     dim3(kCopyThreads), 0, s, p, page_shape(p), dev_status),
                    "pages_compact");
}

extern "C" lcx_status lcx_pages_copy(const lcx_paged_cache *cache, const int32_t *src_pages,
                                     const int32_t *dst_pages, int64_t n, int32_t *dev_status,
                                     void *stream) {
    clear_error();
    PagedParams p;
    lcx_status st = paged_prepare(cache, p);
    if (st != LCX_OK) return st;
    if ((st = entries_ok(src_pages, dst_pages, n, "copy")) != LCX_OK || n == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = launched(launch_dependent(copy_list_kernel, dim3(1), dim3(deciding(n)), 0, s, p,
                                        src_pages, dst_pages, int(n), dev_status),
                       "pages_copy")) != LCX_OK)
        return st;
    return launched(launch_dependent(copy_kernel, dim3(device_sms() * kCopyCtas), dim3(kCopyThreads), 0, s,
                                     p, page_shape(p)),
                    "pages_copy");
}
