// paged_append.cu -- rotate new tokens' keys and queries and write keys and
// values into cache pages (lcx_paged_append); also the rotate pass of packed fp32
// keys that lcx_attn_varlen runs first.
//
// y_p = ms (x_p cos phi - x_q sin phi), y_q = ms (x_p sin phi + x_q cos phi),
// phi = m theta'_i, as in apply_rope.cu, with m the token's position in its own
// sequence ("Long Context: RoPE / YaRN / NTK / MLA", 2.2, 2.4, 6.4).  The angles
// come from the fp64 frequencies: the fp32 table's rounding would move the angle
// at m = 65536 by up to m 2^-25 = 0.002 rad, which fp32 caches can tell.
//
// Bound by HBM: each input vector is read and each output vector written once.
// A CTA owns rows_per_cta tokens and a slice of the heads; one thread owns one
// 16-byte vector of pairs of a token, evaluates their cos/sin once and walks
// the slice.  The token's sequence, position and page are found once per token
// by one thread.
// Measured: 12 prompts (14k tokens, 32 query and 8 kv heads of 128, bf16), 0.46 GB: 81 us,
// 5.7 TB/s of a copy's 6.5; 64 single tokens: 5.6 us, a launch and a chain of loads.
#include <algorithm>

#include "paged.cuh"
#include "rope_angle.cuh"
#include "sm100.cuh"
#include "vec16.cuh"

namespace lcx {
namespace {

constexpr int kThreads = 128;

struct TokenTensor {
    char *p;
    long long st, sh;   // element strides: token, head
};

struct AppendParams {
    TokenTensor k, v, q, qo, ko;        // qo.p, ko.p NULL: not wanted
    char *kp, *vp;                      // pools at the layer, or NULL (packed rotation only)
    long long ks[3], vs[3];             // pool strides: page, slot, head
    const int *ids, *start, *cu;
    const int *table, *lens;
    int *status;
    int n, T, Hq, Hkv, S, MP, P, ps_log2;
    int D, jobs, rows, slices, per;     // jobs per token; tokens per CTA; head slices, heads each
    float ms;
    double theta[64];
};

// Where a token goes: its position and its page's (page << ps_log2 | slot), or
// -1 for a row that is not to be touched.
struct Place {
    int pos;
    long long at;
};

__device__ Place find(const AppendParams &a, int t) {
    Place r;
    r.pos = -1;
    r.at = -1;
    int e = t;
    int first = t;
    if (a.cu) {
        // the last entry whose first row is <= t, if its rows reach t
        int lo = 0, hi = a.n;      // cu[lo] <= t < cu[hi]
        if (t < a.cu[0] || t >= a.cu[a.n]) return r;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= t) lo = mid; else hi = mid;
        }
        e = lo;
        first = a.cu[lo];
    }
    if (e >= a.n) return r;
    if (!a.kp) {                   // packed rotation: positions from 0
        r.pos = t - first;
        r.at = 0;
        return r;
    }
    const int id = a.ids[e], s0 = a.start[e];
    if (id < 0 || s0 < 0) return r;
    const long long pos = (long long)s0 + (t - first);
    if (id >= a.S || pos >= a.lens[id] || (pos >> a.ps_log2) >= a.MP) {
        raise_status(a.status, LCX_ERR_INVALID_ARG);
        return r;
    }
    const int page = a.table[(long long)id * a.MP + (pos >> a.ps_log2)];
    if (page < 0 || page >= a.P) {
        raise_status(a.status, LCX_ERR_INVALID_ARG);
        return r;
    }
    r.pos = int(pos);
    r.at = ((long long)page << a.ps_log2) | (pos & ((1 << a.ps_log2) - 1));
    return r;
}

// One head's vectors of a job rotated: (e1, e2) the pair members (HALF), or the
// one vector at e1 that holds adjacent pairs.
template <typename T, bool kHalf>
__device__ __forceinline__ void rotate(const uint4 &va, const uint4 &vb, const float *c,
                                       const float *s, uint4 &oa, uint4 &ob) {
    constexpr int N = Vec<T>::N;
    if (kHalf) {
        float x1[N], x2[N], y1[N], y2[N];
        unpack(va, x1);
        unpack(vb, x2);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            y1[e] = fmaf(x1[e], c[e], -x2[e] * s[e]);
            y2[e] = fmaf(x1[e], s[e], x2[e] * c[e]);
        }
        oa = pack(y1);
        ob = pack(y2);
    } else {
        float x[N], y[N];
        unpack(va, x);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            y[2 * e] = fmaf(x[2 * e], c[e], -x[2 * e + 1] * s[e]);
            y[2 * e + 1] = fmaf(x[2 * e], s[e], x[2 * e + 1] * c[e]);
        }
        oa = pack(y);
    }
}

template <typename T, bool kHalf>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams a) {
    constexpr int N = Vec<T>::N;
    constexpr int NP = kHalf ? N : N / 2;           // pairs per job
    __shared__ Place place[kThreads];
    wait_previous_kernel();
    pdl_launch_dependents();       // attention over packed fp32 rows may be scheduled
    const int t0 = blockIdx.x * a.rows;
    const int job = threadIdx.x % a.jobs, row = threadIdx.x / a.jobs, t = t0 + row;
    const bool in = row < a.rows && t < a.T;
    const int e1 = job * N, e2 = e1 + a.D / 2;      // HALF: both members; else e1 alone
    // Heads in one list: Hkv keys, Hkv values, Hq queries; this CTA's slice of it.
    const int nv = a.v.p ? a.Hkv : 0, total = a.Hkv + nv + (a.q.p ? a.Hq : 0);
    const int h0 = blockIdx.y * a.per, h1 = min(total, h0 + a.per);
    constexpr int kHB = 8;                          // heads whose loads are in flight together
    uint4 va[kHB], vb[kHB];
    auto load = [&](int b) {
#pragma unroll
        for (int u = 0; u < kHB; ++u) {
            const int h = b + u;
            if (h >= h1) break;
            const bool isk = h < a.Hkv, isv = !isk && h < a.Hkv + nv;
            const TokenTensor &x = isk ? a.k : isv ? a.v : a.q;
            const int hh = isk ? h : isv ? h - a.Hkv : h - a.Hkv - nv;
            const T *src = reinterpret_cast<const T *>(x.p) + t * x.st + hh * x.sh;
            va[u] = __ldcs(reinterpret_cast<const uint4 *>(src + e1));
            if (kHalf) vb[u] = __ldcs(reinterpret_cast<const uint4 *>(src + e2));
        }
    };
    // The first heads' loads go out before the token's place and angles are known
    // (a chain of loads and the sines: some 5 us that nothing else would fill).
    if (in) load(h0);
    if (threadIdx.x < a.rows) {
        Place r;
        r.pos = -1;
        r.at = -1;
        if (t0 + int(threadIdx.x) < a.T) r = find(a, t0 + threadIdx.x);
        place[threadIdx.x] = r;
    }
    __syncthreads();
    if (!in) return;
    const Place w = place[row];
    if (w.at < 0) return;
    float c[NP], s[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        rope_sincos(w.pos, a.theta[job * NP + e], &c[e], &s[e]);
        c[e] *= a.ms;
        s[e] *= a.ms;
    }
    const long long page = a.kp ? w.at >> a.ps_log2 : 0;
    const int slot = int(w.at & ((1 << a.ps_log2) - 1));
    for (int b = h0; b < h1; b += kHB) {
        if (b > h0) load(b);
#pragma unroll
        for (int u = 0; u < kHB; ++u) {
            const int h = b + u;
            if (h >= h1) break;
            const bool isk = h < a.Hkv, isv = !isk && h < a.Hkv + nv;
            uint4 oa = va[u], ob = vb[u];
            if (!isv) rotate<T, kHalf>(va[u], vb[u], c, s, oa, ob);
            auto put = [&](T *dst) {
                __stcs(reinterpret_cast<uint4 *>(dst + e1), oa);
                if (kHalf) __stcs(reinterpret_cast<uint4 *>(dst + e2), ob);
            };
            if (isk) {
                if (a.kp)
                    put(reinterpret_cast<T *>(a.kp) + page * a.ks[0] + slot * a.ks[1] + h * a.ks[2]);
                if (a.ko.p) put(reinterpret_cast<T *>(a.ko.p) + t * a.ko.st + h * a.ko.sh);
            } else if (isv) {
                put(reinterpret_cast<T *>(a.vp) + page * a.vs[0] + slot * a.vs[1] +
                    (h - a.Hkv) * a.vs[2]);
            } else {
                put(reinterpret_cast<T *>(a.qo.p) + t * a.qo.st + (h - a.Hkv - nv) * a.qo.sh);
            }
        }
    }
}

// Launch over a.T tokens: jobs, rows and head slices from the sizes.
lcx_status launch_append(AppendParams &a, int es, bool half, cudaStream_t s) {
    const int vec = 16 / es;
    a.jobs = half ? (a.D / 2) / vec : a.D / vec;
    a.rows = kThreads / a.jobs;
    const int heads = a.Hkv + (a.v.p ? a.Hkv : 0) + (a.q.p ? a.Hq : 0);
    // Many tokens: a CTA of as many tokens as its threads hold walks all heads, the
    // angles evaluated once per token.  Few tokens (a decode step): the heads are cut
    // into slices of at least four until there are about eight CTAs per SM; the angles are
    // evaluated once per slice, which costs less than the walk (64 tokens, 48 heads: 18.3 us
    // walked, 6.5 in slices, 5.6 now that the first loads go out ahead of the token's place).
    const long long ctas = (a.T + a.rows - 1) / a.rows;
    const long long want = std::max<long long>(1, 8ll * device_sms() / ctas);
    a.per = int((heads + want - 1) / want);
    a.per = std::min(heads, std::max(4, (a.per + 3) / 4 * 4));
    a.slices = (heads + a.per - 1) / a.per;
    const dim3 grid{unsigned(ctas), unsigned(a.slices)};
    auto kern = es == 2 ? (half ? append_kernel<__nv_bfloat16, true> : append_kernel<__nv_bfloat16, false>)
                        : (half ? append_kernel<float, true> : append_kernel<float, false>);
    cudaError_t e = launch_dependent(kern, grid, dim3(kThreads), 0, s, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "paged_append launch failed: %s", cudaGetErrorString(e));
    return LCX_OK;
}

}  // namespace

lcx_status check_serving_rope(const lcx_rope_params *r, int64_t D, int64_t seq_len) {
    lcx_status st = check_rope_params(r);
    if (st != LCX_OK) return st;
    if (r->head_dim != D)
        return fail(LCX_ERR_UNSUPPORTED, "rope.head_dim %d: every dim of %lld must be rotated",
                    r->head_dim, (long long)D);
    if ((r->mode == LCX_ROPE_DYNAMIC_NTK || r->mode == LCX_ROPE_FACTORS) && r->seq_len <= 0 &&
        seq_len <= 0)
        return fail(LCX_ERR_INVALID_ARG,
                    "a length-dependent rope mode needs rope.seq_len (the lengths are device data)");
    return LCX_OK;
}

lcx_status rotate_packed(const lcx_rope_params *rope, int64_t seq_len, const void *x,
                         const int64_t *x_strides, void *y, const int *cu, int n,
                         int64_t T, int64_t H, int64_t D, cudaStream_t s) {
    if (T == 0) return LCX_OK;
    AppendParams a = {};
    a.k = {static_cast<char *>(const_cast<void *>(x)), x_strides[0], x_strides[1]};
    a.ko = {static_cast<char *>(y), H * D, D};
    a.cu = cu;
    a.n = n;
    a.T = int(T);
    a.Hkv = int(H);
    a.D = int(D);
    rope_freqs_unchecked(rope, effective_seq_len(rope, seq_len), a.theta, &a.ms);
    return launch_append(a, 4, rope->pairing == LCX_PAIR_HALF, s);
}

}  // namespace lcx

extern "C" lcx_status lcx_paged_append(const lcx_paged_cache *cache,
                                       const lcx_paged_append_args *g, void *stream) {
    using namespace lcx;
    clear_error();
    PagedParams p;
    lcx_status st = paged_prepare(cache, p);
    if (st != LCX_OK) return st;
    if (!g) return fail(LCX_ERR_INVALID_ARG, "args is NULL");
    if ((st = check_serving_rope(&g->rope, p.D, 0)) != LCX_OK) return st;
    if (g->n < 0 || g->T < 0 || g->Hq < 0) return fail(LCX_ERR_INVALID_ARG, "negative size");
    if (g->layer < 0 || g->layer >= p.layers)
        return fail(LCX_ERR_INVALID_ARG, "layer %lld of %d", (long long)g->layer, p.layers);
    if (g->T > (int64_t(1) << 30) || g->n > (int64_t(1) << 30) || g->Hq > 65536)
        return fail(LCX_ERR_UNSUPPORTED, "sizes too large");
    if (!g->cu_new && g->T != g->n)
        return fail(LCX_ERR_INVALID_ARG, "without cu_new every entry has one token (T = n)");
    if (!g->q != !g->q_out) return fail(LCX_ERR_INVALID_ARG, "q and q_out go together");
    if (g->T == 0 || g->n == 0) return LCX_OK;
    if (!g->seq_ids || !g->start) return fail(LCX_ERR_INVALID_ARG, "seq_ids or start is NULL");
    if ((st = check_tokens(g->k, g->k_strides, p.es, "k")) != LCX_OK) return st;
    if ((st = check_tokens(g->v, g->v_strides, p.es, "v")) != LCX_OK) return st;
    if (g->q) {
        if (g->Hq == 0) return fail(LCX_ERR_INVALID_ARG, "q without heads");
        if ((st = check_tokens(g->q, g->q_strides, p.es, "q")) != LCX_OK) return st;
        if ((st = check_tokens(g->q_out, g->q_out_strides, p.es, "q_out")) != LCX_OK) return st;
        if ((st = check_distinct(g->q_out_strides, g->T, g->Hq, "q_out")) != LCX_OK) return st;
    }
    if (g->k_out && ((st = check_tokens(g->k_out, g->k_out_strides, p.es, "k_out")) != LCX_OK ||
                     (st = check_distinct(g->k_out_strides, g->T, p.H, "k_out")) != LCX_OK))
        return st;
    for (int d = 0; d < 2; ++d)
        if ((g->q && g->q == g->q_out && g->q_strides[d] != g->q_out_strides[d]) ||
            (g->k == g->k_out && g->k_strides[d] != g->k_out_strides[d]))
            return fail(LCX_ERR_INVALID_ARG, "in-place rotation needs identical strides");
    AppendParams a = {};
    auto tensor = [](const void *ptr, const int64_t *s) {
        TokenTensor t = {static_cast<char *>(const_cast<void *>(ptr)), s[0], s[1]};
        return t;
    };
    a.k = tensor(g->k, g->k_strides);
    a.v = tensor(g->v, g->v_strides);
    a.q = tensor(g->q, g->q_strides);
    a.qo = tensor(g->q_out, g->q_out_strides);
    a.ko = tensor(g->k_out, g->k_out_strides);
    a.kp = p.k + g->layer * p.ks[0] * p.es;
    a.vp = p.v + g->layer * p.vs[0] * p.es;
    for (int d = 0; d < 3; ++d) {
        a.ks[d] = p.ks[d + 1];
        a.vs[d] = p.vs[d + 1];
    }
    a.ids = g->seq_ids;
    a.start = g->start;
    a.cu = g->cu_new;
    a.table = p.table;
    a.lens = p.lens;
    a.status = g->dev_status;
    a.n = int(g->n);
    a.T = int(g->T);
    a.Hq = int(g->Hq);
    a.Hkv = p.H;
    a.S = p.S;
    a.MP = p.MP;
    a.P = p.P;
    a.ps_log2 = p.ps_log2;
    a.D = p.D;
    rope_freqs_unchecked(&g->rope, g->rope.seq_len, a.theta, &a.ms);
    return launch_append(a, p.es, g->rope.pairing == LCX_PAIR_HALF,
                         static_cast<cudaStream_t>(stream));
}
