// paged_decode.cu -- attention of one new token per sequence over the paged
// key/value cache (lcx_paged_decode).
//
// o = sum_j softmax_j(c <q', k'_j>) v_j over the visible keys, evaluated with a
// running maximum and sum ("8.3 长上下文技术", 8.3.4), q' = q rotated at the
// token's position.  Bound by HBM: every visible key and value is read once.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "rope_angle.cuh"
#include "vec16.cuh"

namespace lcx {
namespace {

constexpr int kWarps = 4;
constexpr int kGB = 8;          // query heads a CTA serves

struct DecodeParams {
    const char *q;
    char *o;
    float *lse;
    const int *ids;
    int *status;
    const char *kp, *vp;        // pools at the layer
    long long ks[3], vs[3];     // pool strides: page, slot, head
    const int *table, *lens;
    long long qs[2], os[2];     // token, head
    int n, Hq, Hkv, G, hb;      // hb: head blocks of a kv head
    int S, MP, P, ps_log2;
    long long window, sinks;
    int rotate, half;
    float c_log2;               // logit scale in log2 units
    double theta[64];
};

template <typename T>
__device__ __forceinline__ float ld(const T *p) {
    return static_cast<float>(*p);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
    paged_decode_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int E = D / 32;   // dims per lane: lane, lane + 32, ..
    __shared__ float sq[kGB][D];
    __shared__ float sm[kWarps][kGB], sl[kWarps][kGB], so[kWarps][kGB][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x / (p.Hkv * p.hb), r = blockIdx.x % (p.Hkv * p.hb);
    const int kvh = r / p.hb, h0 = kvh * p.G + (r % p.hb) * kGB;
    const int nh = min(kGB, (kvh + 1) * p.G - h0);
    const int id = p.ids[e];
    int len = 0;
    if (id >= p.S) {
        if (threadIdx.x == 0) raise_status(p.status, LCX_ERR_INVALID_ARG);
    } else if (id >= 0) {
        len = p.lens[id];
        const long long most = (long long)p.MP << p.ps_log2;
        if (len < 0 || len > most) {
            if (threadIdx.x == 0) raise_status(p.status, LCX_ERR_INVALID_ARG);
            len = int(min(max((long long)len, 0ll), most));
        }
    }
    // q' of the block's heads, fp32
    for (int i = threadIdx.x; i < nh * (D / 2); i += kWarps * 32) {
        const int h = i / (D / 2), pr = i % (D / 2);
        const T *src = reinterpret_cast<const T *>(p.q) + e * p.qs[0] + (h0 + h) * p.qs[1];
        const int a = p.half ? pr : 2 * pr, b = p.half ? pr + D / 2 : 2 * pr + 1;
        float x = ld(src + a), y = ld(src + b), c = 1.f, s = 0.f;
        if (p.rotate) rope_sincos(len - 1, p.theta[pr], &c, &s);
        sq[h][a] = x * c - y * s;
        sq[h][b] = x * s + y * c;
    }
    __syncthreads();
    float m[kGB], l[kGB], acc[kGB][E];
#pragma unroll
    for (int h = 0; h < kGB; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int x = 0; x < E; ++x) acc[h][x] = 0.f;
    }
    for (int j = warp; j < len; j += kWarps) {
        if (p.window > 0 && len - 1 - j >= p.window && j >= p.sinks) continue;
        const int page = p.table[(long long)id * p.MP + (j >> p.ps_log2)];
        if (page < 0 || page >= p.P) {
            if (lane == 0) raise_status(p.status, LCX_ERR_INVALID_ARG);
            continue;
        }
        const int slot = j & ((1 << p.ps_log2) - 1);
        const T *k = reinterpret_cast<const T *>(p.kp) + page * p.ks[0] + slot * p.ks[1] +
                     kvh * p.ks[2];
        const T *v = reinterpret_cast<const T *>(p.vp) + page * p.vs[0] + slot * p.vs[1] +
                     kvh * p.vs[2];
        float kx[E], vx[E];
#pragma unroll
        for (int x = 0; x < E; ++x) {
            kx[x] = ld(k + lane + 32 * x);
            vx[x] = ld(v + lane + 32 * x);
        }
#pragma unroll
        for (int h = 0; h < kGB; ++h) {
            if (h >= nh) break;
            float d = 0.f;
#pragma unroll
            for (int x = 0; x < E; ++x) d = fmaf(sq[h][lane + 32 * x], kx[x], d);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            d *= p.c_log2;
            const float mn = fmaxf(m[h], d);
            const float al = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn);
            const float w = d == -INFINITY ? 0.f : exp2f(d - mn);
            m[h] = mn;
            l[h] = l[h] * al + w;
#pragma unroll
            for (int x = 0; x < E; ++x) acc[h][x] = acc[h][x] * al + w * vx[x];
        }
    }
#pragma unroll
    for (int h = 0; h < kGB; ++h) {
        if (h >= nh) break;
        if (lane == 0) {
            sm[warp][h] = m[h];
            sl[warp][h] = l[h];
        }
#pragma unroll
        for (int x = 0; x < E; ++x) so[warp][h][lane + 32 * x] = acc[h][x];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * D; i += kWarps * 32) {
        const int h = i / D, d = i % D;
        float mx = -INFINITY, z = 0.f, o = 0.f;
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w][h]);
        if (mx != -INFINITY)
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(sm[w][h] - mx);
                z += f * sl[w][h];
                o += f * so[w][h][d];
            }
        const float out = z == 0.f ? 0.f : o / z;   // a NaN sum stays NaN
        T *dst = reinterpret_cast<T *>(p.o) + e * p.os[0] + (h0 + h) * p.os[1];
        dst[d] = static_cast<T>(out);
        if (p.lse && d == 0)
            p.lse[(long long)e * p.Hq + h0 + h] =
                z == 0.f ? -INFINITY : (mx + log2f(z)) * 0.69314718055994531f;
    }
}

}  // namespace
}  // namespace lcx

extern "C" int64_t lcx_paged_decode_workspace_bytes(int64_t n, int64_t Hq, int64_t Hkv,
                                                    int64_t D) {
    if (n < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (D != 64 && D != 128) ||
        n > (int64_t(1) << 20) || Hq > 65536)
        return -1;
    return 0;
}

extern "C" lcx_status lcx_paged_decode(const lcx_paged_cache *cache,
                                       const lcx_paged_decode_args *g, void *workspace,
                                       int64_t workspace_bytes, void *stream) {
    using namespace lcx;
    clear_error();
    PagedParams c;
    lcx_status st = paged_prepare(cache, c);
    if (st != LCX_OK) return st;
    if (!g) return fail(LCX_ERR_INVALID_ARG, "args is NULL");
    if ((st = check_serving_rope(&g->rope, c.D, 0)) != LCX_OK) return st;
    if (g->n < 0 || g->Hq <= 0) return fail(LCX_ERR_INVALID_ARG, "bad sizes");
    if (g->Hq % c.H != 0)
        return fail(LCX_ERR_INVALID_ARG, "Hq (%lld) must be a multiple of Hkv (%d)",
                    (long long)g->Hq, c.H);
    if (g->layer < 0 || g->layer >= c.layers)
        return fail(LCX_ERR_INVALID_ARG, "layer %lld of %d", (long long)g->layer, c.layers);
    if (g->window < 0 || g->sinks < 0)
        return fail(LCX_ERR_INVALID_ARG, "window and sinks must be >= 0");
    if (!(g->softmax_scale >= 0.f) || !std::isfinite(g->softmax_scale))
        return fail(LCX_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
    if (g->flags & ~uint32_t(LCX_DECODE_PREROTATED))
        return fail(LCX_ERR_INVALID_ARG, "unknown flags");
    const int64_t need = lcx_paged_decode_workspace_bytes(g->n, g->Hq, c.H, c.D);
    if (need < 0) return fail(LCX_ERR_UNSUPPORTED, "sizes too large");
    if (g->n == 0) return LCX_OK;
    if (!g->seq_ids) return fail(LCX_ERR_INVALID_ARG, "seq_ids is NULL");
    if ((st = check_tokens(g->q, g->q_strides, c.es, "q")) != LCX_OK) return st;
    if ((st = check_tokens(g->o, g->o_strides, c.es, "o")) != LCX_OK) return st;
    if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return fail(LCX_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < need)
        return fail(LCX_ERR_INVALID_ARG, "workspace holds %lld bytes; %lld needed",
                    (long long)workspace_bytes, (long long)need);
    DecodeParams p = {};
    p.q = static_cast<const char *>(g->q);
    p.o = static_cast<char *>(g->o);
    p.lse = g->lse;
    p.ids = g->seq_ids;
    p.status = g->dev_status;
    p.kp = c.k + g->layer * c.ks[0] * c.es;
    p.vp = c.v + g->layer * c.vs[0] * c.es;
    for (int d = 0; d < 3; ++d) {
        p.ks[d] = c.ks[d + 1];
        p.vs[d] = c.vs[d + 1];
    }
    p.table = c.table;
    p.lens = c.lens;
    for (int d = 0; d < 2; ++d) {
        p.qs[d] = g->q_strides[d];
        p.os[d] = g->o_strides[d];
    }
    p.n = int(g->n);
    p.Hq = int(g->Hq);
    p.Hkv = c.H;
    p.G = p.Hq / p.Hkv;
    p.hb = (p.G + kGB - 1) / kGB;
    p.S = c.S;
    p.MP = c.MP;
    p.P = c.P;
    p.ps_log2 = c.ps_log2;
    p.window = g->window;
    p.sinks = g->sinks;
    p.rotate = (g->flags & LCX_DECODE_PREROTATED) || g->rope.mode == LCX_ROPE_NONE ? 0 : 1;
    p.half = g->rope.pairing == LCX_PAIR_HALF;
    float ms = 1.f;
    rope_freqs_unchecked(&g->rope, g->rope.seq_len, p.theta, &ms);
    const double scale =
        g->softmax_scale > 0.f ? double(g->softmax_scale) : 1.0 / std::sqrt(double(c.D));
    p.c_log2 = float(scale * (p.rotate ? double(ms) : 1.0) * 1.4426950408889634);
    const long long grid = (long long)p.n * p.Hkv * p.hb;
    if (grid > 0x7fffffffLL) return fail(LCX_ERR_UNSUPPORTED, "sizes too large");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned gr = unsigned(grid);
    if (c.es == 2)
        c.D == 128 ? paged_decode_kernel<__nv_bfloat16, 128><<<gr, kWarps * 32, 0, s>>>(p)
                   : paged_decode_kernel<__nv_bfloat16, 64><<<gr, kWarps * 32, 0, s>>>(p);
    else
        c.D == 128 ? paged_decode_kernel<float, 128><<<gr, kWarps * 32, 0, s>>>(p)
                   : paged_decode_kernel<float, 64><<<gr, kWarps * 32, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "paged_decode launch failed: %s", cudaGetErrorString(e));
    return LCX_OK;
}
