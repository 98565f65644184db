// attn_varlen.cu -- fused RoPE + causal attention over packed sequences of
// different lengths (lcx_attn_varlen) and the plan that lays out their work.
//
// o_i = sum_j softmax_j(c <q'_i, k'_j>) v_j over the visible keys j of the same
// sequence ("Long Context: RoPE / YaRN / NTK / MLA", 2.4, 10.1, 10.2), with a
// running maximum and sum ("8.3 长上下文技术", 8.3.4).  Keys are rotated once per
// call into scratch, queries as their tile is loaded.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "paged.cuh"
#include "rope_angle.cuh"
#include "varlen.cuh"
#include "vec16.cuh"

namespace lcx {
namespace {

// ------------------------------------------------------------------ fp32 kernel
// 64 query rows of one head per CTA, key tiles of 64, all products in fp32 on
// the FMA pipe.  Thread (ty, tx) of 16 x 16 owns rows 4 ty .. 4 ty + 3, the scores
// of keys tx + 16 j, and output columns 4 tx + 64 c.
constexpr int kRows = 64, kKeys = 64, kSimtThreads = 256;

template <int D>
struct Simt {
    static constexpr int LD = D + 4;      // padded row of a Q or K tile (floats)
    static constexpr int LP = kKeys + 4;  // padded row of the P tile
    static constexpr int kFloats = kRows * LD + kKeys * LD + kKeys * D + kRows * LP;
    static constexpr int kBytes = kFloats * 4;
};

template <typename T>
__device__ __forceinline__ void load4(const T *src, float (&x)[4]) {
    if constexpr (sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(src);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(src);
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kSimtThreads)
    varlen_simt_kernel(const __grid_constant__ VarlenParams p) {
    using C = Simt<D>;
    extern __shared__ float sm[];
    float *sq = sm, *sk = sq + kRows * C::LD, *sv = sk + kKeys * C::LD, *sp = sv + kKeys * D;
    const int h = blockIdx.x % p.Hq, uu = blockIdx.x / p.Hq;
    const VarlenUnit U = load_unit(p, uu >> 1);
    const int r0 = (uu & 1) * kRows, rows = min(kRows, U.rows - r0);
    if (rows <= 0) return;
    const int g = h / p.G, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int pos0 = U.pos0 + r0;

    // Q tile, rotated in fp32 (rows past the unit: zero)
    const T *q = reinterpret_cast<const T *>(p.q) + (long long)(U.q0 + r0) * p.qs[0] + h * p.qs[1];
    for (int i = threadIdx.x; i < kRows * (D / 2); i += kSimtThreads) {
        const int r = i / (D / 2), pr = i % (D / 2);
        const int a = p.half ? pr : 2 * pr, b = p.half ? pr + D / 2 : 2 * pr + 1;
        float x = 0.f, y = 0.f, c = 1.f, s = 0.f;
        if (r < rows) {
            x = static_cast<float>(q[(long long)r * p.qs[0] + a]);
            y = static_cast<float>(q[(long long)r * p.qs[0] + b]);
            if (p.rotate_q) rope_sincos(pos0 + r, p.theta[pr], &c, &s);
        }
        sq[r * C::LD + a] = x * c - y * s;
        sq[r * C::LD + b] = x * s + y * c;
    }
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    // keys any row of the tile sees: [0, jhi), without (sinks .. jlo) under a window
    const int last = pos0 + rows - 1;
    const int jhi = p.causal ? min(U.nk, last + 1) : U.nk;
    const int jlo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
    for (int j0 = 0; j0 < jhi; j0 += kKeys) {
        if (j0 + kKeys <= jlo && j0 >= p.sinks) continue;
        __syncthreads();
        for (int i = threadIdx.x; i < kKeys * (D / 4); i += kSimtThreads) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
            if (j0 + r < U.nk) {
                const long long row = U.k0 + j0 + r;
                load4(reinterpret_cast<const T *>(p.k) + row * p.ks[0] + g * p.ks[1] + c, x);
                load4(reinterpret_cast<const T *>(p.v) + row * p.vs[0] + g * p.vs[1] + c, y);
            }
            *reinterpret_cast<float4 *>(sk + r * C::LD + c) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(sv + r * D + c) = make_float4(y[0], y[1], y[2], y[3]);
        }
        __syncthreads();
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = *reinterpret_cast<const float4 *>(sq + (4 * ty + i) * C::LD + d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * C::LD + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                    s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                    s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                    s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pos = pos0 + 4 * ty + i;
            float mx = -INFINITY;
            bool seen[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + tx + 16 * j;
                seen[j] = key < U.nk && (!p.causal || key <= pos) &&
                          (p.window <= 0 || pos - key < p.window || key < p.sinks);
                s[i][j] = seen[j] ? s[i][j] * p.c_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o, 16));
            const float mn = fmaxf(m[i], mx);
            const float al = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn);
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = s[i][j] == -INFINITY ? 0.f : exp2f(s[i][j] - mn);
                z += w;
                // hidden weights are marked so that the product skips the value
                sp[(4 * ty + i) * C::LP + tx + 16 * j] = seen[j] ? w : -1.f;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o, 16);
            m[i] = mn;
            l[i] = l[i] * al + z;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] *= al;
        }
        __syncthreads();
#pragma unroll 2
        for (int j = 0; j < kKeys; ++j) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = sp[(4 * ty + i) * C::LP + j];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 v = *reinterpret_cast<const float4 *>(sv + j * D + 64 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (w[i] == -1.f) continue;
                    acc[i][4 * c] = fmaf(w[i], v.x, acc[i][4 * c]);
                    acc[i][4 * c + 1] = fmaf(w[i], v.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(w[i], v.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(w[i], v.w, acc[i][4 * c + 3]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        // a NaN sum (a NaN or infinite score the row does see) stays NaN
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const long long row = U.q0 + r0 + r;
        T *dst = reinterpret_cast<T *>(p.o) + row * p.os[0] + h * p.os[1];
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dst[64 * c + 4 * tx + e] = static_cast<T>(acc[i][4 * c + e] * inv);
        if (p.lse && tx == 0)
            p.lse[(long long)h * p.Tq + row] =
                l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
    }
}

template <typename T, int D>
lcx_status launch_simt(const VarlenParams &p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(varlen_simt_kernel<T, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Simt<D>::kBytes);
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "cudaFuncSetAttribute failed: %s", cudaGetErrorString(e));
    const long long grid = 2ll * p.n_units * p.Hq;
    if (grid > 0x7fffffffLL) return fail(LCX_ERR_UNSUPPORTED, "too many work units");
    varlen_simt_kernel<T, D><<<unsigned(grid), kSimtThreads, Simt<D>::kBytes, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "attn_varlen launch failed: %s", cudaGetErrorString(e));
    return LCX_OK;
}

// Sums over the sequences; false for lengths outside the limits.
bool plan_sums(const int32_t *lq, const int32_t *lk, int64_t n, lcx_varlen_info *x) {
    memset(x, 0, sizeof(*x));
    x->n_seqs = n;
    for (int64_t s = 0; s < n; ++s) {
        if (lq[s] < 0 || lk[s] < 0) return false;
        x->total_q += lq[s];
        x->total_k += lk[s];
        x->max_k = std::max<int64_t>(x->max_k, lk[s]);
        x->n_units[0] += (int64_t(lq[s]) + 127) / 128;
        x->n_units[1] += (int64_t(lq[s]) + 255) / 256;
        if (x->total_q > (1 << 30) || x->total_k > (1 << 30)) return false;
    }
    x->ints = plan_units(n, 1, x->n_units[0]) + 8 * x->n_units[1];
    return true;
}

lcx_status varlen_prepare(const lcx_varlen_args *a, VarlenParams &p, bool *noop) {
    *noop = false;
    if (!a) return fail(LCX_ERR_INVALID_ARG, "args is NULL");
    const lcx_varlen_info &I = a->info;
    lcx_status st = check_serving_rope(&a->rope, a->D, I.max_k > 0 ? I.max_k : 1);
    if (st != LCX_OK) return st;
    if (a->dtype != LCX_BF16 && a->dtype != LCX_F32)
        return fail(LCX_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    if (a->D != 64 && a->D != 128)
        return fail(LCX_ERR_UNSUPPORTED, "head_dim %lld: only 64 and 128", (long long)a->D);
    if (a->Hq <= 0 || a->Hkv <= 0 || a->Tq < 0 || a->Tk < 0)
        return fail(LCX_ERR_INVALID_ARG, "bad sizes");
    if (a->Hq % a->Hkv != 0)
        return fail(LCX_ERR_INVALID_ARG, "Hq (%lld) must be a multiple of Hkv (%lld)",
                    (long long)a->Hq, (long long)a->Hkv);
    if (a->causal != 0 && a->causal != 1) return fail(LCX_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (a->window < 0 || a->sinks < 0)
        return fail(LCX_ERR_INVALID_ARG, "window and sinks must be >= 0");
    if (!a->causal && (a->window != 0 || a->sinks != 0))
        return fail(LCX_ERR_UNSUPPORTED, "window / sinks need causal attention");
    if (a->flags & ~uint32_t(LCX_VARLEN_PREROTATED))
        return fail(LCX_ERR_INVALID_ARG, "unknown flags");
    if (a->reserved0 != 0) return fail(LCX_ERR_INVALID_ARG, "reserved0 must be 0");
    if (a->watchdog_ms < 0 || a->watchdog_ms > 60000)
        return fail(LCX_ERR_INVALID_ARG, "watchdog_ms must be in [0, 60000]");
    if (!(a->softmax_scale >= 0.f) || !std::isfinite(a->softmax_scale))
        return fail(LCX_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
    if (I.n_seqs < 0 || I.total_q < 0 || I.total_k < 0 || I.n_units[0] < 0 || I.n_units[1] < 0 ||
        I.total_q > a->Tq || I.total_k > a->Tk)
        return fail(LCX_ERR_INVALID_ARG, "the plan's rows (%lld, %lld) exceed the tensors' (%lld, %lld)",
                    (long long)I.total_q, (long long)I.total_k, (long long)a->Tq,
                    (long long)a->Tk);
    if (a->Tq > (1 << 30) || a->Tk > (1 << 30) || a->Hq > 65536 || I.n_units[0] > (1 << 24) ||
        I.n_seqs > (1 << 24))
        return fail(LCX_ERR_UNSUPPORTED, "sizes too large");
    if (I.total_q == 0) {
        *noop = true;
        return LCX_OK;
    }
    const int es = a->dtype == LCX_BF16 ? 2 : 4;
    if (!a->plan || (reinterpret_cast<uintptr_t>(a->plan) & 15))
        return fail(LCX_ERR_INVALID_ARG, "plan must be a 16-byte aligned device pointer");
    if ((st = check_tokens(a->q, a->q_strides, es, "q")) != LCX_OK) return st;
    if ((st = check_tokens(a->o, a->o_strides, es, "o")) != LCX_OK) return st;
    if (I.total_k > 0) {
        if ((st = check_tokens(a->k, a->k_strides, es, "k")) != LCX_OK) return st;
        if ((st = check_tokens(a->v, a->v_strides, es, "v")) != LCX_OK) return st;
    }
    const bool rotate = !(a->flags & LCX_VARLEN_PREROTATED) && a->rope.mode != LCX_ROPE_NONE;
    if (rotate && I.total_k > 0) {
        if (!a->k_rot || !aligned16(a->k_rot))
            return fail(LCX_ERR_INVALID_ARG, "k_rot must be a 16-byte aligned device pointer");
        const int64_t need = I.total_k * a->Hkv * a->D * es;
        if (a->k_rot_bytes < need)
            return fail(LCX_ERR_INVALID_ARG, "k_rot holds %lld bytes; %lld needed",
                        (long long)a->k_rot_bytes, (long long)need);
    }
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const char *>(a->q);
    p.k = static_cast<const char *>(rotate ? a->k_rot : a->k);
    p.v = static_cast<const char *>(a->v);
    p.o = static_cast<char *>(a->o);
    p.lse = a->lse;
    p.status = a->dev_status;
    for (int d = 0; d < 2; ++d) {
        p.qs[d] = a->q_strides[d];
        p.ks[d] = rotate ? (d ? a->D : a->Hkv * a->D) : a->k_strides[d];
        p.vs[d] = a->v_strides[d];
        p.os[d] = a->o_strides[d];
    }
    p.Tq = int(a->Tq);
    p.Tk = int(rotate ? I.total_k : a->Tk);
    p.Hq = int(a->Hq);
    p.Hkv = int(a->Hkv);
    p.G = p.Hq / p.Hkv;
    p.causal = a->causal;
    // a window of max_k or more keys hides nothing
    const int64_t big = int64_t(1) << 30;
    p.window = int(a->window >= I.max_k ? 0 : a->window);
    p.sinks = p.window > 0 ? int(std::min(a->sinks, big)) : 0;
    p.rotate_q = rotate ? 1 : 0;
    p.half = a->rope.pairing == LCX_PAIR_HALF;
    float ms = 1.f;
    rope_freqs_unchecked(&a->rope, effective_seq_len(&a->rope, std::max<int64_t>(I.max_k, 1)),
                         p.theta, &ms);
    const double scale =
        a->softmax_scale > 0.f ? double(a->softmax_scale) : 1.0 / std::sqrt(double(a->D));
    // q' is rotated without mscale (folded in here); the rotated keys carry theirs
    p.c_log2 = float(scale * (rotate ? double(ms) : 1.0) * 1.4426950408889634);
    p.timeout_ns = 1000000ull * (unsigned long long)(a->watchdog_ms > 0 ? a->watchdog_ms : 2000);
    return LCX_OK;
}

}  // namespace
}  // namespace lcx

using namespace lcx;

extern "C" int64_t lcx_varlen_plan_ints(const int32_t *lens_q, const int32_t *lens_k, int64_t n) {
    if (n < 0 || n > (1 << 24) || (n > 0 && (!lens_q || !lens_k))) return -1;
    lcx_varlen_info x;
    return plan_sums(lens_q, lens_k, n, &x) ? x.ints : -1;
}

extern "C" lcx_status lcx_varlen_plan(const int32_t *lens_q, const int32_t *lens_k, int64_t n,
                                      int32_t *plan, int64_t ints, lcx_varlen_info *info) {
    clear_error();
    if (n < 0 || (n > 0 && (!lens_q || !lens_k)) || !plan || !info)
        return fail(LCX_ERR_INVALID_ARG, "NULL array or negative count");
    if (n > (1 << 24)) return fail(LCX_ERR_UNSUPPORTED, "too many sequences");
    lcx_varlen_info x;
    if (!plan_sums(lens_q, lens_k, n, &x))
        return fail(LCX_ERR_INVALID_ARG, "lengths must be >= 0 and sum to at most 2^30");
    if (ints < x.ints)
        return fail(LCX_ERR_INVALID_ARG, "plan holds %lld int32; %lld needed", (long long)ints,
                    (long long)x.ints);
    memset(plan, 0, size_t(x.ints) * 4);
    plan[0] = kPlanMagic;
    int32_t *cu_q = plan + plan_cu_q(), *cu_k = plan + plan_cu_k(n);
    for (int64_t s = 0; s < n; ++s) {
        cu_q[s + 1] = cu_q[s] + lens_q[s];
        cu_k[s + 1] = cu_k[s] + lens_k[s];
    }
    for (int which = 0; which < 2; ++which) {
        const int h = which ? 256 : 128;
        std::vector<VarlenUnit> units;
        try {
            units.reserve(size_t(x.n_units[which]));
        } catch (const std::bad_alloc &) {
            return fail(LCX_ERR_INVALID_ARG, "out of host memory for the plan");
        }
        for (int64_t s = 0; s < n; ++s)
            for (int64_t r = 0; r < lens_q[s]; r += h) {
                VarlenUnit u = {};
                u.q0 = cu_q[s] + int(r);
                u.rows = int(std::min<int64_t>(h, lens_q[s] - r));
                u.k0 = cu_k[s];
                u.nk = lens_k[s];
                u.pos0 = lens_k[s] - lens_q[s] + int(r);
                units.push_back(u);
            }
        // Heaviest first: a causal row block's keys end at its last position.  The
        // block scheduler then packs the long blocks first and fills up with the
        // short ones.  Ties keep the packed order (neighbouring rows share keys).
        auto weight = [](const VarlenUnit &u) { return std::min(u.nk, u.pos0 + u.rows); };
        auto before = [&](const VarlenUnit &a, const VarlenUnit &b) {
            const int wa = weight(a), wb = weight(b);
            return wa != wb ? wa > wb : a.q0 < b.q0;
        };
        std::sort(units.begin(), units.end(), before);
        if (!units.empty())
            memcpy(plan + plan_units(n, which, x.n_units[0]), units.data(),
                   units.size() * sizeof(VarlenUnit));
    }
    *info = x;
    return LCX_OK;
}

extern "C" lcx_status lcx_attn_varlen(const lcx_varlen_args *a, void *stream) {
    clear_error();
    VarlenParams p;
    bool noop = false;
    lcx_status st = varlen_prepare(a, p, &noop);
    if (st != LCX_OK || noop) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.rotate_q) {
        st = rotate_packed(&a->rope, std::max<int64_t>(a->info.max_k, 1), a->k, a->k_strides,
                           a->k_rot, a->dtype, a->plan + plan_cu_k(a->info.n_seqs),
                           int(a->info.n_seqs), a->info.total_k, a->Hkv, a->D, s);
        if (st != LCX_OK) return st;
    }
    p.units = reinterpret_cast<const VarlenUnit *>(
        a->plan + plan_units(a->info.n_seqs, 0, a->info.n_units[0]));
    p.n_units = int(a->info.n_units[0]);
    if (a->dtype == LCX_BF16)
        return a->D == 128 ? launch_simt<__nv_bfloat16, 128>(p, s)
                           : launch_simt<__nv_bfloat16, 64>(p, s);
    return a->D == 128 ? launch_simt<float, 128>(p, s) : launch_simt<float, 64>(p, s);
}
