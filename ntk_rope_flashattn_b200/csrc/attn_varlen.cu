// attn_varlen.cu -- fused RoPE + causal attention over packed sequences of
// different lengths (lcx_attn_varlen) and the plan that lays out their work.
//
// o_i = sum_j softmax_j(c <q'_i, k'_j>) v_j over the visible keys j of the same
// sequence ("Long Context: RoPE / YaRN / NTK / MLA", 2.4, 10.1, 10.2), with a
// running maximum and sum ("8.3 长上下文技术", 8.3.4).
//
// bf16: the tcgen05 kernel described here; fp32: the kernel of tf32 products below.
//
// The tcgen05 kernel has a floor of 4 D flops per visible pair and query head on the
// tensor core and, as much again, 128 x 128 exponentials per query and key tile; a
// tile of scores goes through both in turn.  Measured: 4.2k cycles per key tile (2048
// of tensor-core work) and 14-16k per CTA outside of the key loop, the query's copy,
// rotation and the output.  16384 tokens of 32 heads: 1030 TFLOP/s (2.1 ms); 12
// prompts of 200 to 4100: 600 TFLOP/s (384 us); 8 x 2048: 670.  (Persistent CTAs whose
// helpers rotate the next block's queries meanwhile: 560-612 us where this takes 410.
// The rotation's warps take issue slots from the softmax: 4.7-5.8k cycles per tile.)
// One CTA per (row block of the plan, pair of query heads), 16 warps:
//   warps 0-3, 4-7  rotate the query tiles, then softmax of query tile 0, 1: one
//                   thread per row
//   warps 8-11      helpers: rotate along; clean the value tiles at a border
//   warp 12 / 14    TMA producers of Q and K / of V;  warp 13  MMA issuer
//   warp 15         looks whether keys are scaled
// Both tiles multiply the same key tiles, so a K/V tile is loaded once for 256
// query rows, and one tile's softmax overlaps the other's products (order PV0(j),
// S0(j + 1), PV1(j), S1(j + 1)).  With an odd group the two tiles are consecutive
// row blocks of one head.
//
// Operands of QK^T.  Rotated values are not bf16 numbers, and a logit's rounding
// error reaches lse unweakened when a row sees few keys.  q' and k' are therefore
// fp16 (11 bits instead of 8, the same tensor-core rate), each row scaled by a power
// of two when its largest value leaves [2^-6, 2^14) (a query's power goes into c; scaled
// keys, rare, take a slower path), and row blocks that start before position 127, or
// see fewer keys, add the products with the operands' fp16 remainders ("precise":
// their few key tiles cost three products instead of one).  Given rotated inputs
// are bf16 already and enter as they are.
//
// Values at a border.  P is zero where a key is hidden, but zero times an infinite or
// NaN value is NaN, and a tile's last rows may belong to the next sequence.  For the
// tiles that some row does not see completely the helpers clear rows behind the
// sequence and non-finite values before the product, and the rows that do see such a
// value add it at the end.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include <cuda.h>

#include "mma_sync.cuh"
#include "paged.cuh"
#include "rope_angle.cuh"
#include "sm100.cuh"
#include "varlen.cuh"
#include "vec16.cuh"

namespace lcx {
namespace {

// ------------------------------------------------------------------ fp32 kernel
// 64 query rows of one head per CTA, key tiles of 64, 8 warps: warp w has rows
// 16 (w % 4) .. + 15 and, with half = w / 4, the scores of 32 keys and half of the
// output's columns.  Both products are tf32 matrix instructions on two parts of every
// operand, each part a cut of the value (hi + lo within 2^-21 of it): lo hi + hi lo +
// hi hi, three instructions and still above the FMA pipe's rate (254 / 3 against 74
// TFLOP/s).  The matrix instructions cut their sums, so the small products have sums of
// their own and the weighted values of a tile are summed apart and added to the row's
// in fp32.
//
// Fragments come 16 bytes at a time: the sums over d and over keys may take them in any
// order, and a lane's four neighbouring values serve two instructions of Q K^T (d) or
// four column tiles of P V (the columns of a tile are 4 apart).  The scores' own layout
// then is P's operand layout.  One buffer each for K and V: a value tile loads during
// Q K^T, the next key tile during P V.  Two CTAs, 16 warps, per SM: bound by the issue
// of the parts' arithmetic and its latency (four warps of twice the work each: 12 %
// slower, at small sizes 40 %).  4 x 1024 tokens, 32 heads of 128: 745 us, 46 TFLOP/s
// (fp32 products on the FMA pipe: 1075 us).
constexpr int kRows = 64, kKeys = 64, kF32Threads = 256;

template <int D>
struct F32 {
    static constexpr int kCtas = 2;                         // per SM
    static constexpr int CPR = D / 4;                       // 16-byte chunks per row
    static constexpr int kBytes = ((kRows + 2 * kKeys) * D + kRows * kKeys) * 4;
};

// Float offset of chunk c of row r: rows of Q and K are read two at a time, four
// chunks each, rows of V in pairs, four pairs by two chunks, without bank conflicts.
template <int D>
__device__ __forceinline__ int at_qk(int r, int c) {
    return r * D + ((c ^ ((r & 1) << 2)) << 2);
}
template <int D>
__device__ __forceinline__ int at_v(int r, int c) {
    return r * D + ((c ^ (((r >> 1) & 3) << 1)) << 2);
}

template <int D>
__global__ void __launch_bounds__(kF32Threads, F32<D>::kCtas)
    varlen_f32_kernel(const __grid_constant__ VarlenParams p) {
    constexpr int CPR = F32<D>::CPR;
    extern __shared__ __align__(16) float sm[];
    __shared__ float row_part[2][kRows];            // of each half: maxima, at the end sums
    float *sq = sm, *sk = sq + kRows * D, *sv = sk + kKeys * D;
    const int h = blockIdx.x % p.Hq, uu = blockIdx.x / p.Hq;
    const VarlenUnit U = load_unit(p, uu >> 1);
    const int r0 = (uu & 1) * kRows, rows = min(kRows, U.rows - r0);
    if (rows <= 0) {
        // (a plan that does not fit the tensors, or a block of up to kRows rows: no second half)
        if (U.rows <= 0 && threadIdx.x == 0) raise_status(p.status, LCX_ERR_INVALID_ARG);
        wait_previous_kernel();      // what follows in the stream may write k
        return;
    }
    const int g = h / p.G, lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    const int half = threadIdx.x >> 7, t = lane & 3, rl = lane >> 2;
    const int pos0 = U.pos0 + r0;

    // Q tile, rotated in fp32 (rows past the unit: zero)
    const float *q = reinterpret_cast<const float *>(p.q) + (long long)(U.q0 + r0) * p.qs[0] +
                     h * p.qs[1];
    for (int i = threadIdx.x; i < kRows * (D / 2); i += kF32Threads) {
        const int r = i / (D / 2), pr = i % (D / 2);
        const int a = p.half ? pr : 2 * pr, b = p.half ? pr + D / 2 : 2 * pr + 1;
        float x = 0.f, y = 0.f, c = 1.f, s = 0.f;
        if (r < rows) {
            x = q[(long long)r * p.qs[0] + a];
            y = q[(long long)r * p.qs[0] + b];
            if (p.rotate_q) rope_sincos(pos0 + r, p.theta[pr], &c, &s);
        }
        sq[at_qk<D>(r, a >> 2) + (a & 3)] = x * c - y * s;
        sq[at_qk<D>(r, b >> 2) + (b & 3)] = x * s + y * c;
    }
    wait_previous_kernel();          // the rotated keys

    // keys any row of the tile sees: [0, jhi), without (sinks .. jlo) under a window
    const int last = pos0 + rows - 1;
    const int jhi = p.causal ? min(U.nk, last + 1) : U.nk;
    const int jlo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
    auto seen_from = [&](int j) {    // the first tile from j on that is not hidden
        return j + kKeys <= jlo && j >= p.sinks ? jlo / kKeys * kKeys : j;
    };
    const float *kb = reinterpret_cast<const float *>(p.k) + U.k0 * p.ks[0] + g * p.ks[1];
    const float *vb = reinterpret_cast<const float *>(p.v) + U.k0 * p.vs[0] + g * p.vs[1];
    // (a thread copies chunk threadIdx % CPR of every kStep-th row; rows behind the
    // sequence read zero)
    constexpr int kStep = kF32Threads / CPR;
    const int cc = threadIdx.x % CPR, cr = threadIdx.x / CPR;
    auto copy = [&](float *dst, const float *src, long long stride, int j0, bool value) {
#pragma unroll
        for (int i = 0; i < kKeys; i += kStep) {
            const int r = cr + i, row = min(j0 + r, U.nk - 1);
            cp_async16(smem_u32(dst + (value ? at_v<D>(r, cc) : at_qk<D>(r, cc))),
                       src + row * stride + cc * 4, j0 + r < U.nk ? 16 : 0);
        }
    };

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // rows rl, rl + 8 of the warp
    float acc[D / 16][4];  // tile 4 G + e: columns half D/2 + 32 G + 4 (2 t + {0, 1}) + e
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
    const int wrow = warp * 16 + rl, pos = pos0 + wrow;
    const float *qa = sq + wrow * D;
    // the lane's weights, in P's operand layout: eight keys a chunk
    float4 *sp = reinterpret_cast<float4 *>(sv + kKeys * D) + warp * (kKeys / 8) * 32 + lane;
    constexpr int kN = kKeys / 16;   // score tiles of a warp

    int j0 = seen_from(0);
    if (j0 < jhi) copy(sk, kb, p.ks[0], j0, false);
    cp_async_commit();
    while (j0 < jhi) {
        cp_async_wait<0>();
        __syncthreads();             // the keys are there; the last values are read
        copy(sv, vb, p.vs[0], j0, true);
        cp_async_commit();
        float s[kN][4], low[kN][4];  // (rl, rl + 8) x keys 32 half + 8 n + 2 t + {0, 1}
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[n][c] = low[n][c] = 0.f;
        // (not unrolled, here and over the keys below: the code of a key tile then stays
        // in the instruction cache)
#pragma unroll 1
        for (int i = 0; i < D / 16; ++i) {
            const int o = ((4 * i + t) ^ ((rl & 1) << 2)) << 2;
            const float4 x = *reinterpret_cast<const float4 *>(qa + o);
            const float4 y = *reinterpret_cast<const float4 *>(qa + 8 * D + o);
            uint32_t u[kN][4], w[kN][4];
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const float4 k = *reinterpret_cast<const float4 *>(
                    sk + (half * (kKeys / 2) + 8 * n + rl) * D + o);
                tf32_parts(k.x, u[n][0], w[n][0]);
                tf32_parts(k.y, u[n][1], w[n][1]);
                tf32_parts(k.z, u[n][2], w[n][2]);
                tf32_parts(k.w, u[n][3], w[n][3]);
            }
            uint32_t a0[4], b0[4], a1[4], b1[4];
            tf32_parts(x.x, a0[0], b0[0]);
            tf32_parts(y.x, a0[1], b0[1]);
            tf32_parts(x.y, a0[2], b0[2]);
            tf32_parts(y.y, a0[3], b0[3]);
            tf32_parts(x.z, a1[0], b1[0]);
            tf32_parts(y.z, a1[1], b1[1]);
            tf32_parts(x.w, a1[2], b1[2]);
            tf32_parts(y.w, a1[3], b1[3]);
            // (products of one sum stand four and more instructions apart)
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_tf32(low[n], a0, w[n][0], w[n][1]);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_tf32(s[n], a0, u[n][0], u[n][1]);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_tf32(low[n], b0, u[n][0], u[n][1]);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_tf32(s[n], a1, u[n][2], u[n][3]);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_tf32(low[n], a1, w[n][2], w[n][3]);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_tf32(low[n], b1, u[n][2], u[n][3]);
        }
        auto sees = [&](int key, int at) {
            return key < U.nk && (!p.causal || key <= at) &&
                   (p.window <= 0 || at - key < p.window || key < p.sinks);
        };
        const int end = j0 + kKeys - 1, key0 = j0 + half * (kKeys / 2) + 2 * t;
        const bool whole = end < U.nk && (!p.causal || end <= pos0) &&
                           (p.window <= 0 || last - j0 < p.window || end < p.sinks);
        float mx[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = -INFINITY;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[n][2 * r + e];
                    x = whole || sees(key0 + 8 * n + e, pos + 8 * r)
                            ? join(x, low[n][2 * r + e]) * p.c_log2
                            : -INFINITY;
                    mx[r] = fmaxf(mx[r], x);
                }
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            if (t == 0) row_part[half][wrow + 8 * r] = mx[r];
        }
        const int j1 = seen_from(j0 + kKeys);
        __syncthreads();             // both halves' maxima are there, the keys are read
        if (j1 < jhi) copy(sk, kb, p.ks[0], j1, false);
        cp_async_commit();
        float al[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float mn = fmaxf(m[r], fmaxf(mx[r], row_part[half ^ 1][wrow + 8 * r]));
            al[r] = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mn);
            const float ref = mn == -INFINITY ? 0.f : mn;
            float z = 0.f;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[n][2 * r + e];
                    x = exp2f(x - ref);
                    z += x;
                }
            m[r] = mn;
            l[r] = l[r] * al[r] + z;
        }
#pragma unroll
        for (int n = 0; n < kN; ++n)
            sp[(half * kN + n) * 32] = make_float4(s[n][0], s[n][2], s[n][1], s[n][3]);
        cp_async_wait<1>();
        // An infinite or NaN value would reach rows that do not see it, by 0 x: a tile
        // that holds one is cleared of it, and the rows that see it add it.
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < kKeys; i += kStep) {
            const float4 x = *reinterpret_cast<const float4 *>(sv + at_v<D>(cr + i, cc));
            z += 0.f * x.x + 0.f * x.y + 0.f * x.z + 0.f * x.w;
        }
        const bool bad = __syncthreads_or(z != 0.f);   // values and weights are there
        if (bad) {
#pragma unroll 1
            for (int i = 0; i < kKeys; i += kStep) {
                float4 &x = *reinterpret_cast<float4 *>(sv + at_v<D>(cr + i, cc));
                x.x = fabsf(x.x) < INFINITY ? x.x : 0.f;
                x.y = fabsf(x.y) < INFINITY ? x.y : 0.f;
                x.z = fabsf(x.z) < INFINITY ? x.z : 0.f;
                x.w = fabsf(x.w) < INFINITY ? x.w : 0.f;
            }
            __syncthreads();
        }
#pragma unroll
        for (int G = 0; G < D / 64; ++G) {
            float o[4][4], low[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[e][c] = low[e][c] = 0.f;
            const float *vr = sv + 2 * t * D + (((half * CPR / 2 + 8 * G + rl) ^ (2 * t)) << 2);
#pragma unroll 2
            for (int n = 0; n < kKeys / 8; ++n) {
                const float4 w = sp[n * 32];
                const float4 x = *reinterpret_cast<const float4 *>(vr + 8 * n * D);
                const float4 y = *reinterpret_cast<const float4 *>(vr + 8 * n * D + D);
                uint32_t a[4], b[4];
                tf32_parts(w.x, a[0], b[0]);
                tf32_parts(w.y, a[1], b[1]);
                tf32_parts(w.z, a[2], b[2]);
                tf32_parts(w.w, a[3], b[3]);
                const float v0[4] = {x.x, x.y, x.z, x.w}, v1[4] = {y.x, y.y, y.z, y.w};
                uint32_t u0[4], w0[4], u1[4], w1[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    tf32_parts(v0[e], u0[e], w0[e]);
                    tf32_parts(v1[e], u1[e], w1[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_tf32(low[e], a, w0[e], w1[e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_tf32(o[e], a, u0[e], u1[e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_tf32(low[e], b, u0[e], u1[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[4 * G + e][c] =
                        fmaf(acc[4 * G + e][c], al[c >> 1], o[e][c] + low[e][c]);
        }
        if (bad) {
#pragma unroll 1
            for (int r = 0; r < min(kKeys, U.nk - j0); ++r)
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float x = vb[(j0 + r) * p.vs[0] + half * (D / 2) + 32 * (i / 4) +
                                           4 * (2 * t + c) + i % 4];
                        if (fabsf(x) < INFINITY) continue;
                        if (sees(j0 + r, pos)) acc[i][c] += x;
                        if (sees(j0 + r, pos + 8)) acc[i][2 + c] += x;
                    }
        }
        j0 = j1;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t == 0) row_part[half][wrow + 8 * r] = l[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int i = wrow + 8 * r;
        if (i >= rows) continue;
        const float z = row_part[0][i] + row_part[1][i];
        // a NaN sum (a NaN or infinite score the row does see) stays NaN
        const float inv = z == 0.f ? 0.f : 1.f / z;
        const long long row = U.q0 + r0 + i;
        float *dst = reinterpret_cast<float *>(p.o) + row * p.os[0] + h * p.os[1] +
                     half * (D / 2) + 8 * t;
#pragma unroll
        for (int G = 0; G < D / 64; ++G)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<float4 *>(dst + 32 * G + 4 * c) = make_float4(
                    acc[4 * G][2 * r + c] * inv, acc[4 * G + 1][2 * r + c] * inv,
                    acc[4 * G + 2][2 * r + c] * inv, acc[4 * G + 3][2 * r + c] * inv);
        if (p.lse && t == 0 && half == 0)
            p.lse[(long long)h * p.Tq + row] =
                z == 0.f ? -INFINITY : (m[r] + log2f(z)) * 0.69314718055994531f;
    }
}

template <int D>
lcx_status launch_f32(const VarlenParams &p, bool after_keys, cudaStream_t s) {
    auto kern = varlen_f32_kernel<D>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F32<D>::kBytes);
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "cudaFuncSetAttribute failed: %s", cudaGetErrorString(e));
    const long long grid = 2ll * p.n_units * p.Hq;
    if (grid > 0x7fffffffLL) return fail(LCX_ERR_UNSUPPORTED, "too many work units");
    if (after_keys)
        e = launch_dependent(kern, dim3(unsigned(grid)), dim3(kF32Threads), F32<D>::kBytes, s, p);
    else
        kern<<<unsigned(grid), kF32Threads, F32<D>::kBytes, s>>>(p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "attn_varlen launch failed: %s", cudaGetErrorString(e));
    return LCX_OK;
}

// ------------------------------------------------------------------ key rotation
// The rotated keys as the tcgen05 kernel reads them: fp16 parts hi [T][Hkv][D],
// remainders lo alike (rows before kLoRows, all of them with all_lo), one scale per
// row (k' = scale (hi + lo)), and per CTA whether any scale is not 1.
constexpr int kLoRows = 384;   // a precise block's keys: positions below 127 + 256

struct KeyParams {
    const __nv_bfloat16 *k;
    long long st, sh;              // element strides: token, head
    __half *hi, *lo;
    float *scale;
    int *flags;
    const int *cu;                 // first row of each sequence, n + 1
    int n, T, H, all_lo;
    float ms;
    double theta[64];
};

// The power of two that brings amax to [2^13, 2^14) when it leaves [2^-6, 2^14), else 1;
// *undo its reciprocal.  (fp16 keeps 11 bits down to 2^-14 and steps of 2^-24 below: the
// top of its range leaves most room for a row's small values.  fp32 and bf16 values reach
// from 2^-133 to 2^128: powers up to 2^125, so that both are normal numbers.)
__device__ __forceinline__ float range_scale(float amax, float *undo) {
    *undo = 1.f;
    if ((amax >= 0.015625f && amax < 16384.f) || amax == 0.f || !(amax < INFINITY)) return 1.f;
    const int e = max(int(__float_as_uint(amax) >> 23) - 127 - 13, -125);
    *undo = __uint_as_float(uint32_t(127 + e) << 23);
    return __uint_as_float(uint32_t(127 - e) << 23);
}

// 8 values as fp16 parts, and the remainders of such parts.
__device__ __forceinline__ uint4 half_parts(const float (&y)[8]) {
    return make_uint4(pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3]), pack_f16x2(y[4], y[5]),
                      pack_f16x2(y[6], y[7]));
}
__device__ __forceinline__ uint4 half_rest(const float (&y)[8], const uint4 &hi) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
    uint32_t l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = f16x2_to_f32x2(h[e]);
        float a = y[2 * e] - f.x, b = y[2 * e + 1] - f.y;
        a = a == a ? a : 0.f;                 // an infinite value has no remainder
        b = b == b ? b : 0.f;
        l[e] = pack_f16x2(a, b);
    }
    return make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ float abs_max8(const float (&x)[8]) {
    const float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    const float b = fmaxf(fmaxf(fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7])));
    return fmaxf(a, b);
}

// The same of 8 packed fp16 values.
__device__ __forceinline__ float packed_max(const uint4 &h) {
    const __half2 *v = reinterpret_cast<const __half2 *>(&h);
    const __half2 a = __hmax2(__hmax2(__habs2(v[0]), __habs2(v[1])),
                              __hmax2(__habs2(v[2]), __habs2(v[3])));
    return fmaxf(__low2float(a), __high2float(a));
}

// Rotate the pairs of one job: HALF pairs x1[e], x2[e] with angle e; else adjacent
// pairs of x1 with angle e (x2 unused).
template <bool kHalf>
__device__ __forceinline__ void turn(float (&x1)[8], float (&x2)[8], const float *c,
                                     const float *s) {
    if constexpr (kHalf) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 a = make_float2(x1[e], x1[e + 1]), b = make_float2(x2[e], x2[e + 1]);
            const float2 cc = make_float2(c[e], c[e + 1]), ss = make_float2(s[e], s[e + 1]);
            const float2 y1 = fma2(b, make_float2(-ss.x, -ss.y), mul2(a, cc));
            const float2 y2 = fma2(a, ss, mul2(b, cc));
            x1[e] = y1.x; x1[e + 1] = y1.y;
            x2[e] = y2.x; x2[e + 1] = y2.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = x1[2 * e], b = x1[2 * e + 1];
            x1[2 * e] = fmaf(-b, s[e], a * c[e]);
            x1[2 * e + 1] = fmaf(b, c[e], a * s[e]);
        }
    }
}

constexpr int kKeyThreads = 256;

template <int D, bool kHalf>
struct Job {
    static constexpr int CPR = kHalf ? D / 16 : D / 8;   // jobs (lanes) per row
    static constexpr int PPJ = kHalf ? 8 : 4;            // pairs per job
};

template <int D, bool kHalf>
__global__ void __launch_bounds__(kKeyThreads)
    varlen_keys_kernel(const __grid_constant__ KeyParams p) {
    using J = Job<D, kHalf>;
    constexpr int RPC = kKeyThreads / J::CPR;            // tokens per CTA
    __shared__ int pos_of[RPC];
    __shared__ int scaled;
    wait_previous_kernel();
    pdl_launch_dependents();
    const int t0 = blockIdx.x * RPC;
    if (threadIdx.x == 0) scaled = 0;
    if (threadIdx.x < RPC) {
        const int t = t0 + threadIdx.x;
        int lo = 0, hi = p.n;                            // cu[lo] <= t < cu[hi]
        if (t < p.T) {
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.cu[mid] <= t) lo = mid; else hi = mid;
            }
            pos_of[threadIdx.x] = t - p.cu[lo];
        }
    }
    __syncthreads();
    const int q = threadIdx.x % J::CPR, row = threadIdx.x / J::CPR, t = t0 + row;
    const bool in = t < p.T;                             // whole lane groups agree
    const int pos = in ? pos_of[row] : 0;
    float c[J::PPJ], s[J::PPJ];
#pragma unroll
    for (int e = 0; e < J::PPJ; ++e) {
        rope_sincos(pos, p.theta[q * J::PPJ + e], &c[e], &s[e]);
        c[e] *= p.ms;
        s[e] *= p.ms;
    }
    const int e1 = q * 8, e2 = e1 + D / 2;
    const bool want_lo = p.all_lo || pos < kLoRows;
    bool any = false;
    constexpr int kHB = 4;
    for (int b = 0; b < p.H; b += kHB) {
        uint4 va[kHB], vb[kHB];
#pragma unroll
        for (int u = 0; u < kHB; ++u) {
            va[u] = vb[u] = make_uint4(0, 0, 0, 0);
            if (in && b + u < p.H) {
                const __nv_bfloat16 *src = p.k + t * p.st + (b + u) * p.sh;
                va[u] = __ldcs(reinterpret_cast<const uint4 *>(src + e1));
                if (kHalf) vb[u] = __ldcs(reinterpret_cast<const uint4 *>(src + e2));
            }
        }
#pragma unroll
        for (int u = 0; u < kHB; ++u) {
            float x1[8], x2[8];
            unpack(va[u], x1);
            unpack(vb[u], x2);
            turn<kHalf>(x1, x2, c, s);
            float mx = kHalf ? fmaxf(abs_max8(x1), abs_max8(x2)) : abs_max8(x1);
#pragma unroll
            for (int o = 1; o < J::CPR; o <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            float undo;
            const float f = range_scale(mx, &undo);
            if (undo != 1.f) {
                any = true;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x1[e] *= f;
                    x2[e] *= f;
                }
            }
            if (!in || b + u >= p.H) continue;
            const long long at = ((long long)t * p.H + b + u) * D;
            const uint4 h1 = half_parts(x1);
            *reinterpret_cast<uint4 *>(p.hi + at + e1) = h1;
            if (want_lo) *reinterpret_cast<uint4 *>(p.lo + at + e1) = half_rest(x1, h1);
            if (kHalf) {
                const uint4 h2 = half_parts(x2);
                *reinterpret_cast<uint4 *>(p.hi + at + e2) = h2;
                if (want_lo) *reinterpret_cast<uint4 *>(p.lo + at + e2) = half_rest(x2, h2);
            }
            if (q == 0) p.scale[(long long)t * p.H + b + u] = undo;
        }
    }
    if (any) scaled = 1;
    __syncthreads();
    if (threadIdx.x == 0) p.flags[blockIdx.x] = scaled;
}

// ------------------------------------------------------------------ tcgen05 kernel
constexpr int kThreads = 512, kBM = 128, kBN = 128;
constexpr int kRotThreads = 384;    // warps 0-11 rotate the queries
// registers a thread after the warpgroups re-balance: 176 + 176 + 96 + 64 = 4 x 128
constexpr int kRegsSoftmax = 176, kRegsHelp = 96, kRegsIssue = 64;
static_assert(2 * kRegsSoftmax + kRegsHelp + kRegsIssue == 4 * 128, "register file split");
constexpr int kWarpHelp = 8, kWarpTma = 12, kWarpMma = 13, kWarpTmaV = 14, kWarpFlags = 15;
constexpr float kLazy = 15.f;       // log2 growth of a row's maximum that rescales O
constexpr int kMaxBorder = 8;       // border tiles whose non-finite rows are listed

enum Mode { kTwoHeads = 0, kTwoBlocks = 1, kOneTile = 2 };

struct TcParams {
    VarlenParams v;
    const float *k_scale;           // [Tk][Hkv], or NULL: no key is scaled
    const int *k_flags;             // per CTA of the key rotation
    int flag_rows;                  // tokens of such a CTA
    int mode, fp16;                 // fp16: rotated operands; 0: bf16 inputs as they are
    int group_units;                // CTAs per row block and kv head
    int by_head;                    // order of the CTAs (load_block)
    int stall;                      // the producers issue nothing (watchdog test hook)
    float2 step[64];                // cos, sin of the angle between a thread's rows
};

template <int D>
struct Tc {
    static constexpr int kTile = 128 * D * 2;            // a Q, K or V tile
    static constexpr int kBox = 128 * 128;               // its 64-column boxes
    static constexpr int NS = D == 64 ? 4 : 2;           // K stages, and V stages
    static constexpr int kOffK = 2 * kTile;
    static constexpr int kOffV = kOffK + NS * kTile;
    // precise blocks: keys' parts in K stages 0 and 1, values in V stage 0, the query
    // tiles' remainders in V stage 1 and the next 32 KB
    static constexpr int kOffQLo = kOffV + kTile;
    static constexpr int kOffBar = kOffV + NS * kTile + (D == 64 ? 0 : kTile);
    static constexpr int kSmem = kOffBar + 2048 + 1024;  // barriers; alignment slack
    static_assert(kSmem <= 232448, "shared memory budget");
    static constexpr int kColO = 2 * kBN;                // TMEM: S_0, S_1, O_0, O_1
    static_assert(kColO + 2 * D <= 512, "TMEM budget");
};


// The key tiles that rows at positions i0 .. i1 see whole: [0, sf) (sinks) and
// [jl, je).  The others that they visit are border tiles.
struct Full {
    int sf, jl, je;
    __device__ __forceinline__ void set(const VarlenParams &v, int i0, int i1, int nk) {
        const int lim = v.causal ? min(nk - 1, i0) : nk - 1;     // last key all rows see
        je = lim < 0 ? 0 : (lim + 1) / kBN;
        jl = 0;
        sf = 0;
        if (v.window > 0) {
            jl = max(0, i1 - v.window + 1 + kBN - 1) / kBN;
            sf = min(v.sinks / kBN, je);
        }
    }
    __device__ __forceinline__ bool has(int jt) const { return jt < sf || (jt >= jl && jt < je); }
};

// A CTA's work: the row block, its two tiles and the key tiles it visits.
struct Block {
    VarlenUnit u;
    int g, h0, nt, hstep, rstep;    // tile t: head h0 + t hstep, rows from t rstep on
    int ns, jlo, n;                 // key tiles: sink tiles [0, ns), then from jlo on
    Full full;                      // key tiles that every row of the block sees whole
    bool precise;
    __device__ __forceinline__ int tile(int j) const { return j < ns ? j : jlo + (j - ns); }
    __device__ __forceinline__ int pos(int t) const { return u.pos0 + t * rstep; }
    __device__ __forceinline__ int rows(int t) const { return min(kBM, u.rows - t * rstep); }
};

template <int D>
struct Bars {
    static constexpr int NS = Tc<D>::NS;
    Block block;
    Full own[2];                    // tiles that a query tile's own rows see whole
    uint64_t full_q, ready_q, full_k[NS], empty_k[NS], full_v[NS], full_b[NS], clean_v[NS], empty_v[NS];
    uint64_t s_ready[2], p_ready[2], o_ready[2], helped, drain;
    uint32_t tmem_base;
    int abort, k_scaled, n_border, any_bad;
    int border_tile[kMaxBorder];
    uint32_t bad[kMaxBorder][4];    // rows of a border tile with non-finite values
    signed char q_exp[2 * kBM];     // exponents of the query rows' scales
    // per pair (pair e of job q at e CPR + q: a warp's lanes read neighbours), for the
    // query rotation (lanes read different entries, which the
    // parameter space would serve one after the other): the angle of the block's first
    // position and theta (in two fp32 parts) reduced to [-pi, pi], cos and sin of the step
    float base[D / 2];
    float2 theta[D / 2], step[D / 2];
};

__device__ __forceinline__ Block load_block(const TcParams &p) {
    Block b;
    const VarlenParams &v = p.v;
    const int per = v.n_units * p.group_units, all = p.group_units * v.Hkv;
    int g, r;
    if (p.by_head) {            // kv head, row block (heaviest first), the group's heads
        g = int(blockIdx.x) / per;
        r = int(blockIdx.x) % per;
        b.u = load_unit(v, r / p.group_units);
    } else {                    // row block, kv head, the group's heads
        r = int(blockIdx.x) % all;
        g = r / p.group_units;
        b.u = load_unit(v, int(blockIdx.x) / all);
    }
    b.g = g;
    b.hstep = b.rstep = 0;
    b.nt = 1;
    if (p.mode == kTwoHeads) {
        b.h0 = g * v.G + 2 * (r % p.group_units);
        b.nt = 2;
        b.hstep = 1;
    } else {
        b.h0 = g * v.G + r % p.group_units;
        if (p.mode == kTwoBlocks) {
            b.rstep = kBM;
            b.nt = b.u.rows > kBM ? 2 : 1;
        }
    }
    const int pa = b.u.pos0, pb = b.u.pos0 + b.u.rows - 1, nk = b.u.nk;
    const int last = v.causal ? min(pb, nk - 1) : nk - 1;     // last visible key
    b.jlo = 0;
    b.ns = 0;
    if (v.window > 0) {
        b.jlo = max(0, pa - v.window + 1) / kBN;
        b.ns = min((v.sinks + kBN - 1) / kBN, b.jlo);
    }
    b.n = last < 0 ? 0 : b.ns + (last / kBN - b.jlo + 1);
    b.full.set(v, pa, pa + b.rstep * (b.nt - 1) + kBM - 1, nk);
    b.precise = p.fp16 && ((v.causal && pa < 127) || (v.window > 0 && v.window < 128) || nk < 128);
    return b;
}

// 16-byte chunk fc (8 columns) of row r in a tile of 128-byte swizzled boxes.
__device__ __forceinline__ uint32_t chunk_off(int r, int fc) {
    return (fc >> 3) * (128 * 128) + r * 128 + (((fc & 7) ^ (r & 7)) << 4);
}

// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t below(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
}

// Max of 128 values, four chains of 3-input maxima.
__device__ __forceinline__ float row_max(const float (&v)[128]) {
    float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
    for (int e = 4; e + 8 <= 124; e += 8) {
        m0 = max3(m0, v[e], v[e + 1]);
        m1 = max3(m1, v[e + 2], v[e + 3]);
        m2 = max3(m2, v[e + 4], v[e + 5]);
        m3 = max3(m3, v[e + 6], v[e + 7]);
    }
    m0 = max3(m0, v[124], v[125]);
    m1 = max3(m1, v[126], v[127]);
    return fmaxf(max3(m0, m1, m2), m3);
}

// The query tiles rotated in shared memory by the softmax and helper threads (384):
// bf16 -> fp16 parts (and, precise, remainders), one power of two per row.  A thread
// handles the pairs of one job in every RP-th row; two tiles of the same rows share
// the angles, which step by RP positions (at most 15 steps of 2^-23 each), and are
// worked on together: a warp has only its own independent work to hide latency with.
template <int D, bool kHalf>
__device__ __forceinline__ void rotate_queries(const Block &b, int tid, uint8_t *smem,
                                               Bars<D> &bar, volatile int *abort,
                                               uint64_t tmo, bool &ok) {
    using J = Job<D, kHalf>;
    constexpr int RP = kRotThreads / J::CPR;
    const int q = tid % J::CPR, r0 = tid / J::CPR;
    const bool two_blocks = b.rstep != 0 && b.nt == 2, pair = !two_blocks && b.nt == 2;
    const int rows = two_blocks ? 2 * kBM : kBM;
    float c[J::PPJ], s[J::PPJ];
    float2 st[J::PPJ];
#pragma unroll
    for (int e = 0; e < J::PPJ; ++e) {
        // The row's angle r0 theta on top of the block's, r0 < 96 and |theta| <= pi (its
        // whole turns left out): below 48 turns.  2 pi in two parts, the first of 17 bits
        // so that these multiples are exact; within 2^-22 in all.  (The fp64 reduction per
        // thread took 2.3k cycles of the 384 threads.)
        const float2 th = bar.theta[e * J::CPR + q];
        const float r = static_cast<float>(r0);
        const float k = rintf(r * th.x * 0.15915494f);
        float a = fmaf(r, th.x, -k * 6.28314208984375f);
        a = fmaf(k, -4.32173358e-5f, a);
        a = fmaf(r, th.y, a) + bar.base[e * J::CPR + q];
        const float k2 = rintf(a * 0.15915494f);
        a = fmaf(k2, -4.32173358e-5f, fmaf(k2, -6.28314208984375f, a));
        __sincosf(a, &s[e], &c[e]);
        st[e] = bar.step[e * J::CPR + q];
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&bar.full_q, 0, abort, tmo));
    if (!ok) return;
#pragma unroll 1
    for (int R0 = 0; R0 < rows; R0 += RP) {
        const int R = R0 + r0;
        if (R < rows) {
            const int r = R & (kBM - 1), t0 = R >> 7;
            const uint32_t oa = chunk_off(r, q), ob = chunk_off(r, q + D / 16);
            uint8_t *tile = smem + t0 * Tc<D>::kTile;
            float x1[2][8], x2[2][8];
            uint4 va[2], vb[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // (one tile: the second copy is computed and not stored)
                uint8_t *from = tile + (pair ? x : 0) * Tc<D>::kTile;
                va[x] = *reinterpret_cast<const uint4 *>(from + oa);
                if constexpr (kHalf) vb[x] = *reinterpret_cast<const uint4 *>(from + ob);
            }
            uint4 h1[2], h2[2];
            bool in = true;                // the largest value of the job is in range
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                unpack(va[x], x1[x]);
                if constexpr (kHalf) unpack(vb[x], x2[x]);
                turn<kHalf>(x1[x], x2[x], c, s);
                h1[x] = half_parts(x1[x]);
                float mx = packed_max(h1[x]);
                if constexpr (kHalf) {
                    h2[x] = half_parts(x2[x]);
                    mx = fmaxf(mx, packed_max(h2[x]));
                }
                in = in && mx >= 0.015625f && mx < 16384.f;
            }
            int ex[2] = {0, 0};
            // (rows, and the rows of a pass, are whole warps': the warp is together here)
            // without a value out of range in any lane no row maximum is needed
            constexpr uint32_t lanes = 0xffffffffu;
            if (__any_sync(lanes, !in)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float mx = abs_max8(x1[x]);
                    if constexpr (kHalf) mx = fmaxf(mx, abs_max8(x2[x]));
#pragma unroll
                    for (int o = 1; o < J::CPR; o <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(lanes, mx, o));
                    float undo;
                    const float f = range_scale(mx, &undo);
                    ex[x] = int(__float_as_uint(undo) >> 23) - 127;
                    if (ex[x]) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x1[x][e] *= f;
                            if constexpr (kHalf) x2[x][e] *= f;
                        }
                        h1[x] = half_parts(x1[x]);
                        if constexpr (kHalf) h2[x] = half_parts(x2[x]);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (x == 1 && !pair) break;
                uint8_t *to = tile + x * Tc<D>::kTile;
                uint8_t *low = to + Tc<D>::kOffQLo;
                if (q == 0) bar.q_exp[(t0 + x) * kBM + r] = (signed char)ex[x];
                *reinterpret_cast<uint4 *>(to + oa) = h1[x];
                if (b.precise) *reinterpret_cast<uint4 *>(low + oa) = half_rest(x1[x], h1[x]);
                if constexpr (kHalf) {
                    *reinterpret_cast<uint4 *>(to + ob) = h2[x];
                    if (b.precise) *reinterpret_cast<uint4 *>(low + ob) = half_rest(x2[x], h2[x]);
                }
            }
#pragma unroll
            for (int e = 0; e < J::PPJ; ++e) {
                const float nc = fmaf(c[e], st[e].x, -s[e] * st[e].y);
                s[e] = fmaf(c[e], st[e].y, s[e] * st[e].x);
                c[e] = nc;
            }
        }
    }
}

// Whether any key of the block's sequence is scaled (a warp; every lane a part).
__device__ __forceinline__ bool keys_scaled(const TcParams &p, const Block &b, int lane) {
    if (!p.k_scale || b.u.nk == 0) return false;
    const int f0 = b.u.k0 / p.flag_rows, f1 = (b.u.k0 + b.u.nk - 1) / p.flag_rows;
    bool any = false;
#pragma unroll 8
    for (int f = f0 + lane; f <= f1; f += 32) any |= p.k_flags[f] != 0;
    return any;
}

// Multiply a row's scores of key tile jt (TMEM, from taddr on) by the keys' scales and the
// query's, their product first: keys at one end of the exponents meet queries at the other.
__device__ __noinline__ void scale_scores(const TcParams &p, const Block &b, uint32_t taddr,
                                          int jt, float q_scale) {
    const int last = b.u.nk - jt * kBN;
    const float *ks = p.k_scale + (long long)(b.u.k0 + jt * kBN) * p.v.Hkv + b.g;
#pragma unroll 1
    for (int c = 0; c < kBN; c += 32) {
        float x[32];
        tmem_ld32(taddr + c, x);
        uint32_t u[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const float f = c + e < last ? ks[(long long)(c + e) * p.v.Hkv] : 1.f;
            u[e] = __float_as_uint(x[e] * (f * q_scale));
        }
        tmem_st32(taddr + c, u);
    }
}

// 32 bytes to global memory (32-byte aligned).
__device__ __forceinline__ void store32(void *dst, const uint4 &a, const uint4 &b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// Helper thread tw cleans row tw of a border tile's values: a row behind the
// sequence becomes zero, non-finite values become zero and their row is listed.
template <int D>
__device__ __forceinline__ void clean_values(uint8_t *tile, int tw, bool behind, uint32_t *bad,
                                             int *any_bad) {
    uint32_t hit = 0;
    if (behind) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4 *>(tile + chunk_off(tw, c)) = make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 w = *reinterpret_cast<const uint4 *>(tile + chunk_off(tw, c));
            // an exponent of all ones carries into the sign's place
            hit |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                   ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
        }
        hit &= 0x80008000u;
        if (hit) {
            *any_bad = 1;
            for (int c = 0; c < D / 8; ++c) {
                uint32_t *w = reinterpret_cast<uint32_t *>(tile + chunk_off(tw, c));
                for (int e = 0; e < 4; ++e) {
                    if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
                    if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0x0000ffffu;
                }
            }
        }
    }
    const uint32_t rows = __ballot_sync(0xffffffffu, hit != 0);
    if (bad && (tw & 31) == 0) bad[tw >> 5] = rows;
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
    varlen_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tml, const __grid_constant__ CUtensorMap tmv,
                  const __grid_constant__ TcParams p) {
    using C = Tc<D>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sK = smem + C::kOffK, *sV = smem + C::kOffV;
    static_assert(sizeof(Bars<D>) <= 2048, "barrier block");
    Bars<D> &bar = *reinterpret_cast<Bars<D> *>(smem + C::kOffBar);
    const VarlenParams &v = p.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &bar.abort;
    const uint64_t tmo = v.timeout_ns;
    // (the block lives in shared memory: the roles keep of it what their loops need)
    const Block &B = bar.block;
    const Block b0 = load_block(p);

    // The query's way is the longest: its copies go out before anything else.
    if (warp == kWarpTma && lane == 0) {
        mbar_init(&bar.full_q, 1);
        fence_mbar_init();
        if (b0.u.rows > 0 && b0.n > 0 && !p.stall) {
            mbar_arrive_expect_tx(&bar.full_q, b0.nt * C::kTile);
            for (int t = 0; t < b0.nt; ++t)
                for (int x = 0; x < D / 64; ++x)
                    tma_load_4d(smem + t * C::kTile + x * C::kBox, &tmq, &bar.full_q, x * 64,
                                b0.u.q0 + t * b0.rstep, b0.h0 + t * b0.hstep, 0);
        }
    }
    // (the work before the first barrier is spread over the warps: every CTA waits for it)
    if (p.fp16 && threadIdx.x >= 128 && threadIdx.x < 128 + D / 2) {
        const int i = threadIdx.x - 128;
        using J = Job<D, kHalf>;
        const int at = i % J::PPJ * J::CPR + i / J::PPJ;
        // (rows are whole numbers: whole turns of theta leave their angles as they are)
        const double th = rope_reduced(v.theta[i]);
        const float hi = static_cast<float>(th);
        bar.base[at] = rope_reduced_angle((long long)b0.u.pos0, v.theta[i]);
        bar.theta[at] = make_float2(hi, static_cast<float>(th - hi));
        bar.step[at] = p.step[i];
    }
    if (threadIdx.x == 0) {
        mbar_init(&bar.ready_q, kRotThreads + 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar.full_k[s], 1);
            mbar_init(&bar.empty_k[s], 1);
            mbar_init(&bar.full_v[s], 1);
            mbar_init(&bar.full_b[s], 1);
            mbar_init(&bar.clean_v[s], 128);
            mbar_init(&bar.empty_v[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar.s_ready[t], 1);
            mbar_init(&bar.p_ready[t], 128);
            mbar_init(&bar.o_ready[t], 1);
        }
        mbar_init(&bar.helped, 128);
        mbar_init(&bar.drain, 1);
        bar.block = b0;
        for (int t = 0; t < 2; ++t) bar.own[t].set(v, b0.pos(t), b0.pos(t) + kBM - 1, b0.u.nk);
        bar.abort = 0;
        bar.k_scaled = 0;
        bar.n_border = 0;
        bar.any_bad = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(&bar.tmem_base, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_base;
    // K and V stages in use: precise blocks keep the keys' parts in two K stages
    const int mask = B.precise ? 0 : NS - 1, shift = B.precise ? 0 : (NS == 4 ? 2 : 1);
    bool pre = false;   // thread 0: an earlier CTA's wait ran out already
    if (threadIdx.x == 0 && v.status && *reinterpret_cast<volatile int *>(v.status) ==
                                            int(LCX_ERR_TIMEOUT)) {
        pre = true;
        *abort = 1;
    }

    if (B.u.rows <= 0) {
        // (a plan that does not fit the tensors: nothing to do)
        if (threadIdx.x == 0) raise_status(v.status, LCX_ERR_INVALID_ARG);
    } else if ((warp >> 2) == 3) {
        setmaxnreg_dec<kRegsIssue>();
        if (warp == kWarpTma && lane == 0 && B.n > 0 && !p.stall) {
            // ------------------------------------------------ Q and K producer
            tma_prefetch_desc(&tmk);
            wait_previous_kernel();                       // the rotated keys
            uint32_t used = 0;                            // stages with a copy issued
            bool ok = true;
            int j = 0;
            for (; ok && j < B.n; ++j) {
                const int s = j & mask, r = B.u.k0 + B.tile(j) * kBN;
                if (j > mask) ok = mbar_wait(&bar.empty_k[s], ((j >> shift) - 1) & 1, abort, tmo);
                if (!ok) break;
                mbar_arrive_expect_tx(&bar.full_k[s], (B.precise ? 2 : 1) * C::kTile);
                for (int x = 0; x < D / 64; ++x) {
                    tma_load_4d(sK + s * C::kTile + x * C::kBox, &tmk, &bar.full_k[s], x * 64, r,
                                B.g, 0);
                    if (B.precise)
                        tma_load_4d(sK + C::kTile + x * C::kBox, &tml, &bar.full_k[s], x * 64, r,
                                    B.g, 0);
                }
                used |= 1u << s;
            }
            // never leave the CTA with copies in flight: the last one of every stage
            mbar_wait(&bar.full_q, 0, nullptr, tmo);
            for (int s = 0; s <= mask; ++s)
                if (used >> s & 1)
                    mbar_wait(&bar.full_k[s], ((j - 1 - s) >> shift) & 1, nullptr, tmo);
        } else if (warp == kWarpTmaV && lane == 0 && B.n > 0 && !p.stall) {
            // ------------------------------------------------ V producer
            // Border tiles arrive on barriers of their own (full_b), which only the
            // helpers wait for, one phase after the other: a wait by parity must not
            // skip phases.  Bit s of a mask: the parity of a stage's next phase.
            tma_prefetch_desc(&tmv);
            uint32_t used = 0, used_b = 0, phase = 0, phase_b = 0;
            bool ok = true;
            for (int j = 0; ok && j < B.n; ++j) {
                const int s = j & mask;
                if (j > mask) ok = mbar_wait(&bar.empty_v[s], ((j >> shift) - 1) & 1, abort, tmo);
                if (!ok) break;
                const bool border = !B.full.has(B.tile(j));
                uint64_t *full = border ? &bar.full_b[s] : &bar.full_v[s];
                mbar_arrive_expect_tx(full, C::kTile);
                for (int x = 0; x < D / 64; ++x)
                    tma_load_4d(sV + s * C::kTile + x * C::kBox, &tmv, full, x * 64,
                                B.u.k0 + B.tile(j) * kBN, B.g, 0);
                (border ? used_b : used) |= 1u << s;
                (border ? phase_b : phase) ^= 1u << s;
            }
            for (int s = 0; s <= mask; ++s) {
                if (used >> s & 1) mbar_wait(&bar.full_v[s], (phase >> s & 1) ^ 1, nullptr, tmo);
                if (used_b >> s & 1)
                    mbar_wait(&bar.full_b[s], (phase_b >> s & 1) ^ 1, nullptr, tmo);
            }
        } else if (warp == kWarpFlags && B.n > 0 && p.fp16) {
            // ------------------------------------------------ are there scaled keys?
            wait_previous_kernel();
            const bool any = __any_sync(0xffffffffu, keys_scaled(p, B, lane));
            if (lane == 0) {
                bar.k_scaled = any;
                mbar_arrive(&bar.ready_q);
            }
        } else if (warp == kWarpMma && lane == 0 && B.n > 0) {
            // ------------------------------------------------ MMA issuer
            const int n = B.n, nt = B.nt, ns = B.ns, jlo = B.jlo;
            const Full full = B.full;
            const bool precise = B.precise;
            const uint32_t fmt = p.fp16 ? kFmtF16 : kFmtBF16;
            const uint32_t id_s = idesc_f32acc(128, kBN, 0, 0, 0, 0) | (fmt << 7) | (fmt << 10);
            constexpr uint32_t id_pv = idesc_bf16_f32(128, D, 0, 1);   // V as the TMA lands it
            // Every operand's descriptor differs from the first query tile's by a
            // constant: the start address, and for V (MN-major) the leading offset.
            const uint32_t q_lo = uint32_t(sdesc_sw128(smem_u32(smem), 16, 1024));
            constexpr uint32_t dhi = sdesc_hi_sw128(1024);
            constexpr uint32_t kK = C::kOffK >> 4, kQLo = C::kOffQLo >> 4, kT = C::kTile >> 4;
            constexpr uint32_t kV = (C::kOffV >> 4) + (((C::kBox >> 4) - 1) << 16);
            auto product = [&](uint32_t dst, uint32_t qa, uint32_t ka, uint32_t more) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4;
                    mma_ss_w<0>(dst, qa + o, ka + o, dhi, id_s, kk > 0 ? 1u : more);
                }
            };
            auto issue_s = [&](int t, int s) {
                const uint32_t dst = tmem + t * kBN;
                const uint32_t qa = q_lo + t * kT, ka = q_lo + kK + s * kT;
                product(dst, qa, ka, 0);
                if (precise) {
                    // Qh Kl, then Ql Kh
#pragma unroll 1
                    for (int i = 0; i < 2; ++i)
                        product(dst, i ? qa + kQLo : qa, i ? ka : q_lo + kK + kT, 1);
                }
                mma_commit(&bar.s_ready[t]);
            };
            auto issue_pv = [&](int t, int s, bool acc) {
                const uint32_t va = q_lo + kV + s * kT;
                const uint32_t dst = tmem + C::kColO + t * D, pa = tmem + t * kBN;
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    mma_ts_w<0>(dst, pa + kk * 8, va + ((kk * 16 * 128) >> 4), dhi, id_pv,
                                acc || kk > 0);
            };
            uint32_t cleaned = 0, landed = 0;             // next parity of clean_v, full_v
            bool ok = mbar_wait(p.fp16 ? &bar.ready_q : &bar.full_q, 0, abort, tmo);
            if (ok) ok = mbar_wait(&bar.full_k[0], 0, abort, tmo);
            if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int t = 0; t < nt; ++t) issue_s(t, 0);
                mma_commit(&bar.empty_k[0]);
            }
            for (int j = 0; ok && j < n; ++j) {
                const int s = j & mask, jn = j + 1;
                if (!full.has(j < ns ? j : jlo + (j - ns))) {
                    ok = mbar_wait(&bar.clean_v[s], (cleaned >> s) & 1, abort, tmo);
                    cleaned ^= 1u << s;
                } else {
                    ok = mbar_wait(&bar.full_v[s], (landed >> s) & 1, abort, tmo);
                    landed ^= 1u << s;
                }
#pragma unroll 1
                for (int t = 0; ok && t < nt; ++t) {
                    ok = mbar_wait(&bar.p_ready[t], j & 1, abort, tmo);
                    tc_fence_after();
                    if (!ok) break;
                    issue_pv(t, s, j > 0);
                    if (jn == n) mma_commit(&bar.o_ready[t]);
                    if (jn < n) {
                        if (t == 0) {
                            ok = mbar_wait(&bar.full_k[jn & mask], (jn >> shift) & 1, abort, tmo);
                            tc_fence_after();
                            if (!ok) break;
                        }
                        issue_s(t, jn & mask);
                    }
                }
                if (ok) {
                    mma_commit(&bar.empty_v[s]);
                    if (jn < n) mma_commit(&bar.empty_k[jn & mask]);
                }
            }
            // all issued products complete before TMEM is released
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, nullptr, tmo);
        }
    } else if ((warp >> 2) == 2) {
        setmaxnreg_dec<kRegsHelp>();
        // ------------------------------------------------ helpers
        const int tw = threadIdx.x - kWarpHelp * 32;
        bool ok = true;
        if (B.n > 0) {
            if (p.fp16) {
                rotate_queries<D, kHalf>(B, threadIdx.x, smem, bar, abort, tmo, ok);
                if (ok) {
                    fence_proxy_async_smem();
                    mbar_arrive(&bar.ready_q);
                }
            }
            int nb = 0;
            uint32_t phase = 0;
            for (int j = 0; ok && j < B.n; ++j) {
                const int jt = B.tile(j), s = j & mask;
                if (B.full.has(jt)) continue;
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&bar.full_b[s], (phase >> s) & 1, abort, tmo));
                phase ^= 1u << s;
                if (!ok) break;
                if (nb < kMaxBorder && tw == 0) bar.border_tile[nb] = jt;
                clean_values<D>(sV + s * C::kTile, tw, jt * kBN + tw >= B.u.nk,
                                nb < kMaxBorder ? bar.bad[nb] : nullptr, &bar.any_bad);
                ++nb;
                fence_proxy_async_smem();
                mbar_arrive(&bar.clean_v[s]);
            }
            if (tw == 0) bar.n_border = nb;
            mbar_arrive(&bar.helped);
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ------------------------------------------------ softmax of tile t
        const int t = warp >> 2, row = (warp & 3) * 32 + lane;
        bool ok = true;
        if (p.fp16 && B.n > 0) {
            rotate_queries<D, kHalf>(B, threadIdx.x, smem, bar, abort, tmo, ok);
            if (ok) {
                fence_proxy_async_smem();
                mbar_arrive(&bar.ready_q);
            }
        }
        if (t < B.nt) {
            // (a row of scores takes 128 of the 176 registers: what the key loop needs of
            // the block is read again for every tile, while the scores are computed)
            const int n = B.n;
            const uint32_t trow = tmem + (uint32_t((warp & 3) * 32) << 16);
            const uint32_t s_col = t * kBN, o_col = C::kColO + t * D;
            auto q_scale = [&]() {
                return __uint_as_float(uint32_t(127 + bar.q_exp[t * kBM + row]) << 23);
            };
            float m = -INFINITY, l = 0.f, cl2 = v.c_log2;
            bool scaled = false;
            if (p.fp16 && n > 0 && ok) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bar.ready_q, 0, abort, tmo));
                scaled = bar.k_scaled != 0;
                if (!scaled) cl2 *= q_scale();
            }
            for (int j = 0; ok && j < n; ++j) {
                const int jt = B.tile(j);
                const bool whole = bar.own[t].has(jt);
                ok = __all_sync(0xffffffffu, mbar_wait(&bar.s_ready[t], j & 1, abort, tmo));
                if (!ok) break;
                tc_fence_after();
                if (scaled) scale_scores(p, B, trow + s_col, jt, q_scale());
                float x[kBN];
                tmem_ld128(trow + s_col, x);
                if (!whole) {
                    // visible: e <= hi and (no window or e >= lo or e < sk), a bit per
                    // key in four words
                    const int k0 = jt * kBN, nk = B.u.nk, pos = B.pos(t) + row;
                    const int hi = v.causal ? min(pos - k0, nk - 1 - k0) : nk - 1 - k0;
                    const int lo = v.window > 0 ? pos - v.window + 1 - k0 : 0, sk = v.sinks - k0;
#pragma unroll
                    for (int g = 0; g < kBN / 32; ++g) {
                        const uint32_t keep =
                            below(hi + 1 - 32 * g) & (~below(lo - 32 * g) | below(sk - 32 * g));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[32 * g + e] = (keep >> e) & 1 ? x[32 * g + e] : -INFINITY;
                    }
                }
                const float m_new = fmaxf(m, row_max(x) * cl2);
                const bool need = (m != -INFINITY) && (m_new > m + kLazy);
                if (__any_sync(0xffffffffu, need)) {
                    const float alpha = need ? ex2_approx(m - m_new) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(trow + o_col + c * 32, o);
                        uint32_t u[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * alpha);
                        tmem_st32_nowait(trow + o_col + c * 32, u);
                    }
                    tmem_wait_st();
                    if (need) {
                        l *= alpha;
                        m = m_new;
                    }
                }
                if (m == -INFINITY) m = m_new;
                const float mref = m == -INFINITY ? 0.f : m;
                const float2 c2 = make_float2(cl2, cl2), nm2 = make_float2(-mref, -mref);
                float2 sum = make_float2(0.f, 0.f);
                uint32_t pk_[kBN / 2];
#pragma unroll
                for (int e = 0; e < kBN / 2; ++e) {
                    const float2 y = fma2(make_float2(x[2 * e], x[2 * e + 1]), c2, nm2);
                    const float2 w = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                    // P rounded to bf16 for the product; its sum is not
                    pk_[e] = pack_bf16x2(w.x, w.y);
                    sum = add2(sum, w);
                }
                tmem_st64(trow + s_col, pk_);
                l += sum.x + sum.y;
                tc_fence_before();
                mbar_arrive(&bar.p_ready[t]);
            }
            bool bad = false;
            int nb = 0;
            const bool valid = row < B.rows(t);
            const int h = B.h0 + t * B.hstep, pos = B.pos(t) + row;
            if (ok && n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bar.o_ready[t], 0, abort, tmo)) &&
                     __all_sync(0xffffffffu, mbar_wait(&bar.helped, 0, abort, tmo));
                bad = bar.any_bad != 0;
                nb = bar.n_border;
            }
            if (ok) {
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;
                // The rows go through the query tile's place (all its products are done)
                // and out as whole rows: a warp's own 32, so only the warp waits.
                uint8_t *stage = smem + t * C::kTile + row * (D * 2);
                const bool wide =
                    !((reinterpret_cast<uintptr_t>(v.o) | (v.os[0] * 2) | (v.os[1] * 2)) & 31);
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    float o[64];
                    if (n > 0) {
                        tmem_ld64(trow + o_col + c * 64, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 64; ++e) o[e] = 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e] *= inv;
                    if (bad && valid) {
                        // non-finite values of border tiles that this row does see
                        for (int i = 0; i < nb; ++i) {
                            const bool listed = i < kMaxBorder;
                            const int jt = listed ? bar.border_tile[i] : -1;
                            for (int r = 0; listed && r < kBN; ++r) {
                                if (!(bar.bad[i][r >> 5] >> (r & 31) & 1)) continue;
                                const int key = jt * kBN + r;
                                if (key >= B.u.nk || (v.causal && key > pos) ||
                                    (v.window > 0 && pos - key >= v.window && key >= v.sinks))
                                    continue;
                                const __nv_bfloat16 *src =
                                    reinterpret_cast<const __nv_bfloat16 *>(v.v) +
                                    (long long)(B.u.k0 + key) * v.vs[0] + B.g * v.vs[1] + c * 64;
#pragma unroll
                                for (int e = 0; e < 64; ++e) {
                                    const float y = static_cast<float>(src[e]);
                                    if (!(fabsf(y) < INFINITY)) o[e] += y;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4 *>(stage + (((c * 8 + e) ^ (row & 7)) << 4)) =
                            make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]),
                                       pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                       pack_bf16x2(o[8 * e + 4], o[8 * e + 5]),
                                       pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
                }
                __syncwarp();
                const int w0 = (warp & 3) * 32, rows = B.rows(t);
                __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(v.o) +
                                     (long long)(B.u.q0 + t * B.rstep) * v.os[0] + h * v.os[1];
                auto piece = [&](int r, int ch) {
                    return *reinterpret_cast<const uint4 *>(smem + t * C::kTile + r * (D * 2) +
                                                            ((ch ^ (r & 7)) << 4));
                };
                if (wide) {
                    constexpr int CR = D / 16, RI = 32 / CR;   // 32-byte pieces of a row
#pragma unroll
                    for (int i = 0; i < 32; i += RI) {
                        const int r = w0 + i + lane / CR, ch = lane % CR;
                        const uint4 y0 = piece(r, 2 * ch), y1 = piece(r, 2 * ch + 1);
                        if (r < rows) store32(out + r * v.os[0] + ch * 16, y0, y1);
                    }
                } else {
                    constexpr int CR = D / 8, RI = 32 / CR;    // 16-byte pieces
#pragma unroll 4
                    for (int i = 0; i < 32; i += RI) {
                        const int r = w0 + i + lane / CR, ch = lane % CR;
                        const uint4 y = piece(r, ch);
                        if (r < rows) *reinterpret_cast<uint4 *>(out + r * v.os[0] + ch * 8) = y;
                    }
                }
                if (valid && v.lse)
                    v.lse[(long long)h * v.Tq + B.u.q0 + t * B.rstep + row] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            }
        }
    }

    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) {
        // (a CTA without key tiles, too, ends after the key rotation: what follows in
        // the stream may write its inputs)
        wait_previous_kernel();
        if (!pre && bar.abort) raise_status(v.status, LCX_ERR_TIMEOUT);
    }
}

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// [T, H, D] tensor of 16-bit elements -> boxes of 64 columns x 128 rows, 128-byte
// swizzle; rows past T read as zero.
lcx_status token_map(CUtensorMap *map, const void *ptr, int64_t T, int64_t H, int64_t D,
                     const long long *st, const char *name) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(LCX_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(T), cuuint64_t(H), 1};
    // (a single token's or head's stride is never taken)
    const cuuint64_t strides[3] = {cuuint64_t(T > 1 ? st[0] * 2 : D * 2),
                                   cuuint64_t(H > 1 ? st[1] * 2 : D * 2), 16};
    const cuuint32_t box[4] = {64, 128, 1, 1}, ones[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims,
                          strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(LCX_ERR_UNSUPPORTED, "tensor map for %s rejected (CUresult %d)", name, int(r));
    return LCX_OK;
}

// Workspace of rotated keys: fp32, or the parts the tcgen05 kernel reads.
struct KeySpace {
    int64_t lo, scale, flags, bytes;      // offsets (hi, or the fp32 keys, at 0)
};
KeySpace key_space(int64_t total_k, int64_t H, int64_t D, int dtype) {
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    KeySpace k = {};
    if (dtype == LCX_F32) {
        k.bytes = up(total_k * H * D * 4);
        return k;
    }
    k.lo = up(total_k * H * D * 2);
    k.scale = k.lo + up(total_k * H * D * 2);
    k.flags = k.scale + up(total_k * H * 4);
    k.bytes = k.flags + up((total_k / 16 + 1) * 4);
    return k;
}

template <int D, bool kHalf>
lcx_status launch_keys(KeyParams &k, cudaStream_t s) {
    constexpr int rpc = kKeyThreads / Job<D, kHalf>::CPR;
    cudaError_t e = launch_dependent(varlen_keys_kernel<D, kHalf>,
                                     dim3(unsigned((k.T + rpc - 1) / rpc)), dim3(kKeyThreads), 0,
                                     s, k);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "attn_varlen key launch failed: %s", cudaGetErrorString(e));
    return LCX_OK;
}

template <int D, bool kHalf>
lcx_status launch_tc(const CUtensorMap (&m)[4], TcParams &p, bool after_keys, cudaStream_t s) {
    auto kern = varlen_kernel<D, kHalf>;
    p.flag_rows = kKeyThreads / Job<D, kHalf>::CPR;
    // the warpgroups' register shares must add up to what the launch holds
    static const int regs = []() {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, varlen_kernel<D, kHalf>) == cudaSuccess ? fa.numRegs : -1;
    }();
    if (regs * kThreads < (2 * kRegsSoftmax + kRegsHelp + kRegsIssue) * 128)
        return fail(LCX_ERR_CUDA, "attn_varlen kernel built with %d registers per thread; the "
                    "warpgroup register split needs 128", regs);
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "cudaFuncSetAttribute failed: %s", cudaGetErrorString(e));
    const long long grid = (long long)p.v.n_units * p.group_units * p.v.Hkv;
    if (grid > 0x7fffffffLL) return fail(LCX_ERR_UNSUPPORTED, "too many work units");
    if (after_keys)
        e = launch_dependent(kern, dim3(unsigned(grid)), dim3(kThreads), Tc<D>::kSmem, s, m[0],
                             m[1], m[2], m[3], p);
    else
        kern<<<unsigned(grid), kThreads, Tc<D>::kSmem, s>>>(m[0], m[1], m[2], m[3], p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "attn_varlen launch failed: %s", cudaGetErrorString(e));
    return LCX_OK;
}

// The bf16 path: rotated keys (unless given), then the tcgen05 kernel.
lcx_status run_tc(const lcx_varlen_args *a, const VarlenParams &v, cudaStream_t s) {
    const lcx_varlen_info &I = a->info;
    const bool half = v.half != 0, rotate = v.rotate_q != 0;
    TcParams p;
    memset(&p, 0, sizeof(p));
    p.v = v;
    p.fp16 = rotate ? 1 : 0;
    p.stall = (a->flags & LCX_VARLEN_TEST_STALL) ? 1 : 0;
    // Two query tiles per CTA, unless CTAs of one tile each fit the SMs at once (1 x 512
    // tokens of 32/8 heads of 128: one tile 21.3, two 22.9 us; 5 x 128: 26.9 and 18.7; 640
    // behind 8000 keys: 250 and 157; 4096 of 8/2 heads of 64 under a window of 300: 32.1
    // and 22.8).  Causal prompts of 1500 tokens and more are uneven enough for one tile as
    // long as the CTAs of two leave SMs idle (3500 of 8/2 heads of 64: 57.7 and 63.8; 2000
    // of 12/4 heads of 128: 43.2 and 49.2).
    const int64_t one = I.n_units[0] * v.Hq;
    const int64_t pairs = v.G % 2 == 0 ? one / 2 : I.n_units[1] * v.Hq;
    const bool uneven = v.causal && v.window == 0 && I.total_q == I.total_k &&
                        I.total_q >= 1500 * I.n_seqs;
    const int sms = device_sms();
    p.mode = one <= sms || (uneven && pairs < sms) ? kOneTile
             : v.G % 2 == 0                        ? kTwoHeads
                                                   : kTwoBlocks;
    p.group_units = p.mode == kTwoHeads ? v.G / 2 : v.G;
    // Order of the CTAs.  All heads of the heaviest row blocks first balances best.  When
    // the keys and values of all heads exceed what L2 holds for both dies, kv head by kv
    // head reads them from there instead, and the power saved goes into the clock: on a GPU
    // kept busy 12 x 4096 tokens of 32/8 heads of 128 take 2147 against 2313 us, 2 x 26000
    // 11.7 against 12.1 ms, 1 x 32768 9.13 against 9.30, 32 x 1024 585 against 613 us (64 x
    // 512: 465 and 460; after a pause, at full clock, it costs up to 2 %: 2099 and 2075).
    // Heads of 64 and groups of one do not gain: 32 x 1024 tokens of 32/16 heads of 64 504
    // against 470 us, 22000 of 8/8 heads of 128 1184 against 1119.
    p.by_head = a->D == 128 && v.G > 1 && I.total_k * v.Hkv * a->D * 4 > (int64_t(80) << 20);
    const int which = p.mode == kTwoBlocks;
    p.v.units =
        reinterpret_cast<const VarlenUnit *>(a->plan + plan_units(I.n_seqs, which, I.n_units[0]));
    p.v.n_units = int(I.n_units[which]);
    const void *kp = a->k, *lo = a->k;
    long long ks[2] = {v.ks[0], v.ks[1]};
    if (rotate && I.total_k > 0) {
        const KeySpace ws = key_space(I.total_k, v.Hkv, a->D, LCX_BF16);
        char *base = static_cast<char *>(a->workspace);
        KeyParams k = {};
        k.k = static_cast<const __nv_bfloat16 *>(a->k);
        k.st = a->k_strides[0];
        k.sh = a->k_strides[1];
        k.hi = reinterpret_cast<__half *>(base);
        k.lo = reinterpret_cast<__half *>(base + ws.lo);
        k.scale = reinterpret_cast<float *>(base + ws.scale);
        k.flags = reinterpret_cast<int *>(base + ws.flags);
        k.cu = a->plan + plan_cu_k(I.n_seqs);
        k.n = int(I.n_seqs);
        k.T = int(I.total_k);
        k.H = v.Hkv;
        k.all_lo = v.window > 0 && v.window < 128;
        memcpy(k.theta, v.theta, sizeof(k.theta));
        k.ms = v.ms;
        lcx_status st = a->D == 128 ? (half ? launch_keys<128, true>(k, s) : launch_keys<128, false>(k, s))
                                    : (half ? launch_keys<64, true>(k, s) : launch_keys<64, false>(k, s));
        if (st != LCX_OK) return st;
        kp = k.hi;
        lo = k.lo;
        p.k_scale = k.scale;
        p.k_flags = k.flags;
    }
    if (rotate) {
        const int cpr = half ? int(a->D / 16) : int(a->D / 8);
        for (int i = 0; i < a->D / 2; ++i) {
            const double ang = (kRotThreads / cpr) * v.theta[i];
            p.step[i] = make_float2(float(std::cos(ang)), float(std::sin(ang)));
        }
    }
    CUtensorMap m[4];
    lcx_status st;
    if ((st = token_map(&m[0], a->q, a->Tq, v.Hq, a->D, v.qs, "q")) != LCX_OK) return st;
    if (I.total_k > 0) {
        if ((st = token_map(&m[1], kp, v.Tk, v.Hkv, a->D, ks, "k")) != LCX_OK) return st;
        if ((st = token_map(&m[2], lo, v.Tk, v.Hkv, a->D, ks, "k")) != LCX_OK) return st;
        if ((st = token_map(&m[3], a->v, a->Tk, v.Hkv, a->D, v.vs, "v")) != LCX_OK) return st;
    } else {
        m[1] = m[2] = m[3] = m[0];      // no block has a key tile
    }
    const bool dep = p.k_scale != nullptr;
    if (a->D == 128)
        return half ? launch_tc<128, true>(m, p, dep, s) : launch_tc<128, false>(m, p, dep, s);
    return half ? launch_tc<64, true>(m, p, dep, s) : launch_tc<64, false>(m, p, dep, s);
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
    if (a->flags & ~uint32_t(LCX_VARLEN_PREROTATED | LCX_VARLEN_TEST_STALL))
        return fail(LCX_ERR_INVALID_ARG, "unknown flags");
    if ((a->flags & LCX_VARLEN_TEST_STALL) && a->dtype != LCX_BF16)
        return fail(LCX_ERR_UNSUPPORTED, "the stall test hook needs bf16 operands");
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
    if ((st = check_distinct(a->o_strides, a->Tq, a->Hq, "o")) != LCX_OK) return st;
    if (I.total_k > 0) {
        if ((st = check_tokens(a->k, a->k_strides, es, "k")) != LCX_OK) return st;
        if ((st = check_tokens(a->v, a->v_strides, es, "v")) != LCX_OK) return st;
    }
    if (es == 2) {               // a tensor map's strides are positive
        if ((st = check_distinct(a->q_strides, a->Tq, a->Hq, "q")) != LCX_OK ||
            (st = check_distinct(a->k_strides, a->Tk, a->Hkv, "k")) != LCX_OK ||
            (st = check_distinct(a->v_strides, a->Tk, a->Hkv, "v")) != LCX_OK)
            return st;
    }
    const bool rotate = !(a->flags & LCX_VARLEN_PREROTATED) && a->rope.mode != LCX_ROPE_NONE;
    if (rotate && I.total_k > 0) {
        if (!a->workspace || (reinterpret_cast<uintptr_t>(a->workspace) & 255u))
            return fail(LCX_ERR_INVALID_ARG,
                        "workspace must be a 256-byte aligned device pointer");
        const int64_t need = key_space(I.total_k, a->Hkv, a->D, a->dtype).bytes;
        if (a->workspace_bytes < need)
            return fail(LCX_ERR_INVALID_ARG, "workspace holds %lld bytes; %lld needed",
                        (long long)a->workspace_bytes, (long long)need);
    }
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const char *>(a->q);
    p.k = static_cast<const char *>(rotate ? a->workspace : a->k);
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
    p.ms = 1.f;
    if (rotate)
        rope_freqs_unchecked(&a->rope,
                             effective_seq_len(&a->rope, std::max<int64_t>(I.max_k, 1)), p.theta,
                             &p.ms);
    const double scale =
        a->softmax_scale > 0.f ? double(a->softmax_scale) : 1.0 / std::sqrt(double(a->D));
    // q' is rotated without mscale (folded in here); the rotated keys carry theirs
    p.c_log2 = float(scale * double(p.ms) * 1.4426950408889634);
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
    if (a->dtype == LCX_BF16) return run_tc(a, p, s);
    if (p.rotate_q) {
        st = rotate_packed(&a->rope, std::max<int64_t>(a->info.max_k, 1), a->k, a->k_strides,
                           a->workspace, a->plan + plan_cu_k(a->info.n_seqs),
                           int(a->info.n_seqs), a->info.total_k, a->Hkv, a->D, s);
        if (st != LCX_OK) return st;
    }
    p.units = reinterpret_cast<const VarlenUnit *>(
        a->plan + plan_units(a->info.n_seqs, 0, a->info.n_units[0]));
    p.n_units = int(a->info.n_units[0]);
    const bool dep = p.rotate_q && a->info.total_k > 0;
    return a->D == 128 ? launch_f32<128>(p, dep, s) : launch_f32<64>(p, dep, s);
}

extern "C" int64_t lcx_varlen_workspace_bytes(const lcx_varlen_info *info, int64_t Hkv, int64_t D,
                                              int32_t dtype) {
    if (!info || info->total_k < 0 || info->total_k > (1 << 30) || Hkv <= 0 || Hkv > 65536 ||
        (D != 64 && D != 128) || (dtype != LCX_BF16 && dtype != LCX_F32))
        return -1;
    return key_space(info->total_k, Hkv, D, dtype).bytes;
}
