// paged_decode.cu -- attention of one new token per sequence over the paged
// key/value cache (lcx_paged_decode).
//
// o = sum_j softmax_j(c <q', k'_j>) v_j over the visible keys, evaluated with a
// running maximum and sum ("8.3 长上下文技术", 8.3.4), q' = q rotated at the
// token's position; parts over disjoint keys join by rescaling with their maxima
// (8.3.5 step 3).
//
// Bound by HBM: every visible key and value is read once, 4 Hkv D bytes per key
// (bf16) against 4 Hq D flops.  Measured (8 kv heads of 128, bf16): 1.39 GB of keys and
// values in 208 us, 6.7 TB/s, as fast as a copy; 0.35 GB in 64.5 us, 5.4 TB/s (the start,
// the uneven end and the join are 11 us); one sequence of 300 keys in 7.1 us.  fp32:
// 0.40 GB in 86 us, 4.7 TB/s; no pipe is full (issue 46 %, tensor pipe 28 %, DRAM 59 %):
// eight warps an SM wait for one another's chain of parts, product, softmax, product.
//
// Work: the visible keys of each (entry, kv head, block of query heads), a
// "segment", are cut into blocks of 32 to 128 keys; the blocks of all segments in
// order form one list, and every CTA takes an equal stretch of it, so a batch of
// ragged lengths loads the SMs evenly without a plan from the host (lengths are
// device data).  A CTA sees at most two segments whose other blocks lie in other
// CTAs, its first and its last: their parts go to the workspace and a second
// kernel joins them, in CTA order; whole segments are written at once.
//
// Inside a CTA each of the four warps takes a quarter of every block and keeps a
// ring of its own: cp.async copies (16 bytes, any page size and strides, hidden
// keys zero-filled) run two tiles ahead without a barrier between warps, across
// segment borders.  Two CTAs per SM keep 128 KB in flight.
//
// Products: mma.sync with the query heads as the 16 rows.  With at most 8 heads
// the rows hold two bf16 parts of q' (hi in rows 0-7, lo in 8-15) and later of the
// weights, which costs nothing (the rows would be empty) and keeps 16 bits; with 9
// to 16 heads (kWide) q' takes a second product and the weights are rounded to
// bf16.  fp32 pools use tf32 products with two parts of every operand.
#include <algorithm>
#include <cmath>

#include "mma_sync.cuh"
#include "paged.cuh"
#include "rope_angle.cuh"
#include "sm100.cuh"
#include "vec16.cuh"

namespace lcx {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStages = 3;      // ring of a warp: one tile in use, two in flight
constexpr int kHalf = 4096;     // bytes of a tile's keys, and of its values
constexpr float kLazy = 8.f;    // log2 growth of the maximum that moves the reference

template <typename T, int D, bool kWide>
struct Dec {
    static constexpr int ES = sizeof(T);
    static constexpr int ROW = D * ES;            // bytes of a key row
    static constexpr int KT = kHalf / ROW;        // keys of a warp's tile
    static constexpr int BLK = KT * kWarps;       // keys of a block
    static constexpr int HB = kWide ? 16 : 8;     // query heads of a segment
    static constexpr int CPR = ROW / 16;          // 16-byte chunks of a row
    static constexpr int RPI = 32 / CPR;          // rows a warp copies per instruction
    static constexpr int NI = KT / RPI;
    static_assert(!kWide || ES == 2, "wide segments: 16-bit pools");
    // shared memory: rings, q' in two parts and the next segment's q as it comes,
    // the warps' outputs (8 heads x CW columns at a time), their statistics, the
    // rings' visibility masks
    static constexpr int kOffQ = kWarps * kStages * 2 * kHalf;
    static constexpr int kBytesQ = HB * ROW;      // q, and each part of q'
    static constexpr int kOffRaw = kOffQ + 2 * kBytesQ;
    static constexpr int kOffO = kOffRaw + kBytesQ;
    static constexpr int CW = kBytesQ > 2048 ? 32 : 64;
    static constexpr int kOffM = kOffO + kWarps * 8 * CW * 4;
    static constexpr int kOffMask = kOffM + kWarps * 16 * 2 * 4;
    static constexpr int kSmem = kOffMask + kWarps * kStages * 4 + 16;
    static_assert(kSmem <= 115712, "two CTAs per SM");
};

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
    int window, sinks;
    int rotate, half;
    float c_log2;               // logit scale in log2 units
    int ctas, blk;              // CTAs of the attention kernel, keys per block
    float *part_o, *part_ml;    // [2 ctas][HB][D], [2 ctas][HB][2]
    double theta[64];
};

// The visible keys of an entry: [0, ns) and [lo, len), listed so that every tile's
// keys lie in one page of a tile or more: the first from place 0 to nsp (ns rounded
// up to kAlign places), the others from the key loa = lo rounded down on; places
// without a visible key are copied as zeros and masked.
constexpr int kAlign = 32;
struct Entry {
    int id, len, ns, lo, nvis, nblk;
    __device__ __forceinline__ int nsp() const { return (ns + kAlign - 1) & ~(kAlign - 1); }
    __device__ __forceinline__ int loa() const { return lo & ~(kAlign - 1); }
    // key at place v, or -1
    __device__ __forceinline__ int key(int v) const {
        if (v < nsp()) return v < ns ? v : -1;
        const int j = loa() + (v - nsp());
        return j >= lo && j < len ? j : -1;
    }
};
__device__ __forceinline__ Entry load_entry(const DecodeParams &p, int e, bool report) {
    Entry x;
    x.id = p.ids[e];
    x.len = 0;
    bool bad = x.id >= p.S;
    if (x.id >= 0 && !bad) {
        const long long most = (long long)p.MP << p.ps_log2;
        const int len = p.lens[x.id];
        bad = len < 0 || len > most;
        x.len = len < 0 ? 0 : int(min((long long)len, most));
    }
    if (bad && report) raise_status(p.status, LCX_ERR_INVALID_ARG);
    x.lo = p.window > 0 ? max(0, x.len - p.window) : 0;
    x.ns = min(p.sinks, x.lo);
    x.nvis = x.len - x.loa() + x.nsp();
    x.nblk = max(1, (x.nvis + p.blk - 1) / p.blk);   // an empty entry writes its zeros
    return x;
}

// Sum of x over the CTA's threads (4 warps); scratch of 4 ints.
__device__ __forceinline__ int cta_sum(int x, int *scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    return scratch[0] + scratch[1] + scratch[2] + scratch[3];
}

// First block of CTA c's stretch of the list of nb blocks.
__device__ __forceinline__ long long stretch(long long nb, int c, int ctas) {
    return nb * c / ctas;
}

// Position in the block list: block blk of segment (entry e, head block r).
struct Cursor {
    int e, r, blk;
    Entry x;
    __device__ __forceinline__ bool last() const { return blk == x.nblk - 1; }
    __device__ __forceinline__ void next(const DecodeParams &p) {
        if (++blk < x.nblk) return;
        blk = 0;
        if (++r < p.Hkv * p.hb) return;
        r = 0;
        if (++e < p.n) x = load_entry(p, e, false);
    }
};

// What the CTA's threads exchange to find their stretch.
struct Start {
    int sum[4];
    int e, off;
    Entry x;
};

// 16-byte chunk c of row r of a tile with CPR chunks per row, moved so that the
// reads below touch every bank once: 16-bit rows by ldmatrix (8 rows, one chunk);
// fp32 keys by rows r, r + 1 and four chunks, fp32 values by every other row.
template <typename T, int CPR>
__device__ __forceinline__ uint32_t chunk_at(int r, int c, bool value) {
    if constexpr (sizeof(T) == 2)
        return (r * CPR + (c ^ (r & 7))) * 16;
    else
        return (r * CPR + (c ^ (value ? ((r >> 1) & 3) << 1 : (r & 1) << 2))) * 16;
}

// chunk_at of the row `rows` further on (a constant): the tile's base and rows
// are multiples of 128 bytes, so the exclusive-or acts on the offset itself.
template <typename T, int CPR>
__device__ __forceinline__ uint32_t row_at(uint32_t at, int rows, bool value) {
    const int x = sizeof(T) == 2 ? rows & 7 : value ? ((rows >> 1) & 3) << 1 : (rows & 1) << 2;
    return (at ^ (x << 4)) + rows * CPR * 16;
}

// tf32_parts of a factor whose products are not summed apart: an infinite x has no
// second part, so that its products stay infinite.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    tf32_parts(x, hi, lo);
    const float l = __uint_as_float(lo);
    lo = l == l ? lo : 0;
}
// Two values in two bf16 parts each, packed.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pk(x, y);
    lo = pk(x - bf16lo_to_f32(hi), y - bf16hi_to_f32(hi));
}

// ------------------------------------------------------------------ kernel
template <typename T, int D, bool kWide>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_kernel(const __grid_constant__ DecodeParams p) {
    using C = Dec<T, D, kWide>;
    extern __shared__ __align__(128) uint8_t sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c4 = lane & 3;
    uint8_t *ring = sm + warp * kStages * 2 * kHalf;
    uint32_t *mask = reinterpret_cast<uint32_t *>(sm + C::kOffMask) + warp * kStages;
    float *sO = reinterpret_cast<float *>(sm + C::kOffO);     // [warp][8][CW]
    float *sM = reinterpret_cast<float *>(sm + C::kOffM);     // [warp][16][2]
    const int R = p.Hkv * p.hb;
    wait_previous_kernel();
    pdl_launch_dependents();   // the join may be scheduled; it waits for this grid

    // This CTA's stretch [b0, b1) of the block list, and the entry that holds b0:
    // prefix sums over the entries, 128 at a time (up to 128 entries their lengths
    // are loaded once, which a short call's latency consists of).
    Start *st = reinterpret_cast<Start *>(sO);
    Cursor L;
    int nb;
    {
        Entry mine;
        mine.nblk = 0;
        if (threadIdx.x < p.n) mine = load_entry(p, threadIdx.x, blockIdx.x == 0);
        int rest = 0;
        for (int e = threadIdx.x + kThreads; e < p.n; e += kThreads)
            rest += load_entry(p, e, blockIdx.x == 0).nblk;
        long long all = 0;
        if (p.n > kThreads) all = (long long)cta_sum(mine.nblk + rest, st->sum) * R;
        long long before = 0;          // blocks per head block of the entries before
        long long b0 = 0;
        nb = 0;
        for (int base = 0; base < p.n; base += kThreads) {
            if (base > 0) {
                mine.nblk = 0;
                if (base + threadIdx.x < p.n) mine = load_entry(p, base + threadIdx.x, false);
            }
            int incl = mine.nblk;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();
            if (lane == 31) st->sum[warp] = incl;
            if (threadIdx.x == 0) st->e = -1;
            __syncthreads();
            const int s0 = st->sum[0], s1 = st->sum[1], s2 = st->sum[2], s3 = st->sum[3];
            incl += (warp > 0 ? s0 : 0) + (warp > 1 ? s1 : 0) + (warp > 2 ? s2 : 0);
            const int total = s0 + s1 + s2 + s3;
            if (base == 0) {
                if (p.n <= kThreads) all = (long long)total * R;
                b0 = stretch(all, blockIdx.x, p.ctas);
                nb = int(stretch(all, blockIdx.x + 1, p.ctas) - b0);
                if (nb == 0) return;
            }
            const long long end = (before + incl) * R, begin = end - (long long)mine.nblk * R;
            if (begin <= b0 && b0 < end) {
                st->e = base + threadIdx.x;
                st->off = int(b0 - begin);
                st->x = mine;
            }
            before += total;
            __syncthreads();
            if (st->e >= 0) break;
        }
        L.e = st->e;
        if (L.e < 0) return;           // not reached: b0 < all
        L.x = st->x;
        L.r = st->off / L.x.nblk;
        L.blk = st->off % L.x.nblk;
        __syncthreads();
    }
    Cursor W = L;                      // the tile in use; L the next tile to copy
    int first_blk = W.blk;             // first block of the current segment here
    int start_b = 0;                   // the iteration it began in
    int angle_e = -1;                  // the entry cs and sn belong to
    float cs = 1.f, sn = 0.f;

    // Page and slot of this lane's key of the tile at L, loaded one tile early so
    // that the copies do not wait for the table.
    int page = -1, slot = 0;
    bool wanted = false;               // this lane's place holds a visible key
    auto lookup = [&]() {
        const int key = L.x.key(L.blk * C::BLK + warp * C::KT + lane);
        page = -1;
        wanted = lane < C::KT && key >= 0;
        if (wanted) {
            page = __ldg(p.table + (long long)L.x.id * p.MP + (key >> p.ps_log2));
            slot = key & ((1 << p.ps_log2) - 1);
        }
    };
    // pages of a tile or more: all its keys are neighbours in one page, so one page
    // number and one address serve all rows
    const bool run = (1 << p.ps_log2) >= C::KT;
    // This lane's chunk of row lane / CPR: later rows differ by whole rows and an
    // exclusive-or with a constant (chunk_at).
    const int my_row = lane / C::CPR, my_chunk = lane % C::CPR;
    const uint32_t at_k = chunk_at<T, C::CPR>(my_row, my_chunk, false);
    const uint32_t at_v = chunk_at<T, C::CPR>(my_row, my_chunk, true);
    const long long step_k = p.ks[1] * (C::ES * C::RPI), step_v = p.vs[1] * (C::ES * C::RPI);
    int to_copy = nb;
    lookup();
    // q of segment (e, r), as it is, on the way to shared memory (it joins the
    // thread's next copy group)
    auto copy_q = [&](int e, int r) {
        const int kvh = r / p.hb, h0 = kvh * p.G + (r % p.hb) * C::HB;
        const int nh = min(C::HB, (kvh + 1) * p.G - h0);
        const uint32_t dst = smem_u32(sm + C::kOffRaw);
        for (int i = threadIdx.x; i < C::HB * C::CPR; i += kThreads) {
            const int h = i / C::CPR, c = i % C::CPR;
            const char *src = p.q + (e * p.qs[0] + (h0 + h) * p.qs[1]) * C::ES + 16 * c;
            cp_async16(dst + 16 * i, h < nh ? src : p.q, h < nh ? 16 : 0);
        }
    };
    copy_q(W.e, W.r);
    auto copy_tile = [&](int stage) {
        if (to_copy > 0) {
            if (wanted && (page < 0 || page >= p.P)) {
                page = -1;
                raise_status(p.status, LCX_ERR_INVALID_ARG);
            }
            const uint32_t seen = __ballot_sync(0xffffffffu, page >= 0);
            const int kvh = L.r / p.hb;
            const uint32_t dst = smem_u32(ring + stage * 2 * kHalf);
            const char *k0 = p.kp + (kvh * p.ks[2]) * C::ES + 16 * my_chunk;
            const char *w0 = p.vp + (kvh * p.vs[2]) * C::ES + 16 * my_chunk;
            if (run) {
                // the first visible key's page and the slot of row 0
                const int first = max(__ffs(seen) - 1, 0);
                const long long a = max(__shfl_sync(0xffffffffu, page, first), 0);
                const long long sl =
                    seen ? __shfl_sync(0xffffffffu, slot, first) - first + my_row : my_row;
                const char *k = k0 + (a * p.ks[0] + sl * p.ks[1]) * C::ES;
                const char *w = w0 + (a * p.vs[0] + sl * p.vs[1]) * C::ES;
                const uint32_t rows = seen >> my_row;
#pragma unroll
                for (int i = 0; i < C::NI; ++i) {
                    const int bytes = (rows >> (i * C::RPI)) & 1 ? 16 : 0;
                    cp_async16(dst + row_at<T, C::CPR>(at_k, i * C::RPI, false), k, bytes);
                    cp_async16(dst + kHalf + row_at<T, C::CPR>(at_v, i * C::RPI, true), w, bytes);
                    k += step_k;
                    w += step_v;
                }
            } else {
#pragma unroll
                for (int i = 0; i < C::NI; ++i) {
                    const int r = i * C::RPI + my_row;
                    const int pg = __shfl_sync(0xffffffffu, page, r);
                    const int sl = __shfl_sync(0xffffffffu, slot, r);
                    const int bytes = pg >= 0 ? 16 : 0;
                    const long long a = max(pg, 0);
                    const char *k = k0 + (a * p.ks[0] + sl * p.ks[1]) * C::ES;
                    const char *w = w0 + (a * p.vs[0] + sl * p.vs[1]) * C::ES;
                    cp_async16(dst + row_at<T, C::CPR>(at_k, i * C::RPI, false),
                               bytes ? k : p.kp, bytes);
                    cp_async16(dst + kHalf + row_at<T, C::CPR>(at_v, i * C::RPI, true),
                               bytes ? w : p.vp, bytes);
                }
            }
            if (lane == 0) mask[stage] = seen;
            if (--to_copy > 0) {
                L.next(p);
                lookup();
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) copy_tile(s);

    constexpr int NT = D / 8;          // output column tiles
    constexpr uint32_t kAllKeys = C::KT == 32 ? 0xffffffffu : (1u << (C::KT % 32)) - 1;
    constexpr int QF = C::ES == 2 ? (kWide ? 1 : D / 16) : D / 8;
    uint32_t qf[QF][4];                // q' as A fragments (wide: read per tile)
    float acc[NT][4];
    float m[2], l[2];                  // rows g and g + 8 (narrow: row g alone)
    const uint32_t sq = smem_u32(sm + C::kOffQ);
    // where this lane reads its fragments in a tile (16-bit: ldmatrix rows; fp32:
    // 16-byte pieces); other places differ by constants
    const uint32_t rd_k = C::ES == 2 ? chunk_at<T, C::CPR>(lane & 7, lane >> 3, false)
                                     : chunk_at<T, C::CPR>(g, c4, false);
    const uint32_t rd_v = C::ES == 2 ? chunk_at<T, C::CPR>(lane & 15, lane >> 4, true)
                                     : chunk_at<T, C::CPR>(2 * c4, g, true);

    int stage = 0;
    for (int b = 0; b < nb; ++b) {
        // groups of two iterations ago and before have arrived: this tile, and the q
        // of a segment announced that long ago
        cp_async_wait<kStages - 2>();
        if (b == 0 || W.blk == 0) {
            // -------------------------------------------------- a segment starts
            if (b > 0 && b - start_b < 2) cp_async_wait<0>();
            start_b = b;
            first_blk = W.blk;
            if (W.e != angle_e) {
                // one pair per thread; the entry's heads share its angle
                angle_e = W.e;
                if (p.rotate) rope_sincos(W.x.len - 1, p.theta[threadIdx.x % (D / 2)], &cs, &sn);
            }
            __syncthreads();
            {
                constexpr int kStep = kThreads / (D / 2);
                const int pr = threadIdx.x % (D / 2);
                const int a = p.half ? pr : 2 * pr, b2 = p.half ? pr + D / 2 : 2 * pr + 1;
                const T *raw = reinterpret_cast<const T *>(sm + C::kOffRaw);
#pragma unroll 4
                for (int h = threadIdx.x / (D / 2); h < C::HB; h += kStep) {
                    const float x = static_cast<float>(raw[h * D + a]);
                    const float y = static_cast<float>(raw[h * D + b2]);
                    const float u = x * cs - y * sn, w = x * sn + y * cs;
                    if constexpr (C::ES == 2) {
                        // rows h (hi) and HB + h (lo), chunks swizzled
                        auto put = [&](int col, float z) {
                            const uint32_t hi = pk(z, 0.f);
                            const float zl = z - bf16lo_to_f32(hi);
                            const uint32_t lo = pk(zl == zl ? zl : 0.f, 0.f);
                            const int chunk = col >> 3, in = (col & 7) * 2;
                            auto at = [&](int row) {
                                return reinterpret_cast<uint16_t *>(
                                    sm + C::kOffQ + row * C::ROW +
                                    ((chunk ^ (row & 7)) << 4) + in);
                            };
                            *at(h) = uint16_t(hi);
                            *at(C::HB + h) = uint16_t(lo);
                        };
                        put(a, u);
                        put(b2, w);
                    } else {
                        uint32_t *s = reinterpret_cast<uint32_t *>(sm + C::kOffQ);
                        split_tf32(u, s[h * D + a], s[(8 + h) * D + a]);
                        split_tf32(w, s[h * D + b2], s[(8 + h) * D + b2]);
                    }
                }
            }
            __syncthreads();
            if (b + W.x.nblk - W.blk < nb) {       // the stretch goes on behind this segment
                const bool more = W.r + 1 < R;
                copy_q(more ? W.e : W.e + 1, more ? W.r + 1 : 0);
            }
            if constexpr (C::ES == 2 && !kWide) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int row = lane & 15, chunk = 2 * k + (lane >> 4);
                    ldmatrix4(qf[k], sq + row * C::ROW + ((chunk ^ (row & 7)) << 4));
                }
            } else if constexpr (C::ES == 4) {
                // k slots c4 and c4 + 4 of step 2 i + j hold columns 16 i + 4 c4 + 2 j
                // and that + 1, the order in which a key's 16-byte reads arrive
                const uint32_t *s = reinterpret_cast<const uint32_t *>(sm + C::kOffQ);
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    const int col = 16 * (k >> 1) + 4 * c4 + 2 * (k & 1);
                    qf[k][0] = s[g * D + col];
                    qf[k][1] = s[(8 + g) * D + col];
                    qf[k][2] = s[g * D + col + 1];
                    qf[k][3] = s[(8 + g) * D + col + 1];
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
        }
        // ------------------------------------------------------ one tile
        __syncwarp();
        const uint32_t seen = mask[stage];
        const uint32_t kb = smem_u32(ring + stage * 2 * kHalf), vb = kb + kHalf;
        constexpr int NS = C::KT / 8;      // score tiles of 8 keys
        float s[NS][4];
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
        if constexpr (C::ES == 2) {
            // second sums: the products with q's second part (wide), or every other
            // step (shorter chains of dependent products)
            float s2[NS][4];
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s2[j][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
                uint32_t a0[4], a1[4], l0[4], l1[4];
                if constexpr (kWide) {
                    const int row = lane & 15, hc = lane >> 4;
                    auto at = [&](int r, int chunk) {
                        return sq + r * C::ROW + ((chunk ^ (r & 7)) << 4);
                    };
                    ldmatrix4(a0, at(row, 2 * k + hc));
                    ldmatrix4(a1, at(row, 2 * k + 2 + hc));
                    ldmatrix4(l0, at(16 + row, 2 * k + hc));
                    ldmatrix4(l1, at(16 + row, 2 * k + 2 + hc));
                }
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    uint32_t kf[4];        // 8 keys x 32 columns
                    ldmatrix4(kf, kb + (rd_k ^ ((2 * k & 7) << 4)) + (2 * k >> 3) * 128 +
                                      j * 8 * C::ROW);
                    if constexpr (kWide) {
                        mma_bf16(s[j], a0, kf[0], kf[1]);
                        mma_bf16(s2[j], l0, kf[0], kf[1]);
                        mma_bf16(s[j], a1, kf[2], kf[3]);
                        mma_bf16(s2[j], l1, kf[2], kf[3]);
                    } else {
                        mma_bf16(s[j], qf[k], kf[0], kf[1]);
                        mma_bf16(s2[j], qf[k + 1], kf[2], kf[3]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[j][i] = kWide ? join(s[j][i], s2[j][i]) : s[j][i] + s2[j][i];
        } else {
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                // the products with the keys' second parts summed apart: the tensor
                // core cuts its sums, so short chains lose less
                float low[4] = {0.f, 0.f, 0.f, 0.f}, low2[4] = {0.f, 0.f, 0.f, 0.f};
                float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    float4 x;
                    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                                 : "r"(kb + (rd_k ^ ((4 * i & 7) << 4)) + (4 * i >> 3) * 128 +
                                       j * 8 * C::ROW)
                                 : "memory");
                    uint32_t h[4], w[4];
                    tf32_parts(x.x, h[0], w[0]);
                    tf32_parts(x.y, h[1], w[1]);
                    tf32_parts(x.z, h[2], w[2]);
                    tf32_parts(x.w, h[3], w[3]);
                    mma_tf32(low, qf[2 * i], w[0], w[1]);
                    mma_tf32(low2, qf[2 * i + 1], w[2], w[3]);
                    mma_tf32(s[j], qf[2 * i], h[0], h[1]);
                    mma_tf32(s2, qf[2 * i + 1], h[2], h[3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] = join(s[j][i] + s2[i], low[i] + low2[i]);
            }
        }
        // scores of keys 8 j + 2 c4 + {0, 1}: row g in s[j][0..1], row g + 8 in
        // s[j][2..3] (narrow: the second part of row g)
        constexpr int NR = kWide ? 2 : 1;
        if constexpr (!kWide) {
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) s[j][i] = join(s[j][i], s[j][i + 2]);
        }
        if (seen != kAllKeys) {
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!((seen >> (8 * j + 2 * c4 + i)) & 1)) {
                        s[j][i] = -INFINITY;
                        if constexpr (kWide) s[j][i + 2] = -INFINITY;
                    }
        }
        // The running reference m (log2 units) follows the maximum only when that
        // has grown by more than 2^8: the result is the same, the weights stay
        // below 2^8, and the outputs are rescaled a few times per segment instead
        // of in most tiles (a tile with a new maximum in one of 8 heads).
        float mx[NR];
        bool grew = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float x = fmaxf(s[0][2 * r], s[0][2 * r + 1]);
#pragma unroll
            for (int j = 1; j < NS; ++j) x = fmaxf(x, fmaxf(s[j][2 * r], s[j][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            mx[r] = x * p.c_log2;
            grew |= mx[r] > m[r] + kLazy;
        }
        if (__any_sync(0xffffffffu, grew)) {
            float al[2];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float to = fmaxf(m[r], mx[r]);
                al[r] = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - to);
                m[r] = to;
                l[r] *= al[r];
            }
            if constexpr (!kWide) al[1] = al[0];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[j][0] *= al[0];
                acc[j][1] *= al[0];
                acc[j][2] *= al[1];
                acc[j][3] *= al[1];
            }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float mref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                s[j][2 * r] = ex2_approx(fmaf(s[j][2 * r], p.c_log2, -mref));
                s[j][2 * r + 1] = ex2_approx(fmaf(s[j][2 * r + 1], p.c_log2, -mref));
                l[r] += s[j][2 * r] + s[j][2 * r + 1];
            }
        }
        if constexpr (C::ES == 2) {
#pragma unroll
            for (int j = 0; j < NS; j += 2) {
                uint32_t a[4];
                if constexpr (kWide) {
                    a[0] = pk(s[j][0], s[j][1]);
                    a[1] = pk(s[j][2], s[j][3]);
                    a[2] = pk(s[j + 1][0], s[j + 1][1]);
                    a[3] = pk(s[j + 1][2], s[j + 1][3]);
                } else {
                    split_bf16(s[j][0], s[j][1], a[0], a[1]);
                    split_bf16(s[j + 1][0], s[j + 1][1], a[2], a[3]);
                }
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t vf[4];        // 16 keys x 16 columns
                    ldmatrix4_trans(vf, vb + (rd_v ^ ((t & 7) << 4)) + (t >> 3) * 128 +
                                            j * 8 * C::ROW);
                    mma_bf16(acc[t], a, vf[0], vf[1]);
                    mma_bf16(acc[t + 1], a, vf[2], vf[3]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                // k slots c4 and c4 + 4 hold keys 2 c4 and 2 c4 + 1
                uint32_t a[4];
                tf32_parts(s[j][0], a[0], a[1]);
                tf32_parts(s[j][1], a[2], a[3]);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    // columns 32 i + 4 g + {0..3}: one per output tile 4 i + {0..3}
                    float x[2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                     : "=f"(x[k][0]), "=f"(x[k][1]), "=f"(x[k][2]), "=f"(x[k][3])
                                     : "r"(vb + rd_v + i * 128 + (8 * j + k) * C::ROW)
                                     : "memory");
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        uint32_t h0, w0, h1, w1;
                        split_tf32(x[0][t], h0, w0);
                        split_tf32(x[1][t], h1, w1);
                        // (a fresh sum per tile, added in fp32 with rounding)
                        float o[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_tf32(o, a, w0, w1);
                        mma_tf32(o, a, h0, h1);
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[4 * i + t][k] += o[k];
                    }
                }
            }
        }
        __syncwarp();                      // the tile is read: its stage may be refilled
        copy_tile((stage + kStages - 1) % kStages);
        stage = (stage + 1) % kStages;

        if (W.last() || b == nb - 1) {
            // -------------------------------------------------- a segment ends here
            const bool whole = first_blk == 0 && W.last();
            const int kvh = W.r / p.hb, h0 = kvh * p.G + (W.r % p.hb) * C::HB;
            const int nh = min(C::HB, (kvh + 1) * p.G - h0);
            // the stretch's first segment, or a later one that runs past its end
            const int part = 2 * blockIdx.x + (b - (W.blk - first_blk) > 0 ? 1 : 0);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            }
            if (c4 == 0) {
                sM[(warp * 16 + g) * 2] = m[0];
                sM[(warp * 16 + g) * 2 + 1] = l[0];
                if constexpr (kWide) {
                    sM[(warp * 16 + 8 + g) * 2] = m[1];
                    sM[(warp * 16 + 8 + g) * 2 + 1] = l[1];
                }
            }
#pragma unroll
            for (int pass = 0; pass < NR * (D / C::CW); ++pass) {
                const int r = kWide ? pass / (D / C::CW) : 0, part_c = pass % (D / C::CW);
                // this warp's 8 heads x CW columns
                float *dst = sO + (warp * 8 + g) * C::CW;
#pragma unroll
                for (int j = 0; j < C::CW / 8; ++j) {
                    const int t = part_c * (C::CW / 8) + j;
                    const float x = kWide ? acc[t][2 * r] : join(acc[t][0], acc[t][2]);
                    const float y = kWide ? acc[t][2 * r + 1] : join(acc[t][1], acc[t][3]);
                    if constexpr (C::ES == 2) {
                        // columns 8 t + 2 c4, + 1
                        dst[8 * j + 2 * c4] = x;
                        dst[8 * j + 2 * c4 + 1] = y;
                    } else {
                        // tile 4 i + u holds columns 32 i + 4 n + u, n = 2 c4, 2 c4 + 1
                        const int i = j >> 2, u = j & 3;
                        dst[32 * i + 8 * c4 + u] = x;
                        dst[32 * i + 8 * c4 + 4 + u] = y;
                    }
                }
                __syncthreads();
                // CW / 16 columns of one head per thread
                constexpr int CT = C::CW / 16;
                const int hh = threadIdx.x >> 4, col = (threadIdx.x & 15) * CT;
                const int h = 8 * r + hh;
                float mx = -INFINITY, z = 0.f;
                float o[CT];
#pragma unroll
                for (int i = 0; i < CT; ++i) o[i] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sM[(w * 16 + h) * 2]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float mw = sM[(w * 16 + h) * 2];
                    const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - mx);
                    const float lw = sM[(w * 16 + h) * 2 + 1];
                    // (a warp without a key has l = 0 and o = 0; one whose scores are
                    // all NaN has m = -inf and l = NaN, which must show)
                    z += lw == lw ? f * lw : lw;
                    const float fx = lw == lw ? f : lw;
#pragma unroll
                    for (int i = 0; i < CT; ++i)
                        o[i] += fx * sO[(w * 8 + hh) * C::CW + col + i];
                }
                if (h < nh) {
                    if (whole) {
                        const float inv = z == 0.f ? 0.f : 1.f / z;
                        T *out = reinterpret_cast<T *>(p.o) + W.e * p.os[0] +
                                 (h0 + h) * p.os[1] + part_c * C::CW + col;
#pragma unroll
                        for (int i = 0; i < CT; i += 2) {
                            if constexpr (C::ES == 2)
                                *reinterpret_cast<uint32_t *>(out + i) =
                                    pk(o[i] * inv, o[i + 1] * inv);
                            else
                                *reinterpret_cast<float2 *>(out + i) =
                                    make_float2(o[i] * inv, o[i + 1] * inv);
                        }
                        if (p.lse && part_c == 0 && (threadIdx.x & 15) == 0)
                            p.lse[(long long)W.e * p.Hq + h0 + h] =
                                z == 0.f ? -INFINITY : (mx + log2f(z)) * 0.69314718055994531f;
                    } else {
                        float *out =
                            p.part_o + ((long long)part * C::HB + h) * D + part_c * C::CW + col;
#pragma unroll
                        for (int i = 0; i < CT; i += 2)
                            *reinterpret_cast<float2 *>(out + i) = make_float2(o[i], o[i + 1]);
                        if (part_c == 0 && (threadIdx.x & 15) == 0)
                            *reinterpret_cast<float2 *>(p.part_ml + ((long long)part * C::HB + h) * 2) =
                                make_float2(mx, z);
                    }
                }
                __syncthreads();
            }
        }
        W.next(p);
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------------ join
// One CTA per segment: nothing to do when one CTA held all its blocks, else the
// parts of the CTAs that held some, in order.  Everything up to the parts' weights
// is computed by a thread per part; the outputs are then sums of independent loads.
constexpr int kMaxCtas = 320;       // CTAs of the attention kernel, at most

template <typename T, int D, int HB>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ DecodeParams p) {
    __shared__ int sums[3][kWarps];
    __shared__ int part[kMaxCtas];
    __shared__ float weight[HB][kMaxCtas], stat[HB][2];   // stat: maximum, sum
    const int R = p.Hkv * p.hb, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x / R, r = blockIdx.x % R;
    int v[3] = {0, 0, 0};           // blocks of the entries before, of e, behind
    for (int i = threadIdx.x; i < p.n; i += kThreads) {
        const int x = load_entry(p, i, false).nblk;
        v[0] += i < e ? x : 0;
        v[1] += i == e ? x : 0;
        v[2] += i > e ? x : 0;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (lane == 0) sums[k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = sums[k][0] + sums[k][1] + sums[k][2] + sums[k][3];
    const long long all = (long long)(v[0] + v[1] + v[2]) * R;
    const long long s0 = (long long)v[0] * R + (long long)r * v[1], s1 = s0 + v[1];
    // CTA of block x: the largest c with stretch(c) <= x
    auto owner = [&](long long x) {
        int c = int(x * p.ctas / all);
        while (c + 1 < p.ctas && stretch(all, c + 1, p.ctas) <= x) ++c;
        while (stretch(all, c, p.ctas) > x) --c;
        return c;
    };
    const int c0 = owner(s0), c1 = owner(s1 - 1);
    const int kvh = r / p.hb, h0 = kvh * p.G + (r % p.hb) * HB;
    const int nh = min(HB, (kvh + 1) * p.G - h0);
    constexpr int PT = (HB * D / 4 + kThreads - 1) / kThreads;   // 4-column pieces per thread
    float o[PT][4];
#pragma unroll
    for (int i = 0; i < PT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    wait_previous_kernel();
    if (c0 == c1) return;
    const int cnt = c1 + 1 - c0;
    for (int k = threadIdx.x; k < kMaxCtas; k += kThreads) {
        // part of CTA c: its first segment unless its stretch starts before this
        // one; -1 for a CTA without blocks
        int x = -1;
        if (k < cnt) {
            const int c = c0 + k;
            const long long b0 = stretch(all, c, p.ctas);
            if (b0 < stretch(all, c + 1, p.ctas)) x = 2 * c + (b0 < s0 ? 1 : 0);
        }
        part[k] = x;
    }
    __syncthreads();
    // weights: a warp per head
    for (int h = warp; h < nh; h += kWarps) {
        float2 ml[kMaxCtas / 32];
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxCtas / 32; ++k) {
            const int x = part[lane + 32 * k];
            ml[k] = make_float2(-INFINITY, 0.f);
            if (x >= 0)
                ml[k] = *reinterpret_cast<const float2 *>(p.part_ml + ((long long)x * HB + h) * 2);
            mx = fmaxf(mx, ml[k].x);
        }
#pragma unroll
        for (int t = 16; t > 0; t >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, t));
        float z = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCtas / 32; ++k) {
            const float f = ml[k].x == -INFINITY ? 0.f : ex2_approx(ml[k].x - mx);
            const bool nan = ml[k].y != ml[k].y;             // NaN shows
            z += nan ? ml[k].y : f * ml[k].y;
            weight[h][lane + 32 * k] = nan ? ml[k].y : f;
        }
#pragma unroll
        for (int t = 16; t > 0; t >>= 1) z += __shfl_xor_sync(0xffffffffu, z, t);
        if (lane == 0) {
            stat[h][0] = mx;
            stat[h][1] = z;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int at = threadIdx.x + i * kThreads;
        const int h = at / (D / 4), col = at % (D / 4) * 4;
        if (h >= nh) continue;
#pragma unroll 8
        for (int k = 0; k < cnt; ++k) {
            const int x = part[k];
            if (x < 0) continue;
            const float f = weight[h][k];
            const float4 y =
                *reinterpret_cast<const float4 *>(p.part_o + ((long long)x * HB + h) * D + col);
            o[i][0] += f * y.x;
            o[i][1] += f * y.y;
            o[i][2] += f * y.z;
            o[i][3] += f * y.w;
        }
    }
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int at = threadIdx.x + i * kThreads;
        const int h = at / (D / 4), col = at % (D / 4) * 4;
        if (h >= nh) continue;
        const float z = stat[h][1], inv = z == 0.f ? 0.f : 1.f / z;
        T *out = reinterpret_cast<T *>(p.o) + e * p.os[0] + (h0 + h) * p.os[1] + col;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2 *>(out) =
                make_uint2(pk(o[i][0] * inv, o[i][1] * inv), pk(o[i][2] * inv, o[i][3] * inv));
        else
            *reinterpret_cast<float4 *>(out) = make_float4(o[i][0] * inv, o[i][1] * inv,
                                                           o[i][2] * inv, o[i][3] * inv);
        if (p.lse && col == 0)
            p.lse[(long long)e * p.Hq + h0 + h] =
                z == 0.f ? -INFINITY : (stat[h][0] + log2f(z)) * 0.69314718055994531f;
    }
}

constexpr int kMaxHeads = 16;   // query heads of a segment, at most

// Query heads of a segment: 9 and more per kv head share a wide one (16-bit pools).
int segment_heads(int es, int64_t G) { return es == 2 && G > 8 ? 16 : 8; }

// Two CTAs per SM.
int decode_ctas() { return std::min(2 * device_sms(), kMaxCtas); }

int64_t parts_o_bytes(int ctas, int64_t D) { return 2ll * ctas * kMaxHeads * D * 4; }
int64_t parts_bytes(int ctas, int64_t D) {
    return parts_o_bytes(ctas, D) + 2ll * ctas * kMaxHeads * 2 * 4;
}

template <typename T, int D, bool kWide>
lcx_status launch_decode(DecodeParams &p, cudaStream_t s) {
    using C = Dec<T, D, kWide>;
    p.blk = C::BLK;
    auto kern = paged_decode_kernel<T, D, kWide>;
    const long long segments = (long long)p.n * p.Hkv * p.hb;
    if (segments > 0x7fffffffLL) return fail(LCX_ERR_UNSUPPORTED, "sizes too large");
    // no more CTAs than blocks there can be: a sequence's, and what the visible keys'
    // places add under a window (less than kAlign before lo and behind the sinks); the
    // kernels count the blocks of all entries in 32 bits
    const long long places = ((long long)p.MP << p.ps_log2) + (p.window > 0 ? 2 * kAlign : 0);
    const long long most = places / p.blk + 1;
    if (most * p.n > 0x7fffffffLL)
        return fail(LCX_ERR_UNSUPPORTED, "too many entries for sequences of this length");
    p.ctas = int(std::min<long long>(p.ctas, segments * most));
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "cudaFuncSetAttribute failed: %s", cudaGetErrorString(e));
    e = launch_dependent(kern, dim3(unsigned(p.ctas)), dim3(kThreads), C::kSmem, s, p);
    if (e == cudaSuccess && p.ctas > 1)
        e = launch_dependent(join_kernel<T, D, C::HB>, dim3(unsigned(segments)), dim3(kThreads), 0,
                             s, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(LCX_ERR_CUDA, "paged_decode launch failed: %s", cudaGetErrorString(e));
    return LCX_OK;
}

}  // namespace
}  // namespace lcx

extern "C" int64_t lcx_paged_decode_workspace_bytes(int64_t n, int64_t Hq, int64_t Hkv,
                                                    int64_t D) {
    if (n < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (D != 64 && D != 128) ||
        n > (int64_t(1) << 20) || Hq > 65536)
        return -1;
    return lcx::parts_bytes(lcx::decode_ctas(), D);
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
    if ((st = check_distinct(g->o_strides, g->n, g->Hq, "o")) != LCX_OK) return st;
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
    const int heads = segment_heads(c.es, p.G);
    p.hb = (p.G + heads - 1) / heads;
    p.S = c.S;
    p.MP = c.MP;
    p.P = c.P;
    p.ps_log2 = c.ps_log2;
    const int64_t big = int64_t(1) << 30;   // no cache is longer
    p.window = int(g->window >= big ? 0 : g->window);
    p.sinks = int(std::min(g->sinks, big));
    p.rotate = (g->flags & LCX_DECODE_PREROTATED) || g->rope.mode == LCX_ROPE_NONE ? 0 : 1;
    p.half = g->rope.pairing == LCX_PAIR_HALF;
    float ms = 1.f;
    if (p.rotate) rope_freqs_unchecked(&g->rope, g->rope.seq_len, p.theta, &ms);
    const double scale =
        g->softmax_scale > 0.f ? double(g->softmax_scale) : 1.0 / std::sqrt(double(c.D));
    p.c_log2 = float(scale * double(ms) * 1.4426950408889634);
    p.ctas = decode_ctas();
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                          parts_o_bytes(p.ctas, c.D));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.es == 4)
        return c.D == 128 ? launch_decode<float, 128, false>(p, s)
                          : launch_decode<float, 64, false>(p, s);
    if (heads == 16)
        return c.D == 128 ? launch_decode<__nv_bfloat16, 128, true>(p, s)
                          : launch_decode<__nv_bfloat16, 64, true>(p, s);
    return c.D == 128 ? launch_decode<__nv_bfloat16, 128, false>(p, s)
                      : launch_decode<__nv_bfloat16, 64, false>(p, s);
}
