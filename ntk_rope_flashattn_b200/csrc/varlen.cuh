// varlen.cuh -- the plan of a packed-prompt call (lcx_varlen_plan) and what its
// kernels share.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "lcx_internal.h"

namespace lcx {

// Plan layout (int32): 8 zeros, cu_q[n + 1], cu_k[n + 1], then, from a
// 16-byte boundary each, the units of 128 and of 256 query rows, heaviest first.
struct VarlenUnit {
    int q0, rows;     // first packed query row, rows (1..128 or 1..256)
    int k0, nk;       // first packed key row, keys of the sequence
    int pos0;         // position of row q0 (lens_k - lens_q + its index)
    int pad[3];
};
static_assert(sizeof(VarlenUnit) == 32, "plan layout");

inline int64_t plan_cu_q() { return 8; }
inline int64_t plan_cu_k(int64_t n) { return 8 + n + 1; }
inline int64_t plan_units(int64_t n, int which, int64_t n128) {
    const int64_t base = (8 + 2 * (n + 1) + 7) / 8 * 8;
    return base + (which ? 8 * n128 : 0);
}

struct VarlenParams {
    const char *q, *k, *v;
    char *o;
    float *lse;
    int *status;
    const VarlenUnit *units;
    int n_units;
    long long qs[2], ks[2], vs[2], os[2];   // element strides: token, head
    int Tq, Tk, Hq, Hkv, G;
    int causal;
    int window, sinks;
    int rotate_q, half;
    float c_log2;                           // logit scale in log2 units
    unsigned long long timeout_ns;
    float ms;                               // the mode's attention scale (1: not rotated)
    double theta[64];
};

// The unit as the plan holds it, or one without rows when it does not fit the
// tensors of the call (a plan that is not the one of `info`).
__device__ __forceinline__ VarlenUnit load_unit(const VarlenParams &p, int u) {
    const int4 *src = reinterpret_cast<const int4 *>(p.units + u);
    const int4 a = __ldg(src), b = __ldg(src + 1);
    VarlenUnit r;
    r.q0 = a.x;
    r.rows = a.y;
    r.k0 = a.z;
    r.nk = a.w;
    r.pos0 = b.x;
    const bool ok = r.q0 >= 0 && r.rows >= 0 && r.q0 <= p.Tq - r.rows && r.k0 >= 0 && r.nk >= 0 &&
                    r.k0 <= p.Tk - r.nk;
    if (!ok) r.rows = r.nk = 0;
    return r;
}

}  // namespace lcx
