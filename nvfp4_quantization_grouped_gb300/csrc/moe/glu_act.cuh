// glu_act.cuh -- the gated activation of the projections that carry it in their epilogue.
//   a = min(g, L),  z = alpha a,  s = 1 / (1 + e^-z),  b = clamp(u, -L, L) + off,  v = a s b
// SwiGLU is L = inf, alpha = 1, off = 0.  With E = e^-|z| and r = 1 / (1 + E), s and 1 - s are
// r and E r (z >= 0) or E r and r: neither is a difference.  E is within 2^-22 (1 + |z| / 2)
// of itself (one product and the hardware's base-2 exponential), r within 2^-23 or so.
// NaN stays NaN through the clamps.
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "gsa.h"

namespace glu {

struct Act {
    float limit, alpha, off;
};

// False: parameters that the activation kind does not take.
inline bool act_of(int32_t kind, const gsa_act_params *p, Act &a) {
    if (kind == GSA_ACT_SWIGLU) {
        a = {INFINITY, 1.0f, 0.0f};
        return true;
    }
    if (kind != GSA_ACT_CLAMPED_SWIGLU || !p) return false;
    if (!(p->limit > 0.0f) || !std::isfinite(p->limit) || !std::isfinite(p->alpha) || !std::isfinite(p->glu_linear_offset)) return false;
    a = {p->limit, p->alpha, p->glu_linear_offset};
    return true;
}

struct Parts {
    float a, b, z, s, c;   // c = 1 - s
};

__device__ __forceinline__ Parts parts(const Act &A, float g, float u) {
    Parts t;
    t.a = g > A.limit ? A.limit : g;
    t.b = (u > A.limit ? A.limit : u < -A.limit ? -A.limit : u) + A.off;
    t.z = A.alpha * t.a;
    const float e = __expf(-fabsf(t.z)), r = __fdividef(1.0f, 1.0f + e), er = e * r;
    t.s = t.z < 0.0f ? er : r;
    t.c = t.z < 0.0f ? r : er;
    return t;
}

__device__ __forceinline__ float value(const Act &A, float g, float u) {
    const Parts t = parts(A, g, u);
    return t.a * t.s * t.b;
}

// v, and its derivatives by g and u times t.
__device__ __forceinline__ float gradient(const Act &A, float g, float u, float t, float &dg, float &du) {
    const Parts x = parts(A, g, u);
    const float as = x.a * x.s;
    dg = g > A.limit ? 0.0f : t * x.b * __fmaf_rn(x.z * x.s, x.c, x.s);
    du = u > A.limit || u < -A.limit ? 0.0f : t * as;
    return as * x.b;
}

}  // namespace glu
