// glu_act.cuh -- the gated activation of the projections that carry it in their epilogue.
//   a = min(g, L),  z = alpha a,  s = 1 / (1 + e^-z),  b = clamp(u, -L, L) + off,  v = a s b
// SwiGLU is L = inf, alpha = 1, off = 0.  With E = e^-z, s = 1 / (1 + E) and 1 - s = E s: neither
// is a difference of near numbers.  E is the hardware's base-2 exponential (within 2^-22) of a
// product, so within 2^-22 + 3 |z| 2^-24 of itself, the reciprocal within 2^-23; both flush what is
// below 2^-126 to zero (a sigmoid that small is taken as 0; E s, which only comes with it as a
// factor, may then be anything finite).  NaN stays NaN through the clamps.
//   Elements go in pairs: sm_103a multiplies and adds two FP32 values an instruction, which
// halves what the draining warps issue but for the two special functions an element.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "gsa.h"

namespace glu {

struct Act {
    float limit, alpha, off;
    float rate;      // -alpha log2 e
    int clamped;
};

// False: parameters that the activation kind does not take.
inline bool act_of(int32_t kind, const gsa_act_params *p, Act &a) {
    constexpr double kLog2e = 1.4426950408889634;
    if (kind == GSA_ACT_SWIGLU) {
        a = {INFINITY, 1.0f, 0.0f, static_cast<float>(-kLog2e), 0};
        return true;
    }
    if (kind != GSA_ACT_CLAMPED_SWIGLU || !p) return false;
    if (!(p->limit > 0.0f) || !std::isfinite(p->limit) || !std::isfinite(p->alpha) || !std::isfinite(p->glu_linear_offset)) return false;
    a = {p->limit, p->alpha, p->glu_linear_offset, static_cast<float>(-kLog2e * p->alpha), 1};
    return true;
}

__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 d;
    asm("{\n .reg .b64 x, y, d;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 d, x, y;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 x, float y) { return mul2(x, make_float2(y, y)); }

__device__ __forceinline__ float2 add2(float2 x, float y) {
    float2 d;
    asm("{\n .reg .b64 x, y, d;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n add.rn.f32x2 d, x, y;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 d;
    asm("{\n .reg .b64 x, y, z, d;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 d, x, y, z;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float x, float y) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
    return d;
}

// a and b of a pair.
template <bool kClamp> __device__ __forceinline__ void clamp_pair(const Act &A, float2 g, float2 u, float2 &a, float2 &b) {
    if constexpr (kClamp) {
        a = make_float2(min_nan(g.x, A.limit), min_nan(g.y, A.limit));
        b = add2(make_float2(max_nan(min_nan(u.x, A.limit), -A.limit), max_nan(min_nan(u.y, A.limit), -A.limit)), A.off);
    } else {
        a = g, b = u;
    }
}

template <bool kClamp> __device__ __forceinline__ float2 value(const Act &A, float2 g, float2 u) {
    float2 a, b;
    clamp_pair<kClamp>(A, g, u, a, b);
    const float2 t = mul2(a, A.rate);
    const float2 d = add2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), 1.0f);
    return mul2(mul2(a, make_float2(rcp_fast(d.x), rcp_fast(d.y))), b);
}

// v, and its derivatives by g and u times t.
template <bool kClamp> __device__ __forceinline__ float2 gradient(const Act &A, float2 g, float2 u, float2 t, float2 &dg, float2 &du) {
    float2 a, b;
    clamp_pair<kClamp>(A, g, u, a, b);
    const float2 x = mul2(a, A.rate);
    const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
    const float2 d = add2(e, 1.0f);
    const float2 s = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    const float2 as = mul2(a, s), c = mul2(make_float2(fminf(e.x, 0x1p126f), fminf(e.y, 0x1p126f)), s);
    dg = mul2(mul2(t, b), fma2(kClamp ? mul2(as, A.alpha) : as, c, s));
    du = mul2(t, as);
    if constexpr (kClamp) {
        if (g.x > A.limit) dg.x = 0.0f;
        if (g.y > A.limit) dg.y = 0.0f;
        if (fabsf(u.x) > A.limit) du.x = 0.0f;
        if (fabsf(u.y) > A.limit) du.y = 0.0f;
    }
    return mul2(as, b);
}

}  // namespace glu
