// Activation side of the layer's kernels: the effective scale and the codec of
// an 8-element vector under an activation quantiser, and SiLU.
#pragma once

#include "fq_common.h"
#include "fq_internal.h"

namespace fq {

namespace {

// The per-expert tensor scale the quantiser reads (0 where it has none):
// through the scalar cache when e is wave-uniform.
template <int KIND>
__device__ __forceinline__ float act_t(const ActQ& a, int e) {
    return (KIND == K_NVFP4 || (KIND != K_NONE && a.q.source != S_DYNAMIC)) ? sload(a.s, e) : 0.0f;
}

// Effective scale of an 8-element vector under the layer's activation
// quantiser, given its expert's tensor scale t = act_t(a, e).  `bm` is the
// vector's 16-block amax (NVFP4), `gm` its group amax (INT/FP8 per-group
// dynamic), `row_s` the dynamic per-row scale.
template <int KIND>
__device__ __forceinline__ float act_scale_t(const ActQ& a, float t, float bm, float gm, float row_s, float* dfac) {
    *dfac = 1.0f;
    if (KIND == K_NVFP4) {
        const float d6 = 6.0f * t;
        // fl32(bm / d6): Markstein's corrected quotient when every lane's d6
        // is normal, IEEE division otherwise.  Where the corrected form
        // overflows (a NaN) the quotient is far above 448, and fminf takes
        // 448 from both.
        float qd;
        if (__all(d6 >= 0x1p-120f && d6 <= 0x1p120f)) {
            const float inv = rcp_rn(d6);
            const float q0 = bm * inv;
            qd = __builtin_fmaf(__builtin_fmaf(-q0, d6, bm), inv, q0);
        } else {
            qd = bm / d6;
        }
        const float d = e4m3_round(fminf(qd, 448.0f));
        *dfac = d;
        return t * d;
    }
    if (a.q.source != S_DYNAMIC) return t;               // per-expert per-tensor scale
    if (a.q.gran == G_ROW) return row_s;
    return gm / a.q.qdiv;
}

// the same for expert e
template <int KIND>
__device__ __forceinline__ float act_scale(const ActQ& a, int e, float bm, float gm, float row_s, float* dfac) {
    return act_scale_t<KIND>(a, act_t<KIND>(a, e), bm, gm, row_s, dfac);
}

template <int KIND>
__device__ __forceinline__ void quant8(const float* f, float s, float qmin, float qmax, float* y) {
    quant_group<KIND, 8>(f, s, qmin, qmax, [&](int i, const Elem& e) { y[i] = e.q * s; });
}

__device__ __forceinline__ float amax8(const float* f) {
    float m = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
}

// ------------------------------------------------------------------ SiLU ----
// silu(g) = g / (1 + e^-g) in fp32, within (8 + 2|g|) 2^-24 of the exact value
// (relative; results below 2^-126 within that plus (1 + |g|) 2^-149).
// e^-|g| = 2^y, y = -|g| log2(e) clamped at -200 (2^-200 is 0 in fp32):
// 2^y = 2^rint(y) * P(y - rint(y)), P the degree-7 Taylor polynomial of 2^f
// (coefficients (ln 2)^i / i!, rounded to fp32), Horner with one fused
// multiply-add per degree; the 2|g| term is the rounding of y.
__device__ __forceinline__ float exp2_taylor(float y) {
    const float n = rintf(y);
    const float f = y - n;
    float p = 0x1.ffcbfcp-17f;
    p = __builtin_fmaf(p, f, 0x1.430912p-13f);
    p = __builtin_fmaf(p, f, 0x1.5d87fep-10f);
    p = __builtin_fmaf(p, f, 0x1.3b2ab6p-7f);
    p = __builtin_fmaf(p, f, 0x1.c6b08ep-5f);
    p = __builtin_fmaf(p, f, 0x1.ebfbe0p-3f);
    p = __builtin_fmaf(p, f, 0x1.62e430p-1f);
    p = __builtin_fmaf(p, f, 1.0f);
    return ldexpf(p, (int)n);
}

// silu(g) and sigmoid(g), as the forward and the backward both form them,
// without branches and without overflow: with e = e^-|g| in [0, 1] and
// den = 1 + e in [1, 2],
//     g >= 0:  silu = g / den,      sigmoid = 1 / den
//     g <  0:  silu = g e / den,    sigmoid = e / den
// (both are g / (1 + e^-g)).  The quotient is Markstein's correction of
// num RN(1/den) (the rounded quotient while it is normal): where e rounds
// away (den = 1) silu is g exactly, as the exact value rounds; the sign is
// g's, so silu(-0) = -0.
__device__ __forceinline__ float silu_sig(float g, float* sig) {
    const float e = exp2_taylor(fmaxf(-fabsf(g) * 0x1.715476p+0f, -200.0f));
    const float den = 1.0f + e;
    const float inv = rcp_rn(den);
    const float sel = g < 0.0f ? e : 1.0f;
    const float num = g * sel;
    const float q0 = num * inv;
    const float r = __builtin_fmaf(__builtin_fmaf(-q0, den, num), inv, q0);
    *sig = sel * inv;
    return __builtin_copysignf(r, g);
}

}  // namespace

}  // namespace fq
