// Arithmetic of the gated linear recurrence, in channel pairs (sm_103a).
#pragma once

#include "glr_common.cuh"

namespace kda {
namespace glr {

constexpr int SMS = 152;

// ---- arithmetic of channel pairs ------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsq(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float root(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

constexpr float LOG2E = 1.4426950408889634f;
// 1 / (1 + 2^t): sigmoid(x) for t = -x log2(e)
__device__ __forceinline__ float2 sigmoid_of(float2 t) {
    const float2 d = add2(make_float2(ex2(t.x), ex2(t.y)), f2(1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}
// 2^t up to 2^126, whose reciprocal is not flushed to zero: 1 - sigmoid(x) = 2^t sigmoid(x) to its own digits
__device__ __forceinline__ float2 ex2_most(float2 t) { return make_float2(fminf(ex2(t.x), 8.5e37f), fminf(ex2(t.y), 8.5e37f)); }

// What a channel needs besides its rows: -exp(A_log), and the biases times -log2(e).
struct Gate {
    float2 ea, rb, ib;
};
template <typename Args> __device__ __forceinline__ Gate make_gate(const Args& g, int c) {
    Gate k;
    float* f = reinterpret_cast<float*>(&k);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const bool in = c + e < g.C;
        f[e] = in ? -expf(g.A_log[c + e]) : 0.f;
        f[2 + e] = in && g.r_bias ? -LOG2E * g.r_bias[c + e] : 0.f;
        f[4 + e] = in && g.i_bias ? -LOG2E * g.i_bias[c + e] : 0.f;
    }
    return k;
}

// A token's decay a = exp(la) and m^2 = 1 - a^2, for la <= 0.  Near 1 both come from
// q = exp(la) - 1 = la P(la): P interpolates (exp(x) - 1) / x at the six Chebyshev points
// of [-1/2, 0], its last constant set to 1 (relative error 3.1e-9, in fp32 1.7 x 2^-24).  a = 1 + q is then rounded to
// nearest, where an exponential's error has one sign that a state adds up at every
// token, and m^2 = -q (2 + q) keeps its digits (its negative is given).  WIDE: la may lie below -1/2; a channel
// whose exp(A_log) is at most 1/2 never gets there.
constexpr float NEAR = 0.5f;
template <bool WIDE> __device__ __forceinline__ void decay_of(float2 la, float2& a, float2& neg_m2) {
    float2 p = fma2(la, f2(-0.0011234042f), f2(-0.0081896139f));   // (of -q)
    p = fma2(la, p, f2(-0.0416300744f));
    p = fma2(la, p, f2(-0.1666624248f));
    p = fma2(la, p, f2(-0.4999998212f));
    p = fma2(la, p, f2(-1.f));
    const float2 q = mul2(la, p);
    a = fma2(q, f2(-1.f), f2(1.f));
    neg_m2 = mul2(q, add2(q, f2(-2.f)));
    if (WIDE) {
        const float2 t = mul2(la, f2(LOG2E)), e = make_float2(ex2(t.x), ex2(t.y)), em = fma2(e, e, f2(-1.f));
        a = make_float2(la.x < -NEAR ? e.x : a.x, la.y < -NEAR ? e.y : a.y);
        neg_m2 = make_float2(la.x < -NEAR ? em.x : neg_m2.x, la.y < -NEAR ? em.y : neg_m2.y);
    }
}
// 1 / m, finite at m = 0 (there m2 / m is 0)
__device__ __forceinline__ float2 inv_root(float2 neg_m2) {
    const float2 x = fma2(neg_m2, f2(-1.f), f2(1e-36f));
    return make_float2(rsq(x.x), rsq(x.y));
}
// Whether any of the warp's channels may have a decay's logarithm below -NEAR.
__device__ __forceinline__ bool any_wide(const Gate& k) { return __any_sync(0xffffffffu, !(k.ea.x >= -NEAR && k.ea.y >= -NEAR)); }

// h -> A h + B of a run of tokens; A < 0 marks a run that starts anew (a decay never is).
__device__ __forceinline__ float apply(float A, float B, float h) { return A < 0.f ? B : fmaf(A, h, B); }
__device__ __forceinline__ float2 apply(float2 A, float2 B, float2 h) { return make_float2(apply(A.x, B.x, h.x), apply(A.y, B.y, h.y)); }

// What a token does to a channel pair: h -> a h + b.
struct Step {
    float2 a, b;
};
template <bool WIDE> __device__ __forceinline__ Step step_of(const Gate& k, float2 x, float2 r, float2 i) {
    const float2 w = sigmoid_of(fma2(r, f2(-LOG2E), k.rb)), v = sigmoid_of(fma2(i, f2(-LOG2E), k.ib));
    Step s;
    float2 n;
    decay_of<WIDE>(mul2(k.ea, w), s.a, n);
    s.b = mul2(mul2(make_float2(root(-n.x), root(-n.y)), v), x);
    return s;
}
__device__ __forceinline__ float2 silu(float2 z) { return mul2(z, sigmoid_of(mul2(z, f2(-LOG2E)))); }

}  // namespace glr
}  // namespace kda
