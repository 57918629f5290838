// activations.cuh -- the activations of the projections' epilogues and their slopes.
#pragma once
#include "lf_gemm_common.cuh"
#include "lf_ptx_ffn.cuh"

namespace lf {
namespace {

constexpr int ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_NONE = 3;
constexpr float GELU_C2 = 1.5957691216057308f;  // 2 sqrt(2 / pi): gelu_tanh(v) = v sigmoid(GELU_C2 (v + a v^3))
constexpr float GELU_A = 0.044715f;

// 1 / (1 + exp(-v)) in fp32: off by about 2^-21, and for negative v by |v| 2^-24 more,
// what the rounding of its exponent makes of exp(-v).  Below -87, where 1 + exp(-v)
// passes 2^126, it is 0.
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + ex2_approx(-v * LOG2E)); }

// Activations, act(v) = v phi(v), two values at a time: the polynomials of gelu and
// gelu_tanh run in packed operations (2048 x 1024 x 4096 gelu 28.1 -> 25.4 us, 4096 x
// 2048 x 5632 113.3 -> 105.8, e4m3 64.5 -> 60.3); silu's sigmoid, an exponential and a
// reciprocal, is faster one value at a time (2621 x 224 x 12368 40.8 against 41.4).
//
// The standard normal distribution function, with a = |v| and t = 1 / (1 + 0.3 a):
//   Phi(-a) = exp(-a^2 / 2) t Q(t),  Phi(a) = 1 - Phi(-a).
// exp(a^2 / 2) Phi(-a) falls from 1/2 like 1 / a, so divided by t it is smooth over all of
// 0 < t <= 1, and Q of degree 7 comes within 1.8e-7 of it (relative; least squares on
// Chebyshev nodes for a up to 14, reweighted until the errors were level, coefficients
// rounded to fp32; 0.3 was the best of 0.15 to 0.75).  As evaluated here Phi(-a) is off
// by up to 2^-20 + a^2 2^-24: the rest is the rounding of a^2 in the exponent.  One
// polynomial, one exponential and one reciprocal: with normcdff the epilogue of a tile
// took 10 us.
__device__ __forceinline__ float2 normal_cdf(float2 v)
{
    const float2 t = make_float2(__fdividef(1.f, fmaf(0.3f, fabsf(v.x), 1.f)),
                                 __fdividef(1.f, fmaf(0.3f, fabsf(v.y), 1.f)));
    float2 q = fma2(t, both(0.03567476f), both(-0.15720302f));
    q = fma2(t, q, both(0.2063534f));
    q = fma2(t, q, both(-0.05368354f));
    q = fma2(t, q, both(0.12856157f));
    q = fma2(t, q, both(0.09991351f));
    q = fma2(t, q, both(0.12075395f));
    q = fma2(t, q, both(0.1196293f));
    const float2 x = mul2(mul2(v, v), both(-0.5f * LOG2E));
    const float2 e = mul2(mul2(t, q), make_float2(ex2_approx(x.x), ex2_approx(x.y)));
    const float2 r = fma2(e, both(-1.f), both(1.f));
    return make_float2(v.x < 0.f ? e.x : r.x, v.y < 0.f ? e.y : r.y);
}

// phi(v)
template <int ACT>
__device__ __forceinline__ float2 act_phi(float2 v)
{
    if (ACT == ACT_GELU)
        return normal_cdf(v);
    if (ACT == ACT_GELU_TANH)
        v = mul2(both(GELU_C2), fma2(mul2(mul2(both(GELU_A), v), v), v, v));
    return make_float2(sigmoid_f(v.x), sigmoid_f(v.y));
}

// d phi / d v, given p = phi(v)
template <int ACT>
__device__ __forceinline__ float act_dphi(float v, float p)
{
    if (ACT == ACT_SILU)
        return p * (1.f - p);
    if (ACT == ACT_GELU)
        return 0.3989422804014327f * ex2_approx(-0.5f * LOG2E * v * v);
    // (p (1 - p) is 0 long before v^2 would pass fp32's range, and 0 times infinity no number)
    v = fminf(fabsf(v), 0x1p60f);
    return p * (1.f - p) * GELU_C2 * fmaf(3.f * GELU_A * v, v, 1.f);
}

}  // namespace
}  // namespace lf
