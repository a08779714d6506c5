// Device-side building blocks of the transformer-block operators
// (include/emu_block.h): row access at any alignment, sums over the lanes
// that share a row, and the activations with their first two derivatives
// (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "emu_block.h"
#include "emu_device.h"

namespace emu {

// Four floats at a 4-byte aligned address: a global 16-byte access needs no
// more than that on gfx950, so rows of any leading dimension take it.
typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));

// Columns col .. col+3 of a row of `cols` floats; past the end: fill.
__device__ __forceinline__ f32x4_t load4(const float* row, int col, int cols, float fill = 0.0f)
{
    if (col + 4 <= cols) return *reinterpret_cast<const f32x4u_t*>(row + col);
    f32x4_t v = {fill, fill, fill, fill};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < cols) v[e] = row[col + e];
    return v;
}

__device__ __forceinline__ void store4(float* row, int col, int cols, f32x4_t v)
{
    if (col + 4 <= cols) {
        *reinterpret_cast<f32x4u_t*>(row + col) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < cols) row[col + e] = v[e];
}

// x of lane (l + N) % 16 within each row of 16 lanes (DPP row_ror).
template <int N>
__device__ __forceinline__ float ror16(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xf, 0xf, true));
}

// x + x of the lane 16 (32) away.
__device__ __forceinline__ float add_lane16(float x)
{
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float add_lane32(float x)
{
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Sum over the LANES (16, 32 or 64) neighbouring lanes, in every one of them.
template <int LANES>
__device__ __forceinline__ float lane_sum(float x)
{
    static_assert(LANES == 16 || LANES == 32 || LANES == 64, "lanes of one wave");
    x = x + ror16<8>(x);
    x = x + ror16<4>(x);
    x = x + ror16<2>(x);
    x = x + ror16<1>(x);
    if constexpr (LANES >= 32) x = add_lane16(x);
    if constexpr (LANES == 64) x = add_lane32(x);
    return x;
}

// ---- activations ---------------------------------------------------------------

// e^x to about two units in the last place; the rounding error of x log2(e)
// is carried into the result.  x is limited to +-100, where e^x is infinite
// (zero) in FP32 already, so that the correction stays finite.  NaN is not
// kept: callers multiply by a value that keeps it.
__device__ __forceinline__ float exp_f32(float x)
{
    x = __builtin_amdgcn_fmed3f(x, -100.0f, 100.0f);
    const float l2e = 1.44269502162933349609375f;             // log2(e) rounded
    const float l2e_lo = 1.92596299112661746887e-8f;          // log2(e) - l2e
    const float t = x * l2e;
    const float d = __builtin_fmaf(x, l2e_lo, __builtin_fmaf(x, l2e, -t));
    return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(d, 0.693147182464599609375f, 1.0f);
}

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-z)); }

// s = sigmoid(z) and t = 1 - s, both without cancellation.
__device__ __forceinline__ void sigmoid_pair(float z, float& s, float& t)
{
    const float e = exp_f32(-z);
    s = __builtin_amdgcn_rcpf(1.0f + e);
    t = s < 0.5f ? 1.0f - s : e * s;   // (e <= 1 in the second)
}

// The normal distribution's density and cumulative function.  For z <= 0
//   Phi(z) = e^(-z^2/2) G(|z|),  G(y) = erfcx(y / sqrt 2) / 2,
// and Phi(z) = 1 - Phi(-z) above, so that both tails keep their relative
// accuracy.  G is smooth in t = 1 / (1 + 0.35 y): t times a polynomial of
// degree 8, fitted here to the least relative error over y <= 14 (3.2e-8; 5.3
// units of 2^-24 with FP32 roundings), beyond which the exponential is zero.
__device__ __forceinline__ void normal(float z, float& cdf, float& pdf)
{
    const float e = exp_f32(-0.5f * z * z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, __builtin_fabsf(z), 1.0f));
    float p = -0.029145918786525726f;
    p = __builtin_fmaf(p, t, 0.14397163689136505f);
    p = __builtin_fmaf(p, t, -0.2557141184806824f);
    p = __builtin_fmaf(p, t, 0.15917402505874634f);
    p = __builtin_fmaf(p, t, -0.023109741508960724f);
    p = __builtin_fmaf(p, t, 0.10550796240568161f);
    p = __builtin_fmaf(p, t, 0.11983288079500198f);
    p = __builtin_fmaf(p, t, 0.13986186683177948f);
    p = __builtin_fmaf(p, t, 0.13962140679359436f);
    const float low = p * t * e;
    cdf = z < 0.0f ? low : 1.0f - low;
    pdf = 0.398942291736602783203125f * e;
}

// tanh z: its odd series' place is taken below |z| = 0.35 by z times a
// polynomial in z^2 (least relative error 4e-10), above by (1 - e) / (1 + e)
// with e = e^(-2 |z|), where 1 - e loses one bit at most.  NaN kept.
__device__ __forceinline__ float tanh_f32(float z)
{
    const float a = __builtin_fabsf(z);
    const float e = exp_f32(-2.0f * a);
    const float big = (1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e);
    const float q = z * z;
    float p = 0.019361333921551704f;
    p = __builtin_fmaf(p, q, -0.053706347942352295f);
    p = __builtin_fmaf(p, q, 0.13332201540470123f);
    p = __builtin_fmaf(p, q, -0.33333316445350647f);
    p = __builtin_fmaf(p * q, z, z);
    return a >= 0.35f ? __builtin_copysignf(big, z) : p;
}

constexpr float kGeluC = 0.797884583473205566406f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// z limited to where the sigmoidal slopes still change in FP32: their tails
// are exact beyond, and products like z * (slope 0) stay finite.  NaN kept.
__device__ __forceinline__ float limit_z(float z, float lim)
{
    const float c = __builtin_amdgcn_fmed3f(z, -lim, lim);
    return z != z ? z : c;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == EMU_ACT_IDENTITY) return z;
    if constexpr (ACT == EMU_ACT_RELU) return z <= 0.0f ? 0.0f : z;   // (NaN kept)
    if constexpr (ACT == EMU_ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == EMU_ACT_GELU) {
        float c, d;
        normal(z, c, d);
        return z * c;
    }
    if constexpr (ACT == EMU_ACT_GELU_TANH) {
        // (1 + tanh q) / 2 = sigmoid(2 q)
        const float q2 = 2.0f * kGeluC * (z + kGeluA * z * z * z);
        return z * sigmoid(q2);
    }
    if constexpr (ACT == EMU_ACT_TANH) return tanh_f32(z);
    return z;
}

// First (D = 1) or second (D = 2) derivative.
template <int ACT, int D>
__device__ __forceinline__ float act_slope(float z)
{
    static_assert(D == 1 || D == 2, "first or second derivative");
    if constexpr (ACT == EMU_ACT_IDENTITY) return D == 1 ? 1.0f : 0.0f;
    if constexpr (ACT == EMU_ACT_RELU) return D == 2 || z <= 0.0f ? 0.0f : 1.0f;
    if constexpr (ACT == EMU_ACT_SILU) {
        float s, t;
        sigmoid_pair(z, s, t);   // (s t is 0 where z t overflows)
        if constexpr (D == 1) return s * __builtin_fmaf(z, t, 1.0f);
        return s * t * __builtin_fmaf(z, t - s, 2.0f);
    }
    if constexpr (ACT == EMU_ACT_GELU) {
        if constexpr (D == 2) z = limit_z(z, 16.0f);
        float c, d;
        normal(z, c, d);
        if constexpr (D == 1) return __builtin_fmaf(z, d, c);
        return d * __builtin_fmaf(-z, z, 2.0f);
    }
    if constexpr (ACT == EMU_ACT_GELU_TANH) {
        // f = z s, s = sigmoid(p), p = 2 c (z + a z^3): f' = s + z s t p',
        // f'' = s t (2 p' + z (p'' + (t - s) p'^2)), t = 1 - s
        z = limit_z(z, 16.0f);
        const float p = 2.0f * kGeluC * (z + kGeluA * z * z * z);
        const float p1 = 2.0f * kGeluC * __builtin_fmaf(3.0f * kGeluA * z, z, 1.0f);
        float s, t;
        sigmoid_pair(p, s, t);
        if constexpr (D == 1) return __builtin_fmaf(z * p1, s * t, s);
        const float p2 = 12.0f * kGeluC * kGeluA * z;
        return s * t * __builtin_fmaf(z, __builtin_fmaf((t - s) * p1, p1, p2), 2.0f * p1);
    }
    if constexpr (ACT == EMU_ACT_TANH) {
        // 1 - tanh^2 = 4 s t with s = sigmoid(2 z), without the cancellation
        z = limit_z(z, 44.0f);
        float s, t;
        sigmoid_pair(2.0f * z, s, t);
        const float u = 4.0f * s * t;
        if constexpr (D == 1) return z != z ? z : u;   // (the sigmoids drop a NaN)
        return -2.0f * tanh_f32(z) * u;
    }
    return 0.0f;
}

// Value and first derivative together.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& v, float& d)
{
    if constexpr (ACT == EMU_ACT_SILU) {
        float s, t;
        sigmoid_pair(z, s, t);
        v = z * s;
        d = s * __builtin_fmaf(z, t, 1.0f);
    } else if constexpr (ACT == EMU_ACT_GELU) {
        float c, f;
        normal(z, c, f);
        v = z * c;
        d = __builtin_fmaf(z, f, c);
    } else if constexpr (ACT == EMU_ACT_GELU_TANH) {
        const float l = limit_z(z, 16.0f);
        const float p = 2.0f * kGeluC * (l + kGeluA * l * l * l);
        const float p1 = 2.0f * kGeluC * __builtin_fmaf(3.0f * kGeluA * l, l, 1.0f);
        float s, t;
        sigmoid_pair(p, s, t);
        v = z * s;
        d = __builtin_fmaf(l * p1, s * t, s);
    } else {
        v = act_value<ACT>(z);
        d = act_slope<ACT, 1>(z);
    }
}

// f with the activation as a compile-time constant: f.operator()<ACT>().
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f)
{
    switch (act) {
    case EMU_ACT_RELU: f.template operator()<EMU_ACT_RELU>(); break;
    case EMU_ACT_SILU: f.template operator()<EMU_ACT_SILU>(); break;
    case EMU_ACT_GELU: f.template operator()<EMU_ACT_GELU>(); break;
    case EMU_ACT_GELU_TANH: f.template operator()<EMU_ACT_GELU_TANH>(); break;
    case EMU_ACT_TANH: f.template operator()<EMU_ACT_TANH>(); break;
    default: f.template operator()<EMU_ACT_IDENTITY>(); break;
    }
}

}  // namespace emu
