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

__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.707106769084930419921875f); }
__device__ __forceinline__ float normal_pdf(float z) { return 0.398942291736602783203125f * exp_f32(-0.5f * z * z); }

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
    if constexpr (ACT == EMU_ACT_GELU) return z * normal_cdf(z);
    if constexpr (ACT == EMU_ACT_GELU_TANH) {
        // (1 + tanh q) / 2 = sigmoid(2 q)
        const float q2 = 2.0f * kGeluC * (z + kGeluA * z * z * z);
        return z * sigmoid(q2);
    }
    if constexpr (ACT == EMU_ACT_TANH) return tanhf(z);
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
        z = limit_z(z, 88.0f);
        const float s = sigmoid(z);
        const float t = sigmoid(-z);   // 1 - s without its cancellation
        if constexpr (D == 1) return s * __builtin_fmaf(z, t, 1.0f);
        return s * t * __builtin_fmaf(z, t - s, 2.0f);
    }
    if constexpr (ACT == EMU_ACT_GELU) {
        z = limit_z(z, 16.0f);
        if constexpr (D == 1) return __builtin_fmaf(z, normal_pdf(z), normal_cdf(z));
        return normal_pdf(z) * __builtin_fmaf(-z, z, 2.0f);
    }
    if constexpr (ACT == EMU_ACT_GELU_TANH) {
        // f = z s, s = sigmoid(p), p = 2 c (z + a z^3): f' = s + z s t p',
        // f'' = s t (2 p' + z (p'' + (t - s) p'^2)), t = 1 - s
        z = limit_z(z, 16.0f);
        const float p = 2.0f * kGeluC * (z + kGeluA * z * z * z);
        const float p1 = 2.0f * kGeluC * __builtin_fmaf(3.0f * kGeluA * z, z, 1.0f);
        const float s = sigmoid(p), t = sigmoid(-p);
        if constexpr (D == 1) return __builtin_fmaf(z * p1, s * t, s);
        const float p2 = 12.0f * kGeluC * kGeluA * z;
        return s * t * __builtin_fmaf(z, __builtin_fmaf((t - s) * p1, p1, p2), 2.0f * p1);
    }
    if constexpr (ACT == EMU_ACT_TANH) {
        // 1 - tanh^2 = 4 s t with s = sigmoid(2 z), without the cancellation
        z = limit_z(z, 44.0f);
        const float u = 4.0f * sigmoid(2.0f * z) * sigmoid(-2.0f * z);
        if constexpr (D == 1) return z != z ? z : u;   // (the sigmoids drop a NaN)
        return -2.0f * tanhf(z) * u;
    }
    return 0.0f;
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
