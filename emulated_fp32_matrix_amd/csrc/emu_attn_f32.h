// Products of the attention kernels on the FP32 matrix instruction (gfx950
// only): where memory bounds them, short sequences and few rows.
#pragma once

#include "emu_attn_device.h"

namespace emu {

// On v_mfma_f32_16x16x4_f32: lane l holds A[l % 16][l / 16] and B[l / 16][l %
// 16].  Scores contract over d, in any order that A and B share: lane group h
// = l / 16 takes d = 16 c + 4 h + s in step s, so that a 16-byte read feeds
// four steps.  Results contract over the streamed rows, of which step j takes
// 4 h + j; the rows of their A (the result's d) are numbered so that a read of
// VT neighbouring floats feeds VT tiles: tile (c, u) has d = 16 VT c + VT m + u
// in row m.
__device__ __forceinline__ f32x4_t mfma4(float a, float b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// ND tiles of 16 cover a head (dim <= 16 ND); LD is the tile's row length in
// LDS: four more than a multiple of 16, so that the 16 rows of a score's reads
// lie on different banks.
template <int ND>
struct Head {
    static constexpr int VT = ND % 4 == 0 ? 4 : ND % 2 == 0 ? 2 : 1;
    static constexpr int NC = ND / VT;
    static constexpr int LD = 16 * ND + 4;
};

// A wave's own row as the B operand of scores.
template <int ND>
__device__ __forceinline__ void load_own(f32x4_t (&f)[ND], const float* row, bool valid, int h, int dim)
{
#pragma unroll
    for (int c = 0; c < ND; ++c) f[c] = valid ? load4(row, 16 * c + 4 * h, dim) : f32x4_t{};
}

// acc[n] += (16 streamed rows at `tile`)^T . w[n], w as a score's registers
template <int ND, int NT>
__device__ __forceinline__ void results_of(const float* tile, int m, int h, const f32x4_t (&w)[NT], f32x4_t (&acc)[NT][ND])
{
    constexpr int VT = Head<ND>::VT;
    typedef float vec_t __attribute__((ext_vector_type(VT)));
    const float* at = tile + 4 * h * Head<ND>::LD + VT * m;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < Head<ND>::NC; ++c) {
            float a[VT];
            if constexpr (VT == 1) {
                a[0] = at[j * Head<ND>::LD + 16 * c];
            } else {
                const vec_t v = *reinterpret_cast<const vec_t*>(at + j * Head<ND>::LD + 16 * VT * c);
#pragma unroll
                for (int u = 0; u < VT; ++u) a[u] = v[u];
            }
#pragma unroll
            for (int u = 0; u < VT; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][c * VT + u] = mfma4(a[u], w[n][j], acc[n][c * VT + u]);
        }
}

// A result's column (results_of()) to a row of `dim` floats, times f.
template <int ND>
__device__ __forceinline__ void store_own(const f32x4_t (&acc)[ND], float f, float* row, int h, int dim)
{
    constexpr int VT = Head<ND>::VT;
#pragma unroll
    for (int c = 0; c < Head<ND>::NC; ++c) {
        float v[4 * VT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < VT; ++u) v[j * VT + u] = acc[c * VT + u][j] * f;
#pragma unroll
        for (int e = 0; e < VT; ++e)
            store4(row, 16 * VT * c + 4 * VT * h + 4 * e, dim, f32x4_t{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]});
    }
}

template <int ND, int NT>
__device__ __forceinline__ void clear_own(f32x4_t (&acc)[NT][ND])
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < ND; ++t) acc[n][t] = f32x4_t{};
}

}  // namespace emu
