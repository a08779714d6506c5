// The element-wise passes of the transformer-block operators
// (include/emu_block.h): the epilogue of a product that was written out, and
// the backward passes of the activation and of the gated product with their
// own backward passes.
//
// Bound by memory: each array is read or written once, four columns per
// thread and access, several rows per workgroup so that the row and column of
// an access come from one 32-bit division.
#include "emu_block_device.h"
#include "emu_block_launch.h"

namespace emu {
namespace {

constexpr int kGroupsPerWg = 2048;   // 16-byte groups of a workgroup: 8 per thread

struct RowsPlan {
    int rows_per_wg;
    int64_t wgs;
    int groups;      // 16-byte groups per row
};

RowsPlan plan_rows(int64_t rows, int64_t cols)
{
    RowsPlan p;
    p.groups = (int)((cols + 3) / 4);
    int64_t r = kGroupsPerWg / p.groups;
    if (r < 1) r = 1;
    if (r > rows) r = rows;
    p.rows_per_wg = (int)r;
    p.wgs = (rows + r - 1) / r;
    return p;
}

// f(row, col) for the workgroup's share of rows x cols, col a multiple of 4.
template <class F>
__device__ __forceinline__ void each_group(int64_t rows, int groups, int rows_per_wg, F&& f)
{
    for (int64_t wg = blockIdx.x; wg * rows_per_wg < rows; wg += gridDim.x) {
        const int64_t r0 = wg * rows_per_wg;
        const int here = (int)(rows - r0 < rows_per_wg ? rows - r0 : rows_per_wg);
        if (rows_per_wg == 1) {
            for (int c = threadIdx.x; c < groups; c += 256) f(r0, c * 4);
        } else {
            for (int i = threadIdx.x; i < here * groups; i += 256) {
                const int r = (int)((unsigned)i / (unsigned)groups);
                f(r0 + r, (i - r * groups) * 4);
            }
        }
    }
}

__device__ __forceinline__ f32x4_t add_bias(const BlockEpilogue& ep, f32x4_t t, int64_t off, int col, int cols)
{
    if (ep.bias != nullptr) t = t + load4(ep.bias + off, col, cols);
    return t;
}

// t null: a product of zeros (K = 0).
__global__ __launch_bounds__(256) void epilogue_kernel(int64_t M, int N, const float* t, int64_t ldt,
                                                       BlockEpilogue ep, int groups, int rows_per_wg)
{
    with_act(ep.act, [&]<int ACT>() {
        each_group(M, groups, rows_per_wg, [&](int64_t r, int c) {
            f32x4_t z = add_bias(ep, t != nullptr ? load4(t + r * ldt, c, N) : f32x4_t{}, 0, c, N);
            if (ep.Z != nullptr) store4(ep.Z + r * ep.ldz, c, N, z);
            f32x4_t o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = act_value<ACT>(z[e]);
            if (ep.gated) {
                f32x4_t u = add_bias(ep, t != nullptr ? load4(t + r * ldt + N, c, N) : f32x4_t{}, N, c, N);
                if (ep.Z != nullptr) store4(ep.Z + r * ep.ldz + N, c, N, u);
                o = o * u;
            } else if (ep.R != nullptr) {
                o = o + load4(ep.R + r * ep.ldr, c, N);
            }
            store4(ep.C + r * ep.ldc, c, N, o);
        });
    });
}

// Workgroup (i, y): rows of split tile i, 256 threads with one 4-column group
// of C each; parts as ksplit_reduce_kernel's ws.
template <bool GATED>
__global__ __launch_bounds__(256) void split_epilogue_kernel(const float* __restrict__ parts, int segs, int nsplit,
                                                             int split_from, int tiles_n, int th, int64_t M, int64_t N,
                                                             BlockEpilogue ep)
{
    constexpr int TILE = 128, CW = GATED ? 64 : 128, PER_ROW = CW / 4, ROWS = 256 / PER_ROW;
    const int tile = split_from + blockIdx.x;
    const int tm = tile / tiles_n, tn = tile - tm * tiles_n;
    const int r = blockIdx.y * ROWS + (int)threadIdx.x / PER_ROW;
    const int cg = (int)(threadIdx.x % PER_ROW) * 4;
    const int64_t row = (int64_t)tm * th + r, n0 = (int64_t)tn * CW;
    if (row >= M || n0 + cg >= N) return;
    const int cols = N - n0 < CW ? (int)(N - n0) : CW;
    const int64_t stride = (int64_t)nsplit * th * TILE;
    const float* src = parts + ((int64_t)blockIdx.x * th + r) * TILE + (GATED ? (cg >> 4) * 32 + (cg & 15) : cg);
    auto total = [&](const float* q) {
        f32x4_t t = *reinterpret_cast<const f32x4_t*>(q);
        for (int s = 1; s < segs; ++s) t = t + *reinterpret_cast<const f32x4_t*>(q + s * stride);
        return t;
    };
    f32x4_t z = add_bias(ep, total(src), n0, cg, cols);
    f32x4_t u = {};
    if (GATED) u = add_bias(ep, total(src + 16), n0 + N, cg, cols);
    if (ep.Z != nullptr) {
        store4(ep.Z + row * ep.ldz + n0, cg, cols, z);
        if (GATED) store4(ep.Z + row * ep.ldz + n0 + N, cg, cols, u);
    }
    with_act(ep.act, [&]<int ACT>() {
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = act_value<ACT>(z[e]);
    });
    if (GATED)
        z = z * u;
    else if (ep.R != nullptr)
        z = z + load4(ep.R + row * ep.ldr + n0, cg, cols);
    store4(ep.C + row * ep.ldc + n0, cg, cols, z);
}

__global__ __launch_bounds__(256) void copy_rows_kernel(int64_t M, int K, const float* __restrict__ A, int64_t lda,
                                                        float* __restrict__ dst, int64_t ldd, int groups,
                                                        int rows_per_wg)
{
    each_group(M, groups, rows_per_wg,
               [&](int64_t r, int c) { *reinterpret_cast<f32x4_t*>(dst + r * ldd + c) = load4(A + r * lda, c, K); });
}

__global__ __launch_bounds__(256) void act_backward_kernel(int64_t rows, int cols, const float* dy,
                                                           int64_t lddy, const float* z, int64_t ldz, int act,
                                                           float* dz, int64_t lddz, int groups,
                                                           int rows_per_wg)
{
    with_act(act, [&]<int ACT>() {
        each_group(rows, groups, rows_per_wg, [&](int64_t r, int c) {
            const f32x4_t zz = load4(z + r * ldz, c, cols);
            f32x4_t g = load4(dy + r * lddy, c, cols);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = g[e] * act_slope<ACT, 1>(zz[e]);
            store4(dz + r * lddz, c, cols, g);
        });
    });
}

__global__ __launch_bounds__(256) void act_backward2_kernel(int64_t rows, int cols, const float* v,
                                                            int64_t ldv, const float* dy, int64_t lddy,
                                                            const float* z, int64_t ldz, int act, float* gdy,
                                                            int64_t ldgdy, float* gz, int64_t ldgz,
                                                            int groups, int rows_per_wg)
{
    with_act(act, [&]<int ACT>() {
        each_group(rows, groups, rows_per_wg, [&](int64_t r, int c) {
            const f32x4_t zz = load4(z + r * ldz, c, cols), vv = load4(v + r * ldv, c, cols);
            f32x4_t o;
            if (gdy != nullptr) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = vv[e] * act_slope<ACT, 1>(zz[e]);
                store4(gdy + r * ldgdy, c, cols, o);
            }
            if (gz != nullptr) {
                const f32x4_t g = load4(dy + r * lddy, c, cols);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = vv[e] * g[e] * act_slope<ACT, 2>(zz[e]);
                store4(gz + r * ldgz, c, cols, o);
            }
        });
    });
}

__global__ __launch_bounds__(256) void gated_backward_kernel(int64_t M, int F, const float* dh, int64_t lddh,
                                                             const float* Z, int64_t ldz, int act, float* dZ,
                                                             int64_t lddz, int groups, int rows_per_wg)
{
    with_act(act, [&]<int ACT>() {
        each_group(M, groups, rows_per_wg, [&](int64_t r, int c) {
            const f32x4_t g = load4(Z + r * ldz, c, F), u = load4(Z + r * ldz + F, c, F);
            const f32x4_t d = load4(dh + r * lddh, c, F);
            f32x4_t dg, du;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a, s;
                act_both<ACT>(g[e], a, s);
                dg[e] = d[e] * u[e] * s;
                du[e] = d[e] * a;
            }
            store4(dZ + r * lddz, c, F, dg);
            store4(dZ + r * lddz + F, c, F, du);
        });
    });
}

__global__ __launch_bounds__(256) void gated_backward2_kernel(int64_t M, int F, const float* V, int64_t ldv,
                                                              const float* dh, int64_t lddh, const float* Z,
                                                              int64_t ldz, int act, float* gdh, int64_t ldgdh,
                                                              float* gZ, int64_t ldgz, int groups,
                                                              int rows_per_wg)
{
    with_act(act, [&]<int ACT>() {
        each_group(M, groups, rows_per_wg, [&](int64_t r, int c) {
            const f32x4_t g = load4(Z + r * ldz, c, F), u = load4(Z + r * ldz + F, c, F);
            const f32x4_t vg = load4(V + r * ldv, c, F), vu = load4(V + r * ldv + F, c, F);
            f32x4_t s1, o;
#pragma unroll
            for (int e = 0; e < 4; ++e) s1[e] = act_slope<ACT, 1>(g[e]);
            if (gdh != nullptr) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(vg[e] * u[e], s1[e], vu[e] * act_value<ACT>(g[e]));
                store4(gdh + r * ldgdh, c, F, o);
            }
            if (gZ != nullptr) {
                const f32x4_t d = load4(dh + r * lddh, c, F);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = d[e] * __builtin_fmaf(vg[e] * u[e], act_slope<ACT, 2>(g[e]), vu[e] * s1[e]);
                store4(gZ + r * ldgz, c, F, o);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = vg[e] * d[e] * s1[e];
                store4(gZ + r * ldgz + F, c, F, o);
            }
        });
    });
}

int grid_of(const RowsPlan& p) { return (int)(p.wgs < ((int64_t)1 << 20) ? p.wgs : ((int64_t)1 << 20)); }

}  // namespace

hipError_t launch_epilogue(int64_t M, int64_t N, const float* t, int64_t ldt, const BlockEpilogue& ep,
                           hipStream_t s)
{
    const RowsPlan p = plan_rows(M, N);
    hipLaunchKernelGGL(epilogue_kernel, dim3(grid_of(p)), dim3(256), 0, s, M, (int)N, t, ldt, ep, p.groups,
                       p.rows_per_wg);
    return hipGetLastError();
}

hipError_t launch_split_epilogue(const float* parts, int segs, int nsplit, int split_from, int tiles_n, int tile_m,
                                 int64_t M, int64_t N, const BlockEpilogue& ep, hipStream_t s)
{
    if (ep.gated)
        hipLaunchKernelGGL(split_epilogue_kernel<true>, dim3(nsplit, tile_m / 16), dim3(256), 0, s, parts, segs,
                           nsplit, split_from, tiles_n, tile_m, M, N, ep);
    else
        hipLaunchKernelGGL(split_epilogue_kernel<false>, dim3(nsplit, tile_m / 8), dim3(256), 0, s, parts, segs,
                           nsplit, split_from, tiles_n, tile_m, M, N, ep);
    return hipGetLastError();
}

hipError_t launch_copy_rows(int64_t M, int64_t K, const float* A, int64_t lda, float* dst, int64_t ldd,
                            hipStream_t s)
{
    const RowsPlan p = plan_rows(M, K);
    hipLaunchKernelGGL(copy_rows_kernel, dim3(grid_of(p)), dim3(256), 0, s, M, (int)K, A, lda, dst, ldd, p.groups,
                       p.rows_per_wg);
    return hipGetLastError();
}

hipError_t launch_act_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy, const float* z,
                               int64_t ldz, int act, float* dz, int64_t lddz, hipStream_t s)
{
    const RowsPlan p = plan_rows(rows, cols);
    hipLaunchKernelGGL(act_backward_kernel, dim3(grid_of(p)), dim3(256), 0, s, rows, (int)cols, dy, lddy, z,
                       ldz, act, dz, lddz, p.groups, p.rows_per_wg);
    return hipGetLastError();
}

hipError_t launch_act_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv, const float* dy,
                                int64_t lddy, const float* z, int64_t ldz, int act, float* gdy, int64_t ldgdy,
                                float* gz, int64_t ldgz, hipStream_t s)
{
    const RowsPlan p = plan_rows(rows, cols);
    hipLaunchKernelGGL(act_backward2_kernel, dim3(grid_of(p)), dim3(256), 0, s, rows, (int)cols, v, ldv, dy,
                       lddy, z, ldz, act, gdy, ldgdy, gz, ldgz, p.groups, p.rows_per_wg);
    return hipGetLastError();
}

hipError_t launch_gated_backward(int64_t M, int64_t F, const float* dh, int64_t lddh, const float* Z,
                                 int64_t ldz, int act, float* dZ, int64_t lddz, hipStream_t s)
{
    const RowsPlan p = plan_rows(M, F);
    hipLaunchKernelGGL(gated_backward_kernel, dim3(grid_of(p)), dim3(256), 0, s, M, (int)F, dh, lddh, Z, ldz,
                       act, dZ, lddz, p.groups, p.rows_per_wg);
    return hipGetLastError();
}

hipError_t launch_gated_backward2(int64_t M, int64_t F, const float* V, int64_t ldv, const float* dh,
                                  int64_t lddh, const float* Z, int64_t ldz, int act, float* gdh,
                                  int64_t ldgdh, float* gZ, int64_t ldgz, hipStream_t s)
{
    const RowsPlan p = plan_rows(M, F);
    hipLaunchKernelGGL(gated_backward2_kernel, dim3(grid_of(p)), dim3(256), 0, s, M, (int)F, V, ldv, dh, lddh,
                       Z, ldz, act, gdh, ldgdh, gZ, ldgz, p.groups, p.rows_per_wg);
    return hipGetLastError();
}

}  // namespace emu
