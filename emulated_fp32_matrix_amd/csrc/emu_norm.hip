// Layer norm, its backward pass and that pass's own backward pass
// (include/emu_block.h).
//
// All three are bound by memory: the forward reads a row and writes a row,
// the backward reads two and writes one, the second order reads three and
// writes two.  A row is therefore read once, into the registers of LPR lanes
// (16 to 1024 by its length, four columns per 16-byte access), and its sums
// (mean, squared deviations, projections) run across those lanes: by DPP
// rotations and lane swaps within a wave, through LDS beyond it.  Short rows
// share a wave (four rows of 256 columns), so that every lane has several
// loads in flight; the next row is requested before the current one's sums.
// The column sums (weight and bias gradients) stay in registers over all rows
// of a workgroup, then go to one partial row per workgroup, and a second
// launch adds those in order.
#include "emu_block_device.h"
#include "emu_block_launch.h"

namespace emu {
namespace {

template <int LPR_, int NV_>
struct RowShape {
    static constexpr int LPR = LPR_;                  // lanes per row
    static constexpr int NV = NV_;                    // 16-byte groups per lane
    static constexpr int NT = LPR_ < 256 ? 256 : LPR_;
    static constexpr int ROWS = NT / LPR_;            // rows at once per workgroup
    static constexpr int COLS = LPR_ * NV_ * 4;
};

// Sums of N values over the lanes of a row, in all of them.
template <class SH, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* lds)
{
    if constexpr (SH::LPR <= 64) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane_sum<SH::LPR>(v[i]);
    } else {
        constexpr int W = SH::LPR / 64;
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane_sum<64>(v[i]);
        __syncthreads();   // the previous sums have been read
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds[i * W + wave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = lds[i * W];
#pragma unroll
            for (int w = 1; w < W; ++w) s = s + lds[i * W + w];
            v[i] = s;
        }
    }
}

// A lane's columns of a row; zeros past the end.
template <class SH>
__device__ __forceinline__ void load_row(f32x4_t (&v)[SH::NV], const float* row, int li, int cols, float fill = 0.0f)
{
#pragma unroll
    for (int j = 0; j < SH::NV; ++j) v[j] = load4(row, (li + SH::LPR * j) * 4, cols, fill);
}

template <class SH>
__device__ __forceinline__ void load_vec(f32x4_t (&v)[SH::NV], const float* vec, int li, int cols, float none)
{
    if (vec != nullptr) {
        load_row<SH>(v, vec, li, cols);
    } else {
#pragma unroll
        for (int j = 0; j < SH::NV; ++j) v[j] = f32x4_t{none, none, none, none};
    }
}

template <class SH>
__device__ __forceinline__ void store_row(float* row, int li, int cols, const f32x4_t (&v)[SH::NV])
{
#pragma unroll
    for (int j = 0; j < SH::NV; ++j) store4(row, (li + SH::LPR * j) * 4, cols, v[j]);
}

template <class SH>
__device__ __forceinline__ float sum_of(const f32x4_t (&v)[SH::NV])
{
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < SH::NV; ++j) s = s + ((v[j][0] + v[j][1]) + (v[j][2] + v[j][3]));
    return s;
}

template <class SH>
__device__ __forceinline__ float dot_of(const f32x4_t (&v)[SH::NV], const f32x4_t (&u)[SH::NV])
{
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < SH::NV; ++j) {
        const f32x4_t p = v[j] * u[j];
        s = s + ((p[0] + p[1]) + (p[2] + p[3]));
    }
    return s;
}

template <class SH>
__global__ __launch_bounds__(SH::NT) void norm_kernel(int64_t rows, int cols, const float* x, int64_t ldx,
                                                      const float* __restrict__ weight,
                                                      const float* __restrict__ bias, float eps, float* y,
                                                      int64_t ldy, float* mean, float* rstd)
{
    __shared__ float lds[64];
    const int li = threadIdx.x % SH::LPR;
    const int64_t step = (int64_t)gridDim.x * SH::ROWS;
    const float n = (float)cols;
    f32x4_t w[SH::NV], b[SH::NV], v[SH::NV], nx[SH::NV];
    load_vec<SH>(w, weight, li, cols, 1.0f);
    load_vec<SH>(b, bias, li, cols, 0.0f);
    const int64_t r0 = (int64_t)blockIdx.x * SH::ROWS + threadIdx.x / SH::LPR;
    // rows past the end repeat the last one (every lane joins the sums) and
    // are not written
    auto at = [&](int64_t r) { return r < rows ? r : rows - 1; };
    load_row<SH>(v, x + at(r0) * ldx, li, cols);
    for (int64_t rb = (int64_t)blockIdx.x * SH::ROWS; rb < rows; rb += step) {
        const int64_t r = rb + threadIdx.x / SH::LPR;
        if (rb + step < rows) load_row<SH>(nx, x + at(r + step) * ldx, li, cols);
        float s1[1] = {sum_of<SH>(v)};
        row_sum<SH>(s1, lds);
        float mu = s1[0] / n;
        // The sum's rounding, up to a few units of the mean, is a deviation of
        // its own in a row far from zero (1,000,003 in all of 200 columns gave
        // xhat = 1): the centred row's mean is added, which leaves the mean's
        // own rounding.  (Not finite where the row is not or overflows: mu
        // stays.)
        float c = 0.0f;
#pragma unroll
        for (int j = 0; j < SH::NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c = c + ((li + SH::LPR * j) * 4 + e < cols ? v[j][e] - mu : 0.0f);
        float s0[1] = {c};
        row_sum<SH>(s0, lds);
        c = s0[0] / n;
        if (__builtin_fabsf(c) < __builtin_inff()) mu = mu + c;
#pragma unroll
        for (int j = 0; j < SH::NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[j][e] = (li + SH::LPR * j) * 4 + e < cols ? v[j][e] - mu : 0.0f;
        float s2[1] = {dot_of<SH>(v, v)};
        row_sum<SH>(s2, lds);
        const float rs = 1.0f / sqrtf(s2[0] / n + eps);
        if (r < rows) {
#pragma unroll
            for (int j = 0; j < SH::NV; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j][e] = __builtin_fmaf(v[j][e] * rs, w[j][e], b[j][e]);
            store_row<SH>(y + r * ldy, li, cols, v);
            if (li == 0) {
                if (mean != nullptr) mean[r] = mu;
                if (rstd != nullptr) rstd[r] = rs;
            }
        }
#pragma unroll
        for (int j = 0; j < SH::NV; ++j) v[j] = nx[j];
    }
}

// The column sums that a workgroup's threads hold for the columns of their
// lane, added over the rows it ran at once, to out[0 .. cols-1].
template <class SH>
__device__ __forceinline__ void store_columns(f32x4_t (&acc)[SH::NV], int li, int cols, float* out, float* lds)
{
    if constexpr (SH::LPR < 64) {   // rows that share a wave
#pragma unroll
        for (int j = 0; j < SH::NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (SH::LPR == 16) acc[j][e] = add_lane16(acc[j][e]);
                acc[j][e] = add_lane32(acc[j][e]);
            }
    }
    if constexpr (SH::LPR <= 64) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        __syncthreads();
        if (lane < SH::LPR) {
#pragma unroll
            for (int j = 0; j < SH::NV; ++j)
                *reinterpret_cast<f32x4_t*>(lds + wave * SH::COLS + (li + SH::LPR * j) * 4) = acc[j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += SH::NT) {
            float s = lds[c];
#pragma unroll
            for (int w = 1; w < SH::NT / 64; ++w) s = s + lds[w * SH::COLS + c];
            out[c] = s;
        }
    } else {
        store_row<SH>(out, li, cols, acc);
    }
}

template <class SH>
constexpr int column_lds() { return SH::LPR <= 64 ? SH::COLS * (SH::NT / 64) : 4; }

// part: per workgroup one row of 2 * cols (weight sums, then bias sums), or
// null when neither is wanted; with one workgroup dweight and dbias directly.
template <class SH>
__global__ __launch_bounds__(SH::NT) void norm_backward_kernel(
    int64_t rows, int cols, const float* dy, int64_t lddy, const float* __restrict__ x, int64_t ldx,
    const float* __restrict__ weight, const float* __restrict__ mean, const float* __restrict__ rstd,
    float* dx, int64_t lddx, float* pw, float* pb, int64_t pstride)
{
    __shared__ float lds[128];
    __shared__ __attribute__((aligned(16))) float cols_lds[column_lds<SH>()];
    const int li = threadIdx.x % SH::LPR;
    const int64_t step = (int64_t)gridDim.x * SH::ROWS;
    const float inv_n = 1.0f / (float)cols;
    f32x4_t w[SH::NV], aw[SH::NV], ab[SH::NV], g[SH::NV], h[SH::NV], ng[SH::NV], nh[SH::NV];
    load_vec<SH>(w, weight, li, cols, 1.0f);
#pragma unroll
    for (int j = 0; j < SH::NV; ++j) aw[j] = ab[j] = f32x4_t{};
    auto at = [&](int64_t r) { return r < rows ? r : rows - 1; };
    {
        const int64_t r = at((int64_t)blockIdx.x * SH::ROWS + threadIdx.x / SH::LPR);
        load_row<SH>(g, dy + r * lddy, li, cols);
        load_row<SH>(h, x + r * ldx, li, cols);
    }
    for (int64_t rb = (int64_t)blockIdx.x * SH::ROWS; rb < rows; rb += step) {
        const int64_t r = rb + threadIdx.x / SH::LPR;
        const float mu = mean[at(r)], rs = rstd[at(r)];
        if (rb + step < rows) {
            const int64_t rn = at(r + step);
            load_row<SH>(ng, dy + rn * lddy, li, cols);
            load_row<SH>(nh, x + rn * ldx, li, cols);
        }
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < SH::NV; ++j) {
            h[j] = (h[j] - mu) * rs;                       // xhat
            // columns past the end meet dy = 0, but -mu rs may be infinite
            if (cols != SH::COLS) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = (li + SH::LPR * j) * 4 + e < cols ? h[j][e] : 0.0f;
            }
            if (r < rows) {
                aw[j] = aw[j] + g[j] * h[j];
                ab[j] = ab[j] + g[j];
            }
            g[j] = g[j] * w[j];                            // a
            const f32x4_t p = g[j] * h[j];
            s[0] = s[0] + ((g[j][0] + g[j][1]) + (g[j][2] + g[j][3]));
            s[1] = s[1] + ((p[0] + p[1]) + (p[2] + p[3]));
        }
        if (dx != nullptr) {
            row_sum<SH>(s, lds);
            const float ma = s[0] * inv_n, max_ = s[1] * inv_n;
            if (r < rows) {
#pragma unroll
                for (int j = 0; j < SH::NV; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        g[j][e] = rs * __builtin_fmaf(-h[j][e], max_, g[j][e] - ma);
                store_row<SH>(dx + r * lddx, li, cols, g);
            }
        }
#pragma unroll
        for (int j = 0; j < SH::NV; ++j) {
            g[j] = ng[j];
            h[j] = nh[j];
        }
    }
    if (pw != nullptr) store_columns<SH>(aw, li, cols, pw + blockIdx.x * pstride, cols_lds);
    if (pb != nullptr) store_columns<SH>(ab, li, cols, pb + blockIdx.x * pstride, cols_lds);
}

template <class SH>
__global__ __launch_bounds__(SH::NT) void norm_backward2_kernel(
    int64_t rows, int cols, const float* v, int64_t ldv, const float* __restrict__ p,
    const float* __restrict__ q, const float* dy, int64_t lddy, const float* __restrict__ x, int64_t ldx,
    const float* __restrict__ weight, const float* __restrict__ mean, const float* __restrict__ rstd,
    float* gdy, int64_t ldgdy, float* gx, int64_t ldgx, float* pw, int64_t pstride)
{
    __shared__ float lds[128];
    __shared__ __attribute__((aligned(16))) float cols_lds[column_lds<SH>()];
    const int li = threadIdx.x % SH::LPR;
    const int64_t step = (int64_t)gridDim.x * SH::ROWS;
    const float inv_n = 1.0f / (float)cols;
    f32x4_t w[SH::NV], pv[SH::NV], aw[SH::NV];
    load_vec<SH>(w, weight, li, cols, 1.0f);
    load_vec<SH>(pv, p, li, cols, 0.0f);
#pragma unroll
    for (int j = 0; j < SH::NV; ++j) aw[j] = f32x4_t{};
    auto at = [&](int64_t r) { return r < rows ? r : rows - 1; };
    for (int64_t rb = (int64_t)blockIdx.x * SH::ROWS; rb < rows; rb += step) {
        const int64_t r = rb + threadIdx.x / SH::LPR;
        const int64_t ra = at(r);
        const float mu = mean[ra], rs = rstd[ra];
        f32x4_t g[SH::NV], h[SH::NV], u[SH::NV];   // dy, xhat, v
        load_row<SH>(g, dy + ra * lddy, li, cols);
        load_row<SH>(h, x + ra * ldx, li, cols, mu);   // xhat = 0 past the end
        if (v != nullptr) {
            load_row<SH>(u, v + ra * ldv, li, cols);
        } else {
#pragma unroll
            for (int j = 0; j < SH::NV; ++j) u[j] = f32x4_t{};
        }
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};     // sums of v, v xhat, a, a xhat
#pragma unroll
        for (int j = 0; j < SH::NV; ++j) {
            h[j] = (h[j] - mu) * rs;
            const f32x4_t a = g[j] * w[j], uh = u[j] * h[j], ah = a * h[j];
            s[0] = s[0] + ((u[j][0] + u[j][1]) + (u[j][2] + u[j][3]));
            s[1] = s[1] + ((uh[0] + uh[1]) + (uh[2] + uh[3]));
            s[2] = s[2] + ((a[0] + a[1]) + (a[2] + a[3]));
            s[3] = s[3] + ((ah[0] + ah[1]) + (ah[2] + ah[3]));
        }
        row_sum<SH>(s, lds);
        const float mv = s[0] * inv_n, mvx = s[1] * inv_n, ma = s[2] * inv_n, max_ = s[3] * inv_n;
        float t[3] = {0.0f, 0.0f, 0.0f};           // sums of v (P a), h', h' xhat
#pragma unroll
        for (int j = 0; j < SH::NV; ++j) {
            f32x4_t sv, out;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = g[j][e] * w[j][e];
                sv[e] = rs * __builtin_fmaf(-h[j][e], mvx, u[j][e] - mv);
                const float pa = __builtin_fmaf(-h[j][e], max_, a - ma);
                t[0] = t[0] + u[j][e] * pa;
                // the gradient on xhat
                const float hx = __builtin_fmaf(-rs, __builtin_fmaf(u[j][e], max_, a * mvx), pv[j][e] * g[j][e]);
                t[1] = t[1] + hx;
                t[2] = t[2] + hx * h[j][e];
                out[e] = __builtin_fmaf(w[j][e], sv[e], pv[j][e] * h[j][e]);
                if (r < rows) aw[j][e] = __builtin_fmaf(g[j][e], sv[e], aw[j][e]);
                u[j][e] = hx;
            }
            if (gdy != nullptr && r < rows) {
                if (q != nullptr) out = out + load4(q, (li + SH::LPR * j) * 4, cols);
                store4(gdy + r * ldgdy, (li + SH::LPR * j) * 4, cols, out);
            }
        }
        if (gx != nullptr) {
            row_sum<SH>(t, lds);
            const float mh = t[1] * inv_n, mhx = t[2] * inv_n + rs * (t[0] * inv_n);
            if (r < rows) {
#pragma unroll
                for (int j = 0; j < SH::NV; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[j][e] = rs * __builtin_fmaf(-h[j][e], mhx, u[j][e] - mh);
                store_row<SH>(gx + r * ldgx, li, cols, u);
            }
        }
    }
    if (pw != nullptr) store_columns<SH>(aw, li, cols, pw + blockIdx.x * pstride, cols_lds);
}

// out0[c] (and out1[c]) = sum over i < parts of part[i * stride + c] for c <
// cols (and cols <= c < 2 cols), in a fixed order: 64 threads of a column add
// every 64th partial, then their sums are added pairwise.
__global__ __launch_bounds__(1024) void column_join_kernel(const float* __restrict__ part, int parts,
                                                           int64_t stride, int total, int cols, float* out0,
                                                           float* out1)
{
    __shared__ float lds[64][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15);
    const int k = threadIdx.x >> 4;
    float s = 0.0f;
    if (c < total)
        for (int i = k; i < parts; i += 64) s = s + part[i * stride + c];
    lds[k][threadIdx.x & 15] = s;
    __syncthreads();
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        if (k < m) lds[k][threadIdx.x & 15] = lds[k][threadIdx.x & 15] + lds[k + m][threadIdx.x & 15];
        __syncthreads();
    }
    if (k == 0 && c < total) {
        const float r = lds[0][threadIdx.x & 15];
        if (c < cols) {
            if (out0 != nullptr) out0[c] = r;
        } else if (out1 != nullptr) {
            out1[c - cols] = r;
        }
    }
}

__global__ __launch_bounds__(256) void zero_kernel(float* p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

template <class F>
void with_shape(int64_t cols, F&& f)
{
    if (cols <= 64) f(RowShape<16, 1>{});
    else if (cols <= 128) f(RowShape<16, 2>{});
    else if (cols <= 256) f(RowShape<16, 4>{});
    else if (cols <= 512) f(RowShape<32, 4>{});
    else if (cols <= 1024) f(RowShape<64, 4>{});
    else if (cols <= 2048) f(RowShape<256, 2>{});
    else if (cols <= 4096) f(RowShape<256, 4>{});
    else if (cols <= 8192) f(RowShape<512, 4>{});
    else f(RowShape<1024, 4>{});
}

// Workgroups of the passes with column sums: enough rows each (8 per group
// of lanes) that the partial rows are a small part of the traffic.
template <class SH>
int64_t backward_groups(int64_t rows)
{
    const int64_t want = (rows + SH::ROWS * 8 - 1) / (SH::ROWS * 8);
    return want < 1 ? 1 : want > 1024 ? 1024 : want;
}

int64_t parts_of(int64_t rows, int64_t cols)
{
    int64_t p = 1;
    with_shape(cols, [&]<class SH>(SH) { p = backward_groups<SH>(rows); });
    return p;
}

}  // namespace

size_t norm_backward_workspace(int64_t rows, int64_t cols)
{
    const int64_t p = parts_of(rows, cols);
    return p > 1 ? (size_t)p * 2 * (size_t)cols * sizeof(float) : 0;
}

hipError_t launch_zero(float* p, int64_t n, hipStream_t s)
{
    if (p == nullptr || n <= 0) return hipSuccess;
    const int64_t blocks = (n + 255) / 256;
    hipLaunchKernelGGL(zero_kernel, dim3((int)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, p, n);
    return hipGetLastError();
}

hipError_t launch_column_join(const float* part, int64_t parts, int64_t stride, int64_t total, int64_t cols,
                              float* out0, float* out1, hipStream_t s)
{
    hipLaunchKernelGGL(column_join_kernel, dim3((int)((total + 15) / 16)), dim3(1024), 0, s, part, (int)parts,
                       stride, (int)total, (int)cols, out0, out1);
    return hipGetLastError();
}

hipError_t launch_norm(int64_t rows, int64_t cols, const float* x, int64_t ldx, const float* weight,
                       const float* bias, float eps, float* y, int64_t ldy, float* mean, float* rstd,
                       hipStream_t s)
{
    with_shape(cols, [&]<class SH>(SH) {
        const int64_t need = (rows + SH::ROWS - 1) / SH::ROWS;
        const int64_t most = 2048 * 256 / SH::NT;
        hipLaunchKernelGGL(norm_kernel<SH>, dim3((int)(need < most ? need : most)), dim3(SH::NT), 0, s, rows,
                           (int)cols, x, ldx, weight, bias, eps, y, ldy, mean, rstd);
    });
    return hipGetLastError();
}

hipError_t launch_norm_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy, const float* x,
                                int64_t ldx, const float* weight, const float* mean, const float* rstd,
                                float* dx, int64_t lddx, float* dweight, float* dbias, float* ws,
                                hipStream_t s)
{
    const bool sums = dweight != nullptr || dbias != nullptr;
    int64_t parts = 1;
    with_shape(cols, [&]<class SH>(SH) {
        const int64_t need = (rows + SH::ROWS - 1) / SH::ROWS, most = 2048 * 256 / SH::NT;
        const int64_t grid = sums ? backward_groups<SH>(rows) : need < most ? need : most;
        parts = sums ? grid : 1;
        float* pw = dweight == nullptr ? nullptr : parts > 1 ? ws : dweight;
        float* pb = dbias == nullptr ? nullptr : parts > 1 ? ws + cols : dbias;
        hipLaunchKernelGGL(norm_backward_kernel<SH>, dim3((int)grid), dim3(SH::NT), 0, s, rows, (int)cols, dy,
                           lddy, x, ldx, weight, mean, rstd, dx, lddx, pw, pb, 2 * cols);
    });
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && parts > 1) e = launch_column_join(ws, parts, 2 * cols, 2 * cols, cols, dweight, dbias, s);
    return e;
}

hipError_t launch_norm_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv, const float* p,
                                 const float* q, const float* dy, int64_t lddy, const float* x, int64_t ldx,
                                 const float* weight, const float* mean, const float* rstd, float* gdy,
                                 int64_t ldgdy, float* gx, int64_t ldgx, float* gw, float* ws, hipStream_t s)
{
    int64_t parts = 1;
    with_shape(cols, [&]<class SH>(SH) {
        const int64_t need = (rows + SH::ROWS - 1) / SH::ROWS, most = 2048 * 256 / SH::NT;
        const int64_t grid = gw != nullptr ? backward_groups<SH>(rows) : need < most ? need : most;
        parts = gw != nullptr ? grid : 1;
        float* pw = gw == nullptr ? nullptr : parts > 1 ? ws : gw;
        hipLaunchKernelGGL(norm_backward2_kernel<SH>, dim3((int)grid), dim3(SH::NT), 0, s, rows, (int)cols, v,
                           ldv, p, q, dy, lddy, x, ldx, weight, mean, rstd, gdy, ldgdy, gx, ldgx, pw, 2 * cols);
    });
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && parts > 1) e = launch_column_join(ws, parts, 2 * cols, cols, cols, gw, nullptr, s);
    return e;
}

}  // namespace emu
