// The weight-gradient product dW = dZ^T X over many rows, with db = the
// column sums of dZ (include/emu_block.h), on the FP32 matrix instruction
// v_mfma_f32_32x32x2_f32.
//
// Both operands are contiguous along the output's dimensions and strided
// along the summed one, which is how that instruction takes them: lane l
// feeds element (k = l / 32, column l % 32), so a 32-row slab of each operand
// goes to LDS as it lies in memory, without a transpose and without the
// BF16 split (whose pieces would have to be transposed, at twice the vector
// work of the forward product).  FP32 matrix instructions are not bound by
// the chip's power as the BF16 stream is, so the product runs near their
// peak.
//
// One 256-thread workgroup owns a 128 x 128 tile of dW over one segment of
// the rows; 4 waves, 64 x 64 each (2 x 2 instructions' tiles, 64 accumulator
// registers); two workgroups share a CU, so one computes while the other
// waits at its barrier.  The next slab is read to registers during the
// products of the current one and written to the other LDS buffer after
// them.  The tiles of one segment run on one XCD, whose L2 then serves the
// segment's rows to all of them.  The workgroups of the first tile column
// also add up the columns of their dZ slabs.  Segments are written as
// partial tiles and joined in order by a second launch.
#include "emu_block_device.h"
#include "emu_block_launch.h"
#include "emu_tile.h"

namespace emu {
namespace {

constexpr int SLAB = BK * TILE;   // floats of one operand's slab

struct WgradArgs {
    const float* Z;
    const float* X;
    int64_t ldz, ldx, rows;
    int M, N;
    int tiles_n, tiles;
    int segs, seg_steps;   // segments of seg_steps slabs
    float* out;            // dW, or the partial results: seg * pstride + m * ldo + n
    int64_t ldo, pstride;
    float* db;             // db, or its partials: seg * bstride + m; or null
    int64_t bstride;
};

__global__ __launch_bounds__(256, 2) void wgrad_kernel(WgradArgs p)
{
    __shared__ __attribute__((aligned(16))) float smZ[2][SLAB];
    __shared__ __attribute__((aligned(16))) float smX[2][SLAB];
    __shared__ float colsum[TILE];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    const int item = xcd_position(blockIdx.x, gridDim.x);
    const int seg = item / p.tiles;
    const int tile = item - seg * p.tiles;
    const int tm = tile / p.tiles_n, tn = tile - tm * p.tiles_n;
    const int m0 = tm * TILE, n0 = tn * TILE;
    const int64_t k0 = (int64_t)seg * p.seg_steps * BK;
    int64_t kend = k0 + (int64_t)p.seg_steps * BK;
    if (kend > p.rows) kend = p.rows;
    const int steps = (int)((kend - k0 + BK - 1) / BK);

    // thread t copies columns 4 (t % 32) .. +3 of rows t / 32 + 8 r
    const int cr = t >> 5, cc = (t & 31) * 4;
    const int mleft = p.M - m0, nleft = p.N - n0;
    f32x4_t rz[4], rx[4];
    auto load = [&](int step) __attribute__((always_inline)) {
        const int64_t r0 = k0 + (int64_t)step * BK;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t row = r0 + cr + 8 * r;
            if (row < kend) {
                rz[r] = load4(p.Z + row * p.ldz + m0, cc, mleft);
                rx[r] = load4(p.X + row * p.ldx + n0, cc, nleft);
            } else {
                rz[r] = rx[r] = f32x4_t{};
            }
        }
    };
    auto store = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            *reinterpret_cast<f32x4_t*>(&smZ[b][(cr + 8 * r) * TILE + cc]) = rz[r];
            *reinterpret_cast<f32x4_t*>(&smX[b][(cr + 8 * r) * TILE + cc]) = rx[r];
        }
    };

    f32x16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
    const bool sums = p.db != nullptr && tn == 0;
    float bsum = 0.0f;

    if (steps > 0) {
        load(0);
        store(0);
    }
    __syncthreads();
    const int fz = (lane >> 5) * TILE + wm * 64 + (lane & 31);
    const int fx = (lane >> 5) * TILE + wn * 64 + (lane & 31);
    for (int s = 0; s < steps; ++s) {
        const int b = s & 1;
        if (s + 1 < steps) load(s + 1);
#pragma unroll
        for (int k = 0; k < BK; k += 2) {
            float a[2], c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = smZ[b][k * TILE + fz + 32 * i];
                c[i] = smX[b][k * TILE + fx + 32 * i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    // X first: lane l then holds row m = l % 32 and four
                    // consecutive columns per register group
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(c[j], a[i], acc[i][j], 0, 0, 0);
        }
        if (sums) {
            // half of the slab's rows per thread, added among themselves first
            const float* col = &smZ[b][(t >> 7) * 16 * TILE + (t & 127)];
            float part = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k) part = part + col[k * TILE];
            bsum = bsum + part;
        }
        if (s + 1 < steps) store(b ^ 1);
        __syncthreads();
    }

    float* out = p.out + seg * p.pstride;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = m0 + wm * 64 + i * 32 + (lane & 31);
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = n0 + wn * 64 + j * 32 + 8 * q + 4 * (lane >> 5);
                f32x4_t v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
                store4(out + (int64_t)m * p.ldo, n, p.N, v);
            }
    }
    if (sums) {
        if (t >= 128) colsum[t - 128] = bsum;
        __syncthreads();
        if (t < 128 && t < mleft) p.db[seg * p.bstride + m0 + t] = bsum + colsum[t];
    }
}

// dW = the sum of the segments' partial results, in order (four columns per
// thread), then db likewise.
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ part, int segs, int64_t pstride,
                                                         int64_t ldp, int M, int N, float* dW, int64_t lddw,
                                                         const float* __restrict__ bpart, int64_t bstride,
                                                         float* db)
{
    const int groups = (N + 3) / 4;
    const int64_t total = (int64_t)M * groups;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total + (db != nullptr ? M : 0);
         i += (int64_t)gridDim.x * 256) {
        if (i < total) {
            const int m = (int)(i / groups);
            const int c = (int)(i - (int64_t)m * groups) * 4;
            const float* src = part + (int64_t)m * ldp + c;   // (ldp >= 4 * groups: whole groups)
            f32x4_t v = *reinterpret_cast<const f32x4_t*>(src);
            for (int s = 1; s < segs; ++s) v = v + *reinterpret_cast<const f32x4_t*>(src + s * pstride);
            store4(dW + (int64_t)m * lddw, c, N, v);
        } else {
            const float* src = bpart + (i - total);
            float v = src[0];
            for (int s = 1; s < segs; ++s) v = v + src[s * bstride];
            db[i - total] = v;
        }
    }
}

struct WgradPlan {
    int64_t tiles_m, tiles_n, tiles;
    int segs, seg_steps;
    int64_t ldp;      // row of a partial result
};

// Segments: the load of the busiest CU is ceil(tiles * segs / 256) segment
// tiles of ceil(steps / segs) slabs; the fewest segments within 5 % of the
// least load, 64 at most and 4 slabs each at least.
WgradPlan plan_wgrad(int64_t rows, int64_t M, int64_t N)
{
    WgradPlan p;
    p.tiles_m = (M + TILE - 1) / TILE;
    p.tiles_n = N > 0 ? (N + TILE - 1) / TILE : 1;
    p.tiles = p.tiles_m * p.tiles_n;
    const int64_t steps = (rows + BK - 1) / BK;
    int64_t most = steps / 4;
    if (most > 128) most = 128;
    if (most < 1) most = 1;
    auto load = [&](int64_t s) {
        const int64_t items = p.tiles * s, per = (steps + s - 1) / s;
        // (two workgroups per CU hide each other's waits: one alone takes
        // about a quarter longer per slab)
        return (double)((items + 255) / 256) * (double)per * (items <= 256 ? 1.25 : 1.0) + 0.25 * (double)s;
    };
    double best = load(1);
    for (int64_t s = 2; s <= most; ++s)
        if (load(s) < best) best = load(s);
    int64_t segs = 1;
    while (segs < most && load(segs) > 1.05 * best) ++segs;
    p.seg_steps = (int)((steps + segs - 1) / segs);
    if (p.seg_steps < 1) p.seg_steps = 1;
    p.segs = (int)((steps + p.seg_steps - 1) / p.seg_steps);
    if (p.segs < 1) p.segs = 1;
    p.ldp = (N + 3) & ~(int64_t)3;
    return p;
}

}  // namespace

size_t wgrad_workspace(int64_t rows, int64_t M, int64_t N)
{
    const WgradPlan p = plan_wgrad(rows, M, N);
    return p.segs > 1 ? (size_t)p.segs * (size_t)(M * p.ldp + M) * sizeof(float) : 0;
}

hipError_t launch_wgrad(int64_t rows, int64_t M, int64_t N, const float* dZ, int64_t lddz, const float* X,
                        int64_t ldx, float* dW, int64_t lddw, float* db, void* ws, hipStream_t s)
{
    const WgradPlan pl = plan_wgrad(rows, M, N);
    if (pl.tiles * pl.segs >= ((int64_t)1 << 31) || M >= ((int64_t)1 << 31) - TILE ||
        N >= ((int64_t)1 << 31) - TILE)
        return hipErrorInvalidValue;
    WgradArgs a{};
    a.Z = dZ;
    a.X = X;
    a.ldz = lddz;
    a.ldx = ldx;
    a.rows = rows;
    a.M = (int)M;
    a.N = (int)N;
    a.tiles_n = (int)pl.tiles_n;
    a.tiles = (int)pl.tiles;
    a.segs = pl.segs;
    a.seg_steps = pl.seg_steps;
    float* part = static_cast<float*>(ws);
    const int64_t pstride = M * pl.ldp;
    float* bpart = part + pl.segs * pstride;
    if (pl.segs > 1) {
        a.out = part;
        a.ldo = pl.ldp;
        a.pstride = pstride;
        a.db = db != nullptr ? bpart : nullptr;
        a.bstride = M;
    } else {
        a.out = dW;
        a.ldo = lddw;
        a.db = db;
    }
    hipLaunchKernelGGL(wgrad_kernel, dim3((int)(pl.tiles * pl.segs)), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && pl.segs > 1) {
        const int64_t work = M * (pl.ldp / 4) + M;
        const int64_t blocks = (work + 255) / 256;
        hipLaunchKernelGGL(wgrad_join_kernel, dim3((int)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s, part,
                           pl.segs, pstride, pl.ldp, (int)M, (int)N, dW, lddw, bpart, M, db);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace emu
