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
// waits at its barrier.  The next slab goes from registers to the other LDS
// buffer, and the one after it is requested, in quarters between the
// products: with the copies at the start of a step instead, the wave that
// the scheduler favours left its neighbour to finish alone, at 0.83 of the
// matrix unit's cycles (now 0.89; 552,960 x 1024 x 256 in 2,240 us, 129
// TFLOP/s at the 2.1-2.2 GHz that the chip holds under it).  Reading the two
// blocks of a wave as neighbouring columns takes one 8-byte LDS read per
// operand and k instead of two.  The tiles of one segment run on one XCD,
// whose L2 then serves the segment's rows to all of them.  The workgroups of
// the first tile column also add up the columns of the dZ rows they copy
// (no measurable cost).  Segments are written as partial tiles and joined in
// order by a second launch.
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

    // Thread t copies columns 4 (t % 32) .. +3 of rows t / 32 + 8 r of a slab.
    // The buffer descriptors end with the segment's last row, so rows past
    // it read as zeros; columns past M (N) read what follows in memory, or
    // zeros, and only feed outputs that are not stored.
    const int cr = t >> 5, cc = (t & 31) * 4;
    const int mleft = p.M - m0, nleft = p.N - n0;
    const float* zbase = p.Z + k0 * p.ldz + m0;
    const float* xbase = p.X + k0 * p.ldx + n0;
    const uint32_t zoff = (uint32_t)(cr * p.ldz + cc) * 4, xoff = (uint32_t)(cr * p.ldx + cc) * 4;
    const uint32_t zrow = (uint32_t)p.ldz * 32, xrow = (uint32_t)p.ldx * 32;   // bytes of 8 rows
    u32x4_t rz[4], rx[4];
    __amdgpu_buffer_rsrc_t zr, xr;   // the slab that is loaded next
    auto aim = [&](int step) __attribute__((always_inline)) {
        const int64_t left = kend - k0 - (int64_t)step * BK;
        const int rows = left < BK ? (int)left : BK;   // (none left: an empty buffer, zeros)
        zr = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(zbase + (int64_t)step * BK * p.ldz), (short)0,
                                               rows > 0 ? (int)((rows - 1) * p.ldz + mleft) * 4 : 0, 0x00020000);
        xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(xbase + (int64_t)step * BK * p.ldx), (short)0,
                                               rows > 0 && nleft > 0 ? (int)((rows - 1) * p.ldx + nleft) * 4 : 0,
                                               0x00020000);   // (N = 0: X may be null)
    };
    auto load = [&](int r) __attribute__((always_inline)) {
        rz[r] = __builtin_amdgcn_raw_buffer_load_b128(zr, zoff + r * zrow, 0, 0);
        rx[r] = __builtin_amdgcn_raw_buffer_load_b128(xr, xoff + r * xrow, 0, 0);
    };
    const bool sums = p.db != nullptr && tn == 0;
    f32x4_t bsum = {};   // column sums of the rows this thread copies
    auto store = [&](int b, int r) __attribute__((always_inline)) {
        *reinterpret_cast<u32x4_t*>(&smZ[b][(cr + 8 * r) * TILE + cc]) = rz[r];
        *reinterpret_cast<u32x4_t*>(&smX[b][(cr + 8 * r) * TILE + cc]) = rx[r];
    };

    f32x16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};

    // Block i (j) of a wave's 64 rows (columns) of dW holds the rows 2 l + i
    // of lanes l = 0..31: one 8-byte LDS read then gives both blocks' element.
    const int fz = (lane >> 5) * TILE + wm * 64 + 2 * (lane & 31);
    const int fx = (lane >> 5) * TILE + wn * 64 + 2 * (lane & 31);
    auto read = [&](const float* sm, int f, int k) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x2_t*>(&sm[k * TILE + f]);
    };
    // Slab s is in LDS buffer s % 2.  During its step slab s + 1 goes to the
    // other buffer from the registers it was read to during step s - 1, and
    // slab s + 2 is requested into them, a quarter at a time between the
    // products, so that the matrix unit never waits for a wave's copies.
    aim(0);
#pragma unroll
    for (int r = 0; r < 4; ++r) load(r);
    aim(1);
    f32x4_t part[2] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        store(0, r);
        part[r & 1] = part[r & 1] + __builtin_bit_cast(f32x4_t, rz[r]);
        load(r);
    }
    bsum = part[0] + part[1];
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
    for (int s = 0; s < steps; ++s) {
        const int b = s & 1;
        const float *sz = smZ[b], *sx = smX[b];
        // the operands of each k pair are read while the one before is
        // multiplied
        f32x2_t a[2], c[2];
        a[0] = read(sz, fz, 0);
        c[0] = read(sx, fx, 0);
        aim(s + 2);
        part[0] = part[1] = f32x4_t{};
#pragma unroll
        for (int k = 0; k < BK / 2; ++k) {
            if (k + 1 < BK / 2) {
                a[(k + 1) & 1] = read(sz, fz, 2 * k + 2);
                c[(k + 1) & 1] = read(sx, fx, 2 * k + 2);
            }
            if (k % 3 == 2 && k / 3 < 4) {
                const int r = k / 3;
                store(b ^ 1, r);
                if (sums) part[r & 1] = part[r & 1] + __builtin_bit_cast(f32x4_t, rz[r]);
                load(r);
            }
            if (k == BK / 2 - 1) bsum = bsum + (part[0] + part[1]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    // X first: lane l then holds one row of dW and four
                    // columns per register group
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(c[k & 1][j], a[k & 1][i], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_lgkmcnt0();   // this step's writes and reads
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }

    float* out = p.out + seg * p.pstride;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = m0 + wm * 64 + 2 * (lane & 31) + i;
        if (m < p.M) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // columns 2 p + j for p = 8 q + 4 (l / 32) .. +3
                const int n = n0 + wn * 64 + 16 * q + 8 * (lane >> 5);
                const f32x4_t u = {acc[i][0][4 * q], acc[i][1][4 * q], acc[i][0][4 * q + 1], acc[i][1][4 * q + 1]};
                const f32x4_t v = {acc[i][0][4 * q + 2], acc[i][1][4 * q + 2], acc[i][0][4 * q + 3], acc[i][1][4 * q + 3]};
                store4(out + (int64_t)m * p.ldo, n, p.N, u);
                store4(out + (int64_t)m * p.ldo, n + 4, p.N, v);
            }
        }
    }
    if (sums) {
        // (every wave has passed the last step's barrier: the slabs are free)
        float* sum = smZ[0];
        *reinterpret_cast<f32x4_t*>(&sum[cr * TILE + cc]) = bsum;
        wait_lgkmcnt0();
        __builtin_amdgcn_s_barrier();
        if (t < TILE && t < mleft) {
            float v = sum[t];
#pragma unroll
            for (int r = 1; r < 8; ++r) v = v + sum[r * TILE + t];
            p.db[seg * p.bstride + m0 + t] = v;
        }
    }
}

// dW = the sum of the segments' partial results (four columns per thread),
// and db likewise: a workgroup takes 64 groups of columns, its four waves
// every fourth segment each, and adds their sums in order.
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ part, int segs, int64_t pstride,
                                                         int64_t ldp, int M, int N, float* dW, int64_t lddw,
                                                         const float* __restrict__ bpart, int64_t bstride,
                                                         float* db)
{
    __shared__ __attribute__((aligned(16))) f32x4_t sum[4][64];
    const int groups = (N + 3) / 4;
    const int64_t total = (int64_t)M * groups;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i = (int64_t)blockIdx.x * 64 + lane;
    const float* src = nullptr;
    int64_t stride = 0;
    int m = 0, c = 0;
    if (i < total) {
        m = (int)(i / groups);
        c = (int)(i - (int64_t)m * groups) * 4;
        src = part + (int64_t)m * ldp + c;   // (ldp >= 4 * groups: whole groups)
        stride = pstride;
    } else if (db != nullptr && i - total < (M + 3) / 4) {
        src = bpart + (i - total) * 4;       // (bstride is a multiple of 4)
        stride = bstride;
    }
    f32x4_t v = {};
    if (src != nullptr) {
#pragma unroll 8
        for (int s = wave; s < segs; s += 4) v = v + *reinterpret_cast<const f32x4_t*>(src + s * stride);
    }
    sum[wave][lane] = v;
    __syncthreads();
    if (wave != 0 || src == nullptr) return;
    v = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
    if (i < total)
        store4(dW + (int64_t)m * lddw, c, N, v);
    else
        store4(db, (int)(i - total) * 4, M, v);
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
    return p.segs > 1 ? (size_t)p.segs * (size_t)(M * p.ldp + ((M + 3) & ~(int64_t)3)) * sizeof(float) : 0;
}

hipError_t launch_wgrad(int64_t rows, int64_t M, int64_t N, const float* dZ, int64_t lddz, const float* X,
                        int64_t ldx, float* dW, int64_t lddw, float* db, void* ws, hipStream_t s)
{
    const WgradPlan pl = plan_wgrad(rows, M, N);
    if (pl.tiles * pl.segs >= ((int64_t)1 << 31) || lddz > kWgradMaxLd || ldx > kWgradMaxLd || M >= ((int64_t)1 << 31) - TILE ||
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
    const int64_t bstride = (M + 3) & ~(int64_t)3;
    if (pl.segs > 1) {
        a.out = part;
        a.ldo = pl.ldp;
        a.pstride = pstride;
        a.db = db != nullptr ? bpart : nullptr;
        a.bstride = bstride;
    } else {
        a.out = dW;
        a.ldo = lddw;
        a.db = db;
    }
    hipLaunchKernelGGL(wgrad_kernel, dim3((int)(pl.tiles * pl.segs)), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && pl.segs > 1) {
        const int64_t work = M * (pl.ldp / 4) + (db != nullptr ? bstride / 4 : 0);
        if ((work + 63) / 64 >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
        hipLaunchKernelGGL(wgrad_join_kernel, dim3((int)((work + 63) / 64)), dim3(256), 0, s, part, pl.segs, pstride,
                           pl.ldp, (int)M, (int)N, dW, lddw, bpart, bstride, db);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace emu
