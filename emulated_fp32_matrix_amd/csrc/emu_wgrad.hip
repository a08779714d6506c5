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
// A workgroup owns 128 rows x 256 (or 128) columns of dW over one segment of
// the rows of dZ and X; its 8 (4) waves take 64 x 64 each (2 x 2 instructions'
// tiles, 64 accumulator registers), two per SIMD (of one workgroup, or of two
// that share a CU).  The next slab goes from registers to the other LDS
// buffer, and the one after it is requested, a copy at a time between the
// products: with the copies at the start of a step instead, the wave that the
// scheduler favours left its neighbour to finish alone, at 0.83 of the matrix
// unit's cycles (0.89 spread out).  Reading the two blocks of a wave as
// neighbouring columns takes one 8-byte LDS read per operand and k instead of
// two.  256 columns halve the copies of dZ per product and, where dZ is made
// on the way, its making: 552,960 x 1024 x 256 in 2,090 us against 2,165 with
// 128 (139 TFLOP/s of 157; the chip holds 2.1-2.2 GHz under it), with the
// gated product's backward pass 2,530 against 2,920.  The tiles of one
// segment run on one XCD, whose L2 then serves the segment's rows to all of
// them.  The workgroups of the first tile column also add up the columns of
// the dZ rows they copy (no measurable cost).  Segments are written as
// partial tiles and joined in order by a second launch.
#include "emu_block_device.h"
#include "emu_block_launch.h"
#include "emu_tile.h"

namespace emu {
namespace {


// Where the rows of dZ come from: memory (WG_PLAIN), or an activation's
// backward pass that runs on the way to LDS and also writes dZ for the
// input-gradient product: dZ = dY act'(Z) (WG_ACT), or with Z = [g | u]
// dZ = [dY u act'(g) | dY act(g)] (WG_GATED).
enum { WG_PLAIN = 0, WG_ACT = 1, WG_GATED = 2 };

struct WgradArgs {
    const float* Z;        // WG_PLAIN: dZ; else the pre-activations
    const float* X;
    const float* Y;        // WG_ACT, WG_GATED: dY
    float* dZ;             // and the result
    int64_t ldz, ldx, ldy, ldd, rows;
    int M, N;              // columns of dZ (WG_GATED: of each half) and of X
    int tiles_n, tiles;
    int segs, seg_steps;   // segments of seg_steps slabs
    float* out;            // dW, or the partial results: seg * pstride + m * ldo + n
    int64_t ldo, pstride;
    float* db;             // db, or its partials: seg * bstride + m; or null
    int64_t bstride;
};

// WN: waves along N (2 or 4), 64 columns of dW each.
template <int SRC, int ACT, int WN>
__global__ __launch_bounds__(128 * WN, 2) void wgrad_kernel(WgradArgs p)
{
    constexpr int NT = 128 * WN, TN = 64 * WN;
    // columns of dZ per tile and half, 16-byte groups of a row, and copies of
    // a slab per thread
    constexpr int TW = SRC == WG_GATED ? TILE / 2 : TILE;
    constexpr int PER_ROW = TW / 4, ROWS = NT / PER_ROW, COPIES = BK / ROWS;
    constexpr int X_ROWS = NT / (TN / 4);
    static_assert(X_ROWS * 4 == BK && ROWS * COPIES == BK, "four copies of X per thread and slab");
    constexpr int HALVES = SRC == WG_GATED ? 2 : 1;
    constexpr int READS = SRC == WG_PLAIN ? 1 : SRC == WG_ACT ? 2 : 3;   // arrays behind dZ
    __shared__ __attribute__((aligned(16))) float smZ[2][BK * TILE];
    __shared__ __attribute__((aligned(16))) float smX[2][BK * TN];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave / WN, wn = wave % WN;

    const int item = xcd_position(blockIdx.x, gridDim.x);
    const int seg = item / p.tiles;
    const int tile = item - seg * p.tiles;
    const int tm = tile / p.tiles_n, tn = tile - tm * p.tiles_n;
    const int m0 = tm * TW, n0 = tn * TN;
    const int64_t k0 = (int64_t)seg * p.seg_steps * BK;
    int64_t kend = k0 + (int64_t)p.seg_steps * BK;
    if (kend > p.rows) kend = p.rows;
    const int steps = (int)((kend - k0 + BK - 1) / BK);

    // Thread t copies columns 4 (t % PER_ROW) .. +3 of rows t / PER_ROW + ROWS
    // r of a slab of dZ (and of what it is made of), and likewise of X.  The buffer descriptors end with the segment's
    // last row, so rows past it read as zeros (and are not written); columns
    // past M (N) read what follows in memory, or zeros, and only feed outputs
    // that are not stored.
    const int cr = t / PER_ROW, cc = (t % PER_ROW) * 4;
    const int xr = t / (TN / 4), xc = (t % (TN / 4)) * 4;
    const int mleft = p.M - m0, nleft = p.N - n0;
    const int zcols = SRC == WG_GATED ? 2 * p.M - m0 : mleft;   // from m0 to the end of Z's row
    u32x4_t rz[READS][COPIES], rx[4];
    __amdgpu_buffer_rsrc_t bz, bx, by, bd;   // the slab that is loaded next; bd: that is written now
    auto rows_from = [&](int step) __attribute__((always_inline)) {
        const int64_t left = kend - k0 - (int64_t)step * BK;
        return left < BK ? (int)left : BK;   // (none left: an empty buffer, zeros)
    };
    auto buffer = [&](const float* base, int64_t ld, int step, int cols) __attribute__((always_inline)) {
        const int rows = rows_from(step);
        // (cols 0: N = 0, X may be null)
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(base + (k0 + (int64_t)step * BK) * ld), (short)0,
                                                 rows > 0 && cols > 0 ? (int)((rows - 1) * ld + cols) * 4 : 0,
                                                 0x00020000);
    };
    auto aim = [&](int step) __attribute__((always_inline)) {
        bz = buffer(p.Z + m0, p.ldz, step, zcols);
        bx = buffer(p.X + n0, p.ldx, step, nleft);
        if (SRC != WG_PLAIN) by = buffer(p.Y + m0, p.ldy, step, mleft);
    };
    auto offset = [&](int64_t ld, int r) __attribute__((always_inline)) {
        return (uint32_t)((cr + ROWS * r) * ld + cc) * 4;
    };
    auto load_z = [&](int r) __attribute__((always_inline)) {
        rz[0][r] = __builtin_amdgcn_raw_buffer_load_b128(bz, offset(p.ldz, r), 0, 0);
        if constexpr (SRC != WG_PLAIN) rz[1][r] = __builtin_amdgcn_raw_buffer_load_b128(by, offset(p.ldy, r), 0, 0);
        if constexpr (SRC == WG_GATED)
            rz[2][r] = __builtin_amdgcn_raw_buffer_load_b128(bz, offset(p.ldz, r) + (uint32_t)p.M * 4, 0, 0);
    };
    auto load_x = [&](int r) __attribute__((always_inline)) {
        rx[r] = __builtin_amdgcn_raw_buffer_load_b128(bx, (uint32_t)((xr + X_ROWS * r) * p.ldx + xc) * 4, 0, 0);
    };
    const bool first_n = tn == 0;
    const bool sums = p.db != nullptr && first_n;
    f32x4_t bsum[HALVES] = {};   // column sums of the rows this thread copies
    f32x4_t dz[HALVES];          // the copy being made
    auto value = [&](const u32x4_t& v, int e) __attribute__((always_inline)) { return __uint_as_float(v[e]); };
    auto make = [&](int r, int e) __attribute__((always_inline)) {
        if constexpr (SRC == WG_PLAIN) {
            dz[0][e] = value(rz[0][r], e);
        } else if constexpr (SRC == WG_ACT) {
            dz[0][e] = value(rz[1][r], e) * act_slope<ACT, 1>(value(rz[0][r], e));
        } else {
            float a, d;
            act_both<ACT>(value(rz[0][r], e), a, d);
            const float dy = value(rz[1][r], e);
            dz[0][e] = dy * value(rz[2][r], e) * d;
            dz[HALVES - 1][e] = dy * a;
        }
    };
    auto put = [&](int b, int r) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            *reinterpret_cast<f32x4_t*>(&smZ[b][(cr + ROWS * r) * TILE + h * TW + cc]) = dz[h];
            if (sums) bsum[h] = bsum[h] + dz[h];
            if (SRC != WG_PLAIN && first_n) {
                const uint32_t off = offset(p.ldd, r) + (uint32_t)(h * p.M) * 4;
                if (cc + 4 <= mleft) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, dz[h]), bd, off, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (cc + e < mleft)
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(dz[h][e]), bd, off + 4 * e, 0, 0);
                }
            }
        }
    };
    auto put_x = [&](int b, int r) __attribute__((always_inline)) {
        *reinterpret_cast<u32x4_t*>(&smX[b][(xr + X_ROWS * r) * TN + xc]) = rx[r];
    };

    f32x16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};

    // Block i (j) of a wave's 64 rows (columns) of dW holds the rows 2 l + i
    // of lanes l = 0..31: one 8-byte LDS read then gives both blocks' element.
    const int fz = (lane >> 5) * TILE + wm * 64 + 2 * (lane & 31);
    const int fx = (lane >> 5) * TN + wn * 64 + 2 * (lane & 31);
    auto read_z = [&](const float* sm, int k) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x2_t*>(&sm[k * TILE + fz]);
    };
    auto read_x = [&](const float* sm, int k) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x2_t*>(&sm[k * TN + fx]);
    };
    // Slab s is in LDS buffer s % 2.  During its step slab s + 1 goes to the
    // other buffer from the registers it was read to during step s - 1 (with
    // the activation's backward pass on the way, one element of a copy per k
    // pair), and slab s + 2 is requested into them, a copy at a time between
    // the products, so that the matrix unit never waits for a wave's copies.
    aim(0);
#pragma unroll
    for (int r = 0; r < COPIES; ++r) load_z(r);
#pragma unroll
    for (int r = 0; r < 4; ++r) load_x(r);
    aim(1);
    if (SRC != WG_PLAIN) bd = buffer(p.dZ + m0, p.ldd, 0, zcols);
#pragma unroll
    for (int r = 0; r < COPIES; ++r) {
#pragma unroll
        for (int e = 0; e < 4; ++e) make(r, e);
        put(0, r);
        load_z(r);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        put_x(0, r);
        load_x(r);
    }
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
    for (int s = 0; s < steps; ++s) {
        const int b = s & 1;
        const float *sz = smZ[b], *sx = smX[b];
        // the operands of each k pair are read while the one before is
        // multiplied
        f32x2_t a[2], c[2];
        a[0] = read_z(sz, 0);
        c[0] = read_x(sx, 0);
        aim(s + 2);
        if (SRC != WG_PLAIN) bd = buffer(p.dZ + m0, p.ldd, s + 1, zcols);
#pragma unroll
        for (int k = 0; k < BK / 2; ++k) {
            if (k + 1 < BK / 2) {
                a[(k + 1) & 1] = read_z(sz, 2 * k + 2);
                c[(k + 1) & 1] = read_x(sx, 2 * k + 2);
            }
            if (k % 4 == 2) {
                put_x(b ^ 1, k / 4);
                load_x(k / 4);
            }
            if (k % 4 == 0 && k > 0 && k / 4 <= COPIES) {
                put(b ^ 1, k / 4 - 1);
                load_z(k / 4 - 1);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (k / 4 < COPIES) make(k / 4, k % 4);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    // X first: lane l then holds one row of dW and four
                    // columns per register group
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(c[k & 1][j], a[k & 1][i], acc[i][j], 0, 0, 0);
            if (SRC != WG_PLAIN && k / 4 < COPIES) {
                // the activation's vector work between the products
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x402, 8, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (COPIES == 4) {
            put(b ^ 1, 3);
            load_z(3);
        }
        wait_lgkmcnt0();   // this step's writes and reads
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }

    // dZ column m of the tile is row (of dW) row_of(m), if valid
    auto row_of = [&](int m) __attribute__((always_inline)) {
        return SRC == WG_GATED && m >= TW ? p.M + m0 + m - TW : m0 + m;
    };
    auto valid = [&](int m) __attribute__((always_inline)) { return (m % TW) < mleft; };
    float* out = p.out + seg * p.pstride;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = wm * 64 + 2 * (lane & 31) + i;
        if (valid(m)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // columns 2 p + j for p = 8 q + 4 (l / 32) .. +3
                const int n = n0 + wn * 64 + 16 * q + 8 * (lane >> 5);
                const f32x4_t u = {acc[i][0][4 * q], acc[i][1][4 * q], acc[i][0][4 * q + 1], acc[i][1][4 * q + 1]};
                const f32x4_t v = {acc[i][0][4 * q + 2], acc[i][1][4 * q + 2], acc[i][0][4 * q + 3], acc[i][1][4 * q + 3]};
                store4(out + (int64_t)row_of(m) * p.ldo, n, p.N, u);
                store4(out + (int64_t)row_of(m) * p.ldo, n + 4, p.N, v);
            }
        }
    }
    if (sums) {
        // (every wave has passed the last step's barrier: the slabs are free)
        float* sum = smZ[0];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) *reinterpret_cast<f32x4_t*>(&sum[cr * TILE + h * TW + cc]) = bsum[h];
        wait_lgkmcnt0();
        __builtin_amdgcn_s_barrier();
        if (t < TILE && valid(t)) {
            float v = sum[t];
#pragma unroll
            for (int r = 1; r < ROWS; ++r) v = v + sum[r * TILE + t];
            p.db[seg * p.bstride + row_of(t)] = v;
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
    int wn;           // waves along N
    int64_t tiles_m, tiles_n, tiles;
    int segs, seg_steps;
    int64_t ldp;      // row of a partial result
    int64_t rows_out; // rows of dW
    double load;      // of the busiest CU, in products of a 128-column tile and slab
};

// Segments for tiles of 64 wn columns: the load of the busiest CU is ceil(tiles
// * segs / 256) segment tiles of ceil(steps / segs) slabs; the fewest segments
// within 5 % of the least load, 128 at most and 4 slabs each at least.
WgradPlan plan_wgrad(int64_t rows, int64_t M, int64_t N, bool gated, int wn)
{
    WgradPlan p;
    p.wn = wn;
    const int64_t tw = gated ? TILE / 2 : TILE, tn = 64 * wn;
    p.rows_out = gated ? 2 * M : M;
    p.tiles_m = (M + tw - 1) / tw;
    p.tiles_n = N > 0 ? (N + tn - 1) / tn : 1;
    p.tiles = p.tiles_m * p.tiles_n;
    const int64_t steps = (rows + BK - 1) / BK;
    int64_t most = steps / 4;
    if (most > 128) most = 128;
    if (most < 1) most = 1;
    auto load = [&](int64_t s) {
        const int64_t items = p.tiles * s, per = (steps + s - 1) / s;
        // (two workgroups of 128 columns share a CU and hide each other's
        // waits: one alone takes about a quarter longer per slab)
        const double slab = wn == 4 ? 2.0 : items <= 256 ? 1.25 : 1.0;
        return (double)((items + 255) / 256) * (double)per * slab + 0.25 * (double)s;
    };
    double best = load(1);
    for (int64_t s = 2; s <= most; ++s)
        if (load(s) < best) best = load(s);
    int64_t segs = 1;
    while (segs < most && load(segs) > 1.05 * best) ++segs;
    p.load = load(segs);
    p.seg_steps = (int)((steps + segs - 1) / segs);
    if (p.seg_steps < 1) p.seg_steps = 1;
    p.segs = (int)((steps + p.seg_steps - 1) / p.seg_steps);
    if (p.segs < 1) p.segs = 1;
    p.ldp = (N + 3) & ~(int64_t)3;
    return p;
}

WgradPlan plan_wgrad(int64_t rows, int64_t M, int64_t N, bool gated)
{
    const WgradPlan narrow = plan_wgrad(rows, M, N, gated, 2);
    if (N <= 128) return narrow;
    const WgradPlan wide = plan_wgrad(rows, M, N, gated, 4);
    return wide.load <= narrow.load ? wide : narrow;
}

template <int SRC, int WN>
void launch_src(int act, int grid, const WgradArgs& a, hipStream_t s)
{
    auto go = [&]<int ACT>() {
        hipLaunchKernelGGL((wgrad_kernel<SRC, ACT, WN>), dim3(grid), dim3(128 * WN), 0, s, a);
    };
    if constexpr (SRC == WG_PLAIN) {
        go.template operator()<EMU_ACT_IDENTITY>();
    } else {
        switch (act) {
        case EMU_ACT_RELU: go.template operator()<EMU_ACT_RELU>(); break;
        case EMU_ACT_SILU: go.template operator()<EMU_ACT_SILU>(); break;
        case EMU_ACT_GELU: go.template operator()<EMU_ACT_GELU>(); break;
        case EMU_ACT_GELU_TANH: go.template operator()<EMU_ACT_GELU_TANH>(); break;
        case EMU_ACT_TANH: go.template operator()<EMU_ACT_TANH>(); break;
        default: go.template operator()<EMU_ACT_IDENTITY>(); break;
        }
    }
}

}  // namespace

size_t wgrad_workspace(int64_t rows, int64_t M, int64_t N, bool gated)
{
    const WgradPlan p = plan_wgrad(rows, M, N, gated);
    return p.segs > 1 ? (size_t)p.segs * (size_t)(p.rows_out * p.ldp + ((p.rows_out + 3) & ~(int64_t)3)) * sizeof(float) : 0;
}

hipError_t launch_wgrad(int64_t rows, int64_t M, int64_t N, const WgradSource& src, const float* X, int64_t ldx,
                        float* dW, int64_t lddw, float* db, void* ws, hipStream_t s)
{
    const WgradPlan pl = plan_wgrad(rows, M, N, src.gated);
    if (pl.tiles * pl.segs >= ((int64_t)1 << 31) || src.ldz > kWgradMaxLd || ldx > kWgradMaxLd ||
        src.ldy > kWgradMaxLd || src.ldd > kWgradMaxLd || pl.rows_out >= ((int64_t)1 << 31) - TILE ||
        N >= ((int64_t)1 << 31) - TILE)
        return hipErrorInvalidValue;
    WgradArgs a{};
    a.Z = src.Z;
    a.ldz = src.ldz;
    a.Y = src.dY;
    a.ldy = src.ldy;
    a.dZ = src.dZ;
    a.ldd = src.ldd;
    a.X = X;
    a.ldx = ldx;
    a.rows = rows;
    a.M = (int)M;
    a.N = (int)N;
    a.tiles_n = (int)pl.tiles_n;
    a.tiles = (int)pl.tiles;
    a.segs = pl.segs;
    a.seg_steps = pl.seg_steps;
    float* part = static_cast<float*>(ws);
    const int64_t pstride = pl.rows_out * pl.ldp;
    const int64_t bstride = (pl.rows_out + 3) & ~(int64_t)3;
    float* bpart = part + pl.segs * pstride;
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
    const int grid = (int)(pl.tiles * pl.segs);
    auto launch = [&]<int WN>() {
        if (src.gated)
            launch_src<WG_GATED, WN>(src.act, grid, a, s);
        else if (src.dY != nullptr)
            launch_src<WG_ACT, WN>(src.act, grid, a, s);
        else
            launch_src<WG_PLAIN, WN>(0, grid, a, s);
    };
    if (pl.wn == 4)
        launch.template operator()<4>();
    else
        launch.template operator()<2>();
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && pl.segs > 1) {
        const int64_t work = pl.rows_out * (pl.ldp / 4) + (db != nullptr ? bstride / 4 : 0);
        if ((work + 63) / 64 >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
        hipLaunchKernelGGL(wgrad_join_kernel, dim3((int)((work + 63) / 64)), dim3(256), 0, s, part, pl.segs, pstride,
                           pl.ldp, (int)pl.rows_out, (int)N, dW, lddw, bpart, bstride, db);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace emu
