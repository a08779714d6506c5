// The emulated product of few rows with its epilogue in one launch
// (emu_sgemm_act and emu_sgemm_gated of include/emu_block.h in the explicit
// emulated modes): the values of the 128-wide tiles' kernel (emu_gemm_pp.h)
// bit for bit, where those tiles would leave most CUs without one.
//
// Every element of the product is a chain over k per band, each link one
// v_mfma_f32_32x32x16_bf16, and the chain's order is the method's: k is not
// split.  What can run side by side are the tiles and the bands, so a
// workgroup owns 32 rows and 32 columns (gated: 16 gates and the same 16
// ups), and its first four waves, one per SIMD, take the bands: with nine
// products band 2 (three of them), 1, 3 and the pair 0, 4 (two each), with
// six 2, 1 and 0.  The other four waves feed them: each chunk of KC k of A
// and B is read from memory as it is (any alignment; columns behind K read
// as zeros), split to its BF16 planes in registers and written to LDS, one
// chunk ahead of the products, its loads two chunks ahead.  Weights that
// come as planes are copied.  No workspace, no launch for the weights'
// split.  The chain bounds it: KC / 16 k-steps of three MFMAs, 32 cycles
// each, and the LDS reads of their fragments beside them.
#include "emu_gemm_pp.h"

namespace emu {
namespace {

constexpr int FT = 32;                   // rows and columns of a workgroup's tile
constexpr int FPS = FT * LDS_ROW;        // elements per plane of 32 rows x 32 k
constexpr int kGroups = 2;               // groups of 256 threads that load and split
constexpr int kFeeders = 256 * kGroups;

// Where the B operand comes from.
enum { FB_ROWS = 0, FB_COLS = 1, FB_PLANES = 2 };   // N x K, K x N, planes

template <int NB, int KC, int SRC, bool GATED>
__global__ __launch_bounds__(256 + kFeeders) void few_gemm_kernel(int64_t M, int N, int K, const float* __restrict__ A,
                                                       int64_t lda, const float* __restrict__ B, int64_t ldb,
                                                       const uint16_t* __restrict__ planes, BlockEpilogue ep)
{
    static_assert(SRC != FB_COLS || !GATED, "the gated projection's weights are stored N x K");
    constexpr int NP = NB >= 3 ? 3 : NB;
    constexpr int S = KC / BK;           // 32-wide pieces of a chunk
    constexpr int PIECE = 2 * NP * FPS;  // elements of one: A's planes, B's planes
    constexpr int BUF = S * PIECE;
    constexpr int JOIN = NB * 4 * 64;    // f32x4_t of the bands' sums
    constexpr int BYTES = 2 * BUF * 2 > JOIN * 16 ? 2 * BUF * 2 : JOIN * 16;
    __shared__ __attribute__((aligned(16))) char smem[BYTES];
    uint16_t* const sm = reinterpret_cast<uint16_t*>(smem);

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t m0 = (int64_t)blockIdx.y * FT;
    const int tn = blockIdx.x;
    const int n0 = tn * (GATED ? FT / 2 : FT);   // first column of C
    const int chunks = (K + KC - 1) / KC;

    f32x4_t* const join = reinterpret_cast<f32x4_t*>(smem);
    // The products of bands B0 (and B1, if not negative) of every chunk.
    auto multiply = [&]<int B0, int B1>() __attribute__((always_inline)) {
        f32x16_t acc0 = {}, acc1 = {};
        const int off0 = plane_elem(lane & 31, (lane >> 5) * 8), off1 = plane_elem(lane & 31, 16 + (lane >> 5) * 8);
        // the planes that the bands read: band b takes u and v with u + v = b
        constexpr int HI = B0 > B1 ? B0 : B1;
        constexpr bool ALL = B1 >= 0;
        constexpr int LOW = ALL || B0 < NP ? 0 : B0 - NP + 1, TOP = ALL ? NP - 1 : (HI < NP ? HI : NP - 1);
        bf16x8_t fa[2][NP], fb[2][NP];
        // The fragments of 16-wide k-step i of a chunk.
        auto read = [&](const uint16_t* buf, int i) __attribute__((always_inline)) {
            const uint16_t* a = buf + (i >> 1) * PIECE + (i & 1 ? off1 : off0);
#pragma unroll
            for (int u = LOW; u <= TOP; ++u) {
                fa[i & 1][u] = *reinterpret_cast<const bf16x8_t*>(a + u * FPS);
                fb[i & 1][u] = *reinterpret_cast<const bf16x8_t*>(a + (NP + u) * FPS);
            }
        };
        // (as in the 128-wide tiles: A's smallest plane first)
        auto band = [&]<int BAND>(f32x16_t& acc, int i) __attribute__((always_inline)) {
#pragma unroll
            for (int u = NP - 1; u >= 0; --u)
                if (BAND - u >= 0 && BAND - u < NP)
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[i & 1][BAND - u], fa[i & 1][u], acc, 0, 0, 0);
        };
        __syncthreads();   // chunk 0 is there
        for (int c = 0; c < chunks; ++c) {
            const uint16_t* buf = sm + (c & 1) * BUF;
            read(buf, 0);
#pragma unroll
            for (int i = 0; i < 2 * S; ++i) {
                if (i + 1 < 2 * S) read(buf, i + 1);   // a step ahead of their use
                __builtin_amdgcn_sched_barrier(0);
                band.template operator()<B0>(acc0, i);
                if constexpr (B1 >= 0) band.template operator()<B1>(acc1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            join[(B0 * 4 + q) * 64 + lane] = f32x4_t{acc0[4 * q], acc0[4 * q + 1], acc0[4 * q + 2], acc0[4 * q + 3]};
            if constexpr (B1 >= 0)
                join[(B1 * 4 + q) * 64 + lane] = f32x4_t{acc1[4 * q], acc1[4 * q + 1], acc1[4 * q + 2], acc1[4 * q + 3]};
        }
    };
    auto idle = [&]() __attribute__((always_inline)) {
        for (int c = 0; c <= chunks; ++c) __syncthreads();
    };
    auto feed = [&]() __attribute__((always_inline)) {
        // quads of A and 16-byte loads of B per thread and chunk
        constexpr int PA = S / kGroups;
        constexpr int PB = SRC == FB_PLANES ? S * NP * FPS * 2 / (16 * kFeeders) : PA;
        static_assert(PA % 2 == 0 && PA * kGroups == S, "pairs of k of a K x N operand; planes in whole rounds");
        struct Chunk {
            f32x4_t a[PA];
            f32x4_t b[PB];
        };
        const int f = t - 256;
        const int nk = (K + BK - 1) / BK;
        const int grp = f >> 8, row = (f & 255) >> 3, kq = (f & 7) * 4;
        // a thread's quad j of A (and of an N x K operand) is row `row`, from
        // this k of the chunk on
        auto k_of = [&](int j) __attribute__((always_inline)) { return 32 * (kGroups * j + grp) + kq; };
        // of a K x N operand: columns nq .. nq + 3 of this k, and of the next
        // with the next j
        const int pair = 2 * (f >> 3), nq = n0 + kq;
        auto kn_of = [&](int j) __attribute__((always_inline)) { return 64 * kGroups * (j >> 1) + pair + (j & 1); };
        // rows and columns past the end repeat the last ones; they are not stored
        const float* arow = A + (m0 + row < M ? m0 + row : M - 1) * lda;
        const float* brow = B;
        if constexpr (SRC == FB_ROWS) {
            int64_t n = n0 + (GATED ? row & 15 : row);
            if (n >= N) n = N - 1;
            brow = B + (n + (GATED && row >= 16 ? N : 0)) * ldb;
        }
        // The same loads in every chunk: no branches and no masks, which would
        // make them wait for one another.  A quad that crosses K (or N, of
        // a K x N operand) is read from K - 4 on instead and moved up when
        // it is split (up4); K and, there, N are 4 or more.
        auto quad_at = [](const float* row, int i, int n) __attribute__((always_inline)) {
            return (f32x4_t)*reinterpret_cast<const f32x4u_t*>(row + (i < n - 4 ? i : n - 4));
        };
        // Elements i .. i + 3 of a row of n from the quad read for them;
        // zeros behind n.
        auto up4 = [](f32x4_t v, int i, int n) __attribute__((always_inline)) {
            const int d = i - (n - 4);   // up by d, if positive
            const bool one = d > 0 && (d & 1) != 0, two = d > 0 && (d & 2) != 0, out = d >= 4;
            f32x4_t r;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = one ? (e < 3 ? v[e < 3 ? e + 1 : 3] : 0.0f) : v[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = two ? (e < 2 ? v[e < 2 ? e + 2 : 3] : 0.0f) : v[e];
                r[e] = out ? 0.0f : x;
            }
            return r;
        };
        auto load = [&](int c, Chunk& v) __attribute__((always_inline)) {
            const int k0 = c * KC;
#pragma unroll
            for (int j = 0; j < PA; ++j) v.a[j] = quad_at(arow, k0 + k_of(j), K);
            if constexpr (SRC == FB_ROWS) {
#pragma unroll
                for (int j = 0; j < PB; ++j) v.b[j] = quad_at(brow, k0 + k_of(j), K);
            } else if constexpr (SRC == FB_COLS) {
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    const int k = k0 + kn_of(j);
                    v.b[j] = quad_at(brow + (k < K ? k : K - 1) * ldb, nq, N);
                }
            } else {
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    const int e = (j * kFeeders + f) * 8;   // element of the chunk's S x NP planes
                    const int s = e / (NP * FPS), r = e % (NP * FPS);
                    const int kt = c * S + s < nk ? c * S + s : nk - 1;
                    v.b[j] = *reinterpret_cast<const f32x4_t*>(
                        planes + (((int64_t)(tn >> 2) * nk + kt) * NP + r / FPS) * PS + (tn & 3) * FPS + r % FPS);
                }
            }
        };
        auto put = [&](int c, Chunk& v, uint16_t* buf) __attribute__((always_inline)) {
            if (c >= chunks) return;
            const int k0 = c * KC;
            if (k0 + KC > K) {
#pragma unroll
                for (int j = 0; j < PA; ++j) v.a[j] = up4(v.a[j], k0 + k_of(j), K);
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    if constexpr (SRC == FB_ROWS) {
                        v.b[j] = up4(v.b[j], k0 + k_of(j), K);
                    } else {
                        // (a row of a K x N operand, or a 32-wide piece of planes)
                        const bool inside =
                            SRC == FB_COLS ? k0 + kn_of(j) < K : c * S + (j * kFeeders + f) * 8 / (NP * FPS) < nk;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v.b[j][e] = inside ? v.b[j][e] : 0.0f;
                    }
                }
            }
            if (SRC == FB_COLS && n0 + FT > N) {
#pragma unroll
                for (int j = 0; j < PB; ++j) v.b[j] = up4(v.b[j], nq, N);
            }
            auto quad = [&](f32x4_t x, uint16_t* dst) __attribute__((always_inline)) {
                uint32_t w0[NP], w1[NP];
                split_pieces<NP>(x[0], x[1], w0);
                split_pieces<NP>(x[2], x[3], w1);
#pragma unroll
                for (int pl = 0; pl < NP; ++pl) *reinterpret_cast<u32x2_t*>(dst + pl * FPS) = u32x2_t{w0[pl], w1[pl]};
            };
#pragma unroll
            for (int j = 0; j < PA; ++j) quad(v.a[j], buf + (kGroups * j + grp) * PIECE + plane_elem(row, kq));
            if constexpr (SRC == FB_ROWS) {
#pragma unroll
                for (int j = 0; j < PB; ++j) quad(v.b[j], buf + (kGroups * j + grp) * PIECE + NP * FPS + plane_elem(row, kq));
            } else if constexpr (SRC == FB_COLS) {
#pragma unroll
                for (int j = 0; j < PB; j += 2) {
                    const int k = kn_of(j);
                    uint16_t* dst = buf + (k >> 5) * PIECE + NP * FPS;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[NP];
                        split_pieces<NP>(v.b[j][e], v.b[j + 1][e], w);
#pragma unroll
                        for (int pl = 0; pl < NP; ++pl)
                            *reinterpret_cast<uint32_t*>(dst + pl * FPS + plane_elem(kq + e, k & 31)) = w[pl];
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    const int e = (j * kFeeders + f) * 8;
                    const int s = e / (NP * FPS), r = e % (NP * FPS);
                    *reinterpret_cast<f32x4_t*>(buf + s * PIECE + NP * FPS + r) = v.b[j];
                }
            }
        };
        Chunk v[2];
        load(0, v[0]);
        load(1, v[1]);
        put(0, v[0], sm);
        load(2, v[0]);
        __syncthreads();
        for (int c = 0;; c += 2) {
            // chunk c is multiplied, c + 1 split, c + 3 requested
            put(c + 1, v[1], sm + BUF);
            load(c + 3, v[1]);
            __syncthreads();
            if (c + 1 >= chunks) break;
            put(c + 2, v[0], sm);
            load(c + 4, v[0]);
            __syncthreads();
            if (c + 2 >= chunks) break;
        }
    };
    if (wave >= 4) {
        feed();
    } else if constexpr (NB == 5) {
        if (wave == 0) multiply.template operator()<2, -1>();
        else if (wave == 1) multiply.template operator()<1, -1>();
        else if (wave == 2) multiply.template operator()<3, -1>();
        else multiply.template operator()<0, 4>();
    } else {
        // (the largest band, with the most products, first)
        if (wave == 0) multiply.template operator()<NB - 1, -1>();
        else if (NB >= 2 && wave == 1) multiply.template operator()<(NB >= 2 ? NB - 2 : 0), -1>();
        else if (NB >= 3 && wave == 2) multiply.template operator()<0, -1>();
        else idle();
    }
    __syncthreads();

    // Lane l of register group q: row l % 32, columns 8 q + 4 (l / 32) .. +3;
    // gated: groups 0, 1 are the gates of 2, 3.
    if (t >= (GATED ? 128 : 256)) return;
    const int64_t m = m0 + (lane & 31);
    const int col = n0 + 8 * wave + 4 * (lane >> 5);
    if (m >= M || col >= N) return;
    constexpr int Z = GATED ? 2 : 1;
    f32x4_t z[Z];
#pragma unroll
    for (int g = 0; g < Z; ++g) {
        const int q = wave + 2 * g;
        z[g] = join[((NB - 1) * 4 + q) * 64 + lane];
#pragma unroll
        for (int b = NB - 2; b >= 0; --b) {
            const f32x4_t u = join[(b * 4 + q) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[g][e] = __builtin_fmaf(z[g][e], 0.00390625f, u[e]);
        }
        if (ep.bias != nullptr) z[g] = z[g] + load4(ep.bias + (int64_t)g * N, col, N);
        if (ep.Z != nullptr) store4(ep.Z + m * ep.ldz + (int64_t)g * N, col, N, z[g]);
    }
    f32x4_t o;
    with_act(ep.act, [&]<int ACT>() {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = act_value<ACT>(z[0][e]);
    });
    if constexpr (GATED)
        o = o * z[Z - 1];
    else if (ep.R != nullptr)
        o = o + load4(ep.R + m * ep.ldr, col, N);
    store4(ep.C + m * ep.ldc, col, N, o);
}

template <int NB>
void launch_bands(bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, const float* B,
                  int64_t ldb, const uint16_t* planes, const BlockEpilogue& ep, hipStream_t s)
{
    constexpr int KC = 128;
    const int64_t cols = ep.gated ? FT / 2 : FT;
    const dim3 grid((unsigned)((N + cols - 1) / cols), (unsigned)((M + FT - 1) / FT));
    auto go = [&]<int SRC, bool GATED>() {
        hipLaunchKernelGGL((few_gemm_kernel<NB, KC, SRC, GATED>), grid, dim3(256 + kFeeders), 0, s, M, (int)N, (int)K, A, lda, B, ldb,
                           planes, ep);
    };
    if (ep.gated && planes != nullptr)
        go.template operator()<FB_PLANES, true>();
    else if (ep.gated)
        go.template operator()<FB_ROWS, true>();
    else if (planes != nullptr)
        go.template operator()<FB_PLANES, false>();
    else if (trans_b)
        go.template operator()<FB_ROWS, false>();
    else
        go.template operator()<FB_COLS, false>();
}

}  // namespace

hipError_t launch_few_gemm(int nbands, bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                           const float* B, int64_t ldb, const uint16_t* planes, const BlockEpilogue& ep, hipStream_t s)
{
    if (M > (int64_t)65535 * FT || 2 * N >= ((int64_t)1 << 31) || K < 4 || (!trans_b && N < 4) || K >= ((int64_t)1 << 30) ||
        (ep.gated && !trans_b && planes == nullptr))
        return hipErrorInvalidValue;
    switch (nbands) {
    case 5: launch_bands<5>(trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    case 3: launch_bands<3>(trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    case 2: launch_bands<2>(trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    case 1: launch_bands<1>(trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace emu
