// The emulated product of few rows with its epilogue in one launch
// (emu_sgemm_act and emu_sgemm_gated of include/emu_block.h): the values of the
// 128-wide tiles' kernel (emu_gemm_pp.h) bit for bit, where those tiles would
// leave most CUs without one.
//
// Every element of the product is a chain over k per band, each link one
// v_mfma_f32_32x32x16_bf16, and the chain's order is the method's: k is not
// split.  What can run side by side are tiles and bands.  T = 1: a workgroup
// owns 32 rows and 32 columns (gated: 16 gates and the same 16 ups), and its
// first four waves, one per SIMD, take the bands: with nine products band 2
// (three of them), 1, 3 and the pair 0, 4 (two each), with six 2, 1 and 0.
// T = 2: 64 rows and 64 columns, an MFMA tile with all its bands per wave,
// half the splitting per element for shapes that have such tiles for every CU
// (1,024 x 1024 -> 1024, nine products: 24.4 us, T = 1: 43.1).
// The other waves feed them: each chunk of k of A and B (128, T = 2: 64 or 32)
// is read from memory as it is (any alignment; zeros behind K), split to its
// BF16 planes in registers and written to LDS, one chunk ahead of the products,
// its loads two chunks ahead.  Eight feeding waves (four: 12.0 us, not 10.4,
// for 1 x 1024 -> 1024), or four with chunks of 32 where there are more tiles
// than CUs: half the LDS, so that two workgroups share a CU and one's products
// run beside the other's waits (5,003 x 387 -> 771, six products: 42 us, and
// 61 with the 128-wide tiles; 20,000 x 64 -> 64 9.4 -> 7.4).  Weights that come
// as planes are copied.  No workspace, no launch for the weights' split.
// What bounds it: the split, about 10 vector instructions per element of 64
// (128) rows per chunk, with the MFMAs on the same SIMDs: 0.85 us per chunk
// with nine products, 0.72 with three.  64 x 1024 -> 4096, nine products:
// 11.8 us, where reading the weights takes 3.2; the 128-wide tiles 48.7.
#include "emu_gemm_pp.h"

namespace emu {
namespace {

constexpr int FT = 32;                   // rows and columns of an MFMA tile
constexpr int FPS = FT * LDS_ROW;        // elements per plane of 32 rows x 32 k

// Where the B operand comes from.
enum { FB_ROWS = 0, FB_COLS = 1, FB_PLANES = 2 };   // N x K, K x N, planes

// T: a workgroup's tile is 32 T rows by 32 T columns (gated: 16 T gates and
// the same 16 T ups).  FEED: threads that load and split, two quads of each
// operand per chunk.
template <int NB, int T, int FEED, int SRC, bool GATED>
__global__ __launch_bounds__(256 + FEED, FEED == 256 ? 4 : 1) void few_gemm_kernel(int64_t M, int N, int K, const float* __restrict__ A,
                                                            int64_t lda, const float* __restrict__ B, int64_t ldb,
                                                            const uint16_t* __restrict__ planes, BlockEpilogue ep)
{
    static_assert(SRC != FB_COLS || !GATED, "the gated projection's weights are stored N x K");
    static_assert(T == 1 || T == 2, "one MFMA tile by its bands, or four");
    constexpr int NP = NB >= 3 ? 3 : NB;
    constexpr int KC = FEED / (4 * T);     // k of a chunk
    constexpr int S = KC / BK;             // 32-wide pieces of it
    constexpr int PLANE = T * FPS;         // elements of a plane of one piece
    constexpr int PIECE = 2 * NP * PLANE;  // A's planes, B's planes
    constexpr int BUF = S * PIECE;
    constexpr int JB = T == 1 ? NB : 1;    // sums per element at the end: the bands', or theirs together
    constexpr int JOIN = JB * T * T * 4 * 64;
    constexpr int BYTES = 2 * BUF * 2 > JOIN * 16 ? 2 * BUF * 2 : JOIN * 16;
    __shared__ __attribute__((aligned(16))) char smem[BYTES];
    uint16_t* const sm = reinterpret_cast<uint16_t*>(smem);
    f32x4_t* const join = reinterpret_cast<f32x4_t*>(smem);

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t m0 = (int64_t)blockIdx.y * (FT * T);
    const int tn = blockIdx.x;
    const int n0 = tn * (GATED ? FT * T / 2 : FT * T);   // first column of C
    const int chunks = (K + KC - 1) / KC;

    // The chunks' products in the bands of BANDS for one MFMA tile.
    auto multiply = [&]<int... BANDS>() __attribute__((always_inline)) {
        constexpr int n = sizeof...(BANDS);
        constexpr int bands[n] = {BANDS...};
        // planes that they read: band b takes u and v with u + v = b
        constexpr int one = bands[0];
        constexpr int LOW = n > 1 || one < NP ? 0 : one - NP + 1, TOP = n > 1 || one >= NP ? NP - 1 : one;
        f32x16_t acc[n];
#pragma unroll
        for (int i = 0; i < n; ++i) acc[i] = f32x16_t{};
        const int off0 = plane_elem(lane & 31, (lane >> 5) * 8), off1 = plane_elem(lane & 31, 16 + (lane >> 5) * 8);
        const uint16_t* const mine_a = sm + (T == 1 ? 0 : (wave & 1) * FPS);
        const uint16_t* const mine_b = sm + NP * PLANE + (T == 1 ? 0 : (wave >> 1) * FPS);
        // Fragments are read a group ahead of their MFMAs: a group is a 16-wide
        // k-step of the chunk (T = 1, of few MFMAs), or one plane u of A in it
        // (T = 2), with B's planes at the step's first.
        constexpr int NU = TOP - LOW + 1, PER = T == 1 ? 1 : NU, GROUPS = 2 * S * PER;
        bf16x8_t fa[2][NP], fb[2][NP];
        auto read = [&](int b, int g) __attribute__((always_inline)) {
            const int i = g / PER;
            const int at = b * BUF + (i >> 1) * PIECE + (i & 1 ? off1 : off0);
#pragma unroll
            for (int v = TOP; v >= LOW; --v) {
                if (g % PER == 0) fb[i & 1][v] = *reinterpret_cast<const bf16x8_t*>(mine_b + at + v * PLANE);
                if (PER == 1 || v == TOP - g % PER)
                    fa[g & 1][v] = *reinterpret_cast<const bf16x8_t*>(mine_a + at + v * PLANE);
            }
        };
        __builtin_amdgcn_s_setprio(2);   // their SIMD's other waves split beside them
        __syncthreads();   // chunk 0 is there
        for (int c = 0; c < chunks; ++c) {
            const int b = c & 1;
            read(b, 0);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                if (g + 1 < GROUPS) read(b, g + 1);
                __builtin_amdgcn_sched_barrier(0);
                // (as in the 128-wide tiles: A's smallest plane first, and
                // with it B's)
#pragma unroll
                for (int u = TOP; u >= LOW; --u)
#pragma unroll
                    for (int v = TOP; v >= LOW; --v)
#pragma unroll
                        for (int j = 0; j < n; ++j)
                            if (bands[j] == u + v && (PER == 1 || u == TOP - g % PER))
                                acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[g / PER & 1][v], fa[g & 1][u], acc[j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (T == 1) {
#pragma unroll
                for (int j = 0; j < n; ++j)
                    join[(bands[j] * 4 + q) * 64 + lane] =
                        f32x4_t{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
            } else {
                // the bands in order: 0 .. NB - 1
                f32x4_t z;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float sum = acc[n - 1][4 * q + e];
#pragma unroll
                    for (int j = n - 2; j >= 0; --j) sum = __builtin_fmaf(sum, 0.00390625f, acc[j][4 * q + e]);
                    z[e] = sum;
                }
                join[(wave * 4 + q) * 64 + lane] = z;
            }
        }
    };
    auto idle = [&]() __attribute__((always_inline)) {
        for (int c = 0; c <= chunks; ++c) __syncthreads();
    };
    auto feed = [&]() __attribute__((always_inline)) {
        // quads of A and 16-byte loads of B per thread and chunk
        constexpr int PA = 32 * T * KC / 4 / FEED;
        constexpr int PB = SRC == FB_PLANES ? S * NP * PLANE * 2 / (16 * FEED) : PA;
        static_assert(PA == 2, "a pair of k of a K x N operand");
        struct Chunk {
            f32x4_t a[PA];
            f32x4_t b[PB];
        };
        const int f = t - 256;
        const int nk = (K + BK - 1) / BK;
        // a thread's quad j of A (and of an N x K operand): this row, in
        // this piece four k from kq on
        const int kq = (f & 7) * 4;
        auto row_of = [&](int j) __attribute__((always_inline)) { return (j * (FEED / 8) + (f >> 3)) % (32 * T); };
        auto piece_of = [&](int j) __attribute__((always_inline)) { return (j * (FEED / 8) + (f >> 3)) / (32 * T); };
        // of a K x N operand: columns nq .. nq + 3 of chunk rows pair, pair + 1
        const int pair = f / (8 * T) * 2, nr = f % (8 * T) * 4, nq = n0 + nr;
        // rows and columns past the end repeat the last ones; they are not stored
        const float *arow[PA], *brow[PA];
#pragma unroll
        for (int j = 0; j < PA; ++j) {
            const int row = row_of(j);
            arow[j] = A + (m0 + row < M ? m0 + row : M - 1) * lda;
            brow[j] = B;
            if constexpr (SRC == FB_ROWS) {
                int64_t n = n0 + (GATED ? (row >> 5) * 16 + (row & 15) : row);
                if (n >= N) n = N - 1;
                brow[j] = B + (n + (GATED && (row & 16) != 0 ? N : 0)) * ldb;
            }
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
        // element j of the thread's share of the chunk's planes of B
        auto plane_at = [&](int j) __attribute__((always_inline)) { return (j * FEED + f) * 8; };
        auto load = [&](int c, Chunk& v) __attribute__((always_inline)) {
            const int k0 = c * KC;
#pragma unroll
            for (int j = 0; j < PA; ++j) v.a[j] = quad_at(arow[j], k0 + 32 * piece_of(j) + kq, K);
#pragma unroll
            for (int j = 0; j < PB; ++j) {
                if constexpr (SRC == FB_ROWS) {
                    v.b[j] = quad_at(brow[j], k0 + 32 * piece_of(j) + kq, K);
                } else if constexpr (SRC == FB_COLS) {
                    const int k = k0 + pair + j;
                    v.b[j] = quad_at(B + (k < K ? k : K - 1) * ldb, nq, N);
                } else {
                    const int s = plane_at(j) / (NP * PLANE), r = plane_at(j) % (NP * PLANE);
                    const int kt = c * S + s < nk ? c * S + s : nk - 1;
                    v.b[j] = *reinterpret_cast<const f32x4_t*>(
                        planes + (((int64_t)(tn / (4 / T)) * nk + kt) * NP + r / PLANE) * PS + tn % (4 / T) * PLANE + r % PLANE);
                }
            }
        };
        auto put = [&](int c, Chunk& v, uint16_t* buf) __attribute__((always_inline)) {
            if (c >= chunks) return;
            const int k0 = c * KC;
            if (k0 + KC > K) {
#pragma unroll
                for (int j = 0; j < PA; ++j) v.a[j] = up4(v.a[j], k0 + 32 * piece_of(j) + kq, K);
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    if constexpr (SRC == FB_ROWS) {
                        v.b[j] = up4(v.b[j], k0 + 32 * piece_of(j) + kq, K);
                    } else {
                        // (a row of a K x N operand, or a piece of planes)
                        const bool inside = SRC == FB_COLS ? k0 + pair + j < K : c * S + plane_at(j) / (NP * PLANE) < nk;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v.b[j][e] = inside ? v.b[j][e] : 0.0f;
                    }
                }
            }
            if (SRC == FB_COLS && n0 + FT * T > N) {
#pragma unroll
                for (int j = 0; j < PB; ++j) v.b[j] = up4(v.b[j], nq, N);
            }
            auto quad = [&](f32x4_t x, uint16_t* dst) __attribute__((always_inline)) {
                uint32_t w0[NP], w1[NP];
                split_pieces<NP>(x[0], x[1], w0);
                split_pieces<NP>(x[2], x[3], w1);
#pragma unroll
                for (int pl = 0; pl < NP; ++pl) *reinterpret_cast<u32x2_t*>(dst + pl * PLANE) = u32x2_t{w0[pl], w1[pl]};
            };
#pragma unroll
            for (int j = 0; j < PA; ++j) quad(v.a[j], buf + piece_of(j) * PIECE + plane_elem(row_of(j), kq));
            uint16_t* const bufb = buf + NP * PLANE;
            if constexpr (SRC == FB_COLS) {
                uint16_t* dst = bufb + (pair >> 5) * PIECE;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[NP];
                    split_pieces<NP>(v.b[0][e], v.b[1][e], w);
#pragma unroll
                    for (int pl = 0; pl < NP; ++pl)
                        *reinterpret_cast<uint32_t*>(dst + pl * PLANE + plane_elem(nr + e, pair & 31)) = w[pl];
                }
            } else {
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    if constexpr (SRC == FB_ROWS)
                        quad(v.b[j], bufb + piece_of(j) * PIECE + plane_elem(row_of(j), kq));
                    else
                        *reinterpret_cast<f32x4_t*>(bufb + plane_at(j) / (NP * PLANE) * PIECE + plane_at(j) % (NP * PLANE)) =
                            v.b[j];
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
    } else if constexpr (T == 2) {
        if constexpr (NB == 5) multiply.template operator()<0, 1, 2, 3, 4>();
        if constexpr (NB == 3) multiply.template operator()<0, 1, 2>();
        if constexpr (NB == 2) multiply.template operator()<0, 1>();
        if constexpr (NB == 1) multiply.template operator()<0>();
    } else if constexpr (NB == 5) {
        if (wave == 0) multiply.template operator()<2>();
        else if (wave == 1) multiply.template operator()<1>();
        else if (wave == 2) multiply.template operator()<3>();
        else multiply.template operator()<0, 4>();
    } else {
        // (the largest band, with the most products, first)
        if (wave == 0) multiply.template operator()<NB - 1>();
        else if (NB >= 2 && wave == 1) multiply.template operator()<(NB >= 2 ? NB - 2 : 0)>();
        else if (NB >= 3 && wave == 2) multiply.template operator()<0>();
        else idle();
    }
    __syncthreads();

    // Lane l of a tile's register group q: row l % 32, columns 8 q + 4 (l /
    // 32) .. +3; gated: groups 0, 1 are the gates of 2, 3.
    constexpr int Q = GATED ? 2 : 4;   // register groups of a tile that become columns of C
    for (int item = wave; item < T * T * Q; item += (256 + FEED) / 64) {
        const int tile = item / Q, q0 = item % Q;
        const int64_t m = m0 + (tile % T) * FT + (lane & 31);
        const int col = n0 + (tile / T) * (GATED ? FT / 2 : FT) + 8 * q0 + 4 * (lane >> 5);
        if (m >= M || col >= N) continue;
        constexpr int Z = GATED ? 2 : 1;
        f32x4_t z[Z];
#pragma unroll
        for (int g = 0; g < Z; ++g) {
            const f32x4_t* const sums = join + (tile * 4 + q0 + 2 * g) * 64 + lane;
            z[g] = sums[(JB - 1) * 4 * 64];
#pragma unroll
            for (int b = JB - 2; b >= 0; --b) {
                const f32x4_t u = sums[b * 4 * 64];
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
}

template <int NB>
void launch_bands(bool wide, bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                  const float* B, int64_t ldb, const uint16_t* planes, const BlockEpilogue& ep, hipStream_t s)
{
    auto go = [&]<int T, int FEED, int SRC, bool GATED>() {
        const int64_t cols = GATED ? FT * T / 2 : FT * T;
        const dim3 grid((unsigned)((N + cols - 1) / cols), (unsigned)((M + FT * T - 1) / (FT * T)));
        hipLaunchKernelGGL((few_gemm_kernel<NB, T, FEED, SRC, GATED>), grid, dim3(256 + FEED), 0, s, M, (int)N, (int)K, A,
                           lda, B, ldb, planes, ep);
    };
    auto tile = [&]<int T, int FEED>() {
        if (ep.gated && planes != nullptr)
            go.template operator()<T, FEED, FB_PLANES, true>();
        else if (ep.gated)
            go.template operator()<T, FEED, FB_ROWS, true>();
        else if (planes != nullptr)
            go.template operator()<T, FEED, FB_PLANES, false>();
        else if (trans_b)
            go.template operator()<T, FEED, FB_ROWS, false>();
        else
            go.template operator()<T, FEED, FB_COLS, false>();
    };
    if (!wide) return tile.template operator()<1, 512>();
    if constexpr (NB >= 3) {
        const int64_t tiles = (M + FT * 2 - 1) / (FT * 2) * (((ep.gated ? 2 * N : N) + FT * 2 - 1) / (FT * 2));
        if (tiles > 256) return tile.template operator()<2, 256>();
    }
    tile.template operator()<2, 512>();
}

}  // namespace

hipError_t launch_few_gemm(int nbands, bool wide, bool trans_b, int64_t M, int64_t N, int64_t K, const float* A,
                           int64_t lda, const float* B, int64_t ldb, const uint16_t* planes, const BlockEpilogue& ep,
                           hipStream_t s)
{
    if (M > (int64_t)65535 * FT || 2 * N >= ((int64_t)1 << 31) || K < 4 || (!trans_b && N < 4) ||
        K >= ((int64_t)1 << 30) || (ep.gated && !trans_b && planes == nullptr))
        return hipErrorInvalidValue;
    switch (nbands) {
    case 5: launch_bands<5>(wide, trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    case 3: launch_bands<3>(wide, trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    case 2: launch_bands<2>(wide, trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    case 1: launch_bands<1>(wide, trans_b, M, N, K, A, lda, B, ldb, planes, ep, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace emu
