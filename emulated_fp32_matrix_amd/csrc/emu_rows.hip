// The product of few rows with its epilogue in one launch (emu_sgemm_act and
// emu_sgemm_gated of include/emu_block.h in EMU_MODE_AUTO): one token, or the
// tokens of a few atoms, where a launch and one memory latency are most of
// the time.  (Where weights and rows are more, EMU_MODE_AUTO takes the
// emulated kernel of few rows, emu_few.hip.)
//
// FP32 on v_mfma_f32_16x16x4_f32, operands read from memory to registers as
// they are: no split of the weights, no LDS tiles, no second launch.  A
// workgroup owns 16 NT columns (gated: 16 gate and the same 16 up columns) of
// 16 MT rows; 32 columns, where they leave every CU a workgroup, halve the
// reads of A (2,048 x 512 x 256 14.4 -> 12.1 us, 512 x 1024 x 1024 23.8 ->
// 19.8); its 8 waves take every eighth 16-wide slice of k, so that the
// weights, which are what has to be read, stream with 8 waves' loads in
// flight, and their sums are added in LDS in wave order.  The instruction
// sums over 4 k per lane group; a lane's 16-byte load covers k = 16 c + 4 (l /
// 16) .. +3 and feeds one element to each of four instructions (both operands
// in the same order).
#include "emu_block_device.h"
#include "emu_block_launch.h"

namespace emu {
namespace {

constexpr int WAVES = 8;
constexpr int64_t kWide = 256;   // workgroups of 32 columns from which on they are used

template <bool TB, bool GATED, int MT, int NT>
__global__ __launch_bounds__(64 * WAVES) void rows_gemm_kernel(int64_t M, int N, int K, const float* __restrict__ A,
                                                               int64_t lda, const float* __restrict__ B,
                                                               int64_t ldb, BlockEpilogue ep)
{
    static_assert(TB || !GATED, "the gated projection's weights are stored N x K");
    static_assert(NT == 1 || !GATED, "a gated workgroup's second 16 columns are the up projection's");
    constexpr int G = GATED ? 2 : NT;    // 16-column fragments of the weights
    constexpr int U = MT == 4 ? 2 : 4;   // slices of k in flight per wave
    __shared__ __attribute__((aligned(16))) f32x4_t part[WAVES][MT * G][64];

    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int n0 = blockIdx.x * (16 * NT);
    const int kq = (lane >> 4) * 4;
    // rows and columns past the end repeat the last one; they are not stored
    int64_t bcol[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int n = n0 + (GATED ? 0 : 16 * g) + (lane & 15);
        bcol[g] = (n < N ? n : N - 1) + (GATED ? (int64_t)g * N : 0);
    }
    const float* arow[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + 16 * i + (lane & 15);
        arow[i] = A + (m < M ? m : M - 1) * lda;
    }
    auto load_b = [&](int k, int64_t col) __attribute__((always_inline)) {
        if constexpr (TB) {
            return load4(B + col * ldb, k, K);
        } else {
            f32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = k + e < K ? B[(int64_t)(k + e) * ldb + col] : 0.0f;
            return v;
        }
    };

    f32x4_t acc[MT][G];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int g = 0; g < G; ++g) acc[i][g] = f32x4_t{};

    const int slices = (K + 15) / 16;
    for (int c0 = wave; c0 < slices; c0 += WAVES * U) {
        f32x4_t b[U][G], a[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (c0 + u * WAVES) * 16 + kq;   // past the end: zeros
#pragma unroll
            for (int g = 0; g < G; ++g) b[u][g] = load_b(k, bcol[g]);
#pragma unroll
            for (int i = 0; i < MT; ++i) a[u][i] = load4(arow[i], k, K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        // B first: lane l then holds row l % 16 and columns
                        // 4 (l / 16) .. +3
                        acc[i][g] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[u][g][e], a[u][i][e], acc[i][g], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int g = 0; g < G; ++g) part[wave][i * G + g][lane] = acc[i][g];
    __syncthreads();

    if (threadIdx.x >= 64 * MT * NT) return;
    const int i = (threadIdx.x >> 6) % MT, h = (threadIdx.x >> 6) / MT;
    const int64_t m = m0 + 16 * i + (lane & 15);
    if (m >= M) return;
    const int c = n0 + 16 * h + 4 * (lane >> 4);
    if (c >= N) return;
    constexpr int Z = GATED ? 2 : 1;
    f32x4_t z[Z];
#pragma unroll
    for (int g = 0; g < Z; ++g) {
        const int f = i * G + (GATED ? g : h);
        z[g] = part[0][f][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) z[g] = z[g] + part[w][f][lane];
        if (ep.bias != nullptr) z[g] = z[g] + load4(ep.bias + (int64_t)g * N, c, N);
        if (ep.Z != nullptr) store4(ep.Z + m * ep.ldz + (int64_t)g * N, c, N, z[g]);
    }
    f32x4_t o;
    with_act(ep.act, [&]<int ACT>() {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = act_value<ACT>(z[0][e]);
    });
    if constexpr (GATED)
        o = o * z[Z - 1];
    else if (ep.R != nullptr)
        o = o + load4(ep.R + m * ep.ldr, c, N);
    store4(ep.C + m * ep.ldc, c, N, o);
}

template <bool TB, bool GATED>
void launch(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, const float* B, int64_t ldb,
            const BlockEpilogue& ep, hipStream_t s)
{
    auto go = [&]<int MT, int NT>() {
        const int gx = (int)((N + 16 * NT - 1) / (16 * NT));
        hipLaunchKernelGGL((rows_gemm_kernel<TB, GATED, MT, NT>), dim3(gx, (int)((M + 16 * MT - 1) / (16 * MT))),
                           dim3(64 * WAVES), 0, s, M, (int)N, (int)K, A, lda, B, ldb, ep);
    };
    if (M <= 16) {
        go.template operator()<1, 1>();
    } else if (M <= 32) {
        go.template operator()<2, 1>();
    } else {
        // two fragments of columns per workgroup where that leaves every CU one
        if constexpr (!GATED) {
            if (((M + 63) / 64) * ((N + 31) / 32) >= kWide) return go.template operator()<4, 2>();
        }
        go.template operator()<4, 1>();
    }
}

}  // namespace

hipError_t launch_rows_gemm(bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                            const float* B, int64_t ldb, const BlockEpilogue& ep, hipStream_t s)
{
    if (2 * N >= ((int64_t)1 << 31) || K >= ((int64_t)1 << 30) || (ep.gated && !trans_b)) return hipErrorInvalidValue;
    // (gridDim.y holds the row blocks: 65,535 of 64 at most per launch)
    const int64_t most = (int64_t)65535 * 64;
    for (int64_t m = 0; m < M; m += most) {
        const int64_t rows = M - m < most ? M - m : most;
        BlockEpilogue e = ep;
        e.C = ep.C + m * ep.ldc;
        if (ep.Z != nullptr) e.Z = ep.Z + m * ep.ldz;
        if (ep.R != nullptr) e.R = ep.R + m * ep.ldr;
        const float* a = A != nullptr ? A + m * lda : nullptr;   // (null with K = 0)
        if (ep.gated)
            launch<true, true>(rows, N, K, a, lda, B, ldb, e, s);
        else if (trans_b)
            launch<true, false>(rows, N, K, a, lda, B, ldb, e, s);
        else
            launch<false, false>(rows, N, K, a, lda, B, ldb, e, s);
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
    }
    return hipSuccess;
}

}  // namespace emu
