// C ABI of the transformer-block operators (declarations and full contract in
// include/emu_block.h): argument checks, the choice of route and the launches
// on the caller's stream.  Nothing is allocated here: workspaces come from
// the caller.
#include <hip/hip_runtime.h>

#include <cmath>

#include "emu_block.h"
#include "emu_block_launch.h"

namespace {

using emu::BlockEpilogue;

int64_t max1(int64_t v) { return v > 1 ? v : 1; }
bool valid_act(int a) { return a >= EMU_ACT_IDENTITY && a <= EMU_ACT_TANH; }
bool valid_op(int op) { return op == EMU_OP_N || op == EMU_OP_T; }
bool valid_mode(int m) { return m >= EMU_MODE_NATIVE_F32 && m <= EMU_MODE_BF16X1; }
// an array argument of `rows` rows that has to be there
bool bad_array(const void* p, int64_t rows, int64_t cols, int64_t ld)
{
    return ld < max1(cols) || (rows > 0 && cols > 0 && p == nullptr);
}
bool bad_optional(const void* p, int64_t cols, int64_t ld) { return p != nullptr && ld < max1(cols); }
bool bad_workspace(const void* ws, size_t have, size_t need)
{
    return need > 0 && (ws == nullptr || have < need || ((uintptr_t)ws & 255u) != 0);
}

emu_status_t from_hip(hipError_t e)
{
    if (e == hipSuccess) return EMU_STATUS_SUCCESS;
    if (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) return EMU_STATUS_ALLOC_FAILED;
    return EMU_STATUS_LAUNCH_FAILED;
}

hipStream_t stream_of(void* s) { return static_cast<hipStream_t>(s); }

// Columns of the element-wise passes are indexed with 32 bits.
constexpr int64_t kMaxCols = (int64_t)1 << 30;
// The emulated kernel addresses a tile's 128 rows of A with 32-bit byte
// offsets.
constexpr int64_t kMaxK = ((int64_t)1 << 23) - 4;

int bands_of(emu_mode_t mode)
{
    switch (mode) {
    case EMU_MODE_BF16X9: return 5;
    case EMU_MODE_BF16X6: return 3;
    case EMU_MODE_BF16X3: return 2;
    case EMU_MODE_BF16X1: return 1;
    default: return 0;
    }
}

// A product's kernels by predicted time (us), fitted to ten (K, N) and M = 1
// .. 8,192; a slower one is taken only where two are within a tenth.
//
// The one-launch FP32 kernel (launch_rows_gemm): a launch and, per workgroup
// of a CU, a latency and K; a workgroup has 64 rows (or 32, 16) and 16
// columns, or 32 where that still leaves every CU one and in a gated
// projection.
double rows_us(int64_t M, int64_t N, int64_t K, bool is_gated)
{
    const double m64 = (double)((M + 63) / 64), n32 = (double)((N + 31) / 32), n16 = (double)((N + 15) / 16);
    if (M > 32 && (is_gated || m64 * n32 >= 256.0)) {
        const double rounds = std::ceil(m64 * n32 / 256.0);
        // (beyond two the reads of A and the stores weigh more)
        return 2.3 + rounds * (0.9 + 0.0162 * (double)K) * (rounds > 2.0 ? 1.45 : 1.0);
    }
    const double groups = m64 * n16 / 256.0;
    const double per_k = M <= 16 ? 0.0034 : M <= 32 ? 0.0057 : 0.0094;
    return 2.4 + (groups < 1.0 ? 1.0 : groups) * (0.75 + per_k * (double)K);
}

// The one-launch emulated kernel (launch_few_gemm) with its better tile, 32 x
// 32 or (wide) 64 x 64: rounds of a workgroup per CU, each a latency and its
// chunks of 128 or 64 k.
double few_us(int64_t M, int64_t N, int64_t K, int bands, bool& wide)
{
    const int i = bands >= 5 ? 0 : bands >= 3 ? 1 : 2;
    constexpr double narrow_c[3] = {1.0, 0.95, 0.72}, wide_c[3] = {1.3, 1.17, 0.93};
    const double chunks = wide_c[i] * (double)((K + 63) / 64);
    const int64_t tiles32 = (M + 31) / 32 * ((N + 31) / 32), tiles64 = (M + 63) / 64 * ((N + 63) / 64);
    // (more wide tiles than CUs, or any with two planes, share a CU in pairs)
    const double narrow = 0.5 + std::ceil((double)tiles32 / 256.0) * (i == 2 && tiles32 > 256 ? 0.8 : 1.0) *
                                    (2.4 + narrow_c[i] * (double)((K + 127) / 128));
    const double broad =
        0.5 + std::ceil((double)tiles64 / 256.0) * (tiles64 <= 256 ? 3.0 + chunks
                                                    : i == 2       ? 0.8 * (3.0 + chunks)
                                                                   : 2.0 + 0.92 * chunks);
    wide = broad < narrow;
    return wide ? broad : narrow;
}

// The emulated kernel of 128-wide tiles without a K split: its launch (and
// the weights' split's, with 10 bytes per element; where A is copied to
// aligned rows, that launch's), then rounds of tiles of 128 or 64 rows, each
// its k-steps and an epilogue.
double tiles_us(int64_t M, int64_t N, int64_t K, int bands, bool have_planes, bool copies_a)
{
    const int i = bands >= 5 ? 0 : bands >= 3 ? 1 : 2;
    constexpr double tall_c[3] = {1.72, 1.44, 1.1}, low_c[3] = {1.0, 0.92, 0.78};
    const double n = (double)((N + 127) / 128), steps = (double)((K + 31) / 32);
    const double tall = std::ceil((double)((M + 127) / 128) * n / 256.0) * (tall_c[i] * steps + 4.0);
    const double low = std::ceil((double)((M + 63) / 64) * n / 256.0) * (low_c[i] * steps + 2.5);
    return (have_planes ? 4.5 : 8.0 + 10.0 * (double)N * (double)K / 4.0e6) +
           (copies_a ? 4.0 + 8.0 * (double)M * (double)K / 4.0e6 : 0.0) + (low < tall ? low : tall);
}

// The emulated one-launch kernel is taken where it is predicted this much
// faster: the predictions' error.
constexpr double kFewError = 1.1;

// Columns of a product past which the one-launch kernels are not taken: a
// launch holds less than 2^32 threads along the columns, which the FP32 kernel
// spends 32 on each.
constexpr int64_t kOneLaunchCols = (int64_t)1 << 26;

// Below these the kernels' formulas are not asked: the emulated one-launch
// kernel reads four k (and columns of a K x N operand) at a time.
bool few_runs(int64_t M, int64_t N, int64_t K)
{
    return K >= 4 && N >= 4 && M <= ((int64_t)1 << 20) && N <= kOneLaunchCols;
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// How one product with its epilogue runs.
struct Route {
    bool rows;                 // the one-launch FP32 kernel
    bool few, wide;            // the one-launch emulated kernel, and its tile, in
    emu_mode_t mode;           // else: the product's mode,
    emu::GemmPlan plan;        // its plan,
    size_t gemm_bytes;         // and the workspace: the product's own, then
    size_t more_bytes;         // NATIVE_F32: t; else A with 16-byte aligned rows, where it has none
    int64_t ld;                // (leading dimension of either)
};

// g with A as the emulated kernel takes it: 16-byte aligned rows of whole
// 16-byte groups, copied to the workspace where the caller's are not.
bool needs_copy(const emu::GemmArgs& g) { return !emu::fused_a_path(g); }

emu::GemmArgs with_copy(emu::GemmArgs g, const float* copy, int64_t ld)
{
    g.A = copy;
    g.lda = ld;
    g.a_whole_groups = true;
    return g;
}

// (stands for the copy in a workspace query: 16-byte aligned)
const float* const kSomeRows = reinterpret_cast<const float*>((uintptr_t)256);

// N: columns of the product (gated: 2 F).
Route route_of(const emu::GemmArgs& g, bool is_gated, emu_mode_t mode, bool have_planes, int num_cu)
{
    Route r{};
    const bool automatic = mode == EMU_MODE_AUTO;
    r.rows = g.K == 0;
    if (r.rows || g.M == 0 || g.N == 0) return r;
    if (automatic) {
        // what emu_sgemm's AUTO would run (with its K split plan; the
        // library's model leaves out the traffic of the weights' split)
        // against the one-launch kernels.  Measured (us, FP32 / nine
        // products in one launch / AUTO's plan): 1 x 512 x 256 3.6 / 6.8 /
        // 12.1, 2,048 x 512 x 256 12.1 / 9.4 / 17.7, 512 x 1024 x 1024 19.8 /
        // 22.1 / 30.8, 64 x 1024 x 4096 41.1 / 12.1 / 46.3.
        const bool copies = (g.K & 3) != 0;   // (by the shape alone: AUTO's bits do not depend on addresses)
        double plan = emu::api_predict_us(g.M, g.N, g.K) + (have_planes ? -3.5 : 10.0 * (double)g.N * (double)g.K / 4.0e6);
        if (emu::api_select_mode(g.M, g.N, g.K) == EMU_MODE_NATIVE_F32)
            plan += 4.0 + 8.0 * (double)g.M * (double)g.N / 4.5e6;   // the epilogue, a pass of its own
        else if (emu::api_plan(g.M, g.N, g.K, true, num_cu).split == 1)
            plan = std::fmax(plan, tiles_us(g.M, g.N, g.K, 5, have_planes, copies));
        if (copies) plan = std::fmax(plan, emu::api_predict_us(g.M, g.N, g.K) + 4.0 + 8.0 * (double)g.M * (double)g.K / 4.0e6);
        const double rows = have_planes || g.M > ((int64_t)1 << 20) || g.N > kOneLaunchCols ? plan : rows_us(g.M, g.N, g.K, is_gated);
        const double few = few_runs(g.M, g.N, g.K) ? few_us(g.M, g.N, g.K, 5, r.wide) : plan;
        r.rows = rows < plan && rows <= few;
        r.few = !r.rows && kFewError * few < plan;
        r.mode = have_planes || r.few ? EMU_MODE_BF16X9 : (emu_mode_t)emu::api_select_mode(g.M, g.N, g.K);
    } else {
        // the same bits either way.  Measured with nine products (us, one
        // launch / 128-wide tiles): 1 x 1024 x 1024 10.4 / 41.8, 1,024 x 1024
        // x 1024 24.4 / 41.6, 3,000 x 1024 x 1024 67.4 / 63.0, 4,096 x 256 x
        // 512 14.5 / 24.1, 8,192 x 256 x 512 26.1 / 28.0, 100,000 x 64 x 64
        // 22.5 / 47.4.
        r.mode = mode;
        const int bands = bands_of(mode);
        r.few = bands != 0 && few_runs(g.M, g.N, g.K) &&
                kFewError * few_us(g.M, g.N, g.K, bands, r.wide) < tiles_us(g.M, g.N, g.K, bands, have_planes, needs_copy(g));
    }
    if (r.rows || r.few) return r;
    if (r.mode == EMU_MODE_NATIVE_F32) {
        r.gemm_bytes = round256(emu::gemm_native_f32_workspace_bytes(g));
        r.ld = (g.N + 3) & ~(int64_t)3;
        r.more_bytes = (size_t)g.M * (size_t)r.ld * sizeof(float);
    } else {
        emu::GemmArgs f = g;
        if (needs_copy(g)) {
            r.ld = (g.K + 3) & ~(int64_t)3;
            r.more_bytes = (size_t)g.M * (size_t)r.ld * sizeof(float);
            f = with_copy(g, kSomeRows, r.ld);
        }
        r.plan = emu::api_plan(g.M, g.N, g.K, automatic, num_cu);
        r.gemm_bytes = round256(
            emu::gemm_bf16_workspace_bytes(f, bands_of(r.mode), r.plan.split, r.plan.tile_m, r.plan.split_from));
    }
    return r;
}

// The workspace query's device: sizes do not depend on it but through the
// compute units of the plan; without a gfx950 the full chip's count.
int query_cus()
{
    emu::DeviceInfo d;
    return emu::api_current_device(d) ? d.num_cu : 256;
}

emu::GemmArgs gemm_args(bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                        const float* B, int64_t ldb, const void* planes)
{
    emu::GemmArgs g{};
    g.trans_a = false;
    g.trans_b = trans_b;
    g.M = M;
    g.N = N;
    g.K = K;
    g.alpha = 1.0f;
    g.beta = 0.0f;
    g.A = A;
    g.lda = lda;
    g.B = B;
    g.ldb = ldb;
    g.bias = nullptr;
    g.Bplanes = static_cast<const uint16_t*>(planes);
    return g;
}

// The product A . op(B) (columns g.N) and its epilogue (columns n_out).
emu_status_t product(emu::GemmArgs g, int64_t n_out, const BlockEpilogue& ep, emu_mode_t mode, void* ws,
                     size_t ws_bytes, hipStream_t s)
{
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    const Route r = route_of(g, ep.gated != 0, mode, g.Bplanes != nullptr, dev.num_cu);
    if (r.rows && g.N > kOneLaunchCols)   // (K = 0)
        return from_hip(emu::launch_epilogue(g.M, n_out, nullptr, 0, ep, s));
    if (r.rows)
        return from_hip(emu::launch_rows_gemm(g.trans_b, g.M, n_out, g.K, g.A, g.lda, g.B, g.ldb, ep, s));
    if (r.few)
        return from_hip(emu::launch_few_gemm(bands_of(r.mode), r.wide, g.trans_b, g.M, n_out, g.K, g.A, g.lda, g.B, g.ldb,
                                             g.Bplanes, ep, s));
    if (bad_workspace(ws, ws_bytes, r.gemm_bytes + r.more_bytes)) return EMU_STATUS_INVALID_VALUE;
    float* more = reinterpret_cast<float*>(static_cast<char*>(ws) + r.gemm_bytes);
    void* gws = r.gemm_bytes > 0 ? ws : nullptr;
    hipError_t e = hipSuccess;
    if (r.mode == EMU_MODE_NATIVE_F32) {
        g.C = more;
        g.ldc = r.ld;
        e = emu::launch_gemm_native_f32(g, dev, gws, s);
        if (e == hipSuccess) e = emu::launch_epilogue(g.M, n_out, more, r.ld, ep, s);
        return from_hip(e);
    }
    if (needs_copy(g)) {
        e = emu::launch_copy_rows(g.M, g.K, g.A, g.lda, more, r.ld, s);
        g = with_copy(g, more, r.ld);
    }
    if (e == hipSuccess)
        e = emu::launch_gemm_bf16(g, bands_of(r.mode), r.plan.split, r.plan.split_from, r.plan.tile_m, dev, gws, s, &ep);
    return from_hip(e);
}

emu_status_t product_workspace(const emu::GemmArgs& g, bool is_gated, emu_mode_t mode, bool have_planes,
                               size_t* bytes)
{
    *bytes = 0;
    if (g.M == 0 || g.N == 0) return EMU_STATUS_SUCCESS;
    const Route r = route_of(g, is_gated, mode, have_planes, query_cus());
    *bytes = r.gemm_bytes + r.more_bytes;   // (none for one launch)
    return EMU_STATUS_SUCCESS;
}

// A planes pointer that a workspace query stands in for.
const void* const kSomePlanes = reinterpret_cast<const void*>((uintptr_t)256);

bool bad_planes(const void* planes, emu_mode_t mode)
{
    return planes != nullptr && (((uintptr_t)planes & 15u) != 0 || mode == EMU_MODE_NATIVE_F32);
}

}  // namespace

extern "C" {

int emu_block_version(void) { return 100; }

// ---- layer norm -----------------------------------------------------------------

emu_status_t emu_layer_norm(int64_t rows, int64_t cols, const float* x, int64_t ldx, const float* weight,
                            const float* bias, float eps, float* y, int64_t ldy, float* mean, float* rstd,
                            void* stream)
{
    if (rows < 0 || cols < 1 || !(eps >= 0.0f) || bad_array(x, rows, cols, ldx) || bad_array(y, rows, cols, ldy))
        return EMU_STATUS_INVALID_VALUE;
    if (cols > EMU_LAYER_NORM_MAX_COLS) return EMU_STATUS_NOT_SUPPORTED;
    if (rows == 0) return EMU_STATUS_SUCCESS;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    return from_hip(emu::launch_norm(rows, cols, x, ldx, weight, bias, eps, y, ldy, mean, rstd, stream_of(stream)));
}

emu_status_t emu_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes)
{
    if (rows < 0 || cols < 1 || bytes == nullptr) return EMU_STATUS_INVALID_VALUE;
    if (cols > EMU_LAYER_NORM_MAX_COLS) return EMU_STATUS_NOT_SUPPORTED;
    *bytes = emu::norm_backward_workspace(rows, cols);
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_layer_norm_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy, const float* x,
                                     int64_t ldx, const float* weight, const float* mean, const float* rstd,
                                     float* dx, int64_t lddx, float* dweight, float* dbias, void* workspace,
                                     size_t workspace_bytes, void* stream)
{
    if (rows < 0 || cols < 1 || bad_array(dy, rows, cols, lddy) || bad_array(x, rows, cols, ldx) ||
        bad_optional(dx, cols, lddx) || (rows > 0 && (mean == nullptr || rstd == nullptr)))
        return EMU_STATUS_INVALID_VALUE;
    if (cols > EMU_LAYER_NORM_MAX_COLS) return EMU_STATUS_NOT_SUPPORTED;
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (sums && bad_workspace(workspace, workspace_bytes, emu::norm_backward_workspace(rows, cols)))
        return EMU_STATUS_INVALID_VALUE;
    if (!sums && (rows == 0 || dx == nullptr)) return EMU_STATUS_SUCCESS;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    hipStream_t s = stream_of(stream);
    if (rows == 0) {
        hipError_t e = emu::launch_zero(dweight, cols, s);
        if (e == hipSuccess) e = emu::launch_zero(dbias, cols, s);
        return from_hip(e);
    }
    return from_hip(emu::launch_norm_backward(rows, cols, dy, lddy, x, ldx, weight, mean, rstd, dx, lddx, dweight,
                                              dbias, static_cast<float*>(workspace), s));
}

emu_status_t emu_layer_norm_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv, const float* p,
                                      const float* q, const float* dy, int64_t lddy, const float* x,
                                      int64_t ldx, const float* weight, const float* mean, const float* rstd,
                                      float* gdy, int64_t ldgdy, float* gx, int64_t ldgx, float* gw,
                                      void* workspace, size_t workspace_bytes, void* stream)
{
    if (rows < 0 || cols < 1 || bad_optional(v, cols, ldv) || bad_array(dy, rows, cols, lddy) ||
        bad_array(x, rows, cols, ldx) || bad_optional(gdy, cols, ldgdy) || bad_optional(gx, cols, ldgx) ||
        (rows > 0 && (mean == nullptr || rstd == nullptr)))
        return EMU_STATUS_INVALID_VALUE;
    if (cols > EMU_LAYER_NORM_MAX_COLS) return EMU_STATUS_NOT_SUPPORTED;
    if (gw != nullptr && bad_workspace(workspace, workspace_bytes, emu::norm_backward_workspace(rows, cols)))
        return EMU_STATUS_INVALID_VALUE;
    if (gw == nullptr && (rows == 0 || (gdy == nullptr && gx == nullptr))) return EMU_STATUS_SUCCESS;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    hipStream_t s = stream_of(stream);
    if (rows == 0) return from_hip(emu::launch_zero(gw, cols, s));
    return from_hip(emu::launch_norm_backward2(rows, cols, v, ldv, p, q, dy, lddy, x, ldx, weight, mean, rstd, gdy,
                                               ldgdy, gx, ldgx, gw, static_cast<float*>(workspace), s));
}

// ---- activations ------------------------------------------------------------------

emu_status_t emu_act_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy, const float* z,
                              int64_t ldz, emu_act_t act, float* dz, int64_t lddz, void* stream)
{
    if (rows < 0 || cols < 0 || !valid_act(act) || bad_array(dy, rows, cols, lddy) ||
        bad_array(z, rows, cols, ldz) || bad_array(dz, rows, cols, lddz))
        return EMU_STATUS_INVALID_VALUE;
    if (cols > kMaxCols) return EMU_STATUS_NOT_SUPPORTED;
    if (rows == 0 || cols == 0) return EMU_STATUS_SUCCESS;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    return from_hip(emu::launch_act_backward(rows, cols, dy, lddy, z, ldz, act, dz, lddz, stream_of(stream)));
}

emu_status_t emu_act_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv, const float* dy,
                               int64_t lddy, const float* z, int64_t ldz, emu_act_t act, float* gdy,
                               int64_t ldgdy, float* gz, int64_t ldgz, void* stream)
{
    if (rows < 0 || cols < 0 || !valid_act(act) || bad_array(v, rows, cols, ldv) ||
        bad_array(dy, rows, cols, lddy) || bad_array(z, rows, cols, ldz) || bad_optional(gdy, cols, ldgdy) ||
        bad_optional(gz, cols, ldgz))
        return EMU_STATUS_INVALID_VALUE;
    if (cols > kMaxCols) return EMU_STATUS_NOT_SUPPORTED;
    if (rows == 0 || cols == 0 || (gdy == nullptr && gz == nullptr)) return EMU_STATUS_SUCCESS;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    return from_hip(emu::launch_act_backward2(rows, cols, v, ldv, dy, lddy, z, ldz, act, gdy, ldgdy, gz, ldgz,
                                              stream_of(stream)));
}

// ---- linear layer with activation and residual --------------------------------------

emu_status_t emu_sgemm_act_route(emu_op_t transB, int64_t M, int64_t N, int64_t K, int* few)
{
    if (!valid_op(transB) || M < 0 || N < 0 || K < 0 || few == nullptr) return EMU_STATUS_INVALID_VALUE;
    const Route r = route_of(gemm_args(transB == EMU_OP_T, M, N, K, nullptr, max1(K), nullptr, 0, nullptr), false,
                             EMU_MODE_AUTO, false, query_cus());
    *few = M > 0 && N > 0 && K > 0 && r.rows ? 1 : r.few ? 2 : 0;
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_sgemm_act_workspace(emu_op_t transB, int64_t M, int64_t N, int64_t K, const float* A,
                                     int64_t lda, int has_planes, emu_mode_t mode, size_t* bytes)
{
    if (!valid_op(transB) || !valid_mode(mode) || M < 0 || N < 0 || K < 0 || lda < max1(K) || bytes == nullptr ||
        (has_planes && mode == EMU_MODE_NATIVE_F32))
        return EMU_STATUS_INVALID_VALUE;
    return product_workspace(gemm_args(transB == EMU_OP_T, M, N, K, A, lda, nullptr, 0,
                                       has_planes ? kSomePlanes : nullptr),
                             false, mode, has_planes != 0, bytes);
}

emu_status_t emu_sgemm_act(emu_op_t transB, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                           const float* B, int64_t ldb, const void* planes, const float* bias, emu_act_t act,
                           float* Z, int64_t ldz, const float* R, int64_t ldr, float* C, int64_t ldc,
                           emu_mode_t mode, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_op(transB) || !valid_mode(mode) || !valid_act(act) || M < 0 || N < 0 || K < 0)
        return EMU_STATUS_INVALID_VALUE;
    const bool has_c = M > 0 && N > 0;
    if (lda < max1(K) || (planes == nullptr && ldb < (transB == EMU_OP_N ? max1(N) : max1(K))) ||
        bad_array(C, M, N, ldc) || bad_optional(Z, N, ldz) || bad_optional(R, N, ldr) || bad_planes(planes, mode) ||
        (has_c && K > 0 && (A == nullptr || (B == nullptr && planes == nullptr))))
        return EMU_STATUS_INVALID_VALUE;
    if (N > kMaxCols || K > kMaxK) return EMU_STATUS_NOT_SUPPORTED;
    if (!has_c) return EMU_STATUS_SUCCESS;
    const BlockEpilogue ep{(int)act, 0, bias, Z, ldz, R, ldr, C, ldc};
    return product(gemm_args(transB == EMU_OP_T, M, N, K, A, lda, B, ldb, planes), N, ep, mode, workspace,
                   workspace_bytes, stream_of(stream));
}

// ---- gated feed-forward projection -----------------------------------------------------

emu_status_t emu_sgemm_gated_workspace(int64_t M, int64_t F, int64_t K, const float* A, int64_t lda,
                                       int has_planes, emu_mode_t mode, size_t* bytes)
{
    if (!valid_mode(mode) || M < 0 || F < 0 || K < 0 || lda < max1(K) || bytes == nullptr ||
        (has_planes && mode == EMU_MODE_NATIVE_F32) || F > kMaxCols)
        return EMU_STATUS_INVALID_VALUE;
    return product_workspace(gemm_args(true, M, 2 * F, K, A, lda, nullptr, 0, has_planes ? kSomePlanes : nullptr),
                             true, mode, has_planes != 0, bytes);
}

emu_status_t emu_sgemm_gated(int64_t M, int64_t F, int64_t K, const float* A, int64_t lda, const float* W,
                             int64_t ldw, const void* planes, const float* bias, emu_act_t act, float* Z,
                             int64_t ldz, float* C, int64_t ldc, emu_mode_t mode, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    if (!valid_mode(mode) || !valid_act(act) || M < 0 || F < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (F > kMaxCols || K > kMaxK) return EMU_STATUS_NOT_SUPPORTED;
    const bool has_c = M > 0 && F > 0;
    if (lda < max1(K) || (planes == nullptr && ldw < max1(K)) || bad_array(C, M, F, ldc) ||
        bad_optional(Z, 2 * F, ldz) || bad_planes(planes, mode) ||
        (has_c && K > 0 && (A == nullptr || (W == nullptr && planes == nullptr))))
        return EMU_STATUS_INVALID_VALUE;
    if (!has_c) return EMU_STATUS_SUCCESS;
    const BlockEpilogue ep{(int)act, 1, bias, Z, ldz, nullptr, 0, C, ldc};
    return product(gemm_args(true, M, 2 * F, K, A, lda, W, ldw, planes), F, ep, mode, workspace, workspace_bytes,
                   stream_of(stream));
}

emu_status_t emu_presplit_gated_bytes(int64_t F, int64_t K, emu_mode_t mode, size_t* bytes)
{
    if (F < 0 || F > kMaxCols) return EMU_STATUS_INVALID_VALUE;
    return emu_presplit_b_bytes(2 * F, K, mode, bytes);
}

emu_status_t emu_presplit_gated(int64_t F, int64_t K, const float* W, int64_t ldw, emu_mode_t mode, void* planes,
                                void* stream)
{
    if (F < 0 || F > kMaxCols || K < 0 || bands_of(mode) == 0 || ldw < max1(K)) return EMU_STATUS_INVALID_VALUE;
    if (F == 0 || K == 0) return EMU_STATUS_SUCCESS;
    if (W == nullptr || planes == nullptr || ((uintptr_t)planes & 15u) != 0) return EMU_STATUS_INVALID_VALUE;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    return from_hip(emu::launch_presplit_gated(W, ldw, F, K, bands_of(mode), static_cast<uint16_t*>(planes),
                                               stream_of(stream)));
}

emu_status_t emu_gated_backward(int64_t M, int64_t F, const float* dh, int64_t lddh, const float* Z, int64_t ldz,
                                emu_act_t act, float* dZ, int64_t lddz, void* stream)
{
    if (M < 0 || F < 0 || F > kMaxCols || !valid_act(act) || bad_array(dh, M, F, lddh) ||
        bad_array(Z, M, 2 * F, ldz) || bad_array(dZ, M, 2 * F, lddz))
        return EMU_STATUS_INVALID_VALUE;
    if (M == 0 || F == 0) return EMU_STATUS_SUCCESS;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    return from_hip(emu::launch_gated_backward(M, F, dh, lddh, Z, ldz, act, dZ, lddz, stream_of(stream)));
}

emu_status_t emu_gated_backward2(int64_t M, int64_t F, const float* V, int64_t ldv, const float* dh, int64_t lddh,
                                 const float* Z, int64_t ldz, emu_act_t act, float* gdh, int64_t ldgdh, float* gZ,
                                 int64_t ldgz, void* stream)
{
    if (M < 0 || F < 0 || F > kMaxCols || !valid_act(act) || bad_array(V, M, 2 * F, ldv) ||
        bad_array(dh, M, F, lddh) || bad_array(Z, M, 2 * F, ldz) || bad_optional(gdh, F, ldgdh) ||
        bad_optional(gZ, 2 * F, ldgz))
        return EMU_STATUS_INVALID_VALUE;
    if (M == 0 || F == 0 || (gdh == nullptr && gZ == nullptr)) return EMU_STATUS_SUCCESS;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    return from_hip(emu::launch_gated_backward2(M, F, V, ldv, dh, lddh, Z, ldz, act, gdh, ldgdh, gZ, ldgz,
                                                stream_of(stream)));
}

// ---- weight gradient ----------------------------------------------------------------------

emu_status_t emu_wgrad_workspace(int64_t rows, int64_t M, int64_t N, size_t* bytes)
{
    if (rows < 0 || M < 0 || N < 0 || bytes == nullptr) return EMU_STATUS_INVALID_VALUE;
    *bytes = rows == 0 || M == 0 ? 0 : emu::wgrad_workspace(rows, M, N, false);
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_wgrad_gated_workspace(int64_t rows, int64_t F, int64_t N, size_t* bytes)
{
    if (rows < 0 || F < 0 || N < 0 || bytes == nullptr) return EMU_STATUS_INVALID_VALUE;
    *bytes = rows == 0 || F == 0 ? 0 : emu::wgrad_workspace(rows, F, N, true);
    return EMU_STATUS_SUCCESS;
}

}  // extern "C"

namespace {

emu_status_t wgrad(int64_t rows, int64_t M, int64_t N, const emu::WgradSource& src, const float* X, int64_t ldx,
                   float* dW, int64_t lddw, float* db, void* workspace, size_t workspace_bytes, void* stream)
{
    const int64_t out = src.gated ? 2 * M : M;
    if (rows < 0 || M < 0 || N < 0 || bad_array(X, rows, N, ldx) || bad_array(dW, out, N, lddw))
        return EMU_STATUS_INVALID_VALUE;
    for (int64_t ld : {src.ldz, src.ldy, src.ldd, ldx})
        if (ld > emu::kWgradMaxLd) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || (N == 0 && db == nullptr && src.dZ == nullptr)) return EMU_STATUS_SUCCESS;
    if (rows > 0 && bad_workspace(workspace, workspace_bytes, emu::wgrad_workspace(rows, M, N, src.gated)))
        return EMU_STATUS_INVALID_VALUE;
    emu::DeviceInfo dev;
    if (!emu::api_current_device(dev)) return EMU_STATUS_NOT_SUPPORTED;
    hipStream_t s = stream_of(stream);
    if (rows == 0) {
        hipError_t e = hipSuccess;
        if (lddw == N || out == 1) {
            e = emu::launch_zero(dW, out * N, s);
        } else {
            for (int64_t m = 0; m < out && e == hipSuccess; ++m) e = emu::launch_zero(dW + m * lddw, N, s);
        }
        if (e == hipSuccess) e = emu::launch_zero(db, out, s);
        return from_hip(e);
    }
    return from_hip(emu::launch_wgrad(rows, M, N, src, X, ldx, dW, lddw, db, workspace, s));
}

}  // namespace

extern "C" {

emu_status_t emu_wgrad(int64_t rows, int64_t M, int64_t N, const float* dZ, int64_t lddz, const float* X,
                       int64_t ldx, float* dW, int64_t lddw, float* db, void* workspace, size_t workspace_bytes,
                       void* stream)
{
    if (bad_array(dZ, rows, M, lddz)) return EMU_STATUS_INVALID_VALUE;
    emu::WgradSource src{dZ, lddz};
    return wgrad(rows, M, N, src, X, ldx, dW, lddw, db, workspace, workspace_bytes, stream);
}

emu_status_t emu_wgrad_act(int64_t rows, int64_t M, int64_t N, const float* dY, int64_t lddy, const float* Z,
                           int64_t ldz, emu_act_t act, float* dZ, int64_t lddz, const float* X, int64_t ldx,
                           float* dW, int64_t lddw, float* db, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_act(act) || bad_array(dY, rows, M, lddy) || bad_array(Z, rows, M, ldz) || bad_array(dZ, rows, M, lddz))
        return EMU_STATUS_INVALID_VALUE;
    emu::WgradSource src{Z, ldz, dY, lddy, dZ, lddz, (int)act, false};
    return wgrad(rows, M, N, src, X, ldx, dW, lddw, db, workspace, workspace_bytes, stream);
}

emu_status_t emu_wgrad_gated(int64_t rows, int64_t F, int64_t N, const float* dH, int64_t lddh, const float* Z,
                             int64_t ldz, emu_act_t act, float* dZ, int64_t lddz, const float* X, int64_t ldx,
                             float* dW, int64_t lddw, float* db, void* workspace, size_t workspace_bytes,
                             void* stream)
{
    if (!valid_act(act) || F > kMaxCols || bad_array(dH, rows, F, lddh) || bad_array(Z, rows, 2 * F, ldz) ||
        bad_array(dZ, rows, 2 * F, lddz))
        return EMU_STATUS_INVALID_VALUE;
    emu::WgradSource src{Z, ldz, dH, lddh, dZ, lddz, (int)act, true};
    return wgrad(rows, F, N, src, X, ldx, dW, lddw, db, workspace, workspace_bytes, stream);
}

}  // extern "C"
