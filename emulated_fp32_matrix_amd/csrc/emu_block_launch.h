// Internal interface between the C-ABI layer of the transformer-block
// operators (emu_block_api.hip) and their kernels.  Not installed; callers
// use include/emu_block.h.
#pragma once

#include "emu_launch.h"

namespace emu {

// From emu_api.hip: the current device (false unless gfx950), the mode
// EMU_MODE_AUTO runs for a shape and its predicted time, and a launch plan of the emulated kernel:
// AUTO's (K split included) or, without `split`, one that only picks the
// tile height.
bool api_current_device(DeviceInfo& info);
int api_select_mode(int64_t M, int64_t N, int64_t K);
double api_predict_us(int64_t M, int64_t N, int64_t K);
struct GemmPlan {
    int split, tile_m;
    int64_t split_from;
};
GemmPlan api_plan(int64_t M, int64_t N, int64_t K, bool split, int num_cu);

// What follows a matrix product t (include/emu_block.h, emu_sgemm_act and
// emu_sgemm_gated): z = t + bias, then C = act(z) + R, or (gated, t = [g | u],
// bias likewise) C = act(g) * u.
struct BlockEpilogue {
    int act;
    int gated;             // t has 2 N columns
    const float* bias;     // or null
    float* Z;              // receives z, or null
    int64_t ldz;
    const float* R;        // or null
    int64_t ldr;
    float* C;
    int64_t ldc;
};

size_t norm_backward_workspace(int64_t rows, int64_t cols);
hipError_t launch_norm(int64_t rows, int64_t cols, const float* x, int64_t ldx, const float* weight,
                       const float* bias, float eps, float* y, int64_t ldy, float* mean, float* rstd,
                       hipStream_t s);
hipError_t launch_norm_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy, const float* x,
                                int64_t ldx, const float* weight, const float* mean, const float* rstd,
                                float* dx, int64_t lddx, float* dweight, float* dbias, float* ws,
                                hipStream_t s);
hipError_t launch_norm_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv, const float* p,
                                 const float* q, const float* dy, int64_t lddy, const float* x, int64_t ldx,
                                 const float* weight, const float* mean, const float* rstd, float* gdy,
                                 int64_t ldgdy, float* gx, int64_t ldgx, float* gw, float* ws, hipStream_t s);
// n floats of zero.
hipError_t launch_zero(float* p, int64_t n, hipStream_t s);
// out0[c] (c < cols) and out1[c - cols] (cols <= c < total) = the sum over
// i < parts of part[i * stride + c]; out0, out1 may be null.
hipError_t launch_column_join(const float* part, int64_t parts, int64_t stride, int64_t total, int64_t cols,
                              float* out0, float* out1, hipStream_t s);

// C from the product t (M x N, gated: M x 2N; ldt), or from zeros (t null).
hipError_t launch_epilogue(int64_t M, int64_t N, const float* t, int64_t ldt, const BlockEpilogue& ep,
                           hipStream_t s);
// The epilogue of a K-split launch's split tiles (emu_launch.h): t is the sum of
// the segments' partial tiles, in order.  N: columns of C.
hipError_t launch_split_epilogue(const float* parts, int segs, int nsplit, int split_from, int tiles_n, int tile_m,
                                 int64_t M, int64_t N, const BlockEpilogue& ep, hipStream_t s);
// A (M x K, lda) to dst (rows of ldd floats).
hipError_t launch_copy_rows(int64_t M, int64_t K, const float* A, int64_t lda, float* dst, int64_t ldd,
                            hipStream_t s);
hipError_t launch_act_backward(int64_t rows, int64_t cols, const float* dy, int64_t lddy, const float* z,
                               int64_t ldz, int act, float* dz, int64_t lddz, hipStream_t s);
hipError_t launch_act_backward2(int64_t rows, int64_t cols, const float* v, int64_t ldv, const float* dy,
                                int64_t lddy, const float* z, int64_t ldz, int act, float* gdy, int64_t ldgdy,
                                float* gz, int64_t ldgz, hipStream_t s);
hipError_t launch_gated_backward(int64_t M, int64_t F, const float* dh, int64_t lddh, const float* Z,
                                 int64_t ldz, int act, float* dZ, int64_t lddz, hipStream_t s);
hipError_t launch_gated_backward2(int64_t M, int64_t F, const float* V, int64_t ldv, const float* dh,
                                  int64_t lddh, const float* Z, int64_t ldz, int act, float* gdh,
                                  int64_t ldgdh, float* gZ, int64_t ldgz, hipStream_t s);

// The product and its epilogue in one launch, for few rows: A M x K, B N x K
// (trans_b) or K x N; gated: B 2N x K, trans_b.
hipError_t launch_rows_gemm(bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                            const float* B, int64_t ldb, const BlockEpilogue& ep, hipStream_t s);

// The emulated product (nbands of the mode) and its epilogue in one launch, for
// few rows, from B as above or from its planes, in tiles of 64 x 64 (wide) or
// 32 x 32.  K at least 4, and N, of a K x N operand.
hipError_t launch_few_gemm(int nbands, bool wide, bool trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                           const float* B, int64_t ldb, const uint16_t* planes, const BlockEpilogue& ep, hipStream_t s);

// Leading dimensions of the weight-gradient product: its 32-row slabs are
// addressed with 32-bit byte offsets.
constexpr int64_t kWgradMaxLd = ((int64_t)1 << 31) / (4 * 32) - 128;
// dZ of the weight-gradient product: an array (Z, with dY null), or made from
// dY and the pre-activations Z and written to dZ (gated: Z and dZ hold 2 M
// columns, dY M).
struct WgradSource {
    const float* Z;
    int64_t ldz;
    const float* dY = nullptr;
    int64_t ldy = 0;
    float* dZ = nullptr;
    int64_t ldd = 0;
    int act = 0;
    bool gated = false;
};
size_t wgrad_workspace(int64_t rows, int64_t M, int64_t N, bool gated);
hipError_t launch_wgrad(int64_t rows, int64_t M, int64_t N, const WgradSource& src, const float* X, int64_t ldx,
                        float* dW, int64_t lddw, float* db, void* ws, hipStream_t s);

}  // namespace emu
