// Launch of the two-group emulated GEMM with the transformer-block operators'
// epilogue; one translation unit per band count instantiates it
// (emu_gemm_epi_*.hip), so that they compile side by side.
#pragma once

#include "emu_gemm_pp.h"

namespace emu {

// p: as for the plain kernel, with N the columns of C (gated: half the
// product's) and vec_b set when every array of `ep` keeps a tile's rows
// within 32-bit byte offsets.
template <int NB>
void launch_gemm_epi(const Params& p, const BlockEpilogue& ep, int tile_m, int grid, const uint16_t* Wb,
                     hipStream_t s);

#ifdef EMU_GEMM_EPI_INSTANTIATE
namespace {

template <int NB, int TH, int EPI>
void launch_one(const Params& p, const BlockEpilogue& ep, int grid, const uint16_t* Wb, hipStream_t s)
{
    if (p.ksplit > 1)
        hipLaunchKernelGGL((gemm_bf16_pp_kernel<NB, true, false, TH, EPI, BlockEpilogue>), dim3(grid), dim3(512), 0, s,
                           p, Wb, ep);
    else
        hipLaunchKernelGGL((gemm_bf16_pp_kernel<NB, false, false, TH, EPI, BlockEpilogue>), dim3(grid), dim3(512), 0, s,
                           p, Wb, ep);
}

}  // namespace

template <int NB>
void launch_gemm_epi(const Params& p, const BlockEpilogue& ep, int tile_m, int grid, const uint16_t* Wb,
                     hipStream_t s)
{
    if (ep.gated && tile_m == 64)
        launch_one<NB, 64, EPI_GATED>(p, ep, grid, Wb, s);
    else if (ep.gated)
        launch_one<NB, 128, EPI_GATED>(p, ep, grid, Wb, s);
    else if (tile_m == 64)
        launch_one<NB, 64, EPI_ACT>(p, ep, grid, Wb, s);
    else
        launch_one<NB, 128, EPI_ACT>(p, ep, grid, Wb, s);
}

template void launch_gemm_epi<EMU_GEMM_EPI_INSTANTIATE>(const Params&, const BlockEpilogue&, int, int,
                                                        const uint16_t*, hipStream_t);
#endif

}  // namespace emu
