// The transformer-block operators' GEMM with one product (BF16X1).
#define EMU_GEMM_EPI_INSTANTIATE 1
#include "emu_gemm_epi.h"
