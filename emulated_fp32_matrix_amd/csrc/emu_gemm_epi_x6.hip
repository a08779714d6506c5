// The transformer-block operators' GEMM with six products (BF16X6).
#define EMU_GEMM_EPI_INSTANTIATE 3
#include "emu_gemm_epi.h"
