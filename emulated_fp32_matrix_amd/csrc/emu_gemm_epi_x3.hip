// The transformer-block operators' GEMM with three products (BF16X3).
#define EMU_GEMM_EPI_INSTANTIATE 2
#include "emu_gemm_epi.h"
