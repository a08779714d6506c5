// The transformer-block operators' GEMM with nine products (BF16X9).
#define EMU_GEMM_EPI_INSTANTIATE 5
#include "emu_gemm_epi.h"
