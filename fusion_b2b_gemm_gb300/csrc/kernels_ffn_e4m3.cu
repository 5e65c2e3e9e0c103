// Feed-forward kernels with e4m3 operands.
#include "ffn_registry.h"

namespace b2b {
ScaledKernels scaled_kernels() {
  return {gemm_kernel_pair<kGemmE4M3, false, false, kEpiGateQuant, kGemmF16>(),
          {gemm_kernel_pair<kGemmE4M3, false, false, kEpiStore, kGemmF16>(),
           gemm_kernel_pair<kGemmE4M3, false, false, kEpiStore, kGemmBF16>()},
          skinny_kernels<kGemmE4M3, kGemmF16, kEpiGateQuant, true>(),
          {skinny_kernels<kGemmE4M3, kGemmF16, kEpiStore, true>(), skinny_kernels<kGemmE4M3, kGemmBF16, kEpiStore, true>()}};
}
}  // namespace b2b
