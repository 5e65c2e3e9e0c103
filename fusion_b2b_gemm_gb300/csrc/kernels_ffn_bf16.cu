// Feed-forward kernels with bf16 operands.
#include "ffn_registry.h"

namespace b2b {
FfnKernels ffn_kernels_bf16() { return ffn_kernels<kGemmBF16>(); }
}  // namespace b2b
