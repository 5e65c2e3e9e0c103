// Feed-forward kernels with fp16 operands.
#include "ffn_registry.h"

namespace b2b {
FfnKernels ffn_kernels_f16() { return ffn_kernels<kGemmF16>(); }
}  // namespace b2b
