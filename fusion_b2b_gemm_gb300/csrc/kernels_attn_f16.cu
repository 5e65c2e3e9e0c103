// Attention kernels with fp16 operands.
#include "attention_registry.h"

namespace b2b {
AttnKernels attn_kernels_f16() { return attn_kernels<false>(); }
}  // namespace b2b
