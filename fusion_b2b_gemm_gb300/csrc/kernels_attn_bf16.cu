// Attention kernels with bf16 operands.
#include "attention_registry.h"

namespace b2b {
AttnKernels attn_kernels_bf16() { return attn_kernels<true>(); }
}  // namespace b2b
