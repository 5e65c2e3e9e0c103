// The compiled attention kernels of one operand type.
#pragma once

#include "attention.cuh"

namespace b2b {

struct AttnKernels {
  const void* main[2];  // padded head size 64, 128
  int smem[2];          // dynamic shared memory of each
  const void* combine;
};

template <bool BF16>
AttnKernels attn_kernels() {
  return {{reinterpret_cast<const void*>(&attn_kernel<BF16, 64>), reinterpret_cast<const void*>(&attn_kernel<BF16, 128>)},
          {AttnShape<64>::kBytes, AttnShape<128>::kBytes},
          reinterpret_cast<const void*>(&attn_combine_kernel<BF16>)};
}

AttnKernels attn_kernels_f16();
AttnKernels attn_kernels_bf16();

}  // namespace b2b
