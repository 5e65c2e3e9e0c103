// The compiled kernels of the feed-forward operators.
#pragma once

#include "gemm.cuh"
#include "quantize.cuh"

namespace b2b {

// A GEMM and the kernel that joins the parts of tiles cut along k.
struct GemmKernel {
  const void* main;
  const void* combine;
};

template <int IN, bool AMN, bool BMN, int EPI, int OUT>
GemmKernel gemm_kernel_pair() {
  return {reinterpret_cast<const void*>(&gemm_kernel<IN, AMN, BMN, EPI, OUT>),
          reinterpret_cast<const void*>(&gemm_combine_kernel<EPI, OUT>)};
}

// By operand type: the products of the block and of its backward pass.
struct FfnKernels {
  GemmKernel gate;       // H = act(X.Wg) * (X.Wu)
  GemmKernel down;       // Y = H.Wd
  GemmKernel gate_grad;  // dG, dU from dY.Wd^T
  GemmKernel dx;         // dG.Wg^T + dU.Wu^T
  GemmKernel dw;         // X^T.dG, X^T.dU, H^T.dY
  GemmKernel dw_add;     // the same, added to fp32
  const void* quantize_rows;
  const void* quantize_tiles;
};

template <int T>
FfnKernels ffn_kernels() {
  return {gemm_kernel_pair<T, false, true, kEpiGate, T>(),
          gemm_kernel_pair<T, false, true, kEpiStore, T>(),
          gemm_kernel_pair<T, false, false, kEpiGateGrad, T>(),
          gemm_kernel_pair<T, false, false, kEpiStore, T>(),
          gemm_kernel_pair<T, true, true, kEpiStore, T>(),
          gemm_kernel_pair<T, true, true, kEpiAdd, T>(),
          reinterpret_cast<const void*>(&quantize_rows_kernel<T>),
          reinterpret_cast<const void*>(&quantize_tiles_kernel<T>)};
}
FfnKernels ffn_kernels_f16();
FfnKernels ffn_kernels_bf16();

// e4m3 operands; `product` by type of the result.
struct ScaledKernels {
  GemmKernel gate;        // quantised H
  GemmKernel product[2];  // f16, bf16
};
ScaledKernels scaled_kernels();

}  // namespace b2b
