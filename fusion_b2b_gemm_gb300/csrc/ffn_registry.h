// The compiled kernels of the feed-forward operators.
#pragma once

#include "gemm.cuh"
#include "quantize.cuh"
#include "skinny.cuh"

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

// The kernels for tiles of 16, 32, 64 and (16-bit operands) 128 rows.
struct SkinnyKernels {
  const void* main[4];
  int smem[4], threads[4], sizes, columns, depth;
  bool k_major;  // order of the weights
  bool gate;
  SkinnyCost cost;
};
template <int IN, int OUT, int EPI, bool KM>
SkinnyKernels skinny_kernels() {
  constexpr bool F8 = IN == kGemmE4M3, GATE = EPI == kEpiGate || EPI == kEpiGateQuant;
  SkinnyKernels k = {{reinterpret_cast<const void*>(&skinny_kernel<IN, OUT, EPI, KM, 16>), reinterpret_cast<const void*>(&skinny_kernel<IN, OUT, EPI, KM, 32>),
                      reinterpret_cast<const void*>(&skinny_kernel<IN, OUT, EPI, KM, 64>), nullptr},
                     {SkinnyShape<F8, GATE, 16>::kBytes, SkinnyShape<F8, GATE, 32>::kBytes, SkinnyShape<F8, GATE, 64>::kBytes, 0},
                     {SkinnyShape<F8, GATE, 16>::kThreads, SkinnyShape<F8, GATE, 32>::kThreads, SkinnyShape<F8, GATE, 64>::kThreads, 0},
                     3,
                     SkinnyShape<F8, GATE, 16>::kColumns,
                     SkinnyShape<F8, GATE, 16>::kDepth,
                     KM,
                     GATE,
                     SkinnyShape<F8, GATE, 16>::cost(KM)};
  if constexpr (!F8) {
    k.main[3] = reinterpret_cast<const void*>(&skinny_kernel<IN, OUT, EPI, KM, 128>);
    k.smem[3] = SkinnyShape<F8, GATE, 128>::kBytes;
    k.threads[3] = SkinnyShape<F8, GATE, 128>::kThreads;
    k.sizes = 4;
  }
  return k;
}

// By operand type: the products of the block and of its backward pass.
struct FfnKernels {
  GemmKernel gate;       // H = act(X.Wg) * (X.Wu)
  GemmKernel down;       // Y = H.Wd
  GemmKernel gate_grad;  // dG, dU from dY.Wd^T
  GemmKernel dx;         // dG.Wg^T + dU.Wu^T
  GemmKernel dw;         // X^T.dG, X^T.dU, H^T.dY
  GemmKernel dw_add;     // the same, added to fp32
  SkinnyKernels gate_few, down_few, gate_grad_few, dx_few;
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
          skinny_kernels<T, T, kEpiGate, false>(),
          skinny_kernels<T, T, kEpiStore, false>(),
          skinny_kernels<T, T, kEpiGateGrad, true>(),
          skinny_kernels<T, T, kEpiStore, true>(),
          reinterpret_cast<const void*>(&quantize_rows_kernel<T>),
          reinterpret_cast<const void*>(&quantize_tiles_kernel<T>)};
}
FfnKernels ffn_kernels_f16();
FfnKernels ffn_kernels_bf16();

// e4m3 operands; `product` by type of the result.
struct ScaledKernels {
  GemmKernel gate;        // quantised H
  GemmKernel product[2];  // f16, bf16
  SkinnyKernels gate_few, product_few[2];
};
ScaledKernels scaled_kernels();

}  // namespace b2b
