// 16-bit values to e4m3 with a power-of-two scale for each block: 128 values of
// a row (activations) or 128 x 128 values (weights).  Bound by memory: 2 bytes
// read and 1 written for each value, once.
#pragma once

#include "gemm.cuh"

namespace b2b {

constexpr int kQuantThreads = 256;

struct QuantParams {
  long long rows, cols;  // cols a multiple of 8
  const void* x;
  long long x_ld;
  uint8_t* q;
  long long q_ld;
  float* scale;          // of (row or row block, column block)
  long long scale_row, scale_k;
};

// Blocks of 128 of a row: 16 lanes take a block, 8 values each, so a warp takes
// two rows; a thread block 16 rows of kQuantBlocks column blocks, whose loads
// overlap (one at a time: 2048 x 4096 in 8.2 us, four 7.4 us).
constexpr int kQuantBlocks = 4;
template <int T>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const __grid_constant__ QuantParams p) {
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 15;
  const long long row = static_cast<long long>(blockIdx.x) * (kQuantThreads / 16) + (threadIdx.x >> 4);
  for (long long kb0 = static_cast<long long>(blockIdx.y) * kQuantBlocks; kb0 * 128 < p.cols; kb0 += static_cast<long long>(gridDim.y) * kQuantBlocks) {
    uint4 w[kQuantBlocks];
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
      const long long col = (kb0 + i) * 128 + lane * 8;
      w[i] = make_uint4(0, 0, 0, 0);
      if (row < p.rows && col < p.cols)
        w[i] = gemm::load(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.x_ld + col));
    }
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
      const long long kb = kb0 + i, col = kb * 128 + lane * 8;
      float v[8];
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gemm::unpack16<T>((&w[i].x)[e], v[2 * e], v[2 * e + 1]);
        top = max(top, max(__float_as_uint(v[2 * e]) & 0x7fffffffu, __float_as_uint(v[2 * e + 1]) & 0x7fffffffu));
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      float inv;
      const float scale = gemm::block_scale(top, inv);
      if (row < p.rows && col < p.cols)
        *reinterpret_cast<uint2*>(p.q + row * p.q_ld + col) =
            make_uint2(gemm::pack_e4m3(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       gemm::pack_e4m3(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
      if (lane == 0 && row < p.rows && kb * 128 < p.cols) p.scale[row * p.scale_row + kb * p.scale_k] = scale;
    }
  }
}

// Blocks of 128 x 128: one for a thread block, 16 lanes to a row, 8 rows a thread.
template <int T>
__global__ void __launch_bounds__(kQuantThreads) quantize_tiles_kernel(const __grid_constant__ QuantParams p) {
  __shared__ uint32_t tops[kQuantThreads / 32];
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 15;
  for (long long kb = blockIdx.y; kb * 128 < p.cols; kb += gridDim.y) {
    const long long row0 = static_cast<long long>(blockIdx.x) * 128 + (threadIdx.x >> 4), col = kb * 128 + lane * 8;
    uint4 w[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long row = row0 + 16 * i;
      w[i] = make_uint4(0, 0, 0, 0);
      if (row < p.rows && col < p.cols)
        w[i] = gemm::load(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.x_ld + col));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, b;
        gemm::unpack16<T>((&w[i].x)[e], a, b);
        top = max(top, max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) top = max(top, tops[i]);
    __syncthreads();
    float inv;
    const float scale = gemm::block_scale(top, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long row = row0 + 16 * i;
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) gemm::unpack16<T>((&w[i].x)[e], v[2 * e], v[2 * e + 1]);
      if (row < p.rows && col < p.cols)
        *reinterpret_cast<uint2*>(p.q + row * p.q_ld + col) =
            make_uint2(gemm::pack_e4m3(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       gemm::pack_e4m3(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    }
    if (threadIdx.x == 0) p.scale[blockIdx.x * p.scale_row + kb * p.scale_k] = scale;
  }
}

}  // namespace b2b
