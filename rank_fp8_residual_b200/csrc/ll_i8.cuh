// Int8 matrix product with scales (sm_100a):
//
//   y[m, n] = bf16( act( sx[m] * sw[n] * sum_k xq[m, k] wq[n, k] + bias[n] ) )
//
// xq [M, K] int8 codes with one scale per token, wq [N, K] int8 codes with
// one scale per output feature.  The sum is exact in int32 (K <= 131056 keeps
// it below 2^31 even for codes of -128), so the order in which partial sums
// are added does not change the result.
#pragma once
#include <cstdint>
#include <cuda.h>

#include "ptx.cuh"

namespace llk {

constexpr int kI8MaxK = 131056;

// A 64 x 64 tile per block, four int8 products per dp4a.
__global__ void __launch_bounds__(256) ll_i8_simple_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                                                           const int8_t* __restrict__ wq, const float* __restrict__ sw,
                                                           const uint16_t* __restrict__ bias, uint16_t* __restrict__ y,
                                                           int M, int N, int K, int gelu) {
  __shared__ int xs[64][17], ws[64][17];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tm = threadIdx.x >> 4, tn = threadIdx.x & 15;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 64) {
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
    int4 xv = make_int4(0, 0, 0, 0), wv = xv;
    if (k0 + c < K) {
      if (m0 + r < M) xv = *reinterpret_cast<const int4*>(xq + static_cast<size_t>(m0 + r) * K + k0 + c);
      if (n0 + r < N) wv = *reinterpret_cast<const int4*>(wq + static_cast<size_t>(n0 + r) * K + k0 + c);
    }
    __syncthreads();
    const int w = c / 4;
    xs[r][w] = xv.x; xs[r][w + 1] = xv.y; xs[r][w + 2] = xv.z; xs[r][w + 3] = xv.w;
    ws[r][w] = wv.x; ws[r][w + 1] = wv.y; ws[r][w + 2] = wv.z; ws[r][w + 3] = wv.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[tm + 16 * i][k], ws[tn + 16 * j][k], acc[i][j]);
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
      if (m >= M || n >= N) continue;
      float v = fmaf(static_cast<float>(acc[i][j]), sx[m] * sw[n], bias ? bf16_bits_to_float(bias[n]) : 0.f);
      if (gelu) v = gelu_tanh(v);
      y[static_cast<size_t>(m) * N + n] = to_bf16_bits(v);
    }
}

}  // namespace llk
