// Row kernels of the int8 path (sm_100a): the RMS norm with the residual's
// addition and an int8 output, and the per-row int8 quantisation.
//
//   h[k]     = bf16(x[k] + residual[k])      (h = x without a residual)
//   u[k]     = h[k] * w[k]                   (u = h without a gain)
//   rstd     = 1 / sqrt(sum_k h[k]^2 / K + eps)
//   y[k]     = bf16(u[k] * rstd)
//   a        = max_k |u[k]|
//   codes[k] = the integer nearest to 127 u[k] / a, ties to even
//   scale    = a * rstd / 127                (quantisation alone: a / 127)
//
// codes * scale stands for u * rstd, and rstd cancels in the code: it is the
// rounding of a quotient of exact values.  (A bf16 has 8 significant bits, so
// u has 16 and is exact in binary32.)  The norm is of h as stored, the values
// that the next block's residual adds to.
//
// Rounding to the nearest code: t = u * (127 / a) in binary32 is within
// 1.6e-5 of the quotient for |t| <= 127 (two roundings of 2^-24), so its
// rounding n is right unless t lies within kBorder of a border between two
// integers.  There e = 127 u - n a decides: 127 u and n a are exact (23 bits),
// and so is their difference (|e| <= a / 2 + a 2^-16 on u's grid, whose
// exponent is at most 8 below a's), so comparing 2 e with a is exact too.
#pragma once
#include <cstdint>
#include <cuda.h>

#include "ptx.cuh"

namespace llk {

struct RowsParams {
  const uint16_t* x;         // bf16 [M, K]; h may be the same buffer
  const uint16_t* residual;  // bf16 [M, K] or nullptr; h may be the same buffer
  const uint16_t* w;         // bf16 [K] or nullptr
  uint16_t* h;               // bf16 [M, K] or nullptr
  uint16_t* y;               // bf16 [M, K] or nullptr
  int8_t* codes;             // [M, K] or nullptr
  float* scale;              // [M] (with codes)
  float eps;
  int M, K;
  int norm;                  // 0: quantisation alone
};

constexpr float kBorder = 0.49996f;
constexpr int kRowsMaxChunks = 8;  // 16-byte chunks of a row per thread
constexpr int kRowsMaxK = 1024 * kRowsMaxChunks * 8;

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// The integer nearest to 127 u / a (ties to even) as a float; inv = 127 / a.
__device__ __forceinline__ float code_of(float u, float a, float inv) {
  float n = rintf(__fmul_rn(u, inv));
  const float t = __fmul_rn(u, inv);
  if (fabsf(t - n) > kBorder) {
    const float e2 = 2.f * fmaf(-n, a, 127.f * u);
    const bool odd = (static_cast<int>(n) & 1) != 0;
    if (e2 > a || (e2 == a && odd)) n += 1.f;
    else if (e2 < -a || (e2 == -a && odd)) n -= 1.f;
  }
  return n;
}

// One block per row (rows strided over the grid), the row's h in registers
// (kC chunks of 8 values per thread).
template <int kC>
__global__ void __launch_bounds__(1024) ll_rows_i8_kernel(const RowsParams p) {
  __shared__ float s_ss[32];
  __shared__ uint32_t s_mx[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nw = blockDim.x >> 5;
  const int nv = p.K >> 3;
  // Sum over the block (every thread gets it).
  auto block_sum = [&](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) s_ss[warp] = v;
    __syncthreads();
    float t = lane < nw ? s_ss[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
  };
  auto block_max = [&](uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) s_mx[warp] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < nw ? s_mx[lane] : 0u);
  };
  for (int m = blockIdx.x; m < p.M; m += gridDim.x) {
    const size_t row = static_cast<size_t>(m) * p.K;
    uint4 hv[kC];
    float ss = 0.f;
    uint32_t mx = 0;  // |u| as bits: NaN above infinity above every finite value
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      hv[j] = make_uint4(0, 0, 0, 0);
      if (c >= nv) continue;
      hv[j] = reinterpret_cast<const uint4*>(p.x + row)[c];
      uint32_t* hw = reinterpret_cast<uint32_t*>(&hv[j]);
      if (p.residual) {
        const uint4 r = reinterpret_cast<const uint4*>(p.residual + row)[c];
        const uint32_t* rw = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          hw[i] = pack_bf16x2(bf16_lo(hw[i]) + bf16_lo(rw[i]), bf16_hi(hw[i]) + bf16_hi(rw[i]));
        if (p.h) reinterpret_cast<uint4*>(p.h + row)[c] = hv[j];
      }
      uint4 wv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
      if (p.w) wv = __ldg(reinterpret_cast<const uint4*>(p.w) + c);
      const uint32_t* ww = reinterpret_cast<const uint32_t*>(&wv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float h0 = bf16_lo(hw[i]), h1 = bf16_hi(hw[i]);
        ss = fmaf(h0, h0, ss);
        ss = fmaf(h1, h1, ss);
        mx = max(mx, __float_as_uint(h0 * bf16_lo(ww[i])) & 0x7FFFFFFFu);
        mx = max(mx, __float_as_uint(h1 * bf16_hi(ww[i])) & 0x7FFFFFFFu);
      }
    }
    mx = block_max(mx);
    const bool bad = mx >= 0x7F800000u;
    float a = __uint_as_float(mx);
    float rstd = 1.f;
    if (p.norm) {
      ss = block_sum(ss);
      rstd = 1.f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
      if (isinf(ss) && !bad) {
        // Finite values whose squares overflow: the squares of h * 2^-64,
        // beside which eps does not count.
        float s2 = 0.f;
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          const uint32_t* hw = reinterpret_cast<const uint32_t*>(&hv[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float h0 = bf16_lo(hw[i]) * 0x1p-64f, h1 = bf16_hi(hw[i]) * 0x1p-64f;
            s2 = fmaf(h0, h0, s2);
            s2 = fmaf(h1, h1, s2);
          }
        }
        s2 = block_sum(s2);
        rstd = 0x1p-64f / sqrtf(s2 / static_cast<float>(p.K));
      }
    }
    if (p.codes && threadIdx.x == 0)
      p.scale[m] = bad ? __uint_as_float(0x7FC00000u) : (p.norm ? a * rstd : a) / 127.f;
    // Rows far from 1 are scaled by a power of two, so that 127 / a and 127 u
    // stay finite and normal.
    const float pre = a > 0x1p100f ? 0x1p-60f : (a < 0x1p-60f ? 0x1p60f : 1.f);
    a *= pre;
    const float inv = a > 0.f ? 127.f / a : 0.f;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      if (c >= nv) continue;
      const uint32_t* hw = reinterpret_cast<const uint32_t*>(&hv[j]);
      uint4 wv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
      if (p.w) wv = __ldg(reinterpret_cast<const uint4*>(p.w) + c);
      const uint32_t* ww = reinterpret_cast<const uint32_t*>(&wv);
      uint4 yv;
      uint32_t* yw = reinterpret_cast<uint32_t*>(&yv);
      uint32_t cw[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u0 = bf16_lo(hw[i]) * bf16_lo(ww[i]), u1 = bf16_hi(hw[i]) * bf16_hi(ww[i]);
        yw[i] = pack_bf16x2(u0 * rstd, u1 * rstd);
        if (p.codes && !bad) {
          const int c0 = static_cast<int>(code_of(u0 * pre, a, inv)), c1 = static_cast<int>(code_of(u1 * pre, a, inv));
          cw[i >> 1] |= (static_cast<uint32_t>(c0 & 0xFF) | (static_cast<uint32_t>(c1 & 0xFF) << 8)) << (16 * (i & 1));
        }
      }
      if (p.y) reinterpret_cast<uint4*>(p.y + row)[c] = yv;
      if (p.codes) reinterpret_cast<uint2*>(p.codes + row)[c] = make_uint2(cw[0], cw[1]);
    }
  }
}

}  // namespace llk
