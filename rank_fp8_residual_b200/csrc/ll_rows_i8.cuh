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
// The nearest code.  p = 127 u has 23 bits: exact.  From y ~ 1 / a (within
// 2^-22), q0 = p y is within 4 units in the last place (ulp) of t = p / a;
// e = p - q0 a is exact by one fused multiply-add (a multiple of ulp(q0) *
// ulp16(a) and below 2^24 of them), and q = q0 + e y (Markstein's correction,
// IBM J. Res. Dev. 34, 1990) is t + d, |d| < 2^-19 ulp, rounded once.  That
// suffices: a border n + 1/2 is a binary32 number, so a t on a border gives q
// = t, and adding 1.5 * 2^23 rounds it to the even integer; any other t is
// at least 2^-s / (2 A) away from a border, with A < 65026 the 16-bit
// significand of a and 2^-s the ratio of u's unit to a's, while half an ulp of
// t is at most 2^-s / 2^17: q stays on t's side of the border.
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
  float eps, inv_k;          // inv_k: 1 / K
  int M, K;
};

constexpr float kRound = 12582912.f;  // 1.5 * 2^23
constexpr int kRowsMaxK = 1024 * 8 * 8;  // 1024 threads with 8 chunks of 8 values each
// Threads per row that a kernel with c chunks per thread may have.
constexpr int rows_max_threads(int c) { return c == 4 ? 256 : 1024; }

// Products of the low and the high bf16 of two words in binary32 (exact: 16
// bits), added to c.  The mixed-precision fused multiply-add takes the bf16
// halves as they are, on the multiply-add pipe; unpacking them first costs an
// operation each on the pipe that already bounds these kernels.
__device__ __forceinline__ float fma_lo(uint32_t a, uint32_t b, float c) {
  float d;
  asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
      "fma.rn.f32.bf16 %0, al, bl, %3;\n\t}"
      : "=f"(d)
      : "r"(a), "r"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float fma_hi(uint32_t a, uint32_t b, float c) {
  float d;
  asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
      "fma.rn.f32.bf16 %0, ah, bh, %3;\n\t}"
      : "=f"(d)
      : "r"(a), "r"(b), "f"(c));
  return d;
}
constexpr uint32_t kOnes = 0x3F803F80u;  // two bf16 ones
constexpr uint32_t k127s = 0x42FE42FEu;  // two bf16 127s
// Two maxima of magnitudes, NaN where either is.
__device__ __forceinline__ uint32_t absmax2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.NaN.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// bf16(a + b): rounding the exact sum once is also what rounding the
// binary32 sum gives (24 >= 2 * 8 + 2 bits).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// max(a, |b|), NaN if either is.
__device__ __forceinline__ float absmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The code of p / a in the low byte, p = 127 u (see above).
__device__ __forceinline__ uint32_t code_of(float p, float a, float y) {
  const float q0 = p * y;
  return __float_as_uint(fmaf(fmaf(-q0, a, p), y, q0) + kRound);
}
__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// One row per blockIdx.x and threadIdx.y: kC chunks of eight values for each
// of blockDim.x threads (a multiple of 32; one warp where blockDim.y > 1).
// kNorm: the norm, else the quantisation alone.
//
// A norm's u stays in registers between the maximum and the codes up to four
// chunks per thread; with eight it would spill, so there h stays (packed) and
// the products are taken once more.
template <int kC, bool kNorm>
__global__ void __launch_bounds__(rows_max_threads(kC)) ll_rows_i8_kernel(const RowsParams p) {
  __shared__ float s_sum[2][32];
  __shared__ uint32_t s_max[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nw = blockDim.x >> 5;
  const int nv = p.K >> 3;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int m = blockIdx.x * blockDim.y + threadIdx.y;
  if (m >= p.M) return;  // a whole warp, and no barrier follows for rows of one warp
  const size_t row = static_cast<size_t>(m) * p.K;
  uint4 hv[kC], rv[kC];
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    const int c = threadIdx.x + j * blockDim.x;
    hv[j] = c < nv ? reinterpret_cast<const uint4*>(p.x + row)[c] : make_uint4(0, 0, 0, 0);
    if (kNorm && p.residual)
      rv[j] = c < nv ? reinterpret_cast<const uint4*>(p.residual + row)[c] : make_uint4(0, 0, 0, 0);
  }
  const auto gain = [&](int c) {
    return p.w && c < nv ? __ldg(reinterpret_cast<const uint4*>(p.w) + c) : make_uint4(kOnes, kOnes, kOnes, kOnes);
  };
  constexpr bool kKeep = kC <= 4;
  float u[kKeep ? kC : 1][8];  // of the norm
  float ss = 0.f;
  uint32_t mx = 0;  // max |u| as bits: NaN above infinity above every finite value
  if (kNorm) {
    float am = 0.f;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      if (p.residual) {
        hv[j].x = add_bf16x2(hv[j].x, rv[j].x);
        hv[j].y = add_bf16x2(hv[j].y, rv[j].y);
        hv[j].z = add_bf16x2(hv[j].z, rv[j].z);
        hv[j].w = add_bf16x2(hv[j].w, rv[j].w);
        if (p.h && c < nv) reinterpret_cast<uint4*>(p.h + row)[c] = hv[j];
      }
      const uint4 wv = gain(c);
      const uint32_t hw[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w}, ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss = fma_lo(hw[i], hw[i], ss);
        ss = fma_hi(hw[i], hw[i], ss);
        const float u0 = fma_lo(hw[i], ww[i], 0.f), u1 = fma_hi(hw[i], ww[i], 0.f);
        am = absmax_nan(absmax_nan(am, u0), u1);
        if (kKeep) {
          u[j][2 * i] = u0;
          u[j][2 * i + 1] = u1;
        }
      }
    }
    mx = __float_as_uint(am);
  } else {
    uint32_t m2 = 0;  // two bf16 magnitudes (positive: the order of the bits is that of the values)
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      m2 = absmax2_nan(m2, hv[j].x);
      m2 = absmax2_nan(m2, hv[j].y);
      m2 = absmax2_nan(m2, hv[j].z);
      m2 = absmax2_nan(m2, hv[j].w);
    }
    mx = max(m2 << 16, m2 & 0xFFFF0000u);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  const auto warp_sum = [](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  if (kNorm) ss = warp_sum(ss);
  if (nw > 1) {
    if (lane == 0) {
      s_max[warp] = mx;
      s_sum[0][warp] = ss;
    }
    __syncthreads();
    mx = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
    if (kNorm) ss = warp_sum(lane < nw ? s_sum[0][lane] : 0.f);
  }
  float a = __uint_as_float(mx), rstd = 1.f;
  const bool bad = mx >= 0x7F800000u;
  if (kNorm) {
    if (p.y || threadIdx.x == 0) rstd = 1.f / sqrtf(fmaf(ss, p.inv_k, p.eps));
    if (isinf(ss) && !bad) {
      // Finite values whose squares overflow: the squares of h * 2^-64,
      // beside which eps does not count.  h comes from memory once more: as
      // this thread stored it, or from inputs that nothing has written.
      float s2 = 0.f;
      for (int c = threadIdx.x; c < nv; c += blockDim.x) {
        uint4 v = reinterpret_cast<const uint4*>((p.h ? p.h : p.x) + row)[c];
        if (p.residual && !p.h) {
          const uint4 r = reinterpret_cast<const uint4*>(p.residual + row)[c];
          v = make_uint4(add_bf16x2(v.x, r.x), add_bf16x2(v.y, r.y), add_bf16x2(v.z, r.z), add_bf16x2(v.w, r.w));
        }
        const uint32_t hw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float h0 = fma_lo(hw[i], kOnes, 0.f) * 0x1p-64f, h1 = fma_hi(hw[i], kOnes, 0.f) * 0x1p-64f;
          s2 = fmaf(h0, h0, s2);
          s2 = fmaf(h1, h1, s2);
        }
      }
      s2 = warp_sum(s2);
      if (nw > 1) {
        if (lane == 0) s_sum[1][warp] = s2;
        __syncthreads();
        s2 = warp_sum(lane < nw ? s_sum[1][lane] : 0.f);
      }
      rstd = 0x1p-64f / sqrtf(s2 * p.inv_k);
    }
  }
  if (p.codes && threadIdx.x == 0)
    p.scale[m] = bad ? __int_as_float(0x7FC00000) : (kNorm ? a * rstd : a) / 127.f;
  // Rows far from 1 are scaled by a power of two, so that 1 / a, 127 u and
  // the corrections stay finite and normal.
  const float pre = a > 0x1p100f ? 0x1p-60f : (a < 0x1p-60f ? 0x1p80f : 1.f);
  const float pre127 = 127.f * pre;
  a *= pre;
  const float yr = a > 0.f ? __frcp_rn(a) : 0.f;
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    const int c = threadIdx.x + j * blockDim.x;
    if (c >= nv) break;
    float v[8];  // 127 u
    if (kNorm) {
      float(&uj)[8] = u[kKeep ? j : 0];
      if (!kKeep) {
        const uint4 wv = gain(c);
        const uint32_t hw[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w}, ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uj[2 * i] = fma_lo(hw[i], ww[i], 0.f);
          uj[2 * i + 1] = fma_hi(hw[i], ww[i], 0.f);
        }
      }
      if (p.y)
        reinterpret_cast<uint4*>(p.y + row)[c] =
            make_uint4(pack_bf16x2(uj[0] * rstd, uj[1] * rstd), pack_bf16x2(uj[2] * rstd, uj[3] * rstd),
                       pack_bf16x2(uj[4] * rstd, uj[5] * rstd), pack_bf16x2(uj[6] * rstd, uj[7] * rstd));
      if (!p.codes) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = uj[i] * pre127;
    } else {
      const uint32_t hw[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = fma_lo(hw[i], k127s, 0.f);
        v[2 * i + 1] = fma_hi(hw[i], k127s, 0.f);
      }
      if (pre127 != 127.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = fma_lo(hw[i], kOnes, 0.f) * pre127;
          v[2 * i + 1] = fma_hi(hw[i], kOnes, 0.f) * pre127;
        }
      }
    }
    uint2 out = make_uint2(0u, 0u);
    if (!bad) {
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = code_of(v[i], a, yr);
      out = make_uint2(pack_codes(r[0], r[1], r[2], r[3]), pack_codes(r[4], r[5], r[6], r[7]));
    }
    reinterpret_cast<uint2*>(p.codes + row)[c] = out;
  }
}

}  // namespace llk
