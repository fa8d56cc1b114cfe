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
#include <math_constants.h>

#include "ptx.cuh"
#include "ptx_i8.cuh"

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
// Threads per row that a kernel may have: 1024, or 256 for four and eight
// chunks per thread with u kept.
constexpr int rows_max_threads(int c, bool keep) { return c >= 4 && keep ? 256 : 1024; }

// The two bf16 of a word.
__device__ __forceinline__ float2 bf16x2_to_f32x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
// The two products of the bf16 of two words, exact in binary32 (-0 added keeps
// a zero's sign), by the multiplier that takes bf16 operands as they lie
// (16384 x 4096 without residual 41.3 us with the gain unpacked, 40.4 so).
__device__ __forceinline__ float2 mul_bf16x2(uint32_t a, uint32_t b) {
  float2 r;
  asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %2;\n\tmov.b32 {bl, bh}, %3;\n\t"
      "fma.rn.f32.bf16 %0, al, bl, 0f80000000;\n\tfma.rn.f32.bf16 %1, ah, bh, 0f80000000;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kOnes = 0x3F803F80u;  // two bf16 ones
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
// max(a, |b.x|, |b.y|) for a >= 0, NaN if any is.
__device__ __forceinline__ float absmax_nan(float a, float2 b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b.x), "f"(b.y));
  return r;
}

// The codes of p / a in the low bytes, p = 127 u (see above); na = -a, y ~ 1 / a.
__device__ __forceinline__ float2 codes_of(float2 p, float2 na, float2 y) {
  const float2 q0 = mul2(p, y);
  return add2(fma2(fma2(q0, na, p), y, q0), make_float2(kRound, kRound));
}
__device__ __forceinline__ uint32_t pack_codes(float2 a, float2 b) {
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

// The norm of a row that leaves binary32's range: squares or products that
// overflow (finite ones are finite here, below 2^256), products all below
// 2^-100 (the largest then has too few bits to spare: exact here), NaN and
// infinities, which are marked.  In binary64, where 127 u is exact and the
// quotient's rounding cannot cross n + 1/2.  h comes from memory once more:
// as this thread stored it, or from inputs that nothing has written.  A row
// of zeros under a gain comes here too (3630 x 4096 of nothing else 34 us,
// ordinary rows 17).
__device__ __forceinline__ void norm_row_far(const RowsParams& p, unsigned m) {
  __shared__ double s_far[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5, nv = p.K >> 3;
  const size_t row = static_cast<size_t>(m) * p.K;
  const auto load = [&](int c, uint32_t* hw, uint32_t* ww) {
    uint4 v = reinterpret_cast<const uint4*>((p.h ? p.h : p.x) + row)[c];
    if (p.residual && !p.h) {
      const uint4 r = reinterpret_cast<const uint4*>(p.residual + row)[c];
      v = make_uint4(add_bf16x2(v.x, r.x), add_bf16x2(v.y, r.y), add_bf16x2(v.z, r.z), add_bf16x2(v.w, r.w));
    }
    const uint4 w = p.w ? reinterpret_cast<const uint4*>(p.w)[c] : make_uint4(kOnes, kOnes, kOnes, kOnes);
    hw[0] = v.x, hw[1] = v.y, hw[2] = v.z, hw[3] = v.w;
    ww[0] = w.x, ww[1] = w.y, ww[2] = w.z, ww[3] = w.w;
  };
  double ss = 0., a = 0.;
  for (int c = threadIdx.x; c < nv; c += blockDim.x) {
    uint32_t hw[4], ww[4];
    load(c, hw, ww);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = bf16x2_to_f32x2(hw[i]), w = bf16x2_to_f32x2(ww[i]);
      ss += static_cast<double>(h.x) * h.x + static_cast<double>(h.y) * h.y;
      const double u0 = fabs(static_cast<double>(h.x) * w.x), u1 = fabs(static_cast<double>(h.y) * w.y);
      a = isfinite(u0) && isfinite(u1) ? fmax(a, fmax(u0, u1)) : CUDART_INF;
    }
  }
  const auto reduce = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      a = fmax(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
  };
  reduce();
  if (nw > 1) {
    if (lane == 0) {
      s_far[0][warp] = ss;
      s_far[1][warp] = a;
    }
    __syncthreads();
    ss = lane < nw ? s_far[0][lane] : 0.;
    a = lane < nw ? s_far[1][lane] : 0.;
    reduce();
  }
  const bool bad = isinf(a);
  const double rstd = 1. / sqrt(ss / p.K + p.eps);
  if (p.codes && threadIdx.x == 0) p.scale[m] = bad ? CUDART_NAN_F : static_cast<float>(a * rstd / 127.);
  for (int c = threadIdx.x; c < nv; c += blockDim.x) {
    uint32_t hw[4], ww[4];
    load(c, hw, ww);
    uint32_t o[4];
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = bf16x2_to_f32x2(hw[i]), w = bf16x2_to_f32x2(ww[i]);
      const double u0 = static_cast<double>(h.x) * w.x, u1 = static_cast<double>(h.y) * w.y;
      o[i] = pack_bf16x2(static_cast<float>(u0 * rstd), static_cast<float>(u1 * rstd));
      if (!bad && a > 0.) {
        const uint32_t c0 = __double2int_rn(127. * u0 / a) & 255, c1 = __double2int_rn(127. * u1 / a) & 255;
        out[i >> 1] |= (c0 | c1 << 8) << (i & 1) * 16;
      }
    }
    if (p.y) reinterpret_cast<uint4*>(p.y + row)[c] = make_uint4(o[0], o[1], o[2], o[3]);
    if (p.codes) reinterpret_cast<uint2*>(p.codes + row)[c] = make_uint2(out[0], out[1]);
  }
}

// One row per blockIdx.x and threadIdx.y: kC chunks of eight values for each
// of blockDim.x threads (a multiple of 32; one warp where blockDim.y > 1).
// kNorm: the norm, else the quantisation alone.
//
// kKeep: a norm's u stays in registers between the maximum and the codes, in
// blocks of up to 256 threads.  Beyond, that would cost the second block on an
// SM, so h stays, packed, and the products are taken once more (4000 x 16384
// with residual 68.8 us by 512 threads, 90 with u kept; by 256 68.7, without
// residual 47.5 and 42.7).  Rows of more than 16384 values are those of 512 to
// 1024 threads, one block on an SM: 4000 x 24576 158 us with residual (the bytes
// take 107), 108 without (46); 2000 x 65536 182 (142) and 116 (61).
//
// One or two chunks serve batches of few rows, where registers are free and
// loads in flight are not: the second bound lets the compiler use 64 (1000 x
// 4096 with residual 8.0 -> 7.4 us).
template <int kC, bool kNorm, bool kKeep>
__global__ void __launch_bounds__(rows_max_threads(kC, kKeep), kC <= 2 ? 1 : 0) ll_rows_i8_kernel(const RowsParams p) {
  __shared__ __align__(16) float s_sum[32];
  __shared__ __align__(16) uint32_t s_max[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nw = blockDim.x >> 5;
  const int nv = p.K >> 3;
  pdl_launch_dependents();
  pdl_wait_primary();
  const unsigned m = blockIdx.x * blockDim.y + threadIdx.y;  // may pass 2^31 behind the last row
  if (m >= static_cast<unsigned>(p.M)) return;  // a whole warp, and no barrier follows for rows of one warp
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
    return c < nv ? reinterpret_cast<const uint4*>(p.w)[c] : make_uint4(kOnes, kOnes, kOnes, kOnes);
  };
  constexpr bool kAhead = kC <= 4 || kKeep;  // the gains' loads go out with x's
  uint4 wv[kAhead ? kC : 1];
  if (kNorm && kAhead && p.w) {
#pragma unroll
    for (int j = 0; j < kC; ++j) wv[kAhead ? j : 0] = gain(threadIdx.x + j * blockDim.x);
  }
  float2 u[kKeep ? kC : 1][4];  // of the norm
  float ss = 0.f;
  uint32_t mx = 0;  // max |u| as bits: NaN above infinity above every finite value
  if (kNorm) {
    float am = 0.f;
    float2 s2 = make_float2(0.f, 0.f);
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
      const uint32_t hw[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w};
      float2 uj[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uj[i] = bf16x2_to_f32x2(hw[i]);
        s2 = fma2(uj[i], uj[i], s2);
      }
      if (p.w) {
        const uint4 wj = kAhead ? wv[kAhead ? j : 0] : gain(c);
        const uint32_t ww[4] = {wj.x, wj.y, wj.z, wj.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) uj[i] = mul_bf16x2(hw[i], ww[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        am = absmax_nan(am, uj[i]);
        if (kKeep) u[j][i] = uj[i];
      }
    }
    ss = s2.x + s2.y;
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
      s_sum[warp] = ss;
    }
    __syncthreads();
    if (nw <= 8) {  // few enough to add up without shuffles (16384 x 8192 with residual 134.9 -> 134.4 us, 2048 x 8192 20.4 -> 19.8)
      const uint4 m4 = *reinterpret_cast<const uint4*>(s_max);
      const float4 t4 = *reinterpret_cast<const float4*>(s_sum);
      mx = max(m4.x, m4.y);
      ss = t4.x + t4.y;
      if (nw > 2) mx = max(mx, m4.z), ss += t4.z;
      if (nw > 3) mx = max(mx, m4.w), ss += t4.w;
      if (nw > 4) {
        const uint4 m5 = reinterpret_cast<const uint4*>(s_max)[1];
        const float4 t5 = reinterpret_cast<const float4*>(s_sum)[1];
        mx = max(mx, m5.x), ss += t5.x;
        if (nw > 5) mx = max(mx, m5.y), ss += t5.y;
        if (nw > 6) mx = max(mx, m5.z), ss += t5.z;
        if (nw > 7) mx = max(mx, m5.w), ss += t5.w;
      }
    } else {
      mx = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
      if (kNorm) ss = warp_sum(lane < nw ? s_sum[lane] : 0.f);
    }
  }
  float a = __uint_as_float(mx), rstd = 1.f;
  const bool bad = !kNorm && mx >= 0x7F800000u;
  if (kNorm) {
    if (mx >= 0x7F800000u || isinf(ss) || (p.w && a < 0x1p-100f)) return norm_row_far(p, m);  // alike in all threads of the row
    if (p.y || threadIdx.x == 0) rstd = 1.f / sqrtf(fmaf(ss, p.inv_k, p.eps));
  }
  if (p.codes && threadIdx.x == 0) {
    const bool big = a > 1.f;  // then a * rstd may overflow where the scale does not, else a / 127 underflow
    const float t = (big ? a : a * rstd) / 127.f;
    p.scale[m] = bad ? CUDART_NAN_F : (big ? t * rstd : t);
  }
  // Rows far from 1 are scaled by a power of two, so that 1 / a, 127 u and
  // the corrections stay finite and normal.
  const float pre = a > 0x1p100f ? 0x1p-60f : (a < 0x1p-60f ? 0x1p80f : 1.f);
  const float pre127 = 127.f * pre;
  a *= pre;
  const float yr = a > 0.f ? __fdividef(1.f, a) : 0.f;
  const float2 y2 = make_float2(yr, yr), na2 = make_float2(-a, -a), p127 = make_float2(pre127, pre127);
  const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    const int c = threadIdx.x + j * blockDim.x;
    if (c >= nv) break;
    float2 v[4];
    if (kNorm && kKeep) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = u[j][i];
    } else {
      const uint32_t hw[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w};
      if (kNorm && p.w) {
        const uint4 wj = gain(c);
        const uint32_t ww[4] = {wj.x, wj.y, wj.z, wj.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul_bf16x2(hw[i], ww[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = bf16x2_to_f32x2(hw[i]);
      }
    }
    if (kNorm) {
      if (p.y) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 t = mul2(v[i], r2);
          o[i] = pack_bf16x2(t.x, t.y);
        }
        reinterpret_cast<uint4*>(p.y + row)[c] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (!p.codes) continue;
    }
    uint2 out = make_uint2(0u, 0u);
    if (!bad) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = codes_of(mul2(v[i], p127), na2, y2);
      out = make_uint2(pack_codes(v[0], v[1]), pack_codes(v[2], v[3]));
    }
    reinterpret_cast<uint2*>(p.codes + row)[c] = out;
  }
}

}  // namespace llk
