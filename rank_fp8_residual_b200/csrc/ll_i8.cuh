// Int8 matrix product with scales (sm_100a):
//
//   y[m, n] = bf16( act( sx[m] * sw[n] * sum_k xq[m, k] wq[n, k] + bias[n] ) )
//
// xq [M, K] int8 codes with one scale per token, wq [N, K] int8 codes with
// one scale per output feature, both K-major.  The sum is exact in int32
// (K <= 131056 keeps it below 2^31 even for codes of -128), so the order in
// which partial sums are added does not change the result.  Both kernels run
// on tcgen05 kind::i8 (32 products deep per instruction, twice the bf16
// rate) with int32 accumulators in TMEM.
//
// Neither kernel keeps state between launches: tiles are dealt out by index
// and split sums meet in distributed shared memory, so launches of one layer
// may overlap.  Both are programmatic dependents of the kernel before them:
// the weight (the layer's own copy) is loaded at once, everything the
// caller owns only after griddepcontrol.wait; and both let their dependents
// launch only after their TMEM is allocated, so that a waiting dependent
// cannot hold the columns that a CTA of theirs still needs.
#pragma once
#include <cstdint>
#include <cuda.h>

#include "ll_kernels.cuh"
#include "ptx.cuh"

namespace llk {

constexpr int kI8MaxK = 131056;

// Instruction descriptor of tcgen05.mma kind::i8: int32 accumulation, signed
// A and B, both K-major.
__host__ __device__ __forceinline__ constexpr uint32_t idesc_i8(int m, int n) {
  return (2u << 4)                                  // D format: s32
         | (1u << 7)                                // A format: s8
         | (1u << 10)                               // B format: s8
         | (static_cast<uint32_t>(n >> 3) << 17)    // N / 8
         | (static_cast<uint32_t>(m >> 4) << 24);   // M / 16
}

__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two binary32 values at once (the packed multiply-add of sm_100).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float ex2(float v) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float rcp(float v) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}

// Two neighbouring outputs of a token from their sums: sm is the token's
// scale, s = (scale, scale, bias, bias) of the two features.  GELU:
// v / 2 (1 + tanh(z)) = v / (1 + exp(-2 z)), z = sqrt(2 / pi) (v + 0.044715 v^3);
// exp(-2 z) as a power of two: -2 z log2(e) = v (-2.3022082 - 0.10294324 v^2).
template <int kAct>
__device__ __forceinline__ uint32_t i8_out2(int a0, int a1, float sm, const float4& s) {
  float2 v = fma2(mul2(make_float2(s.x, s.y), make_float2(sm, sm)),
                  make_float2(static_cast<float>(a0), static_cast<float>(a1)), make_float2(s.z, s.w));
  if constexpr (kAct == kActGelu) {
    const float2 t = mul2(v, fma2(mul2(v, v), make_float2(-0.10294324f, -0.10294324f),
                                  make_float2(-2.3022082f, -2.3022082f)));
    v = mul2(v, make_float2(rcp(1.f + ex2(t.x)), rcp(1.f + ex2(t.y))));
  }
  return pack_bf16x2(v.x, v.y);
}

// ==================================================== many tokens: CTA pairs
struct I8Params {
  CUtensorMap tm_x;  // s8 xq [M, K]  box {128, 128},    128B swizzle
  CUtensorMap tm_w;  // s8 wq [N, K]  box {128, fn / 2}, 128B swizzle
  CUtensorMap tm_y;  // bf16 y [M, N] box {32, 32},      64B swizzle
  const float* sx;       // [M]
  const float4* sb;      // [N rounded up / 2] (scale, scale, bias, bias) of two features
  int M, N, K;
  int fn;                  // features per tile: a multiple of 32, 32..256
  int n_ttiles, n_ftiles;  // tiles of 256 tokens and fn features
  int withhold;            // debug: the producers issue nothing, so every consumer's wait runs out
  Watch watch;
};

constexpr int kI8Ring = 192 * 1024;
constexpr int kI8MaxStages = 8;
constexpr int kI8EpiWarps = 8;
constexpr int kI8Threads = 32 * (2 + kI8EpiWarps);
constexpr int kI8Stage = 2 * 32 * 64;  // per epilogue warp: two 32 x 32 bf16 staging buffers
constexpr int kI8Group = 8;            // token tiles per raster group

__host__ __device__ constexpr int i8_stage_bytes(int fn) { return 128 * 128 + fn * 64; }
__host__ __device__ constexpr int i8_stages(int fn) {
  return kI8Ring / i8_stage_bytes(fn) < kI8MaxStages ? kI8Ring / i8_stage_bytes(fn) : kI8MaxStages;
}
__host__ __device__ constexpr int i8_smem_bytes() { return kI8Ring + kI8EpiWarps * kI8Stage + 1024 + 256; }

__device__ __forceinline__ void i8_tile_coords(const I8Params& p, int T, int& tt, int& ft) {
  const int per_group = kI8Group * p.n_ftiles;
  const int g = T / per_group;
  const int first = g * kI8Group;
  const int gsize = min(kI8Group, p.n_ttiles - first);
  const int idx = T - g * per_group;
  ft = idx / gsize;
  tt = first + idx % gsize;
}

// A tile is 256 tokens x fn features of one CTA pair: each CTA stages its 128
// token rows and its fn / 2 feature rows per 128-deep K step and holds the
// accumulator of its tokens x all fn features, twice, so that a tile's
// epilogue runs under the next tile's products.  Warps: 0 TMA producer, 1
// MMA issuer (leader) and TMEM allocator, 2-9 epilogue (lane quadrant
// warp % 4; two warps share a quadrant and take alternate 32-column chunks).
template <int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    ll_i8_kernel(const __grid_constant__ I8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align1024(smem_raw);
  uint8_t* epi = ring + kI8Ring;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + kI8EpiWarps * kI8Stage);  // leader: both CTAs' loads landed
  uint64_t* empty = full + kI8MaxStages;                                      // both: the MMAs are done with the slot
  uint64_t* tfull = empty + kI8MaxStages;                                     // both: accumulator buffer ready
  uint64_t* tempty = tfull + 2;                                               // leader: both CTAs' epilogues done
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int fn = p.fn;
  const int sb = i8_stage_bytes(fn);
  const int ns = i8_stages(fn);
  const int nS = (p.K + 127) / 128;  // K steps of 128 (a step past K loads as zeros)
  const int tiles = p.n_ttiles * p.n_ftiles;
  const int cid = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kI8MaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kI8EpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_x);
    tma_prefetch_desc(&p.tm_w);
    tma_prefetch_desc(&p.tm_y);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tbase = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
      int slot = 0;
      uint32_t ph = 0;
      bool ok = !p.withhold, issued = false;
      // The weight rows of the ring's first lap come before the wait.
      const int lap = min(ns, nS);
      if (ok) {
        int tt, ft;
        i8_tile_coords(p, cid, tt, ft);
        for (int s = 0; s < lap; ++s) {
          if (leader) mbar_arrive_expect_tx(&full[s], 2u * sb);
          tma_load_2d_pair(ring + s * sb + 16384, &p.tm_w, full0 + 8u * s, s * 128, ft * fn + (fn / 2) * static_cast<int>(rank));
        }
        issued = true;
      }
      pdl_wait_primary();
      for (int T = cid; T < tiles && ok; T += pairs) {
        int tt, ft;
        i8_tile_coords(p, T, tt, ft);
        const int t0 = tt * 256 + 128 * static_cast<int>(rank);
        const int f0 = ft * fn + (fn / 2) * static_cast<int>(rank);
        for (int s = 0; s < nS; ++s) {
          const bool first = T == cid && s < lap;
          const uint32_t bar = full0 + 8u * slot;
          uint8_t* dst = ring + slot * sb;
          if (!first) {
            if (!mbar_wait(&empty[slot], ph ^ 1, p.watch, kErrTimeoutProducer)) { ok = false; break; }
            if (leader) mbar_arrive_expect_tx(&full[slot], 2u * sb);
            tma_load_2d_pair(dst + 16384, &p.tm_w, bar, s * 128, f0);
          }
          tma_load_2d_pair(dst, &p.tm_x, bar, s * 128, t0);
          if (++slot == ns) { slot = 0; ph ^= 1; }
        }
      }
      if (!ok && issued) {
        // Loads already issued must land before the CTA exits; they
        // complete on leader barriers whose other arrivals may never come
        // now, so wait a bounded settle time far above any load latency.
        const uint64_t c0 = clock_cycles();
        while (clock_cycles() - c0 < 400000ull) {  // >= 200 us at any clock up to 2 GHz
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // --------------------------------------------- MMA issuer (leader)
      pdl_wait_primary();
      const uint32_t id = idesc_i8(256, fn);
      int slot = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int T = cid; T < tiles && ok; T += pairs, ++it) {
        const int buf = it & 1;
        if (!mbar_wait_cl(&tempty[buf], ((it >> 1) & 1) ^ 1, p.watch, kErrTimeoutMma)) break;
        tc_fence_after();
        const uint32_t d = tbase + 256u * buf;
        for (int s = 0; s < nS; ++s) {
          if (!mbar_wait_cl(&full[slot], ph, p.watch, kErrTimeoutMma)) { ok = false; break; }
          tc_fence_after();
          const uint32_t base = smem_u32(ring + slot * sb);
          const uint64_t dx = sdesc_kmajor_sw128(base);
          const uint64_t dw = sdesc_kmajor_sw128(base + 16384);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_i8_pair(d, dx + 2 * kk, dw + 2 * kk, id, (s | kk) != 0 ? 1u : 0u);
          tc_commit_pair(&empty[slot], 0x3);
          if (++slot == ns) { slot = 0; ph ^= 1; }
        }
        if (ok) tc_commit_pair(&tfull[buf], 0x3);
      }
      // No MMA may still run when TMEM is released.
      tc_commit_pair(drain, 0x1);
      mbar_wait_drain(drain, 0, p.watch);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // TMEM lane = token row of this CTA; column = feature of the tile.
    pdl_wait_primary();
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = epi + (warp - 2) * kI8Stage;
    const uint32_t tl = tbase + ((32u * q) << 16);
    const uint32_t tempty_leader = mapa_shared(smem_u32(&tempty[0]), 0);
    const int sw = (lane >> 1) & 3;  // 64-byte swizzle phase of this lane's staging row
    int it = 0, eb = 0;
    for (int T = cid; T < tiles; T += pairs, ++it) {
      int tt, ft;
      i8_tile_coords(p, T, tt, ft);
      const int buf = it & 1;
      const int trow = tt * 256 + 128 * static_cast<int>(rank) + 32 * q;
      const int tok = trow + lane;
      const float sm = tok < p.M ? __ldg(p.sx + tok) : 0.f;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], (it >> 1) & 1, p.watch, kErrTimeoutEpilogue))) break;
      tc_fence_after();
      const uint32_t acc = tl + 256u * buf;
      for (int c = half; c < fn / 32; c += 2) {
        const int f = ft * fn + 32 * c;
        uint32_t v[32];
        tmem_ld32_wait(acc + 32u * c, v);
        const float4* sb4 = p.sb + f / 2;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = i8_out2<kAct>(static_cast<int>(v[2 * i]), static_cast<int>(v[2 * i + 1]), sm, __ldg(sb4 + i));
        if (lane == 0) tma_store_wait_read<1>();
        __syncwarp();
        uint8_t* st = stg + eb * (32 * 64);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(st + lane * 64 + 16 * (j ^ sw)) =
              make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (trow < p.M && f < p.N) tma_store_2d(&p.tm_y, st, f, trow);
          tma_store_commit();
        }
        eb ^= 1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(&tempty[buf]);
        else
          mbar_arrive_cluster(tempty_leader + 8u * buf);
      }
    }
    if (lane == 0) tma_store_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's MMAs and epilogues are done with both TMEMs
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

// ============================================ few tokens: streaming the weight
struct I8StreamParams {
  CUtensorMap tm_x;  // s8 xq [M, K] box {128, Mt},  128B swizzle
  CUtensorMap tm_w;  // s8 wq [N, K] box {128, 128}, 128B swizzle
  const float* sx;   // [M]
  const float4* sb;  // [N rounded up / 2] (scale, scale, bias, bias) of two features
  uint16_t* y;       // [M, N] bf16 bits
  int M, N, K;
  int Mt;            // MMA N: tokens padded to a multiple of 16, 16..256
  int tmem_cols;     // power of two >= Mt, at least 32
  int splits;        // CTAs of a cluster that share a tile's K steps
  int steps;         // K steps of 128 per split
  int withhold;
  Watch watch;
};

constexpr int kIsThreads = 192;  // 0 TMA producer, 1 MMA issuer and TMEM allocator, 2-5 epilogue
constexpr int kIsRing = 208 * 1024;
constexpr int kIsMaxStages = 12;
constexpr int kIsMaxSplit = 8;

__host__ __device__ constexpr int is_stage_bytes(int Mt) { return 16384 + Mt * 128; }
__host__ __device__ constexpr int is_stages(int Mt) {
  return kIsRing / is_stage_bytes(Mt) < kIsMaxStages ? kIsRing / is_stage_bytes(Mt) : kIsMaxStages;
}
__host__ __device__ constexpr int is_smem_bytes(int Mt) { return is_stages(Mt) * is_stage_bytes(Mt) + 1024 + 256; }

// One CTA (or a cluster that splits K) per tile of 128 features x all tokens:
// the weight is read once from HBM, features on the MMA's M side, tokens on
// its N side.  The int32 sums go through shared memory ([token][feature]), and
// the CTAs of a cluster add them over distributed shared memory, each for
// every splits-th token.
template <int kAct>
__global__ void __launch_bounds__(kIsThreads, 1) ll_i8_stream_kernel(const __grid_constant__ I8StreamParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align1024(smem_raw);
  const int sb = is_stage_bytes(p.Mt), ns = is_stages(p.Mt);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + ns * sb);
  uint64_t* empty = full + kIsMaxStages;
  uint64_t* acc_full = empty + kIsMaxStages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int f0 = blockIdx.x * 128;
  const int z = blockIdx.y;  // split of K = rank in the cluster
  const int s0 = z * p.steps;
  const int n = min((p.K + 127) / 128 - s0, p.steps);  // K steps of this CTA (>= 1 by the plan)

  if (threadIdx.x == 0) {
    for (int s = 0; s < ns; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    // The weight of the ring's first lap: the layer's own memory.
    if (!p.withhold)
      for (int i = 0; i < min(ns, n); ++i) {
        mbar_arrive_expect_tx(&full[i], sb);
        tma_load_2d(ring + i * sb, &p.tm_w, &full[i], (s0 + i) * 128, f0);
      }
    tma_prefetch_desc(&p.tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tbase = *tmem_slot;
  bool ok = true;
  pdl_wait_primary();

  if (warp == 0) {
    if (lane == 0 && !p.withhold) {
      for (int i = 0; i < min(ns, n); ++i) tma_load_2d(ring + i * sb + 16384, &p.tm_x, &full[i], (s0 + i) * 128, 0);
      int slot = 0, i = ns;
      uint32_t ph = 0;
      for (; i < n; ++i) {
        if (!mbar_wait(&empty[slot], ph, p.watch, kErrTimeoutProducer)) { ok = false; break; }
        mbar_arrive_expect_tx(&full[slot], sb);
        tma_load_2d(ring + slot * sb, &p.tm_w, &full[slot], (s0 + i) * 128, f0);
        tma_load_2d(ring + slot * sb + 16384, &p.tm_x, &full[slot], (s0 + i) * 128, 0);
        if (++slot == ns) { slot = 0; ph ^= 1; }
      }
      if (!ok)  // let every load already issued land before the CTA can exit
        for (int j = max(0, i - ns); j < i; ++j) mbar_wait_drain(&full[j % ns], (j / ns) & 1, p.watch);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id = idesc_i8(128, p.Mt);
      int slot = 0;
      uint32_t ph = 0;
      for (int i = 0; i < n; ++i) {
        if (!mbar_wait(&full[slot], ph, p.watch, kErrTimeoutMma)) break;
        tc_fence_after();
        const uint32_t base = smem_u32(ring + slot * sb);
        const uint64_t dw = sdesc_kmajor_sw128(base);
        const uint64_t dx = sdesc_kmajor_sw128(base + 16384);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_i8(tbase, dw + 2 * kk, dx + 2 * kk, id, (i | kk) != 0 ? 1u : 0u);
        tc_commit(&empty[slot]);
        if (++slot == ns) { slot = 0; ph ^= 1; }
        if (i + 1 == n) tc_commit(acc_full);
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0, p.watch);
    }
  } else {
    // The sums as [token][feature] in the ring, which is idle once the last
    // MMA is done: a warp's lanes are 32 features of one token.
    const int q = warp & 3;
    int* part = reinterpret_cast<int*>(ring) + 32 * q + lane;
    if (__all_sync(0xffffffffu, mbar_wait(acc_full, 0, p.watch, kErrTimeoutEpilogue))) {
      tc_fence_after();
      for (int c = 0; c < p.Mt; c += 16) {
        uint32_t v[16];
        tmem_ld16_wait(tbase + ((32u * q) << 16) + c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * 128] = static_cast<int>(v[i]);
      }
    } else {
      ok = false;
    }
  }
  tc_fence_before();
  ok = __syncthreads_and(ok);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, p.tmem_cols);
  }
  // After a timeout the sums are incomplete; the CTA still takes part in both
  // cluster barriers.
  if (p.splits > 1) cluster_sync();
  const uint32_t part = smem_u32(ring);
  for (int i = threadIdx.x; ok && i < ((p.M - z + p.splits - 1) / p.splits) * 64; i += kIsThreads) {
    const int m = z + (i >> 6) * p.splits, c = (i & 63) * 2;
    if (f0 + c >= p.N) continue;
    const uint32_t off = part + static_cast<uint32_t>((m * 128 + c) * 4);
    int2 acc = make_int2(0, 0);
    if (p.splits == 1) {
      acc = *reinterpret_cast<const int2*>(ring + (m * 128 + c) * 4);
    } else {
#pragma unroll
      for (int r = 0; r < kIsMaxSplit; ++r)
        if (r < p.splits) {
          const int2 v = ld_shared_cluster_i2(mapa_shared(off, static_cast<uint32_t>(r)));
          acc.x += v.x;
          acc.y += v.y;
        }
    }
    *reinterpret_cast<uint32_t*>(p.y + static_cast<size_t>(m) * p.N + f0 + c) =
        i8_out2<kAct>(acc.x, acc.y, __ldg(p.sx + m), __ldg(p.sb + (f0 + c) / 2));
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync();  // no CTA leaves while a peer still reads its sums
}

// (scale, scale, bias, bias) of two features as the epilogues read them, zeros
// behind the last feature (a tile may end there).
__global__ void ll_i8_scale_bias_kernel(const float* __restrict__ scale, const uint16_t* __restrict__ bias,
                                        float4* __restrict__ sb, int N, int N_pad) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < N_pad / 2; i += gridDim.x * blockDim.x) {
    const bool in = 2 * i < N;  // N is even
    const float2 s = in ? make_float2(scale[2 * i], scale[2 * i + 1]) : make_float2(0.f, 0.f);
    sb[i] = in && bias ? make_float4(s.x, s.y, bf16_bits_to_float(bias[2 * i]), bf16_bits_to_float(bias[2 * i + 1]))
                       : make_float4(s.x, s.y, 0.f, 0.f);
  }
}

}  // namespace llk
