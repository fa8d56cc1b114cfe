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
#include "ptx_i8.cuh"

namespace llk {

constexpr int kI8MaxK = 131056;

// A time far above any load's or MMA's latency, that a CTA's own ones in flight
// get to complete after an error, whatever the limit of the waits.
constexpr uint64_t kI8SettleCycles = 400000;  // >= 200 us at any clock up to 2 GHz
__device__ __forceinline__ void i8_settle() {
  const uint64_t c0 = clock_cycles();
  while (clock_cycles() - c0 < kI8SettleCycles) {
  }
}
// The wait for MMAs or loads in flight, on the barrier that they complete on.
__device__ __forceinline__ void i8_drain(uint64_t* bar, uint32_t parity, const Watch& w) {
  mbar_wait_drain(bar, parity, Watch{w.status, max(w.timeout_ns, kI8SettleCycles / 2)});
}

// Two outputs from their sums: scaled by their tokens' scales sm, then s =
// (scale, scale, bias, bias) of their features.  The sum takes one scale after
// the other, as the formula's factors may be far from 1 where their product with
// it is not, and the token's first in every kernel, so that a token's outputs
// do not depend on the batch (and so the kernel) that it comes in.  GELU:
// v / 2 (1 + tanh(z)) = v / (1 + exp(-2 z)), z = sqrt(2 / pi) (v + 0.044715 v^3);
// exp(-2 z) as a power of two: -2 z log2(e) = v (-2.3022082 - 0.10294324 v^2).
template <int kAct>
__device__ __forceinline__ uint32_t i8_out2(int a0, int a1, float2 sm, const float4& s) {
  float2 v = fma2(mul2(make_float2(static_cast<float>(a0), static_cast<float>(a1)), sm), make_float2(s.x, s.y),
                  make_float2(s.z, s.w));
  if constexpr (kAct == kActGelu) {
    const float2 t = mul2(v, fma2(mul2(v, v), make_float2(-0.10294324f, -0.10294324f),
                                  make_float2(-2.3022082f, -2.3022082f)));
    v = mul2(v, make_float2(rcp(1.f + ex2(t.x)), rcp(1.f + ex2(t.y))));
  }
  return pack_bf16x2(v.x, v.y);
}

// Scales of the 16 tokens from m0 on (0 behind the last).
__device__ __forceinline__ void i8_token_scales(float (&v)[16], const float* sx, int m0, int M) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = 0.f;
    if (m0 + i < M) v[i] = ld_ahead(sx + m0 + i);
  }
}

// Outputs of one feature (this lane's; s, b its scale and bias) for 16 tokens
// whose scales are sm, into a staging tile [token][32 features]: lanes of
// neighbouring features swap halves, so that each writes one token's pair.
template <int kAct>
__device__ __forceinline__ void i8_stage_tokens(const uint32_t (&v)[16], const float (&sm)[16], float s, float b,
                                                uint8_t* tile, int lane) {
  uint32_t* d = reinterpret_cast<uint32_t*>(tile + (lane & 1) * 64) + lane / 2;
  const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
  const float4 sb = make_float4(s, s, b, b);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const uint32_t w =
        i8_out2<kAct>(static_cast<int>(v[i]), static_cast<int>(v[i + 1]), make_float2(sm[i], sm[i + 1]), sb);
    d[16 * i] = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), sel);
  }
}

// The same for the 16 tokens from m0 on, straight to y (few tokens, where the
// staging's round trip would show): 64 bytes of a token's row per warp.
template <int kAct>
__device__ __forceinline__ void i8_store_tokens(const uint32_t (&v)[16], const float (&sm)[16], int m0, int M, int N,
                                                int f, float s, float b, uint16_t* __restrict__ y) {
  uint16_t* d = y + static_cast<size_t>(m0) * N + f;
  const float4 sb = make_float4(s, s, b, b);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const uint32_t w =
        i8_out2<kAct>(static_cast<int>(v[i]), static_cast<int>(v[i + 1]), make_float2(sm[i], sm[i + 1]), sb);
    if (f < N && m0 + i < M) d[static_cast<size_t>(i) * N] = static_cast<uint16_t>(w);
    if (f < N && m0 + i + 1 < M) d[static_cast<size_t>(i + 1) * N] = static_cast<uint16_t>(w >> 16);
  }
}

// ==================================================== many tokens: CTA pairs
//
// A tile is 256 rows of one operand (a) x up to 256 of the other (b), of one
// CTA pair: each CTA stages its 128 rows of a and half of b's per 128-deep K
// step and holds the accumulator of its rows of a x all of b's, twice, so that a
// tile's epilogue runs under the next tile's products.  kSwap = false: a is the
// tokens, b the features; a thread of the epilogue owns a token, and the outputs
// go through shared memory and TMA stores.  kSwap = true: a is the features, b
// the tokens (batches whose tokens would fill tiles of 256 badly); a thread
// owns a feature.
struct I8Params {
  CUtensorMap tm_x;  // s8 xq [M, K]  box {128, rows}, 128B swizzle
  CUtensorMap tm_w;  // s8 weight panels [K / 128][N][128]  box {128, rows, 1}, 128B swizzle
  CUtensorMap tm_y;  // bf16 y [M, N] box {32, 32}, 64B swizzle, or {32, 16} without (kSwap)
  const float* sx;       // [M]
  const float4* sb;      // [N rounded up / 2] (scale, scale, bias, bias) of two features
  int M, N, K;
  int na, nb;            // tiles of a and b
  int w;                 // rows of b per tile: a multiple of 32, 64..256
  int withhold;          // debug: the producers issue nothing, so every consumer's wait runs out
  Watch watch;
};

constexpr int kI8Ring = 192 * 1024;
constexpr int kI8MaxStages = 9;
constexpr int kI8EpiWarps = 8;
constexpr int kI8Threads = 32 * (2 + kI8EpiWarps);
constexpr int kI8Stage = 2 * 32 * 64;  // per epilogue warp: two 32 x 32 bf16 staging buffers
constexpr int kI8Group = 8;            // tiles of a per raster group

// A ring slot: 128 rows of a and w / 2 of b, 128 codes each.
__host__ __device__ constexpr int i8_slot_bytes(int w) { return 16384 + w * 64; }
__host__ __device__ constexpr int i8_stages(int w) {
  return kI8Ring / i8_slot_bytes(w) < kI8MaxStages ? kI8Ring / i8_slot_bytes(w) : kI8MaxStages;
}
__host__ __device__ constexpr int i8_smem_bytes() { return kI8Ring + kI8EpiWarps * kI8Stage + 1024 + 256; }

// Groups of kI8Group tiles of a, a fastest: the tiles in flight share their
// rows of both operands in L2.
__device__ __forceinline__ void i8_tile_coords(const I8Params& p, int T, int& ta, int& tb) {
  const int per_group = kI8Group * p.nb;
  const int g = T / per_group;
  const int first = g * kI8Group;
  const int gsize = min(kI8Group, p.na - first);
  const int idx = T - g * per_group;
  tb = idx / gsize;
  ta = first + idx % gsize;
}

// Warps: 0 TMA producer, 1 MMA issuer (leader) and TMEM allocator, 2-9
// epilogue (lane quadrant warp % 4; two warps share a quadrant and take
// alternate chunks of columns).
template <int kAct, bool kSwap>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    ll_i8_kernel(const __grid_constant__ I8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align1024(smem_raw);
  uint8_t* epi = ring + kI8Ring;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + kI8EpiWarps * kI8Stage);  // leader: both CTAs' loads landed
  uint64_t* empty = full + kI8MaxStages;                                         // both: the MMAs are done with the slot
  uint64_t* tfull = empty + kI8MaxStages;                                        // both: accumulator buffer ready
  uint64_t* tempty = tfull + 2;                                               // leader: both CTAs' epilogues done
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int nS = (p.K + 127) / 128;  // K steps of 128 (a step past K loads as zeros)

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
  const int pid = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const int tiles = p.na * p.nb;
  const int w = p.w, slot_bytes = i8_slot_bytes(w), stages = i8_stages(w);
  bool done = true;  // no wait of this thread ran out

  if (warp == 0) {
    // ------------------------------------------- TMA producer (both CTAs)
    const uint32_t one = elect_one();
    const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0), ring0 = smem_u32(ring);
    int slot = 0, ta, tb;
    uint32_t ph = 0;
    bool ok = !p.withhold;
    const int lap = min(stages, nS);
    auto load_x = [&](int slot, int s) {
      if (kSwap)
        load_2d_pair_one(ring0 + slot * slot_bytes + 16384, &p.tm_x, full0 + 8u * slot, s * 128, tb * w + (w / 2) * rank, one);
      else
        load_2d_pair_one(ring0 + slot * slot_bytes, &p.tm_x, full0 + 8u * slot, s * 128, ta * 256 + 128 * rank, one);
    };
    auto load_w = [&](int slot, int s) {
      if (leader) expect_one(&full[slot], 2u * slot_bytes, one);
      if (kSwap)
        load_3d_pair_one(ring0 + slot * slot_bytes, &p.tm_w, full0 + 8u * slot, 0, ta * 256 + 128 * rank, s, one);
      else
        load_3d_pair_one(ring0 + slot * slot_bytes + 16384, &p.tm_w, full0 + 8u * slot, 0, tb * w + (w / 2) * rank, s, one);
    };
    if (ok) {
      // The weight rows of the ring's first lap come before the wait.
      i8_tile_coords(p, pid, ta, tb);
      for (int s = 0; s < lap; ++s) load_w(s, s);
    }
    pdl_wait_primary();
    for (int T = pid; T < tiles && ok; T += pairs) {
      i8_tile_coords(p, T, ta, tb);
      for (int s = 0; s < nS; ++s) {
        if (T != pid || s >= lap) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ph ^ 1, p.watch, kErrTimeoutProducer));
          if (!ok) break;
          load_w(slot, s);
        }
        load_x(slot, s);
        if (++slot == stages) { slot = 0; ph ^= 1; }
      }
    }
    done = ok;
  } else if (warp == 1) {
    if (leader) {
      // --------------------------------------------- MMA issuer (leader)
      pdl_wait_primary();
      const uint32_t one = elect_one();
      const uint32_t id = idesc_i8(256, w);
      const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(ring)), db0 = sdesc_kmajor_sw128(smem_u32(ring) + 16384);
      int slot = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int T = pid; T < tiles && ok; T += pairs, ++it) {
        const int buf = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_cl(&tempty[buf], ((it >> 1) & 1) ^ 1, p.watch, kErrTimeoutMma));
        const uint32_t d = tbase + 256u * buf;
        for (int s = 0; s < nS && ok; ++s) {
          ok = __all_sync(0xffffffffu, mbar_wait_cl(&full[slot], ph, p.watch, kErrTimeoutMma));
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = da0 + static_cast<uint64_t>(slot * (slot_bytes >> 4));
          const uint64_t db = db0 + static_cast<uint64_t>(slot * (slot_bytes >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_i8_pair(d, da + 2 * kk, db + 2 * kk, id, (s | kk) != 0 ? 1u : 0u, one);
          commit_one_pair(&empty[slot], 0x3, one);
          if (++slot == stages) { slot = 0; ph ^= 1; }
        }
        if (ok) commit_one_pair(&tfull[buf], 0x3, one);
      }
      // No MMA may still run when TMEM is released.
      commit_one_pair(drain, 0x1, one);
      if (one) i8_drain(drain, 0, p.watch);
      __syncwarp();
      done = ok;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // TMEM lane = row of a of this CTA; column = row of b.
    pdl_wait_primary();
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = epi + (warp - 2) * kI8Stage;
    const uint32_t tl = tbase + ((32u * q) << 16);
    const uint32_t tempty_leader = mapa_shared(smem_u32(&tempty[0]), 0);
    const int sw = (lane >> 1) & 3;  // 64-byte swizzle phase of this lane's staging row
    int it = 0, eb = 0;
    for (int T = pid; T < tiles; T += pairs, ++it) {
      int ta, tb;
      i8_tile_coords(p, T, ta, tb);
      const int b0 = tb * w, buf = it & 1;
      const int row0 = ta * 256 + 128 * rank + 32 * q;
      const int row = row0 + lane;
      float sm = 0.f, bias = 0.f;  // kSwap: scale and bias of the feature; else the token's scale
      if (kSwap) {
        if (row < p.N) {
          const float4 s2 = __ldg(p.sb + row / 2);
          sm = row & 1 ? s2.y : s2.x;
          bias = row & 1 ? s2.w : s2.z;
        }
      } else if (row < p.M) {
        sm = ld_ahead(p.sx + row);
      }
      float4 sb[16];  // of the next chunk's features
      auto load_sb = [&](int c) {
        const float4* sb4 = p.sb + (b0 + c) / 2;
#pragma unroll
        for (int i = 0; i < 16; ++i) sb[i] = ldg_ahead(sb4 + i);
      };
      float sx[16];  // kSwap: of the next chunk's tokens
      if (kSwap)
        i8_token_scales(sx, p.sx, b0 + 16 * half, p.M);
      else if (32 * half < w)
        load_sb(32 * half);
      done = __all_sync(0xffffffffu, mbar_wait(&tfull[buf], (it >> 1) & 1, p.watch, kErrTimeoutEpilogue));
      if (!done) break;
      tc_fence_after();
      const uint32_t acc = tl + 256u * buf;
      if constexpr (kSwap) {
        for (int c = 16 * half; c < w && b0 + c < p.M; c += 32) {
          uint32_t v[16];
          tmem_ld16_wait(acc + c, v);
          if (lane == 0) tma_store_wait_read<1>();
          __syncwarp();
          uint8_t* st = stg + eb * (16 * 64);
          i8_stage_tokens<kAct>(v, sx, sm, bias, st, lane);
          fence_proxy_async_smem();
          __syncwarp();
          store_2d_one(&p.tm_y, smem_u32(st), row0, b0 + c, row0 < p.N, lane == 0);
          if (c + 32 < w) i8_token_scales(sx, p.sx, b0 + c + 32, p.M);
          eb ^= 1;
        }
      } else {
        for (int c = 32 * half; c < w; c += 64) {
          const int f = b0 + c;
          uint32_t v[32];
          tmem_ld32_wait(acc + c, v);
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = i8_out2<kAct>(static_cast<int>(v[2 * i]), static_cast<int>(v[2 * i + 1]), make_float2(sm, sm), sb[i]);
          if (c + 64 < w) load_sb(c + 64);
          if (lane == 0) tma_store_wait_read<1>();
          __syncwarp();
          uint8_t* st = stg + eb * (32 * 64);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(st + lane * 64 + 16 * (j ^ sw)) =
                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          store_2d_one(&p.tm_y, smem_u32(st), f, row0, row0 < p.M && f < p.N, lane == 0);
          eb ^= 1;
        }
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
  // Where a wait ran out, loads that the producer has issued may be in flight,
  // and the barriers of the leader that they complete on never be waited for:
  // they must land before the CTA exits.
  if (!__syncthreads_and(done) && !p.withhold) i8_settle();
  cluster_sync();  // the pair's MMAs and epilogues are done with both TMEMs
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

// ============================================ few tokens: streaming the weight
struct I8StreamParams {
  CUtensorMap tm_x;  // s8 xq [M, K] box {128, Mt},  128B swizzle
  CUtensorMap tm_w;  // s8 weight panels [K / 128][N][128] box {128, 128, 1}, 128B swizzle
  CUtensorMap tm_y;  // bf16 y [M, N] box {32, 16} (16 epilogue warps)
  const float* sx;   // [M]
  const float4* sb;  // [N rounded up / 2] (scale, scale, bias, bias) of two features
  uint16_t* y;       // [M, N] bf16 bits
  int M, N, K;
  int Mt;            // MMA N: tokens padded to a multiple of 16, 16..256
  int tmem_cols;     // power of two >= Mt, at least 32
  int splits;        // CTAs of a cluster that share a tile's K steps
  int steps;         // K steps of 128 per split
  int stages;        // ring slots
  int withhold;
  Watch watch;
};

// Warps: 0 TMA producer, 1 MMA issuer and TMEM allocator, the rest epilogue.
__host__ __device__ constexpr int is_threads(int epi_warps) { return 32 * (2 + epi_warps); }
constexpr int kIsMaxStages = 12;
constexpr int kIsMaxSplit = 8;
// The small ring leaves room for a second CTA on the SM: the next kernel's,
// whose weight loads then start under this kernel's end.
constexpr int kIsRingSmall = 108 * 1024, kIsRingLarge = 208 * 1024;

__host__ __device__ constexpr int is_stage_bytes(int Mt) { return 16384 + Mt * 128; }
__host__ __device__ constexpr int is_stages(int Mt, int ring) {
  return ring / is_stage_bytes(Mt) < kIsMaxStages ? ring / is_stage_bytes(Mt) : kIsMaxStages;
}
__host__ __device__ constexpr int is_smem_bytes(int Mt, int ring) {
  return is_stages(Mt, ring) * is_stage_bytes(Mt) + 1024 + 256;
}

// One CTA (or a cluster that splits K) per tile of 128 features x all tokens:
// the weight is read once from HBM, features on the MMA's M side, tokens on
// its N side.  Without a split the outputs go straight from TMEM to global
// memory (a warp's lanes are 32 features of a token), or through staging tiles
// and TMA stores by 16 epilogue warps, a launch for more than 32 tokens.  With one the int32 sums
// go through shared memory ([token][feature]), and the CTAs of the cluster add
// them over distributed shared memory, each for every splits-th token.
//
// 56 registers with 16 epilogue warps (8 have room for 102), so that the next
// kernel's CTA fits beside one of the small ring.
template <int kAct, int kEpiWarps>
__global__ void __launch_bounds__(is_threads(kEpiWarps), kEpiWarps > 8 ? 2 : 1)
    ll_i8_stream_kernel(const __grid_constant__ I8StreamParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align1024(smem_raw);
  const int sb = is_stage_bytes(p.Mt), ns = p.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + ns * sb);
  uint64_t* empty = full + kIsMaxStages;
  uint64_t* acc_full = empty + kIsMaxStages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int f0 = blockIdx.x * 128;
  const int z = blockIdx.y;  // split of K = rank in the cluster
  const int s0 = z * p.steps;
  constexpr bool kStaged = kEpiWarps > 8;  // outputs go through staging tiles; no split then
  const bool split = !kStaged && p.splits > 1;
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
        tma_load_3d(ring + i * sb, &p.tm_w, &full[i], 0, f0, s0 + i);
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
  int issued = 0;  // K steps whose loads warp 0 has issued
  pdl_wait_primary();

  if (warp == 0) {
    if (!p.withhold) {
      const uint32_t one = elect_one();
      const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(&full[0]);
      for (int i = 0; i < min(ns, n); ++i)
        load_2d_one(ring0 + i * sb + 16384, &p.tm_x, full0 + 8u * i, (s0 + i) * 128, 0, one);
      int slot = 0, i = ns;
      uint32_t ph = 0;
      for (; i < n; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ph, p.watch, kErrTimeoutProducer));
        if (!ok) break;
        expect_one(&full[slot], sb, one);
        load_3d_one(ring0 + slot * sb, &p.tm_w, full0 + 8u * slot, 0, f0, s0 + i, one);
        load_2d_one(ring0 + slot * sb + 16384, &p.tm_x, full0 + 8u * slot, (s0 + i) * 128, 0, one);
        if (++slot == ns) { slot = 0; ph ^= 1; }
      }
      issued = min(i, n);
    }
  } else if (warp == 1) {
    const uint32_t one = elect_one();
    const uint32_t id = idesc_i8(128, p.Mt);
    const uint64_t dw0 = sdesc_kmajor_sw128(smem_u32(ring)), dx0 = sdesc_kmajor_sw128(smem_u32(ring) + 16384);
    int slot = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], ph, p.watch, kErrTimeoutMma));
      if (!ok) break;
      tc_fence_after();
      const uint64_t dw = dw0 + static_cast<uint64_t>(slot * (sb >> 4)), dx = dx0 + static_cast<uint64_t>(slot * (sb >> 4));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_i8(tbase, dw + 2 * kk, dx + 2 * kk, id, (i | kk) != 0 ? 1u : 0u, one);
      commit_one(&empty[slot], one);
      if (i + 1 == n) commit_one(acc_full, one);
      if (++slot == ns) { slot = 0; ph ^= 1; }
    }
    commit_one(drain, one);
    if (one) i8_drain(drain, 0, p.watch);
    __syncwarp();
  } else {
    // TMEM lane = feature, column = token; the warps of a lane quadrant take
    // turns at blocks of 16 tokens.
    constexpr int kTurn = 16 * kEpiWarps / 4;
    const int q = warp & 3, turn = (warp - 2) >> 2;
    const int f = f0 + 32 * q + lane;
    const float4 s2 = f < p.N ? __ldg(p.sb + f / 2) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float s = f & 1 ? s2.y : s2.x, b = f & 1 ? s2.w : s2.z;
    int* part = reinterpret_cast<int*>(ring) + 32 * q + lane;
    float sx[16];  // of the next block's tokens
    if (!split) i8_token_scales(sx, p.sx, 16 * turn, p.M);
    if (__all_sync(0xffffffffu, mbar_wait(acc_full, 0, p.watch, kErrTimeoutEpilogue))) {
      tc_fence_after();
      for (int c = 16 * turn; c < p.Mt; c += kTurn) {
        uint32_t v[16];
        tmem_ld16_wait(tbase + ((32u * q) << 16) + c, v);
        if (split) {
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * 128] = static_cast<int>(v[i]);
        } else if (!kStaged) {
          i8_store_tokens<kAct>(v, sx, c, p.M, p.N, f, s, b, p.y);
          i8_token_scales(sx, p.sx, c + kTurn, p.M);
        } else {
          if (lane == 0) tma_store_wait_read<1>();
          __syncwarp();
          uint8_t* st = ring + (2 * (warp - 2) + ((c / kTurn) & 1)) * (16 * 64);  // the MMAs are done with the ring
          i8_stage_tokens<kAct>(v, sx, s, b, st, lane);
          fence_proxy_async_smem();
          __syncwarp();
          store_2d_one(&p.tm_y, smem_u32(st), f0 + 32 * q, c, f0 + 32 * q < p.N && c < p.M, lane == 0);
          i8_token_scales(sx, p.sx, c + kTurn, p.M);
        }
      }
      if (kStaged && lane == 0) tma_store_wait<0>();
    } else {
      ok = false;
    }
  }
  tc_fence_before();
  ok = __syncthreads_and(ok);
  if (!ok && warp == 0)  // loads that are in flight must land before the CTA exits
    for (int j = max(0, issued - ns); j < issued; ++j) i8_drain(&full[j % ns], (j / ns) & 1, p.watch);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, p.tmem_cols);
  }
  if (!split) return;
  // After a timeout the sums are incomplete; the CTA still takes part in both
  // cluster barriers.
  cluster_sync();
  const int c = 4 * lane;  // a warp's lanes are a token's 128 features
  if (ok && f0 + c < p.N) {
    const float4 s0v = __ldg(p.sb + (f0 + c) / 2), s1v = __ldg(p.sb + (f0 + c) / 2 + 1);
    const uint32_t part = smem_u32(ring) + 4 * c;
    for (int m = z + warp * p.splits; m < p.M; m += (2 + kEpiWarps) * p.splits) {
      const float sx = ld_ahead(p.sx + m);
      const float2 sm = make_float2(sx, sx);
      int4 v[kIsMaxSplit];
#pragma unroll
      for (int r = 0; r < kIsMaxSplit; ++r)
        if (r < p.splits) v[r] = ld_shared_cluster_i4(mapa_shared(part + 512u * m, static_cast<uint32_t>(r)));
      int4 a = v[0];
#pragma unroll
      for (int r = 1; r < kIsMaxSplit; ++r)
        if (r < p.splits) {
          a.x += v[r].x;
          a.y += v[r].y;
          a.z += v[r].z;
          a.w += v[r].w;
        }
      *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(m) * p.N + f0 + c) =
          make_uint2(i8_out2<kAct>(a.x, a.y, sm, s0v), i8_out2<kAct>(a.z, a.w, sm, s1v));
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while a peer still reads its sums
}

// The weight as the kernels read it: panels of 128 codes of every row,
// [K / 128][N][128], so that a tile's load of one K step is one contiguous
// piece of memory; zeros behind K.
__global__ void ll_i8_panels_kernel(const int8_t* __restrict__ w, int8_t* __restrict__ panels, int N, int K) {
  const int nc = (K + 127) / 128 * 8;  // 16-byte chunks of a padded row
  const size_t total = static_cast<size_t>(N) * nc;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const int c = static_cast<int>(i % nc);
    const size_t n = i / nc;
    const uint4 v = 16 * c < K ? *reinterpret_cast<const uint4*>(w + n * K + 16 * c) : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(panels + (static_cast<size_t>(c / 8) * N + n) * 128 + 16 * (c % 8)) = v;
  }
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
