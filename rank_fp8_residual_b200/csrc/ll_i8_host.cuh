// Host side of the int8 operators of include/rank_fp8_residual.h: the row
// kernels (ll_rows_i8.cuh) and the int8 layer (ll_i8.cuh).  Included by
// ll_api.cu, whose helpers it uses.
#pragma once

#include <new>

#include "ll_i8.cuh"
#include "ll_rows_i8.cuh"

// The int8 layer.  Its forwards change nothing here, on the host or on the
// device (except the status word after a timeout), so they may run on any
// streams at once.
struct ll_i8_layer {
  int N = 0, K = 0, device = 0, num_sms = 0;
  bool ready = false;
  int8_t* W = nullptr;   // panels [K / 128][N][128]
  float4* sb = nullptr;  // [N_pad / 2] (scale, scale, bias, bias), zeros behind the last feature
  int N_pad = 0;         // room for a tile of 256 features that starts at the last one
  int* status = nullptr;
  CUtensorMap tm_w[7];   // maps of W with boxes of 32, 48 .. 128 rows (half of the pair kernel's widths)
  int clusters[llk::kIsMaxSplit + 1] = {};  // co-resident clusters of that many CTAs of the streaming kernel
  int pairs = 0;                            // co-resident CTA pairs of the pair kernel
  int epilogue = LL_EPILOGUE_NONE;
  int withhold = 0;
  uint64_t timeout_ns = 2000000000ull;
};

namespace {

int current_device_sms(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
    cudaGetLastError();
    return LL_ERR_CUDA;
  }
  return LL_OK;
}

// Makes a device current for a scope.
struct DeviceScope {
  int prev = -1;
  explicit DeviceScope(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess || prev == dev || cudaSetDevice(dev) != cudaSuccess) prev = -1;
  }
  ~DeviceScope() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

template <bool kNorm>
cudaError_t launch_rows_i8_as(const llk::RowsParams& p, int chunks, bool keep, const cudaLaunchConfig_t& cfg) {
  using namespace llk;
  switch (chunks) {
    case 1: return cudaLaunchKernelEx(&cfg, ll_rows_i8_kernel<1, kNorm, true>, p);
    case 2: return cudaLaunchKernelEx(&cfg, ll_rows_i8_kernel<2, kNorm, true>, p);
    case 4:
      if constexpr (kNorm)
        if (keep) return cudaLaunchKernelEx(&cfg, ll_rows_i8_kernel<4, true, true>, p);
      return cudaLaunchKernelEx(&cfg, ll_rows_i8_kernel<4, kNorm, false>, p);
    default:
      if constexpr (kNorm)
        if (keep) return cudaLaunchKernelEx(&cfg, ll_rows_i8_kernel<8, true, true>, p);
      return cudaLaunchKernelEx(&cfg, ll_rows_i8_kernel<8, kNorm, false>, p);
  }
}

int launch_rows_i8(const llk::RowsParams& p, bool norm, int sms, cudaStream_t st) {
  const int nv = p.K / 8;
  // Chunks of eight values per thread.  Few rows: as many threads as there
  // are (latency).  Many: four chunks, whose loads are in flight together.
  // Norm with residual, us with 1 / 2 / 4 chunks: 100 x 8192 2.8 / 3.2 / 3.2,
  // 400 x 4096 5.0 / 3.9 / 4.2, 3630 x 4096 29.2 / 19.9 / 18.0, 16384 x 4096
  // 118 / 78 / 69.  Eight where four would need more than 1024 threads.
  // Many long rows whose norm's u fits 256 threads by eight chunks take those
  // (us with 4 / 8: 4000 x 16384 68.8 / 68.7 and 47.5 / 42.7 without residual,
  // 4000 x 12288 56.0 / 54.2 and 41.4 / 39.1; but 400 x 16384 10.7 / 11.0), and
  // shorter ones without a residual: half as much to load beside the same
  // work, and half the warps to join (1400 x 8192 11.4 / 11.1, 16384 x 8192
  // 89.8 / 80.7, 5000 x 6144 23.0 / 22.5; but 16384 x 4096 41.0 / 42.3, and
  // with residual 16384 x 8192 134 / 137).
  int c = p.M <= 2 * sms ? 1 : (p.M <= 8 * sms && nv <= 512 ? 2 : 4);
  if (norm && c == 4 && p.M > 8 * sms && nv <= 2048 && nv > (p.residual ? 1024 : 640)) c = 8;
  while (c < 8 && nv > 1024 * c) c *= 2;
  while (c > 1 && nv <= 16 * c) c /= 2;
  const int threads = ((nv + c - 1) / c + 31) / 32 * 32;
  // Rows of one warp: four per block (16384 x 512 11.1 us, one per block 19.9).
  const int rows = threads == 32 && p.M > 2 * sms ? 4 : 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((static_cast<unsigned>(p.M) + rows - 1) / rows);
  cfg.blockDim = dim3(threads, rows);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool keep = threads <= llk::rows_max_threads(c, true);
  if ((norm ? launch_rows_i8_as<true>(p, c, keep, cfg) : launch_rows_i8_as<false>(p, c, false, cfg)) == cudaSuccess) return LL_OK;
  cudaGetLastError();
  return LL_ERR_CUDA;
}

using I8Fn = void (*)(llk::I8Params);
using I8StreamFn = void (*)(llk::I8StreamParams);
I8Fn kernel_i8(int epilogue, bool swap) {
  using namespace llk;
  if (epilogue == LL_EPILOGUE_GELU_TANH) return swap ? ll_i8_kernel<kActGelu, true> : ll_i8_kernel<kActGelu, false>;
  return swap ? ll_i8_kernel<kActNone, true> : ll_i8_kernel<kActNone, false>;
}
template <int kEpiWarps>
I8StreamFn kernel_i8_stream_as(int epilogue) {
  return epilogue == LL_EPILOGUE_GELU_TANH ? llk::ll_i8_stream_kernel<llk::kActGelu, kEpiWarps>
                                           : llk::ll_i8_stream_kernel<llk::kActNone, kEpiWarps>;
}
I8StreamFn kernel_i8_stream(int epilogue, int epi_warps) {
  return epi_warps == 16 ? kernel_i8_stream_as<16>(epilogue) : kernel_i8_stream_as<8>(epilogue);
}

// Per device: the kernels' shared-memory limits, and how many clusters of
// the streaming kernel fit at once.
bool setup_i8(ll_i8_layer* h) {
  using namespace llk;
  for (int e : {LL_EPILOGUE_NONE, LL_EPILOGUE_GELU_TANH})
    if (cudaFuncSetAttribute(kernel_i8(e, false), cudaFuncAttributeMaxDynamicSharedMemorySize, i8_smem_bytes()) != cudaSuccess ||
        cudaFuncSetAttribute(kernel_i8(e, true), cudaFuncAttributeMaxDynamicSharedMemorySize, i8_smem_bytes()) != cudaSuccess ||
        cudaFuncSetAttribute(kernel_i8_stream(e, 8), cudaFuncAttributeMaxDynamicSharedMemorySize, kIsRingLarge + 1280) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel_i8_stream(e, 16), cudaFuncAttributeMaxDynamicSharedMemorySize, kIsRingLarge + 1280) !=
            cudaSuccess)
      return false;
  for (int s = 2; s <= kIsMaxSplit; ++s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = static_cast<unsigned>(s);
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(h->num_sms, s);
    cfg.blockDim = dim3(is_threads(8));
    cfg.dynamicSmemBytes = kIsRingLarge + 1280;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&h->clusters[s], kernel_i8_stream(LL_EPILOGUE_NONE, 8), &cfg) != cudaSuccess)
      return false;
  }
  h->clusters[1] = h->num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(h->num_sms);
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = i8_smem_bytes();
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel_i8(LL_EPILOGUE_NONE, false), &cfg) != cudaSuccess || n < 1) return false;
  h->pairs = std::min(n, h->num_sms / 2);
  return true;
}

bool make_weight_maps(ll_i8_layer* h) {
  for (int i = 0; i < 7; ++i)
    if (!make_map3(&h->tm_w[i], h->W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 128, h->N, (h->K + 127) / 128, 128, 128ull * h->N,
                   128, 32 + 16 * i, 1, CU_TENSOR_MAP_SWIZZLE_128B))
      return false;
  return true;
}
const CUtensorMap& weight_map(const ll_i8_layer* h, int rows) { return h->tm_w[(rows - 32) / 16]; }

constexpr int kI8MaxRows = 0x7FFFFFFF - 511;  // of either operand: a tile's rows behind the last still count in an int
constexpr int kI8StreamMaxM = 256;  // the MMA's N

// What a forward of M tokens runs, and the model's cycles.  The model's rates
// are fitted to measured times (at about 1.75 GHz); it ranks plans and is not a
// prediction of the time:
//   a CTA's loads arrive at 66 bytes a cycle (w = 64, 128 and 256 of the pair
//   kernel: 310, 367 and 565 cycles per K step), the weight at 5.7 TB/s;
//   products of a 256 x w step take 2.2 w cycles (2 w alone);
//   start and end cost 5,000 (pair) or 5,560 (streaming), and the last tile's
//   epilogue 4,500 per 256 columns (10,000 with kSwap: its shuffles and scales
//   token by token, and what a choice against measured crossovers leaves open: over
//   some 150 sizes of up to 3630 tokens every plan that 11,000 chose otherwise
//   was slower, 100 x 1024 -> 28000 12.3 against 9.8 us) or 42 per token
//   (streaming), 5 % of which starts under the kernel before;
//   a streaming launch with 16 epilogue warps all but hides them (60 per token
//   above 25).
struct I8Plan {
  bool stream;
  int splits, steps;  // streaming: CTAs per tile and K steps of each
  bool swap;          // pairs: orientation, tiles of a and b, and b's width
  int na, nb, w;
  double cycles;
};

double i8_weight_cycles(const ll_i8_layer* h) { return static_cast<double>(h->N) * h->K * 3.07e-4; }

I8Plan i8_plan_pair(const ll_i8_layer* h, int M) {
  const int pairs = h->pairs;
  const double steps = (h->K + 127) / 128;
  I8Plan best{};
  best.cycles = -1;
  for (bool swap : {false, true}) {
    const int na = ((swap ? h->N : M) + 255) / 256, b = swap ? M : h->N;
    for (int w = 256; w >= 64; w -= 32) {
      const int nb = (b + w - 1) / w;
      const double waves = std::ceil(static_cast<double>(na) * nb / pairs);
      const double loop = waves * (steps * std::max(2.2 * w, (16384.0 + 64.0 * w) / 66.0) + 200.0);
      const double cycles = 5000.0 + std::max(loop, i8_weight_cycles(h)) + (swap ? 10000.0 : 4500.0) * w / 256;
      if (best.cycles < 0 || cycles < 0.98 * best.cycles) best = I8Plan{false, 0, 0, swap, na, nb, w, cycles};
    }
  }
  return best;
}

// Twice the epilogue warps, and outputs by staging tiles and TMA stores, where
// a launch without a split has more than 32 tokens (64 x 4096 -> 16384 13.9 ->
// 13.15 us, 80 x 8192 -> 8192 15.8 -> 15.7); with a split the warps only move
// sums (128 x 8192 -> 2048 8.4 -> 8.7).
bool i8_staged(int splits, int Mt) { return splits == 1 && Mt > 32; }

// The small ring where the next kernel's start under this one's end counts for
// more than loads in flight (us small / large: 1 x 4096 -> 4096 4.95 / 5.44, 32 x
// 4096 -> 4096 5.70 / 6.03; 64 x 8192 -> 2048 7.4 / 7.0, 64 x 4096 -> 16384 15.3 /
// 13.8; with four K steps or fewer they fit it anyway).  At least four slots: a
// split's sums (512 bytes per token) go where the ring was, and 4 (16384 +
// 128 Mt) >= 512 Mt.
bool is_small_ring(int steps, int Mt) {
  return llk::is_stages(Mt, llk::kIsRingSmall) >= 4 && (Mt <= 32 || steps <= 4);
}

I8Plan i8_plan_stream(const ll_i8_layer* h, int M) {
  const int tiles = (h->N + 127) / 128, steps = (h->K + 127) / 128, Mt = (M + 15) / 16 * 16;
  // As many CTAs as fit at once share the K steps of a tile.
  int s = 1;
  while (s < std::min(llk::kIsMaxSplit, steps) && tiles <= h->clusters[s + 1]) ++s;
  I8Plan p{};
  p.stream = true;
  p.steps = (steps + s - 1) / s;
  p.splits = (steps + p.steps - 1) / p.steps;
  const double waves = std::ceil(static_cast<double>(tiles) * p.splits / h->num_sms);
  const double step = (16384.0 + 128.0 * Mt) / 66.0, loop = std::max(waves * p.steps * step, i8_weight_cycles(h));
  if (!i8_staged(p.splits, Mt))
    p.cycles = 0.95 * (loop + 5560.0 + 42.0 * M);
  else if (waves == 1)
    p.cycles = loop + 60.0 * M - 1500.0;
  else  // one CTA per SM: its rounds follow one another (us, streaming / pair / swapped: 40 x 4096 -> 19000 22.7 / 22.3 /
        // 20.4, 64 x 1024 -> 28000 10.2 / 12.5 / 8.7, 64 x 128 -> 19000 3.6 / 6.3 / 4.8)
    p.cycles = 0.95 * std::max(waves * (p.steps * step + std::min(5800.0, 2000.0 + 450.0 * p.steps)),
                               i8_weight_cycles(h));
  return p;
}

// Measured (us, streaming / pair / swapped, the best width of each): 1024 ->
// 1024: M = 128 6.1 / 4.4 / 4.6; 4096 -> 4096: 64 7.8 / 9.6 / 8.8, 256 12.1 /
// 9.6 / 10.1; 4096 -> 16384: 96 13.8 / 16.5 / 14.7, 160 15.2 / 16.7 / 16.2, 200
// 17.9 / 17.3 / 18.1, 256 18.5 / 17.4 / 18.8; 1024 -> 16384: 128 6.8 / 9.0 / 8.4;
// 2048 -> 8192: 65 7.7 / 8.1 / 7.3; 8192 -> 8192: 100 16.1 / 16.8 / 16.0; 8192 ->
// 2048: 256 13.6 / 14.1 / 13.8.
I8Plan i8_plan(const ll_i8_layer* h, int M) {
  const I8Plan pair = i8_plan_pair(h, M);
  if (M > kI8StreamMaxM) return pair;
  const I8Plan stream = i8_plan_stream(h, M);
  return pair.cycles < stream.cycles ? pair : stream;
}

int launch_i8_stream(const ll_i8_layer* h, const I8Plan& plan, const void* codes, const float* scale, void* y, int M,
                     cudaStream_t st) {
  using namespace llk;
  I8StreamParams p;
  p.Mt = (M + 15) / 16 * 16;
  if (!make_map(&p.tm_x, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, M, h->K, h->K, 128, p.Mt, CU_TENSOR_MAP_SWIZZLE_128B))
    return LL_ERR_CUDA;
  p.tm_w = weight_map(h, 128);
  p.sx = scale;
  p.sb = h->sb;
  p.y = static_cast<uint16_t*>(y);
  p.M = M;
  p.N = h->N;
  p.K = h->K;
  p.tmem_cols = next_pow2_ge32(p.Mt);
  p.withhold = h->withhold;
  p.watch = Watch{h->status, h->timeout_ns};
  p.steps = plan.steps;
  p.splits = plan.splits;
  const int ring = is_small_ring(p.steps, p.Mt) ? kIsRingSmall : kIsRingLarge;
  p.stages = is_stages(p.Mt, ring);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = static_cast<unsigned>(p.splits);
  attr[1].val.clusterDim.z = 1;
  const int epi_warps = i8_staged(p.splits, p.Mt) ? 16 : 8;
  if (epi_warps == 16 &&
      !make_map(&p.tm_y, y, kBF16, M, h->N, 2ull * h->N, 32, 16, CU_TENSOR_MAP_SWIZZLE_NONE))
    return LL_ERR_CUDA;
  cfg.gridDim = dim3((h->N + 127) / 128, p.splits);
  cfg.blockDim = dim3(is_threads(epi_warps));
  cfg.dynamicSmemBytes = is_smem_bytes(p.Mt, ring);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel_i8_stream(h->epilogue, epi_warps), p) == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

int launch_i8(const ll_i8_layer* h, const I8Plan& plan, const void* codes, const float* scale, void* y, int M,
              cudaStream_t st) {
  using namespace llk;
  I8Params p;
  p.na = plan.na;
  p.nb = plan.nb;
  p.w = plan.w;
  if (!make_map(&p.tm_x, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, M, h->K, h->K, 128, plan.swap ? p.w / 2 : 128,
                CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.tm_y, y, kBF16, M, h->N, 2ull * h->N, 32, plan.swap ? 16 : 32,
                plan.swap ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B))
    return LL_ERR_CUDA;
  p.tm_w = weight_map(h, plan.swap ? 128 : p.w / 2);
  p.sx = scale;
  p.sb = h->sb;
  p.M = M;
  p.N = h->N;
  p.K = h->K;
  p.withhold = h->withhold;
  p.watch = Watch{h->status, h->timeout_ns};
  const long long tiles = static_cast<long long>(p.na) * p.nb;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<long long>(tiles, h->pairs)));
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = i8_smem_bytes();
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel_i8(h->epilogue, plan.swap), p) == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

void free_i8(ll_i8_layer* h) {
  cudaFree(h->W);
  cudaFree(h->sb);
  cudaFree(h->status);
  delete h;
}

}  // namespace

extern "C" {

int ll_rmsnorm_i8(const void* x, const void* residual, const void* weight, float eps, int M, int K, void* h, void* y,
                  void* codes, float* scale, void* stream) {
  g_last_error = LL_OK;
  if (M < 0 || K < 16 || K % 16 != 0 || !std::isfinite(eps) || eps < 1e-30f) return fail(LL_ERR_INVALID_ARG);
  if (K > llk::kRowsMaxK) return fail(LL_ERR_UNSUPPORTED);
  if (M == 0) return LL_OK;
  if (!x || (codes == nullptr) != (scale == nullptr) || (!codes && !y) || (h && !residual))
    return fail(LL_ERR_INVALID_ARG);
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16) || !aligned(y, 16) ||
      !aligned(codes, 16) || !aligned(scale, 4))
    return fail(LL_ERR_INVALID_ARG);
  const size_t n = static_cast<size_t>(M) * K;
  // Each output against every input and every other output; h may be x or
  // residual itself.
  const void* outs[4] = {h, y, codes, scale};
  const size_t out_bytes[4] = {2 * n, 2 * n, n, 4 * static_cast<size_t>(M)};
  const void* ins[3] = {x, residual, weight};
  const size_t in_bytes[3] = {2 * n, 2 * n, 2 * static_cast<size_t>(K)};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    for (int j = 0; j < 3; ++j) {
      if (!ins[j] || (i == 0 && j < 2 && outs[i] == ins[j])) continue;
      if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j])) return fail(LL_ERR_INVALID_ARG);
    }
    for (int j = 0; j < i; ++j)
      if (outs[j] && overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j])) return fail(LL_ERR_INVALID_ARG);
  }
  int dev = 0, sms = 0;
  if (current_device_sms(&dev, &sms) != LL_OK) return fail(LL_ERR_CUDA);
  for (const void* p : {x, residual, weight, static_cast<const void*>(h), static_cast<const void*>(y),
                        static_cast<const void*>(codes), static_cast<const void*>(scale)})
    if (p && !is_device_ptr_on(p, dev)) return fail(LL_ERR_INVALID_ARG);
  llk::RowsParams rp{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual),
                     static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(h), static_cast<uint16_t*>(y),
                     static_cast<int8_t*>(codes), scale, eps, 1.f / static_cast<float>(K), M, K};
  const int rc = launch_rows_i8(rp, true, sms, static_cast<cudaStream_t>(stream));
  return rc == LL_OK ? LL_OK : fail(rc);
}

int ll_quantize_i8(const void* x, int M, int K, void* codes, float* scale, void* stream) {
  g_last_error = LL_OK;
  if (M < 0 || K < 16 || K % 16 != 0) return fail(LL_ERR_INVALID_ARG);
  if (K > llk::kRowsMaxK) return fail(LL_ERR_UNSUPPORTED);
  if (M == 0) return LL_OK;
  if (!x || !codes || !scale || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4))
    return fail(LL_ERR_INVALID_ARG);
  const size_t n = static_cast<size_t>(M) * K, ns = 4 * static_cast<size_t>(M);
  if (overlaps(codes, n, x, 2 * n) || overlaps(scale, ns, x, 2 * n) || overlaps(scale, ns, codes, n))
    return fail(LL_ERR_INVALID_ARG);
  int dev = 0, sms = 0;
  if (current_device_sms(&dev, &sms) != LL_OK) return fail(LL_ERR_CUDA);
  if (!is_device_ptr_on(x, dev) || !is_device_ptr_on(codes, dev) || !is_device_ptr_on(scale, dev))
    return fail(LL_ERR_INVALID_ARG);
  llk::RowsParams rp{static_cast<const uint16_t*>(x), nullptr, nullptr, nullptr, nullptr, static_cast<int8_t*>(codes),
                     scale, 0.f, 0.f, M, K};
  const int rc = launch_rows_i8(rp, false, sms, static_cast<cudaStream_t>(stream));
  return rc == LL_OK ? LL_OK : fail(rc);
}

ll_i8_handle ll_i8_create(int N, int K) {
  g_last_error = LL_OK;
  if (N < 1 || N % 8 != 0 || K < 16 || K % 16 != 0) {
    fail(LL_ERR_INVALID_ARG);
    return nullptr;
  }
  if (K > llk::kI8MaxK || N > kI8MaxRows) {
    fail(LL_ERR_UNSUPPORTED);
    return nullptr;
  }
  int dev = 0, sms = 0, major = 0, minor = 0;
  if (current_device_sms(&dev, &sms) != LL_OK ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    cudaGetLastError();
    fail(LL_ERR_CUDA);
    return nullptr;
  }
  if (major != 10 || minor != 0) {
    fail(LL_ERR_UNSUPPORTED);
    return nullptr;
  }
  ll_i8_layer* h = new (std::nothrow) ll_i8_layer();
  if (!h) {
    fail(LL_ERR_OOM);
    return nullptr;
  }
  h->N = N;
  h->K = K;
  h->device = dev;
  h->num_sms = sms;
  h->N_pad = (N + 511) / 256 * 256;
  if (cudaMalloc(&h->W, static_cast<size_t>(N) * ((K + 127) / 128 * 128)) != cudaSuccess ||
      cudaMalloc(&h->sb, sizeof(float4) * (h->N_pad / 2)) != cudaSuccess || cudaMalloc(&h->status, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    free_i8(h);
    fail(LL_ERR_OOM);
    return nullptr;
  }
  if (!setup_i8(h) || !encode_fn() || !make_weight_maps(h) || cudaMemset(h->status, 0, sizeof(int)) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    free_i8(h);
    fail(LL_ERR_CUDA);
    return nullptr;
  }
  return h;
}

int ll_i8_set_weights(ll_i8_handle h, const void* codes, const float* scale, const void* bias) {
  g_last_error = LL_OK;
  if (!h || !codes || !scale || !aligned(codes, 16) || !aligned(scale, 4) || !aligned(bias, 2))
    return fail(LL_ERR_INVALID_ARG);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(LL_ERR_CUDA);
  }
  if (dev != h->device || !is_device_ptr_on(codes, dev) || !is_device_ptr_on(scale, dev) ||
      (bias && !is_device_ptr_on(bias, dev)))
    return fail(LL_ERR_INVALID_ARG);
  const size_t sb = sizeof(float) * h->N;
  float* host = static_cast<float*>(std::malloc(sb));
  if (!host) return fail(LL_ERR_OOM);
  // A forward still running reads the weights that this call replaces.
  bool ok = cudaDeviceSynchronize() == cudaSuccess &&
            cudaMemcpy(host, scale, sb, cudaMemcpyDeviceToHost) == cudaSuccess;
  bool finite = true;
  for (int n = 0; ok && n < h->N; ++n) finite &= std::isfinite(host[n]);
  std::free(host);
  if (ok && !finite) return fail(LL_ERR_INVALID_ARG);
  if (ok) {
    h->ready = false;
    llk::ll_i8_panels_kernel<<<h->num_sms * 8, 256>>>(static_cast<const int8_t*>(codes), h->W, h->N, h->K);
    llk::ll_i8_scale_bias_kernel<<<(h->N_pad / 2 + 255) / 256, 256>>>(scale, static_cast<const uint16_t*>(bias), h->sb, h->N,
                                                                 h->N_pad);
    ok = cudaGetLastError() == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess;
  }
  if (!ok) {
    cudaGetLastError();
    return fail(LL_ERR_CUDA);
  }
  h->ready = true;
  return LL_OK;
}

int ll_i8_set_epilogue(ll_i8_handle h, int epilogue) {
  g_last_error = LL_OK;
  if (!h || epilogue < LL_EPILOGUE_NONE || epilogue > LL_EPILOGUE_GEGLU_TANH) return fail(LL_ERR_INVALID_ARG);
  if (epilogue == LL_EPILOGUE_GEGLU_TANH) return fail(LL_ERR_UNSUPPORTED);
  h->epilogue = epilogue;
  return LL_OK;
}

int ll_i8_forward(ll_i8_handle h, const void* codes, const float* scale, void* y, int M, void* stream) {
  g_last_error = LL_OK;
  if (!h || M < 0) return fail(LL_ERR_INVALID_ARG);
  if (!h->ready) return fail(LL_ERR_NOT_READY);
  if (M > kI8MaxRows) return fail(LL_ERR_UNSUPPORTED);
  if (M == 0) return LL_OK;
  if (!codes || !scale || !y || !aligned(codes, 16) || !aligned(scale, 4) || !aligned(y, 16))
    return fail(LL_ERR_INVALID_ARG);
  const size_t yb = 2 * static_cast<size_t>(M) * h->N;
  if (overlaps(y, yb, codes, static_cast<size_t>(M) * h->K) || overlaps(y, yb, scale, 4 * static_cast<size_t>(M)))
    return fail(LL_ERR_INVALID_ARG);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(LL_ERR_CUDA);
  }
  if (dev != h->device || !is_device_ptr_on(codes, dev) || !is_device_ptr_on(scale, dev) || !is_device_ptr_on(y, dev))
    return fail(LL_ERR_INVALID_ARG);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const I8Plan plan = i8_plan(h, M);
  const int rc = plan.stream ? launch_i8_stream(h, plan, codes, scale, y, M, st) : launch_i8(h, plan, codes, scale, y, M, st);
  if (rc != LL_OK) cudaGetLastError();
  return rc == LL_OK ? LL_OK : fail(rc);
}

int ll_i8_plan(int N, int K, int M, int num_sms, int* kernel, int* tile_features, int* tile_tokens, int* splits) {
  g_last_error = LL_OK;
  if (N < 1 || N % 8 != 0 || K < 16 || K % 16 != 0 || M < 1 || num_sms < 2) return fail(LL_ERR_INVALID_ARG);
  if (K > llk::kI8MaxK || N > kI8MaxRows || M > kI8MaxRows) return fail(LL_ERR_UNSUPPORTED);
  ll_i8_layer view;  // what the planning reads
  view.N = N;
  view.K = K;
  view.num_sms = num_sms;
  view.pairs = num_sms / 2;
  for (int s = 1; s <= llk::kIsMaxSplit; ++s) view.clusters[s] = num_sms / s;
  const I8Plan p = i8_plan(&view, M);
  if (kernel) *kernel = p.stream ? LL_I8_STREAM : p.swap ? LL_I8_PAIR_SWAP : LL_I8_PAIR;
  if (tile_features) *tile_features = p.stream ? 128 : p.swap ? 256 : p.w;
  if (tile_tokens) *tile_tokens = p.stream ? (M + 15) / 16 * 16 : p.swap ? p.w : 256;
  if (splits) *splits = p.stream ? p.splits : 1;
  return LL_OK;
}

int ll_i8_status(ll_i8_handle h) {
  g_last_error = LL_OK;
  if (!h) return fail(LL_ERR_INVALID_ARG);
  const DeviceScope on(h->device);
  int v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&v, h->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) {
    cudaGetLastError();
    return fail(LL_ERR_CUDA);
  }
  if (v == 0) return LL_OK;
  cudaMemset(h->status, 0, sizeof(int));
  cudaDeviceSynchronize();
  return LL_ERR_DEVICE_TIMEOUT;
}

int ll_i8_set_debug(ll_i8_handle h, int withhold_producer, uint64_t timeout_ns) {
  g_last_error = LL_OK;
  if (!h || timeout_ns == 0) return fail(LL_ERR_INVALID_ARG);
  h->withhold = withhold_producer ? 1 : 0;
  h->timeout_ns = timeout_ns;
  return LL_OK;
}

void ll_i8_destroy(ll_i8_handle h) {
  if (!h) return;
  const DeviceScope on(h->device);
  cudaDeviceSynchronize();
  free_i8(h);
  cudaGetLastError();
}

}  // extern "C"
