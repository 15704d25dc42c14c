// Attention of a chunk of new tokens over a paged LoopKV cell (sm_100a): the
// choice between the kernels of chunk_few.cuh (at most 16 rows of a KV head, 4-bit
// and 2-bit cells) and chunk_tensor.cuh (everything else), and their launches.
#include <mutex>

#include "chunk_few.cuh"
#include "chunk_tensor.cuh"

namespace loopkv {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxSplits = 8;  // the portable cluster size

int current_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) dev = -1;
  return dev;
}

int sm_count(int dev) {
  static std::mutex mu;
  static int count[kMaxDevices] = {};
  if (dev < 0) return 148;
  std::lock_guard<std::mutex> lock(mu);
  if (count[dev] == 0) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
    count[dev] = sms;
  }
  return count[dev];
}

// One launch of `units` groups of `splits` CTAs, a cluster each.
template <typename Kernel, typename... Args>
cudaError_t launch_clusters(Kernel kern, int64_t units, int splits, int threads, size_t smem, cudaStream_t stream,
                            const ChunkAttnParams& p, Args... args) {
  if (units * splits > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * splits), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  if (splits > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kern, p, args..., splits);
}

// Shared-memory limit of a kernel (MT < 0: of -MT warps, for few rows), once a device.
template <int KIND, int D, int MT, typename Kernel>
cudaError_t prepare_once(Kernel kern, size_t smem, int dev) {
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (dev >= 0) done[dev] = true;
  return cudaSuccess;
}

// Clusters of `splits` CTAs that the device holds at once (a cluster stays within
// one group of SMs, so these are fewer than the SMs would give).
template <int KIND, int D, int MT, typename Kernel>
int64_t resident_clusters(Kernel kern, int splits, int threads, size_t smem, int dev) {
  static std::mutex mu;
  static int64_t cache[kMaxDevices][kMaxSplits + 1] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && cache[dev][splits]) return cache[dev][splits];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(splits, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = splits;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1) clusters = 1;
  if (dev >= 0) cache[dev][splits] = clusters;
  return clusters;
}

template <int KIND, int D, int MT>
cudaError_t launch_mt(const ChunkAttnParams& p, cudaStream_t stream) {
  using L = ChunkSmem<D, MT>;
  // At most as many CTAs an SM as its tensor memory serves (2 x 256 columns, or
  // one of 512): the request keeps further ones out, whose allocation would wait.
  constexpr size_t kSmem = MT * (2 * kStepKeys + D) > 256 && L::kBytes < 120 * 1024 ? 120 * 1024 : L::kBytes;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
  const int dev = current_device();
  static constexpr auto kern = chunk_tensor_kernel<KIND, D, MT>;
  const cudaError_t e = prepare_once<KIND, D, MT>(kern, kSmem, dev);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.chunk.T) << p.g_log2;
  const int64_t row_tiles = (rows + MT * 128 - 1) / (MT * 128);
  const int64_t units = row_tiles * p.Hkv * p.chunk.B;
  const int64_t keys = static_cast<int64_t>(p.max_stored) + (p.k_cur.p ? p.chunk.T : 0);
  const int64_t key_tiles = (keys + kTileKeys - 1) / kTileKeys;
  // as many splits as all run at once, of at least two tiles each
  int splits = 1;
  while (splits < kMaxSplits && key_tiles >= splits * 4 &&
         units <= resident_clusters<KIND, D, MT>(kern, splits * 2, chunk_threads<MT>(), kSmem, dev))
    splits *= 2;
  return launch_clusters(kern, units, splits, chunk_threads<MT>(), kSmem, stream, p, static_cast<int>(row_tiles));
}

// Few rows, CTAs of WARPS warps.  With `best`, each split's cost is compared with
// it, and it, warps and splits are set where that is less; without, the launch.
template <int KIND, int D, int WARPS>
cudaError_t few_w(const ChunkAttnParams& p, int64_t units, int64_t groups, int dev, int* warps, int* splits, int64_t* best,
                  cudaStream_t stream) {
  using L = FewSmem<KIND, D, WARPS>;
  static_assert(kFewWarpsPerSm / WARPS * (L::kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
  static constexpr auto kern = chunk_few_kernel<KIND, D, WARPS>;
  const cudaError_t e = prepare_once<KIND, D, -WARPS>(kern, L::kBytes, dev);
  if (e != cudaSuccess) return e;
  if (!best) return launch_clusters(kern, units, *splits, WARPS * 32, L::kBytes, stream, p);
  auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t sms = sm_count(dev);
  for (int s = 1; s <= kMaxSplits; s *= 2) {
    const int64_t at_once = s == 1 ? sms * (kFewWarpsPerSm / WARPS)
                                   : resident_clusters<KIND, D, -WARPS>(kern, s, WARPS * 32, L::kBytes, dev);
    const int64_t waves = ceil_div(units, at_once);
    // CTAs on the busiest SM; a cluster's fill an SM before they go to the next
    int64_t load = ceil_div(units * s, sms);
    const int64_t packed = s == 1 ? 1 : s < kFewWarpsPerSm / WARPS ? s : kFewWarpsPerSm / WARPS;
    load = load > waves * packed ? load : waves * packed;
    const int64_t busiest = load * ceil_div(groups, s), serial = waves * ceil_div(groups, s * WARPS) * 6;
    const int64_t cost = (busiest > serial ? busiest : serial) + waves * (s == 1 ? 25 : 45);
    if (cost < *best) *best = cost, *splits = s, *warps = WARPS;
  }
  return cudaSuccess;
}

// Few rows: the CTA size and split of least estimated time, in the time that an
// SM with twelve warps at work takes a 32-token group (440 cycles): what the
// busiest SM has to read, or six for each group that a warp takes one after
// another; and for each wave of CTAs their start and end, 25, or 45 as clusters.
// Measured with heads of 128 and 4 bits, 512 (sequence, head) pairs of 4100 tokens:
// CTAs of 12 warps 151 us, of 6 warps 135, of 3 warps 126 (one wave), of 3 warps in
// clusters of two 136.  16 pairs of 16384: 12 warps alone 122 us, in clusters of
// four 40 (taken), of eight (which do not all run at once) 52, 6 warps in clusters
// of eight 39; 16 pairs of 1024: 14 taken, 12 the best.  With heads of 64 and 2
// bits, half the work a group, the same choices: 512 pairs of 4100 78 us (the
// best), 128 pairs 25 (the best), 16 pairs of 16384 27 (best 25), of 1024 9.0 (8.4).
template <int KIND, int D>
cudaError_t launch_few(const ChunkAttnParams& p, cudaStream_t stream) {
  const int dev = current_device();
  const int64_t units = static_cast<int64_t>(p.Hkv) * p.chunk.B;
  const int64_t groups = (static_cast<int64_t>(p.max_stored) + kGroup - 1) / kGroup + (p.k_cur.p ? 1 : 0);
  int warps = kFewWarpsPerSm, splits = 1;
  int64_t best = INT64_MAX;
  cudaError_t e = few_w<KIND, D, 12>(p, units, groups, dev, &warps, &splits, &best, stream);
  if (e == cudaSuccess) e = few_w<KIND, D, 6>(p, units, groups, dev, &warps, &splits, &best, stream);
  if (e == cudaSuccess) e = few_w<KIND, D, 3>(p, units, groups, dev, &warps, &splits, &best, stream);
  if (e != cudaSuccess) return e;
  switch (warps) {
    case 3: return few_w<KIND, D, 3>(p, units, groups, dev, &warps, &splits, nullptr, stream);
    case 6: return few_w<KIND, D, 6>(p, units, groups, dev, &warps, &splits, nullptr, stream);
    default: return few_w<KIND, D, 12>(p, units, groups, dev, &warps, &splits, nullptr, stream);
  }
}

template <int KIND, int D>
cudaError_t launch_t(const ChunkAttnParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.chunk.T) << p.g_log2;
  if constexpr (KIND != LOOPKV_CELL_BF16)
    if (rows <= kFewRows) return launch_few<KIND, D>(p, stream);
  return rows > 128 ? launch_mt<KIND, D, 2>(p, stream) : launch_mt<KIND, D, 1>(p, stream);
}

}  // namespace

cudaError_t launch_chunk_attention(int kind, int head_dim, const ChunkAttnParams& p, cudaStream_t stream) {
  switch (kind * 1000 + head_dim) {
    case LOOPKV_CELL_Q4 * 1000 + 128: return launch_t<LOOPKV_CELL_Q4, 128>(p, stream);
    case LOOPKV_CELL_Q4 * 1000 + 64: return launch_t<LOOPKV_CELL_Q4, 64>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 128: return launch_t<LOOPKV_CELL_Q2, 128>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 64: return launch_t<LOOPKV_CELL_Q2, 64>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 128: return launch_t<LOOPKV_CELL_BF16, 128>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 64: return launch_t<LOOPKV_CELL_BF16, 64>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace loopkv
