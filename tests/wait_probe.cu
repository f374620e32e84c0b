// Four warps walk rings of bulk copies with the bounded waits of the paged kernels.
// One warp expects a copy that nobody issues, so its wait runs out; every warp must
// leave, with its own copies landed and the reason recorded.
#include "../bit_quantized_kv_02_gb300/csrc/kvq_pages_attn.cuh"

using namespace kvq;

namespace {

constexpr int kProbeWarps = 4, kProbeStages = 3, kProbeSteps = 9, kProbeBytes = 1024;
constexpr unsigned long long kProbeLimit = 30000000ull;  // 30 ms

// done[w]: steps that warp w read; landed[w]: bit i, its copy i steps further is there
// when it leaves; sums[w]: of the words that it read.
__global__ void ring_probe(const uint32_t* src, int lost_warp, int lost_step, int* err, int* done, int* landed,
                           unsigned* sums) {
  __shared__ __align__(128) char ring[kProbeWarps][kProbeStages][kProbeBytes];
  __shared__ __align__(8) uint64_t bars[kProbeWarps][kProbeStages];
  __shared__ int dead;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar = smem_u32(bars[warp]);
  if (lane < kProbeStages) mbar_init(bar + lane * 8, 1);
  if (threadIdx.x == 0) dead = 0;
  fence_mbar_init();
  __syncthreads();
  auto bring = [&](int step) {
    const int s = step % kProbeStages;
    if (lane == 0) {
      mbar_expect(bar + s * 8, kProbeBytes);
      if (warp != lost_warp || step != lost_step)
        bulk_load(smem_u32(ring[warp][s]), src + step * (kProbeBytes / 4), kProbeBytes, bar + s * 8);
    }
    __syncwarp();
  };
  for (int i = 0; i < kProbeStages; ++i) bring(i);
  int step = 0, stage = 0, phase = 0, there = 0;
  unsigned sum = 0;
  for (; step < kProbeSteps; ++step) {
    if (!warp_wait(bar + stage * 8, phase, &dead, err, kProbeLimit)) {
      const int n = min(kProbeStages, kProbeSteps - step);
      ring_drain<kProbeStages>(bar, stage, phase, n, kProbeLimit);
      for (int i = 0; i < n; ++i)
        there |= (int)mbar_try(bar + (stage + i) % kProbeStages * 8, phase ^ (stage + i >= kProbeStages)) << i;
      break;
    }
    for (int i = lane; i < kProbeBytes / 4; i += 32) sum += reinterpret_cast<volatile uint32_t*>(ring[warp][stage])[i];
    fence_async();
    __syncwarp();
    if (step + kProbeStages < kProbeSteps) bring(step + kProbeStages);
    if (++stage == kProbeStages) stage = 0, phase ^= 1;
  }
  atomicAdd(&sums[warp], sum);
  __syncthreads();
  if (lane == 0) done[warp] = step, landed[warp] = there;
}

}  // namespace

// out: [1 + 3 * kProbeWarps] ints (device): error word, done, landed, sums; src: [kProbeSteps * 256] words (device)
extern "C" int wait_probe(const void* src, int lost_warp, int lost_step, void* out) {
  int* o = static_cast<int*>(out);
  ring_probe<<<1, kProbeWarps * 32>>>(static_cast<const uint32_t*>(src), lost_warp, lost_step, o, o + 1,
                                      o + 1 + kProbeWarps,
                                      reinterpret_cast<unsigned*>(o + 1 + 2 * kProbeWarps));
  const cudaError_t e = cudaDeviceSynchronize();
  return (int)e;
}
