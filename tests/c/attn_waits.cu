// What the attention kernels do when a wait is given up, on one CTA: a barrier that nobody arrives at is
// given up after its polls, with the error code and the flag for the other waits set; and bar_drain returns
// when the copies that are on their way to a ring of stages are there, though nobody waited for them.
// Prints: the seconds that a kernel's wait takes to be given up, then "ok" or what differs.
#include <cstdio>
#include <vector>

#include "kvx_attn_tma.cuh"

using namespace kvx;

constexpr int kStages = 4, kBytes = 16384, kPolls = 256;

struct Result {
  int32_t waited, lost, error, second;
  uint64_t ns;
};

__device__ uint64_t now() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// One warp.  Fills `fills` stages in turn without waiting for any but those that it fills again.
__global__ void waits(const char *src, char *dst, int fills, Result *out) {
  extern __shared__ __align__(128) char ring[];
  __shared__ uint64_t full[kStages], never;
  __shared__ int32_t lost, error;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) bar_init(&full[i], 1);
    bar_init(&never, 1);
    lost = error = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint32_t stage = 0, phase = 1;
  if (threadIdx.x == 0) {
    for (int f = 0; f < fills; ++f) {
      // (bounded, and met: the fill before of this stage has been sent)
      for (int n = 0; n < 1 << 16 && !bar_try(&full[stage], phase); ++n) {}
      bar_expect(&full[stage], kBytes);
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       smem_u32(ring + stage * kBytes)),
                   "l"(src + f * kBytes), "r"(kBytes), "r"(smem_u32(&full[stage])) : "memory");
      if (++stage == kStages) stage = 0, phase ^= 1;
    }
    bar_drain<kStages>(full, stage, phase);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kStages * kBytes; i += blockDim.x) dst[i] = ring[i];
  if (threadIdx.x == 0) {
    Result r;
    const uint64_t a = now();
    r.waited = bar_wait(&never, 0, &lost, &error, kPolls);
    r.ns = now() - a;
    r.lost = lost, r.error = error;
    r.second = bar_wait(&never, 0, &lost, &error);  // given up at once, because the first was
    *out = r;
  }
}

int main() {
  char *src, *dst;
  Result *res;
  const int most = 11;
  if (cudaMalloc(&src, most * kBytes) || cudaMalloc(&dst, kStages * kBytes) || cudaMalloc(&res, sizeof(Result))) return 2;
  std::vector<char> in(most * kBytes), got(kStages * kBytes);
  for (size_t i = 0; i < in.size(); ++i) in[i] = (char)(i * 31 + i / 251);
  cudaMemcpy(src, in.data(), in.size(), cudaMemcpyHostToDevice);
  if (cudaFuncSetAttribute(waits, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * kBytes)) return 2;
  double seconds = 0;
  for (int fills : {kStages, kStages + 1, 2 * kStages, most}) {
    waits<<<1, 32, kStages * kBytes>>>(src, dst, fills, res);
    Result r;
    if (cudaMemcpy(&r, res, sizeof(r), cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
    cudaMemcpy(got.data(), dst, got.size(), cudaMemcpyDeviceToHost);
    seconds = r.ns * 1e-9 / (kPolls + 1) * (kAttnPolls + 1.0);
    if (r.waited || r.second || r.lost != 1 || r.error != KVX_ERR_TIMEOUT) {
      printf("wait %d second %d lost %d error %d\n", r.waited, r.second, r.lost, r.error);
      return 1;
    }
    for (int s = 0; s < kStages; ++s) {
      const int f = (fills - 1 - s) / kStages * kStages + s;  // the last fill of stage s
      for (int i = 0; i < kBytes; ++i)
        if (got[s * kBytes + i] != in[f * kBytes + i]) {
          printf("fills %d stage %d byte %d\n", fills, s, i);
          return 1;
        }
    }
  }
  printf("%.3f\nok\n", seconds);
  return 0;
}
