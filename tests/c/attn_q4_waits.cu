// What becomes of a 4-bit pool's copies on their way when a wait is given up, on one CTA: a warp fills a ring of stages by
// copies of 16 bytes whose arrivals (a lane each, 32 a stage) are the copies' own, without anyone waiting for them; its last
// copies and bar_drain are all that stands between them and the ring's end, as in the 4-bit kernel's producer warp.
// Prints "ok" or what differs.
#include <cstdio>
#include <vector>

#include "kvx_attn_tma.cuh"

using namespace kvx;

constexpr int kStages = 3, kBytes = 16384, kPolls = 256;

struct Result {
  int32_t waited, lost, error;
};

__global__ void fill(const char *src, char *dst, int fills, Result *out) {
  extern __shared__ __align__(128) char ring[];
  __shared__ uint64_t full[kStages], never;
  __shared__ int32_t lost, error;
  const int lane = threadIdx.x;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) bar_init(&full[i], 32);
    bar_init(&never, 1);
    lost = error = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint32_t stage = 0, phase = 1;
  for (int f = 0; f < fills; ++f) {
    // (bounded, and met: the fill before of this stage is on its way)
    for (int n = 0; n < 1 << 16 && !bar_try(&full[stage], phase); ++n) {}
    __syncwarp();
    for (int i = lane * 16; i < kBytes; i += 512)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(ring + stage * kBytes + i)),
                   "l"(src + f * kBytes + i) : "memory");
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&full[stage])) : "memory");
    if (++stage == kStages) stage = 0, phase ^= 1;
  }
  Result r;
  r.waited = bar_wait(&never, 0, &lost, &error, kPolls);
  cp_async_commit();
  cp_async_wait<0>();
  bar_drain<kStages>(full, stage, phase);
  __syncthreads();
  for (int i = lane; i < kStages * kBytes; i += 32) dst[i] = ring[i];
  r.lost = lost, r.error = error;
  if (lane == 0) *out = r;
}

int main() {
  char *src, *dst;
  Result *res;
  const int most = 11;
  if (cudaMalloc(&src, most * kBytes) || cudaMalloc(&dst, kStages * kBytes) || cudaMalloc(&res, sizeof(Result))) return 2;
  std::vector<char> in(most * kBytes), got(kStages * kBytes);
  for (size_t i = 0; i < in.size(); ++i) in[i] = (char)(i * 29 + i / 241);
  cudaMemcpy(src, in.data(), in.size(), cudaMemcpyHostToDevice);
  if (cudaFuncSetAttribute(fill, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * kBytes)) return 2;
  for (int fills : {kStages, kStages + 1, 2 * kStages, most}) {
    fill<<<1, 32, kStages * kBytes>>>(src, dst, fills, res);
    Result r;
    if (cudaMemcpy(&r, res, sizeof(r), cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
    cudaMemcpy(got.data(), dst, got.size(), cudaMemcpyDeviceToHost);
    if (r.waited || r.lost != 1 || r.error != KVX_ERR_TIMEOUT) {
      printf("wait %d lost %d error %d\n", r.waited, r.lost, r.error);
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
  printf("ok\n");
  return 0;
}
