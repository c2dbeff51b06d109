// kvx_attn_general.cu -- the plain kernel of kvx_shared_attention: any type, head_dim and
// alignment.
//
// A CTA of 128 threads works one piece of up to 16 rows: the queries and 32 keys at a time sit in
// shared memory as 32-bit values; each warp scores four rows, a lane a key, and takes the
// running maximum and sum of its rows with shuffles; then every thread adds the tile's weighted
// values into its one or two columns of all 16 rows, held in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kvx_attn.cuh"
#include "kvx_launch.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = kAttnGeneralRows;
constexpr int kKeys = 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__nv_fp8_e4m3 x) { return (float)x; }

template <typename KV, typename IO, int NC>
__global__ void __launch_bounds__(kThreads) attn_general_kernel(const AttnParams p) {
  extern __shared__ float sm[];
  const int D = p.head_dim, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *sq = sm;                       // [kRows][D]
  float *sk = sq + kRows * D;           // [kKeys][D + 1]
  float *sv = sk + kKeys * (D + 1);     // [kKeys][D]
  float *sp = sv + kKeys * D;           // [kRows][kKeys]
  float *sc = sp + kRows * kKeys;       // [kRows]: rescale of the tile
  __shared__ int64_t soff[kKeys];
  __shared__ int32_t slim[kRows];
  attn_wait_prior();
  const int g = blockIdx.x / p.kv_heads, head = blockIdx.x - g * p.kv_heads;
  __shared__ int64_t scan[2 * (kThreads / 32) + 4];
  __shared__ int32_t error;
  if (tid == 0) error = 0;
  const AttnLine line = attn_line<kThreads>(p, g, scan);
  attn_pieces(p, g, head, line, [&](const AttnPiece &item) {
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kThreads) {
      const int r = i / D, d = i - r * D;
      float x = 0.f;
      if (r < item.rows) {
        const int row = item.row0 + r, t = row / p.group;
        const IO *q = reinterpret_cast<const IO *>(p.q + t * p.q_tok +
                                                   (head * p.group + row - t * p.group) * p.q_head);
        x = to_f(q[d]) * p.scale_log2;
      }
      sq[i] = x;
    }
    if (tid < kRows) slim[tid] = tid < item.rows ? attn_limit(p, (item.row0 + tid) / p.group) : 0;
    float acc[kRows][NC], m[kRows / 4], l[kRows / 4];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[r][c] = 0.f;
#pragma unroll
    for (int r = 0; r < kRows / 4; ++r) m[r] = -INFINITY, l[r] = 0.f;
    __syncthreads();
    int most = 0, least = INT32_MAX;
    for (int r = 0; r < item.rows; ++r) most = max(most, slim[r]), least = min(least, slim[r]);
    const int end = min(item.key1, most);
    for (int k0 = max(item.key0, item.low); k0 < end; k0 += kKeys) {
      const int nk = min(kKeys, end - k0);
      __syncthreads();  // the tile before has been read
      if (tid < nk) soff[tid] = attn_key_offset(p, item.table, k0 + tid, &error) + head * p.pool.head_stride;
      __syncthreads();
      for (int i = tid; i < kKeys * D; i += kThreads) {
        const int j = i / D, d = i - j * D;
        float x = 0.f, y = 0.f;
        if (j < nk) {
          x = to_f(reinterpret_cast<const KV *>(p.pool.k + soff[j])[d]);
          y = to_f(reinterpret_cast<const KV *>(p.pool.v + soff[j])[d]);
        }
        sk[j * (D + 1) + d] = x;
        sv[j * D + d] = y;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        const int r = warp * (kRows / 4) + i;
        float s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(sq[r * D + d], sk[lane * (D + 1) + d], s);
        if (lane >= nk || k0 + lane >= slim[r]) s = -INFINITY;
        float top = s;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        top = fmaxf(top, m[i]);
        const float base = top == -INFINITY ? 0.f : top;
        const float e = exp2f(s - base), f = exp2f(m[i] - base);
        float sum = e;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = top;
        sp[r * kKeys + lane] = e;
        if (lane == 0) sc[r] = f;
      }
      __syncthreads();
      // where some row's mask falls into the tile, what masked rows' keys hold must not be
      // multiplied by their weight of 0 (it may be an infinity or NaN)
      const bool mixed = k0 + nk > least;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = tid + c * kThreads;
        if (d < D) {
#pragma unroll
          for (int r = 0; r < kRows; ++r) acc[r][c] *= sc[r];
          for (int j = 0; j < nk; ++j) {
            const float v = sv[j * D + d];
            if (mixed) {
#pragma unroll
              for (int r = 0; r < kRows; ++r)
                if (k0 + j < slim[r]) acc[r][c] = fmaf(sp[r * kKeys + j], v, acc[r][c]);
            } else {
#pragma unroll
              for (int r = 0; r < kRows; ++r) acc[r][c] = fmaf(sp[r * kKeys + j], v, acc[r][c]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = tid + c * kThreads;
      if (d < D)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r < item.rows) p.part_o[(item.part + r) * D + d] = acc[r][c];
    }
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        const int r = warp * (kRows / 4) + i;
        if (r < item.rows) p.part_m[item.part + r] = m[i], p.part_l[item.part + r] = l[i];
      }
  });
  __syncthreads();
  if (tid == 0) p.errors[blockIdx.x] = error;
}

template <typename KV, typename IO>
cudaError_t launch(const AttnParams &p, cudaStream_t s) {
  const size_t smem = sizeof(float) * ((size_t)p.head_dim * (kRows + 2 * kKeys) + kKeys +
                                       kRows * kKeys + kRows);
  const void *fn = p.head_dim <= kThreads ? (const void *)attn_general_kernel<KV, IO, 1>
                                          : (const void *)attn_general_kernel<KV, IO, 2>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
  if (e != cudaSuccess) return e;
  void *args[] = {const_cast<AttnParams *>(&p)};
  return launch_pdl(fn, dim3(p.groups * p.kv_heads), dim3(kThreads), args, s, smem);
}

}  // namespace

cudaError_t launch_attn_general(const AttnParams &p, int32_t dtype, int32_t io, cudaStream_t s) {
  if (dtype == KVX_F32) return launch<float, float>(p, s);
  if (dtype == KVX_F16) return launch<__half, __half>(p, s);
  if (dtype == KVX_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(p, s);
  if (io == KVX_F16) return launch<__nv_fp8_e4m3, __half>(p, s);
  return launch<__nv_fp8_e4m3, __nv_bfloat16>(p, s);
}

}  // namespace kvx
