// kvx_attn_general.cu -- the plain kernel of kvx_shared_attention: any type, head_dim and
// alignment, and what 32-bit pools take.
//
// A CTA of 128 threads works one piece of up to 16 rows: the queries and 32 keys at a time sit in
// shared memory as 32-bit values, rows padded to a multiple of four columns.  Each warp scores four
// rows, a lane a key, four columns at a time, and takes the running maximum and sum of its rows with
// shuffles; then every thread adds the tile's weighted values into its one or two columns of all 16
// rows, held in registers, four keys at a time.  The next tile's elements are on their way meanwhile
// where 16-byte loads are possible.  Pieces of up to four rows (kFew) take one row a warp and leave the
// other twelve out: 32 decode requests of 4 rows in 32 bits 219 -> 182 us.
//
// Bound: shared-memory reads (5 of 16 bytes for 64 multiply-adds) and the barriers of a tile.  Up to 128
// columns three CTAs share an SM (168 registers; two took 1208 us for 117 decode requests of 7 rows and
// 4016 shared tokens in 32 bits, 8 kv heads; three 909 us; four, at 128 registers with spills, 1027 us).
// With kFew 894 us: 15 TFLOP/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "kvx_attn.cuh"
#include "kvx_launch.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = kAttnGeneralRows, kFew = 4;
constexpr int kKeys = 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__nv_fp8_e4m3 x) { return (float)x; }

// Rows of D columns padded to pitch(D): a multiple of four, and 16-byte reads of eight rows of one
// column lie in different banks.
__host__ __device__ constexpr int pitch(int D) { return (D + 3) / 4 * 4 + 4; }

template <typename KV>
__device__ __forceinline__ void unpack(const uint4 &v, float *o) {
  const KV *e = reinterpret_cast<const KV *>(&v);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(KV)); ++i) o[i] = to_f(e[i]);
}

// NC: columns a thread.  VEC: 16-byte loads.
template <typename KV, typename IO, int NC, bool VEC>
__global__ void __launch_bounds__(kThreads, NC == 1 ? 3 : 2) attn_general_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ float4 smem4[];
  const int D = p.head_dim, P = pitch(D), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *sq = reinterpret_cast<float *>(smem4);  // [kRows][P]
  float *sk = sq + kRows * P;           // [kKeys][P]
  float *sv = sk + kKeys * P;           // [kKeys][P]
  float *sp = sv + kKeys * P;           // [kRows][kKeys]
  float *sc = sp + kRows * kKeys;       // [kRows]: rescale of the tile
  __shared__ int32_t slim[kRows];
  __shared__ int64_t scan[2 * (kThreads / 32) + 4];
  __shared__ int64_t soff[kKeys];
  __shared__ int32_t error;
  constexpr int kElems = 16 / sizeof(KV);             // of a 16-byte load
  constexpr int kMost = VEC ? kKeys * NC * 128 / kElems / kThreads : 1;  // loads a thread and tile, K or V
  attn_wait_prior();
  if (tid == 0) error = 0;
  const int g = blockIdx.x / p.kv_heads, head = blockIdx.x - g * p.kv_heads;
  const AttnLine line = attn_line<kThreads>(p, g, scan);
  if (D % 4 != 0)  // columns past D are 0 throughout
    for (int i = tid; i < (kRows + 2 * kKeys) * P; i += kThreads) sq[i] = 0.f;
  attn_pieces(p, g, head, line, [&](const AttnPiece &item) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c) {  // all rows' elements of a column are on their way together
      const int d = tid + c * kThreads;
      float x[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int row = item.row0 + r, t = row / p.group;
        const IO *q = reinterpret_cast<const IO *>(p.q + t * p.q_tok +
                                                   (int64_t)(head * p.group + row - t * p.group) * p.q_head);
        x[r] = r < item.rows && d < D ? to_f(q[d]) * p.scale_log2 : 0.f;
      }
      if (d < D)
#pragma unroll
        for (int r = 0; r < kRows; ++r) sq[r * P + d] = x[r];
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
    const bool few = item.rows <= kFew;  // the first row of each warp alone
    const int begin = max(item.key0, item.low), end = min(item.key1, most);
    // every warp looks all keys of a tile up, a lane a key: the offsets then go by shuffles
    auto look = [&](int k0) -> int64_t {
      return k0 + lane < end ? attn_key_offset(p, item.table, k0 + lane, &error) + head * p.pool.head_stride : 0;
    };
    const int chunks = D / kElems;  // VEC: D is a multiple of kElems
    uint4 rk[kMost], rv[kMost];
    auto fetch = [&](int64_t off) {
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        const int e = i * kThreads + tid, j = e / chunks, c = e - j * chunks;
        const int64_t o = __shfl_sync(~0u, off, j & 31) + c * 16;  // a row has whole warps' loads or its lanes agree
        if (j < kKeys) {
          rk[i] = *reinterpret_cast<const uint4 *>(p.pool.k + o);
          rv[i] = *reinterpret_cast<const uint4 *>(p.pool.v + o);
        }
      }
    };
    if (VEC && begin < end) fetch(look(begin));
    for (int k0 = begin; k0 < end; k0 += kKeys) {
      const int nk = min(kKeys, end - k0);
      __syncthreads();  // the tile before has been read
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          const int e = i * kThreads + tid, j = e / chunks, c = e - j * chunks;
          if (j >= kKeys) continue;
          float x[kElems], y[kElems];
          unpack<KV>(rk[i], x);
          unpack<KV>(rv[i], y);
#pragma unroll
          for (int w = 0; w < kElems; w += 4) {
            float4 a = make_float4(x[w], x[w + 1], x[w + 2], x[w + 3]), b = make_float4(y[w], y[w + 1], y[w + 2], y[w + 3]);
            if (j >= nk) a = b = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(sk + j * P + c * kElems + w) = a;
            *reinterpret_cast<float4 *>(sv + j * P + c * kElems + w) = b;
          }
        }
        if (k0 + kKeys < end) fetch(look(k0 + kKeys));
      } else {
        if (tid < 32) soff[lane] = look(k0);
        __syncthreads();
        for (int i = tid; i < kKeys * D; i += kThreads) {
          const int j = i / D, d = i - j * D;
          const int64_t o = soff[j];
          float x = 0.f, y = 0.f;
          if (j < nk) {
            x = to_f(reinterpret_cast<const KV *>(p.pool.k + o)[d]);
            y = to_f(reinterpret_cast<const KV *>(p.pool.v + o)[d]);
          }
          sk[j * P + d] = x;
          sv[j * P + d] = y;
        }
      }
      __syncthreads();
      float s[kRows / 4] = {};
      const float4 *kr = reinterpret_cast<const float4 *>(sk + lane * P);
      const float4 *qr = reinterpret_cast<const float4 *>(sq + warp * P);  // row i of a warp: 4 i + warp
      auto scores = [&](auto rows_) {
#pragma unroll 4
        for (int d = 0; d < (D + 3) / 4; ++d) {
          const float4 k = kr[d];
#pragma unroll
          for (int i = 0; i < decltype(rows_)::value; ++i) {
            const float4 q = qr[i * P + d];
            s[i] = fmaf(q.x, k.x, s[i]), s[i] = fmaf(q.y, k.y, s[i]);
            s[i] = fmaf(q.z, k.z, s[i]), s[i] = fmaf(q.w, k.w, s[i]);
          }
        }
      };
      if (few) scores(std::integral_constant<int, kFew / 4>{});
      else scores(std::integral_constant<int, kRows / 4>{});
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        const int r = i * 4 + warp;
        if (few && i >= kFew / 4) continue;
        if (lane >= nk || k0 + lane >= slim[r]) s[i] = -INFINITY;
        float top = s[i];
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        top = fmaxf(top, m[i]);
        const float base = top == -INFINITY ? 0.f : top;
        const float e = exp2f(s[i] - base), f = exp2f(m[i] - base);
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
          auto add = [&](auto rows_) {
            constexpr int R = decltype(rows_)::value;
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r][c] *= sc[r];
            if (mixed) {
              for (int j = 0; j < nk; ++j) {
                const float v = sv[j * P + d];
#pragma unroll
                for (int r = 0; r < R; ++r)
                  if (k0 + j < slim[r]) acc[r][c] = fmaf(sp[r * kKeys + j], v, acc[r][c]);
              }
            } else {  // keys past nk are 0 and weigh 0
              for (int j = 0; j < nk; j += 4) {
                const float v0 = sv[j * P + d], v1 = sv[(j + 1) * P + d], v2 = sv[(j + 2) * P + d], v3 = sv[(j + 3) * P + d];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                  const float4 w = *reinterpret_cast<const float4 *>(sp + r * kKeys + j);
                  acc[r][c] = fmaf(w.x, v0, acc[r][c]), acc[r][c] = fmaf(w.y, v1, acc[r][c]);
                  acc[r][c] = fmaf(w.z, v2, acc[r][c]), acc[r][c] = fmaf(w.w, v3, acc[r][c]);
                }
              }
            }
          };
          if (few) add(std::integral_constant<int, kFew>{});
          else add(std::integral_constant<int, kRows>{});
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
        const int r = i * 4 + warp;
        if (r < item.rows) p.part_m[item.part + r] = m[i], p.part_l[item.part + r] = l[i];
      }
  });
  __syncthreads();
  if (tid == 0) p.errors[blockIdx.x] = error;
}

template <typename KV, typename IO, int NC>
cudaError_t launch_c(const AttnParams &p, bool vec, cudaStream_t s) {
  const size_t smem = sizeof(float) * ((size_t)pitch(p.head_dim) * (kRows + 2 * kKeys) + kRows * kKeys + kRows);
  const void *fn = vec ? (const void *)attn_general_kernel<KV, IO, NC, true>
                       : (const void *)attn_general_kernel<KV, IO, NC, false>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
  if (e != cudaSuccess) return e;
  void *args[] = {const_cast<AttnParams *>(&p)};
  return launch_pdl(fn, dim3(p.groups * p.kv_heads), dim3(kThreads), args, s, smem);
}

template <typename KV, typename IO>
cudaError_t launch(const AttnParams &p, bool vec, cudaStream_t s) {
  return p.head_dim <= kThreads ? launch_c<KV, IO, 1>(p, vec, s) : launch_c<KV, IO, 2>(p, vec, s);
}

}  // namespace

cudaError_t launch_attn_general(const AttnParams &p, int32_t dtype, int32_t io, bool vec, cudaStream_t s) {
  if (dtype == KVX_F32) return launch<float, float>(p, vec, s);
  if (dtype == KVX_F16) return launch<__half, __half>(p, vec, s);
  if (dtype == KVX_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(p, vec, s);
  if (io == KVX_F16) return launch<__nv_fp8_e4m3, __half>(p, vec, s);
  return launch<__nv_fp8_e4m3, __nv_bfloat16>(p, vec, s);
}

}  // namespace kvx
