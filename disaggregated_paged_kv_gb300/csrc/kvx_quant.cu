// kvx_quant.cu -- rows quantised as they are written into a pool, and read back.
//
// A thread has eight neighbouring elements of a head (16 bytes of 16-bit values), so a 4-bit group of 32
// is four lanes': its least and greatest value take two shuffles each, its codes are four words side by
// side, and one lane writes scale and low.  The four such pieces of a thread are loaded before anything is
// waited for; as in the row copy kernel, the planner's verdict (or, for few tokens, the CTA's own check of
// every index) is looked at between the loads and the first store, so that a call writes all or nothing.
//
// Bound: bytes, 2 + 5/8 of them an element of a 16-bit tensor and a 4-bit pool.
#include <cuda_bf16.h>

#include "kvx_launch.cuh"
#include "kvx_quant.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;  // of a thread, on their way together

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float *o, float x) { *o = x; }
__device__ __forceinline__ void from_f(__half *o, float x) { *o = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16 *o, float x) { *o = __float2bfloat16_rn(x); }

// The smaller and the greater of two, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two E4M3 numbers, lo in the low byte; beyond +-448 the greatest.
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t from_e4m3x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

constexpr float kMost = 61440.f;  // what low + 15 * scale can reach without passing f16's end

// The codes of this lane's eight elements, element i in bits 4 i .., and the group's (scale, low), which all
// four lanes of the group get.  Steps are rounded one by one (no fused multiply-add), as kvx.h says.
__device__ __forceinline__ uint32_t encode(float (&x)[8], uint32_t *pair) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = min_nan(lo, x[i]), hi = max_nan(hi, x[i]);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(~0u, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(~0u, hi, o));
  }
  if (isnan(lo)) {
    *pair = 0x7fff0000u;
    return 0;
  }
  // (clamping the ends is clamping the values: codes past them are clamped below)
  const __half low = __float2half_rn(fminf(fmaxf(lo, -kMost), kMost));
  const float base = __half2float(low);
  const float reach = __fsub_rn(fminf(fmaxf(hi, -kMost), kMost), base);
  const __half scale = __float2half_rn(fmaxf(__fmul_rn(reach, 1.f / 15.f), 0.f));
  *pair = (uint32_t)__half_as_ushort(scale) | (uint32_t)__half_as_ushort(low) << 16;
  const float s = __half2float(scale), r = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t codes = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float y = fminf(fmaxf(x[i], -kMost), kMost);
    const float c = fminf(fmaxf(__fmul_rn(__fsub_rn(y, base), r), 0.f), 15.f);
    // the nearest whole number, ties to even, in the low bits of c + 1.5 * 2^23
    codes = codes << 4 | (__float_as_uint(__fadd_rn(c, 12582912.f)) & 15u);
  }
  return codes;
}

// An element of a group.
__device__ __forceinline__ float decode(uint32_t code, float scale, float low) {
  // 2^23 + code, less 2^23
  return __fmaf_rn(__uint_as_float(0x4b000000u | code) - 8388608.f, scale, low);
}

// Where a piece is: N elements of one head of one token.
struct Piece {
  char *pool;       // the head vector; nullptr: nothing to be done
  char *data;       // the elements in k or v
  int32_t d;        // first element in the head
};

template <int N>
__device__ __forceinline__ Piece piece_at(const QuantArgs &q, int p, int64_t at, int64_t most, int e) {
  Piece x = {nullptr, nullptr, 0};
  if (at >= most) return x;
  const int32_t per_head = q.head_dim / N, per_row = per_head * q.heads;
  int64_t i;
  int32_t c;
  if (most <= INT32_MAX) {
    i = (uint32_t)at / (uint32_t)per_row;
    c = (int32_t)((uint32_t)at - (uint32_t)i * (uint32_t)per_row);
  } else {
    i = at / per_row;
    c = (int32_t)(at - i * per_row);
  }
  const int32_t h = c / per_head;
  x.d = (c - h * per_head) * N;
  const int32_t slot = q.slots[i];
  const int64_t row = q.rows ? (int64_t)q.rows[i] : i;
  if (slot < 0 || slot >= q.pool.num_slots || row < 0 || row >= q.n_rows) return x;
  int64_t off;
  if (q.pool.hnd) {
    const int32_t page = slot / q.pool.page_size, in = slot - page * q.pool.page_size;
    off = page * q.pool.page_bytes + ((int64_t)h * q.pool.page_size + in) * q.pool.seg_bytes;
  } else {
    off = slot * q.pool.slot_stride + (int64_t)h * q.pool.seg_bytes;
  }
  x.pool = q.base[p] + off;
  x.data = (p & 1 ? q.v : q.k) + (p >> 1) * q.layer_stride + row * q.token_stride + h * q.head_stride + (int64_t)x.d * e;
  return x;
}

// False: some index is out of range, and nothing may be written.
__device__ __forceinline__ bool all_in_range(const QuantArgs &q) {
  int bad = 0;
  for (int64_t i = threadIdx.x; i < q.n; i += kThreads) {
    const int32_t s = q.slots[i];
    bad |= s < 0 || s >= q.pool.num_slots;
    if (q.rows) bad |= q.rows[i] < 0 || q.rows[i] >= q.n_rows;
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *q.status = bad ? KVX_ERR_OUT_OF_RANGE : KVX_OK;
  return !bad;
}

// N elements of IO as they stand in memory.
template <typename IO, int N>
struct Raw {
  static constexpr int kBytes = N * (int)sizeof(IO), kVecs = kBytes / 16;
  alignas(16) IO e[N];
  __device__ __forceinline__ void load(const char *s, bool wide) {
    if (N > 1 && wide) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4 *>(e)[i] = reinterpret_cast<const uint4 *>(s)[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = reinterpret_cast<const IO *>(s)[i];
    }
  }
  __device__ __forceinline__ void store(char *s, bool wide) const {
    if (N > 1 && wide) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4 *>(s)[i] = reinterpret_cast<const uint4 *>(e)[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) reinterpret_cast<IO *>(s)[i] = e[i];
    }
  }
};

// N: elements of a piece, eight, or one where an 8-bit pool's head vectors are no multiple of that.
template <typename IO, bool Q4, int N>
__global__ void __launch_bounds__(kThreads) store_kernel(const __grid_constant__ QuantArgs q) {
  const int p = blockIdx.y;
  const int64_t most = q.n * (q.head_dim / N * q.heads), step = (int64_t)gridDim.x * (kPieces * kThreads);
  bool first = true, ok = true;
  // behind the planner the rows are complete (it has waited for whoever wrote them)
  if (q.check) asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t at = (int64_t)blockIdx.x * (kPieces * kThreads) + threadIdx.x; first || at - threadIdx.x < most; at += step) {
    Piece x[kPieces];
    Raw<IO, N> raw[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      x[u] = piece_at<N>(q, p, at + u * kThreads, most, sizeof(IO));
      if (x[u].pool) raw[u].load(x[u].data, q.wide);
    }
    if (first) {
      if (q.check) {
        ok = all_in_range(q);
      } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        ok = *(volatile int32_t *)q.status == KVX_OK;
      }
      first = false;
    }
    if (!ok) return;
    const float scale = q.scale[p & 1];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if constexpr (Q4) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[u].pool ? __fmul_rn(to_f(raw[u].e[i]), scale) : 0.f;
        uint32_t pair;
        const uint32_t codes = encode(y, &pair);
        if (x[u].pool) {
          uint32_t *o = reinterpret_cast<uint32_t *>(x[u].pool);
          o[x[u].d / 8] = codes;
          if (x[u].d % KVX_Q4_GROUP == 0) o[q.head_dim / 8 + x[u].d / KVX_Q4_GROUP] = pair;
        }
      } else if (x[u].pool) {
        if constexpr (N == 8) {
          uint32_t w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            w[i] = (uint32_t)to_e4m3x2(__fmul_rn(to_f(raw[u].e[4 * i]), scale), __fmul_rn(to_f(raw[u].e[4 * i + 1]), scale)) |
                   (uint32_t)to_e4m3x2(__fmul_rn(to_f(raw[u].e[4 * i + 2]), scale), __fmul_rn(to_f(raw[u].e[4 * i + 3]), scale)) << 16;
          *reinterpret_cast<uint2 *>(x[u].pool + x[u].d) = make_uint2(w[0], w[1]);
        } else {
          x[u].pool[x[u].d] = (char)to_e4m3x2(__fmul_rn(to_f(raw[u].e[0]), scale), 0.f);
        }
      }
    }
  }
}

template <typename IO, bool Q4, int N>
__global__ void __launch_bounds__(kThreads) load_kernel(const __grid_constant__ QuantArgs q) {
  const int p = blockIdx.y;
  const int64_t most = q.n * (q.head_dim / N * q.heads), step = (int64_t)gridDim.x * (kPieces * kThreads);
  bool first = true, ok = true;
  if (q.check) asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t at = (int64_t)blockIdx.x * (kPieces * kThreads) + threadIdx.x; first || at - threadIdx.x < most; at += step) {
    Piece x[kPieces];
    uint32_t w[kPieces][2];  // codes and (scale, low), or eight E4M3 numbers
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      x[u] = piece_at<N>(q, p, at + u * kThreads, most, sizeof(IO));
      w[u][0] = w[u][1] = 0;
      if (!x[u].pool) continue;
      if constexpr (Q4) {
        const uint32_t *o = reinterpret_cast<const uint32_t *>(x[u].pool);
        w[u][0] = o[x[u].d / 8], w[u][1] = o[q.head_dim / 8 + x[u].d / KVX_Q4_GROUP];
      } else if constexpr (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(x[u].pool + x[u].d);
        w[u][0] = v.x, w[u][1] = v.y;
      } else {
        w[u][0] = (uint8_t)x[u].pool[x[u].d];
      }
    }
    if (first) {
      if (q.check) {
        ok = all_in_range(q);
      } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        ok = *(volatile int32_t *)q.status == KVX_OK;
      }
      first = false;
    }
    if (!ok) return;
    const float scale = q.scale[p & 1];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if (!x[u].pool) continue;
      Raw<IO, N> out;
      if constexpr (Q4) {
        const float s = __half2float(__ushort_as_half((uint16_t)w[u][1]));
        const float low = __half2float(__ushort_as_half((uint16_t)(w[u][1] >> 16)));
#pragma unroll
        for (int i = 0; i < 8; ++i) from_f(&out.e[i], __fmul_rn(decode(w[u][0] >> (4 * i) & 15u, s, low), scale));
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const uint32_t v = from_e4m3x2((uint16_t)(w[u][i >> 2] >> ((i & 2) * 8)));
          from_f(&out.e[i], __fmul_rn(__half2float(__ushort_as_half((uint16_t)v)), scale));
          if constexpr (N > 1)
            from_f(&out.e[i + 1], __fmul_rn(__half2float(__ushort_as_half((uint16_t)(v >> 16))), scale));
        }
      }
      out.store(x[u].data, q.wide);
    }
  }
}

template <typename IO, bool Q4, int N>
cudaError_t launch(const QuantArgs &q, bool store, cudaStream_t s) {
  const void *fn = store ? (const void *)store_kernel<IO, Q4, N> : (const void *)load_kernel<IO, Q4, N>;
  const int64_t pieces = q.n * (q.head_dim / N * q.heads), per = kPieces * kThreads;
  const int64_t grid = (pieces + per - 1) / per, most = 1 << 30;
  void *args[] = {const_cast<QuantArgs *>(&q)};
  return launch_pdl(fn, dim3((unsigned)(grid < most ? grid : most), (unsigned)q.planes), dim3(kThreads), args, s);
}

template <typename IO>
cudaError_t launch_io(const QuantArgs &q, bool store, bool q4, cudaStream_t s) {
  if (q4) return launch<IO, true, 8>(q, store, s);
  return q.words ? launch<IO, false, 8>(q, store, s) : launch<IO, false, 1>(q, store, s);
}

}  // namespace

cudaError_t launch_quant(const QuantArgs &q, bool store, bool q4, int32_t dtype, cudaStream_t s) {
  if (dtype == KVX_F16) return launch_io<__half>(q, store, q4, s);
  if (dtype == KVX_BF16) return launch_io<__nv_bfloat16>(q, store, q4, s);
  return launch_io<float>(q, store, q4, s);
}

}  // namespace kvx
