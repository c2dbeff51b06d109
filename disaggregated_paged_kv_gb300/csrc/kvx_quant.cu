// kvx_quant.cu -- rows quantised as they are written into a pool, and read back.
//
// A thread has 16 neighbouring elements of a head (8-bit pools: eight), so a 4-bit group of 32 is two lanes'.
// Which head and which elements depends on the thread alone; it takes a few tokens in turn, whose slots
// give the rows, so that an element costs a handful of instructions beside its bytes.  All rows of a turn are
// loaded before anything is waited for; as in the row copy kernel, the planner's verdict (or, for few
// tokens, the CTA's own check of every index) is looked at between the first loads and the first store: a
// call writes all or nothing.
//
// Bound: bytes, 2 + 5/8 of them an element of a 16-bit tensor and a 4-bit pool, and instructions close behind: an element
// costs about five to encode and four to decode.  2048 tokens of 36 layers of 8 heads of 128, written from bf16 and read
// back, 152 us (the bytes take 103); 20000 tokens of 28 layers of 2 heads read back 136 us (111), 5.5 TB/s.  Stores alone keep
// 69 % of the issue slots busy.  A call of few tokens is 2.3 us on the GPU, less than its host side.
#include <cuda_bf16.h>

#include <type_traits>

#include "kvx_launch.cuh"
#include "kvx_quant.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 256;

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

// Two 32-bit floats at a time.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

constexpr float kMost = 61440.f;  // what low + 15 * scale can reach without passing f16's end

// Least and greatest of a thread's elements, by pairs where they come as 16-bit numbers; NaN if any is.
template <typename IO, int N>
__device__ __forceinline__ void ends(const IO (&e)[N], float *lo, float *hi) {
  if constexpr (sizeof(IO) == 4) {
    float a = e[0], b = e[0];
#pragma unroll
    for (int i = 1; i < N; ++i) a = min_nan(a, e[i]), b = max_nan(b, e[i]);
    *lo = a, *hi = b;
  } else {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(e);
    uint32_t a = w[0], b = w[0];
#pragma unroll
    for (int i = 1; i < N / 2; ++i) {
      if constexpr (std::is_same<IO, __half>::value) {
        asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(w[i]));
        asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(b) : "r"(w[i]));
      } else {
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(w[i]));
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(w[i]));
      }
    }
    IO x[2], y[2];
    *reinterpret_cast<uint32_t *>(x) = a, *reinterpret_cast<uint32_t *>(y) = b;
    *lo = min_nan(to_f(x[0]), to_f(x[1])), *hi = max_nan(to_f(y[0]), to_f(y[1]));
  }
}

// The codes of this lane's 16 elements times mul, element i in bits 4 i .., and the group's (scale, low), which both
// lanes of the group get.  Steps are rounded one by one (no fused multiply-add), as kvx.h says.  live: the elements
// are some token's (a group's lanes agree).
template <bool SCALED, typename IO>
__device__ __forceinline__ uint64_t encode(const IO (&e)[16], bool live, float mul, uint32_t *pair) {
  float lo, hi;
  ends(e, &lo, &hi);
  lo = min_nan(lo, __shfl_xor_sync(~0u, lo, 1));
  hi = max_nan(hi, __shfl_xor_sync(~0u, hi, 1));
  if (SCALED) lo = __fmul_rn(lo, mul), hi = __fmul_rn(hi, mul);  // (mul > 0: the ends of the products)
  const bool nan = isnan(lo);
  const float least = fminf(fmaxf(lo, -kMost), kMost), most = fminf(fmaxf(hi, -kMost), kMost);
  const __half low = __float2half_rn(least);
  const float base = __half2float(low);
  const __half scale = __float2half_rn(fmaxf(__fmul_rn(__fsub_rn(most, base), 1.f / 15.f), 0.f));
  *pair = nan ? 0x7fff0000u : (uint32_t)__half_as_ushort(scale) | (uint32_t)__half_as_ushort(low) << 16;
  const float s = __half2float(scale), r = s > 0.f ? __frcp_rn(s) : 0.f;
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = to_f(e[i]);
  if (SCALED)
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], mul);
  // A code is the nearest whole number, ties to even: the low bits of c + 1.5 * 2^23.  (Clamping the ends is clamping the
  // values: codes past them are clamped here.)  No code can be below 0 where no value is below the low, none
  // above 15 where the scale is a normal number, within 2^-11 of a 15th of the reach.
  const bool plain = !nan && base <= lo && hi <= kMost && s >= 0x1p-14f;
  if (__all_sync(~0u, plain || !live)) {
    const uint64_t base2 = pair2(-base, -base), r2 = pair2(r, r);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      unpair2(mul2(add2(pair2(y[i], y[i + 1]), base2), r2), y[i], y[i + 1]);
      // (as pairs, product and sum would become one operation with one rounding)
      y[i] = __fadd_rn(y[i], 12582912.f), y[i + 1] = __fadd_rn(y[i + 1], 12582912.f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      y[i] = __fadd_rn(fminf(fmaxf(__fmul_rn(__fsub_rn(y[i], base), r), 0.f), 15.f), 12582912.f);
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 7; i >= 0; --i) w[k] = w[k] * 16u + __float_as_uint(y[8 * k + i]);
    w[k] -= 0x4b400000u * 0x11111111u;  // what 1.5 * 2^23 has left of its bits
  }
  return nan ? 0 : (uint64_t)w[1] << 32 | w[0];
}

// Eight elements from their codes, SCALED: times scale.
template <bool SCALED>
__device__ __forceinline__ void decode(uint32_t codes, float step, float low, float scale, float (&o)[8]) {
  // 2^23 + 16^i code, less 2^23, times step / 16^i: all exact, and rounded once with the low
  const uint64_t less = pair2(-8388608.f, -8388608.f), low2 = pair2(low, low), scale2 = pair2(scale, scale);
  const uint64_t step01 = pair2(step, step * 0x1p-4f), step23 = pair2(step * 0x1p-8f, step * 0x1p-12f);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w = k ? codes >> 16 : codes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t c = pair2(__uint_as_float((w & (0xfu << (8 * i))) | 0x4b000000u), __uint_as_float((w & (0xf0u << (8 * i))) | 0x4b000000u));
      uint64_t y = fma2(add2(c, less), i ? step23 : step01, low2);
      if (SCALED) y = mul2(y, scale2);
      unpair2(y, o[4 * k + 2 * i], o[4 * k + 2 * i + 1]);
    }
  }
}

// Which elements of a row a thread has, wherever the row is.
template <int N>
struct Place {
  int32_t first, step;   // its first token's place among the CTA's, and how far apart its tokens are
  int32_t d;             // first element in the head
  char *pool, *data;     // the head vector and the elements in row 0 (HND: token 0 of page 0)
  bool any;
  __device__ __forceinline__ Place(const QuantArgs &q, int p, int32_t part, int e) {
    const int32_t per_head = q.head_dim / N, per_row = per_head * q.heads;
    int32_t c = threadIdx.x;
    first = 0, step = 1;
    if (per_row < kThreads) {
      step = kThreads / per_row;
      first = c / per_row;
      c -= first * per_row;
      any = first < step;
    } else {
      c += part * kThreads;
      any = c < per_row;
    }
    const int32_t h = c / per_head;
    d = (c - h * per_head) * N;
    pool = q.base[p] + h * (int64_t)q.pool.seg_bytes * (q.pool.hnd ? q.pool.page_size : 1);
    data = (p & 1 ? q.v : q.k) + (p >> 1) * q.layer_stride + h * q.head_stride + (int64_t)d * e;
  }
};

// a * b, in one instruction where b has 31 bits.
__device__ __forceinline__ int64_t times(int32_t a, int64_t b) {
  return (b >> 31) == 0 ? (int64_t)((uint64_t)(uint32_t)a * (uint32_t)b) : a * b;
}

// A token's head vector in the pool and its elements outside; nullptr: no token, or an index out of range.
struct Row {
  char *pool, *data;
};

template <int N>
__device__ __forceinline__ Row row_at(const QuantArgs &q, const Place<N> &x, int64_t i) {
  Row r = {nullptr, nullptr};
  if (!x.any || i >= q.n) return r;
  const int32_t slot = q.slots[i], row = q.rows ? q.rows[i] : (int32_t)i;
  if ((uint32_t)slot >= (uint32_t)q.pool.num_slots || (uint32_t)row >= (uint32_t)q.n_rows) return r;
  if (q.pool.hnd) {
    const int32_t page = q.pool.ps_shift >= 0 ? slot >> q.pool.ps_shift : slot / q.pool.page_size;
    r.pool = x.pool + times(page, q.pool.page_bytes) + times(slot - page * q.pool.page_size, q.pool.seg_bytes);
  } else {
    r.pool = x.pool + times(slot, q.pool.slot_stride);
  }
  r.data = x.data + times(row, q.token_stride);
  return r;
}

// False: some index is out of range, and nothing may be written.  (For up to kSmallMaxTokens tokens: a longer
// list read by every CTA costs more than the planner's launch.)
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

// Rows of a turn, on their way together: two, which leaves registers for five CTAs an SM.  (20000 tokens of 28 layers read:
// turns of one, two and four rows 159, 133 and 153 us.  2048 tokens of 36 layers, written and read: stores of one, two,
// four and eight rows 155, 152, 156 and 185 us, with as many CTAs as they leave room for.)
template <typename IO>
constexpr int kStoreTurn = sizeof(IO) == 4 ? 1 : 2;
constexpr int kLoadTurn = 2;

// The first look at the verdict: whether anything may be written.
__device__ __forceinline__ bool may_write(const QuantArgs &q) {
  if (q.check) return all_in_range(q);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  return *(volatile int32_t *)q.status == KVX_OK;
}

// Calls f(first token of a turn) for this CTA's tokens; blockIdx.x counts them, its parts of long rows within.
template <int N, int T, typename F>
__device__ __forceinline__ void turns(const QuantArgs &q, int32_t step, F f) {
  const int64_t block = blockIdx.x / q.parts;
  for (int32_t k = 0; k < q.turns; ++k) {
    const int64_t i = (block * q.turns + k) * (T * step);
    if (i >= q.n && k > 0) return;
    if (!f(i, k == 0)) return;
  }
}

// N: elements of a thread: 16 (4-bit pools), 8, or 1 where an 8-bit pool's head vectors are no multiple of that.
template <typename IO, bool Q4, int N, bool SCALED>
__global__ void __launch_bounds__(kThreads, 5) store_kernel(const __grid_constant__ QuantArgs q) {
  constexpr int T = kStoreTurn<IO>;
  const int p = blockIdx.y;
  const Place<N> x(q, p, (int32_t)(blockIdx.x % q.parts), sizeof(IO));
  const float scale = q.scale[p & 1];
  // behind the planner the rows are complete (it has waited for whoever wrote them)
  if (q.check) asm volatile("griddepcontrol.wait;" ::: "memory");
  turns<N, T>(q, x.step, [&](int64_t i0, bool first) {
    Row r[T];
    Raw<IO, N> raw[T];
#pragma unroll
    for (int u = 0; u < T; ++u) {
      r[u] = row_at<N>(q, x, i0 + x.first + u * x.step);
      if (r[u].pool) raw[u].load(r[u].data, q.wide);
    }
    if (first && !may_write(q)) return false;
#pragma unroll
    for (int u = 0; u < T; ++u) {
      if constexpr (Q4) {
        uint32_t pair;
        const uint64_t codes = encode<SCALED>(raw[u].e, r[u].pool != nullptr, scale, &pair);
        if (r[u].pool) {
          uint32_t *o = reinterpret_cast<uint32_t *>(r[u].pool) + x.d / 8;
          if (q.words) *reinterpret_cast<uint64_t *>(o) = codes;
          else o[0] = (uint32_t)codes, o[1] = (uint32_t)(codes >> 32);
          if (x.d % KVX_Q4_GROUP == 0) reinterpret_cast<uint32_t *>(r[u].pool)[q.head_dim / 8 + x.d / KVX_Q4_GROUP] = pair;
        }
      } else if (r[u].pool) {
        if constexpr (N == 8) {
          uint32_t w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            w[i] = (uint32_t)to_e4m3x2(__fmul_rn(to_f(raw[u].e[4 * i]), scale), __fmul_rn(to_f(raw[u].e[4 * i + 1]), scale)) |
                   (uint32_t)to_e4m3x2(__fmul_rn(to_f(raw[u].e[4 * i + 2]), scale), __fmul_rn(to_f(raw[u].e[4 * i + 3]), scale)) << 16;
          *reinterpret_cast<uint2 *>(r[u].pool + x.d) = make_uint2(w[0], w[1]);
        } else {
          r[u].pool[x.d] = (char)to_e4m3x2(__fmul_rn(to_f(raw[u].e[0]), scale), 0.f);
        }
      }
    }
    return true;
  });
}

template <typename IO, bool Q4, int N, bool SCALED>
__global__ void __launch_bounds__(kThreads) load_kernel(const __grid_constant__ QuantArgs q) {
  constexpr int T = kLoadTurn;
  const int p = blockIdx.y;
  const Place<N> x(q, p, (int32_t)(blockIdx.x % q.parts), sizeof(IO));
  const float scale = q.scale[p & 1];
  if (q.check) asm volatile("griddepcontrol.wait;" ::: "memory");
  turns<N, T>(q, x.step, [&](int64_t i0, bool first) {
    Row r[T];
    uint32_t w[T][3];  // codes and (scale, low), or eight E4M3 numbers
#pragma unroll
    for (int u = 0; u < T; ++u) {
      r[u] = row_at<N>(q, x, i0 + x.first + u * x.step);
      if (!r[u].pool) continue;
      if constexpr (Q4) {
        const uint32_t *o = reinterpret_cast<const uint32_t *>(r[u].pool);
        if (q.words) {
          const uint2 v = *reinterpret_cast<const uint2 *>(o + x.d / 8);
          w[u][0] = v.x, w[u][1] = v.y;
        } else {
          w[u][0] = o[x.d / 8], w[u][1] = o[x.d / 8 + 1];
        }
        w[u][2] = o[q.head_dim / 8 + x.d / KVX_Q4_GROUP];
      } else if constexpr (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(r[u].pool + x.d);
        w[u][0] = v.x, w[u][1] = v.y;
      } else {
        w[u][0] = (uint8_t)r[u].pool[x.d];
      }
    }
    if (first && !may_write(q)) return false;
#pragma unroll
    for (int u = 0; u < T; ++u) {
      if (!r[u].pool) continue;
      Raw<IO, N> out;
      if constexpr (Q4) {
        const float s = __half2float(__ushort_as_half((uint16_t)w[u][2]));
        const float low = __half2float(__ushort_as_half((uint16_t)(w[u][2] >> 16)));
#pragma unroll
        for (int k = 0; k < N / 8; ++k) {
          float y[8];
          decode<SCALED>(w[u][k], s, low, scale, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) from_f(&out.e[8 * k + i], y[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const uint32_t v = from_e4m3x2((uint16_t)(w[u][i >> 2] >> ((i & 2) * 8)));
          from_f(&out.e[i], __fmul_rn(__half2float(__ushort_as_half((uint16_t)v)), scale));
          if constexpr (N > 1)
            from_f(&out.e[i + 1], __fmul_rn(__half2float(__ushort_as_half((uint16_t)(v >> 16))), scale));
        }
      }
      out.store(r[u].data, q.wide);
    }
    return true;
  });
}

constexpr int kSms = 152;

template <typename IO, bool Q4, int N>
cudaError_t launch(QuantArgs &q, bool store, cudaStream_t s) {
  // (an 8-bit pool's elements are multiplied in any case)
  const bool scaled = !Q4 || q.scale[0] != 1.f || q.scale[1] != 1.f;
  const void *fn = store ? (const void *)store_kernel<IO, Q4, N, true> : (const void *)load_kernel<IO, Q4, N, true>;
  if constexpr (Q4)
    if (!scaled) fn = store ? (const void *)store_kernel<IO, Q4, N, false> : (const void *)load_kernel<IO, Q4, N, false>;
  const int64_t per_row = (int64_t)(q.head_dim / N) * q.heads, turn = store ? kStoreTurn<IO> : kLoadTurn;
  const int64_t step = per_row < kThreads ? kThreads / per_row : 1;  // tokens of a pass
  q.parts = (int32_t)((per_row + kThreads - 1) / kThreads);
  const int64_t all = (q.n + turn * step - 1) / (turn * step);
  // some turns a CTA where that still leaves each SM many CTAs
  const int64_t many = all * q.parts * q.planes / (kSms * 16), least = all * q.parts / INT32_MAX + 1;  // (a grid has 31 bits)
  q.turns = (int32_t)(many < 1 ? 1 : many > 8 ? (least > 8 ? 2 * least : 8) : many);
  const int64_t grid = (all + q.turns - 1) / q.turns * q.parts;
  void *args[] = {&q};
  return launch_pdl(fn, dim3((unsigned)grid, (unsigned)q.planes), dim3(kThreads), args, s);
}

template <typename IO>
cudaError_t launch_io(QuantArgs &q, bool store, bool q4, cudaStream_t s) {
  if (q4) return launch<IO, true, 16>(q, store, s);
  return q.words ? launch<IO, false, 8>(q, store, s) : launch<IO, false, 1>(q, store, s);
}

}  // namespace

cudaError_t launch_quant(QuantArgs &q, bool store, bool q4, int32_t dtype, cudaStream_t s) {
  if (dtype == KVX_F16) return launch_io<__half>(q, store, q4, s);
  if (dtype == KVX_BF16) return launch_io<__nv_bfloat16>(q, store, q4, s);
  return launch_io<float>(q, store, q4, s);
}

}  // namespace kvx
