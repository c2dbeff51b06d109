// kvx_attn_narrow.cu -- shared attention for few rows a key: decode steps and short drafts.
//
// A piece's keys are read once and meet at most 64 rows, so the loads bound it: 4 D bytes of K
// and V a key and head against 4 D operations a row.  A CTA of four warps keeps three tiles of 64
// keys in flight with asynchronous 16-byte copies (two CTAs an SM: 128 KB of 16-bit tiles at
// D = 128), placed by page look-ups that run two tiles ahead of the copies.  The products are
// m16n8k16 ones with Q and P in registers: a warp takes 16 rows, and warps that have no rows of
// their own (16 or 32 rows in all) take other keys of the tile instead, each with its own running
// maximum and sum, joined in shared memory at the piece's end.  tcgen05 would need 128 rows.
// 8-bit keys and values go through registers, where they become the 16-bit type of q (exactly).
#include <type_traits>

#include "kvx_attn.cuh"
#include "kvx_attn_mma.cuh"
#include "kvx_launch.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 128;
constexpr int kTileKeys = kAttnKeyTile;
constexpr int kStages = 3;
constexpr int kRing = 4;  // tiles of key offsets: one more than the stages

template <int D>
struct Smem {
  alignas(128) char kv[kStages][2][kTileKeys * D * 2];
  int64_t off[kRing][kTileKeys];
  int32_t lim[kAttnNarrowRows];
  float m[4][16], l[4][16];
};

// Byte place of 16-byte chunk c of row r in a tile of D 16-bit columns: rows of eight chunks (or
// sixteen) whose low three bits are exchanged by the row, so that eight rows of one chunk lie in
// different banks.
template <int D>
__device__ __forceinline__ uint32_t place(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

template <typename T, bool FP8, int D>
struct Narrow {
  static constexpr int kChunks = D / 8;               // 16-byte chunks of a 16-bit row
  static constexpr int kRaw = FP8 ? D / 16 : D / 8;   // of a row in the pool
  static constexpr int kPer = kTileKeys * kRaw / kThreads;  // copies a thread and tile, K or V
  static constexpr int kStep = kThreads / kRaw;       // rows between a thread's copies

  const AttnParams &p;
  Smem<D> &sm;
  const int h, tid, lane, warp;
  uint4 raw[FP8 ? 2 * kPer : 1];  // 8-bit tile on its way

  __device__ __forceinline__ void load(const AttnPiece &x, int tile, int stage) {
    const int c = tid % kRaw, r0 = tid / kRaw, k0 = x.key0 + tile * kTileKeys;
    const int64_t *off = sm.off[tile % kRing];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + i * kStep;
      const bool ok = k0 + r < x.key1;
      const int64_t o = off[r] + c * 16;
      if constexpr (FP8) {
        raw[i] = ok ? __ldg(reinterpret_cast<const uint4 *>(p.pool.k + o)) : make_uint4(0, 0, 0, 0);
        raw[kPer + i] = ok ? __ldg(reinterpret_cast<const uint4 *>(p.pool.v + o)) : make_uint4(0, 0, 0, 0);
      } else {
        cp_async16(smem_u32(sm.kv[stage][0]) + place<D>(r, c), p.pool.k + o, ok);
        cp_async16(smem_u32(sm.kv[stage][1]) + place<D>(r, c), p.pool.v + o, ok);
      }
    }
  }

  // The 8-bit tile in registers to its stage, as 16-bit values.
  __device__ __forceinline__ void store_raw(int stage) {
    if constexpr (FP8) {
      const int c = tid % kRaw, r0 = tid / kRaw;
#pragma unroll
      for (int i = 0; i < 2 * kPer; ++i) {
        const int r = r0 + (i % kPer) * kStep;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[2 * k] = from_e4m3x2<T>((uint16_t)w[k]);
          o[2 * k + 1] = from_e4m3x2<T>((uint16_t)(w[k] >> 16));
        }
        char *base = sm.kv[stage][i / kPer];
        *reinterpret_cast<uint4 *>(base + place<D>(r, 2 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(base + place<D>(r, 2 * c + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }

  // RG groups of 16 rows; 4 / RG warps share the keys of a tile for each.
  template <int RG>
  __device__ __forceinline__ void piece(const AttnPiece &x) {
    constexpr int KP = 4 / RG, NB = RG;  // NB blocks of 16 keys a warp and tile
    const int rg = warp % RG, kp = warp / RG, c4 = lane & 3, r8 = lane >> 2;
    __syncthreads();  // the piece before has left the shared memory
    if (tid < 16 * RG) sm.lim[tid] = tid < x.rows ? p.limit[(x.row0 + tid) / p.group] : 0;
    // where the piece ends for its longest row, and from where on rows differ: rows whose mask
    // leaves nothing of the piece do not count, their sums are dropped at the end
    __syncthreads();
    int most = 0, least = INT32_MAX;
    for (int r = 0; r < x.rows; ++r) {
      const int v = sm.lim[r];
      most = max(most, v);
      if (v > x.key0) least = min(least, v);
    }
    AttnPiece y = x;
    y.key1 = min(x.key1, most);
    const int nt = max(0, (y.key1 - x.key0 + kTileKeys - 1) / kTileKeys);
    const int lim0 = sm.lim[rg * 16 + r8], lim1 = sm.lim[rg * 16 + r8 + 8];

    // page look-ups: thread j < 64 does key j of each tile
    auto look = [&](int tile) -> int64_t {
      const int pos = y.key0 + tile * kTileKeys + tid;
      return tid < kTileKeys && pos < y.key1
                 ? attn_key_offset(p, y.table, pos) + h * p.pool.head_stride : 0;
    };
    for (int t = 0; t < kStages && t < nt; ++t) {
      const int64_t o = look(t);
      if (tid < kTileKeys) sm.off[t][tid] = o;
    }
    int64_t next = look(kStages);
    __syncthreads();

    if constexpr (!FP8) {
#pragma unroll
      for (int t = 0; t < kStages - 1; ++t) {
        if (t < nt) load(y, t, t);
        cp_async_commit();
      }
    } else if (nt > 0) {
      load(y, 0, 0);
      store_raw(0);
      if (nt > 1) load(y, 1, 1);
    }

    uint32_t q[D / 16][4];
    {
      const int ra = rg * 16 + r8, rb = ra + 8;
      const T *qa = nullptr, *qb = nullptr;
      auto at = [&](int r) {
        const int row = x.row0 + r, t = row / p.group;
        return reinterpret_cast<const T *>(p.q + t * p.q_tok + (int64_t)(h * p.group + row - t * p.group) * p.q_head);
      };
      if (ra < x.rows) qa = at(ra);
      if (rb < x.rows) qb = at(rb);
      auto get = [&](const T *s, int d) -> uint32_t {
        if (!s) return 0;
        const uint16_t *u = reinterpret_cast<const uint16_t *>(s) + d;
        if (p.q_even) return *reinterpret_cast<const uint32_t *>(u);
        return u[0] | (uint32_t)u[1] << 16;
      };
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][0] = get(qa, k * 16 + 2 * c4);
        q[k][1] = get(qb, k * 16 + 2 * c4);
        q[k][2] = get(qa, k * 16 + 2 * c4 + 8);
        q[k][3] = get(qb, k * 16 + 2 * c4 + 8);
      }
    }

    float o[D / 8][4] = {}, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int odd = 0;
    for (int t = 0; t < nt; ++t) {
      const int stage = t % kStages;
      if constexpr (!FP8) cp_async_wait<kStages - 2>();
      __syncthreads();  // tile t is there, and everyone is done with tile t - 1
      if constexpr (!FP8) {
        if (t + kStages - 1 < nt) load(y, t + kStages - 1, (t + kStages - 1) % kStages);
        cp_async_commit();
      } else {
        if (t + 1 < nt) store_raw((t + 1) % kStages);
        if (t + 2 < nt) load(y, t + 2, 0);
      }
      if (tid < kTileKeys) sm.off[(t + kStages) % kRing][tid] = next;
      next = look(t + kStages + 1);
      const int k0 = y.key0 + t * kTileKeys;
      if (k0 + kTileKeys > least && least < y.key1) {
        // some row's mask falls into the tile: what it hides must not meet the row's weight of 0
        // as an infinity or NaN, so such values are taken out here and added to the rows that do
        // see them at the end
        for (int i = tid; i < kTileKeys * kChunks; i += kThreads) {
          uint4 *v = reinterpret_cast<uint4 *>(sm.kv[stage][1]) + i;
          uint32_t w[4] = {v->x, v->y, v->z, v->w};
          bool any = false;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (odd2<T>(w[k])) {
              if (odd2<T>(w[k] & 0xffffu)) w[k] &= 0xffff0000u;
              if (odd2<T>(w[k] & 0xffff0000u)) w[k] &= 0xffffu;
              any = true;
            }
          if (any) *v = make_uint4(w[0], w[1], w[2], w[3]), odd = 1;
        }
        __syncthreads();
      }

      const uint32_t kb = smem_u32(sm.kv[stage][0]), vb = smem_u32(sm.kv[stage][1]);
      float s[NB][2][4];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int row = (kp * NB + b) * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[b][n][i] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t kf[4];
          ldmatrix4(kf, kb + place<D>(row, k * 2 + ((lane >> 3) & 1)));
          mma16816<T>(s[b][0], q[k], kf[0], kf[1]);
          mma16816<T>(s[b][1], q[k], kf[2], kf[3]);
        }
      }
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = k0 + (kp * NB + b) * 16 + n * 8 + 2 * c4 + i;
            s[b][n][i] = key < lim0 && key < y.key1 ? s[b][n][i] * p.scale_log2 : -INFINITY;
            s[b][n][i + 2] = key < lim1 && key < y.key1 ? s[b][n][i + 2] * p.scale_log2 : -INFINITY;
            t0 = fmaxf(t0, s[b][n][i]);
            t1 = fmaxf(t1, s[b][n][i + 2]);
          }
      t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, 1));
      t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, 1));
      t0 = fmaxf(fmaxf(t0, __shfl_xor_sync(~0u, t0, 2)), m0);
      t1 = fmaxf(fmaxf(t1, __shfl_xor_sync(~0u, t1, 2)), m1);
      if (__any_sync(~0u, t0 > m0 || t1 > m1)) {
        const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - t0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - t1);
        l0 *= f0, l1 *= f1;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
        m0 = t0, m1 = t1;
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t a[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            s[b][n][i] = ex2(s[b][n][i] - b0);
            s[b][n][i + 2] = ex2(s[b][n][i + 2] - b1);
            l0 += s[b][n][i];
            l1 += s[b][n][i + 2];
          }
          // the weights are rounded to the values' type for the product; their sum is not
          a[2 * n] = pack2<T>(s[b][n][0], s[b][n][1]);
          a[2 * n + 1] = pack2<T>(s[b][n][2], s[b][n][3]);
        }
        const int row = (kp * NB + b) * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t vf[4];
          ldmatrix4t(vf, vb + place<D>(row, n * 2 + (lane >> 4)));
          mma16816<T>(o[2 * n], a, vf[0], vf[1]);
          mma16816<T>(o[2 * n + 1], a, vf[2], vf[3]);
        }
      }
    }
    l0 += __shfl_xor_sync(~0u, l0, 1);
    l1 += __shfl_xor_sync(~0u, l1, 1);
    l0 += __shfl_xor_sync(~0u, l0, 2);
    l1 += __shfl_xor_sync(~0u, l1, 2);

    // the warps' parts through shared memory (over the tiles) to the piece's place
    if constexpr (!FP8) cp_async_wait<0>();
    odd = __syncthreads_or(odd);
    constexpr int kPitch = D + 4;
    float *so = reinterpret_cast<float *>(&sm.kv[0][0][0]);
    static_assert(4 * 16 * (D + 4) * 4 <= kStages * 2 * kTileKeys * D * 2, "the parts fit the tiles");
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      float *a = so + (warp * 16 + r8) * kPitch + n * 8 + 2 * c4;
      a[0] = o[n][0], a[1] = o[n][1];
      a[8 * kPitch] = o[n][2], a[8 * kPitch + 1] = o[n][3];
    }
    if (c4 == 0) {
      sm.m[warp][r8] = m0, sm.m[warp][r8 + 8] = m1;
      sm.l[warp][r8] = l0, sm.l[warp][r8 + 8] = l1;
    }
    __syncthreads();
    for (int i = tid; i < x.rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i - r * (D / 4)) * 4, g = r >> 4, rr = r & 15;
      float top = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < KP; ++k) top = fmaxf(top, sm.m[k * RG + g][rr]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < KP; ++k) {
        const int w = k * RG + g;
        if (sm.l[w][rr] == 0.f) continue;  // saw nothing: its sums may be anything times 0
        const float f = ex2(sm.m[w][rr] - top);
        const float4 v = *reinterpret_cast<const float4 *>(so + (w * 16 + rr) * kPitch + d);
        acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
        l = fmaf(f, sm.l[w][rr], l);
      }
      if (odd) {  // infinities and NaN that were taken out, for the rows that see them
        const int end = min(sm.lim[r], y.key1);
        const int from = y.key0 + (max(least, y.key0) - y.key0) / kTileKeys * kTileKeys;
        for (int key = from; key < end; ++key) {
          const char *v = p.pool.v + attn_key_offset(p, y.table, key) + h * p.pool.head_stride;
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (FP8) {
              const uint32_t u = from_e4m3x2<__half>(reinterpret_cast<const uint8_t *>(v)[d + k]);
              e[k] = __half2float(*reinterpret_cast<const __half *>(&u));
            } else {
              e[k] = (float)reinterpret_cast<const T *>(v)[d + k];
            }
            e[k] = isfinite(e[k]) ? 0.f : e[k];
          }
          acc.x += e[0], acc.y += e[1], acc.z += e[2], acc.w += e[3];
        }
      }
      *reinterpret_cast<float4 *>(p.part_o + (x.part + r) * D + d) = acc;
      if (d == 0) p.part_m[x.part + r] = top, p.part_l[x.part + r] = l;
    }
  }
};

template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kThreads, 2) attn_narrow_kernel(const AttnParams p) {
  extern __shared__ char raw_smem[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw_smem);
  attn_wait_prior();
  const int g = blockIdx.x / p.kv_heads, h = blockIdx.x - g * p.kv_heads, tid = threadIdx.x;
  Narrow<T, FP8, D> n{p, sm, h, tid, tid & 31, tid >> 5, {}};
  attn_pieces(p, g, h, [&](const AttnPiece &x) {
    if (x.rows <= 16) n.template piece<1>(x);
    else if (x.rows <= 32) n.template piece<2>(x);
    else n.template piece<4>(x);
  });
}

template <typename T, bool FP8, int D>
cudaError_t launch(const AttnParams &p, cudaStream_t s) {
  const void *fn = (const void *)attn_narrow_kernel<T, FP8, D>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  void *args[] = {const_cast<AttnParams *>(&p)};
  return launch_pdl(fn, dim3(p.groups * p.kv_heads), dim3(kThreads), args, s, sizeof(Smem<D>));
}

template <typename T, bool FP8>
cudaError_t launch_d(const AttnParams &p, cudaStream_t s) {
  return p.head_dim == 64 ? launch<T, FP8, 64>(p, s) : launch<T, FP8, 128>(p, s);
}

}  // namespace

cudaError_t launch_attn_narrow(const AttnParams &p, int32_t dtype, int32_t io, cudaStream_t s) {
  if (dtype == KVX_F16) return launch_d<__half, false>(p, s);
  if (dtype == KVX_BF16) return launch_d<__nv_bfloat16, false>(p, s);
  if (io == KVX_F16) return launch_d<__half, true>(p, s);
  return launch_d<__nv_bfloat16, true>(p, s);
}

}  // namespace kvx
