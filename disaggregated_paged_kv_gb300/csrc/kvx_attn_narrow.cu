// kvx_attn_narrow.cu -- shared attention for few rows a key: decode steps and short drafts.
//
// A piece's keys are read once and meet at most 64 rows, so the loads bound it: 4 D bytes of K
// and V a key and head (16-bit pool) against 4 D operations a row.  A CTA has four producer warps that
// fill a ring of tiles of 64 keys and run on into the next piece, and four consumer warps; two
// CTAs an SM keep about 190 KB of tiles in the ring.  A tile comes by tensor copies, one a page and
// head; tiles that end inside a page or mix two tables, and pages that are no multiple of eight
// tokens, come by 16-byte copies key by key.
//
// The products are m16n8k16 ones with Q and P in registers (tcgen05 would need 128 rows): a warp
// takes 16 rows, and warps without rows of their own (16 or 32 rows in all) take other keys of the
// tile, each with its own running maximum and sum, joined in shared memory at the piece's end.
//
// Measured: 64 decode requests of 1500 own tokens (bf16, 8 kv heads of 4 rows, 128 columns) behind 2048
// shared ones 92 us, the prefix beside it in the wide kernel; where it has all SMs it reads 1.57 GB at 6.2
// TB/s, 92 % of a plain copy's rate.
//
// 8-bit pools: E4M3 values become f16 in registers, exactly.  Queries become f16 too, each row
// scaled by a power of two so that its greatest element is below 2^15: what falls below f16's range
// then is less than 2^-39 of that element.
#include <type_traits>

#include "kvx_attn.cuh"
#include "kvx_attn_mma.cuh"
#include "kvx_attn_tma.cuh"
#include "kvx_launch.cuh"

namespace kvx {
namespace {

constexpr int kConsumers = 128;
constexpr int kThreads = kConsumers + 128;
constexpr int kTileKeys = kAttnKeyTile;

template <bool FP8, int D>
struct Smem {
  static constexpr int kTile = kTileKeys * D * (FP8 ? 1 : 2);  // bytes of K, and of V
  static constexpr int kStages = 98304 / (2 * kTile) < 6 ? 98304 / (2 * kTile) : 6;
  alignas(1024) char kv[kStages][2][kTile];
  float part[2][D / 4][32];  // half of a warp's sums, on their way to the warp that adds them up
  float ml[2][5][32];
  int64_t scan[2 * (kThreads / 32) + 4];
  uint64_t full[kStages], empty[kStages];
  int32_t lost, error;
};

// Byte place of 16-byte chunk c of row r in a tile as it comes.
template <bool FP8, int D>
__device__ __forceinline__ uint32_t spot(int r, int c) {
  if constexpr (FP8) return place8<D>(r, c);
  else return place<D>(r, c);
}

// Loads two neighbouring 16-bit elements; even: their address is a multiple of four.
__device__ __forceinline__ uint32_t load2(const char *s, int d, bool even) {
  const uint16_t *u = reinterpret_cast<const uint16_t *>(s) + d;
  if (even) return *reinterpret_cast<const uint32_t *>(u);
  return u[0] | (uint32_t)u[1] << 16;
}

template <typename IO, bool FP8, int D>
struct Consumer {
  using T = typename std::conditional<FP8, __half, IO>::type;  // of the products
  using S = Smem<FP8, D>;
  static constexpr float kShift = weight_shift<T>(0.f);
  const AttnParams &p;
  S &sm;
  const int h, lane, warp;
  int stage;
  uint32_t phase;

  // RG groups of 16 rows; 4 / RG warps share the keys of a tile for each.
  template <int RG>
  __device__ __forceinline__ void piece(const AttnPiece &x) {
    constexpr int KP = 4 / RG;
    constexpr int NB = RG < 2 ? 1 : 2;      // blocks of 16 keys at a time
    constexpr int kSteps = RG / NB;         // and how often that is a tile
    const int rg = warp % RG, kp = warp / RG, c4 = lane & 3, r8 = lane >> 2;
    const int ra = rg * 16 + r8, rb = ra + 8;
    const char *qa = nullptr, *qb = nullptr;
    int lim0 = 0, lim1 = 0;
    {
      auto at = [&](int r, int *lim) {
        const int row = x.row0 + r, t = row / p.group;
        *lim = min(attn_limit(p, t), x.key1);
        return p.q + t * p.q_tok + (int64_t)(h * p.group + row - t * p.group) * p.q_head;
      };
      if (ra < x.rows) qa = at(ra, &lim0);
      if (rb < x.rows) qb = at(rb, &lim1);
    }
    // 8-bit pools: columns 4 c4 .. 4 c4 + 3 of a block, as the keys' fragments have them
    uint32_t q[D / 16][4];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int d0 = k * 16 + (FP8 ? 4 : 2) * c4, d1 = d0 + (FP8 ? 2 : 8);
      q[k][0] = qa ? load2(qa, d0, p.q_even) : 0;
      q[k][1] = qb ? load2(qb, d0, p.q_even) : 0;
      q[k][2] = qa ? load2(qa, d1, p.q_even) : 0;
      q[k][3] = qb ? load2(qb, d1, p.q_even) : 0;
    }
    float sc0 = p.scale_log2, sc1 = p.scale_log2;
    if constexpr (FP8 && std::is_same<IO, __nv_bfloat16>::value) {
      uint32_t ma = 0, mb = 0;  // greatest magnitudes, by their bits
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        ma = max(ma, max(max(q[k][0] & 0x7fffu, q[k][0] >> 16 & 0x7fffu), max(q[k][2] & 0x7fffu, q[k][2] >> 16 & 0x7fffu)));
        mb = max(mb, max(max(q[k][1] & 0x7fffu, q[k][1] >> 16 & 0x7fffu), max(q[k][3] & 0x7fffu, q[k][3] >> 16 & 0x7fffu)));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        ma = max(ma, __shfl_xor_sync(~0u, ma, o));
        mb = max(mb, __shfl_xor_sync(~0u, mb, o));
      }
      const float fa = half_scale(ma, &sc0), fb = half_scale(mb, &sc1);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = i & 1 ? fb : fa;
          q[k][i] = pack2<__half>(__uint_as_float(q[k][i] << 16) * f, __uint_as_float(q[k][i] & 0xffff0000u) * f);
        }
    }
    // from where on rows of this warp differ in what they see; rows whose mask leaves nothing of
    // the piece do not count, their sums are dropped at the end
    int least = INT32_MAX;
    if (lim0 > x.key0) least = lim0;
    if (lim1 > x.key0) least = min(least, lim1);
    for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(~0u, least, o));
    if (least >= x.key1) least = INT32_MAX;

    float o[D / 8][4] = {}, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int odd = 0;
    for (int k0 = x.key0; k0 < x.key1; k0 += kTileKeys) {
      bar_wait(&sm.full[stage], phase, &sm.lost, &sm.error);  // (given up: what follows is of no account)
      __syncwarp();
      const uint32_t kb = smem_u32(sm.kv[stage][0]), vb = smem_u32(sm.kv[stage][1]);
      const bool mixed = k0 + kTileKeys > least;
#pragma unroll
      for (int step = 0; step < kSteps; ++step) {
        const int b0 = (kp * kSteps + step) * NB;  // first block of 16 keys
        const int low = max(x.low - k0, 0);        // keys of the tile before the seg's first
        float s[NB][2][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][n][i] = 0.f;
          const int row = (b0 + b) * 16 + (lane & 7) + ((lane >> 4) << 3);
          if constexpr (FP8) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t f[4];
              ldmatrix4(f, kb + place8<D>(row, k * 2 + ((lane >> 3) & 1)));
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  mma16816<T>(s[b][n], q[2 * k + e], from_e4m3x2((uint16_t)f[2 * n + e]),
                              from_e4m3x2((uint16_t)(f[2 * n + e] >> 16)));
            }
          } else {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t f[4];
              ldmatrix4(f, kb + place<D>(row, k * 2 + ((lane >> 3) & 1)));
              mma16816<T>(s[b][0], q[k], f[0], f[1]);
              mma16816<T>(s[b][1], q[k], f[2], f[3]);
            }
          }
        }
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int key = (b0 + b) * 16 + n * 8 + 2 * c4 + i;
              s[b][n][i] = key < lim0 - k0 && key >= low ? s[b][n][i] * sc0 : -INFINITY;
              s[b][n][i + 2] = key < lim1 - k0 && key >= low ? s[b][n][i + 2] * sc1 : -INFINITY;
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
        const float base0 = m0 == -INFINITY ? 0.f : m0 - kShift, base1 = m1 == -INFINITY ? 0.f : m1 - kShift;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t a[4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s[b][n][i] = ex2(s[b][n][i] - base0);
              s[b][n][i + 2] = ex2(s[b][n][i + 2] - base1);
              l0 += s[b][n][i];
              l1 += s[b][n][i + 2];
            }
            // the weights are rounded to the values' type for the product; their sum is not
            a[2 * n] = pack2<T>(s[b][n][0], s[b][n][1]);
            a[2 * n + 1] = pack2<T>(s[b][n][2], s[b][n][3]);
          }
          const int row = (b0 + b) * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
          for (int n = 0; n < D / 16; n += FP8 ? 2 : 1) {
            uint32_t f[4];
            if constexpr (FP8) {
              // 16 columns as pairs of bytes: a register has two keys of an even and an odd column
              ldmatrix4t(f, vb + place8<D>(row, n + (lane >> 4)));
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t u = __byte_perm(f[e], 0, 0x3120);
                v[2 * e] = from_e4m3x2((uint16_t)u);
                v[2 * e + 1] = from_e4m3x2((uint16_t)(u >> 16));
              }
              if (mixed)
#pragma unroll
                for (int e = 0; e < 8; ++e) odd |= clean2(v[e]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                mma16816<T>(o[2 * n + 2 * e], a, v[4 * e], v[4 * e + 2]);
                mma16816<T>(o[2 * n + 2 * e + 1], a, v[4 * e + 1], v[4 * e + 3]);
              }
            } else {
              ldmatrix4t(f, vb + place<D>(row, n * 2 + (lane >> 4)));
              if (mixed)
#pragma unroll
                for (int e = 0; e < 4; ++e) odd |= clean2(f[e]);
              mma16816<T>(o[2 * n], a, f[0], f[1]);
              mma16816<T>(o[2 * n + 1], a, f[2], f[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&sm.empty[stage]);
      if (++stage == S::kStages) stage = 0, phase ^= 1;
    }
    l0 += __shfl_xor_sync(~0u, l0, 1);
    l1 += __shfl_xor_sync(~0u, l1, 1);
    l0 += __shfl_xor_sync(~0u, l0, 2);
    l1 += __shfl_xor_sync(~0u, l1, 2);
    odd = __any_sync(~0u, odd);

    // warps that shared the rows' keys: the upper half of them hands its sums to the lower half
#pragma unroll
    for (int half = KP / 2; half >= 1; half >>= 1) {
      const bool gives = kp >= half && kp < 2 * half, takes = kp < half;
      const int slot = RG == 2 ? rg : kp % half;
      float f0 = 1.f, f1 = 1.f, g0 = 0.f, g1 = 0.f;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (gives) {
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sm.part[slot][n * 4 + i][lane] = o[part * (D / 16) + n][i];
          if (part == 0) {
            sm.ml[slot][0][lane] = m0, sm.ml[slot][1][lane] = m1, sm.ml[slot][2][lane] = l0;
            sm.ml[slot][3][lane] = l1, sm.ml[slot][4][lane] = __int_as_float(odd);
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (takes) {
          if (part == 0) {
            const float n0 = sm.ml[slot][0][lane], n1 = sm.ml[slot][1][lane];
            const float k0 = sm.ml[slot][2][lane], k1 = sm.ml[slot][3][lane];
            odd |= __float_as_int(sm.ml[slot][4][lane]);
            const float t0 = fmaxf(m0, n0), t1 = fmaxf(m1, n1);
            // a sum of 0: nothing was seen, and what the products left may be anything times 0
            f0 = l0 == 0.f ? 0.f : ex2(m0 - t0), f1 = l1 == 0.f ? 0.f : ex2(m1 - t1);
            g0 = k0 == 0.f ? 0.f : ex2(n0 - t0), g1 = k1 == 0.f ? 0.f : ex2(n1 - t1);
            if (l0 == 0.f)
#pragma unroll
              for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = 0.f;
            if (l1 == 0.f)
#pragma unroll
              for (int n = 0; n < D / 8; ++n) o[n][2] = o[n][3] = 0.f;
            l0 = l0 * f0 + k0 * g0, l1 = l1 * f1 + k1 * g1;
            if (k0 == 0.f) g0 = 0.f;
            m0 = t0, m1 = t1;
          }
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            float(&a)[4] = o[part * (D / 16) + n];
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = sm.part[slot][n * 4 + i][lane];
            a[0] = a[0] * f0 + (g0 == 0.f ? 0.f : g0 * v[0]), a[1] = a[1] * f0 + (g0 == 0.f ? 0.f : g0 * v[1]);
            a[2] = a[2] * f1 + (g1 == 0.f ? 0.f : g1 * v[2]), a[3] = a[3] * f1 + (g1 == 0.f ? 0.f : g1 * v[3]);
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
    }
    if (kp != 0) return;
    if (l0 == 0.f)
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = 0.f;
    if (l1 == 0.f)
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][2] = o[n][3] = 0.f;
    if (odd) {  // infinities and NaN that were taken out, for the rows that see them
      for (int key = max(x.low, x.key0 + (least - x.key0) / kTileKeys * kTileKeys); key < x.key1; ++key) {
        const char *v = p.pool.v + attn_key_offset(p, x.table, key, &sm.error) + h * p.pool.head_stride;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float e;
            if constexpr (FP8) {
              const uint32_t u = from_e4m3x2(reinterpret_cast<const uint8_t *>(v)[column(n, i, c4)]);
              e = __half2float(*reinterpret_cast<const __half *>(&u));
            } else {
              e = (float)reinterpret_cast<const T *>(v)[column(n, i, c4)];
            }
            if (!isfinite(e)) {
              if (key < lim0) o[n][i] += e;
              if (key < lim1) o[n][i + 2] += e;
            }
          }
      }
    }
#pragma unroll
    for (int up = 0; up < 2; ++up) {
      if ((up ? rb : ra) >= x.rows) continue;
      const int64_t at = x.part + (up ? rb : ra);
      float *d = p.part_o + at * D;
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        if constexpr (FP8)
          *reinterpret_cast<float4 *>(d + n * 8 + 4 * c4) =
              make_float4(o[n][2 * up], o[n + 1][2 * up], o[n][2 * up + 1], o[n + 1][2 * up + 1]);
        else
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2 *>(d + (n + e) * 8 + 2 * c4) = make_float2(o[n + e][2 * up], o[n + e][2 * up + 1]);
      }
      if (c4 == 0) p.part_m[at] = (up ? m1 : m0) - kShift, p.part_l[at] = up ? l1 : l0;
    }
  }

  // The column that element i of sum n has in this lane.
  static __device__ __forceinline__ int column(int n, int i, int c4) {
    return FP8 ? (n >> 1) * 16 + 4 * c4 + 2 * i + (n & 1) : n * 8 + 2 * c4 + i;
  }

  // Takes infinities and NaN out of a packed pair; 1 if there were any.
  static __device__ __forceinline__ int clean2(uint32_t &w) {
    if (!odd2<T>(w)) return 0;
    if (odd2<T>(w & 0xffffu)) w &= 0xffff0000u;
    if (odd2<T>(w & 0xffff0000u)) w &= 0xffffu;
    return 1;
  }
};

template <typename IO, bool FP8, int D>
__global__ void __launch_bounds__(kThreads, 2)
attn_narrow_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnTma tma,
                   const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ char raw_smem[];
  using S = Smem<FP8, D>;
  S &sm = *reinterpret_cast<S *>(raw_smem + (-smem_u32(raw_smem) & 1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) bar_init(&sm.full[i], 128), bar_init(&sm.empty[i], 4);
    sm.lost = sm.error = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (!p.after_wide) attn_wait_prior();
  else if (tid == 0) attn_wait_announced(p);  // for the others by the barrier below
  const int g = blockIdx.x / p.kv_heads, h = blockIdx.x - g * p.kv_heads;
  __syncthreads();
  const AttnLine line = attn_line<kThreads>(p, g, sm.scan);
  attn_release_next();  // the join takes its place as CTAs end, and waits for the last
  int stage = 0;        // of the producers
  uint32_t phase = 1;

  if (warp < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    Consumer<IO, FP8, D> c{p, sm, h, lane, warp, 0, 0};
    attn_pieces(p, g, h, line, [&](const AttnPiece &x) {
      if (x.rows <= 16) c.template piece<1>(x);
      else if (x.rows <= 32) c.template piece<2>(x);
      else c.template piece<4>(x);
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // (no kernel's end lies between the pool's writes and these copies)
    if (p.after_wide) asm volatile("fence.proxy.async.global;" ::: "memory");
    constexpr int kRaw = FP8 ? D / 16 : D / 8;  // 16-byte chunks of a row
    constexpr int kPer = 32 / kRaw;             // rows of a copy of all lanes
    // lane pairs (K and V) of the warps take the boxes of a tile in turn
    const int boxes = tma.rows > 0 ? kTileKeys / tma.rows : 1, kv = lane & 1, pw = warp - 4;
    const int box = (lane >> 1) * 4 + pw;
    bool lost = false;  // a wait was given up: nothing more is sent on its way
    attn_pieces(p, g, h, line, [&](const AttnPiece &x) {
      if (lost) return;
      const int tiles = (x.key1 - x.key0 + kTileKeys - 1) / kTileKeys;
      // a tile of keys that all count (its boxes each lie in a page: tiles begin at multiples of them)
      auto regular = [&](int j) {
        return tma.rows > 0 && x.key0 + j * kTileKeys >= x.low && x.key0 + (j + 1) * kTileKeys <= x.key1;
      };
      // look-ups a tile ahead: the page of this lane's box, or of key 16 pw + lane % 16
      auto look = [&](int j) -> int32_t {
        if (j >= tiles) return 0;
        const bool reg = regular(j);
        const int pos = x.key0 + j * kTileKeys + (reg ? box * tma.rows : pw * 16 + (lane & 15));
        if (reg ? box >= boxes : pos < x.low || pos >= x.key1) return 0;
        int pg, o;
        attn_split(p, pos, &pg, &o);
        return attn_entry(p, x.table, pg);
      };
      int32_t next = look(0);
      for (int j = 0; j < tiles; ++j) {
        const int32_t id = next;
        next = look(j + 1);
        lost = !__all_sync(~0u, bar_wait(&sm.empty[stage], phase, &sm.lost, &sm.error));
        if (lost) return;
        if (regular(j)) {
          // (a box may arrive before the tile's bytes are announced: the stage is not full before
          // thread 0 has arrived)
          if (tid == kConsumers) bar_expect(&sm.full[stage], 2 * S::kTile);
          if (box < boxes) {
            char *dst = sm.kv[stage][kv] + box * tma.rows * D * (FP8 ? 1 : 2);
            int pg, o;
            attn_split(p, x.key0 + j * kTileKeys + box * tma.rows, &pg, &o);
            const int row = (int)(attn_checked(p, id, &sm.error) * tma.page_y + h * tma.head_y + o);
            if constexpr (FP8) tma_load(dst, kv ? &v_map : &k_map, h * tma.head_x, row, &sm.full[stage]);
            else tma_load4(dst, kv ? &v_map : &k_map, h * tma.head_x, row >> 3, &sm.full[stage]);
          }
          if (tid != kConsumers) bar_arrive(&sm.full[stage]);
        } else {
          const int c = lane % kRaw, pos = x.key0 + j * kTileKeys + pw * 16 + (lane & 15);
          int64_t off = -1;
          if (pos >= x.low && pos < x.key1) {
            int pg, o;
            attn_split(p, pos, &pg, &o);
            off = attn_checked(p, id, &sm.error) * p.pool.page_stride + o * p.pool.tok_stride + h * p.pool.head_stride;
          }
          const uint32_t kd = smem_u32(sm.kv[stage][0]), vd = smem_u32(sm.kv[stage][1]);
#pragma unroll
          for (int i = 0; i < 16 / kPer; ++i) {
            const int r = i * kPer + lane / kRaw;
            const int64_t at = __shfl_sync(~0u, off, r);
            const bool ok = at >= 0;
            cp_async16(kd + spot<FP8, D>(pw * 16 + r, c), p.pool.k + (ok ? at : 0) + c * 16, ok);
            cp_async16(vd + spot<FP8, D>(pw * 16 + r, c), p.pool.v + (ok ? at : 0) + c * 16, ok);
          }
          // this thread's arrival when its copies are there
          asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&sm.full[stage])) : "memory");
        }
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
    });
    cp_async_commit();
    cp_async_wait<0>();
  }
  __syncthreads();
  if (sm.lost) {
    if (warp >= 4) bar_drain<S::kStages>(sm.full, stage, phase);
    __syncthreads();
  }
  if (tid == 0) p.errors[blockIdx.x] = sm.error;
  if (p.after_wide) attn_wait_prior();  // the join's wait for this kernel covers the wide one as well
}

template <typename IO, bool FP8, int D>
cudaError_t launch(const AttnParams &p, bool hnd, cudaStream_t s) {
  const void *fn = (const void *)attn_narrow_kernel<IO, FP8, D>;
  constexpr int kSmem = (int)sizeof(Smem<FP8, D>) + 1024;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  AttnTma tma;
  CUtensorMap km, vm;
  attn_make_tma(p, kTileKeys, FP8, hnd, &tma, &km, &vm);
  void *args[] = {const_cast<AttnParams *>(&p), &tma, &km, &vm};
  return launch_pdl(fn, dim3(p.groups * p.kv_heads), dim3(kThreads), args, s, kSmem);
}

template <typename IO, bool FP8>
cudaError_t launch_d(const AttnParams &p, bool hnd, cudaStream_t s) {
  return p.head_dim == 64 ? launch<IO, FP8, 64>(p, hnd, s) : launch<IO, FP8, 128>(p, hnd, s);
}

}  // namespace

cudaError_t launch_attn_narrow(const AttnParams &p, int32_t dtype, int32_t io, bool hnd, cudaStream_t s) {
  if (dtype == KVX_F16) return launch_d<__half, false>(p, hnd, s);
  if (dtype == KVX_BF16) return launch_d<__nv_bfloat16, false>(p, hnd, s);
  if (io == KVX_F16) return launch_d<__half, true>(p, hnd, s);
  return launch_d<__nv_bfloat16, true>(p, hnd, s);
}

}  // namespace kvx
