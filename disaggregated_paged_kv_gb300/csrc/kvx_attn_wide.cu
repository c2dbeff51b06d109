// kvx_attn_wide.cu -- shared attention for many rows a key: the prefix of a batch, and prompts.
//
// A CTA (one per SM) has a unit of two tiles of 128 rows and walks its keys in tiles of 128.  Both
// products run on the 5th-generation tensor cores with their sums in tensor memory (512 columns):
// S = Q K^T of either row tile (128 columns each) and O += P V (head_dim columns each); the weights
// P overlay the first half of their S as 16-bit values and are the product's A operand from there.
// The two row tiles alternate: while one's scores become weights, the tensor cores work for the
// other.  Warps 0-3 and 4-7 do the softmax of the tiles (a thread a row, so no exchange between
// threads), warps 8-11 bring in the queries and the keys and values by page look-up, warp 12
// issues the products.
//
// Bound: 4 D operations a score on the tensor cores (1024 cycles for 128 x 128 scores at D = 128)
// against one exponential and about five instructions a score on four warps.  Measured: eight prompts
// behind a shared prefix, 842 GFLOP in all, 682-708 us with the plan and the join (1.19-1.23 PFLOP/s); the tensor
// cores are busy 61-64 % of this kernel's time and wait for weights in the rest.  Two threads a row, each with
// half of its keys, took longer (749 against 704 us then).
//
// A row's sums refer to a maximum that is renewed only when a score passes it by 2^8 (f16: 2^2): the factor
// between the two cancels in the quotient, weights stay in range (see weight_shift), and the sums in
// tensor memory are rescaled a few times in all instead of with every tile.
#include <cuda.h>

#include <type_traits>

#include "kvx_attn.cuh"
#include "kvx_attn_mma.cuh"
#include "kvx_attn_tma.cuh"
#include "kvx_launch.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 512;
constexpr int kKeys = kAttnWideKeys;

template <bool FP8, int D>
struct Smem {
  static constexpr int kStages = FP8 ? 3 : 5;  // of one K or V tile each, as 16-bit values
  static constexpr int kRawStages = FP8 ? 3 : 1;
  alignas(1024) char q[2][128 * D * 2];
  alignas(1024) char kv[kStages][kKeys * D * 2];
  alignas(1024) char raw[kRawStages][FP8 ? kKeys * D : 128];  // 8-bit tiles as they come
  int64_t off[kKeys];
  uint64_t q_full, full[kStages], empty[kStages], raw_full[kRawStages];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_empty[2], drained;
  // of the piece, by its parity: the least position that a live row does not see, and whether
  // infinities or NaN were taken out of the V tiles from there on.  Pieces of one or two tiles fit the ring
  // together, so that the loads may be two pieces ahead: they write a pair anew when the 256 softmax threads
  // have read it.
  int32_t least[2], odd[2];
  uint64_t odd_read[2];
  int32_t warp_least[4];
  int32_t lost, error;
  int64_t scan[2 * (kThreads / 32)];
  uint32_t tmem;
};

// ---- tensor memory and products --------------------------------------------------------------
// One lane of the warp issues (lead != 0 there); the others pass by.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add, uint32_t lead) {
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add, uint32_t lead) {
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead) : "memory");
}
// The barrier is arrived at when all products issued before are done.
__device__ __forceinline__ void mma_commit(uint64_t *b, uint32_t lead) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %1, 0;\n"
               "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
               ::"r"(smem_u32(b)), "r"(lead) : "memory");
}
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// All loads before are there; the registers go through, so that no use of them comes before.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]),"+r"(r[1]),"+r"(r[2]),"+r"(r[3]),"+r"(r[4]),"+r"(r[5]),"+r"(r[6]),"+r"(r[7]),
               "+r"(r[8]),"+r"(r[9]),"+r"(r[10]),"+r"(r[11]),"+r"(r[12]),"+r"(r[13]),"+r"(r[14]),"+r"(r[15]),
               "+r"(r[16]),"+r"(r[17]),"+r"(r[18]),"+r"(r[19]),"+r"(r[20]),"+r"(r[21]),"+r"(r[22]),"+r"(r[23]),
               "+r"(r[24]),"+r"(r[25]),"+r"(r[26]),"+r"(r[27]),"+r"(r[28]),"+r"(r[29]),"+r"(r[30]),"+r"(r[31]) :: "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]),"+r"(r[1]),"+r"(r[2]),"+r"(r[3]),"+r"(r[4]),"+r"(r[5]),"+r"(r[6]),"+r"(r[7]),
               "+r"(r[8]),"+r"(r[9]),"+r"(r[10]),"+r"(r[11]),"+r"(r[12]),"+r"(r[13]),"+r"(r[14]),"+r"(r[15]) :: "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t a) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t a) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Two 32-bit floats at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
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
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
}

// A matrix operand in shared memory, D 16-bit columns a row: groups of eight rows, in them blocks of
// 64 columns, in them eight rows of 128 bytes whose 16-byte chunks are exchanged by the row (128-byte
// swizzle).  So eight rows are D * 16 bytes, blocks 1024 bytes apart.
template <int D>
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(1024 >> 4) << 16 | (uint64_t)(D * 16 >> 4) << 32 |
         1ull << 46 | 2ull << 61;
}

struct WidePiece {
  int32_t row0, rows, key0, tiles, key1, table;
  bool first, whole;
};

// Calls f(piece) for every piece of group g, whose part of the line is [w, end), beginning in unit u; f
// returns false to stop.
template <typename F>
__device__ __forceinline__ void wide_pieces(const AttnParams &p, int u, int64_t w, int64_t end, F f) {
  for (; w < end; ++u) {
    const AttnUnit x = p.planned ? p.units[u] : attn_plain_unit(p, u);
    if (w >= x.tile0 + x.key_tiles) continue;
    const int kt = (int)(w - x.tile0);
    WidePiece y;
    y.row0 = x.row0, y.rows = x.rows, y.table = x.table;
    y.tiles = (int)min((int64_t)(x.key_tiles - kt), end - w);
    y.key0 = kt * kKeys;
    y.key1 = (int32_t)min((int64_t)x.key1, (int64_t)y.key0 + (int64_t)y.tiles * kKeys);
    y.first = kt == 0;
    y.whole = y.first && y.tiles == x.key_tiles;
    if (!f(y)) return;
    w += y.tiles;
  }
}

// The token of local row i of a piece; its row's member of the group is (row0 + i) % group.
__device__ __forceinline__ int row_token(const AttnParams &p, const WidePiece &x, int i) {
  const int t = (x.row0 + i) / p.group;
  return x.table < 0 && p.planned ? p.prefix_tok[t] : t;
}

template <typename IO, bool FP8, int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnTma tma,
                 const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ char raw_smem[];
  using S = Smem<FP8, D>;
  using T = typename std::conditional<FP8, __half, IO>::type;  // of the products
  // (f16: little room above the maximum, so that the weights keep their range below it)
  constexpr float kRenew = std::is_same<T, __half>::value ? 2.f : 8.f, kShift = weight_shift<T>(kRenew);
  constexpr int kStages = S::kStages;
  S &sm = *reinterpret_cast<S *>(raw_smem + (-smem_u32(raw_smem) & 1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    bar_init(&sm.q_full, 256);
    for (int i = 0; i < S::kRawStages; ++i) bar_init(&sm.raw_full[i], 1);
    for (int i = 0; i < kStages; ++i) bar_init(&sm.full[i], 128), bar_init(&sm.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm.s_full[i], 1), bar_init(&sm.p_full[i][0], 128), bar_init(&sm.p_full[i][1], 128);
      bar_init(&sm.o_full[i], 1), bar_init(&sm.o_empty[i], 128);
      bar_init(&sm.odd_read[i], 256);
    }
    bar_init(&sm.drained, 1);
    sm.lost = sm.error = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  attn_wait_prior();
  if (blockIdx.x == 0) {
    if (tid == 0) attn_announce(p);
    __syncthreads();
  }
  attn_release_next();  // the narrow kernel may take SMs that this one does not use
  // this CTA's part of the line, and whether it has one
  const int g = blockIdx.x / p.kv_heads, h = blockIdx.x - g * p.kv_heads;
  int64_t w0, w1, quota;
  if (p.planned) {
    quota = p.head->wide_quota;
    w1 = p.head->units ? p.head->wide_tiles : 0;
  } else {
    int64_t before, mine;
    int32_t bad;
    w1 = attn_plain_wide(p);
    const int64_t own = attn_plain_total<kThreads>(p, sm.scan, &before, &mine, &bad);
    quota = max((int64_t)1, attn_up(w1, attn_share(p, own, w1).wide_groups));
  }
  w0 = g * quota;
  w1 = min(w1, w0 + quota);
  if (w0 >= w1) {
    if (tid == 0) p.errors[p.groups * p.kv_heads + blockIdx.x] = 0;
    if (warp == 12)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem) : "memory");
    return;
  }
  const int unit0 = p.planned ? p.start[p.groups + g] : (int)(w0 / attn_plain_unit(p, 0).key_tiles);
  constexpr uint32_t tm = 0;  // all 512 columns are this CTA's, so they begin at the first
  auto wait = [&](uint64_t *b, uint32_t parity) {
    return bar_wait(b, parity, &sm.lost, &sm.error);
  };

  // where the loads are in the rings
  uint32_t stage = 0, phase = 1, raw_in = 0, raw_in_phase = 1;

  if (warp < 8) {
    // ---- softmax of row tile t, a thread a row ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int t = warp >> 2, r = tid & 127;
    const uint32_t tmS = tm + t * 128, tmO = tm + 256 + t * D;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    uint32_t s_phase = 0, o_phase = 0, parity = 0;
    wide_pieces(p, unit0, w0, w1, [&](const WidePiece &x) {
      const int i = t * 128 + r;
      const bool active = x.rows > t * 128;
      const bool live = i < x.rows;
      const int token = live ? row_token(p, x, i) : 0;
      const int lim = live ? min(attn_limit(p, token), x.key1) : 0;
      const int member = (x.row0 + i) % p.group;
      float scale = p.scale_log2;
      if (active) {  // this row's queries; the products of the piece before are done with the last
        float f = 1.f;
        if constexpr (FP8 && std::is_same<IO, __nv_bfloat16>::value) {  // see attn_narrow_kernel
          const uint16_t *u = reinterpret_cast<const uint16_t *>(p.q + token * p.q_tok + (int64_t)(h * p.group + member) * p.q_head);
          uint32_t most = 0;
          if (live) {
            if (p.q_vec) {
#pragma unroll 8
              for (int c = 0; c < D / 8; ++c) {
                const uint4 w = reinterpret_cast<const uint4 *>(u)[c];
                most = max(most, max(max(max(w.x & 0x7fffu, w.x >> 16 & 0x7fffu), max(w.y & 0x7fffu, w.y >> 16 & 0x7fffu)),
                                     max(max(w.z & 0x7fffu, w.z >> 16 & 0x7fffu), max(w.w & 0x7fffu, w.w >> 16 & 0x7fffu))));
              }
            } else {
              for (int d = 0; d < D; ++d) most = max(most, u[d] & 0x7fffu);
            }
          }
          f = half_scale(most, &scale);
          // a row of zeros has the factor 2^-126: the product with a small scale must not be 0, by which
          // masked scores of -infinity are multiplied (any number as small gives the same weights)
          scale = fmaxf(scale, 1.17549435e-38f);
        }
        const char *src = p.q + token * p.q_tok + (int64_t)(h * p.group + member) * p.q_head;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
          uint4 w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            w[c] = make_uint4(0, 0, 0, 0);
            if (live && p.q_vec) w[c] = *reinterpret_cast<const uint4 *>(src + (c0 + c) * 16);
          }
          if (live && !p.q_vec) {
            const uint16_t *u = reinterpret_cast<const uint16_t *>(src) + c0 * 8;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              w[c].x = u[8 * c] | (uint32_t)u[8 * c + 1] << 16, w[c].y = u[8 * c + 2] | (uint32_t)u[8 * c + 3] << 16;
              w[c].z = u[8 * c + 4] | (uint32_t)u[8 * c + 5] << 16, w[c].w = u[8 * c + 6] | (uint32_t)u[8 * c + 7] << 16;
            }
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if constexpr (FP8 && std::is_same<IO, __nv_bfloat16>::value) {
              uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = pack2<__half>(__uint_as_float(v[e] << 16) * f, __uint_as_float(v[e] & 0xffff0000u) * f);
              w[c] = make_uint4(v[0], v[1], v[2], v[3]);
            }
            *reinterpret_cast<uint4 *>(sm.q[t] + place<D>(r, c0 + c)) = w[c];
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      bar_arrive(&sm.q_full);
      float m = -INFINITY;
      uint64_t l2 = pair(0.f, 0.f);
      if (active) {
        for (int j = 0; j < x.tiles; ++j) {
          if (!__all_sync(~0u, wait(&sm.s_full[t], s_phase))) return false;
          s_phase ^= 1;
          fence_after();
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s[c], tmS + lanes + c * 32);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
          const int seen = lim - (x.key0 + j * kKeys);
          if (seen < kKeys) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (c * 32 + k >= seen) s[c][k] = 0xff800000u;
          }
          float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            t0 = max3(t0, s[0][k], s[0][k + 1]), t1 = max3(t1, s[1][k], s[1][k + 1]);
            t2 = max3(t2, s[2][k], s[2][k + 1]), t3 = max3(t3, s[3][k], s[3][k + 1]);
          }
          const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * scale;
          const bool renew = top > m + (kRenew + kShift) || (m == -INFINITY && top > m);
          if (__any_sync(~0u, renew)) {
            const float f = !renew ? 1.f : m == -INFINITY ? 0.f : ex2(m - (top - kShift));
            if (renew) m = top - kShift;
            l2 = mul2(l2, pair(f, f));
            if (j > 0) {  // S of this tile is done, so are the products before it
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(o, tmO + lanes + c * 16);
                tmem_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(tmO + lanes + c * 16, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : -m;
          const uint64_t scale2 = pair(scale, scale), base2 = pair(base, base);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float a, b;
              unpair(fma2(pair(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), scale2, base2), a, b);
              a = ex2(a), b = ex2(b);
              l2 = add2(l2, pair(a, b));
              w[k] = pack2<T>(a, b);  // rounded to the values' type for the product; the sum is not
            }
            tmem_st16(tmS + lanes + c * 16, w);
            if (c & 1) {  // the products with the first 64 keys need not wait for the others
              tmem_wait_st();
              fence_before();
              bar_arrive(&sm.p_full[t][c >> 1]);
            }
          }
        }
      }
      if (!__all_sync(~0u, wait(&sm.o_full[t], o_phase))) return false;
      o_phase ^= 1;
      fence_after();
      const int odd = *(volatile int32_t *)&sm.odd[parity], least = *(volatile int32_t *)&sm.least[parity];
      bar_arrive(&sm.odd_read[parity]);
      if (active) {
        float l, l_odd;
        unpair(l2, l, l_odd);
        l += l_odd;
        const int qh = h * p.group + member;
        const int64_t part = attn_wide_part(p, x.first, g, h) + (x.first ? (int64_t)token * p.group + member : i);
        const bool direct = x.whole && x.table >= 0;
        const float inv = l == 0.f ? 0.f : p.v_scale / l;
        IO *out = reinterpret_cast<IO *>(p.out + (int64_t)token * p.out_tok + (int64_t)qh * p.out_head);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(o, tmO + lanes + c * 32);
          tmem_wait_ld(o);
          if (!live) continue;
          if (l == 0.f) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          } else if (odd) {
            // infinities and NaN that were taken out of tiles that some row's mask falls into
            for (int key = x.key0; key < lim; ++key) {
              const char *v = p.pool.v + attn_key_offset(p, key < p.prefix_len ? -1 : x.table, key, &sm.error) +
                              h * p.pool.head_stride;
              const int tile1 = x.key0 + ((key - x.key0) / kKeys + 1) * kKeys;
              if (tile1 <= least) continue;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                float e;
                if constexpr (FP8) {
                  const uint32_t u = from_e4m3x2(reinterpret_cast<const uint8_t *>(v)[c * 32 + k]);
                  e = __half2float(*reinterpret_cast<const __half *>(&u));
                } else {
                  e = (float)reinterpret_cast<const T *>(v)[c * 32 + k];
                }
                if (!isfinite(e)) o[k] = __float_as_uint(__uint_as_float(o[k]) + e);
              }
            }
          }
          if (direct) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              w[k] = pack2<IO>(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
            if (p.out_vec) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                reinterpret_cast<uint4 *>(out + c * 32)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                reinterpret_cast<uint16_t *>(out)[c * 32 + 2 * k] = (uint16_t)w[k];
                reinterpret_cast<uint16_t *>(out)[c * 32 + 2 * k + 1] = (uint16_t)(w[k] >> 16);
              }
            }
          } else {
            float *d = p.part_o + part * D + c * 32;
#pragma unroll
            for (int k = 0; k < 32; k += 8)  // whole sectors
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(d + k), "r"(o[k]),
                           "r"(o[k + 1]), "r"(o[k + 2]), "r"(o[k + 3]), "r"(o[k + 4]), "r"(o[k + 5]),
                           "r"(o[k + 6]), "r"(o[k + 7]) : "memory");
          }
        }
        if (live) {
          if (direct) {
            if (p.lse)
              p.lse[(int64_t)token * p.q_heads + qh] =
                  l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
          } else {
            p.part_m[part] = m;
            p.part_l[part] = l;
          }
        }
        fence_before();
      }
      bar_arrive(&sm.o_empty[t]);
      parity ^= 1;
      return true;
    });
  } else if (warp < 12) {
    // ---- loads ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int i = tid - 256;
    constexpr int kRaw = FP8 ? D / 16 : D / 8;         // 16-byte chunks of a row in the pool
    constexpr int kStep = 128 / kRaw, kPer = kKeys / kStep;
    const int c = i % kRaw, r0 = i / kRaw;
    uint32_t parity = 0, read_phase = 1, raw_out = 0, raw_phase = 0;
    uint64_t *pend[2] = {nullptr, nullptr};  // barriers of copies on their way, the older first
    auto arrive = [&](uint64_t *b) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      bar_arrive(b);
    };
    auto flush = [&]() {
      if (pend[0]) {
        cp_async_wait<1>();
        arrive(pend[0]);
      }
      if (pend[1]) {
        cp_async_wait<0>();
        arrive(pend[1]);
      }
      pend[0] = pend[1] = nullptr;
    };
    auto sent = [&](uint64_t *b) {  // the copies for b have been issued
      cp_async_commit();
      if (pend[0]) {
        cp_async_wait<2>();
        arrive(pend[0]);
      }
      pend[0] = pend[1], pend[1] = b;
    };
    // A wait that was given up is not waited for again (see bar_wait): these threads then run
    // through what is left without waiting, since they meet at barriers of their own, and send nothing more
    // on its way.
    bool lost = false;  // a warp's lanes agree
    wide_pieces(p, unit0, w0, w1, [&](const WidePiece &x) {
      const int boxes = tma.rows > 0 ? kKeys / tma.rows : 1, pw = warp - 8;
      // page look-ups: lane l of warp w has box 4 l + w of a regular tile
      const int box = lane * 4 + pw;
      auto box_page = [&](int j) -> int32_t {  // as it stands in the table; checked when it is used
        int pg, off;
        const int pos = x.key0 + j * kKeys + box * tma.rows;
        if (pos >= x.key1 || box >= boxes) return 0;
        attn_split(p, pos, &pg, &off);
        return attn_entry(p, pos < p.prefix_len ? -1 : x.table, pg);
      };
      const int32_t page0 = box_page(0);
      // from where on live rows differ in what they see
      int least = INT32_MAX;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = i + k * 128;
        const int v = r < x.rows ? attn_limit(p, row_token(p, x, r)) : 0;
        if (v > x.key0) least = min(least, v);
      }
      for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(~0u, least, o));
      if (lane == 0) sm.warp_least[warp - 8] = least;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      least = min(min(sm.warp_least[0], sm.warp_least[1]), min(sm.warp_least[2], sm.warp_least[3]));
      if (least >= x.key1) least = INT32_MAX;
      lost |= !__all_sync(~0u, i != 0 || wait(&sm.odd_read[parity], read_phase));
      if (i == 0) sm.least[parity] = least, sm.odd[parity] = 0;
      asm volatile("bar.sync 1, 128;" ::: "memory");  // odd is 0 before anyone sets it

      // a tile that tensor copies can bring: whole, the same for all live rows, and no box of it
      // partly in the prefix
      auto regular = [&](int j) {
        const int k0 = x.key0 + j * kKeys;
        return tma.rows > 0 && k0 + kKeys <= x.key1 && k0 + kKeys <= least &&
               (k0 >= p.prefix_len || k0 + kKeys <= p.prefix_len || p.prefix_len % tma.rows == 0);
      };
      auto box_row = [&](int j, int32_t id) -> int {
        int pg, off;
        attn_split(p, x.key0 + j * kKeys + box * tma.rows, &pg, &off);
        return (int)(attn_checked(p, id, &sm.error) * tma.page_y + h * tma.head_y + off);
      };
      auto look = [&](int j) -> int64_t {  // of any tile, key by key
        const int pos = x.key0 + j * kKeys + i;
        return pos < x.key1
                   ? attn_key_offset(p, pos < p.prefix_len ? -1 : x.table, pos, &sm.error) + h * p.pool.head_stride : 0;
      };
      // this lane's box of K (kv 0) or V (1); a lane of each warp at most has work for short tiles
      auto tensor = [&](int j, int kv, int32_t id, char *dst, uint64_t *bar) {
        if (box >= boxes) return;
        const CUtensorMap *map = kv ? &v_map : &k_map;
        const int row = box_row(j, id);
        if constexpr (FP8) tma_load(dst + box * tma.rows * D, map, h * tma.head_x, row, bar);
        else tma_load4(dst + box * tma.rows * D * 2, map, h * tma.head_x, row >> 3, bar);
      };
      auto convert = [&](const uint4 &v, char *dst, int r) {  // 16 8-bit values to their places
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] = from_e4m3x2((uint16_t)w[e]);
          o[2 * e + 1] = from_e4m3x2((uint16_t)(w[e] >> 16));
        }
        *reinterpret_cast<uint4 *>(dst + place<D>(r, 2 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(dst + place<D>(r, 2 * c + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
      };

      // 8-bit tiles come by tensor copies some stages ahead of their conversion
      int ahead = 0;
      int32_t ahead_page = page0, ahead_next = FP8 ? box_page(1) : 0;
      auto fetch = [&](int upto) {  // up to tile and half number `upto`
        for (; ahead < min(upto, 2 * x.tiles); ++ahead) {
          if (regular(ahead >> 1) && !lost) {
            if (i == 0) bar_expect(&sm.raw_full[raw_in], kKeys * D);
            tensor(ahead >> 1, ahead & 1, ahead_page, sm.raw[raw_in], &sm.raw_full[raw_in]);
            if (++raw_in == S::kRawStages) raw_in = 0, raw_in_phase ^= 1;
          }
          if (ahead & 1) ahead_page = ahead_next, ahead_next = box_page((ahead + 3) >> 1);
        }
      };
      int32_t next_page = page0;
      for (int j = 0; j < x.tiles; ++j) {
        const int k0 = x.key0 + j * kKeys;
        const bool reg = regular(j);
        const int32_t page = next_page;
        if constexpr (!FP8) next_page = box_page(j + 1);
        if (!reg) {
          // key by key; the tile that used these offsets before is done with by everyone
          const int64_t o = look(j);
          asm volatile("bar.sync 1, 128;" ::: "memory");
          sm.off[i] = o;
          asm volatile("bar.sync 1, 128;" ::: "memory");
        }
        const int64_t *off = sm.off;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const char *plane = (kv ? p.pool.v : p.pool.k) + c * 16;
          uint4 raw[FP8 ? kPer : 1];
          if constexpr (FP8) {
            if (reg) {
              fetch(2 * j + kv + S::kRawStages);
            } else {
#pragma unroll
              for (int k = 0; k < kPer; ++k) {
                const int r = r0 + k * kStep;
                raw[k] = k0 + r < x.key1 ? __ldg(reinterpret_cast<const uint4 *>(plane + off[r])) : make_uint4(0, 0, 0, 0);
              }
            }
          }
          bool there = bar_try(&sm.empty[stage], phase);
          if (!there) {
            flush();  // nothing that is there is held back meanwhile
            there = wait(&sm.empty[stage], phase);
          }
          lost |= !__all_sync(~0u, there);
          char *dst = sm.kv[stage];
          if constexpr (FP8) {
            if (reg) {
              lost |= !__all_sync(~0u, wait(&sm.raw_full[raw_out], raw_phase));
#pragma unroll
              for (int k = 0; k < kPer; ++k)
                raw[k] = *reinterpret_cast<const uint4 *>(sm.raw[raw_out] + place8<D>(r0 + k * kStep, c));
              asm volatile("bar.sync 1, 128;" ::: "memory");  // the raw stage may be filled again
              if (++raw_out == S::kRawStages) raw_out = 0, raw_phase ^= 1;
            }
          }
          if (lost) continue;
          if constexpr (FP8) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) convert(raw[k], dst, r0 + k * kStep);
          } else if (reg) {
            flush();
            // one arrival for the tile's bytes and one for each thread's boxes: those of a thread may
            // arrive before the bytes are announced, the stage is not full before the thread is
            if (i == 0) bar_expect(&sm.full[stage], kKeys * D * 2);
            tensor(j, kv, page, dst, &sm.full[stage]);
            if (i != 0) bar_arrive(&sm.full[stage]);
          } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              const int r = r0 + k * kStep;
              cp_async16(smem_u32(dst) + place<D>(r, c), plane + off[r], k0 + r < x.key1);
            }
          }
          if (kv && k0 + kKeys > least) {
            // see attn_narrow_kernel: values that are not finite, where some row's mask falls into
            // the tile; a thread looks at the chunks that it has copied itself
            cp_async_commit();
            cp_async_wait<0>();
            bool any = false;
#pragma unroll 1
            for (int k = 0; k < kPer * (FP8 ? 2 : 1); ++k) {
              const int r = r0 + (FP8 ? k >> 1 : k) * kStep;
              uint4 *v = reinterpret_cast<uint4 *>(dst + place<D>(r, FP8 ? 2 * c + (k & 1) : c));
              uint32_t w[4] = {v->x, v->y, v->z, v->w};
              bool here = false;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (odd2<T>(w[e])) {
                  if (odd2<T>(w[e] & 0xffffu)) w[e] &= 0xffff0000u;
                  if (odd2<T>(w[e] & 0xffff0000u)) w[e] &= 0xffffu;
                  here = true;
                }
              if (here) *v = make_uint4(w[0], w[1], w[2], w[3]);
              any |= here;
            }
            if (any) *(volatile int32_t *)&sm.odd[parity] = 1;
          }
          if (FP8) arrive(&sm.full[stage]);
          else if (!reg) sent(&sm.full[stage]);
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
      }
      flush();
      asm volatile("bar.sync 1, 128;" ::: "memory");  // everyone has read warp_least
      read_phase ^= parity;
      parity ^= 1;
      return true;
    });
  } else {
    // ---- products ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 12) {  // all lanes walk along, so that what they agree on stays in uniform registers
      const uint32_t lead = elect_lane();
      // (a wait that was given up is not waited for again, and what is then computed is of no account)
      auto wait_all = [&](uint64_t *b, uint32_t parity) {
        wait(b, parity);
        __syncwarp();
      };
      constexpr uint32_t kFmt = std::is_same<T, __half>::value ? 0u : 1u;
      constexpr uint32_t kBase = 1u << 4 | kFmt << 7 | kFmt << 10 | (128u >> 4) << 24;
      constexpr uint32_t kDescS = kBase | (uint32_t)(kKeys >> 3) << 17;
      constexpr uint32_t kDescO = kBase | (uint32_t)(D >> 3) << 17 | 1u << 16;  // V read across its rows
      // (everything is a function of t by arithmetic and the loops over t are unrolled: one thread issues
      // a product every 64 cycles and has no time for tables in memory)
      uint32_t q_phase = 0, p_phase = 0, oe_phase = 1;
      phase = 0;
      const uint64_t q0 = operand<D>(smem_u32(sm.q[0])), kv0 = operand<D>(smem_u32(sm.kv[0]));
      constexpr uint64_t kTileStep = 128 * D * 2 >> 4;
      auto scores = [&](int t, uint32_t kst) {
        const uint64_t qd = q0 + t * kTileStep, kd = kv0 + kst * kTileStep;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t step = (uint64_t)((k >> 2) * (1024 >> 4) + (k & 3) * 2);
          mma_ss(tm + t * 128, qd + step, kd + step, kDescS, k > 0, lead);
        }
      };
      // About five products wait in the tensor cores' queue, 350 cycles: no two waits stand together, and
      // stages are given back as soon as their last product has been issued.
      wide_pieces(p, unit0, w0, w1, [&](const WidePiece &x) {
        const int tiles = x.tiles;
        const bool two = x.rows > 128;
        wait_all(&sm.q_full, q_phase);
        wait_all(&sm.full[stage], phase);
        q_phase ^= 1;
        fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (t == 0 || two) {
            scores(t, stage);
            mma_commit(&sm.s_full[t], lead);
          }
        mma_commit(&sm.empty[stage], lead);
        if (++stage == kStages) stage = 0, phase ^= 1;
        wait_all(&sm.full[stage], phase);
        for (int j = 0; j < tiles; ++j) {
          const uint32_t vst = stage;
          if (++stage == kStages) stage = 0, phase ^= 1;
          const uint32_t kst = stage, k_phase = phase;  // of the next tile's keys
          const bool more = j + 1 < tiles;
          if (more && ++stage == kStages) stage = 0, phase ^= 1;  // now its values
          const uint64_t vd = kv0 + vst * kTileStep;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (j == 0) wait_all(&sm.o_empty[t], oe_phase);
            if (t == 0 || two) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k) {
                if (k % (kKeys / 32) == 0) {
                  wait_all(&sm.p_full[t][k / (kKeys / 32)], p_phase >> t & 1);
                  fence_after();
                }
                mma_ts(tm + 256 + t * D, tm + t * 128 + k * 8, vd + (uint64_t)(k * (2 * D * 16 >> 4)), kDescO,
                       j > 0 || k > 0, lead);
              }
            }
            if (t == 1) mma_commit(&sm.empty[vst], lead);
            if (more) {
              if (t == 0) wait_all(&sm.full[kst], k_phase);
              else wait_all(&sm.full[stage], phase);
              if (t == 0 || two) {
                scores(t, kst);
                mma_commit(&sm.s_full[t], lead);
              }
            } else {
              mma_commit(&sm.o_full[t], lead);
            }
          }
          p_phase ^= two ? 3 : 1;
          if (more) mma_commit(&sm.empty[kst], lead);
        }
        oe_phase ^= 1;
        return true;
      });
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (sm.lost) {  // products and copies in flight end before their memory is given up
    if (warp == 12) {
      mma_commit(&sm.drained, elect_lane());  // (the lane that has issued them)
      for (uint32_t n = 0; n < kAttnDrainPolls && !bar_try(&sm.drained, 0); ++n) {}
    } else if (warp >= 8 && warp < 12) {
      bar_drain<kStages>(sm.full, stage, phase);
      if constexpr (FP8) bar_drain<S::kRawStages>(sm.raw_full, raw_in, raw_in_phase);
    }
    __syncthreads();
  }
  if (tid == 0) p.errors[p.groups * p.kv_heads + blockIdx.x] = sm.error;
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem) : "memory");
}

template <typename IO, bool FP8, int D>
cudaError_t launch(const AttnParams &p, bool hnd, cudaStream_t s) {
  const void *fn = (const void *)attn_wide_kernel<IO, FP8, D>;
  constexpr int kSmem = (int)sizeof(Smem<FP8, D>) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  AttnTma tma;
  CUtensorMap km, vm;
  attn_make_tma(p, kKeys, FP8, hnd, &tma, &km, &vm);
  void *args[] = {const_cast<AttnParams *>(&p), &tma, &km, &vm};
  return launch_pdl(fn, dim3(p.wide_groups * p.kv_heads), dim3(kThreads), args, s, kSmem);
}

template <typename IO, bool FP8>
cudaError_t launch_d(const AttnParams &p, bool hnd, cudaStream_t s) {
  return p.head_dim == 64 ? launch<IO, FP8, 64>(p, hnd, s) : launch<IO, FP8, 128>(p, hnd, s);
}

}  // namespace

cudaError_t launch_attn_wide(const AttnParams &p, int32_t dtype, int32_t io, bool hnd, cudaStream_t s) {
  if (dtype == KVX_F16) return launch_d<__half, false>(p, hnd, s);
  if (dtype == KVX_BF16) return launch_d<__nv_bfloat16, false>(p, hnd, s);
  if (io == KVX_F16) return launch_d<__half, true>(p, hnd, s);
  return launch_d<__nv_bfloat16, true>(p, hnd, s);
}

}  // namespace kvx
