// kvx_attn_q4.cu -- shared attention over a 4-bit pool for few rows a key: decode steps and short drafts.
//
// An element is low + code * scale, with a scale and a low for every 32 elements of a head (a group).  Codes go
// into the tensor cores as they are: the 4 bits, masked out of a word, are the f16 number code * 2^-24 (or
// 2^-20), exactly, so that unpacking is one AND an element pair.  With the scales left for later,
//   <q, k>       = sum_g scale_g <q_g, code_g> + low_g sum(q_g)
//   sum_j p_j v_j = sum_j (p_j scale_gj) code_j + p_j low_gj :
// the scores' sums of a group are multiplied by its scale in 32 bits; the weights, which are rounded to f16 for
// the product in any case, are multiplied by the scales of their keys' values, group by group, and rounded once more.
// The lows are a product of their own: (scale, low) words as they stand are its operand, against the sums of the
// queries (as two f16 numbers, so exact to 2^-22) and against the weights.
//
// Keys are the rows of both products (m16n8k16, M = 16 keys, N = 8 query rows; then M = 16 columns, K = 16
// keys): the eight columns suit a group of up to eight query heads.  A warp walks blocks of 16 keys that it
// brings in itself, 80 (or 40) bytes of K and V a key, into a ring of its own: no barrier within a piece.  The
// warps of a CTA share a piece's blocks, and where it has more than eight rows its rows; their sums are joined in
// shared memory at its end.
#include <type_traits>

#include "kvx_attn.cuh"
#include "kvx_attn_mma.cuh"
#include "kvx_launch.cuh"
#include "kvx_quant.cuh"

namespace kvx {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kBlock = 16;    // keys at a time
constexpr int kRows = 8;      // of a warp
constexpr int kPieces = 32;   // listed at a time
constexpr float kTop = 13.f;  // the greatest weight is about 2^kTop (see weight_shift), less for scales above 1
constexpr float kRenew = 2.f; // by so many powers of two may a score pass what weights refer to

template <int D>
struct Smem {
  static constexpr int kPitch = D == 128 ? 80 : 48;  // eight rows' 16-byte chunks lie in different banks
  static constexpr int kStages = 3;
  static constexpr int kStage = 2 * kBlock * kPitch;  // keys, then values
  static constexpr int kSum = D + 4;                  // floats of a row on its way to be joined
  alignas(128) char ring[kWarps][kStages][kStage];
  alignas(16) float sum[kWarps][kRows][kSum];
  float base[kWarps][kRows], l[kWarps][kRows];
  AttnPiece pieces[kPieces];
  int64_t scan[2 * kWarps + 4];
  int32_t n_pieces, more, error;
};

template <int B>
__device__ __forceinline__ void cp_async(uint32_t dst, const char *src) {
  if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// ... or zeros.
template <int B>
__device__ __forceinline__ void cp_async_if(uint32_t dst, const char *src, bool ok) {
  const int n = ok ? B : 0;
  if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t (&r)[2], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix2t(uint32_t (&r)[2], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float low_half(uint32_t x) { return __half2float(__ushort_as_half((uint16_t)x)); }
__device__ __forceinline__ bool odd_word(uint32_t x) { return odd2<__half>(x); }

// How a piece's rows and keys are shared by the warps: 2^split sets of eight rows, the others take other blocks.
__device__ __forceinline__ int split_of(int rows) { return rows <= 8 ? 0 : rows <= 16 ? 1 : rows <= 32 ? 2 : 3; }

// A piece's blocks of 16 keys, from the one that its first key is in.
struct Blocks {
  int32_t start, count;
  __device__ __forceinline__ Blocks(const AttnPiece &x) {
    start = max(x.key0, x.low) / kBlock * kBlock;
    count = x.key1 > max(x.key0, x.low) ? (x.key1 - start + kBlock - 1) / kBlock : 0;
  }
};

// Brings a warp's blocks in, in the order in which they are worked.
template <int D>
struct Loader {
  using S = Smem<D>;
  static constexpr int kChunk = D / 8;  // bytes of a copy: a head vector is five of them
  const AttnParams &p;
  S &sm;
  const int h, lane, warp;
  int piece = -1, block = 0, count = 0, step = 1, stage = 0;
  int32_t start = 0, low = 0, key1 = 0, table = 0;
  int32_t id = 0;            // the page of the block to be sent next (whole blocks in a page)
  int32_t off[5], dst[5];    // this lane's copies of a block in a page: from its first key's head vector, in a stage

  __device__ __forceinline__ Loader(const AttnParams &p, S &sm, int h, int lane, int warp)
      : p(p), sm(sm), h(h), lane(lane), warp(warp) {
#pragma unroll
    for (int r = 0; r < 5; ++r) {
      const int j = r * 32 + lane, row = j / 5, c = j - row * 5;
      off[r] = (row & 15) * (int32_t)p.pool.tok_stride + c * kChunk;
      dst[r] = row * S::kPitch + c * kChunk;
    }
  }
  // The next block that is this warp's.
  __device__ __forceinline__ void next() {
    block += step;
    while (block >= count) {
      if (++piece >= sm.n_pieces) return;
      const AttnPiece &x = sm.pieces[piece];
      const Blocks b(x);
      const int split = split_of(x.rows);
      start = b.start, count = b.count, low = x.low, key1 = x.key1, table = x.table;
      block = warp >> split, step = kWarps >> split;
    }
    if (p.paged_blocks) {
      int32_t pg, o;
      attn_split(p, start + block * kBlock, &pg, &o);
      id = attn_entry(p, table, pg);
    }
  }
  __device__ __forceinline__ void begin() {
    piece = -1, block = count = 0, step = 1;
    next();
  }
  __device__ __forceinline__ void send() {
    if (piece < sm.n_pieces) {
      const uint32_t to = smem_u32(sm.ring[warp][stage]);
      const int32_t pos = start + block * kBlock;
      if (p.paged_blocks && pos >= low && pos + kBlock <= key1) {
        int32_t pg, o;
        attn_split(p, pos, &pg, &o);
        const int64_t at = attn_checked(p, id, &sm.error) * p.pool.page_stride + o * p.pool.tok_stride + h * p.pool.head_stride;
        const char *k = p.pool.k + at, *v = p.pool.v + at;
#pragma unroll
        for (int r = 0; r < 5; ++r) {
          const bool val = r == 2 ? lane >= 16 : r > 2;  // copies 80 on are of the values
          cp_async<kChunk>(to + dst[r], (val ? v : k) + off[r]);
        }
      } else {
        const int32_t mine = pos + (lane & 15);
        int64_t at = -1;
        if (mine >= low && mine < key1) at = attn_key_offset(p, table, mine, &sm.error) + h * p.pool.head_stride;
#pragma unroll
        for (int r = 0; r < 5; ++r) {
          const int j = r * 32 + lane, row = j / 5, c = j - row * 5;
          const int64_t from = __shfl_sync(~0u, at, row & 15);
          cp_async_if<kChunk>(to + dst[r], (row >= 16 ? p.pool.v : p.pool.k) + (from < 0 ? 0 : from + c * kChunk), from >= 0);
        }
      }
      next();
    }
    cp_async_commit();
    if (++stage == S::kStages) stage = 0;
  }
};

template <typename IO, int D>
struct Worker {
  using S = Smem<D>;
  static constexpr int G = D / KVX_Q4_GROUP;
  const AttnParams &p;
  S &sm;
  Loader<D> &load;
  const int h, lane, warp;
  int stage = 0;

  // Eight elements of a query row from d on, as 32-bit numbers.
  __device__ __forceinline__ void eight(const char *row, int d, float (&o)[8]) const {
    uint32_t w[4];
    if (p.q_vec) {
      const uint4 v = *reinterpret_cast<const uint4 *>(row + d * 2);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint16_t *u = reinterpret_cast<const uint16_t *>(row) + d;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = u[2 * i] | (uint32_t)u[2 * i + 1] << 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<IO, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        o[2 * i] = f.x, o[2 * i + 1] = f.y;
      } else {
        o[2 * i] = __uint_as_float(w[i] << 16), o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }

  __device__ __forceinline__ void piece(const AttnPiece &x) {
    const int split = split_of(x.rows), set = warp & ((1 << split) - 1), c4 = lane & 3, r8 = lane >> 2;
    const Blocks blocks(x);
    // ---- queries: of row set * 8 + r8, elements 8 c4 .. 8 c4 + 7 of every group, so that a word of codes
    // (eight elements of a key) meets them: pairs (0, 4), (1, 5), (2, 6), (3, 7), the odd ones divided by 16,
    // by which their codes are greater
    uint32_t q[G][2][2], qs[2];
    float factor = 1.f;
    {
      const int r = set * kRows + r8;
      const bool live = r < x.rows;
      const int row = x.row0 + (live ? r : 0), t = row / p.group;
      const char *src = p.q + t * p.q_tok + (int64_t)(h * p.group + row - t * p.group) * p.q_head;
      float e[G][8];
      uint32_t most = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        eight(src, g * KVX_Q4_GROUP + 8 * c4, e[g]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!live) e[g][i] = 0.f;
          most = max(most, __float_as_uint(e[g][i]) & 0x7fffffffu);
        }
      }
      most = max(most, __shfl_xor_sync(~0u, most, 1));
      most = max(most, __shfl_xor_sync(~0u, most, 2));
      const float f = half_scale(most >> 16, &factor);  // (the upper bits of a 32-bit number are bf16's)
      float mine = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) e[g][i] *= f, sum += e[g][i];
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        if (c4 == g) mine = sum;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          q[g][k][0] = pack2<__half>(e[g][2 * k], e[g][2 * k + 4]);
          q[g][k][1] = pack2<__half>(e[g][2 * k + 1] * 0.0625f, e[g][2 * k + 5] * 0.0625f);
        }
      }
      mine *= 0.03125f;  // of at most 32 numbers up to 2^15: back into f16's range
      const __half hi = __float2half_rn(mine);
      qs[0] = (uint32_t)__half_as_ushort(hi) << 16;  // against (scale, low): nothing of the scale
      qs[1] = (uint32_t)__half_as_ushort(__float2half_rn(mine - __half2float(hi))) << 16;
    }
    // ---- of this lane's rows, set * 8 + 2 c4 and the one behind
    float sc[2], base[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int lim[2];
    const int first = max(x.key0, x.low);
    int least = INT32_MAX;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sc[i] = p.scale_log2 * __shfl_sync(~0u, factor, (2 * c4 + i) * 4);
      const int r = set * kRows + 2 * c4 + i;
      lim[i] = r < x.rows ? min(attn_limit(p, (x.row0 + r) / p.group), x.key1) : 0;
      if (lim[i] > first) least = min(least, lim[i]);
    }
    least = min(least, __shfl_xor_sync(~0u, least, 1));
    least = min(least, __shfl_xor_sync(~0u, least, 2));
    float o[G][2][4] = {}, z[4] = {};  // z: of the unit of (scale, low) words that is r8's
    float top = kTop;
    int odd = 0;
    const float limit0 = r8 & 1 ? INFINITY : 1.f;  // of values' scales: at first 1
    float limit = limit0;

#pragma unroll 1
    for (int b = warp >> split; b < blocks.count; b += kWarps >> split) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      load.send();
      const uint32_t kt = smem_u32(sm.ring[warp][stage]), vt = kt + kBlock * S::kPitch;
      if (++stage == S::kStages) stage = 0;
      const int pos = blocks.start + b * kBlock;
      const bool mixed = pos + kBlock > least || pos < x.low || pos + kBlock > x.key1;
      const uint32_t row16 = (uint32_t)((lane & 15) * S::kPitch);  // (addresses of ldmatrix: 16 keys, two chunks)
      // ---- scores of keys r8 and r8 + 8
      float s[4] = {};
      {
        float a[4] = {};
        uint32_t w[2];
        ldmatrix2(w, kt + row16 + D / 2);
        const uint32_t f[4] = {w[0], w[1], w[0], w[1]};
        mma16816<__half>(a, f, qs[0], qs[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = a[i] * 0x1p-19f;
      }
      uint32_t ks[2][G];  // (scale, low) of the two keys
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const char *at = sm.ring[warp][0] + (kt - smem_u32(sm.ring[warp][0])) + (r8 + 8 * i) * S::kPitch + D / 2;
        if constexpr (G == 4) {
          const uint4 v = *reinterpret_cast<const uint4 *>(at);
          ks[i][0] = v.x, ks[i][1] = v.y, ks[i][2] = v.z, ks[i][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(at);
          ks[i][0] = v.x, ks[i][1] = v.y;
        }
      }
#pragma unroll
      for (int g = 0; g < G; g += 2) {
        uint32_t w[4];
        ldmatrix4(w, kt + row16 + (g + (lane >> 4)) * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t u = w[2 * e], v = w[2 * e + 1];
          float a[4] = {};
          const uint32_t f0[4] = {u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u};
          mma16816<__half>(a, f0, q[g + e][0][0], q[g + e][0][1]);
          const uint32_t u8 = u >> 8, v8 = v >> 8;
          const uint32_t f1[4] = {u8 & 0x000f000fu, v8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x00f000f0u};
          mma16816<__half>(a, f1, q[g + e][1][0], q[g + e][1][1]);
          const float s0 = low_half(ks[0][g + e]), s1 = low_half(ks[1][g + e]);
          s[0] = fmaf(a[0], s0, s[0]), s[1] = fmaf(a[1], s0, s[1]);
          s[2] = fmaf(a[2], s1, s[2]), s[3] = fmaf(a[3], s1, s[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = s[i] * 0x1p24f * sc[i & 1];
      if (mixed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = pos + r8 + (i >> 1) * 8;
          if (key < x.low || key >= lim[i & 1]) s[i] = -INFINITY;
        }
      }
      // ---- the values' (scale, low) words, a unit a lane's row; what weights refer to
      uint32_t zw[2];
      ldmatrix2t(zw, vt + row16 + D / 2);
      if (mixed) {
        // (infinities and NaN of keys that some row does not see are taken out and put back at the end)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (odd_word(zw[i] & 0xffffu)) zw[i] &= 0xffff0000u, odd = 1;
          if (odd_word(zw[i] & 0xffff0000u)) zw[i] &= 0xffffu, odd = 1;
        }
      }
      {
        const float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
        const __half2 zm = __hmax2(*reinterpret_cast<const __half2 *>(&zw[0]), *reinterpret_cast<const __half2 *>(&zw[1]));
        const float big = fmaxf(__low2float(zm), __high2float(zm));
        const float edge = top + kRenew;
        // (a row that has seen nothing yet has a base of -infinity, and any score passes it)
        if (__any_sync(~0u, t0 - base[0] > edge || t1 - base[1] > edge || big > limit)) {
          float n0 = t0, n1 = t1, up = limit0 < INFINITY ? big : 0.f;
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, d));
            n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, d));
          }
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, d));
          float now = top;
          if (up > 1.f) now = fminf(top, kTop - (float)(ilogbf(fminf(up, 65504.f)) + 1));
          limit = limit0 < INFINITY ? exp2f(kTop - now) : INFINITY;
          // the greatest score so far, or what stood for it
          const float m0 = fmaxf(base[0] + top, n0), m1 = fmaxf(base[1] + top, n1);
          const float b0 = m0 - now, b1 = m1 - now;
          const float f0 = base[0] == -INFINITY ? 0.f : ex2(base[0] - b0), f1 = base[1] == -INFINITY ? 0.f : ex2(base[1] - b1);
          l[0] *= f0, l[1] *= f1;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 2; ++k) o[g][k][0] *= f0, o[g][k][1] *= f1, o[g][k][2] *= f0, o[g][k][3] *= f1;
          z[0] *= f0, z[1] *= f1;
          base[0] = b0, base[1] = b1, top = now;
        }
      }
      // ---- weights, their rows and keys exchanged: row r8, keys 2 c4, 2 c4 + 1 and 8 behind
      const float from0 = base[0] == -INFINITY ? 0.f : base[0], from1 = base[1] == -INFINITY ? 0.f : base[1];
      s[0] = ex2(s[0] - from0), s[1] = ex2(s[1] - from1), s[2] = ex2(s[2] - from0), s[3] = ex2(s[3] - from1);
      l[0] += s[0] + s[2], l[1] += s[1] + s[3];
      // rounded to f16 for the products; their sum is not
      const uint32_t p0 = transpose8(pack2<__half>(s[0], s[1])), p1 = transpose8(pack2<__half>(s[2], s[3]));
      {
        const uint32_t f[4] = {zw[0], 0, zw[1], 0};
        mma16816<__half>(z, f, p0, p1);
      }
      uint32_t vs[4][G];  // (scale, low) of keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const char *at = sm.ring[warp][0] + (vt - smem_u32(sm.ring[warp][0])) + (2 * c4 + (i & 1) + 8 * (i >> 1)) * S::kPitch + D / 2;
        if constexpr (G == 4) {
          const uint4 v = *reinterpret_cast<const uint4 *>(at);
          vs[i][0] = v.x, vs[i][1] = v.y, vs[i][2] = v.z, vs[i][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(at);
          vs[i][0] = v.x, vs[i][1] = v.y;
        }
        if (mixed)
#pragma unroll
          for (int g = 0; g < G; ++g)
            if (odd_word(vs[i][g] & 0xffffu)) vs[i][g] = 0, odd = 1;
      }
#pragma unroll
      for (int g = 0; g < G; g += 2) {
        uint32_t w[4];
        ldmatrix4t(w, vt + row16 + (g + (lane >> 4)) * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t b0 = mul_half2(p0, __byte_perm(vs[0][g + e], vs[1][g + e], 0x5410));
          const uint32_t b1 = mul_half2(p1, __byte_perm(vs[2][g + e], vs[3][g + e], 0x5410));
          const uint32_t u = w[2 * e], v = w[2 * e + 1], u8 = u >> 8, v8 = v >> 8;
          const uint32_t f0[4] = {u & 0x000f000fu, u8 & 0x000f000fu, v & 0x000f000fu, v8 & 0x000f000fu};
          mma16816<__half>(o[g + e][0], f0, b0, b1);
          const uint32_t f1[4] = {u & 0x00f000f0u, u8 & 0x00f000f0u, v & 0x00f000f0u, v8 & 0x00f000f0u};
          mma16816<__half>(o[g + e][1], f1, b0, b1);
        }
      }
    }
    // ---- the warp's sums: columns 32 g + 4 r8 .. + 3 of its two rows
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l[0] += __shfl_xor_sync(~0u, l[0], d);
      l[1] += __shfl_xor_sync(~0u, l[1], d);
    }
    odd = __any_sync(~0u, odd);
    __syncthreads();  // the sums of the piece before have been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool none = lim[i] <= first || l[i] == 0.f;  // (a row that sees nothing of the piece has worked on all)
      const int r = 2 * c4 + i;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float low = __shfl_sync(~0u, z[i], (2 * g + 1) * 4 + c4);
        float v[4] = {fmaf(o[g][0][i], 0x1p24f, low), fmaf(o[g][1][i], 0x1p20f, low),
                      fmaf(o[g][0][2 + i], 0x1p24f, low), fmaf(o[g][1][2 + i], 0x1p20f, low)};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = none ? 0.f : v[k];
        if (odd && !none) put_back(x, g, lim[i], least, v);
        *reinterpret_cast<float4 *>(&sm.sum[warp][r][g * KVX_Q4_GROUP + 4 * r8]) = make_float4(v[0], v[1], v[2], v[3]);
      }
      if (r8 == 0) sm.base[warp][r] = none ? -INFINITY : base[i], sm.l[warp][r] = none ? 0.f : l[i];
    }
    __syncthreads();
    // ---- all warps join the sums of those that shared rows, a float4 of a row at a time
    const int sets = 1 << split;
    for (int i = threadIdx.x; i < x.rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4), w0 = r >> 3, in = r & 7;
      float m = -INFINITY;
      for (int w = w0; w < kWarps; w += sets) m = fmaxf(m, sm.base[w][in]);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      for (int w = w0; w < kWarps; w += sets) {
        const float bw = sm.base[w][in];
        if (bw == -INFINITY) continue;
        const float f = ex2(bw - m);
        const float4 v = *reinterpret_cast<const float4 *>(&sm.sum[w][in][c * 4]);
        a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
        sum = fmaf(f, sm.l[w][in], sum);
      }
      const int64_t at = x.part + r;
      *reinterpret_cast<float4 *>(p.part_o + at * D + c * 4) = a;
      if (c == 0) p.part_m[at] = m, p.part_l[at] = sum;
    }
  }

  // Adds the elements that are not finite of keys that a row sees, from the first block that was looked through.
  __device__ __noinline__ void put_back(const AttnPiece &x, int g, int lim, int least, float (&v)[4]) const {
    const int first = max(x.key0, x.low), c0 = g * KVX_Q4_GROUP + 4 * (lane >> 2);
    const int split = split_of(x.rows), start = first / kBlock * kBlock;
    for (int key = first; key < lim; ++key) {
      const int b = (key - start) / kBlock, pos = start + b * kBlock;
      if (b % (kWarps >> split) != warp >> split) continue;  // another warp's
      if (!(pos + kBlock > least || pos < x.low || pos + kBlock > x.key1)) continue;
      const char *at = p.pool.v + attn_key_offset(p, x.table, key, &sm.error) + h * p.pool.head_stride;
      const uint32_t pair = reinterpret_cast<const uint32_t *>(at)[D / 8 + g];
      if (!odd_word(pair)) continue;
      const uint32_t codes = reinterpret_cast<const uint16_t *>(at)[c0 / 4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += fmaf((float)(codes >> (4 * k) & 15u), low_half(pair), low_half(pair >> 16));
    }
  }
};

template <typename IO, int D>
__global__ void __launch_bounds__(kThreads, 2) attn_q4_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ char raw_smem[];
  using S = Smem<D>;
  S &sm = *reinterpret_cast<S *>(raw_smem + (-smem_u32(raw_smem) & 127));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sm.error = 0;
  // (what lies between the head vectors of a stage is read with them, and has to be finite)
  for (int i = tid; i < (int)sizeof(sm.ring) / 16; i += kThreads) reinterpret_cast<uint4 *>(sm.ring)[i] = make_uint4(0, 0, 0, 0);
  if (!p.after_wide) attn_wait_prior();
  else if (tid == 0) attn_wait_announced(p);  // for the others by the barrier below
  const int g = blockIdx.x / p.kv_heads, h = blockIdx.x - g * p.kv_heads;
  __syncthreads();
  const AttnLine line = attn_line<kThreads>(p, g, sm.scan);
  attn_release_next();  // the join takes its place as CTAs end, and waits for the last
  Loader<D> load(p, sm, h, lane, warp);
  Worker<IO, D> work{p, sm, load, h, lane, warp};
  for (int done = 0;; done += kPieces) {
    int n = 0;
    attn_pieces(p, g, h, line, [&](const AttnPiece &x) {
      if (tid == 0 && n >= done && n < done + kPieces) sm.pieces[n - done] = x;
      ++n;
    });
    if (tid == 0) sm.n_pieces = min(n - done, kPieces);
    __syncthreads();
    load.begin();
#pragma unroll 1
    for (int i = 0; i < S::kStages - 1; ++i) load.send();
#pragma unroll 1
    for (int i = 0; i < sm.n_pieces; ++i) work.piece(sm.pieces[i]);
    __syncthreads();
    if (n <= done + kPieces) break;
    // what was sent for no block is nothing: the ring begins anew
    cp_async_wait<0>();
    load.stage = work.stage = 0;
  }
  cp_async_wait<0>();
  if (tid == 0) p.errors[blockIdx.x] = sm.error;
  if (p.after_wide) attn_wait_prior();  // the join's wait for this kernel covers the wide one as well
}

template <typename IO, int D>
cudaError_t launch(const AttnParams &p, cudaStream_t s) {
  const void *fn = (const void *)attn_q4_kernel<IO, D>;
  constexpr int kSmem = (int)sizeof(Smem<D>) + 128;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  void *args[] = {const_cast<AttnParams *>(&p)};
  return launch_pdl(fn, dim3(p.groups * p.kv_heads), dim3(kThreads), args, s, kSmem);
}

}  // namespace

cudaError_t launch_attn_q4(const AttnParams &p, int32_t io, cudaStream_t s) {
  if (io == KVX_F16) return p.head_dim == 64 ? launch<__half, 64>(p, s) : launch<__half, 128>(p, s);
  return p.head_dim == 64 ? launch<__nv_bfloat16, 64>(p, s) : launch<__nv_bfloat16, 128>(p, s);
}

}  // namespace kvx
