// kvx_attn_q4.cu -- shared attention over a 4-bit pool for few rows a key: decode steps and short drafts.
//
// An element is low + code * scale, with a scale and a low for every 32 elements of a head (a group).  Codes go
// into the tensor cores as they are: the 4 bits, masked out of a word, are the f16 number code * 2^-24 (or
// 2^-20), exactly, so that unpacking is one AND an element pair.  With the scales left for later,
//   <q, k>       = sum_g scale_g <q_g, code_g> + low_g sum(q_g)
//   sum_j p_j v_j = sum_j (p_j scale_gj) code_j + p_j low_gj :
// the scores' sums of a group are multiplied by its scale in 32 bits; the weights, which are rounded to f16 for
// the product in any case, are multiplied by the scales of their keys' values, group by group, and rounded once more.  So
// that such a product is a normal f16 number, the scales are first multiplied by a power of two (see Worker::piece); where that
// would cost bits, or rows differ in what they see, the products are made in 32 bits (all of a call's: 256 requests 119 -> 136 us).
// The lows are a product of their own: (scale, low) words as they stand are its operand, against the sums of the
// queries (as two f16 numbers, so exact to 2^-22) and against the weights.
//
// Keys are the rows of both products (m16n8k16, M = 16 keys, N = 8 query rows; then M = 16 columns, K = 16
// keys): the eight columns suit a group of up to eight query heads.
//
// A head vector is 80 (or 40) bytes, so a CTA has up to eight neighbouring heads (a chunk).  A producer warp fills a ring
// of stages of 16 to 128 keys, by a tensor copy of 16 tokens of all heads where pages are multiples of that, else by
// a bulk copy a token; eight warps share the heads, the rows where there are more than eight, and blocks of 16 keys.
// Cycles of an SM a key and head (the memory's rate is 6.8): copies of 16 bytes by the computing warps themselves, a
// head a CTA, took 16, 9 of them for the copies alone (each fetches whole sectors of 32 bytes).  A bulk copy takes the
// copy engine some 45 cycles whatever its size: two a token of eight heads are 11.  By tensor copies it is 7.5 to 8.
//
// Bound: instructions, some 390 a block of 16 keys and head, close before the memory for long requests, and begins and ends of
// units for short ones.  In a graph, join included: one request of 2^20 tokens, 8 x 4 heads of 128, 267 us (its bytes 197), 328
// in pages of one token; one of 131072 tokens 63 us (25); 256 requests of 1000 to 2000 tokens 118 us (73); 64 of them behind
// 2048 shared tokens 61 us (19).
#include <type_traits>

#include "kvx_attn.cuh"
#include "kvx_attn_mma.cuh"
#include "kvx_attn_tma.cuh"
#include "kvx_launch.cuh"
#include "kvx_quant.cuh"

namespace kvx {
namespace {

constexpr int kWarps = kAttnQ4Warps, kThreads = kWarps * 32 + 32;
constexpr int kBlock = 16;    // keys at a time
constexpr int kRows = 8;      // of a warp
constexpr int kPieces = 32;   // listed at a time
constexpr int kStages = 3;
constexpr float kTop = 13.f;  // the greatest weight is about 2^kTop (see weight_shift)
constexpr float kRenew = 2.f; // by so many powers of two may a score pass what weights refer to
constexpr float kLeast = 0x1p-10f;  // scales this far below the greatest, or further, are multiplied in 32 bits

template <int D>
struct Smem {
  // head vectors of keys and of values, of at most 128 (key, head) pairs, tokens padded by up to 16 bytes
  static constexpr int kHalf = 128 * q4_bytes(D) + (D == 128 ? 1024 : 512);
  static constexpr int kSum = D + 4;  // floats of a row on its way to be joined
  alignas(128) char ring[kStages][2 * kHalf];
  alignas(16) float sum[kWarps][kRows][kSum];
  float base[kWarps][kRows], l[kWarps][kRows];
  uint32_t vector[128];  // where a stage's keys are, for copies of a part of a head
  AttnPiece pieces[kPieces];
  int64_t scan[2 * (kThreads / 32) + 4];
  uint64_t full[kStages], empty[kStages];
  int32_t n_pieces, lost, error;
};

// Copies 16 or 8 bytes, or zeros.
template <int B>
__device__ __forceinline__ void cp_async_if(uint32_t dst, const char *src, bool ok) {
  const int n = ok ? B : 0;
  if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *b) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const char *src, int bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t (&r)[2], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix2t(uint32_t (&r)[2], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t (&r)[2], uint32_t a) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t load_shared(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
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

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }
// Magnitudes of two f16 numbers, 0 for an infinity or NaN.
__device__ __forceinline__ __half2 finite_abs2(uint32_t x) {
  return as_half2((odd_word(x & 0xffffu) ? 0 : x & 0x7fffu) | (odd_word(x & 0xffff0000u) ? 0 : x & 0x7fff0000u));
}
// Of a positive normal number; and 2^e, e from -126 to 127.
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two 32-bit floats at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// What a CTA's warps have of a piece: slots of a chunk's heads (a power of two), and by each head's warps 2^split sets of
// eight rows and the blocks of 16 keys that are left to share.
struct Share {
  int32_t warps;      // a head's
  int32_t sets, keys; // sets * keys = warps
  int32_t start, stages;
  __device__ __forceinline__ Share(const AttnParams &p, const AttnPiece &x) {
    warps = kWarps >> p.slot_shift;
    sets = x.rows <= 8 ? 1 : x.rows <= 16 ? 2 : x.rows <= 32 ? 4 : 8;
    keys = warps / sets;
    const int32_t first = max(x.key0, x.low), stage = kBlock * warps;
    start = first / kBlock * kBlock;
    stages = x.key1 > first ? (x.key1 - start + stage - 1) / stage : 0;
  }
};

// Brings the stages of all pieces in, in order, by one warp.
template <int D>
struct Producer {
  using S = Smem<D>;
  static constexpr int kBytes = q4_bytes(D), kChunk = D / 8;  // of a head vector, and of a fifth of it
  const AttnParams &p;
  S &sm;
  const CUtensorMap *k_map, *v_map;
  const int h0, heads, lane;
  uint32_t stage = 0, phase = 1;
  bool lost = false;  // a wait was given up: nothing more is sent on its way

  // The page of position pos of a piece (a request's table, or the prefix's), as it stands there.
  __device__ __forceinline__ int32_t page_of(const AttnPiece &x, int32_t pos) const {
    if (pos < x.low || pos >= x.key1) return 0;
    int32_t pg, o;
    attn_split(p, pos, &pg, &o);
    return attn_entry(p, x.table, pg);
  }
  __device__ __forceinline__ void piece(const AttnPiece &x) {
    if (lost) return;
    const Share w(p, x);
    const int32_t keys = kBlock * w.warps;
    // look-ups, a stage ahead of their use: of blocks of 16 tokens, the lane pair's (lanes of K and V); of tokens, lane's,
    // lane + 32's and so on (16 keys: lanes of K and V)
    const bool boxes = p.q4_copies == kAttnQ4Boxes, pairs = keys == 16 && !boxes;
    int32_t id[4] = {};
    auto look = [&](int j) {
      if (j >= w.stages) return;
      const int32_t pos = w.start + j * keys;
      if (boxes) {
        if (lane >> 1 < w.warps) id[0] = page_of(x, max(pos + (lane >> 1) * kBlock, x.low));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i == 0 || i * 32 < keys) id[i] = page_of(x, pos + (pairs ? lane & 15 : i * 32 + lane));
      }
    };
    look(0);
    for (int j = 0; j < w.stages; ++j) {
      const int32_t pos = w.start + j * keys;
      int32_t now[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) now[i] = id[i];
      look(j + 1);
      lost = !__all_sync(~0u, bar_wait(&sm.empty[stage], phase, &sm.lost, &sm.error));
      if (lost) return;
      const uint32_t to = smem_u32(sm.ring[stage]);
      if (boxes) {
        // 16 tokens of all heads, whole: what lies beside the piece's keys, or the chunk's heads, is masked or not looked at
        const int32_t at = pos + (lane >> 1) * kBlock;
        if (lane == 0) bar_expect(&sm.full[stage], 2 * min(w.warps, (x.key1 - pos + kBlock - 1) / kBlock) * p.q4_block_pitch);
        if (lane >> 1 < w.warps && at < x.key1) {
          int32_t pg, o;
          attn_split(p, at, &pg, &o);
          const int32_t page = attn_checked(p, now[0], &sm.error);
          // (see attn_q4_maps)
          const int32_t cx = p.q4_runs ? o * (kBytes / 8) : 0, cy = p.q4_runs ? page * p.kv_heads + h0 : page * p.page_size + o;
          tma_load3(to + (lane >> 1) * p.q4_block_pitch + (lane & 1) * p.q4_v_off, lane & 1 ? v_map : k_map, cx, cy,
                    p.q4_runs ? 0 : h0 >> p.q4_pair, &sm.full[stage]);
        }
      } else if (p.q4_copies == kAttnQ4Tokens) {
        const int32_t first = max(pos, x.low), last = min(pos + keys, x.key1), bytes = heads * kBytes;
        if (lane == 0) bar_expect(&sm.full[stage], 2 * (last - first) * bytes);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t key = pairs ? lane & 15 : i * 32 + lane, at = pos + key;
          if ((i > 0 && i * 32 >= keys) || at < first || at >= last) continue;
          int32_t pg, o;
          attn_split(p, at, &pg, &o);
          const int64_t off = attn_checked(p, now[i], &sm.error) * p.pool.page_stride + o * p.pool.tok_stride + h0 * p.pool.head_stride;
          const uint32_t dst = to + key * p.q4_key_pitch;
          if (p.q4_v_off == bytes) {  // a token's values are behind its keys, here and there
            if (!pairs || lane < 16) bulk_copy(dst, p.pool.k + off, 2 * bytes, &sm.full[stage]);
          } else {
            if (!pairs || lane < 16) bulk_copy(dst, p.pool.k + off, bytes, &sm.full[stage]);
            if (!pairs || lane >= 16) bulk_copy(dst + p.q4_v_off, p.pool.v + off, bytes, &sm.full[stage]);
          }
        }
      } else {
        // a fifth of a head vector at a time; head vectors by their number in the plane (see AttnParams::page_vectors)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t key = i * 32 + lane, at = pos + key;
          if (key >= keys) continue;
          uint32_t n = ~0u;
          if (at >= x.low && at < x.key1) {
            int32_t pg, o;
            attn_split(p, at, &pg, &o);
            n = (uint32_t)attn_checked(p, now[i], &sm.error) * p.page_vectors + (uint32_t)o;
          }
          sm.vector[key] = n;
        }
        __syncwarp();
        const int chunks = heads * 5;
        for (int i = lane; i < keys * chunks; i += 32) {
          const int key = i / chunks, c = i - key * chunks, head = c / 5;
          const uint32_t n = sm.vector[key];
          const bool ok = n != ~0u;
          const int64_t off = (ok ? (int64_t)((uint64_t)n * (uint32_t)p.pool.tok_stride) : 0) + (h0 + head) * p.pool.head_stride + (c - head * 5) * kChunk;
          const uint32_t dst = to + key * p.q4_key_pitch + head * p.q4_head_pitch + (c - head * 5) * kChunk;
          cp_async_if<kChunk>(dst, p.pool.k + off, ok);
          cp_async_if<kChunk>(dst + p.q4_v_off, p.pool.v + off, ok);
        }
        // this lane's arrival when its copies are there
        asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&sm.full[stage])) : "memory");
        __syncwarp();  // (before the places are written anew)
      }
      if (++stage == kStages) stage = 0, phase ^= 1;
    }
  }
};

template <typename IO, int D>
struct Worker {
  using S = Smem<D>;
  static constexpr int G = D / KVX_Q4_GROUP;
  const AttnParams &p;
  S &sm;
  const int h, slot, sub, lane, warp;  // the kv head, its place in the chunk, and the warp's place among its
  uint32_t stage = 0, phase = 0;

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
    const Share share(p, x);
    const int set = sub & (share.sets - 1), first_block = sub / share.sets, c4 = lane & 3, r8 = lane >> 2;
    // ---- queries: of row set * 8 + r8, elements 8 c4 .. 8 c4 + 7 of every group, so that a word of codes
    // (eight elements of a key) meets them: pairs (0, 4), (1, 5), (2, 6), (3, 7), the odd ones divided by 16,
    // by which their codes are greater
    // (kept in shared memory, a group's four words of a lane together, where the warp's sums go in the end)
    if (share.warps > 1) head_sync(share);  // the sums of the piece before have been read
    const uint32_t q_at = smem_u32(&sm.sum[warp][0][0]) + lane * 16;
    uint32_t qs[2];
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
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(q_at + g * 512), "r"(pack2<__half>(e[g][0], e[g][4])),
                     "r"(pack2<__half>(e[g][1] * 0.0625f, e[g][5] * 0.0625f)), "r"(pack2<__half>(e[g][2], e[g][6])),
                     "r"(pack2<__half>(e[g][3] * 0.0625f, e[g][7] * 0.0625f)) : "memory");
      }
      mine *= 0.03125f;  // of at most 32 numbers up to 2^15: back into f16's range
      const __half hi = __float2half_rn(mine);
      qs[0] = (uint32_t)__half_as_ushort(hi) << 16;  // against (scale, low): nothing of the scale
      qs[1] = (uint32_t)__half_as_ushort(__float2half_rn(mine - __half2float(hi))) << 16;
    }
    // ---- of this lane's rows, set * 8 + 2 c4 and the one behind
    // (a base below any score: nothing seen yet)
    float sc[2], base[2] = {-3.40282347e38f, -3.40282347e38f}, l[2] = {0.f, 0.f};
    int lim[2];
    const int first = max(x.key0, x.low);
    int least = INT32_MAX, most = 0;  // of the warp's rows that see some of the piece
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sc[i] = p.scale_log2 * __shfl_sync(~0u, factor, (2 * c4 + i) * 4);
      const int r = set * kRows + 2 * c4 + i;
      lim[i] = r < x.rows ? min(attn_limit(p, (x.row0 + r) / p.group), x.key1) : 0;
      if (lim[i] > first) least = min(least, lim[i]), most = max(most, lim[i]);
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      least = min(least, __shfl_xor_sync(~0u, least, d));
      most = max(most, __shfl_xor_sync(~0u, most, d));
    }
    float o[G][2][4] = {}, z[4] = {};  // z: of the unit of (scale, low) words that is r8's
    int odd = 0;
    // Weights' products with the values' scales are f16 numbers, up_by times what they are.  up_by is a power of two, by which
    // the greatest scale of the piece so far comes to 1/2 .. 1, the same for all rows.  While no other scale but 0 then is below
    // kLeast, scales times up_by are exact, and products of weights far below the greatest are normal numbers still.  From
    // the first that is below, and from where on rows differ in what they see, products are made in 32 bits and rounded once, and up_by
    // is of row r8, by its greatest product in the block.
    float up_by = 0x1p15f;
    bool apart = false;
    const uint32_t kp = p.q4_key_pitch, mine = (slot >> p.q4_pair) * p.q4_head_pitch + (slot & p.q4_pair) * q4_bytes(D);
    const uint32_t row16 = mine + (lane & 15) * kp, row8 = mine + r8 * kp;

#pragma unroll 1
    for (int j = 0; j < share.stages; ++j) {
      bar_wait(&sm.full[stage], phase, &sm.lost, &sm.error);  // (given up: what follows is of no account)
      __syncwarp();
      const uint32_t ring = smem_u32(sm.ring[stage]);
#pragma unroll 1
      for (int b = first_block; b < share.warps; b += share.keys) {
      const int pos = share.start + (j * share.warps + b) * kBlock;
      if (pos >= x.key1) break;
      const uint32_t kt = ring + b * p.q4_block_pitch, vt = kt + p.q4_v_off;
      const bool mixed = pos + kBlock > least || pos < x.low;  // (no row sees further than key1)
      // ---- scores of keys r8 and r8 + 8
      float s[4];
      uint32_t ks[2][G];  // (scale, low) of the two keys
#pragma unroll
      for (int i = 0; i < 2; ++i) load_shared(ks[i], kt + row8 + 8 * i * kp + D / 2);
      {
        float a[4] = {};
        uint32_t w[2];
        if constexpr (G == 4) {
          ldmatrix2(w, kt + row16 + D / 2);
        } else {
          w[0] = c4 == 0 ? ks[0][0] : c4 == 1 ? ks[0][1] : 0, w[1] = c4 == 0 ? ks[1][0] : c4 == 1 ? ks[1][1] : 0;
        }
        const uint32_t f[4] = {w[0], w[1], w[0], w[1]};
        mma16816<__half>(a, f, qs[0], qs[1]);
        unpair(mul2(pair(a[0], a[1]), pair(0x1p-19f, 0x1p-19f)), s[0], s[1]);
        unpair(mul2(pair(a[2], a[3]), pair(0x1p-19f, 0x1p-19f)), s[2], s[3]);
      }
#pragma unroll
      for (int g = 0; g < G; g += 2) {
        uint32_t w[4];
        if constexpr (G == 4) {
          ldmatrix4(w, kt + row16 + (g + (lane >> 4)) * 16);
        } else {  // (head vectors of 40 bytes: an odd one is off 16 bytes)
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = load_shared(kt + row8 + 8 * (i & 1) * kp + (i >> 1) * 16 + c4 * 4);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t u = w[2 * e], v = w[2 * e + 1];
          float a[4] = {};
          uint32_t q[4];
          load_shared(q, q_at + (g + e) * 512);
          const uint32_t f0[4] = {u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u};
          mma16816<__half>(a, f0, q[0], q[1]);
          const uint32_t u8 = u >> 8, v8 = v >> 8;
          const uint32_t f1[4] = {u8 & 0x000f000fu, v8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x00f000f0u};
          mma16816<__half>(a, f1, q[2], q[3]);
          const float s0 = low_half(ks[0][g + e]), s1 = low_half(ks[1][g + e]);
          s[0] = fmaf(a[0], s0, s[0]), s[1] = fmaf(a[1], s0, s[1]);
          s[2] = fmaf(a[2], s1, s[2]), s[3] = fmaf(a[3], s1, s[3]);
        }
      }
      const uint64_t up24 = pair(0x1p24f, 0x1p24f), sc2 = pair(sc[0], sc[1]);
      unpair(mul2(mul2(pair(s[0], s[1]), up24), sc2), s[0], s[1]);
      unpair(mul2(mul2(pair(s[2], s[3]), up24), sc2), s[2], s[3]);
      if (mixed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = pos + r8 + (i >> 1) * 8;
          if (key < x.low || key >= lim[i & 1]) s[i] = -INFINITY;
        }
      }
      // ---- the values' (scale, low) words, a unit a lane's row
      uint32_t zw[2];
      if constexpr (G == 4) {
        ldmatrix2t(zw, vt + row16 + D / 2);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) zw[i] = transpose8(c4 < 2 ? load_shared(vt + row8 + 8 * i * kp + D / 2 + c4 * 4) : 0);
      }
      if (mixed) {
        // Nothing of keys that no row sees; infinities and NaN of keys that some row does not see are taken out and put
        // back at the end.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = pos + 2 * c4 + 8 * i;
          if (key < x.low || key >= most) zw[i] &= 0xffff0000u;
          if (key + 1 < x.low || key + 1 >= most) zw[i] &= 0xffffu;
          if (odd_word(zw[i] & 0xffffu)) zw[i] &= 0xffff0000u, odd = 1;
          if (odd_word(zw[i] & 0xffff0000u)) zw[i] &= 0xffffu, odd = 1;
        }
      }
      // ---- weights; what they refer to is renewed where a score passes it by far, up_by where a scale asks for it
      float e[4] = {s[0] - base[0], s[1] - base[1], s[2] - base[0], s[3] - base[1]};
      uint32_t zs[2];  // the scales times up_by
      auto scales_fit = [&]() {
        // (units of scales; lows are of no account)
        const __half2 none = as_half2(0), by = __float2half2_rn(up_by), s0 = as_half2(r8 & 1 ? 0 : zw[0]), s1 = as_half2(r8 & 1 ? 0 : zw[1]);
        const __half2 a = __hmul2(s0, by), b = __hmul2(s1, by);
        zs[0] = as_word(a), zs[1] = as_word(b);
        // (0 counts as 1)
        const __half2 a1 = __hadd2(__habs2(a), __heq2(s0, none)), b1 = __hadd2(__habs2(b), __heq2(s1, none));
        return __hbge2(__hmin2(a1, b1), __float2half2_rn(kLeast)) && __hble2(__hmax2(a1, b1), as_half2(0x3c003c00u));
      };
      if (least < most && pos + kBlock > least) apart = true;  // rows differ in what they see, from here to the end
      const bool fit = scales_fit() || apart;
      if (__any_sync(~0u, fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])) > kTop + kRenew || !fit)) {
        float n0 = fmaxf(s[0], s[2]), n1 = fmaxf(s[1], s[3]), change = 1.f;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, d));
          n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, d));
        }
        if (!apart) {
          const __half2 most2 = r8 & 1 ? as_half2(0) : __hmax2(finite_abs2(zw[0]), finite_abs2(zw[1]));
          float up = fmaxf(__low2float(most2), __high2float(most2));
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, d));
          if (up * up_by > 1.f) {
            const float now = power_of_2(-1 - exponent(up));
            change = now * __frcp_rn(up_by), up_by = now;
          }
          apart = !__all_sync(~0u, scales_fit());
        }
        // each row by its own scores: what others see is nothing to it
        const float b0 = n0 > base[0] + (kTop + kRenew) ? n0 - kTop : base[0], b1 = n1 > base[1] + (kTop + kRenew) ? n1 - kTop : base[1];
        const float f0 = ex2(base[0] - b0), f1 = ex2(base[1] - b1);
        l[0] *= f0, l[1] *= f1;
        scale_sums(o, f0 * change, f1 * change);
        z[0] *= f0, z[1] *= f1;
        base[0] = b0, base[1] = b1;
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = s[i] - base[i & 1];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = ex2(e[i]);
      l[0] += e[0] + e[2], l[1] += e[1] + e[3];
      // rounded to f16 for the products (their sum is not), rows and keys exchanged: row r8, keys 2 c4, 2 c4 + 1 and 8 behind
      const uint32_t p0 = transpose8(pack2<__half>(e[0], e[1])), p1 = transpose8(pack2<__half>(e[2], e[3]));
      {
        const uint32_t f[4] = {zw[0], 0, zw[1], 0};
        mma16816<__half>(z, f, p0, p1);
      }
      if (apart) {
        __half2 h[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          h[i] = r8 & 1 ? as_half2(0) : finite_abs2(zw[i]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) h[i] = __hmax2(h[i], as_half2(__shfl_xor_sync(~0u, as_word(h[i]), d)));
        }
        float m = fmaxf(fmaxf(low_half(p0) * __low2float(h[0]), low_half(p0 >> 16) * __high2float(h[0])),
                        fmaxf(low_half(p1) * __low2float(h[1]), low_half(p1 >> 16) * __high2float(h[1])));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
        float change = 1.f;
        if (m > 0.f && !(m * up_by >= 1.f && m * up_by <= 0x1p14f)) {
          const float now = power_of_2(13 - exponent(m));
          change = now * __frcp_rn(up_by), up_by = now;
        }
        if (__any_sync(~0u, change != 1.f)) scale_sums(o, __shfl_sync(~0u, change, c4 * 8), __shfl_sync(~0u, change, c4 * 8 + 4));
      }
      auto values = [&](auto exact) {
#pragma unroll
        for (int g = 0; g < G; g += 2) {
          uint32_t w[4];
          if constexpr (G == 4) {
            ldmatrix4t(w, vt + row16 + (g + (lane >> 4)) * 16);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = transpose8(load_shared(vt + row8 + 8 * (i & 1) * kp + (i >> 1) * 16 + c4 * 4));
          }
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            // the group's scales of keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9, from the lanes whose row is their unit
            const int from = (g + e2) * 8 + c4;
            uint32_t b0, b1;
            if constexpr (decltype(exact)::value) {
              b0 = __shfl_sync(~0u, zw[0], from), b1 = __shfl_sync(~0u, zw[1], from);
              b0 = pack2<__half>(low_half(p0) * up_by * low_half(b0), low_half(p0 >> 16) * up_by * low_half(b0 >> 16));
              b1 = pack2<__half>(low_half(p1) * up_by * low_half(b1), low_half(p1 >> 16) * up_by * low_half(b1 >> 16));
            } else {
              b0 = mul_half2(p0, __shfl_sync(~0u, zs[0], from)), b1 = mul_half2(p1, __shfl_sync(~0u, zs[1], from));
            }
            const uint32_t u = w[2 * e2], v = w[2 * e2 + 1], u8 = u >> 8, v8 = v >> 8;
            const uint32_t f0[4] = {u & 0x000f000fu, u8 & 0x000f000fu, v & 0x000f000fu, v8 & 0x000f000fu};
            mma16816<__half>(o[g + e2][0], f0, b0, b1);
            const uint32_t f1[4] = {u & 0x00f000f0u, u8 & 0x00f000f0u, v & 0x00f000f0u, v8 & 0x00f000f0u};
            mma16816<__half>(o[g + e2][1], f1, b0, b1);
          }
        }
      };
      if (apart) values(std::true_type());
      else values(std::false_type());
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&sm.empty[stage]);
      if (++stage == kStages) stage = 0, phase ^= 1;
    }
    // ---- the warp's sums: columns 32 g + 4 r8 .. + 3 of its two rows
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l[0] += __shfl_xor_sync(~0u, l[0], d);
      l[1] += __shfl_xor_sync(~0u, l[1], d);
    }
    odd = __any_sync(~0u, odd);
    const int64_t part = x.part + h * x.head_step;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float down = __frcp_rn(__shfl_sync(~0u, up_by, (2 * c4 + i) * 4));
      const bool none = lim[i] <= first || l[i] == 0.f;  // (a row that sees nothing of the piece has worked on all)
      const int in = 2 * c4 + i, r = set * kRows + in;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float low = __shfl_sync(~0u, z[i], (2 * g + 1) * 4 + c4);
        float v[4] = {fmaf(o[g][0][i], 0x1p24f * down, low), fmaf(o[g][1][i], 0x1p20f * down, low),
                      fmaf(o[g][0][2 + i], 0x1p24f * down, low), fmaf(o[g][1][2 + i], 0x1p20f * down, low)};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = none ? 0.f : v[k];
        const float4 out = make_float4(v[0], v[1], v[2], v[3]);
        const int d = g * KVX_Q4_GROUP + 4 * r8;
        if (share.keys > 1) *reinterpret_cast<float4 *>(&sm.sum[warp][in][d]) = out;
        else if (r < x.rows) *reinterpret_cast<float4 *>(p.part_o + (part + r) * D + d) = out;
      }
      const float m = none ? -INFINITY : base[i], sum = none ? 0.f : l[i];
      if (r8 == 0) {
        if (share.keys > 1) sm.base[warp][in] = m, sm.l[warp][in] = sum;
        else if (r < x.rows) p.part_m[part + r] = m, p.part_l[part + r] = sum;
      }
    }
    if (odd) {
      __syncwarp();
      put_back(x, share, part, set, least, lim[0] <= first || l[0] == 0.f ? 0 : lim[0], lim[1] <= first || l[1] == 0.f ? 0 : lim[1]);
    }
    if (share.keys == 1) return;
    head_sync(share);
    // ---- the head's warps join the sums of those that shared rows, a float4 of a row at a time
    const int w00 = slot * share.warps;
    for (int i = sub * 32 + lane; i < x.rows * (D / 4); i += share.warps * 32) {
      const int r = i / (D / 4), c = i % (D / 4), w0 = w00 + (r >> 3), in = r & 7;
      float m = -INFINITY;
      for (int w = w0; w < w00 + share.warps; w += share.sets) m = fmaxf(m, sm.base[w][in]);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      for (int w = w0; w < w00 + share.warps; w += share.sets) {
        const float bw = sm.base[w][in];
        if (bw == -INFINITY) continue;
        const float f = ex2(bw - m);
        const float4 v = *reinterpret_cast<const float4 *>(&sm.sum[w][in][c * 4]);
        a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
        sum = fmaf(f, sm.l[w][in], sum);
      }
      const int64_t at = part + r;
      *reinterpret_cast<float4 *>(p.part_o + at * D + c * 4) = a;
      if (c == 0) p.part_m[at] = m, p.part_l[at] = sum;
    }
  }

  // The sums of a lane's two rows, times a factor each.
  __device__ __forceinline__ static void scale_sums(float (&o)[G][2][4], float f0, float f1) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int k = 0; k < 2; ++k) o[g][k][0] *= f0, o[g][k][1] *= f1, o[g][k][2] *= f0, o[g][k][3] *= f1;
  }

  // The warps of a head.
  __device__ __forceinline__ void head_sync(const Share &share) const {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(share.warps * 32) : "memory");
  }

  // Adds the elements that are not finite of keys that a row sees, of the blocks that were looked through, to the sums
  // as they have been written.
  __device__ __forceinline__ void put_back(const AttnPiece &x, const Share &share, int64_t part, int set, int least, int lim0, int lim1) const {
    const int first = max(x.key0, x.low), c4 = lane & 3, r8 = lane >> 2;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const int in = 2 * c4 + i, lim = i ? lim1 : lim0;
#pragma unroll 1
      for (int key = first; key < lim; ++key) {
        const int b = (key - share.start) / kBlock, pos = share.start + b * kBlock;
        if (b % share.warps % share.keys != sub / share.sets) continue;  // another warp's
        if (!(pos + kBlock > least || pos < x.low)) continue;
        const char *at = p.pool.v + attn_key_offset(p, x.table, key, &sm.error) + h * p.pool.head_stride;
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
          const uint32_t pair = reinterpret_cast<const uint32_t *>(at)[D / 8 + g];
          if (!odd_word(pair)) continue;
          const int d = g * KVX_Q4_GROUP + 4 * r8;
          const uint32_t codes = reinterpret_cast<const uint16_t *>(at)[d / 4];
          float *o = share.keys > 1 ? &sm.sum[warp][in][d] : p.part_o + (part + set * kRows + in) * D + d;
          for (int k = 0; k < 4; ++k) o[k] += fmaf((float)(codes >> (4 * k) & 15u), low_half(pair), low_half(pair >> 16));
        }
      }
    }
  }
};

template <typename IO, int D>
__global__ void __launch_bounds__(kThreads, 2) attn_q4_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ char raw_smem[];
  using S = Smem<D>;
  S &sm = *reinterpret_cast<S *>(raw_smem + (-smem_u32(raw_smem) & 127));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x / p.group_ctas, h0 = (blockIdx.x - g * p.group_ctas) * p.chunk;
  const int heads = min(p.chunk, p.kv_heads - h0), warps = kWarps >> p.slot_shift;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i)
      bar_init(&sm.full[i], p.q4_copies == kAttnQ4Parts ? 32 : 1), bar_init(&sm.empty[i], heads * warps);
    sm.lost = sm.error = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // (what no copy has written is read with the rest, and masked by finite numbers)
  for (int i = tid; i < (int)sizeof(sm.ring) / 16; i += kThreads) reinterpret_cast<uint4 *>(sm.ring)[i] = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (!p.after_wide) attn_wait_prior();
  else if (tid == 0) attn_wait_announced(p);  // for the others by the barrier below
  __syncthreads();
  const AttnLine line = attn_line<kThreads>(p, g, sm.scan);
  attn_release_next();  // the join takes its place as CTAs end, and waits for the last
  // Calls f(piece) for the CTA's pieces, listed some at a time; all threads come along.
  auto all_pieces = [&](auto f) {
    for (int done = 0;; done += kPieces) {
      int n = 0;
      attn_pieces(p, g, 0, line, [&](const AttnPiece &x) {
        if (tid == 0 && n >= done && n < done + kPieces) sm.pieces[n - done] = x;
        ++n;
      });
      if (tid == 0) sm.n_pieces = max(0, min(n - done, kPieces));
      __syncthreads();
      const int count = sm.n_pieces;
#pragma unroll 1
      for (int i = 0; i < count; ++i) f(sm.pieces[i]);
      __syncthreads();
      if (n <= done + kPieces) break;
    }
  };
  Producer<D> producer{p, sm, &k_map, &v_map, h0, heads, lane};
  if (warp < kWarps) {
    const int slot = warp / warps;
    Worker<IO, D> work{p, sm, h0 + slot, slot, warp - slot * warps, lane, warp};
    all_pieces([&](const AttnPiece &x) {
      if (slot < heads) work.piece(x);
    });
  } else {
    // (no kernel's end lies between the pool's writes and these copies)
    if (p.after_wide) asm volatile("fence.proxy.async.global;" ::: "memory");
    all_pieces([&](const AttnPiece &x) {
      producer.piece(x);
    });
  }
  if (sm.lost) {
    if (warp == kWarps) {
      cp_async_commit();
      cp_async_wait<0>();
      bar_drain<kStages>(sm.full, producer.stage, producer.phase);
    }
    __syncthreads();
  }
  if (tid < heads) p.errors[g * p.kv_heads + h0 + tid] = sm.error;
  if (p.after_wide) attn_wait_prior();  // the join's wait for this kernel covers the wide one as well
}

template <typename IO, int D>
cudaError_t launch(const AttnParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map, cudaStream_t s) {
  const void *fn = (const void *)attn_q4_kernel<IO, D>;
  constexpr int kSmem = (int)sizeof(Smem<D>) + 128;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  void *args[] = {const_cast<AttnParams *>(&p), const_cast<CUtensorMap *>(&k_map), const_cast<CUtensorMap *>(&v_map)};
  return launch_pdl(fn, dim3(p.groups * p.group_ctas), dim3(kThreads), args, s, kSmem);
}

}  // namespace

cudaError_t launch_attn_q4(const AttnParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map, int32_t io, cudaStream_t s) {
  if (io == KVX_F16) return p.head_dim == 64 ? launch<__half, 64>(p, k_map, v_map, s) : launch<__half, 128>(p, k_map, v_map, s);
  return p.head_dim == 64 ? launch<__nv_bfloat16, 64>(p, k_map, v_map, s) : launch<__nv_bfloat16, 128>(p, k_map, v_map, s);
}

}  // namespace kvx
