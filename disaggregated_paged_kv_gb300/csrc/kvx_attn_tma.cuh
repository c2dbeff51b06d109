// kvx_attn_tma.cuh -- how the tensor-core attention kernels bring key and value tiles to shared
// memory: barriers with bounded waits, tensor copies of whole pages, and the tiles' arrangement.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "kvx_attn.cuh"
#include "kvx_attn_mma.cuh"

namespace kvx {

// How tiles come by tensor copies: boxes of `rows` (a multiple of 8) consecutive tokens of one page
// and head.  A plane is seen as [group of 8 tokens][block of 64 16-bit columns][token][column] (8-bit
// pools: [token][column]), so that a box arrives as the matrix operand's own arrangement.
struct AttnTma {
  int32_t rows;       // 0: no tensor copies (pages too short, or too many rows for an index)
  int32_t head_x;     // a head's first block (8-bit pools: column): head * head_x
  int64_t page_y, head_y;  // first token of (page, head): page * page_y + head * head_y
};

// A tile of D 16-bit columns a row: groups of eight rows, in them blocks of 64 columns, in them eight
// rows of 128 bytes whose 16-byte chunks are exchanged by the row (128-byte swizzle), so that eight rows
// of one chunk lie in different banks.  Byte place of 16-byte chunk c (of D / 8) of row r.
template <int D>
__device__ __forceinline__ uint32_t place(int r, int c) {
  return (uint32_t)((r >> 3) * (D * 16) + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The same of an 8-bit tile as it comes: rows of D bytes, chunks exchanged by the row.
template <int D>
__device__ __forceinline__ uint32_t place8(int r, int c) {
  return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// No wait of a kernel takes as many polls unless it is lost.
constexpr uint32_t kAttnPolls = 1u << 19;

// ---- barriers ------------------------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint64_t *b, int n) {
  asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ void bar_expect(uint64_t *b, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load4(void *dst, const CUtensorMap *map, int z, int y, uint64_t *b) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(0), "r"(0), "r"(z), "r"(y), "r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int x, int y, uint64_t *b) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(b)) : "memory");
}
// Waits for a phase.  False when the wait is given up: after so many polls (a poll waits some
// microseconds itself), or because some other wait of the CTA was.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, int32_t *lost, int32_t *error,
                                         uint32_t polls = kAttnPolls) {
  for (uint32_t n = 0; !bar_try(b, parity); ++n) {
    if (*(volatile int32_t *)lost) return false;
    if (n == polls) {
      *(volatile int32_t *)lost = 1;
      *(volatile int32_t *)error = KVX_ERR_TIMEOUT;
      return false;
    }
  }
  return true;
}

// When a wait of the CTA was given up: waits until what a thread has sent on its way to a ring of Stages
// stages is there (stage and phase: those of the `empty` barrier that it would wait for next), so that nothing
// arrives in memory that the CTA has given back.  A stage that some threads did not fill any more is never
// full; after kAttnDrainPolls polls its copies, which depend on nothing, are there.
constexpr uint32_t kAttnDrainPolls = 1u << 11;
template <int Stages>
__device__ __forceinline__ void bar_drain(uint64_t *full, uint32_t stage, uint32_t phase) {
  for (uint32_t i = 0; i < Stages; ++i) {
    const uint32_t parity = i < stage ? phase ^ 1 : phase;
    for (uint32_t n = 0; n < kAttnDrainPolls && !bar_try(&full[i], parity); ++n) {}
  }
}

// The planes of a call as AttnTma says, for tiles of `keys` keys.  Boxes are whole groups of 8 tokens of a
// page; with other pages, or more rows than an index counts, the tiles come key by key (t->rows 0).
void attn_make_tma(const AttnParams &p, int keys, bool fp8, bool hnd, AttnTma *t, CUtensorMap *km,
                   CUtensorMap *vm);

}  // namespace kvx
