// kvx_quant.cuh -- what the host hands the kernels of kvx_store_kv and kvx_load_kv, and the arithmetic of
// 4-bit groups.
#pragma once

#include <cuda_fp16.h>

#include "kvx_internal.cuh"

namespace kvx {

struct QuantArgs {
  Side pool;
  const int32_t *slots, *rows;   // rows: nullptr: token i is row i
  int64_t n, n_rows;
  int32_t planes;                // 2 * layers, K and V in turn
  int32_t heads, head_dim;
  int32_t check;                 // 1: every CTA checks every index; 0: *status is the planner's verdict
  int32_t wide;                  // k, v and their strides are multiples of 16 bytes
  int32_t words;                 // head vectors are on 8-byte boundaries (8-bit pools: and multiples of that)
  int32_t parts, turns;          // of a row, where it is more than a CTA's; of a CTA (set by launch_quant)
  char *k, *v;
  int64_t layer_stride, token_stride, head_stride;  // bytes
  float scale[2];                // of K and V: store: 1 / scale
  int32_t *status;
  char *base[KVX_MAX_PLANES];
};

cudaError_t launch_quant(QuantArgs &q, bool store, bool q4, int32_t dtype, cudaStream_t s);

// A head vector of a KVX_Q4 pool: head_dim / 2 bytes of codes, then the groups' (scale, low).
__host__ __device__ __forceinline__ constexpr int32_t q4_bytes(int32_t head_dim) { return head_dim / 8 * 5; }

}  // namespace kvx
