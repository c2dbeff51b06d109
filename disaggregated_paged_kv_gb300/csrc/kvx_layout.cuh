// kvx_layout.cuh -- the layout handle behind kvx_layout_t, shared by the host sides of every call.
#pragma once

#include <cstdint>

#include "kvx.h"

struct kvx_layout {
  int32_t num_layers, kv_heads, head_dim, elem, kind, page_size;
  int32_t dtype;      // kvx_dtype: copies use only its width, attention its values
  int32_t kv_planes;  // planes per layer: 2 (K, V) or 1 (MLA latent)
  int32_t vec;        // widest access (16, 8, 4, 2, 1 bytes) every row and head vector allows
  int32_t planes;
  int64_t num_slots;
  int64_t row_bytes, seg_bytes;
  int64_t slot_stride;  // NHD
  int64_t page_bytes;   // HND
  int64_t extent;       // bytes one plane spans from its start
  uintptr_t lo, hi;     // envelope of all planes
  uintptr_t plane[KVX_MAX_PLANES];
};
