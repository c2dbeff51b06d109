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

inline bool ranges_overlap(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) {
  return a0 < b1 && b0 < a1;
}

inline bool layout_overlaps_range(const kvx_layout *l, uintptr_t b0, uintptr_t b1) {
  if (!ranges_overlap(l->lo, l->hi, b0, b1)) return false;
  for (int p = 0; p < l->planes; ++p)
    if (ranges_overlap(l->plane[p], l->plane[p] + l->extent, b0, b1)) return true;
  return false;
}
