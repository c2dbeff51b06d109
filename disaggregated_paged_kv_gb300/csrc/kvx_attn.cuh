// kvx_attn.cuh -- what the kernels of kvx_shared_attention share.
//
// Rows and parts.  A row is (query token t, query head); the G = q_heads / kv_heads rows of a
// token that read one kv head lie together: row r of kv head h is token r / G, query head
// h * G + r % G.  The keys of a row are cut into the common prefix and the request's own
// positions, and each of the two into splits; a split of a run of rows is an item, which one CTA
// works through with a running maximum and sum.  It leaves, per row, the unnormalised sum
// o = sum_j e^(s_j - m) v_j in 32 bits, m and l = sum_j e^(s_j - m), and the join kernel adds the
// parts of a row in a fixed order:
//   M = max m_i,  out = sum_i e^(m_i - M) o_i / sum_i e^(m_i - M) l_i.
// Scores are kept in units of log 2 (scale * k_scale * log2 e is folded into one factor), so the
// exponential is exp2.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kvx.h"

namespace kvx {

constexpr int kAttnSplitTile = 64;   // splits are cut at multiples of this many keys
constexpr int kAttnMinSplit = 128;   // and are not made shorter than this

// Where a layer's rows are: element row (page id, offset in page, kv head) starts at
// plane + id * page_stride + offset * tok_stride + head * head_stride (bytes), in either kind of
// layout.
struct AttnPool {
  const char *k, *v;
  int64_t page_stride, tok_stride, head_stride;
  int64_t num_pages;     // valid ids are [0, num_pages)
  int32_t page_size;
  int32_t page_shift;    // log2(page_size), or -1
};

// One seg: the prefix (rows of all tokens) or a request (its own rows, its own positions).
struct AttnSeg {
  int64_t part;    // first partial row; kv head h, split s, local row i is partial row
                   // part + ((int64_t)h * splits + s) * rows + i
  int32_t row0;    // first row
  int32_t rows;
  int32_t key0, key1;
  int32_t splits;  // 0: no keys
  int32_t chunk;   // keys per split
};

struct AttnItem {
  int64_t part;    // partial row of the item's first row
  int32_t row0;    // first row, and how many (at most the kernel's tile)
  int32_t rows;
  int32_t key0, key1;
  int32_t table;   // request whose row names the pages; -1: the prefix list
  int32_t head;    // kv head
};

struct AttnHeader {
  int32_t n_items;
  int32_t prefix_splits;
  int32_t pad[14];
};

struct AttnParams {
  AttnPool pool;
  const int32_t *tables;
  int64_t table_stride;
  const int32_t *prefix_pages;
  const int32_t *seq_lens, *q_start;
  const char *q;
  char *out;
  int64_t q_tok, q_head, out_tok, out_head;  // bytes
  float *lse;
  float scale_log2;   // scale * k_scale * log2(e)
  float v_scale;
  int32_t n_q, n_reqs, q_heads, kv_heads, group, head_dim;
  int32_t page_size, max_pages, prefix_len;
  int32_t row_tile;   // most rows of an item
  int32_t target;     // items wanted
  int32_t max_items;
  // workspace
  AttnHeader *head;
  AttnSeg *segs;      // [1 + n_reqs]: the prefix, then the requests
  int32_t *item_base; // [2 + n_reqs]
  int32_t *limit;     // [n_q]: positions that a token sees
  int32_t *owner;     // [n_q]: its request, -1: none
  AttnItem *items;
  float *part_m, *part_l, *part_o;
  int64_t max_parts;
  int32_t *status;
};

// The page id of position pos for an item's table, checked: an id outside the pool is reported
// and read as page 0.
__device__ __forceinline__ int32_t attn_page(const AttnParams &p, int32_t table, int64_t pg) {
  const int32_t id = table < 0 ? p.prefix_pages[pg] : p.tables[table * p.table_stride + pg];
  if ((uint32_t)id >= (uint64_t)p.pool.num_pages) {
    atomicMax(p.status, (int32_t)KVX_ERR_OUT_OF_RANGE);
    return 0;
  }
  return id;
}

// Byte offset in a plane of position pos, kv head 0.
__device__ __forceinline__ int64_t attn_key_offset(const AttnParams &p, int32_t table, int32_t pos) {
  int32_t pg, off;
  if (p.pool.page_shift >= 0) {
    pg = pos >> p.pool.page_shift;
    off = pos & (p.page_size - 1);
  } else {
    pg = pos / p.page_size;
    off = pos - pg * p.page_size;
  }
  return attn_page(p, table, pg) * p.pool.page_stride + off * p.pool.tok_stride;
}

__device__ __forceinline__ void attn_wait_prior() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void attn_release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

cudaError_t launch_attn_general(const AttnParams &p, int32_t dtype, int32_t io, int grid,
                                cudaStream_t s);
constexpr int kAttnGeneralRows = 16;

}  // namespace kvx
