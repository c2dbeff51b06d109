// kvx_attn.cuh -- what the kernels of kvx_shared_attention share.
//
// Rows and parts.  A row is (query token t, query head); the G = q_heads / kv_heads rows of a
// token that read one kv head lie together: row r of kv head h is token r / G, query head
// h * G + r % G.  Three kinds of work, each a set of rows with the keys they all read:
//   own      a request's rows and its positions behind the prefix;
//   prefix   the rows of many requests and the prefix;
//   prompt   a request with several tokens, more than 64 rows in all, and all its positions, prefix
//            included: it takes tiles of rows of its own, and one pass needs no join.
// The narrow kernel (and the plain one) takes units of up to row_tile rows: own work, and the
// prefix where there are few rows in all.  The wide kernel takes units of up to 256 rows: the
// prefix and prompts.  A unit's keys are cut into tiles, all units' key tiles stand in a line, each as
// long as its cost, and the line is dealt out evenly: group g of kv_heads CTAs, one CTA a head, takes
// the tiles that begin in [g * quota, (g + 1) * quota).  So every CTA has about the same work whatever
// the lengths, and the CTAs of a group read the heads of the same rows at the same time.
//
// A piece is what a CTA has of one unit.  It is worked through with a running maximum and sum and
// leaves, per row, the unnormalised sum o = sum_j e^(s_j - m) v_j in 32 bits, m and
// l = sum_j e^(s_j - m).  The piece that begins a unit leaves them at the rows' own place, one that
// goes on with a unit (there is at most one in a group) at the group's place.  The join adds the
// pieces of a row in the order of the line, so results do not depend on scheduling:
//   M = max m_i,  out = sum_i e^(m_i - M) o_i / sum_i e^(m_i - M) l_i.
// Scores are kept in units of log 2 (scale * k_scale * log2 e is folded into one factor), so the
// exponential is exp2.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kvx.h"

namespace kvx {

constexpr int kAttnKeyTile = 64;       // of the narrow and the plain kernel
constexpr int kAttnGeneralRows = 16;   // rows of a unit, plain kernel
constexpr int kAttnNarrowRows = 64;    // narrow kernel
constexpr int kAttnWideKeys = 128;     // key tile of the wide kernel
constexpr int kAttnWideRows = 256;     // rows of its units

constexpr int kAttnWritten = -2;

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

// Work of the narrow line: the prefix (first) or a request's own positions.
struct AttnSeg {
  int64_t tile0;       // where its first key tile begins in the line
  int32_t row0, rows;
  int32_t cost;        // of a tile
  int32_t low;         // its first position; tiles begin at multiples of their length, so that they
  int32_t key0, key1;  // hold whole pages: key0 is the first tile's begin, at most low
  int32_t key_tiles;   // of each unit; 0: no keys (or no rows)
  int32_t pad;
};

// A unit of the wide line.  table: the request of a prompt, -1: the prefix, whose rows are those
// of the tokens of prefix_tok.
struct AttnUnit {
  int64_t tile0;
  int32_t row0, rows;
  int32_t key_tiles, key1;
  int32_t table;
  int32_t pad;
};

struct AttnHeader {
  int64_t tiles, quota;            // the narrow line, and a group's part of it
  int64_t wide_tiles, wide_quota;
  int32_t refused;                 // 0, or the kvx_status that the arguments were refused with
  int32_t units;
  int32_t pad[6];
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
  int32_t key_bytes;     // of an element of the pool
  int32_t row_tile;      // rows of a narrow unit
  int32_t unit_cost;     // what a unit's begin and end cost, in tiles of up to 16 rows
  int32_t groups;        // groups of kv_heads CTAs, narrow line
  int32_t wide_groups;   // of the wide line; 0: no wide kernel
  int32_t planned;       // 1: the plan kernel has laid the work out.  0: one query token a request,
                         // and every kernel works its part out from the lengths
  int32_t after_wide;    // the narrow kernel runs beside the end of the wide kernel
  int32_t q_even;        // q's heads start on 4-byte boundaries
  int32_t q_vec;         // on 16-byte boundaries
  int32_t out_vec;       // out's heads do
  uint64_t call;         // unlike any other call's (see attn_announce)
  // workspace
  AttnHeader *head;
  uint64_t *ready;       // [1], calls with a wide kernel
  AttnSeg *segs;         // [1 + n_reqs]: the prefix, then the requests
  AttnUnit *units;
  int32_t *start;        // [groups + wide_groups]: the seg, or unit, that a group begins in
  int32_t *unit_base;    // [2 + n_reqs]: first wide unit of the prefix and of each request
  int32_t *prompt;       // [n_reqs]: INT32_MIN: prompt work; else what to add to a token for its
                         // place in prefix_tok
  int32_t *limit;        // [n_q]: positions that a token sees
  int32_t *owner;        // [n_q]: its request, -1: none, kAttnWritten: nothing is left to be joined
  int32_t *prefix_tok;   // [n_q]: tokens whose requests are not prompts, in order
  int32_t *prefix_at;    // [n_q]: a token's place in prefix_tok
  // part rows: [kv_heads][n_q * G] of own work's first pieces; the same of the prefix's and
  // prompts' first pieces; then pieces that go on, [groups][kv_heads][row_tile] and
  // [wide_groups][kv_heads][256]
  float *part_m, *part_l, *part_o;
  int32_t *errors;       // [n_errors]: one word of each CTA of the kernels before the join
  int32_t n_errors;
  int32_t *status;
};

// The page id of entry pg of a table (-1: the prefix list), as it stands there.
__device__ __forceinline__ int32_t attn_entry(const AttnParams &p, int32_t table, int64_t pg) {
  return table < 0 ? p.prefix_pages[pg] : p.tables[table * p.table_stride + pg];
}

// A page id checked: one outside the pool is reported in *error (of the CTA) and read as page 0.
// (Apart from the load, so that a look-up ahead of its use is not waited for at the check.)
__device__ __forceinline__ int32_t attn_checked(const AttnParams &p, int32_t id, int32_t *error) {
  if ((uint32_t)id >= (uint64_t)p.pool.num_pages) {
    *(volatile int32_t *)error = KVX_ERR_OUT_OF_RANGE;
    return 0;
  }
  return id;
}

// Page and offset of a position.
__device__ __forceinline__ void attn_split(const AttnParams &p, int32_t pos, int32_t *pg, int32_t *off) {
  if (p.pool.page_shift >= 0) {
    *pg = pos >> p.pool.page_shift;
    *off = pos & (p.page_size - 1);
  } else {
    *pg = pos / p.page_size;
    *off = pos - *pg * p.page_size;
  }
}

// Byte offset in a plane of position pos, kv head 0.
__device__ __forceinline__ int64_t attn_key_offset(const AttnParams &p, int32_t table, int32_t pos, int32_t *error) {
  int32_t pg, off;
  attn_split(p, pos, &pg, &off);
  return attn_checked(p, attn_entry(p, table, pg), error) * p.pool.page_stride + off * p.pool.tok_stride;
}

// A request's query tokens and length as the kernels use them: clamped into what can be
// addressed, whatever the arrays hold.
struct AttnReq {
  int32_t t0, n, len;
};

__device__ __forceinline__ AttnReq attn_request(const AttnParams &p, int b, int32_t *bad) {
  AttnReq r;
  r.t0 = b;
  r.n = 1;
  if (p.q_start) {
    const int32_t a = p.q_start[b], z = p.q_start[b + 1];
    if (a < 0 || z < a || z > p.n_q || (b == 0 && a != 0)) {
      *bad = max(*bad, (int32_t)KVX_ERR_INVALID_ARG);
      r.t0 = 0, r.n = 0;
    } else {
      r.t0 = a, r.n = z - a;
    }
  }
  r.len = p.seq_lens[b];
  if (r.len < 0) {
    *bad = max(*bad, (int32_t)KVX_ERR_INVALID_ARG);
    r.len = 0;
  } else if (r.len > (int64_t)p.max_pages * p.page_size || r.len > KVX_ATTN_MAX_POSITIONS) {
    // (so that a tile's end, and what the lanes of a warp look up behind it, are 32-bit positions)
    *bad = max(*bad, (int32_t)KVX_ERR_OUT_OF_RANGE);
    r.len = 0;
  }
  return r;
}

// Positions that token t sees.
__device__ __forceinline__ int32_t attn_limit(const AttnParams &p, int32_t t) {
  return p.planned ? p.limit[t] : max(0, p.seq_lens[t]);
}

// a / b for a >= 0, b > 0; in 32 bits, an order of magnitude sooner, where that is enough.
__device__ __forceinline__ int64_t attn_div(int64_t a, int64_t b) {
  if (((a | b) >> 31) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
__device__ __forceinline__ int64_t attn_up(int64_t a, int64_t b) { return attn_div(a + b - 1, b); }

// What a tile of a unit with that many rows costs: with up to 16 rows it is the bytes, with more the
// products, which four warps share between 16-row groups.  (Tiles of 64 rows take 2 to 4 times the time of
// tiles of 16 rows, depending on what else the SM has.)
__host__ __device__ __forceinline__ int32_t attn_cost(int32_t rows, int32_t row_tile) {
  const int32_t r = rows < row_tile ? rows : row_tile;
  return r <= 16 ? 1 : r <= 32 ? 2 : 4;
}

__device__ __forceinline__ int64_t attn_units(const AttnParams &p, int32_t rows) {
  return rows <= p.row_tile ? rows > 0 : attn_up(rows, p.row_tile);
}

// The length of a unit and of a seg in the line.  A unit's begin and end (its queries, joining its warps,
// its results) come behind its tiles.
__device__ __forceinline__ int64_t attn_unit_length(const AttnParams &p, const AttnSeg &g) {
  return g.key_tiles > 0 ? (int64_t)g.key_tiles * g.cost + p.unit_cost : 0;
}
__device__ __forceinline__ int64_t attn_length(const AttnParams &p, const AttnSeg &g) {
  return attn_units(p, g.rows) * attn_unit_length(p, g);
}

__device__ __forceinline__ void attn_tile_seg(const AttnParams &p, AttnSeg *g) {
  g->cost = attn_cost(g->rows, p.row_tile);
  g->key0 = g->low / kAttnKeyTile * kAttnKeyTile;
  if (g->rows > 0 && g->key1 > g->low)
    g->key_tiles = (int32_t)attn_up((int64_t)g->key1 - g->key0, kAttnKeyTile);
}

// Seg s of a call without a plan (its tile0 aside).
__device__ __forceinline__ AttnSeg attn_plain_seg(const AttnParams &p, int s, int32_t *bad) {
  AttnSeg g = {};
  if (s == 0) {
    if (p.wide_groups == 0) g.rows = p.n_q * p.group, g.key1 = p.prefix_len;
  } else {
    const AttnReq r = attn_request(p, s - 1, bad);
    g.row0 = r.t0 * p.group, g.rows = p.group;
    g.low = p.prefix_len, g.key1 = r.len;
  }
  attn_tile_seg(p, &g);
  return g;
}

// First part row of a piece of a narrow unit that starts at row0 (see AttnParams).
__device__ __forceinline__ int64_t attn_part(const AttnParams &p, bool prefix, bool first, int g,
                                             int h, int32_t row0) {
  const int64_t all = (int64_t)p.n_q * p.group;
  if (first) return ((prefix ? p.kv_heads : 0) + h) * all + row0;
  return 2 * p.kv_heads * all + ((int64_t)g * p.kv_heads + h) * p.row_tile;
}
// The same of the wide line: the place of row 0 of head h for first pieces, of the unit's first
// row for those that go on.
__device__ __forceinline__ int64_t attn_wide_part(const AttnParams &p, bool first, int g, int h) {
  const int64_t all = (int64_t)p.n_q * p.group;
  if (first) return (p.kv_heads + h) * all;
  return 2 * p.kv_heads * all + (int64_t)p.groups * p.kv_heads * p.row_tile +
         ((int64_t)g * p.kv_heads + h) * kAttnWideRows;
}

// The last of n entries (of segs or units) that starts at or before tile w: empty ones before it
// share its start.
template <typename E>
__device__ __forceinline__ int attn_find(const E *e, int n, int64_t w) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (e[mid].tile0 <= w) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A piece: keys [key0, key1), those below low left out, for rows [row0, row0 + rows).
struct AttnPiece {
  int64_t part;
  int32_t row0, rows, low, key0, key1, table;
};

// How many groups of each line have work.  Both lines at once, on SMs of their own, where that is
// estimated to end sooner than one after the other on all: the narrow line is bound by the bytes, which
// half of the SMs read nearly as fast as all of them (311 against 260 us for 1.57 GB), the wide line by its
// SMs.  Every kernel that needs it works it out by itself, in whole numbers, from the same totals.
struct AttnShare {
  int32_t groups, wide_groups;
};

// The GPU's SMs, and measured times in ns: of a CTA's tile of 128 keys and 256 rows; of a narrow CTA's unit
// of cost, two CTAs on the SM, at least, and of 16 bytes of a tile; of 1 MB at the memory's rate; and what a launch takes before and after its tiles.
constexpr int kAttnSms = 152;
constexpr int64_t kAttnWideNs = 2100, kAttnNarrowNs = 900, kAttnNarrowPs = 470, kAttnMbNs = 160,
                  kAttnStartNs = 10000;

__device__ __forceinline__ AttnShare attn_share(const AttnParams &p, int64_t own, int64_t wide) {
  AttnShare s = {p.groups, p.wide_groups};
  if (p.wide_groups < 2 || own == 0 || wide == 0) return s;
  const int64_t bytes = (int64_t)kAttnKeyTile * p.head_dim * p.key_bytes * 2;  // of a narrow tile
  const int64_t tiles = max(own - (int64_t)p.n_reqs * p.unit_cost, (int64_t)0);
  const int64_t floor_ns = (tiles * p.kv_heads * bytes >> 20) * kAttnMbNs;
  const int64_t unit_ns = max(kAttnNarrowNs, bytes / 16 * kAttnNarrowPs / 1000);
  auto narrow_ns = [&](int64_t groups) {
    return kAttnStartNs + max(attn_up(own, groups) * unit_ns, floor_ns);
  };
  auto wide_ns = [&](int64_t groups) { return kAttnStartNs + attn_up(wide, groups) * kAttnWideNs; };
  int64_t best = (wide_ns(p.wide_groups) + narrow_ns(p.groups)) * 9 / 10;  // a tenth sooner, or not at all
  int at = p.wide_groups;
  for (int g = 1 + (threadIdx.x & 31); g < p.wide_groups; g += 32) {
    const int left = (kAttnSms - g * p.kv_heads) * 2 / p.kv_heads;
    if (left < 1) continue;
    const int64_t a = wide_ns(g), b = narrow_ns(left), both = a > b ? a : b;
    if (both < best) best = both, at = g;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const int64_t b = __shfl_xor_sync(~0u, best, o);
    const int g = __shfl_xor_sync(~0u, at, o);
    if (b < best || (b == best && g < at)) best = b, at = g;
  }
  if (at < p.wide_groups) s.wide_groups = at, s.groups = min(p.groups, (kAttnSms - at * p.kv_heads) * 2 / p.kv_heads);
  return s;
}

// The wide line of a call without a plan: the prefix and all rows.
__device__ __forceinline__ int attn_plain_units(const AttnParams &p) {
  return p.prefix_len > 0 ? (int)attn_up((int64_t)p.n_q * p.group, kAttnWideRows) : 0;
}
__device__ __forceinline__ AttnUnit attn_plain_unit(const AttnParams &p, int u) {
  AttnUnit x = {};
  x.row0 = u * kAttnWideRows;
  x.rows = min(kAttnWideRows, p.n_q * p.group - x.row0);
  x.key1 = p.prefix_len;
  x.key_tiles = (int32_t)attn_up(p.prefix_len, kAttnWideKeys);
  x.tile0 = (int64_t)u * x.key_tiles;
  x.table = -1;
  return x;
}
__device__ __forceinline__ int64_t attn_plain_wide(const AttnParams &p) {
  return p.wide_groups ? (int64_t)attn_plain_units(p) * attn_plain_unit(p, 0).key_tiles : 0;
}

// The length of the narrow line of a call without a plan, added up by the CTA's Threads threads; *before,
// *mine: where the thread's segs begin and how long they are; returns the verdict on the arguments in
// *bad.  sm: two words a warp.
template <int Threads>
__device__ __forceinline__ int64_t attn_plain_total(const AttnParams &p, int64_t *sm, int64_t *before,
                                                    int64_t *mine, int32_t *bad) {
  constexpr int kWarps = Threads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = 1 + p.n_reqs;
  const int per = (n + Threads - 1) / Threads, s0 = min(tid * per, n), s1 = min(s0 + per, n);
  *bad = 0;
  *mine = 0;
  for (int s = s0; s < s1; ++s) *mine += attn_length(p, attn_plain_seg(p, s, bad));
  int64_t x = *mine;
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  for (int o = 16; o; o >>= 1) *bad = max(*bad, __shfl_xor_sync(~0u, *bad, o));
  if (lane == 31) sm[warp] = x, sm[kWarps + warp] = *bad;
  __syncthreads();
  int64_t total = 0;
  *before = x - *mine;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) *before += sm[i];
    total += sm[i];
    *bad = max(*bad, (int32_t)sm[kWarps + i]);
  }
  return total;
}

// Where a CTA's part of the narrow line begins.
struct AttnLine {
  int64_t w, end;     // its tiles
  int64_t tile0;      // first tile of seg
  int32_t seg;
};

// Group g's part, found by the CTA's Threads threads: by a search in the plan, or without one by adding
// up all lengths (the first CTA then leaves what the join needs).  sm: two words a warp and four more.
template <int Threads>
__device__ __forceinline__ AttnLine attn_line(const AttnParams &p, int g, int64_t *sm) {
  AttnLine l = {};
  if (p.planned) {
    const int64_t quota = p.head->quota;
    l.seg = p.start[g];
    if (p.head->refused) return l;
    l.w = g * quota;
    l.end = min(p.head->tiles, l.w + quota);
    if (l.w < l.end) l.tile0 = p.segs[l.seg].tile0;
    return l;
  }
  constexpr int kWarps = Threads / 32;
  const int tid = threadIdx.x, n = 1 + p.n_reqs;
  const int per = (n + Threads - 1) / Threads, s0 = min(tid * per, n), s1 = min(s0 + per, n);
  int32_t bad;
  int64_t before, mine;
  const int64_t total = attn_plain_total<Threads>(p, sm, &before, &mine, &bad), wide = attn_plain_wide(p);
  const AttnShare share = attn_share(p, total, wide);
  const int64_t quota = max((int64_t)1, attn_up(total, share.groups));
  if (blockIdx.x == 0) {
    int64_t at = before;
    for (int s = s0; s < s1; ++s) {
      AttnSeg g = attn_plain_seg(p, s, &bad);
      g.tile0 = at;
      p.segs[s] = g;
      at += attn_length(p, g);
    }
    if (tid == 0) {
      p.head->tiles = total, p.head->quota = quota, p.head->refused = bad;
      p.head->wide_quota = share.wide_groups ? max((int64_t)1, attn_up(wide, share.wide_groups)) : 1;
    }
  }
  l.w = g * quota;
  l.end = min(total, l.w + quota);
  if (bad || l.w >= l.end) {
    l.end = l.w;
    return l;
  }
  if (before <= l.w && l.w < before + mine) {
    int64_t at = before;
    for (int s = s0; s < s1; ++s) {
      const int64_t next = at + attn_length(p, attn_plain_seg(p, s, &bad));
      if (l.w < next) {
        sm[2 * kWarps] = s, sm[2 * kWarps + 1] = at;
        break;
      }
      at = next;
    }
  }
  __syncthreads();
  l.seg = (int32_t)sm[2 * kWarps];
  l.tile0 = sm[2 * kWarps + 1];
  return l;
}

// Calls f(piece) for every piece of group g, kv head h of the narrow line, l being its part.
template <typename F>
__device__ __forceinline__ void attn_pieces(const AttnParams &p, int g, int h, const AttnLine &l, F f) {
  int64_t w = l.w, tile0 = l.tile0;
  int32_t none = 0;
  for (int s = l.seg; w < l.end; ++s) {
    const AttnSeg seg = p.planned ? p.segs[s] : attn_plain_seg(p, s, &none);
    const int64_t unit_length = attn_unit_length(p, seg), length = attn_units(p, seg.rows) * unit_length;
    for (int64_t from = max(w - tile0, (int64_t)0), to = min(length, l.end - tile0); from < to;) {
      // the unit's tiles that begin in this group's part: kt .. kt + take - 1
      const int unit = (int)attn_div(from, unit_length);
      const int64_t begin = unit * unit_length;
      const int kt = (int)attn_up(from - begin, seg.cost);
      const int take = (int)min((int64_t)seg.key_tiles, attn_up(to - begin, seg.cost)) - kt;
      from = begin + unit_length;
      if (take <= 0) continue;
      AttnPiece x;
      x.row0 = seg.row0 + unit * p.row_tile;
      x.rows = min(p.row_tile, seg.rows - unit * p.row_tile);
      x.low = seg.low;
      x.key0 = seg.key0 + kt * kAttnKeyTile;
      x.key1 = (int32_t)min((int64_t)seg.key1, (int64_t)x.key0 + (int64_t)take * kAttnKeyTile);
      x.table = s - 1;
      x.part = attn_part(p, s == 0, kt == 0, g, h, x.row0);
      f(x);
    }
    tile0 += length;
    w = max(w, tile0);
  }
}

__device__ __forceinline__ void attn_wait_prior() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void attn_release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// What was there before the wide kernel (the plan, the queries, the pool) is visible to a kernel beside
// it, which does not wait for the wide kernel's end, by a release and an acquire: a thread of the wide
// kernel that has waited for all before stores the call's number, and only then lets its successor in; a
// thread of the narrow kernel that reads the number sees what the other saw.  One that reads anything else
// waits for the wide kernel's end.  The join clears the word, so that a call captured into a graph, whose
// number is the same in every replay, does not find its own of the time before.
__device__ __forceinline__ void attn_announce(const AttnParams &p) {
  asm volatile("st.release.gpu.global.b64 [%0], %1;" ::"l"(p.ready), "l"(p.call) : "memory");
}
__device__ __forceinline__ void attn_wait_announced(const AttnParams &p) {
  uint64_t x;
  asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(x) : "l"(p.ready) : "memory");
  if (x != p.call) attn_wait_prior();
}

// vec: heads are whole 16-byte pieces on 16-byte boundaries.
cudaError_t launch_attn_general(const AttnParams &p, int32_t dtype, int32_t io, bool vec, cudaStream_t s);
// head_dim 64 or 128, 16-bit or 8-bit pool with 16-byte aligned heads.
cudaError_t launch_attn_narrow(const AttnParams &p, int32_t dtype, int32_t io, bool hnd, cudaStream_t s);
cudaError_t launch_attn_wide(const AttnParams &p, int32_t dtype, int32_t io, bool hnd, cudaStream_t s);

}  // namespace kvx
