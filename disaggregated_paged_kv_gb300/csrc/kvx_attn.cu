// kvx_attn.cu -- kvx_shared_attention: checks, the plan, the join, and the choice of kernels.
//
// Lengths and query starts are device data, so the work is laid out on the device: a one-CTA
// plan kernel adds up the key tiles of all units, and the kernels behind it walk that line with a
// grid that does not depend on it.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvx_attn.cuh"
#include "kvx_attn_tma.cuh"
#include "kvx_internal.cuh"
#include "kvx_launch.cuh"
#include "kvx_layout.cuh"

namespace kvx {
namespace {

constexpr int kPlanCta = 1024;

// Exclusive block-wide sum; *total gets the whole.
__device__ __forceinline__ int64_t block_excl(int64_t x, int64_t *total, int64_t *sm) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, y, d);
    if (lane >= d) y += u;
  }
  __syncthreads();
  if (lane == 31) sm[w] = y;
  __syncthreads();
  int64_t z = lane < nw ? sm[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, z, d);
    if (lane >= d) z += u;
  }
  *total = __shfl_sync(~0u, z, 31);
  const int64_t before = __shfl_sync(~0u, z, (w + 31) & 31);
  return (w ? before : 0) + y - x;
}

// The last b in [0, n) with base[b] <= x.
__device__ __forceinline__ int last_at_or_before(const int32_t *base, int n, int32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanCta) attn_plan_kernel(const AttnParams p) {
  __shared__ int64_t sm[32];
  // the first requests' own first token, count, length and place (see AttnParams::prompt): calls of up to
  // kPlanCta requests read them from here
  __shared__ int32_t s_t0[kPlanCta + 1], s_len[kPlanCta], s_prompt[kPlanCta];
  attn_release_next();  // what follows may take its place, and waits for this kernel's end itself
  attn_wait_prior();
  const int tid = threadIdx.x, n = p.n_reqs;
  const bool small = n <= kPlanCta;
  auto req = [&](int b) -> AttnReq {
    if (small) return AttnReq{s_t0[b], s_t0[b + 1] - s_t0[b], s_len[b]};
    int32_t none = 0;
    return attn_request(p, b, &none);
  };
  auto place_of = [&](int b) -> int32_t { return small ? s_prompt[b] : p.prompt[b]; };
  int32_t bad = 0, most = 0;
  // check; how far the longest request reaches; which requests are prompts
  int64_t many = 0, plain = 0;
  for (int b0 = 0; b0 < n; b0 += kPlanCta) {
    const int b = b0 + tid;
    int64_t mine = 0, total;
    AttnReq r = {};
    bool prompt = false;
    if (b < n) {
      r = attn_request(p, b, &bad);
      most = max(most, r.len);
      // (one token, of however many heads, shares the batch's pass over the prefix)
      prompt = p.wide_groups > 0 && r.n > 1 && (int64_t)r.n * p.group > kAttnNarrowRows;
      mine = prompt ? 0 : r.n;
    }
    const int64_t at = plain + block_excl(mine, &total, sm);
    if (b < n) {
      // a request's first place in prefix_tok, as an offset from its first token; prompts: none
      p.prompt[b] = prompt ? INT32_MIN : (int32_t)(at - r.t0);
      if (small) {
        s_t0[b] = r.t0, s_len[b] = r.len, s_prompt[b] = p.prompt[b];
        if (b == n - 1) s_t0[n] = r.t0 + r.n;
      }
      many += prompt;
    }
    plain += total;
  }
  for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(~0u, most, o));
  __syncthreads();
  if ((tid & 31) == 0) sm[tid >> 5] = most;
  const int any_range = __syncthreads_or(bad == KVX_ERR_OUT_OF_RANGE);
  const int any_arg = __syncthreads_or(bad == KVX_ERR_INVALID_ARG);
  const int any_prompt = __syncthreads_or(many > 0);
  for (int i = 0; i < 32; ++i) most = max(most, (int32_t)sm[i]);
  const bool refused = any_range || any_arg;
  const int32_t prefix = min(p.prefix_len, most);  // no further than some request reaches
  if (tid == 0) {
    p.head->refused = any_range ? KVX_ERR_OUT_OF_RANGE : any_arg ? KVX_ERR_INVALID_ARG : KVX_OK;
  }
  // what each token sees, and whose it is
  const int32_t last = refused || n == 0 ? 0 : p.q_start ? p.q_start[n] : n;
  for (int t = tid; t < p.n_q; t += kPlanCta) {
    int b = -1, sees = 0;
    if (t < last) {
      b = p.q_start ? last_at_or_before(small ? s_t0 : p.q_start, n, t) : t;
      const AttnReq r = req(b);
      sees = max(0, r.len - r.n + (t - r.t0) + 1);
      const int32_t at = place_of(b);
      if (at != INT32_MIN) p.prefix_tok[at + t] = t, p.prefix_at[t] = at + t;
    }
    p.owner[t] = b;
    p.limit[t] = sees;
  }
  // the narrow line
  int64_t tiles = 0;
  for (int s0 = 0; s0 <= n; s0 += kPlanCta) {
    const int s = s0 + tid;
    AttnSeg g = {};
    int64_t mine = 0;
    if (s <= n && !refused) {
      if (s == 0) {
        if (p.wide_groups == 0) {
          g.rows = (int32_t)plain * p.group;
          g.key1 = prefix;
        }
      } else if (place_of(s - 1) != INT32_MIN) {
        const AttnReq r = req(s - 1);
        g.row0 = r.t0 * p.group;
        g.rows = r.n * p.group;
        g.low = p.prefix_len;
        g.key1 = r.len;
      }
      attn_tile_seg(p, &g);
      mine = attn_length(p, g);
    }
    int64_t total;
    g.tile0 = tiles + block_excl(mine, &total, sm);
    if (s <= n) p.segs[s] = g;
    tiles += total;
  }
  // the wide line: units first, then their tiles
  int64_t units = 0, wide = 0;
  if (p.wide_groups > 0 && !refused) {
    for (int s0 = 0; s0 <= n; s0 += kPlanCta) {
      const int s = s0 + tid;
      int64_t mine = 0, total;
      if (s == 0) mine = prefix > 0 ? attn_up(plain * p.group, kAttnWideRows) : 0;
      else if (s <= n && any_prompt && place_of(s - 1) == INT32_MIN)
        mine = attn_up((int64_t)req(s - 1).n * p.group, kAttnWideRows);
      const int64_t at = units + block_excl(mine, &total, sm);
      if (s <= n) p.unit_base[s] = (int32_t)at;
      units += total;
      if (!any_prompt) break;
    }
    __syncthreads();
    for (int64_t u0 = 0; u0 < units; u0 += kPlanCta) {
      const int64_t u = u0 + tid;
      AttnUnit x = {};
      int64_t total;
      if (u < units) {
        const int s = any_prompt ? last_at_or_before(p.unit_base, n + 1, (int32_t)u) : 0;
        const int tile = (int)(u - (s ? p.unit_base[s] : 0));
        x.table = s - 1;
        x.row0 = tile * kAttnWideRows;
        if (s == 0) {
          x.rows = (int32_t)min((int64_t)kAttnWideRows, plain * p.group - x.row0);
          x.key1 = prefix;
        } else {
          const AttnReq r = req(s - 1);
          x.rows = min(kAttnWideRows, r.n * p.group - x.row0);
          // as far as its last row sees
          x.key1 = max(0, r.len - r.n + (x.row0 + x.rows - 1) / p.group + 1);
          x.row0 += r.t0 * p.group;
        }
        x.key_tiles = (int32_t)attn_up(x.key1, kAttnWideKeys);
      }
      x.tile0 = wide + block_excl(x.key_tiles, &total, sm);
      if (u < units) p.units[u] = x;
      wide += total;
    }
  }
  const AttnShare share = attn_share(p, tiles, wide);
  const int64_t quota = max((int64_t)1, attn_up(tiles, share.groups));
  const int64_t wide_quota = p.wide_groups > 0 ? max((int64_t)1, attn_up(wide, share.wide_groups)) : 1;
  if (tid == 0) {
    p.head->tiles = tiles;
    p.head->quota = quota;
    p.head->units = (int32_t)units;
    p.head->wide_tiles = wide;
    p.head->wide_quota = wide_quota;
  }
  __syncthreads();
  // tokens of prompts whose rows the wide kernel writes itself, being in one piece
  if (any_prompt && !refused)
    for (int t = tid; t < last; t += kPlanCta) {
      const int b = p.owner[t];
      if (p.prompt[b] != INT32_MIN) continue;
      const int at = (t - req(b).t0) * p.group;  // (there may be no query starts)
      bool whole = true;
      for (int u = at / kAttnWideRows; u <= (at + p.group - 1) / kAttnWideRows; ++u) {
        const AttnUnit x = p.units[p.unit_base[1 + b] + u];
        whole = whole && x.key_tiles > 0 && x.tile0 / wide_quota == (x.tile0 + x.key_tiles - 1) / wide_quota;
      }
      if (whole) p.owner[t] = kAttnWritten;
    }
  for (int g = tid; g < p.groups + p.wide_groups; g += kPlanCta)
    p.start[g] = g < p.groups ? attn_find(p.segs, n + 1, g * quota)
                 : units > 0  ? attn_find(p.units, (int)units, (g - p.groups) * wide_quota) : 0;
}

__device__ __forceinline__ void put(float *o, float x) { *o = x; }
__device__ __forceinline__ void put(__half *o, float x) { *o = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16 *o, float x) { *o = __float2bfloat16_rn(x); }

constexpr int kJoinWarps = 4;

// The pieces of a row.  The first is at the row's own place, piece i, of group g, at more + g * step; g is
// g0 + i, or (cost > 0) where a group's part is shorter than a tile that of the i-th tile.
struct RowPieces {
  int64_t first, more, step, begin;
  int32_t count, g0, cost;
};

__device__ __forceinline__ RowPieces narrow_pieces(const AttnParams &p, const AttnSeg &s, int64_t quota,
                                                   bool prefix, int h, int32_t r) {
  RowPieces x = {};
  if (s.key_tiles == 0) return x;
  const int unit = s.rows <= p.row_tile ? 0 : (r - s.row0) / p.row_tile, row0 = s.row0 + unit * p.row_tile;
  x.begin = s.tile0 + unit * attn_unit_length(p, s);
  x.g0 = (int)attn_div(x.begin, quota);
  if (s.cost <= quota) {
    x.count = (int)attn_div(x.begin + (int64_t)(s.key_tiles - 1) * s.cost, quota) - x.g0 + 1;
  } else {
    x.count = s.key_tiles;
    x.cost = s.cost;
  }
  x.first = attn_part(p, prefix, true, 0, h, row0) + (r - row0);
  x.more = attn_part(p, prefix, false, 0, h, row0) + (r - row0);
  x.step = (int64_t)p.kv_heads * p.row_tile;
  return x;
}

// A block joins the parts of `heads` query heads of one token, a warp a head at a time, prefix splits
// first, in order.  DK: head_dim, 0: any.  Bound: reading the parts (4 D bytes a row and piece), or for few
// rows the chain of a row's pieces.  Cold, 3100 tokens of 32 heads (prompts) 28 us, 64 tokens of 32 heads
// 7 us, one token with 38 pieces a row 18 us.
// W: the warps of a row, each with a stretch of its pieces, whose sums are added up in order; 1 but for few rows of
// 4-bit pools, whose narrow line has many more groups (one token of 304 pieces a row, cold: 15.5 us).
template <typename IO, int DK, int W>
__global__ void __launch_bounds__((W > 1 ? W : kJoinWarps) * 32) attn_join_kernel(const __grid_constant__ AttnParams p, int heads) {
  constexpr int kWarps = W > 1 ? W : kJoinWarps;
  attn_wait_prior();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x;
  const AttnHeader head = *p.head;
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the call's verdict
    int32_t e = head.refused;
    for (int i = threadIdx.x; i < p.n_errors; i += kWarps * 32) e = max(e, p.errors[i]);
    for (int o = 16; o; o >>= 1) e = max(e, __shfl_xor_sync(~0u, e, o));
    __shared__ int32_t worst[kWarps];
    if (lane == 0) worst[warp] = e;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < kWarps; ++i) e = max(e, worst[i]);
      *p.status = e;
      if (p.wide_groups > 0) *p.ready = 0;
    }
  }
  if (t >= p.n_q) return;
  const int b = p.planned ? p.owner[t] : t;
  if (b == kAttnWritten) return;
  const int D = DK ? DK : p.head_dim;
  const bool some = b >= 0 && !head.refused;
  const bool prompt = some && p.planned && p.prompt[b] == INT32_MIN;
  AttnSeg seg[2] = {};
  if (some && p.wide_groups == 0) seg[0] = p.segs[0];
  if (some) seg[1] = p.segs[1 + b];
  const int units = p.planned ? head.units : attn_plain_units(p);
  // of the wide line: the token's unit 0, and its first row's place among those of its kind of work
  int unit0 = 0, lead = 0, wide_row = t * p.group;
  if (some && p.wide_groups > 0 && p.planned) {
    if (prompt) unit0 = p.unit_base[1 + b], lead = p.q_start ? p.q_start[b] * p.group : b * p.group;
    else wide_row = p.prefix_at[t] * p.group;
  }
  const int qh1 = min(p.q_heads, (int)(blockIdx.y + 1) * heads);
  for (int qh = blockIdx.y * heads + (W > 1 ? 0 : warp); qh < qh1; qh += W > 1 ? 1 : kJoinWarps) {
    const int h = qh / p.group, member = qh - h * p.group, r = t * p.group + member;
    // the pieces of the row: those of the prefix (or of the prompt), then the request's own
    RowPieces pre = {}, own = {};
    if (some && p.wide_groups > 0) {
      const int wr = wide_row + member, u = unit0 + (wr - lead) / kAttnWideRows;
      if (u < units) {
        const AttnUnit x = p.planned ? p.units[u] : attn_plain_unit(p, u);
        if (x.key_tiles > 0 && x.table == (prompt ? b : -1)) {
          pre.g0 = (int)attn_div(x.tile0, head.wide_quota);
          pre.count = (int)attn_div(x.tile0 + x.key_tiles - 1, head.wide_quota) - pre.g0 + 1;
          if (prompt && pre.count == 1) continue;  // the wide kernel has written the result
          pre.first = attn_wide_part(p, true, 0, h) + r;
          pre.more = attn_wide_part(p, false, 0, h) + (wr - x.row0);
          pre.step = (int64_t)p.kv_heads * kAttnWideRows;
        }
      }
    } else {
      pre = narrow_pieces(p, seg[0], head.quota, true, h, r);
    }
    own = narrow_pieces(p, seg[1], head.quota, false, h, r);
    const int n0 = pre.count, n = n0 + own.count;
    auto part = [&](int i) {
      const bool k = i >= n0;
      i -= k ? n0 : 0;
      if (i == 0) return k ? own.first : pre.first;
      const int cost = k ? own.cost : pre.cost;
      int g = (k ? own.g0 : pre.g0) + i;
      if (cost) g = (int)attn_div((k ? own.begin : pre.begin) + (int64_t)i * cost, head.quota);
      return (k ? own.more : pre.more) + g * (k ? own.step : pre.step);
    };
    // lane i has part i (of 32 at a time); all lanes then add the parts, neighbouring columns a lane
    float top = -INFINITY, l = 0.f;
    constexpr int kCols = DK ? DK / 32 : KVX_ATTN_MAX_HEAD_DIM / 32;
    float acc[kCols] = {};
    const int per = W > 1 ? (n + W - 1) / W : n, begin = W > 1 ? min(warp * per, n) : 0, end = W > 1 ? min(begin + per, n) : n;
    for (int i0 = begin; i0 < end; i0 += 32) {
      const int left = min(32, end - i0);
      int64_t at = 0;
      float m = -INFINITY, pl = 0.f;
      if (lane < left) {
        at = part(i0 + lane);
        m = p.part_m[at];
        pl = p.part_l[at];
      }
      float now = m;
#pragma unroll
      for (int o = 16; o; o >>= 1) now = fmaxf(now, __shfl_xor_sync(~0u, now, o));
      now = fmaxf(now, top);
      const float base = now == -INFINITY ? 0.f : now;
      if (i0 > begin) {  // more than 32 parts: what the first ones gave refers to the greatest so far
        const float f = top == -INFINITY ? 0.f : exp2f(top - base);
        l *= f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] *= f;
      }
      top = now;
      const float f = exp2f(m - base);
      l = fmaf(f, pl, l);
#pragma unroll 8
      for (int i = 0; i < left; ++i) {
        const float *o = p.part_o + __shfl_sync(~0u, at, i) * D;
        const float w = __shfl_sync(~0u, f, i);
        if constexpr (DK == 128) {
          const float4 v = *reinterpret_cast<const float4 *>(o + lane * 4);
          acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
          acc[2] = fmaf(w, v.z, acc[2]), acc[3] = fmaf(w, v.w, acc[3]);
        } else if constexpr (DK == 64) {
          const float2 v = *reinterpret_cast<const float2 *>(o + lane * 2);
          acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
        } else {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c * 32 + lane < D) acc[c] = fmaf(w, o[c * 32 + lane], acc[c]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    if constexpr (W > 1) {
      __shared__ float s_acc[W][kCols * 32], s_top[W], s_l[W];
      __syncthreads();  // (the head before has been added up)
#pragma unroll
      for (int c = 0; c < kCols; ++c) s_acc[warp][c * 32 + lane] = acc[c];
      if (lane == 0) s_top[warp] = top, s_l[warp] = l;
      __syncthreads();
      if (warp != 0) continue;
      top = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_top[w]);
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = exp2f(s_top[w] - base);
        l = fmaf(f, s_l[w], l);
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = fmaf(f, s_acc[w][c * 32 + lane], acc[c]);
      }
    }
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
    IO *out = reinterpret_cast<IO *>(p.out + t * p.out_tok + qh * p.out_head);
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const int d = DK ? lane * kCols + c : c * 32 + lane;
      if (DK || d < D) put(out + d, l == 0.f ? 0.f : acc[c] * inv);
    }
    if (p.lse && lane == 0)
      p.lse[(int64_t)t * p.q_heads + qh] =
          l == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(l)) * 0.693147180559945309f;
  }
}

constexpr int kDeepWarps = 16;

template <typename IO>
const void *join_kernel(int D, bool deep) {
  if (deep) return D == 64 ? (const void *)attn_join_kernel<IO, 64, kDeepWarps> : (const void *)attn_join_kernel<IO, 128, kDeepWarps>;
  return D == 64    ? (const void *)attn_join_kernel<IO, 64, 1>
         : D == 128 ? (const void *)attn_join_kernel<IO, 128, 1>
                    : (const void *)attn_join_kernel<IO, 0, 1>;
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

}  // namespace

void attn_make_tma(const AttnParams &p, int keys, bool fp8, bool hnd, AttnTma *t, CUtensorMap *km,
                   CUtensorMap *vm) {
  *t = AttnTma{};
  std::memset(km, 0, sizeof(*km));
  std::memset(vm, 0, sizeof(*vm));
  const int64_t pages = p.pool.num_pages, D = p.head_dim;
  const int64_t all = hnd ? pages * p.kv_heads * p.page_size : pages * p.page_size;
  if (p.page_size % 8 != 0 || all > INT32_MAX || !encoder()) return;
  int rows = keys;
  while (p.page_size % rows != 0) rows >>= 1;
  const cuuint64_t pitch = (cuuint64_t)p.pool.tok_stride;
  const cuuint64_t columns = (cuuint64_t)(hnd ? D : D * p.kv_heads);
  const cuuint64_t dims8[2] = {columns, (cuuint64_t)all}, strides8[1] = {pitch};
  const cuuint32_t box8[2] = {(cuuint32_t)D, (cuuint32_t)rows};
  const cuuint64_t dims[4] = {64, 8, columns / 64, (cuuint64_t)(all / 8)}, strides[3] = {pitch, 128, pitch * 8};
  const cuuint32_t box[4] = {64, 8, (cuuint32_t)(D / 64), (cuuint32_t)(rows / 8)}, one[4] = {1, 1, 1, 1};
  for (int kv = 0; kv < 2; ++kv)
    if (encoder()(kv ? vm : km, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                  fp8 ? 2 : 4, const_cast<char *>(kv ? p.pool.v : p.pool.k), fp8 ? dims8 : dims,
                  fp8 ? strides8 : strides, fp8 ? box8 : box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  fp8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return;
  t->rows = rows;
  t->head_x = hnd ? 0 : (int32_t)(fp8 ? D : D / 64);
  t->page_y = hnd ? (int64_t)p.kv_heads * p.page_size : p.page_size;
  t->head_y = hnd ? p.page_size : 0;
}

bool attn_q4_maps(const AttnParams &p, CUtensorMap *km, CUtensorMap *vm) {
  const cuuint64_t S = p.head_bytes, ps = p.page_size, pages = p.pool.num_pages, H = p.kv_heads;
  if (!encoder()) return false;
  cuuint64_t dims[3], strides[2];
  cuuint32_t box[3];
  const cuuint32_t one[3] = {1, 1, 1};
  if (p.q4_runs) {
    dims[0] = ps * S / 8, dims[1] = pages * H, dims[2] = 1;
    strides[0] = ps * S, strides[1] = ps * S * pages * H;
    box[0] = (cuuint32_t)(16 * S / 8), box[1] = p.chunk, box[2] = 1;
  } else {
    dims[0] = (S << p.q4_pair) / 8, dims[1] = pages * ps, dims[2] = H >> p.q4_pair;
    strides[0] = p.pool.tok_stride, strides[1] = S << p.q4_pair;
    box[0] = (cuuint32_t)dims[0], box[1] = 16, box[2] = p.chunk >> p.q4_pair;
  }
  for (int kv = 0; kv < 2; ++kv)
    if (encoder()(kv ? vm : km, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<char *>(kv ? p.pool.v : p.pool.k), dims, strides,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

namespace {

// Calls with one query token a request do without the plan kernel up to this many requests.
constexpr int kPlanReqs = 2048;

// Operations from which the wide kernel takes the prefix and prompts (about 1200 TFLOP/s behind some 12
// us) instead of the narrow one, 64 rows at a time (about 290 TFLOP/s, no launch of its own): kWideWork; but
// already kWideBeside where the requests' own rows may come to kWideBytes, so that the two kernels can run
// side by side (see attn_share).  64 requests of 1000-2000 tokens behind 2048 shared ones (2.1e9): 102
// us with the narrow kernel alone, 93 us side by side.
constexpr double kWideWork = 4.5e9, kWideBeside = 0.7e9, kWideBytes = 2e8;

// The same of 4-bit pools, whose wide kernel takes some 20 us to begin and whose other one reads short tiles at about 100
// TFLOP/s.  64 requests of 1000-2000 tokens behind 2048 shared ones (2.1e9): 57 us without the wide kernel (then; 61 now), 64
// to 78 with it; 100-1000 tokens behind 4096 (4.3e9): 55 and 42.
constexpr double kQ4WideWork = 2.5e9;

// A narrow unit's begin and end take about as long as some tiles of 16 rows.  Counted as 0, 2, 3 and 4 of
// them: 95 requests of up to 25 own tokens behind 1360 shared ones 121, 66, 57 and 53 us; 96 FP8 decode
// requests 60, 52, 59 and 60 us; 256 decode requests of 4096 own tokens 350, 344, 342 and 366 us.  The plain
// kernel's tiles take so long that they do not tell.
constexpr int32_t kNarrowUnitCost = 2;

// The same of 4-bit pools where a CTA has one head; the more places for heads it has, the longer its tiles take.  Counted as 2, 8,
// 12, 16 and 24: 95 requests of 4-81 own tokens of 1 x 4 heads of 64 behind 6859 shared ones 58, 37, 33, 32 and 29 us; 91 of
// 1-1208 of 2 x 8 heads behind 16944 65, and 56 from 8 on; 125 of 31-358 of 1 x 6 heads 18.8, 18.2, 18.6, 20.5 and 21.1.
constexpr int32_t kQ4UnitCost = 12;

struct Sizes {
  int64_t ready_off, segs_off, units_off, start_off, base_off, prompt_off, limit_off, owner_off, tok_off, at_off;
  int64_t m_off, l_off, o_off, errors_off, errors, total;
  int32_t groups, wide_groups;
};

// Whether the tensor-core kernels take a layout.
bool tensor_cores(const kvx_layout *l) {
  if (l->dtype == KVX_Q4)  // copies of a fifth of a head vector, head vectors counted in 32 bits
    return (l->head_dim == 64 || l->head_dim == 128) && l->vec >= l->head_dim / 8 && l->slot_stride <= INT32_MAX &&
           (l->kind == KVX_NHD || l->num_slots * l->kv_heads < (int64_t)1 << 32);
  return l->elem <= 2 && (l->head_dim == 64 || l->head_dim == 128) && l->vec == 16;
}

bool q4_kernel(const kvx_layout *l) { return l->dtype == KVX_Q4 && tensor_cores(l); }

// kv heads of a CTA: 1, but up to `most` (of eight) in the 4-bit kernel, as evenly as it goes, and pairs where a head
// vector is no whole number of 16-byte pieces.
int chunk_of(const kvx_layout *l, int most) {
  if (!q4_kernel(l)) return 1;
  const int chunks = (l->kv_heads + most - 1) / most, c = (l->kv_heads + chunks - 1) / chunks;
  return l->head_dim == 64 && c % 2 != 0 && l->kv_heads > 1 ? c + 1 : c;
}
int slot_shift_of(int chunk) {
  int s = 0;
  while (1 << s < chunk) ++s;
  return s;
}
int row_tile_of(const kvx_layout *l, int chunk) {
  if (q4_kernel(l)) return 8 * (kAttnQ4Warps >> slot_shift_of(chunk));
  return tensor_cores(l) ? kAttnNarrowRows : kAttnGeneralRows;
}
int group_ctas_of(const kvx_layout *l, int chunk) { return (l->kv_heads + chunk - 1) / chunk; }

// How many heads of a CTA suit calls of n_q tokens of n_reqs requests: eight warps have eight rows each, and a unit of
// more rows than they have for its heads reads the keys again.
int q4_most_heads(int64_t n_q, int64_t n_reqs, int64_t group) {
  int most = kAttnQ4Warps;
  while (most > 1 && n_q * group > 8 * (kAttnQ4Warps / most) * n_reqs) most /= 2;
  return most;
}

// How many groups of CTAs: as many as are resident at once.
Sizes sizes(const kvx_layout *l, int64_t n_q, int64_t n_reqs, int64_t q_heads, bool wide, int chunk) {
  Sizes z = {};
  const int64_t kv_heads = l->kv_heads, D = l->head_dim, row_tile = row_tile_of(l, chunk);
  const int64_t rows = n_q * (q_heads / kv_heads);
  const int64_t per_sm = !tensor_cores(l) && D <= 128 ? 3 : 2;
  z.groups = (int32_t)std::max((int64_t)1, kAttnSms * per_sm / group_ctas_of(l, chunk));
  z.wide_groups = wide ? (int32_t)std::max((int64_t)1, kAttnSms / kv_heads) : 0;
  z.errors = z.groups * kv_heads + z.wide_groups * kv_heads;
  const int64_t parts = 2 * n_q * q_heads + z.groups * kv_heads * row_tile +
                        z.wide_groups * kv_heads * kAttnWideRows;
  // prompts have more than kAttnNarrowRows rows each
  const int64_t units = wide ? 2 * (rows / kAttnWideRows) + rows / kAttnNarrowRows + 2 : 0;
  int64_t at = sizeof(AttnHeader);
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = align_up(at + bytes, 256);
    return here;
  };
  z.ready_off = take(8);
  z.segs_off = take((int64_t)sizeof(AttnSeg) * (n_reqs + 1));
  z.units_off = take((int64_t)sizeof(AttnUnit) * units);
  z.start_off = take(4 * (z.groups + z.wide_groups));
  z.base_off = take(4 * (n_reqs + 2));
  z.prompt_off = take(4 * n_reqs);
  z.limit_off = take(4 * n_q);
  z.owner_off = take(4 * n_q);
  z.tok_off = take(4 * n_q);
  z.at_off = take(4 * n_q);
  z.errors_off = take(4 * z.errors);
  z.m_off = take(4 * parts);
  z.l_off = take(4 * parts);
  z.o_off = take(4 * parts * D);
  z.total = at;
  return z;
}

bool shape_ok(const kvx_layout *l, int64_t n_q, int64_t n_reqs, int64_t q_heads, int64_t prefix) {
  return l && l->kv_planes == 2 && l->head_dim <= KVX_ATTN_MAX_HEAD_DIM && n_q >= 0 &&
         n_reqs >= 0 && n_reqs <= KVX_MAX_TABLE_REQUESTS && q_heads >= 1 &&
         q_heads % l->kv_heads == 0 && prefix >= 0 && prefix <= KVX_ATTN_MAX_POSITIONS &&
         n_q * q_heads <= (int64_t)1 << 30;
}

// Whether a call may have work for the wide kernel: more rows than the narrow kernel has in a unit (and than 4-bit pools' may
// have, whose units are of 8 to 64 rows).
bool takes_wide(const kvx_layout *l, int64_t n_q, int64_t q_heads) {
  return tensor_cores(l) && n_q * (q_heads / l->kv_heads) > kAttnNarrowRows;
}

// A number that no word of a workspace holds by chance: calls are counted from the process's first one's
// time, and mixed (splitmix64; every step can be undone, so no two counts give the same).
uint64_t next_call() {
  static std::atomic<uint64_t> calls{(uint64_t)std::chrono::system_clock::now().time_since_epoch().count() << 20};
  uint64_t x = calls.fetch_add(1, std::memory_order_relaxed) * 0x9e3779b97f4a7c15u;
  x = (x ^ (x >> 30)) * 0xbf58476d1ce4e5b9u;
  x = (x ^ (x >> 27)) * 0x94d049bb133111ebu;
  return x ^ (x >> 31);
}

bool mult(const void *p, uintptr_t a) { return (uintptr_t)p % a == 0; }

static_assert(sizeof(kvx_attn_args) == 152, "the binding mirrors this structure");

}  // namespace
}  // namespace kvx

extern "C" size_t kvx_attention_workspace_size(kvx_layout_t pool, int32_t n_q, int32_t n_reqs,
                                               int32_t q_heads, int32_t prefix_len) {
  if (!kvx::shape_ok(pool, n_q, n_reqs, q_heads, prefix_len)) return 0;
  // (whatever number of heads a CTA has: fewer tokens or requests may take another)
  int64_t most = 0;
  for (int heads = kvx::kAttnQ4Warps; heads >= 1; heads /= 2)
    most = std::max(most, kvx::sizes(pool, n_q, n_reqs, q_heads, kvx::takes_wide(pool, n_q, q_heads), kvx::chunk_of(pool, heads)).total);
  return (size_t)most;
}

extern "C" kvx_status kvx_shared_attention(kvx_layout_t pool, const kvx_attn_args *args,
                                           void *d_ws, size_t ws_bytes, int32_t *d_status,
                                           kvx_stream_t stream) {
  using namespace kvx;
  if (!pool || !args || !d_status) return KVX_ERR_INVALID_ARG;
  const kvx_attn_args &a = *args;
  if (a.reserved != 0 || a.reserved2 != 0 || !shape_ok(pool, a.n_q, a.n_reqs, a.q_heads, a.prefix_len) ||
      a.layer < 0 || a.layer >= pool->num_layers || a.page_size < 1 || a.max_pages < 1 ||
      a.table_stride < a.max_pages || a.n_prefix_pages < 0 || a.page_size > pool->num_slots)
    return KVX_ERR_INVALID_ARG;
  if (pool->dtype == KVX_FP8 || pool->dtype == KVX_Q4 ? (a.q_dtype != KVX_F16 && a.q_dtype != KVX_BF16)
                             : a.q_dtype != pool->dtype)
    return KVX_ERR_INVALID_ARG;
  if (pool->kind == KVX_HND_PAGED && pool->page_size != a.page_size) return KVX_ERR_INVALID_ARG;
  if ((int64_t)a.n_prefix_pages * a.page_size < a.prefix_len ||
      (a.prefix_len > 0 && !a.prefix_pages))
    return KVX_ERR_INVALID_ARG;
  if (!a.q_start && a.n_q != a.n_reqs) return KVX_ERR_INVALID_ARG;
  if (a.n_reqs > 0 && (!a.tables || !a.seq_lens)) return KVX_ERR_INVALID_ARG;
  if (a.n_q > 0 && (!a.q || !a.out)) return KVX_ERR_INVALID_ARG;
  if (!std::isfinite(a.scale) || !std::isfinite(a.k_scale) || !std::isfinite(a.v_scale))
    return KVX_ERR_INVALID_ARG;
  const int64_t io = a.q_dtype == KVX_F32 ? 4 : 2, most = ((int64_t)1 << 40);
  for (int64_t x : {a.q_token_stride, a.q_head_stride, a.out_token_stride, a.out_head_stride,
                    a.table_stride})
    if (x < 0 || x > most) return KVX_ERR_INVALID_ARG;
  // the last element's byte, past any memory: offsets within q and out are 64-bit numbers
  auto reach = [&](int64_t token, int64_t head) {
    return ((double)token * std::max(0, a.n_q - 1) + (double)head * (a.q_heads - 1) + pool->head_dim) * io;
  };
  if (reach(a.q_token_stride, a.q_head_stride) > 0x1p60 || reach(a.out_token_stride, a.out_head_stride) > 0x1p60)
    return KVX_ERR_INVALID_ARG;
  if (!mult(a.q, io) || !mult(a.out, io)) return KVX_ERR_ALIGNMENT;
  for (const void *q : {(const void *)a.tables, (const void *)a.prefix_pages,
                        (const void *)a.seq_lens, (const void *)a.q_start, (const void *)a.lse,
                        (const void *)d_status})
    if (!mult(q, 4)) return KVX_ERR_ALIGNMENT;
  if (a.n_q > 0) {
    const uintptr_t b0 = (uintptr_t)a.out;
    const uintptr_t b1 = b0 + ((a.n_q - 1) * a.out_token_stride + (a.q_heads - 1) * a.out_head_stride +
                               pool->head_dim) * io;
    if (layout_overlaps_range(pool, b0, b1)) return KVX_ERR_OVERLAP;
  }
  // What the wide kernel may have: the prefix, and with several tokens a request prompts, whose keys
  // only the tables bound.  Below kWideWork operations its launch costs more than it saves.  It takes
  // the greatest score from the greatest product, so the factor between them has to be above 0.
  const double room = (double)a.max_pages * a.page_size;
  const bool q4 = q4_kernel(pool);
  const bool beside = (room - a.prefix_len) * a.n_reqs * pool->row_bytes * 2 >= kWideBytes;
  const double wide_keys = a.q_start ? (double)a.max_pages * a.page_size : (double)a.prefix_len;
  const bool wide = takes_wide(pool, a.n_q, a.q_heads) &&
                    4.0 * pool->head_dim * a.q_heads * a.n_q * wide_keys >= (q4 ? kQ4WideWork : beside ? kWideBeside : kWideWork) &&
                    a.scale * a.k_scale > 0.f;
  const int chunk = chunk_of(pool, q4_most_heads(a.n_q, a.n_reqs, a.q_heads / pool->kv_heads));
  const Sizes z = sizes(pool, a.n_q, a.n_reqs, a.q_heads, wide, chunk);
  if (!d_ws || !mult(d_ws, 256) || (int64_t)ws_bytes < z.total) return KVX_ERR_NO_WORKSPACE;

  AttnParams p;
  std::memset(&p, 0, sizeof(p));
  const int64_t seg = pool->seg_bytes;
  p.pool.k = reinterpret_cast<const char *>(pool->plane[2 * a.layer]);
  p.pool.v = reinterpret_cast<const char *>(pool->plane[2 * a.layer + 1]);
  const bool hnd = pool->kind == KVX_HND_PAGED;
  p.pool.page_stride = hnd ? pool->page_bytes : pool->slot_stride * a.page_size;
  p.pool.tok_stride = hnd ? seg : pool->slot_stride;
  p.pool.head_stride = hnd ? seg * a.page_size : seg;
  p.pool.num_pages = pool->num_slots / a.page_size;
  p.pool.page_size = a.page_size;
  p.pool.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == (1 << i)) p.pool.page_shift = i;
  p.tables = a.tables;
  p.table_stride = a.table_stride;
  p.prefix_pages = a.prefix_pages;
  p.seq_lens = a.seq_lens;
  p.q_start = a.q_start;
  p.q = static_cast<const char *>(a.q);
  p.out = static_cast<char *>(a.out);
  p.q_tok = a.q_token_stride * io;
  p.q_head = a.q_head_stride * io;
  p.out_tok = a.out_token_stride * io;
  p.out_head = a.out_head_stride * io;
  p.lse = a.lse;
  p.scale_log2 = (float)((double)a.scale * a.k_scale * 1.4426950408889634);
  p.v_scale = a.v_scale;
  p.n_q = a.n_q;
  p.n_reqs = a.n_reqs;
  p.q_heads = a.q_heads;
  p.kv_heads = pool->kv_heads;
  p.group = a.q_heads / pool->kv_heads;
  p.head_dim = pool->head_dim;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.prefix_len = a.prefix_len;
  p.row_tile = row_tile_of(pool, chunk);
  p.few_rows = q4 ? 8 : 16;
  p.key_shift = q4 ? 5 : 6;
  static_assert(1 << 5 == kAttnQ4KeyTile && 1 << 6 == kAttnKeyTile, "tiles of these kernels");
  p.group_ctas = group_ctas_of(pool, chunk);
  p.chunk = chunk;
  p.tile_ns = (int32_t)(q4 ? kAttnQ4TileNs << slot_shift_of(chunk) : std::max(kAttnNarrowNs, (pool->seg_bytes << p.key_shift) * 2 / 16 * kAttnNarrowPs / 1000));
  p.wide_ns = (int32_t)(q4 ? kAttnQ4WideNs : kAttnWideNs);
  p.wide_start_ns = (int32_t)(q4 ? kAttnQ4WideStartNs : kAttnStartNs);
  p.head_bytes = (int32_t)pool->seg_bytes;
  CUtensorMap k_map = {}, v_map = {};  // of the 4-bit kernel's boxes
  if (q4) {
    p.slot_shift = slot_shift_of(chunk);
    p.page_vectors = (uint32_t)(hnd ? (int64_t)a.page_size * pool->kv_heads : a.page_size);
    const int32_t keys = 16 * (kAttnQ4Warps >> p.slot_shift), S = (int32_t)seg;  // of a stage; of a head vector
    const bool even = ((uintptr_t)p.pool.k | (uintptr_t)p.pool.v) % 16 == 0 && a.page_size % 16 == 0;
    p.q4_runs = hnd || (pool->kv_heads == 1 && pool->slot_stride == S);
    p.q4_pair = !p.q4_runs && S % 16 != 0;  // (40 bytes are no whole pieces of 16, two heads' are)
    const bool boxes = even && (p.q4_runs ? p.pool.num_pages * pool->kv_heads <= INT32_MAX && (int64_t)a.page_size * S / 8 <= INT32_MAX
                                          : pool->slot_stride % 16 == 0 && (!p.q4_pair || (pool->kv_heads | p.chunk) % 2 == 0)) &&
                       attn_q4_maps(p, &k_map, &v_map);  // (a driver that makes none: the other copies do without)
    const bool tokens = !hnd && pool->vec == 16 && p.chunk * S % 16 == 0;
    p.q4_copies = boxes ? kAttnQ4Boxes : tokens ? kAttnQ4Tokens : kAttnQ4Parts;
    if (boxes) {
      p.q4_key_pitch = S << p.q4_pair, p.q4_head_pitch = 16 * S << p.q4_pair;
      p.q4_block_pitch = 16 * S * p.chunk, p.q4_v_off = 16 * S * kAttnQ4Warps;
    } else if (tokens) {
      // an odd number of 16-byte pieces a token: eight tokens' lie in different banks
      const bool together = p.group_ctas == 1 && p.pool.v - p.pool.k == pool->row_bytes;
      p.q4_pair = 0;
      p.q4_head_pitch = S;
      p.q4_key_pitch = (p.chunk * S * (together ? 2 : 1)) | 16;
      p.q4_v_off = together ? p.chunk * S : keys * p.q4_key_pitch;
      p.q4_block_pitch = 16 * p.q4_key_pitch;
    } else {
      p.q4_pair = 0;
      p.q4_key_pitch = S, p.q4_head_pitch = S * keys, p.q4_block_pitch = 16 * S, p.q4_v_off = 128 * S;
    }
  }
  p.unit_cost = q4 ? std::max(kNarrowUnitCost, kQ4UnitCost >> p.slot_shift) : tensor_cores(pool) ? kNarrowUnitCost : 0;
  const uintptr_t q_at = (uintptr_t)a.q | (uintptr_t)p.q_tok | (uintptr_t)p.q_head;
  p.q_even = q_at % 4 == 0;
  p.q_vec = q_at % 16 == 0;
  p.out_vec = ((uintptr_t)a.out | (uintptr_t)p.out_tok | (uintptr_t)p.out_head) % 16 == 0;
  p.groups = z.groups;
  p.wide_groups = z.wide_groups;
  // a single token a request, and not so many requests that every CTA's adding them up tells
  p.planned = a.n_q == 0 || a.q_start || a.n_reqs > kPlanReqs;
  p.after_wide = wide;
  char *ws = static_cast<char *>(d_ws);
  p.head = reinterpret_cast<AttnHeader *>(ws);
  p.ready = reinterpret_cast<uint64_t *>(ws + z.ready_off);
  p.call = wide ? next_call() : 0;
  p.segs = reinterpret_cast<AttnSeg *>(ws + z.segs_off);
  p.units = reinterpret_cast<AttnUnit *>(ws + z.units_off);
  p.start = reinterpret_cast<int32_t *>(ws + z.start_off);
  p.unit_base = reinterpret_cast<int32_t *>(ws + z.base_off);
  p.prompt = reinterpret_cast<int32_t *>(ws + z.prompt_off);
  p.prefix_tok = reinterpret_cast<int32_t *>(ws + z.tok_off);
  p.prefix_at = reinterpret_cast<int32_t *>(ws + z.at_off);
  p.limit = reinterpret_cast<int32_t *>(ws + z.limit_off);
  p.owner = reinterpret_cast<int32_t *>(ws + z.owner_off);
  p.part_m = reinterpret_cast<float *>(ws + z.m_off);
  p.part_l = reinterpret_cast<float *>(ws + z.l_off);
  p.part_o = reinterpret_cast<float *>(ws + z.o_off);
  p.errors = reinterpret_cast<int32_t *>(ws + z.errors_off);
  p.n_errors = a.n_q > 0 ? (int32_t)z.errors : 0;
  p.status = d_status;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void *kargs[] = {&p};
  // The wide kernel goes first: the narrow one does not wait for it, and takes over its SMs one by
  // one as its CTAs end.
  cudaError_t e = cudaSuccess;
  if (p.planned) e = launch_pdl((const void *)attn_plan_kernel, dim3(1), dim3(kPlanCta), kargs, s);
  if (a.n_q > 0) {
    if (e == cudaSuccess && wide) e = launch_attn_wide(p, pool->dtype, a.q_dtype, hnd, s);
    if (e == cudaSuccess)
      e = q4                   ? launch_attn_q4(p, k_map, v_map, a.q_dtype, s)
          : tensor_cores(pool) ? launch_attn_narrow(p, pool->dtype, a.q_dtype, hnd, s)
                             : launch_attn_general(p, pool->dtype, a.q_dtype, pool->vec == 16 && pool->seg_bytes % 16 == 0, s);
  }
  if (e == cudaSuccess) {
    // all warps that an SM has for a row, while there is a row or two an SM
    const bool deep = q4 && a.n_q > 0 && (int64_t)a.n_q * a.q_heads <= 2 * kAttnSms;
    const void *join = a.q_dtype == KVX_F32   ? join_kernel<float>(pool->head_dim, false)
                       : a.q_dtype == KVX_F16 ? join_kernel<__half>(pool->head_dim, deep)
                                              : join_kernel<__nv_bfloat16>(pool->head_dim, deep);
    // a warp a row while that fills the GPU; then a block a token, which reads what is the token's once
    int heads = kJoinWarps;
    if ((int64_t)a.n_q * a.q_heads > (int64_t)kJoinWarps * kAttnSms * 16 || a.q_heads > kJoinWarps * 65535)
      heads = a.q_heads;
    if (deep) heads = 1;
    void *jargs[] = {&p, &heads};
    e = launch_pdl(join, dim3((unsigned)std::max(1, a.n_q), (unsigned)((a.q_heads + heads - 1) / heads)),
                   dim3((deep ? kDeepWarps : kJoinWarps) * 32), jargs, s);
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return KVX_ERR_CUDA;
  }
  return KVX_OK;
}
