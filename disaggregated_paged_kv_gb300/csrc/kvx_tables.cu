// kvx_tables.cu -- block tables and slot maps of a batch, from its lengths.
//
// Two exclusive sums over the requests (new tokens, pages taken) say where everything goes; the
// rest is writing.  The whole batch is checked before anything is written:
//   tables_plan   a few CTAs, each of which adds up all lengths (4-8 bytes a request) and checks
//                 its share of the page ids that the call is going to use; the first one leaves
//                 the sums in the workspace, every one its verdict.
//   tables_fill   a grid over the new tokens, in chunks of 4096: slots, positions and the table
//                 entry of every page that begins among them, then the shared prefix entries.
// Up to kTabThreads requests with room for no more than kOneTokens tokens (decode steps, drafts,
// short prompts) are one CTA's work in one launch, tables_one.
// Bound: the writes (8 bytes a token, 4 a page) for prompts, launch latency for a decode step.  Kernel
// times with cold caches: one request 5.4 us, 256 requests 8.2 us (a call 21 us; in two launches it took
// 36), 1024 prompts of 100-8000 tokens 7 and 25 us for 35 MB, the call itself 24 us.
#include <cstring>

#include "kvx_internal.cuh"
#include "kvx_launch.cuh"
#include "kvx_layout.cuh"

namespace kvx {
namespace {

constexpr int kTabThreads = 1024;
constexpr int kTabMaxCtas = 32;
constexpr int kFillThreads = 256;
constexpr int kFillChunk = 16 * kFillThreads;  // tokens a CTA writes at a time

constexpr int kOneTokens = 8192;

struct TabParams {
  kvx_tables_args a;
  int64_t num_pages;
  int32_t page_shift;  // log2(page_size), or -1
  int32_t ctas;        // of tables_plan
  int64_t prefix_tokens;
  // workspace
  int32_t *verdict;    // [kTabMaxCtas]
  int64_t *totals;     // tokens, pages
  int32_t *tok_base;   // [n_reqs + 1]
  int32_t *page_base;  // [n_reqs + 1]
  int32_t *status;
};

struct TabLayout {
  int64_t totals_off, tok_off, page_off, total;
};

constexpr TabLayout tab_layout(int64_t n) {
  TabLayout L{};
  L.totals_off = 4 * kTabMaxCtas;
  L.tok_off = 256;
  L.page_off = align_up(L.tok_off + 4 * (n + 1), 256);
  L.total = align_up(L.page_off + 4 * (n + 1), 256);
  return L;
}

__device__ __forceinline__ int64_t div_page(const TabParams &p, int64_t x) {
  return p.page_shift >= 0 ? x >> p.page_shift : x / p.a.page_size;
}

struct Span {
  int64_t start, end;  // positions that are new
  int64_t have, need;  // pages before and after
};

__device__ __forceinline__ Span span_of(const TabParams &p, int b, int32_t *bad) {
  const int32_t oldn = p.a.old_lens ? p.a.old_lens[b] : 0, newn = p.a.new_lens[b];
  Span s;
  s.start = oldn;
  if (oldn == 0 && newn > 0) s.start = p.prefix_tokens;
  s.end = newn;
  if (oldn < 0 || newn < s.start) {
    *bad = max(*bad, (int32_t)KVX_ERR_INVALID_ARG);
    s.start = s.end = 0;
  }
  const int64_t up = p.a.page_size - 1;
  s.have = div_page(p, s.start + up);
  s.need = div_page(p, s.end + up);
  return s;
}

// Exclusive block-wide sums of two 64-bit values; *ta, *tb get the totals.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t *ta, int64_t *tb,
                                            int64_t (*sm)[2]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t x = a, y = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, x, d), v = __shfl_up_sync(~0u, y, d);
    if (lane >= d) x += u, y += v;
  }
  if (lane == 31) sm[w][0] = x, sm[w][1] = y;
  __syncthreads();
  if (w == 0) {
    int64_t p = lane < nw ? sm[lane][0] : 0, q = lane < nw ? sm[lane][1] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(~0u, p, d), v = __shfl_up_sync(~0u, q, d);
      if (lane >= d) p += u, q += v;
    }
    sm[lane][0] = p, sm[lane][1] = q;
  }
  __syncthreads();
  const int64_t oa = w ? sm[w - 1][0] : 0, ob = w ? sm[w - 1][1] : 0;
  *ta = sm[nw - 1][0], *tb = sm[nw - 1][1];
  a = oa + x - a;
  b = ob + y - b;
  __syncthreads();
}

__device__ __forceinline__ bool page_ok(const TabParams &p, int32_t id) {
  return id >= 0 && id < p.num_pages;
}

// span_of, with the row's room checked and (page: read the table) the page that is filled further.
__device__ __forceinline__ Span checked_span(const TabParams &p, int b, bool page, int32_t *bad) {
  const Span s = span_of(p, b, bad);
  if (max(s.need, s.have) > p.a.max_pages) {
    *bad = max(*bad, (int32_t)KVX_ERR_OUT_OF_RANGE);
  } else if (page && s.end > s.start && p.a.old_lens && p.a.old_lens[b] > 0 &&
             s.start < s.have * p.a.page_size &&
             !page_ok(p, p.a.tables[b * p.a.table_stride + s.have - 1])) {
    *bad = max(*bad, (int32_t)KVX_ERR_OUT_OF_RANGE);
  }
  return s;
}

// Whether request b is new and has tokens: its row begins with the shared prefix.
__device__ __forceinline__ bool takes_prefix(const TabParams &p, int b) {
  return !(p.a.old_lens && p.a.old_lens[b] != 0) && p.a.new_lens[b] != 0;
}

// Cursor, totals, and every page id that the call is going to use (prefix: those of the shared prefix as
// well), by thread at of step.
__device__ __forceinline__ void check_ids(const TabParams &p, int64_t cur, int64_t tokens,
                                          int64_t pages, bool prefix, int64_t at, int64_t step,
                                          int32_t *bad) {
  if (cur < 0) {
    *bad = max(*bad, (int32_t)KVX_ERR_INVALID_ARG);
  } else if (cur + pages > p.a.n_free || tokens > p.a.max_tokens) {
    *bad = max(*bad, (int32_t)KVX_ERR_OUT_OF_RANGE);
  } else {
    for (int64_t i = at; i < pages; i += step)
      if (!page_ok(p, p.a.free_pages[cur + i])) *bad = max(*bad, (int32_t)KVX_ERR_OUT_OF_RANGE);
    for (int64_t i = at; prefix && i < p.a.n_prefix_pages; i += step)
      if (!page_ok(p, p.a.prefix_pages[i])) *bad = max(*bad, (int32_t)KVX_ERR_OUT_OF_RANGE);
  }
}

__global__ void __launch_bounds__(kTabThreads) tables_plan_kernel(const TabParams p) {
  __shared__ int64_t sm[32][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = p.a.n_reqs, tid = threadIdx.x;
  int32_t bad = 0;
  int64_t tokens = 0, pages = 0;
  bool prefix = false;
  for (int b0 = 0; b0 < n; b0 += kTabThreads) {
    const int b = b0 + tid;
    int64_t cnt = 0, take = 0;
    if (b < n) {
      prefix = prefix || takes_prefix(p, b);
      const Span s = checked_span(p, b, blockIdx.x == 0, &bad);
      cnt = s.end - s.start;
      take = s.need - s.have;
    }
    int64_t tc, tp;
    block_scan2(cnt, take, &tc, &tp, sm);
    if (blockIdx.x == 0 && b < n) {
      // sums past 31 bits are refused below: what is cut off here is never used
      p.tok_base[b] = (int32_t)(tokens + cnt);
      p.page_base[b] = (int32_t)(pages + take);
    }
    tokens += tc;
    pages += tp;
  }
  const int64_t cur = p.a.cursor ? p.a.cursor[0] : 0;
  check_ids(p, cur, tokens, pages, __syncthreads_or(prefix), (int64_t)blockIdx.x * kTabThreads + tid,
            (int64_t)p.ctas * kTabThreads, &bad);
  const int any_range = __syncthreads_or(bad == KVX_ERR_OUT_OF_RANGE);
  const int any_arg = __syncthreads_or(bad == KVX_ERR_INVALID_ARG);
  if (tid == 0) {
    p.verdict[blockIdx.x] = any_range ? KVX_ERR_OUT_OF_RANGE : any_arg ? KVX_ERR_INVALID_ARG : 0;
    if (blockIdx.x == 0) {
      p.totals[0] = tokens;
      p.totals[1] = cur + pages;
      p.tok_base[n] = (int32_t)tokens;
      p.page_base[n] = (int32_t)pages;
    }
  }
}

// The last b in [lo, hi] with base[b] <= i.
__device__ __forceinline__ int find_request(const int32_t *base, int lo, int hi, int32_t i) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Slots, positions and new table entries of all tokens, and the shared prefix entries, by CTA cta
// of ctas with Threads threads.  cur: the cursor before the call.
template <int Threads>
__device__ __forceinline__ void fill(const TabParams &p, const int32_t *tok_base,
                                     const int32_t *page_base, int32_t tokens, int64_t cur, int cta,
                                     int ctas) {
  constexpr int kChunk = 16 * Threads;  // tokens at a time: 4 x 4 consecutive a thread
  const int n = p.a.n_reqs, tid = threadIdx.x;
  int32_t none = 0;
  for (int64_t c0 = (int64_t)cta * kChunk; c0 < tokens; c0 += (int64_t)ctas * kChunk) {
    const int32_t last = (int32_t)min(c0 + kChunk, (int64_t)tokens) - 1;
    const int lo = find_request(tok_base, 0, n - 1, (int32_t)c0);
    const int hi = find_request(tok_base, lo, n - 1, last);
#pragma unroll
    for (int g = 0; g < kChunk / (4 * Threads); ++g) {
      const int32_t i0 = (int32_t)c0 + (g * Threads + tid) * 4;
      if (i0 > last) break;
      int b = find_request(tok_base, lo, hi, i0);
      Span s = span_of(p, b, &none);
      int32_t q0 = tok_base[b], q1 = tok_base[b + 1];
      int64_t page = -1;
      int32_t id = 0, slot[4], at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int32_t i = i0 + k;
        if (i > last) break;
        while (i >= q1) {  // the next request that has new tokens
          ++b;
          q0 = q1, q1 = tok_base[b + 1];
          if (i < q1) s = span_of(p, b, &none);
          page = -1;
        }
        const int64_t pos = s.start + (i - q0);
        const int64_t pg = div_page(p, pos);
        const int32_t off = (int32_t)(pos - pg * p.a.page_size);
        if (pg != page) {
          page = pg;
          id = pg < s.have ? p.a.tables[b * p.a.table_stride + pg]
                           : p.a.free_pages[cur + page_base[b] + (pg - s.have)];
        }
        if (off == 0) p.a.tables[b * p.a.table_stride + pg] = id;
        slot[k] = (int32_t)((int64_t)id * p.a.page_size + off);
        at[k] = (int32_t)pos;
      }
      const bool wide = i0 + 3 <= last;
      if (wide && ((uintptr_t)p.a.slots & 15) == 0)
        *reinterpret_cast<int4 *>(p.a.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      else
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i0 + k <= last) p.a.slots[i0 + k] = slot[k];
      if (p.a.positions) {
        if (wide && ((uintptr_t)p.a.positions & 15) == 0)
          *reinterpret_cast<int4 *>(p.a.positions + i0) = make_int4(at[0], at[1], at[2], at[3]);
        else
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (i0 + k <= last) p.a.positions[i0 + k] = at[k];
      }
    }
  }
  // the shared prefix at the head of every new request's row, a CTA per row
  if (p.a.n_prefix_pages > 0)
    for (int b = cta; b < n; b += ctas) {
      if (!takes_prefix(p, b)) continue;
      for (int j = tid; j < p.a.n_prefix_pages; j += Threads)
        p.a.tables[b * p.a.table_stride + j] = p.a.prefix_pages[j];
    }
}

__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const TabParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = p.a.n_reqs, tid = threadIdx.x;
  const int32_t bad = tid < p.ctas ? p.verdict[tid] : 0;
  const int any_range = __syncthreads_or(bad == KVX_ERR_OUT_OF_RANGE);
  const int any_arg = __syncthreads_or(bad == KVX_ERR_INVALID_ARG);
  if (blockIdx.x == 0 && tid == 0)
    *p.status = any_range ? KVX_ERR_OUT_OF_RANGE : any_arg ? KVX_ERR_INVALID_ARG : KVX_OK;
  if (any_range || any_arg) return;
  const int64_t next = p.totals[1];
  const int64_t gtid = (int64_t)blockIdx.x * kFillThreads + tid, gstep = (int64_t)gridDim.x * kFillThreads;
  for (int64_t b = gtid; b <= n; b += gstep) p.a.q_start[b] = p.tok_base[b];
  if (gtid == 0) *p.a.next_cursor = (int32_t)next;
  // the cursor as it was: next_cursor may be the same word, so it is not read again here
  fill<kFillThreads>(p, p.tok_base, p.page_base, (int32_t)p.totals[0], next - p.page_base[n],
                     blockIdx.x, gridDim.x);
}

// The whole call in one CTA, a request a thread, the sums in shared memory.
__global__ void __launch_bounds__(kTabThreads) tables_one_kernel(const TabParams p) {
  __shared__ int64_t sm[32][2];
  __shared__ int32_t tok_base[kTabThreads + 1], page_base[kTabThreads + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = p.a.n_reqs, b = threadIdx.x;
  const int64_t cur = p.a.cursor ? p.a.cursor[0] : 0;
  int32_t bad = 0;
  int64_t cnt = 0, take = 0, tokens, pages;
  bool prefix = false;
  if (b < n) {
    prefix = takes_prefix(p, b);
    const Span s = checked_span(p, b, true, &bad);
    cnt = s.end - s.start;
    take = s.need - s.have;
  }
  block_scan2(cnt, take, &tokens, &pages, sm);
  if (b < n) tok_base[b] = (int32_t)cnt, page_base[b] = (int32_t)take;
  if (b == n % kTabThreads) tok_base[n] = (int32_t)tokens, page_base[n] = (int32_t)pages;
  check_ids(p, cur, tokens, pages, __syncthreads_or(prefix), b, kTabThreads, &bad);
  const int any_range = __syncthreads_or(bad == KVX_ERR_OUT_OF_RANGE);
  const int any_arg = __syncthreads_or(bad == KVX_ERR_INVALID_ARG);
  if (b == 0) *p.status = any_range ? KVX_ERR_OUT_OF_RANGE : any_arg ? KVX_ERR_INVALID_ARG : KVX_OK;
  if (any_range || any_arg) return;
  for (int i = b; i <= n; i += kTabThreads) p.a.q_start[i] = tok_base[i];
  if (b == 0) *p.a.next_cursor = (int32_t)(cur + pages);
  fill<kTabThreads>(p, tok_base, page_base, (int32_t)tokens, cur, 0, 1);
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3) == 0; }

static_assert(sizeof(kvx_tables_args) == 120, "the binding mirrors this structure");

}  // namespace
}  // namespace kvx

extern "C" size_t kvx_tables_workspace_size(int32_t n_reqs) {
  if (n_reqs < 0 || n_reqs > KVX_MAX_TABLE_REQUESTS) return 0;
  return (size_t)kvx::tab_layout(n_reqs).total;
}

extern "C" kvx_status kvx_block_tables(kvx_layout_t pool, const kvx_tables_args *args, void *d_ws,
                                       size_t ws_bytes, int32_t *d_status, kvx_stream_t stream) {
  using namespace kvx;
  if (!pool || !args || !d_status) return KVX_ERR_INVALID_ARG;
  const kvx_tables_args &a = *args;
  if (a.reserved != 0 || a.n_reqs < 0 || a.n_reqs > KVX_MAX_TABLE_REQUESTS || a.page_size < 1 ||
      a.n_prefix_pages < 0 || a.max_pages < 1 || a.table_stride < a.max_pages || a.n_free < 0 ||
      a.max_tokens < 0 || a.max_tokens > INT32_MAX)
    return KVX_ERR_INVALID_ARG;
  if (a.table_stride > ((int64_t)1 << 56) / KVX_MAX_TABLE_REQUESTS) return KVX_ERR_INVALID_ARG;
  if (pool->kind == KVX_HND_PAGED && pool->page_size != a.page_size) return KVX_ERR_INVALID_ARG;
  if (a.n_reqs > 0 && (!a.new_lens || !a.tables)) return KVX_ERR_INVALID_ARG;
  if ((a.n_prefix_pages > 0 && !a.prefix_pages) || (a.n_free > 0 && !a.free_pages) ||
      (a.max_tokens > 0 && !a.slots) || !a.next_cursor || !a.q_start)
    return KVX_ERR_INVALID_ARG;
  for (const void *q : {(const void *)a.old_lens, (const void *)a.new_lens,
                        (const void *)a.prefix_pages, (const void *)a.tables,
                        (const void *)a.free_pages, (const void *)a.cursor,
                        (const void *)a.next_cursor, (const void *)a.q_start,
                        (const void *)a.slots, (const void *)a.positions, (const void *)d_status})
    if (!aligned4(q)) return KVX_ERR_ALIGNMENT;
  const TabLayout L = tab_layout(a.n_reqs);
  if (!d_ws || ((uintptr_t)d_ws & 255) != 0 || (int64_t)ws_bytes < L.total)
    return KVX_ERR_NO_WORKSPACE;
  TabParams p;
  std::memset(&p, 0, sizeof(p));
  p.a = a;
  p.num_pages = pool->num_slots / a.page_size;
  p.page_shift = -1;
  for (int32_t s = 0; s < 31; ++s)
    if (a.page_size == (1 << s)) p.page_shift = s;
  p.prefix_tokens = (int64_t)a.n_prefix_pages * a.page_size;
  char *ws = static_cast<char *>(d_ws);
  p.verdict = reinterpret_cast<int32_t *>(ws);
  p.totals = reinterpret_cast<int64_t *>(ws + L.totals_off);
  p.tok_base = reinterpret_cast<int32_t *>(ws + L.tok_off);
  p.page_base = reinterpret_cast<int32_t *>(ws + L.page_off);
  p.status = d_status;
  // one more CTA for every 8192 page ids there may be to check
  const int64_t ids = (int64_t)a.n_free + a.n_prefix_pages;
  p.ctas = (int32_t)(1 + ids / 8192 < kTabMaxCtas ? 1 + ids / 8192 : kTabMaxCtas);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void *kargs[] = {&p};
  cudaError_t e;
  if (a.n_reqs <= kTabThreads && a.max_tokens <= kOneTokens &&
      (int64_t)a.n_reqs * a.n_prefix_pages <= kOneTokens) {
    e = launch_pdl((const void *)tables_one_kernel, dim3(1), dim3(kTabThreads), kargs, s);
  } else {
    e = launch_pdl((const void *)tables_plan_kernel, dim3(p.ctas), dim3(kTabThreads), kargs, s);
    if (e == cudaSuccess) {
      const int64_t chunks = (a.max_tokens + kFillChunk - 1) / kFillChunk;
      const int64_t rows = a.n_prefix_pages > 0 ? a.n_reqs : 1;
      const int64_t most = chunks > rows ? chunks : rows;
      const int64_t grid = most < 1 ? 1 : most < 152 * 8 ? most : 152 * 8;
      e = launch_pdl((const void *)tables_fill_kernel, dim3((unsigned)grid), dim3(kFillThreads),
                     kargs, s);
    }
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return KVX_ERR_CUDA;
  }
  return KVX_OK;
}
