// gdn_slots.cu -- block tables, slots and positions of a serving step from request lengths.
// Request b has ctx_b cached tokens and new_b new ones; with P tokens per page
//   cu_b    = sum_{i<b} new_i                                  (packed token offsets)
//   need_b  = ceil((ctx_b + new_b) / P) - ceil(ctx_b / P),  first_b = sum_{i<b} need_i
// (both lengths at most what a row of the table holds) and token j of request b is at position
// ctx_b + j, on the request's page number i = position / P: an old page (block_table) below
// ceil(ctx_b / P), else entry first_b + i - ceil(ctx_b / P) of the free list.
//
// Integer work on a few KB: bound by latency, so one launch.  Every CTA scans the lengths
// itself (SM_NT at a time, 64-bit sums) up to the tokens that it owns, rather than wait for
// a scan kernel: the lengths come from L2.  A token finds its request by a binary search in
// shared memory.  The token at the first row of a new page writes the page's entry of
// block_table (each new page has exactly one such token); CTA 0 writes the per-request
// outputs.  Pages are numbered by the requests before, so that a cut at the last token row
// changes only the request that it falls on and those behind it, which have no token here.
#include <string.h>

#include "gdn_internal.h"
#include "gdn_launch.cuh"

namespace gdn {
namespace {

constexpr int SM_NT = 256;      // threads per CTA, requests per scan step
constexpr int SM_TOK = 1024;    // tokens per CTA

struct SlotArgs {
  uint32_t P;
  int64_t B, max_blocks, pages, n_free, n_tokens;
  const int32_t* ctx;
  const int32_t* nw;
  const int32_t* free_pages;
  int32_t* table;
  int32_t* seq_len;
  int32_t* cu;
  int32_t* pos;
  int32_t* slots;
  int32_t* used;
  int32_t* status;
};

__device__ __forceinline__ int32_t sat31(int64_t x) {
  return x > 0x7fffffff ? 0x7fffffff : (int32_t)x;
}

__device__ __forceinline__ uint32_t ceil_div(uint32_t x, uint32_t d) {
  return x == 0 ? 0 : (x - 1) / d + 1;
}

// inclusive sums of two values over the CTA's threads, in thread order
__device__ __forceinline__ void scan2(int64_t& x, int64_t& y, int64_t (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ux = __shfl_up_sync(0xffffffffu, x, o), uy = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += ux;
      y += uy;
    }
  }
  if (lane == 31) {
    part[warp][0] = x;
    part[warp][1] = y;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    x += part[w][0];
    y += part[w][1];
  }
}

__global__ void __launch_bounds__(SM_NT) k_slot_map(SlotArgs ar) {
  __shared__ int64_t part[SM_NT / 32][2];
  __shared__ int64_t s_cu[SM_NT + 1], s_first[SM_NT + 1];
  __shared__ uint32_t s_ctx[SM_NT];
  after_previous();
  before_next();
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * SM_TOK;
  const int64_t t1 = t0 + SM_TOK < ar.n_tokens ? t0 + SM_TOK : ar.n_tokens;
  const uint32_t cap = (uint32_t)(ar.max_blocks * ar.P);  // below 2^31
  const bool lead = blockIdx.x == 0;
  int bad = 0;
  int64_t cu0 = 0, first0 = 0;  // sums over the requests of earlier steps
  for (int64_t b0 = 0; b0 < ar.B && (lead || cu0 < t1); b0 += SM_NT) {
    const int64_t b = b0 + tid;
    uint32_t c = 0, n = 0;  // below 2^31 each: their sum fits 32 bits, and divides in 32
    if (b < ar.B) {
      const int32_t ci = ar.ctx[b], ni = ar.nw[b];
      c = ci < 0 ? 0 : ci;
      n = ni < 0 ? 0 : ni;
      if (ci < 0 || ni < 0 || c + n > cap) bad = 1;
    }
    const auto pages_of = [&](uint32_t x) { return ceil_div(min(x, cap), ar.P); };
    const int64_t need = pages_of(c + n) - pages_of(c);  // the table takes no others
    int64_t cu = n, first = need;
    scan2(cu, first, part);
    if (tid == 0) {
      s_cu[0] = cu0;
      s_first[0] = first0;
    }
    s_cu[tid + 1] = cu0 + cu;
    s_first[tid + 1] = first0 + first;
    s_ctx[tid] = c;
    if (lead && b < ar.B) {
      // tokens past n_tokens have no row: the step is the one without them, lengths and pages too
      const int64_t room = ar.n_tokens - (cu0 + cu - n);
      const uint32_t kept = room < (int64_t)n ? (uint32_t)(room > 0 ? room : 0) : n;
      ar.seq_len[b] = (int32_t)min(c + kept, cap);
      ar.cu[b + 1] = (int32_t)min(cu0 + cu, ar.n_tokens);
      if (room >= 0 && kept < n) {  // the one request that the end falls on
        const int64_t taken = first0 + first - need + pages_of(c + kept) - pages_of(c);
        ar.used[0] = sat31(taken);
        bad = 1;
      }
    }
    __syncthreads();
    const int64_t lo = s_cu[0] > t0 ? s_cu[0] : t0;
    const int64_t hi = s_cu[SM_NT] < t1 ? s_cu[SM_NT] : t1;
    for (int64_t t = lo + tid; t < hi; t += SM_NT) {
      int l = 0, r = SM_NT;  // s_cu[l] <= t < s_cu[r]
      while (r - l > 1) {
        const int m = (l + r) >> 1;
        if (s_cu[m] <= t) l = m; else r = m;
      }
      const uint32_t p = s_ctx[l] + (uint32_t)(t - s_cu[l]), i = p / ar.P;
      const uint32_t held = ceil_div(s_ctx[l], ar.P);
      int32_t page = -1;
      if (i < ar.max_blocks) {
        int32_t* entry = ar.table + (b0 + l) * ar.max_blocks + i;
        if (i < held) {
          page = *entry;
        } else {
          const int64_t f = s_first[l] + (i - held);
          if (f < ar.n_free) page = ar.free_pages[f];
          if (page < 0 || page >= ar.pages) page = -1;
          if (p == i * ar.P) *entry = page;
        }
      }
      const bool ok = page >= 0 && page < ar.pages;
      if (!ok) bad = 1;
      ar.pos[t] = sat31(p);
      ar.slots[t] = ok ? (int32_t)((uint32_t)page * ar.P + (p - i * ar.P)) : -1;
    }
    cu0 = s_cu[SM_NT];
    first0 = s_first[SM_NT];
    __syncthreads();
  }
  // padding rows (cu0 is the total here unless this CTA's tokens end before it)
  for (int64_t t = (cu0 > t0 ? cu0 : t0) + tid; t < t1; t += SM_NT) {
    ar.pos[t] = 0;
    ar.slots[t] = -1;
  }
  if (lead && tid == 0) {
    ar.cu[0] = 0;
    if (cu0 <= ar.n_tokens) {
      ar.used[0] = sat31(first0);
      if (first0 > ar.n_free) bad = 1;
    }
  }
  if (bad && ar.status) atomicOr(ar.status, kStatusClamped);
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool ok4(const void* p, int64_t n) { return n == 0 || (p && aligned4(p)); }

// An array of n int32 in memory.
struct Span {
  uintptr_t first, last;  // bytes; empty: first > last
  Span(const void* p, int64_t n) {
    first = n > 0 ? (uintptr_t)p : 1;
    const uintptr_t left = (UINTPTR_MAX - first) / 4;
    last = n > 0 ? first + 4 * ((uint64_t)n < left ? (uintptr_t)n : left) - 1 : 0;
  }
  bool meets(const Span& o) const {
    return first <= last && o.first <= o.last && first <= o.last && o.first <= last;
  }
};

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_slot_map(const gdn_slot_problem* p, const int32_t* ctx_len,
                                   const int32_t* new_len, const int32_t* free_pages,
                                   int32_t* block_table, int32_t* seq_len, int32_t* cu_seqlens,
                                   int32_t* positions, int32_t* slots, int32_t* used,
                                   int32_t* status, void* stream) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->page_size < 1 || p->B < 0 || p->max_blocks < 0 || p->pages < 0 || p->n_free < 0 ||
      p->n_tokens < 0)
    return GDN_ERR_INVALID_ARG;
  constexpr int64_t top = 0x7fffffff;
  if (p->B > top || p->n_free > top || p->n_tokens > top || p->pages > top / p->page_size ||
      p->max_blocks > top / p->page_size)
    return GDN_ERR_UNSUPPORTED;
  if (!ok4(ctx_len, p->B) || !ok4(new_len, p->B) || !ok4(free_pages, p->n_free) ||
      !ok4(block_table, p->B * p->max_blocks) || !ok4(seq_len, p->B) || !ok4(cu_seqlens, 1) ||
      !ok4(positions, p->n_tokens) || !ok4(slots, p->n_tokens) || !ok4(used, 1) ||
      ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  // CTAs read lengths, pages and table entries while others write: nothing may lie on anything
  const Span in[] = {{ctx_len, p->B}, {new_len, p->B}, {free_pages, p->n_free}};
  const Span out[] = {{block_table, p->B * p->max_blocks}, {seq_len, p->B},
                      {cu_seqlens, p->B + 1}, {positions, p->n_tokens},
                      {slots, p->n_tokens}, {used, 1}};
  for (const Span& o : out) {
    for (const Span& i : in)
      if (o.meets(i)) return GDN_ERR_INVALID_ARG;
    for (const Span& other : out)
      if (&other != &o && o.meets(other)) return GDN_ERR_INVALID_ARG;
  }
  SlotArgs ar;
  memset(&ar, 0, sizeof(ar));
  ar.P = (uint32_t)p->page_size;
  ar.B = p->B;
  ar.max_blocks = p->max_blocks;
  ar.pages = p->pages;
  ar.n_free = p->n_free;
  ar.n_tokens = p->n_tokens;
  ar.ctx = ctx_len;
  ar.nw = new_len;
  ar.free_pages = free_pages;
  ar.table = block_table;
  ar.seq_len = seq_len;
  ar.cu = cu_seqlens;
  ar.pos = positions;
  ar.slots = slots;
  ar.used = used;
  ar.status = status;
  const int64_t ctas = p->n_tokens > 0 ? (p->n_tokens + SM_TOK - 1) / SM_TOK : 1;
  const cudaError_t e =
      launch_behind(k_slot_map, dim3((unsigned)ctas), SM_NT, 0, (cudaStream_t)stream, ar);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
