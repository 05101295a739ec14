// gdn_attn_split.cuh -- attention of one new token per request over a paged cache: what does not
// depend on how the cache holds its numbers.  The work of all requests is divided evenly over one
// wave of CTAs (Schedule), each piece of it runs over its tokens (Piece, of the cache's type), and
// the parts of split pieces are added up (finish, k_attn_join).
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "gdn_internal.h"
#include "gdn_launch.cuh"

namespace gdn {
namespace {

constexpr int AT_W = 4;            // warps per CTA
constexpr int AT_NT = 32 * AT_W;
constexpr int AT_G = 8;            // query heads per product
constexpr int AT_SMS = 152;
constexpr float AT_LAZY = 8.f;     // log2 units
constexpr float AT_LOG2E = 1.4426950408889634f;
// What a piece costs beside its tiles, in units (its first loads and its end): without it a CTA
// with many short requests lags (61 ragged requests 128 against 102 us; 2 to 5: the same).
constexpr int AT_START = 1;

// Keys per warp tile, CTAs per SM and parts, for NG groups of AT_G query heads per piece: the K
// and V tiles and the accumulators of D x 8 NG fill most of a CTA's share of the registers.
// kParts > 1: the two tiles do not fit; they go by that many parts of D.
template <int KEYS, int CTAS, int PARTS>
struct Fit {
  static constexpr int kKeys = KEYS, kCtas = CTAS, kParts = PARTS;
};
template <int D, typename T, int NG> struct Cfg;

// What a cache of type T gives: the type of q and o, and the elements of a lane's load of V.
template <typename T> struct Cache {
  using Out = T;
  template <int D> static constexpr int el() { return 16 / (int)sizeof(T); }
};
// Shared memory of a CTA: kORow (floats of a row of o), kBytes.
template <int D, typename T, int NG> struct Smem;
// run(): tokens [0, n) of request b, units [t0, t1) of CTA tiles, into the warp's Acc.
template <int D, typename T, int NG> struct Piece;

// Parts of pieces in the workspace: slot 2c of CTA c is the piece that began before it, slot
// 2c + 1 the one that goes on behind it.  Join c tells of the piece that goes on from CTA c to
// CTA c + 1, if one does.
struct __align__(16) Join {
  int32_t b, h;         // request, piece of it
  int32_t first, last;  // CTAs that it begins and ends in (last < 0: none goes on)
};

struct AttnArgs {
  int64_t B, Hq, Hk, pages, max_blocks, qs;
  int P, G, HG;   // tokens per page, query heads per key head, pieces of them
  float sl;       // scale log2(e)
  float lazy;     // how far a score may be above its reference, in units of the unscaled scores
  const void *q, *kc, *vc;
  const float *ksc, *vsc;  // 8-bit caches: [pages][P / 16][Hk]
  const int32_t *table, *len;
  void* o;
  float* lse;
  Join* join;     // [CTAs]
  float2* ml;     // [CTAs][2][AT_G NG] reference score (unscaled) and sum
  float* acc;     // [CTAs][2][AT_G NG][D]
  int32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a warp keeps of its piece.
template <int D, int NG> struct Acc {
  float o[NG][D / 16][4];    // O^T tiles
  float m[NG][2], l[NG][2];  // heads 2t, 2t + 1: reference score (unscaled), this lane's sum
};

// The 4 warps' results joined, AT_G heads at a time: to o and lse (slot < 0), or as the partial
// piece `slot`.
template <int D, typename T, int NG>
__device__ void finish(const AttnArgs& ar, char* smem, float2 (*ml)[AT_G], int64_t b, int h0,
                       int heads, const Acc<D, NG>& a, int64_t slot) {
  constexpr int kORow = Smem<D, T, NG>::kORow, EL = Cache<T>::template el<D>();
  using TO = typename Cache<T>::Out;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  float* so = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    __syncthreads();  // every warp is done with Q, or with the heads before these
    if (g == 0) {
      ml[warp][2 * t] = make_float2(a.m[q][0], a.l[q][0]);
      ml[warp][2 * t + 1] = make_float2(a.m[q][1], a.l[q][1]);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int d = EL * (g + 8 * (i / (EL / 2))) + 2 * (i % (EL / 2));
      *reinterpret_cast<float2*>(so + (warp * AT_G + 2 * t) * kORow + d) =
          make_float2(a.o[q][i][0], a.o[q][i][2]);
      *reinterpret_cast<float2*>(so + (warp * AT_G + 2 * t + 1) * kORow + d) =
          make_float2(a.o[q][i][1], a.o[q][i][3]);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < min(AT_G, heads - q * AT_G) * (D / 2); x += AT_NT) {
      const int h = x / (D / 2), d = (x % (D / 2)) * 2, hp = q * AT_G + h;
      float m = -INFINITY, l = 0.f;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < AT_W; ++w) m = fmaxf(m, ml[w][h].x);
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < AT_W; ++w) {
        const float f = ex2((ml[w][h].x - base) * ar.sl);
        const float2 y = *reinterpret_cast<const float2*>(so + (w * AT_G + h) * kORow + d);
        l = fmaf(ml[w][h].y, f, l);
        o.x = fmaf(y.x, f, o.x);
        o.y = fmaf(y.y, f, o.y);
      }
      if (slot >= 0) {
        const int64_t at = slot * (AT_G * NG) + hp;
        *reinterpret_cast<float2*>(ar.acc + at * D + d) = o;
        if (d == 0) ar.ml[at] = make_float2(m, l);
        continue;
      }
      const float r = l != 0.f ? 1.f / l : 0.f;  // nothing counted: zero, not 0 / 0
      const int64_t row = b * ar.Hq + h0 + hp;
      TO* out = reinterpret_cast<TO*>(ar.o) + row * D + d;
      if constexpr (sizeof(TO) == 2)
        *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(o.x * r, o.y * r);
      else
        *reinterpret_cast<float2*>(out) = make_float2(o.x * r, o.y * r);
      if (d == 0 && ar.lse)
        ar.lse[row] = (base * ar.sl + log2f(l)) * 0.69314718055994531f;
    }
  }
}

// How the work is divided.  The units of request b are those of its
// pieces (key head x AT_G NG query heads) in a row, each its CTA tiles behind AT_START; the
// W units of all requests are divided over C CTAs, CTA c taking [W c / C, W (c + 1) / C).
// Each warp finds its way by itself: a lane sums up a run of requests, one scan over the lanes.
// AHEAD: read past the first-level cache, for a caller that has not waited for the kernel before
// it (the lengths were written before that one began).
template <int D, typename T, int NG, bool AHEAD>
struct Schedule {
  static constexpr int TK = Cfg<D, T, NG>::kKeys * AT_W;  // keys per CTA tile
  const AttnArgs& ar;
  int64_t W, incl, excl;  // all units; up to and before this lane's run
  int C, run, per;        // CTAs with work, requests per run, pieces per request

  __device__ __forceinline__ int length(int64_t b) const {
    const int32_t n = AHEAD ? __ldcg(ar.len + b) : ar.len[b];
    const int64_t cap = ar.max_blocks * ar.P;
    return (int)(n < 0 ? 0 : n > cap ? cap : n);
  }
  static __device__ __forceinline__ int tiles(int n) { return n > 0 ? (n - 1) / TK + 1 : 0; }
  __device__ __forceinline__ int64_t units(int64_t b) const {
    const int n = tiles(length(b));
    return n > 0 ? (int64_t)(n + AT_START) * per : 0;
  }
  static __device__ __forceinline__ int64_t scan(int64_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
  __device__ __forceinline__ Schedule(const AttnArgs& a, int ctas) : ar(a) {
    const int lane = threadIdx.x & 31;
    per = (int)ar.Hk * ar.HG;
    run = (int)((ar.B + 31) / 32);
    const int64_t b0 = (int64_t)lane * run, b1 = min(ar.B, b0 + run);
    int64_t sum = 0;
#pragma unroll 4
    for (int64_t b = b0; b < b1; ++b) sum += units(b);
    incl = scan(sum);
    excl = incl - sum;
    W = __shfl_sync(0xffffffffu, incl, 31);
    C = (int)(W < ctas ? W : ctas);
  }
  __device__ __forceinline__ int64_t first(int c) const { return W * c / C; }
  // the CTA of unit u: the last c with first(c) <= u
  __device__ __forceinline__ int cta_of(int64_t u) const { return (int)(((u + 1) * C - 1) / W); }
  // the request of unit u (0 <= u < W) and the unit's number in it
  __device__ __forceinline__ void find(int64_t u, int64_t* b, int64_t* r) const {
    const int lane = threadIdx.x & 31;
    const int own = __ffs(__ballot_sync(0xffffffffu, incl > u)) - 1;
    int64_t at = __shfl_sync(0xffffffffu, excl, own), b0 = (int64_t)own * run;
    if (run > 1) {
      const int64_t end = min(ar.B, b0 + run);
      for (;; b0 += 32) {
        const int64_t n = b0 + lane < end ? units(b0 + lane) : 0, x = scan(n);
        const unsigned over = __ballot_sync(0xffffffffu, at + x > u);
        if (over) {
          const int i = __ffs(over) - 1;
          at += __shfl_sync(0xffffffffu, x - n, i);
          b0 += i;
          break;
        }
        at += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    *b = b0;
    *r = u - at;
  }
};

template <int D, typename T, int NG>
__global__ void __launch_bounds__(AT_NT, Cfg<D, T, NG>::kCtas) k_attn_decode(AttnArgs ar) {
  constexpr int GP = AT_G * NG;
  using TO = typename Cache<T>::Out;
  extern __shared__ __align__(16) char smem[];
  __shared__ float2 ml[AT_W][AT_G];
  after_previous();
  before_next();
  const int tid = threadIdx.x, c = blockIdx.x;
  const Schedule<D, T, NG, false> sc(ar, gridDim.x);
  int bad = 0;
  if (c == 0)
    for (int64_t b = tid; b < ar.B; b += AT_NT) bad |= sc.length(b) != ar.len[b];
  // requests without tokens
  for (int64_t b = c; b < ar.B; b += gridDim.x)
    if (sc.length(b) == 0) {
      TO* o = reinterpret_cast<TO*>(ar.o) + b * ar.Hq * D;
      for (int64_t i = tid; i < ar.Hq * D; i += AT_NT) o[i] = (TO)0.f;
      if (ar.lse)
        for (int64_t i = tid; i < ar.Hq; i += AT_NT) ar.lse[b * ar.Hq + i] = -INFINITY;
    }
  Join goes_on{0, 0, 0, -1};
  if (c < sc.C) {
    int64_t u = sc.first(c), b, r;
    const int64_t u1 = sc.first(c + 1);
    sc.find(u, &b, &r);
    int n = sc.length(b), nt = sc.tiles(n), w = nt + AT_START;
    int h = (int)(r / w), r0 = (int)(r % w);  // piece of the request, unit in it
    while (u < u1) {
      const int r1 = (int)(u1 - u < w - r0 ? r0 + (u1 - u) : w);
      const int t0 = max(0, r0 - AT_START), t1 = max(0, r1 - AT_START);
      if (t0 < t1) {
        const int hk = h / ar.HG, hg = h % ar.HG, heads = min(GP, ar.G - hg * GP);
        Acc<D, NG> a;
        Piece<D, T, NG>::run(ar, smem, b, n, hk, hg, t0, t1, a, &bad);
        const int64_t slot = t0 == 0 && t1 == nt ? -1 : t0 == 0 ? 2 * c + 1 : 2 * c;
        finish<D, T, NG>(ar, smem, ml, b, hk * ar.G + hg * GP, heads, a, slot);
        if (t1 < nt) {  // the share ends in this piece, whose tile 0 is unit u - r0 + AT_START
          const int64_t tile0 = u - r0 + AT_START;
          goes_on = Join{(int32_t)b, h, sc.cta_of(tile0), sc.cta_of(tile0 + nt - 1)};
        }
      }
      u += r1 - r0;
      r0 = 0;
      if (u < u1 && ++h == sc.per) {
        h = 0;
        do n = sc.length(++b); while (n == 0);
        nt = sc.tiles(n);
        w = nt + AT_START;
      }
    }
  }
  if (tid == 0) ar.join[c] = goes_on;
  if (bad && ar.status) atomicOr(ar.status, kStatusClamped);
}

constexpr int AJ_NT = 32 * AT_G;  // a warp per query head
constexpr int AJ_FEW = 8;        // parts that one warp adds up by itself
constexpr int AJ_DC = 64;         // columns per item of a CTA

template <typename T>
__device__ __forceinline__ void store_o(T* o, float4 x, float r) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x * r, x.y * r);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x.z * r, x.w * r);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(o) = make_float4(x.x * r, x.y * r, x.z * r, x.w * r);
  }
}
__device__ __forceinline__ void add_scaled(float4& a, const float4& x, float f) {
  a.x = fmaf(x.x, f, a.x);
  a.y = fmaf(x.y, f, a.y);
  a.z = fmaf(x.z, f, a.z);
  a.w = fmaf(x.w, f, a.w);
}

// Adds up the parts of the pieces that were split.  CTA x serves the piece that goes on from CTA
// x of the pass above to CTA x + 1: a piece of n parts has n - 1 CTAs.  They share its items (a
// query head and AJ_DC columns), 16 parts at a time; or, with up to AJ_FEW parts (a batch: hundreds
// of pieces of 2 or 3), or up to 32 where the CTAs would have to take several items each, the
// first of them does it alone, a warp per query head (517 tokens, 9 parts, 32 items: 9.4 us for
// the whole call against 12.7 shared; 10 parts of 3 items: 13.4 shared, 14.3 alone).  Which piece
// it is, a CTA works out from the lengths while the pass still runs where one load per warp tells
// them (the kernels in front of the pass wrote them; 8 requests of 1000 tokens 11.9 against 12.8
// us); with more requests all CTAs together would wait for the same few lines of L2 (400 requests
// of 100 tokens 102 us), and it reads what the pass wrote down (44 us).
template <int D, typename T, int NG>
__global__ void __launch_bounds__(AJ_NT) k_attn_join(AttnArgs ar) {
  using TO = typename Cache<T>::Out;
  constexpr int GP = AT_G * NG, NW = AJ_NT / 32, MAXC = AT_SMS * Cfg<D, T, NG>::kCtas;
  __shared__ float s_w[MAXC], s_red[NW][2];
  __shared__ float4 s_o[AJ_NT / 16][AJ_DC / 4];
  const int x = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Join j{0, 0, 0, -1};
  if (ar.B <= 32) {
    const Schedule<D, T, NG, true> sc(ar, gridDim.x);
    if (x < sc.C) {
      int64_t b, r;
      const int64_t u = sc.first(x + 1) - 1;  // CTA x's last unit, in piece [start, start + w)
      sc.find(u, &b, &r);
      const int w = sc.tiles(sc.length(b)) + AT_START;
      const int64_t tile0 = u - r % w + AT_START;
      j = Join{(int32_t)b, (int32_t)(r / w), sc.cta_of(tile0), sc.cta_of(tile0 + w - AT_START - 1)};
    }
    after_previous();
    if (x < j.first || x >= j.last) return;
  } else {
    after_previous();
    j = ar.join[x];
    if (j.last < 0) return;
  }
  before_next();
  const int c = j.first, n = j.last - c + 1;
  const int hk = j.h / ar.HG, hg = j.h % ar.HG, heads = min(GP, ar.G - hg * GP);
  const int64_t row0 = (int64_t)j.b * ar.Hq + hk * ar.G + hg * GP;
  // parts: slot 2c + 1 of the piece's first CTA c, slot 2i of the CTAs behind it
  if (n <= AJ_FEW || (n <= 32 && heads * (D / AJ_DC) > n - 1)) {
    if (x > c) return;
    for (int g = warp; g < heads; g += NW) {
      auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * GP + g; };
      const float2 ml = lane < n ? ar.ml[slot(lane)] : make_float2(-INFINITY, 0.f);
      float m = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.f : m, f = ex2((ml.x - base) * ar.sl);
      float l = ml.y * f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      constexpr int V = D >= 128 ? D / 128 : 1;  // columns 4 lane + 128 v
      const bool in = D >= 128 || lane * 4 < D;
      float4 a[V];
#pragma unroll
      for (int v = 0; v < V; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < n; i0 += AJ_FEW)
#pragma unroll
        for (int j = 0; j < AJ_FEW; ++j) {
          const int i = i0 + j;
          const float fi = __shfl_sync(0xffffffffu, f, i);
          const float* part = ar.acc + slot(i) * D + lane * 4;
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (i < n && in) add_scaled(a[v], *reinterpret_cast<const float4*>(part + v * 128), fi);
        }
      const float q = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (in) store_o(reinterpret_cast<TO*>(ar.o) + (row0 + g) * D + lane * 4 + v * 128, a[v], q);
      if (lane == 0 && ar.lse) ar.lse[row0 + g] = (base * ar.sl + log2f(l)) * 0.69314718055994531f;
    }
    return;
  }
  for (int item = x - c; item < heads * (D / AJ_DC); item += n - 1) {
    const int g = item % heads, d0 = item / heads * AJ_DC, col = tid % 16, first = tid / 16;
    auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * GP + g; };
    float m = -INFINITY, l = 0.f;
    for (int i = tid; i < n; i += AJ_NT) m = fmaxf(m, ar.ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();  // the last item's readers are done
    if (lane == 0) s_red[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, s_red[w][0]);
    const float base = m == -INFINITY ? 0.f : m;
    for (int i = tid; i < n; i += AJ_NT) {
      const float2 y = ar.ml[slot(i)];
      const float f = ex2((y.x - base) * ar.sl);
      s_w[i] = f;
      l = fmaf(y.y, f, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) s_red[warp][1] = l;
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = first; i < n; i += AJ_NT / 16)
      add_scaled(a, *reinterpret_cast<const float4*>(ar.acc + slot(i) * D + d0 + col * 4), s_w[i]);
    s_o[first][col] = a;
    __syncthreads();
    if (tid < AJ_DC / 4) {
      a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < AJ_NT / 16; ++i) add_scaled(a, s_o[i][tid], 1.f);
      l = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) l += s_red[w][1];
      store_o(reinterpret_cast<TO*>(ar.o) + (row0 + g) * D + d0 + tid * 4, a,
              l != 0.f ? 1.f / l : 0.f);
      if (tid == 0 && d0 == 0 && ar.lse)
        ar.lse[row0 + g] = (base * ar.sl + log2f(l)) * 0.69314718055994531f;
    }
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool ok16(const void* p, int64_t n) { return n == 0 || (p && aligned16(p)); }
bool ok4(const void* p, int64_t n) { return n == 0 || (p && ((uintptr_t)p & 3u) == 0); }

gdn_status check_problem(const gdn_attn_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (p->B < 0 || p->Hq < 1 || p->Hk < 1 || p->Hq % p->Hk != 0 || p->pages < 0 ||
      p->max_blocks < 0 || p->page_size < 1 || p->D < 1 || !isfinite(p->scale) ||
      !isfinite(fmaxf(p->scale, 0.f) * AT_LOG2E))
    return GDN_ERR_INVALID_ARG;
  const int64_t unit = p->dtype == GDN_BF16 ? 8 : 4;  // elements in 16 bytes
  if (p->q_stride != 0 && (p->q_stride < p->Hq * p->D || p->q_stride % unit != 0))
    return GDN_ERR_INVALID_ARG;
  if ((p->D != 64 && p->D != 128 && p->D != 256) || p->page_size % 16 != 0)
    return GDN_ERR_UNSUPPORTED;
  constexpr int64_t top = 0x7fffffff;
  if (p->pages > top / p->page_size || p->max_blocks > top / p->page_size || p->Hq > top ||
      p->B > top / p->Hq)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// CTAs of the pass and the workspace's parts (a fixed count per kind, so that results do not
// depend on the device).
struct Plan {
  int ctas;
  size_t ml, acc, total;
};
template <int D, typename T, int NG>
Plan plan_of() {
  Plan pl;
  pl.ctas = AT_SMS * Cfg<D, T, NG>::kCtas;
  const size_t parts = (size_t)pl.ctas * 2 * AT_G * NG;
  pl.ml = (pl.ctas * sizeof(Join) + 255) & ~(size_t)255;
  pl.acc = pl.ml + ((parts * sizeof(float2) + 255) & ~(size_t)255);
  pl.total = pl.acc + parts * D * sizeof(float);
  return pl;
}
template <int D, typename T>
size_t workspace_of() {
  const size_t a = plan_of<D, T, 1>().total, b = plan_of<D, T, 2>().total;
  return a > b ? a : b;
}

// The call's arguments but for the workspace's and the scales.
inline AttnArgs args_of(const gdn_attn_problem* p, const void* q, const void* k_cache,
                        const void* v_cache, const int32_t* block_table, const int32_t* seq_len,
                        void* o, float* lse, int32_t* status, float lazy) {
  AttnArgs ar;
  memset(&ar, 0, sizeof(ar));
  ar.B = p->B;
  ar.Hq = p->Hq;
  ar.Hk = p->Hk;
  ar.pages = p->pages;
  ar.max_blocks = p->max_blocks;
  ar.qs = p->q_stride ? p->q_stride : p->Hq * p->D;
  ar.P = p->page_size;
  ar.G = (int)(p->Hq / p->Hk);
  ar.sl = (p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->D)) * AT_LOG2E;
  ar.lazy = fminf(lazy / ar.sl, 1e30f);
  ar.q = q;
  ar.kc = k_cache;
  ar.vc = v_cache;
  ar.table = block_table;
  ar.len = seq_len;
  ar.o = o;
  ar.lse = lse;
  ar.status = status;
  return ar;
}

template <int D, typename T, int NG>
cudaError_t launch(AttnArgs ar, char* ws, cudaStream_t st) {
  const Plan pl = plan_of<D, T, NG>();
  ar.HG = (ar.G + AT_G * NG - 1) / (AT_G * NG);
  ar.join = (Join*)ws;
  ar.ml = (float2*)(ws + pl.ml);
  ar.acc = (float*)(ws + pl.acc);
  cudaError_t e = cudaSuccess;
  if constexpr (Smem<D, T, NG>::kBytes > 48 * 1024)
    e = allow_smem<k_attn_decode<D, T, NG>>(Smem<D, T, NG>::kBytes);
  if (e == cudaSuccess)
    e = launch_behind(k_attn_decode<D, T, NG>, dim3(pl.ctas), AT_NT, Smem<D, T, NG>::kBytes, st, ar);
  if (e != cudaSuccess) return e;
  return launch_behind(k_attn_join<D, T, NG>, dim3(pl.ctas), AJ_NT, 0, st, ar);
}

}  // namespace
}  // namespace gdn
