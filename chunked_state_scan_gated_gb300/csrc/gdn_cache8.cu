// gdn_cache8.cu -- a paged key-value cache in 8 bits, written and read back.  A block is 16 tokens
// of one head; with s its scale (a power of two) and x an element:
//   code = e4m3(x / s),  value = code s,   s = min { 2^e >= 2^-100 : 448 2^e >= |x| of the block }
// A power of two costs no accuracy (e4m3 is a floating-point type: what matters is that nothing
// overflows and little falls below 2^-6 s), x / s and code s are exact, and when a later token
// raises the scale of a block that is partly filled, its earlier codes only move their exponents.
//
// Both are bound by HBM (write: width + 1 bytes per element, read: 1 + width).  A CTA takes 16
// packed token rows and finds their requests with one 32-way search per row; in write8 the rows
// that open a block (the first row of a request or of a block) lead, and a warp takes one block of
// one head at a time, its rows in registers: one pass for the scale and the codes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <string.h>

#include <type_traits>

#include "gdn_internal.h"
#include "gdn_launch.cuh"

namespace gdn {
namespace {

constexpr int C8_NT = 256;
constexpr int C8_W = C8_NT / 32;
constexpr int C8_ROWS = 16;   // packed token rows of a CTA
constexpr int C8_BLOCK = 16;  // tokens that share a scale
constexpr int C8_MANY = 4096, C8_CTAS = 608;  // requests beyond which there are so many CTAs at most

struct Cache8Args {
  int64_t N, B, pages, max_blocks, ks, vs;
  int P, Hk;
  const void *k, *v;  // write8
  void *ko, *vo;      // read8
  uint8_t *kc, *vc;
  float *ksc, *vsc;
  const int32_t *table, *ctx, *cu;
  int32_t* status;
};

// The last b in [0, B) with cu[b] <= t, or -1; by the whole warp.
__device__ __forceinline__ int64_t request_of(const int32_t* cu, int64_t B, int64_t t) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = B;
  while (true) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < hi && cu[at] <= t);
    if (m == 0) return -1;
    lo += (31 - __clz(m)) * step;
    if (step == 1) return lo;
    hi = min(hi, lo + step);
  }
}

// The same where offsets may be anything: they count as cut to [0, N] and raised to the largest before
// them, so the request is the one in front of the first that is above t; from the first offset on.
__device__ __forceinline__ int64_t request_through(const Cache8Args& ar, int64_t t, int64_t* first,
                                                   int64_t* end) {
  const int lane = threadIdx.x & 31, n = (int)ar.N;
  int top = 0;
  for (int64_t i0 = 0; i0 <= ar.B; i0 += 32) {
    const int64_t i = i0 + lane;
    const int c = i <= ar.B ? max(0, min(ar.cu[i], n)) : 0;
    const unsigned over = __ballot_sync(0xffffffffu, c > t);
    const int k = over ? __ffs(over) - 1 : 32;
    top = max(top, __reduce_max_sync(0xffffffffu, lane < k ? c : 0));
    if (over) {
      *first = top;
      *end = __shfl_sync(0xffffffffu, c, k);
      return i0 + k - 1;
    }
  }
  return -1;
}

// Where 16 token rows are: request, position in it, end of its packed rows (0: none).
struct Rows {
  int64_t t0;   // the first
  int ordered;  // whether the offsets are in order
  int64_t pos[C8_ROWS];
  int32_t b[C8_ROWS], end[C8_ROWS];
  int32_t lead[C8_ROWS];
};

// ORDERED: the offsets are in order and within the rows.
template <bool WRITE, bool ORDERED>
__device__ __forceinline__ void find_rows(const Cache8Args& ar, int64_t t0, Rows* r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < C8_ROWS / C8_W; ++i) {
    const int slot = warp + i * C8_W;
    const int64_t t = t0 + slot;
    int64_t b = -1, first = 0, end = 0, ctx = 0;
    if (t < ar.N) b = ORDERED ? request_of(ar.cu, ar.B, t) : request_through(ar, t, &first, &end);
    if (b >= 0) {
      if (ORDERED) {
        first = ar.cu[b];
        end = ar.cu[b + 1];
      }
      if (WRITE) ctx = max(ar.ctx[b], 0);
      if (end <= t) end = 0;
    } else {
      end = 0;
    }
    if (lane == 0) {
      r->b[slot] = (int32_t)b;
      r->end[slot] = (int32_t)end;
      r->pos[slot] = ctx + t - first;
      r->lead[slot] = end > 0 && (t == first || (ctx + t - first) % C8_BLOCK == 0);
    }
  }
}

// A CTA's first rows.  Only all offsets together tell whether they are in order, and no launch before
// this one looks at them: every CTA does, while its rows are searched for as if they were (37 requests
// of 500 to 4000 tokens, bf16: written 105.5 us without that, 106.9 with it at 8 heads of 128, 65 and 68
// at 2 of 256; read back the same; 250 tokens 4.9 and 5.1).
template <bool WRITE>
__device__ __forceinline__ void find_first_rows(const Cache8Args& ar, Rows* r, int* bad) {
  const int64_t t0 = (int64_t)blockIdx.x * C8_ROWS, b0 = threadIdx.x;
  const int32_t c0 = b0 < ar.B ? ar.cu[b0] : 0, c1 = b0 < ar.B ? ar.cu[b0 + 1] : 0;
  find_rows<WRITE, true>(ar, t0, r);
  int out = c0 < 0 || c0 > ar.N || c1 < c0;
#pragma unroll 8
  for (int b = (int)b0 + C8_NT; b < (int)ar.B; b += C8_NT) {
    const int32_t x = ar.cu[b], y = ar.cu[b + 1];
    out |= x < 0 || x > (int)ar.N || y < x;
  }
  if (b0 == 0) out |= ar.cu[ar.B] > ar.N;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    *bad = out;
    if (WRITE)
      for (int64_t b = b0; b < ar.B; b += C8_NT) *bad |= ar.ctx[b] < 0;
  }
  if (threadIdx.x == 0) r->t0 = t0;
  out = __syncthreads_or(out);
  if (threadIdx.x == 0) r->ordered = !out;
  if (out) {
    find_rows<WRITE, false>(ar, t0, r);
    __syncthreads();
  }
}
template <bool WRITE>
__device__ __forceinline__ void find_more_rows(const Cache8Args& ar, Rows* r) {
  const int64_t t0 = r->t0 + (int64_t)gridDim.x * C8_ROWS;
  __syncthreads();  // the rows before are done
  if (threadIdx.x == 0) r->t0 = t0;
  if (r->ordered) find_rows<WRITE, true>(ar, t0, r);
  else find_rows<WRITE, false>(ar, t0, r);
  __syncthreads();
}

// Cache row of position pos of request b, or -1.
__device__ __forceinline__ int64_t cache_row(const Cache8Args& ar, int64_t b, int64_t pos) {
  const int64_t i = pos / ar.P;
  if (i >= ar.max_blocks) return -1;
  const int64_t page = ar.table[b * ar.max_blocks + i];
  return page >= 0 && page < ar.pages ? page * ar.P + pos % ar.P : -1;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
template <typename T>
__device__ __forceinline__ float element(const uint4& v, int i) {
  if constexpr (sizeof(T) == 2)
    return __uint_as_float(i & 1 ? word(v, i >> 1) & 0xffff0000u : word(v, i >> 1) << 16);
  else
    return __uint_as_float(word(v, i));
}

// Two e4m3 codes of a and b (ties to even); what is not finite becomes NaN (FINITE: there is none).
template <bool FINITE>
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  uint32_t r = c;
  if (!FINITE && !(fabsf(a) < INFINITY)) r |= 0x7fu;
  if (!FINITE && !(fabsf(b) < INFINITY)) r |= 0x7f00u;
  return r;
}
// The larger of m and |elements| of v, as bits (two 16-bit maxima for bf16).
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t m, const uint4& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) m = __vmaxu2(m, word(v, i) & 0x7fff7fffu);
    else m = max(m, word(v, i) & 0x7fffffffu);
  }
  return m;
}
// Two numbers of two codes, the first in x.
__device__ __forceinline__ float2 values2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The smallest power of two s >= 2^-100 with 448 s >= top (finite, not negative).
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t bits = __float_as_uint(top);
  // top = m 2^e with m in [1, 2): 448 = 1.75 2^8
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

// CTAs per SM: a block's rows are D sizeof(T) / 8 registers of a thread, and what bounds the call is
// how many blocks are on their way (63,000 tokens of 8 heads of 128, bf16: 110 us with 2 CTAs, 91
// with 3, 85 with 4, 80% of the measured copy rate; of 2 heads of 256: 71 with 2, 55 with 3).
template <int D, typename T>
constexpr int write_ctas() {
  constexpr int x = D * (int)sizeof(T) / 8;
  return x <= 16 ? 5 : x <= 32 ? 4 : x <= 64 ? 3 : 1;
}

template <int D, typename T, bool MANY>
__global__ void __launch_bounds__(C8_NT, write_ctas<D, T>()) k_cache_write8(Cache8Args ar) {
  constexpr int EL = 16 / (int)sizeof(T);       // elements of a load
  constexpr int LR = D / EL;                    // loads of a row
  constexpr int RPI = LR >= 32 ? 1 : 32 / LR;   // rows a warp loads at once
  constexpr int CPL = LR > 32 ? LR / 32 : 1;    // loads of a row per lane
  constexpr int NIT = C8_BLOCK / RPI;
  __shared__ Rows rows;
  after_previous();
  before_next();
  int bad = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  find_first_rows<true>(ar, &rows, &bad);
  while (true) {  // MANY: several runs of rows
    const unsigned leads = __ballot_sync(0xffffffffu, lane < C8_ROWS && rows.lead[lane & 15]);
    const int per = 2 * ar.Hk, units = __popc(leads) * per;
    for (int u = blockIdx.y * C8_W + warp; u < units; u += gridDim.y * C8_W) {
      const int slot = __fns(leads, 0, u / per + 1), h = (u % per) >> 1;
      const bool isv = u & 1;
      const int64_t t0 = rows.t0 + slot, pos = rows.pos[slot];
      const int in = (int)(pos % C8_BLOCK);  // earlier tokens of the block
      const int n = min(C8_BLOCK - in, (int)(rows.end[slot] - t0));
      const int64_t row = cache_row(ar, rows.b[slot], pos);
      if (row < 0) {
        bad = 1;
        continue;
      }
      const int64_t ts = isv ? ar.vs : ar.ks;
      const T* src = reinterpret_cast<const T*>(isv ? ar.v : ar.k) + t0 * ts + (int64_t)h * D;
      float* sc = (isv ? ar.vsc : ar.ksc) + (row / C8_BLOCK) * ar.Hk + h;
      uint8_t* dst = (isv ? ar.vc : ar.kc) + (row * ar.Hk + h) * (int64_t)D;  // the first new row
      const int64_t dr = (int64_t)ar.Hk * D;
      const int r0 = LR >= 32 ? 0 : lane / LR, c0 = LR >= 32 ? lane : lane % LR;
      uint4 x[NIT][CPL];
#pragma unroll
      for (int i = 0; i < NIT; ++i)
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          x[i][c] = make_uint4(0, 0, 0, 0);
          if (i * RPI + r0 < n)
            x[i][c] = *reinterpret_cast<const uint4*>(src + (i * RPI + r0) * ts +
                                                      (c0 + c * 32) * EL);
        }
      const float before = in > 0 ? *sc : 0.f;
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < NIT; ++i)
#pragma unroll
        for (int c = 0; c < CPL; ++c) bits = top_bits<T>(bits, x[i][c]);
      if (sizeof(T) == 2) bits = max(bits << 16, bits & 0xffff0000u);
      bits = __reduce_max_sync(0xffffffffu, bits);
      const bool finite = bits < 0x7f800000u;  // uniform in the warp
      float top = __uint_as_float(bits);
      if (!finite) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < NIT; ++i)
#pragma unroll
          for (int c = 0; c < CPL; ++c)
#pragma unroll
            for (int e = 0; e < EL; ++e) {
              const float y = fabsf(element<T>(x[i][c], e));
              top = fmaxf(top, y < INFINITY ? y : 0.f);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const float s = fmaxf(scale_for(top), before), inv = 1.f / s;  // powers of two: exact
      if (in > 0 && s != before) {
        // the earlier tokens' codes at the new scale, 16 bytes at a time
        const float f = before * inv;
        for (int j = lane; j < in * (D / 16); j += 32) {
          uint4* at = reinterpret_cast<uint4*>(dst - (in - j / (D / 16)) * dr + j % (D / 16) * 16);
          uint4 v = *at;
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = values2(w[i] & 0xffffu), b = values2(w[i] >> 16);
            w[i] = codes2<false>(a.x * f, a.y * f) | codes2<false>(b.x * f, b.y * f) << 16;
          }
          *at = v;
        }
      }
      auto store = [&](auto fin) {
        constexpr bool kFin = decltype(fin)::value;
#pragma unroll
        for (int i = 0; i < NIT; ++i)
          if (i * RPI + r0 < n)
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
              uint32_t w[EL / 4];
#pragma unroll
              for (int e = 0; e < EL; e += 4) {
                const uint4& v = x[i][c];
                w[e / 4] =
                    codes2<kFin>(element<T>(v, e) * inv, element<T>(v, e + 1) * inv) |
                    codes2<kFin>(element<T>(v, e + 2) * inv, element<T>(v, e + 3) * inv) << 16;
              }
              uint8_t* at = dst + (i * RPI + r0) * dr + (c0 + c * 32) * EL;
              if constexpr (EL == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
              else *reinterpret_cast<uint32_t*>(at) = w[0];
            }
      };
      if (finite) store(std::true_type());
      else store(std::false_type());
      if (lane == 0) *sc = s;
    }
    if (!MANY || rows.t0 + (int64_t)gridDim.x * C8_ROWS >= ar.N) break;
    find_more_rows<true>(ar, &rows);
  }
  if (bad && ar.status) atomicOr(ar.status, kStatusClamped);
}

template <int D, typename T, bool MANY>
__global__ void __launch_bounds__(C8_NT) k_cache_read8(Cache8Args ar) {
  constexpr int CH = D / 16;  // 16-byte loads of a head's row
  __shared__ Rows rows;
  __shared__ int64_t at[C8_ROWS];  // cache rows
  after_previous();
  before_next();
  int bad = 0;
  find_first_rows<false>(ar, &rows, &bad);
  while (true) {
    if (threadIdx.x < C8_ROWS) {
      int64_t r = -2;  // no token
      if (rows.end[threadIdx.x] > 0) {
        r = cache_row(ar, rows.b[threadIdx.x], rows.pos[threadIdx.x]);
        if (r < 0) bad = 1;
      }
      at[threadIdx.x] = r;
    }
    __syncthreads();
    const int per = ar.Hk * CH, all = C8_ROWS * per * 2;
#pragma unroll 4
    for (int i = blockIdx.y * C8_NT + threadIdx.x; i < all; i += gridDim.y * C8_NT) {
      const int slot = i / (2 * per), j = i % (2 * per);
      const bool isv = j >= per;
      const int c = isv ? j - per : j;
      const int64_t r = at[slot];
      if (r == -2) continue;
      T* out = reinterpret_cast<T*>(isv ? ar.vo : ar.ko) +
               ((rows.t0 + slot) * per + c) * 16;
      uint4 v = make_uint4(0, 0, 0, 0);
      float s = 0.f;
      if (r >= 0) {
        v = *reinterpret_cast<const uint4*>((isv ? ar.vc : ar.kc) + (r * per + c) * 16);
        s = (isv ? ar.vsc : ar.ksc)[(r / C8_BLOCK) * ar.Hk + c / CH];
      }
      float x[16];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 a = values2(word(v, w) & 0xffffu), b = values2(word(v, w) >> 16);
        x[4 * w] = a.x * s;
        x[4 * w + 1] = a.y * s;
        x[4 * w + 2] = b.x * s;
        x[4 * w + 3] = b.y * s;
      }
      if constexpr (sizeof(T) == 2) {
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 z = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
          y[e] = *reinterpret_cast<const uint32_t*>(&z);
        }
        reinterpret_cast<uint4*>(out)[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4*>(out)[1] = make_uint4(y[4], y[5], y[6], y[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          reinterpret_cast<float4*>(out)[e] =
              make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
      }
    }
    if (!MANY || rows.t0 + (int64_t)gridDim.x * C8_ROWS >= ar.N) break;
    find_more_rows<false>(ar, &rows);
  }
  if (bad && ar.status) atomicOr(ar.status, kStatusClamped);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool ok16(const void* p, int64_t n) { return n == 0 || (p && aligned16(p)); }
bool ok4(const void* p, int64_t n) { return n == 0 || (p && ((uintptr_t)p & 3u) == 0); }

gdn_status check(const gdn_cache8_problem* p, const void* k, const void* v, const void* kc,
                 const void* vc, const float* ks, const float* vs, const int32_t* table,
                 const int32_t* cu, const int32_t* status) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (p->B < 0 || p->N < 0 || p->Hk < 1 || p->pages < 0 || p->max_blocks < 0 ||
      p->page_size < 1 || p->D < 1)
    return GDN_ERR_INVALID_ARG;
  if (p->Hk > 0x7fffffff / 1024) return GDN_ERR_UNSUPPORTED;
  const int64_t unit = p->dtype == GDN_BF16 ? 8 : 4, row = p->Hk * p->D;
  for (int64_t s : {p->k_stride, p->v_stride})
    if (s != 0 && (s < row || s % unit != 0)) return GDN_ERR_INVALID_ARG;
  if ((p->D != 64 && p->D != 128 && p->D != 256) || p->page_size % C8_BLOCK != 0)
    return GDN_ERR_UNSUPPORTED;
  constexpr int64_t top = 0x7fffffff;
  if (p->pages > top / p->page_size || p->max_blocks > top / p->page_size ||
      p->N > top / p->Hk || p->B > (1 << 20))
    return GDN_ERR_UNSUPPORTED;
  const int64_t cached = p->pages;
  if (!ok16(k, p->N) || !ok16(v, p->N) || !ok16(kc, cached) || !ok16(vc, cached) ||
      !ok16(ks, cached) || !ok16(vs, cached) || !ok4(table, p->B * p->max_blocks) ||
      !ok4(cu, 1) || ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

template <template <int, typename, bool> class K>
cudaError_t run(const gdn_cache8_problem* p, const Cache8Args& ar, int items, cudaStream_t st) {
  // CTAs along the rows; with very many requests so few that all of them reading all offsets costs
  // little, each for several runs of rows (100,000 requests of a token, one head of 64: written 194 us
  // without that limit and 160 with it, read back 113 and 80; 1,048,576: 1760 and 955 with it).
  int64_t x = (p->N + C8_ROWS - 1) / C8_ROWS;
  const bool many = p->B > C8_MANY && x > C8_CTAS;
  if (many) x = C8_CTAS;
  // few rows (a decode step): the heads of a CTA's rows go to several
  int64_t y = x >= 304 ? 1 : (304 + x - 1) / x;
  if (y > items) y = items;
  const dim3 grid((unsigned)x, (unsigned)(y < 1 ? 1 : y));
  auto go = [&](auto d, auto t) {
    return many ? launch_behind(K<d(), decltype(t), true>::fn(), grid, C8_NT, 0, st, ar)
                : launch_behind(K<d(), decltype(t), false>::fn(), grid, C8_NT, 0, st, ar);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  using D256 = std::integral_constant<int, 256>;
  if (p->dtype == GDN_BF16) {
    const __nv_bfloat16 t{};
    return p->D == 64 ? go(D64(), t) : p->D == 128 ? go(D128(), t) : go(D256(), t);
  }
  return p->D == 64 ? go(D64(), 0.f) : p->D == 128 ? go(D128(), 0.f) : go(D256(), 0.f);
}
template <int D, typename T, bool MANY> struct Write {
  static auto fn() { return k_cache_write8<D, T, MANY>; }
};
template <int D, typename T, bool MANY> struct Read {
  static auto fn() { return k_cache_read8<D, T, MANY>; }
};

Cache8Args args(const gdn_cache8_problem* p, const int32_t* table, const int32_t* cu,
                int32_t* status) {
  Cache8Args ar;
  memset(&ar, 0, sizeof(ar));
  ar.N = p->N;
  ar.B = p->B;
  ar.pages = p->pages;
  ar.max_blocks = p->max_blocks;
  ar.P = p->page_size;
  ar.Hk = (int)p->Hk;
  ar.ks = p->k_stride ? p->k_stride : p->Hk * p->D;
  ar.vs = p->v_stride ? p->v_stride : p->Hk * p->D;
  ar.table = table;
  ar.cu = cu;
  ar.status = status;
  return ar;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_cache_write8(const gdn_cache8_problem* p, const void* k, const void* v,
                            const int32_t* block_table, const int32_t* ctx_len,
                            const int32_t* cu_seqlens, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, int32_t* status, void* stream) {
  const gdn_status s = check(p, k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                             status);
  if (s != GDN_OK) return s;
  if (!ok4(ctx_len, p->B)) return GDN_ERR_INVALID_ARG;
  if (p->N == 0 || p->B == 0) return GDN_OK;
  Cache8Args ar = args(p, block_table, cu_seqlens, status);
  ar.k = k;
  ar.v = v;
  ar.kc = (uint8_t*)k_cache;
  ar.vc = (uint8_t*)v_cache;
  ar.ksc = k_scale;
  ar.vsc = v_scale;
  ar.ctx = ctx_len;
  // a warp per block and head, of which 16 rows have 16 at most
  const int items = (int)((2 * p->Hk * C8_ROWS + C8_W - 1) / C8_W);
  const cudaError_t e = run<Write>(p, ar, items, (cudaStream_t)stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_cache_read8(const gdn_cache8_problem* p, const void* k_cache, const void* v_cache,
                           const float* k_scale, const float* v_scale,
                           const int32_t* block_table, const int32_t* cu_seqlens, void* k,
                           void* v, int32_t* status, void* stream) {
  const gdn_status s = check(p, k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                             status);
  if (s != GDN_OK) return s;
  if (p->N == 0 || p->B == 0) return GDN_OK;
  Cache8Args ar = args(p, block_table, cu_seqlens, status);
  ar.ko = k;
  ar.vo = v;
  ar.kc = (uint8_t*)const_cast<void*>(k_cache);
  ar.vc = (uint8_t*)const_cast<void*>(v_cache);
  ar.ksc = const_cast<float*>(k_scale);
  ar.vsc = const_cast<float*>(v_scale);
  const int items = (int)((2 * p->Hk * (p->D / 16) * C8_ROWS + C8_NT - 1) / C8_NT);
  const cudaError_t e = run<Read>(p, ar, items, (cudaStream_t)stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
