// gdn_rope.cu -- RMSNorm of every query and key head with the position rotation.  Per head row
// x of D elements at position t, r = 1 / sqrt(mean(x^2) + eps), n = x r w, and for i < R/2 with
// c = rope_scale cos(t inv_freq[i]), s = rope_scale sin(t inv_freq[i]):
//   y1 = n1 c - n2 s,  y2 = n2 c + n1 s      on the pairs (i, i + R/2) or (2i, 2i + 1)
// Backward: dn1 = dy1 c + dy2 s, dn2 = dy2 c - dy1 s (the transposed rotation), g = dn w,
//   dx = r (g - x r mean(g x r)),  dw = sum over rows of dn x r.
// The angle is formed in revolutions: t * (inv_freq / 2 pi) as an exact two-term product, its
// integer part dropped, so positions past 2^20 lose nothing (angle()).
//
// Bound by HBM (2 row accesses forward, 3 backward).  A warp takes one token and a run of its
// heads: the token's R/2 angles are computed once, into the warp's own shared memory (no CTA
// barrier), and serve all its heads.  A row is held 8 elements per lane (16 bytes of bf16) by
// LPR = 8, 16 or 32 lanes, so a warp holds 32 / LPR heads at a time, and the loads of RO_UNR such
// groups are issued together.  The halves of a rotated head meet through shuffles.  With many
// tokens a warp takes all heads of its token; with few (decode) as few as one group, which
// repeats the angles but spreads a token over many SMs.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using namespace vec;

constexpr int RO_NT = 256;     // 8 warps
constexpr int RO_W = RO_NT / 32;
constexpr int RO_UNR = 4;      // head groups whose loads are issued together
constexpr int RO_BCTAS = 304;  // CTAs of the backward at most (2 per SM of a 152-SM GPU)
constexpr int RO_MAXD = 256;   // 8 elements per lane
constexpr int RO_FILL = 152 * 16;  // warps that keep the GPU busy

struct RopeArgs {
  int64_t N, T, qs, ks, vs, n_slots;
  int Hq, Hk, D, R, inter;
  int heads, chunk, chunks;     // rows of a token, rows per warp (in heads), warps per token
  float eps, rscale, inv_d;
  const void *q, *k, *v;
  const float *wq, *wk, *inv_freq;
  const int32_t* pos;
  const int32_t* slots;
  void *q_out, *k_out, *v_out;  // forward: outputs or caches; backward: dq, dk
  const void *dq_out, *dk_out;
  float* part;                  // [CTAs][2][D] partial dwq, dwk
  int32_t* status;
};

__device__ __forceinline__ void ld8(const float* p, float (&v)[8]) {
  float a[4], b[4];
  ld4(p, a);
  ld4(p + 4, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[j + 4] = b[j];
  }
}
// cos and sin of t * f, t any int32, f fp32.  In revolutions u = t f / (2 pi), with
// 1/(2 pi) as the sum of two fp32 numbers: t is split into two parts that are exact in fp32
// and f / (2 pi) into hi + lo, the product with hi is exact as value and remainder of an
// fma, and only the fraction goes into sincospi.  What is left is the rounding of the
// fraction (2^-24 revolutions) and of lo (t f 2^-51 revolutions: 2^-22 at t = 2^29).
__device__ __forceinline__ void angle(int32_t t, float f, float* c, float* s) {
  constexpr float kHi = 0x1.45f306p-3f, kLo = 0x1.b9391p-28f;  // 1/(2 pi) = kHi + kLo
  const float hi = __fmul_rn(f, kHi);
  const float lo = fmaf(f, kHi, -hi) + f * kLo;
  const int32_t th = t & ~0xffff, tl = t & 0xffff;  // t = th + tl, both exact in fp32
  float u = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float x = (float)(k ? tl : th);
    const float p = __fmul_rn(x, hi);  // not contracted: its remainder is added below
    u += (p - rintf(p)) + fmaf(x, hi, -p) + x * lo;
  }
  u -= rintf(u);
  sincospif(2.f * u, s, c);
}

// Two fp32 numbers in a register pair: Blackwell's packed arithmetic halves the instructions.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 un(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// A row's 8 elements of one lane, as loaded; from(): the same of another lane of the row.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  template <int LPR> __device__ __forceinline__ Raw from(int lane) const {
    Raw r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = __shfl_sync(0xffffffffu, w[j], lane, LPR);
    return r;
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  }
};
template <> struct Raw<float> {
  float w[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
  }
  template <int LPR> __device__ __forceinline__ Raw from(int lane) const {
    Raw r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = __shfl_sync(0xffffffffu, w[j], lane, LPR);
    return r;
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = f2(w[2 * j], w[2 * j + 1]);
  }
};
__device__ __forceinline__ void put(float* p, const F2 (&v)[4]) {
  const float2 a = un(v[0]), b = un(v[1]), c = un(v[2]), d = un(v[3]);
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
  *(reinterpret_cast<float4*>(p) + 1) = make_float4(c.x, c.y, d.x, d.y);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const F2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = un(v[j]);
    const __nv_bfloat162 x = __floats2bfloat162_rn(a.x, a.y);
    w[j] = *reinterpret_cast<const uint32_t*>(&x);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// A row's partner elements: of the pair's other half (another lane), or of the neighbour.
template <bool INTER, int LPR, typename T>
__device__ __forceinline__ void partner(const Raw<T>& raw, const F2 (&x)[4], int other,
                                        F2 (&y)[4]) {
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = un(x[j]);
      y[j] = f2(a.y, a.x);
    }
  } else {
    raw.template from<LPR>(other).get(y);
  }
}

// sum over the LPR lanes of a row
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of the token's angles into the warp's cs[0 .. R/2) and cs[RO_MAXD / 2 ..)
__device__ __forceinline__ void angles(const RopeArgs& ar, int64_t n, float* cs) {
  const int lane = threadIdx.x & 31;
  const int32_t t = ar.pos ? ar.pos[n] : (int32_t)(n % ar.T);
  __syncwarp();  // the last token's readers are done
  for (int i = lane; i < ar.R / 2; i += 32) {
    float c, s;
    angle(t, ar.inv_freq[i], &c, &s);
    cs[i] = c * ar.rscale;
    cs[RO_MAXD / 2 + i] = s * ar.rscale;
  }
  __syncwarp();
}

// A lane's view of the rotation: y_j = x_j c_j + xp_j s_j with xp the partner elements and the
// sign of the pair's side in s (sgn = -1: the transposed rotation); c = 1, s = 0 past R.
template <bool INTER>
__device__ __forceinline__ void turn(const RopeArgs& ar, const float* cs, int e, float sgn,
                                     float (&c)[8], float (&s)[8]) {
  const bool in = e < ar.R, first = e < ar.R / 2;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = INTER ? (e + j) / 2 : first ? e + j : e + j - ar.R / 2;
    c[j] = in ? cs[i] : 1.f;
    const bool neg = INTER ? !(j & 1) : first;
    s[j] = in ? (neg ? -sgn : sgn) * cs[RO_MAXD / 2 + i] : 0.f;
  }
}
// The lane (of LPR) that holds the partner elements: its own past R (where they do not count).
__device__ __forceinline__ int other_lane(const RopeArgs& ar, int e) {
  if (e >= ar.R) return e / 8;
  return (e < ar.R / 2 ? e + ar.R / 2 : e - ar.R / 2) / 8;
}

// The heads of one kind (query, key) of a token: y = f (x (w c) + xp (w_p s)).
template <bool INTER, int LPR, typename T>
__device__ __forceinline__ void norm_heads(const RopeArgs& ar, const T* src, T* dst,
                                           const float* w, int h, int end, int64_t n, float* cs,
                                           bool* have, bool store) {
  constexpr int RPL = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR, e = (lane & (LPR - 1)) * 8;
  const bool in = e < ar.D;
  const int other = INTER ? 0 : other_lane(ar, e);
  src += (int64_t)(h + sub) * ar.D + e;
  dst += (int64_t)(h + sub) * ar.D + e;
  F2 A[4], Bq[4];
  bool first = true;
  for (; h < end; h += RO_UNR * RPL) {
    Raw<T> raw[RO_UNR];
#pragma unroll
    for (int u = 0; u < RO_UNR; ++u) {
      if (in && h + u * RPL + sub < end) raw[u].load(src + u * RPL * ar.D);
      else raw[u].zero();
    }
    if (first) {  // under the first loads
      if (!*have) angles(ar, n, cs);
      *have = true;
      first = false;
      float c[8], s[8], wv[8] = {}, wp[8] = {};
      turn<INTER>(ar, cs, e, 1.f, c, s);
      if (in) {
        ld8(w + e, wv);
        if constexpr (!INTER) ld8(w + other * 8, wp);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p0 = INTER ? wv[2 * j + 1] : wp[2 * j], p1 = INTER ? wv[2 * j] : wp[2 * j + 1];
        A[j] = f2(wv[2 * j] * c[2 * j], wv[2 * j + 1] * c[2 * j + 1]);
        Bq[j] = f2(p0 * s[2 * j], p1 * s[2 * j + 1]);
      }
    }
#pragma unroll
    for (int u = 0; u < RO_UNR; ++u) {
      if (h + u * RPL >= end) break;
      F2 x[4], y[4];
      raw[u].get(x);
      F2 ss = mul(x[0], x[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) ss = fma(x[j], x[j], ss);
      const float2 s2 = un(ss);
      const float f = rsqrtf(fmaf(row_sum<LPR>(s2.x + s2.y), ar.inv_d, ar.eps));
      partner<INTER, LPR>(raw[u], x, other, y);
      const F2 ff = f2(f, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul(fma(y[j], Bq[j], mul(x[j], A[j])), ff);
      if (store && in && h + u * RPL + sub < end) put(dst + u * RPL * ar.D, y);
    }
    src += RO_UNR * RPL * ar.D;
    dst += RO_UNR * RPL * ar.D;
  }
}

// CACHE: k and v rows go to the caches
template <bool CACHE, bool INTER, int LPR, typename T>
__global__ void __launch_bounds__(RO_NT) k_qk_norm_rope_fwd(RopeArgs ar) {
  __shared__ __align__(16) float s_cs[RO_W][RO_MAXD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t task = (int64_t)blockIdx.x * RO_W + warp;
  if (task >= ar.N * ar.chunks) return;
  const int64_t n = task / ar.chunks;
  const int h0 = (int)(task % ar.chunks) * ar.chunk, h1 = min(h0 + ar.chunk, ar.heads);
  int64_t dst = n;
  if (CACHE) {
    dst = ar.slots[n];
    if (dst < 0 || dst >= ar.n_slots) {
      if (dst != -1 && lane == 0 && h0 == 0 && ar.status) atomicOr(ar.status, kStatusClamped);
      dst = -1;
    }
  }
  bool have = false;
  if (h0 < ar.Hq)
    norm_heads<INTER, LPR>(ar, reinterpret_cast<const T*>(ar.q) + n * ar.qs,
                           reinterpret_cast<T*>(ar.q_out) + n * ar.Hq * ar.D, ar.wq, h0,
                           min(h1, ar.Hq), n, s_cs[warp], &have, true);
  const int k0 = max(h0 - ar.Hq, 0), k1 = min(h1 - ar.Hq, ar.Hk);
  if (k0 < k1 && dst >= 0)
    norm_heads<INTER, LPR>(ar, reinterpret_cast<const T*>(ar.k) + n * ar.ks,
                           reinterpret_cast<T*>(ar.k_out) + dst * ar.Hk * ar.D, ar.wk, k0, k1, n,
                           s_cs[warp], &have, true);
  if (CACHE && dst >= 0) {
    const int v0 = max(h0 - ar.Hq - ar.Hk, 0), v1 = h1 - ar.Hq - ar.Hk;
    constexpr int EL = 16 / (int)sizeof(T);
    const T* src = reinterpret_cast<const T*>(ar.v) + n * ar.vs;
    T* out = reinterpret_cast<T*>(ar.v_out) + dst * ar.Hk * ar.D;
    for (int i = v0 * ar.D + lane * EL; i < v1 * ar.D; i += 32 * EL)
      *reinterpret_cast<uint4*>(out + i) = *reinterpret_cast<const uint4*>(src + i);
  }
}

// The gradients of the heads of one kind of a token.  With dn the turned dy:
//   dx = f w dn - x f^3 sum(dn x w) / D,   dw += f dn x
template <bool INTER, int LPR, int UNR, typename T>
__device__ __forceinline__ void grad_heads(const RopeArgs& ar, const T* xs, const T* gs, T* dst,
                                           const float* w, int h, int end, int64_t n, float* cs,
                                           bool* have, F2 (&dw)[4]) {
  constexpr int RPL = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR, e = (lane & (LPR - 1)) * 8;
  const bool in = e < ar.D;
  const int other = INTER ? 0 : other_lane(ar, e);
  const int64_t at = (int64_t)(h + sub) * ar.D + e;
  xs += at;
  gs += at;
  dst += at;
  F2 C[4], S[4], W[4];
  bool first = true;
  for (; h < end; h += UNR * RPL) {
    Raw<T> rx[UNR], rg[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      if (in && h + u * RPL + sub < end) {
        rx[u].load(xs + u * RPL * ar.D);
        rg[u].load(gs + u * RPL * ar.D);
      } else {
        rx[u].zero();
        rg[u].zero();
      }
    }
    if (first) {
      if (!*have) angles(ar, n, cs);
      *have = true;
      first = false;
      float c[8], s[8], wv[8] = {};
      turn<INTER>(ar, cs, e, -1.f, c, s);
      if (in) ld8(w + e, wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        C[j] = f2(c[2 * j], c[2 * j + 1]);
        S[j] = f2(s[2 * j], s[2 * j + 1]);
        W[j] = f2(wv[2 * j], wv[2 * j + 1]);
      }
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      if (h + u * RPL >= end) break;
      F2 x[4], g[4], y[4];
      rx[u].get(x);
      rg[u].get(g);
      partner<INTER, LPR>(rg[u], g, other, y);
      F2 ss = mul(x[0], x[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) ss = fma(x[j], x[j], ss);
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = fma(y[j], S[j], mul(g[j], C[j]));  // dn
      F2 dot = f2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = mul(g[j], x[j]);
        g[j] = mul(g[j], W[j]);
        dot = fma(g[j], x[j], dot);
      }
      const float2 s2 = un(ss), d2 = un(dot);
      const float f = rsqrtf(fmaf(row_sum<LPR>(s2.x + s2.y), ar.inv_d, ar.eps));
      const float m = -(row_sum<LPR>(d2.x + d2.y) * ar.inv_d) * f * f * f;
      const F2 ff = f2(f, f), mm = f2(m, m);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dw[j] = fma(y[j], ff, dw[j]);  // absent rows hold zeros
        g[j] = fma(x[j], mm, mul(g[j], ff));
      }
      if (in && h + u * RPL + sub < end) put(dst + u * RPL * ar.D, g);
    }
    xs += UNR * RPL * ar.D;
    gs += UNR * RPL * ar.D;
    dst += UNR * RPL * ar.D;
  }
}

// Persistent: a warp takes tasks in a fixed stride and keeps its lanes' dwq, dwk in registers.
template <bool INTER, int LPR, typename T>
__global__ void __launch_bounds__(RO_NT, 2) k_qk_norm_rope_bwd(RopeArgs ar) {
  __shared__ __align__(16) float s_cs[RO_W][RO_MAXD];
  __shared__ float red[RO_W][RO_MAXD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
  const int e = (lane & (LPR - 1)) * 8;
  constexpr int UNR = sizeof(T) == 2 ? RO_UNR : RO_UNR / 2;
  F2 dw[2][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) dw[0][j] = dw[1][j] = f2(0.f, 0.f);
  for (int64_t task = (int64_t)blockIdx.x * RO_W + warp; task < ar.N * ar.chunks;
       task += (int64_t)gridDim.x * RO_W) {
    const int64_t n = task / ar.chunks;
    const int h0 = (int)(task % ar.chunks) * ar.chunk, h1 = min(h0 + ar.chunk, ar.heads);
    bool have = false;
    if (h0 < ar.Hq)
      grad_heads<INTER, LPR, UNR>(ar, reinterpret_cast<const T*>(ar.q) + n * ar.qs,
                                  reinterpret_cast<const T*>(ar.dq_out) + n * ar.Hq * ar.D,
                                  reinterpret_cast<T*>(ar.q_out) + n * ar.Hq * ar.D, ar.wq, h0,
                                  min(h1, ar.Hq), n, s_cs[warp], &have, dw[0]);
    const int k0 = max(h0 - ar.Hq, 0), k1 = h1 - ar.Hq;
    if (k0 < k1)
      grad_heads<INTER, LPR, UNR>(ar, reinterpret_cast<const T*>(ar.k) + n * ar.ks,
                                  reinterpret_cast<const T*>(ar.dk_out) + n * ar.Hk * ar.D,
                                  reinterpret_cast<T*>(ar.k_out) + n * ar.Hk * ar.D, ar.wk, k0,
                                  k1, n, s_cs[warp], &have, dw[1]);
  }
  for (int z = 0; z < 2; ++z) {  // this CTA's dwq, dwk: lanes of equal elements, then warps in order
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 d = un(z ? dw[1][j] : dw[0][j]);
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        d.x += __shfl_xor_sync(0xffffffffu, d.x, o);
        d.y += __shfl_xor_sync(0xffffffffu, d.y, o);
      }
      if (e < ar.D && sub == 0) {
        red[warp][e + 2 * j] = d.x;
        red[warp][e + 2 * j + 1] = d.y;
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < ar.D; c += RO_NT) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < RO_W; ++w) s += red[w][c];
      ar.part[((int64_t)blockIdx.x * 2 + z) * ar.D + c] = s;
    }
  }
}

// dwq, dwk = sums over the n_part CTA partials in fp64: 32 columns per CTA, warp w adds the
// partials w, w + 8, ... in order, then warp 0 adds the 8 warp sums in order.
__global__ void __launch_bounds__(RO_NT) k_qk_norm_rope_dw(int n_part, int D,
                                                           const float* __restrict__ part,
                                                           float* dwq, float* dwk) {
  __shared__ double acc[RO_NT / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (e < 2 * D)
    for (int p = warp; p < n_part; p += RO_NT / 32) s += part[(int64_t)p * 2 * D + e];
  acc[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && e < 2 * D) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < RO_NT / 32; ++w) t += acc[w][lane];
    float* out = e < D ? dwq : dwk;
    if (out) out[e < D ? e : e - D] = (float)t;
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool ok16(const void* p, int64_t n) { return n == 0 || (p && aligned16(p)); }
bool ok4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

gdn_status check_problem(const gdn_rope_problem* p, RopeArgs* ar) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (p->N < 0 || p->T < 0 || p->Hq < 0 || p->Hk < 0 || (p->Hq == 0 && p->Hk == 0) || p->D < 1 ||
      p->R < 0 || p->R > p->D || !(p->eps >= 0.f) || !isfinite(p->rope_scale))
    return GDN_ERR_INVALID_ARG;
  if (p->D % 8 != 0 || p->D > RO_MAXD || p->R % 16 != 0) return GDN_ERR_UNSUPPORTED;
  constexpr int64_t top = 0x7fffffff;
  if (p->Hq > top || p->Hk > top || p->N > top / (p->Hq + p->Hk)) return GDN_ERR_UNSUPPORTED;
  const int64_t unit = p->dtype == GDN_BF16 ? 8 : 4;  // elements in 16 bytes
  const int64_t heads[3] = {p->Hq, p->Hk, p->Hk};
  const int64_t given[3] = {p->q_stride, p->k_stride, p->v_stride};
  int64_t stride[3];
  for (int i = 0; i < 3; ++i) {
    stride[i] = given[i] ? given[i] : heads[i] * p->D;
    if (stride[i] < heads[i] * p->D || stride[i] % unit != 0) return GDN_ERR_INVALID_ARG;
  }
  memset(ar, 0, sizeof(*ar));
  ar->N = p->N;
  ar->T = p->T > 0 ? p->T : (p->N > 0 ? p->N : 1);
  ar->qs = stride[0];
  ar->ks = stride[1];
  ar->vs = stride[2];
  ar->Hq = (int)p->Hq;
  ar->Hk = (int)p->Hk;
  ar->D = p->D;
  ar->R = p->R;
  ar->inter = p->interleaved ? 1 : 0;
  ar->eps = p->eps;
  ar->inv_d = 1.f / (float)p->D;
  ar->rscale = p->rope_scale;
  return GDN_OK;
}

// The operands that every form has.
bool inputs_ok(const RopeArgs& ar, const void* q, const void* k, const float* wq,
               const float* wk, const float* inv_freq, const int32_t* pos) {
  return ok16(q, ar.N * ar.Hq) && ok16(k, ar.N * ar.Hk) && ok16(wq, ar.Hq) && ok16(wk, ar.Hk) &&
         ok16(inv_freq, ar.R) && ok4(pos);
}

// Splits the heads of a token over warps: all of them to one warp when the tokens alone fill
// the GPU, else runs of whole load groups.
void split_heads(RopeArgs* ar, int heads) {
  const int rpl = ar->D > 128 ? 1 : ar->D > 64 ? 2 : 4, group = rpl;
  ar->heads = heads;
  int64_t warps = ar->N > 0 ? (RO_FILL + ar->N - 1) / ar->N : 1;  // wanted per token
  const int64_t most = (heads + group - 1) / group;
  if (warps > most) warps = most;
  if (warps < 1) warps = 1;
  const int64_t chunk = (heads + warps - 1) / warps;
  ar->chunk = (int)((chunk + group - 1) / group * group);
  ar->chunks = (heads + ar->chunk - 1) / ar->chunk;
}

int64_t bwd_ctas(const RopeArgs& ar) {
  const int64_t n = (ar.N * ar.chunks + RO_W - 1) / RO_W;
  return n < RO_BCTAS ? n : RO_BCTAS;
}

// Runs f with the lanes per row, the pairing and the type as template arguments.
template <typename F>
void with_types(const RopeArgs& ar, int dtype, F f) {
  auto lanes = [&](auto inter, auto t) {
    if (ar.D <= 64) f(std::integral_constant<int, 8>(), inter, t);
    else if (ar.D <= 128) f(std::integral_constant<int, 16>(), inter, t);
    else f(std::integral_constant<int, 32>(), inter, t);
  };
  auto pairs = [&](auto t) {
    if (ar.inter) lanes(std::true_type(), t);
    else lanes(std::false_type(), t);
  };
  if (dtype == GDN_BF16) pairs(__nv_bfloat16());
  else pairs(0.f);
}

template <bool CACHE>
gdn_status launch_fwd(const RopeArgs& ar, int dtype, cudaStream_t st) {
  const unsigned ctas = (unsigned)((ar.N * ar.chunks + RO_W - 1) / RO_W);
  with_types(ar, dtype, [&](auto lpr, auto inter, auto t) {
    k_qk_norm_rope_fwd<CACHE, inter(), lpr(), decltype(t)><<<ctas, RO_NT, 0, st>>>(ar);
  });
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_qk_norm_rope_fwd(const gdn_rope_problem* p, const void* q, const void* k,
                                const float* wq, const float* wk, const float* inv_freq,
                                const int32_t* positions, void* q_out, void* k_out,
                                void* stream) {
  RopeArgs ar;
  gdn_status s = check_problem(p, &ar);
  if (s != GDN_OK) return s;
  if (p->N == 0) return GDN_OK;
  if (!inputs_ok(ar, q, k, wq, wk, inv_freq, positions) || !ok16(q_out, ar.Hq) ||
      !ok16(k_out, ar.Hk))
    return GDN_ERR_INVALID_ARG;
  ar.q = q;
  ar.k = k;
  ar.wq = wq;
  ar.wk = wk;
  ar.inv_freq = inv_freq;
  ar.pos = positions;
  ar.q_out = q_out;
  ar.k_out = k_out;
  split_heads(&ar, ar.Hq + ar.Hk);
  return launch_fwd<false>(ar, p->dtype, (cudaStream_t)stream);
}

gdn_status gdn_qk_norm_rope_cache(const gdn_rope_problem* p, const void* q, const void* k,
                                  const void* v, const float* wq, const float* wk,
                                  const float* inv_freq, const int32_t* positions,
                                  int64_t n_slots, const int32_t* slots, void* q_out,
                                  void* k_cache, void* v_cache, int32_t* status, void* stream) {
  RopeArgs ar;
  gdn_status s = check_problem(p, &ar);
  if (s != GDN_OK) return s;
  if (n_slots < 0) return GDN_ERR_INVALID_ARG;
  if (n_slots > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
  if (p->N == 0) return GDN_OK;
  if (!inputs_ok(ar, q, k, wq, wk, inv_freq, positions) || !ok16(v, ar.Hk) ||
      !ok16(q_out, ar.Hq) || !ok16(k_cache, n_slots * ar.Hk) || !ok16(v_cache, n_slots * ar.Hk) ||
      !slots || !ok4(slots) || ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  ar.q = q;
  ar.k = k;
  ar.v = v;
  ar.wq = wq;
  ar.wk = wk;
  ar.inv_freq = inv_freq;
  ar.pos = positions;
  ar.n_slots = n_slots;
  ar.slots = slots;
  ar.q_out = q_out;
  ar.k_out = k_cache;
  ar.v_out = v_cache;
  ar.status = status;
  split_heads(&ar, ar.Hq + 2 * ar.Hk);
  return launch_fwd<true>(ar, p->dtype, (cudaStream_t)stream);
}

gdn_status gdn_qk_norm_rope_bwd_workspace_size(const gdn_rope_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  RopeArgs ar;
  gdn_status s = check_problem(p, &ar);
  if (s != GDN_OK) return s;
  split_heads(&ar, ar.Hq + ar.Hk);
  *bytes = (size_t)bwd_ctas(ar) * 2 * (size_t)ar.D * sizeof(float);
  return GDN_OK;
}

gdn_status gdn_qk_norm_rope_bwd(const gdn_rope_problem* p, const void* q, const void* k,
                                const float* wq, const float* wk, const float* inv_freq,
                                const int32_t* positions, const void* dq_out,
                                const void* dk_out, void* dq, void* dk, float* dwq, float* dwk,
                                void* workspace, size_t workspace_bytes, void* stream) {
  RopeArgs ar;
  gdn_status s = check_problem(p, &ar);
  if (s != GDN_OK) return s;
  if (!inputs_ok(ar, q, k, wq, wk, inv_freq, positions) || !ok16(dq_out, ar.N * ar.Hq) ||
      !ok16(dk_out, ar.N * ar.Hk) || !ok16(dq, ar.N * ar.Hq) || !ok16(dk, ar.N * ar.Hk) ||
      !ok16(dwq, ar.Hq) || !ok16(dwk, ar.Hk))
    return GDN_ERR_INVALID_ARG;
  split_heads(&ar, ar.Hq + ar.Hk);
  const int64_t ctas = bwd_ctas(ar);
  const size_t need = (size_t)ctas * 2 * (size_t)ar.D * sizeof(float);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return GDN_ERR_WORKSPACE;
  ar.q = q;
  ar.k = k;
  ar.wq = wq;
  ar.wk = wk;
  ar.inv_freq = inv_freq;
  ar.pos = positions;
  ar.dq_out = dq_out;
  ar.dk_out = dk_out;
  ar.q_out = dq;
  ar.k_out = dk;
  ar.part = (float*)workspace;
  cudaStream_t st = (cudaStream_t)stream;
  if (ctas > 0) {
    with_types(ar, p->dtype, [&](auto lpr, auto inter, auto t) {
      k_qk_norm_rope_bwd<inter(), lpr(), decltype(t)><<<(unsigned)ctas, RO_NT, 0, st>>>(ar);
    });
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  k_qk_norm_rope_dw<<<(unsigned)((2 * ar.D + 31) / 32), RO_NT, 0, st>>>(
      (int)ctas, ar.D, (const float*)workspace, ar.Hq ? dwq : nullptr, ar.Hk ? dwk : nullptr);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
