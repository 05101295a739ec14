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
  float eps, rscale;
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

// A row's 8 elements of one lane, as loaded.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
__device__ __forceinline__ void put(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  uint32_t* w = &u.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&x);
  }
  *reinterpret_cast<uint4*>(p) = u;
}

// sum over the LPR lanes of a row
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of the token's angles into the warp's cs[0 .. R/2) and cs[128 ..)
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

// The rotation of a row held 8 elements per lane (element 8 l + j, l the lane in the row);
// sgn = -1 transposes.
template <int LPR>
__device__ __forceinline__ void rotate(const RopeArgs& ar, const float* cs, float sgn,
                                       float (&n)[8]) {
  const int l = threadIdx.x & (LPR - 1), e = l * 8;
  if (ar.inter) {
    if (e < ar.R) {
      const float4 c = *reinterpret_cast<const float4*>(cs + e / 2);
      const float4 s = *reinterpret_cast<const float4*>(cs + RO_MAXD / 2 + e / 2);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = n[2 * j], b = n[2 * j + 1], sj = sgn * ss[j];
        n[2 * j] = a * cc[j] - b * sj;
        n[2 * j + 1] = b * cc[j] + a * sj;
      }
    }
    return;
  }
  const int half = ar.R / 16;  // lanes per half
  const bool first = l < half;
  const int other = first ? l + half : l - half;
  const float sg = first ? -sgn : sgn;
  const float* at = cs + (first ? e : e - ar.R / 2);
  const bool in = e < ar.R;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      c = *reinterpret_cast<const float4*>(at + 4 * z);
      s = *reinterpret_cast<const float4*>(at + RO_MAXD / 2 + 4 * z);
    }
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float m = __shfl_sync(0xffffffffu, n[4 * z + j], other, LPR);
      if (in) n[4 * z + j] = n[4 * z + j] * cc[j] + m * (sg * ss[j]);
    }
  }
}

// One head row: its input, output and kind.
struct Row {
  int kind;  // 0 query, 1 key, 2 value (cache form), -1 none
  int h;     // head of its kind
};
__device__ __forceinline__ Row row_of(const RopeArgs& ar, int h, int end) {
  if (h >= end) return Row{-1, 0};
  if (h < ar.Hq) return Row{0, h};
  if (h < ar.Hq + ar.Hk) return Row{1, h - ar.Hq};
  return Row{2, h - ar.Hq - ar.Hk};
}

// CACHE: k and v rows go to the caches
template <bool CACHE, int LPR, typename T>
__global__ void __launch_bounds__(RO_NT) k_qk_norm_rope_fwd(RopeArgs ar) {
  __shared__ __align__(16) float s_cs[RO_W][RO_MAXD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
  const int e = (lane & (LPR - 1)) * 8;
  constexpr int RPL = 32 / LPR;
  const int64_t task = (int64_t)blockIdx.x * RO_W + warp;
  if (task >= ar.N * ar.chunks) return;
  const int64_t n = task / ar.chunks;
  const int h0 = (int)(task % ar.chunks) * ar.chunk;
  const int end = min(h0 + ar.chunk, ar.heads);
  const bool in = e < ar.D;
  int64_t dst = n;
  if (CACHE) {
    dst = ar.slots[n];
    if (dst < 0 || dst >= ar.n_slots) {
      if (dst != -1 && lane == 0 && h0 == 0 && ar.status) atomicOr(ar.status, kStatusClamped);
      dst = -1;
    }
  }
  const T* src[3] = {reinterpret_cast<const T*>(ar.q) + n * ar.qs + e,
                     reinterpret_cast<const T*>(ar.k) + n * ar.ks + e,
                     reinterpret_cast<const T*>(ar.v) + n * ar.vs + e};
  bool have = false;
  for (int hb = h0; hb < end; hb += RO_UNR * RPL) {
    Raw<T> raw[RO_UNR];
#pragma unroll
    for (int u = 0; u < RO_UNR; ++u) {
      const Row r = row_of(ar, hb + u * RPL + sub, end);
      raw[u].zero();
      if (r.kind >= 0 && in)
        raw[u].load((r.kind == 0 ? src[0] : r.kind == 1 ? src[1] : src[2]) + (int64_t)r.h * ar.D);
    }
    if (!have) angles(ar, n, s_cs[warp]);  // under the first loads
    have = true;
#pragma unroll
    for (int u = 0; u < RO_UNR; ++u) {
      if (hb + u * RPL >= end) break;
      const Row r = row_of(ar, hb + u * RPL + sub, end);
      float v[8], w[8] = {};
      raw[u].get(v);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
      const float f = rsqrtf(row_sum<LPR>(ss) / (float)ar.D + ar.eps);
      if (in && r.kind >= 0 && r.kind < 2) ld8((r.kind == 0 ? ar.wq : ar.wk) + e, w);
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[j] * (f * w[j]);
      rotate<LPR>(ar, s_cs[warp], 1.f, y);
      if (r.kind < 0 || !in || (CACHE && r.kind > 0 && dst < 0)) continue;
      const int64_t at = (r.kind == 0 ? n * ar.Hq : dst * ar.Hk) + r.h;
      T* out = reinterpret_cast<T*>(r.kind == 0 ? ar.q_out : r.kind == 1 ? ar.k_out : ar.v_out);
      if (CACHE && r.kind == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[j];
      }
      put(out + at * ar.D + e, y);
    }
  }
}

// Persistent: a warp takes tasks in a fixed stride and keeps its lanes' dwq, dwk in registers.
template <int LPR, typename T>
__global__ void __launch_bounds__(RO_NT, 2) k_qk_norm_rope_bwd(RopeArgs ar) {
  __shared__ __align__(16) float s_cs[RO_W][RO_MAXD];
  __shared__ float red[RO_W][RO_MAXD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
  const int e = (lane & (LPR - 1)) * 8;
  constexpr int RPL = 32 / LPR, UNR = sizeof(T) == 2 ? RO_UNR : RO_UNR / 2;
  const bool in = e < ar.D;
  float dw[2][8] = {};
  for (int64_t task = (int64_t)blockIdx.x * RO_W + warp; task < ar.N * ar.chunks;
       task += (int64_t)gridDim.x * RO_W) {
    const int64_t n = task / ar.chunks;
    const int h0 = (int)(task % ar.chunks) * ar.chunk;
    const int end = min(h0 + ar.chunk, ar.heads);
    bool have = false;
    for (int hb = h0; hb < end; hb += UNR * RPL) {
      Raw<T> rx[UNR], rg[UNR];
#pragma unroll
      for (int u = 0; u < UNR; ++u) {
        const Row r = row_of(ar, hb + u * RPL + sub, end);
        rx[u].zero();
        rg[u].zero();
        if (r.kind >= 0 && in) {
          const bool isq = r.kind == 0;
          const int64_t hd = (int64_t)r.h * ar.D + e;
          rx[u].load(reinterpret_cast<const T*>(isq ? ar.q : ar.k) + n * (isq ? ar.qs : ar.ks) +
                     hd);
          rg[u].load(reinterpret_cast<const T*>(isq ? ar.dq_out : ar.dk_out) +
                     n * (isq ? ar.Hq : ar.Hk) * ar.D + hd);
        }
      }
      if (!have) angles(ar, n, s_cs[warp]);
      have = true;
#pragma unroll
      for (int u = 0; u < UNR; ++u) {
        if (hb + u * RPL >= end) break;
        const Row r = row_of(ar, hb + u * RPL + sub, end);
        const bool isq = r.kind == 0;
        float x[8], g[8], w[8] = {};
        rx[u].get(x);
        rg[u].get(g);
        rotate<LPR>(ar, s_cs[warp], -1.f, g);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        const float f = rsqrtf(row_sum<LPR>(ss) / (float)ar.D + ar.eps);
        if (in && r.kind >= 0) ld8((isq ? ar.wq : ar.wk) + e, w);
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] *= f;
          const float d = g[j] * x[j];
          dw[0][j] += isq ? d : 0.f;
          dw[1][j] += isq ? 0.f : d;  // absent rows hold zeros
          g[j] *= w[j];
          dot = fmaf(g[j], x[j], dot);
        }
        const float m = row_sum<LPR>(dot) / (float)ar.D;
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = f * (g[j] - x[j] * m);
        if (r.kind >= 0 && in)
          put(reinterpret_cast<T*>(isq ? ar.q_out : ar.k_out) +
                  (n * (isq ? ar.Hq : ar.Hk) + r.h) * ar.D + e,
              g);
      }
    }
  }
  for (int z = 0; z < 2; ++z) {  // this CTA's dwq, dwk: lanes of equal elements, then warps in order
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) dw[z][j] += __shfl_xor_sync(0xffffffffu, dw[z][j], o);
    __syncthreads();
    if (in && sub == 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) red[warp][e + j] = dw[z][j];
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

template <bool CACHE, typename T>
void launch_fwd_t(const RopeArgs& ar, cudaStream_t st) {
  const unsigned ctas = (unsigned)((ar.N * ar.chunks + RO_W - 1) / RO_W);
  if (ar.D <= 64) k_qk_norm_rope_fwd<CACHE, 8, T><<<ctas, RO_NT, 0, st>>>(ar);
  else if (ar.D <= 128) k_qk_norm_rope_fwd<CACHE, 16, T><<<ctas, RO_NT, 0, st>>>(ar);
  else k_qk_norm_rope_fwd<CACHE, 32, T><<<ctas, RO_NT, 0, st>>>(ar);
}
template <bool CACHE>
gdn_status launch_fwd(const RopeArgs& ar, int dtype, cudaStream_t st) {
  if (dtype == GDN_BF16) launch_fwd_t<CACHE, __nv_bfloat16>(ar, st);
  else launch_fwd_t<CACHE, float>(ar, st);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
template <typename T>
void launch_bwd(const RopeArgs& ar, unsigned ctas, cudaStream_t st) {
  if (ar.D <= 64) k_qk_norm_rope_bwd<8, T><<<ctas, RO_NT, 0, st>>>(ar);
  else if (ar.D <= 128) k_qk_norm_rope_bwd<16, T><<<ctas, RO_NT, 0, st>>>(ar);
  else k_qk_norm_rope_bwd<32, T><<<ctas, RO_NT, 0, st>>>(ar);
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
    if (p->dtype == GDN_BF16) launch_bwd<__nv_bfloat16>(ar, (unsigned)ctas, st);
    else launch_bwd<float>(ar, (unsigned)ctas, st);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  k_qk_norm_rope_dw<<<(unsigned)((2 * ar.D + 31) / 32), RO_NT, 0, st>>>(
      (int)ctas, ar.D, (const float*)workspace, ar.Hq ? dwq : nullptr, ar.Hk ? dwk : nullptr);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
