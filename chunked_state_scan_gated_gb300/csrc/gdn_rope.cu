// gdn_rope.cu -- RMSNorm of every query and key head with the position rotation.  Per head row
// x of D elements at position t, r = 1 / sqrt(mean(x^2) + eps), n = x r w, and for i < R/2 with
// c = rope_scale cos(t inv_freq[i]), s = rope_scale sin(t inv_freq[i]):
//   y1 = n1 c - n2 s,  y2 = n2 c + n1 s      on the pairs (i, i + R/2) or (2i, 2i + 1)
// Backward: dn1 = dy1 c + dy2 s, dn2 = dy2 c - dy1 s (the transposed rotation), g = dn w,
//   dx = r (g - x r mean(g x r)),  dw = sum over rows of dn x r.
// The angle is formed in revolutions: t * (inv_freq / 2 pi) as an exact two-term product, its
// integer part dropped, so positions past 2^20 lose nothing (angle()).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using namespace vec;

constexpr int RO_NT = 256;     // 8 warps
constexpr int RO_BCTAS = 608;  // CTAs of the backward at most (4 per SM of a 152-SM GPU)
constexpr int RO_MAXD = 256;   // 8 elements per lane

struct RopeArgs {
  int64_t N, T, qs, ks, vs, n_slots;
  int Hq, Hk, D, R, inter;
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ void ld8(const T* p, float (&v)[8]) {
  float a[4], b[4];
  ld4(p, a);
  ld4(p + 4, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[j + 4] = b[j];
  }
}
template <typename T>
__device__ __forceinline__ void st8(T* p, const float (&v)[8]) {
  float a[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a[j] = v[j];
    b[j] = v[j + 4];
  }
  st4(p, a);
  st4(p + 4, b);
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

// The rotation of a row held 8 elements per lane (element 8 lane + j); sgn = -1 transposes.
__device__ __forceinline__ void rotate(const RopeArgs& ar, int32_t t, float sgn, float (&n)[8]) {
  const int lane = threadIdx.x & 31, e = lane * 8;
  if (ar.inter) {
    if (e < ar.R)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float c, s;
        angle(t, ar.inv_freq[e / 2 + j], &c, &s);
        c *= ar.rscale;
        s *= sgn * ar.rscale;
        const float a = n[2 * j], b = n[2 * j + 1];
        n[2 * j] = a * c - b * s;
        n[2 * j + 1] = b * c + a * s;
      }
    return;
  }
  const int half = ar.R / 16;  // lanes per half
  const bool first = lane < half;
  const int other = first ? lane + half : lane - half;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = __shfl_sync(0xffffffffu, n[j], other & 31);
    if (e < ar.R) {
      float c, s;
      angle(t, ar.inv_freq[(first ? e : e - ar.R / 2) + j], &c, &s);
      c *= ar.rscale;
      s *= sgn * ar.rscale;
      n[j] = first ? n[j] * c - m * s : n[j] * c + m * s;
    }
  }
}

// Mode 0: outputs; mode 1: k and v rows into the caches
template <int Mode, typename T>
__global__ void __launch_bounds__(RO_NT) k_qk_norm_rope_fwd(RopeArgs ar) {
  const int lane = threadIdx.x & 31, e = lane * 8;
  const int H = ar.Hq + ar.Hk;
  const int64_t row = (int64_t)blockIdx.x * (RO_NT / 32) + (threadIdx.x >> 5);
  if (row >= ar.N * H) return;
  const int64_t n = row / H;
  const int h = (int)(row % H);
  const bool isq = h < ar.Hq, in = e < ar.D;
  const int hk = h - ar.Hq;
  int64_t dst = n;
  if (Mode == 1 && !isq) {
    dst = ar.slots[n];
    if (dst < 0 || dst >= ar.n_slots) {
      if (dst != -1 && lane == 0 && hk == 0 && ar.status) atomicOr(ar.status, kStatusClamped);
      return;
    }
  }
  const T* x = isq ? reinterpret_cast<const T*>(ar.q) + n * ar.qs + (int64_t)h * ar.D
                   : reinterpret_cast<const T*>(ar.k) + n * ar.ks + (int64_t)hk * ar.D;
  float v[8] = {}, w[8] = {};
  if (in) {
    ld8(x + e, v);
    ld8((isq ? ar.wq : ar.wk) + e, w);
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
  const float r = rsqrtf(warp_sum(ss) / (float)ar.D + ar.eps);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= r * w[j];
  rotate(ar, ar.pos ? ar.pos[n] : (int32_t)(n % ar.T), 1.f, v);
  T* y = isq ? reinterpret_cast<T*>(ar.q_out) + (n * ar.Hq + h) * ar.D
             : reinterpret_cast<T*>(ar.k_out) + (dst * ar.Hk + hk) * ar.D;
  if (in) st8(y + e, v);
  if (Mode == 1 && !isq && in) {
    ld8(reinterpret_cast<const T*>(ar.v) + n * ar.vs + (int64_t)hk * ar.D + e, v);
    st8(reinterpret_cast<T*>(ar.v_out) + (dst * ar.Hk + hk) * ar.D + e, v);
  }
}

template <typename T>
__global__ void __launch_bounds__(RO_NT) k_qk_norm_rope_bwd(RopeArgs ar) {
  __shared__ float red[RO_NT / 32][RO_MAXD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = lane * 8;
  const int H = ar.Hq + ar.Hk;
  const bool in = e < ar.D;
  float dw[2][8] = {}, wq[8] = {}, wk[8] = {};
  if (in) {
    if (ar.Hq) ld8(ar.wq + e, wq);
    if (ar.Hk) ld8(ar.wk + e, wk);
  }
  for (int64_t row = (int64_t)blockIdx.x * (RO_NT / 32) + warp; row < ar.N * H;
       row += (int64_t)gridDim.x * (RO_NT / 32)) {
    const int64_t n = row / H;
    const int h = (int)(row % H);
    const bool isq = h < ar.Hq;
    const int hk = h - ar.Hq;
    const int64_t src = isq ? n * ar.qs + (int64_t)h * ar.D : n * ar.ks + (int64_t)hk * ar.D;
    const int64_t out = isq ? (n * ar.Hq + h) * ar.D : (n * ar.Hk + hk) * ar.D;
    float x[8] = {}, g[8] = {};
    if (in) {
      ld8(reinterpret_cast<const T*>(isq ? ar.q : ar.k) + src + e, x);
      ld8(reinterpret_cast<const T*>(isq ? ar.dq_out : ar.dk_out) + out + e, g);
    }
    rotate(ar, ar.pos ? ar.pos[n] : (int32_t)(n % ar.T), -1.f, g);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    const float r = rsqrtf(warp_sum(ss) / (float)ar.D + ar.eps);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] *= r;
      const float d = g[j] * x[j];
      if (isq) dw[0][j] += d; else dw[1][j] += d;
      g[j] *= isq ? wq[j] : wk[j];
      dot = fmaf(g[j], x[j], dot);
    }
    const float m = warp_sum(dot) / (float)ar.D;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = r * (g[j] - x[j] * m);
    if (in) st8(reinterpret_cast<T*>(isq ? ar.q_out : ar.k_out) + out + e, g);
  }
  for (int z = 0; z < 2; ++z) {  // this CTA's dwq, dwk: its 8 warps added in order
    __syncthreads();
    if (in)
#pragma unroll
      for (int j = 0; j < 8; ++j) red[warp][e + j] = dw[z][j];
    __syncthreads();
    for (int c = threadIdx.x; c < ar.D; c += RO_NT) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < RO_NT / 32; ++w) s += red[w][c];
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

int64_t bwd_ctas(const RopeArgs& ar) {
  const int64_t n = (ar.N * (ar.Hq + ar.Hk) + RO_NT / 32 - 1) / (RO_NT / 32);
  return n < RO_BCTAS ? n : RO_BCTAS;
}

template <int Mode>
gdn_status launch_fwd(const RopeArgs& ar, int dtype, cudaStream_t st) {
  const int64_t rows = ar.N * (ar.Hq + ar.Hk);
  const unsigned ctas = (unsigned)((rows + RO_NT / 32 - 1) / (RO_NT / 32));
  if (dtype == GDN_BF16)
    k_qk_norm_rope_fwd<Mode, __nv_bfloat16><<<ctas, RO_NT, 0, st>>>(ar);
  else
    k_qk_norm_rope_fwd<Mode, float><<<ctas, RO_NT, 0, st>>>(ar);
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
  return launch_fwd<0>(ar, p->dtype, (cudaStream_t)stream);
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
  return launch_fwd<1>(ar, p->dtype, (cudaStream_t)stream);
}

gdn_status gdn_qk_norm_rope_bwd_workspace_size(const gdn_rope_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  RopeArgs ar;
  gdn_status s = check_problem(p, &ar);
  if (s != GDN_OK) return s;
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
    if (p->dtype == GDN_BF16)
      k_qk_norm_rope_bwd<__nv_bfloat16><<<(unsigned)ctas, RO_NT, 0, st>>>(ar);
    else
      k_qk_norm_rope_bwd<float><<<(unsigned)ctas, RO_NT, 0, st>>>(ar);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  k_qk_norm_rope_dw<<<(unsigned)((2 * ar.D + 31) / 32), RO_NT, 0, st>>>(
      (int)ctas, ar.D, (const float*)workspace, ar.Hq ? dwq : nullptr, ar.Hk ? dwk : nullptr);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
