// gdn_step.cu -- the core for one token per row over a pool of states (serving).  Per row and
// V head, with the row's state S [dk,dv] and the normalised q, k of gdn_fwd:
//   S' = alpha (S - beta k (S^T k)^T) + beta k v^T,   o = S'^T q
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int ST_NT = 128;  // one thread per state column

struct StepArgs {
  int64_t B, Ts, Hqk, H, r, n_slots;
  int dk, dv, l2norm;
  float eps, scale;
  const int32_t* slots;
  const void *q, *k, *v, *a, *b;
  const float *A_log, *dt_bias;
  float* state;
  void* o;
  int32_t* status;
};

__device__ __forceinline__ float ldf(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void stf(float* p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, int64_t i, float x) {
  p[i] = __float2bfloat16_rn(x);
}

__device__ __forceinline__ float block_sum(float x, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < ST_NT / 32; ++w) s += red[w];
  __syncthreads();
  return s;
}

// The state of row b, or -1 (uniform over the CTA): its slot when that is in range and no
// earlier row has it.
__device__ __forceinline__ int64_t row_slot(const StepArgs& ar, int64_t b, bool lead) {
  if (!ar.slots) return b;
  const int32_t s = ar.slots[b];
  if (s == -1) return -1;
  bool bad = s < -1 || s >= ar.n_slots;
  int dup = 0;
  for (int64_t i = threadIdx.x; i < b; i += ST_NT) dup |= ar.slots[i] == s;
  bad = __syncthreads_or(dup) || bad;
  if (!bad) return s;
  if (lead && threadIdx.x == 0 && ar.status) atomicOr(ar.status, kStatusClamped);
  return -1;
}

template <typename T>
__global__ void __launch_bounds__(ST_NT) k_step(StepArgs ar) {
  __shared__ float qs[kMaxHeadDim], ks[kMaxHeadDim], red[ST_NT / 32];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / ar.H, h = blockIdx.x % ar.H, hq = h / ar.r;
  const int64_t row = b * ar.Ts;
  const int64_t slot = row_slot(ar, b, h == 0);
  T* o = reinterpret_cast<T*>(ar.o) + (row * ar.H + h) * ar.dv;
  if (slot < 0) {
    if (tid < ar.dv) stf(o, tid, 0.f);
    return;
  }
  const int64_t qk = (row * ar.Hqk + hq) * ar.dk;
  float q = 0.f, k = 0.f;
  if (tid < ar.dk) {
    q = ldf(reinterpret_cast<const T*>(ar.q), qk + tid);
    k = ldf(reinterpret_cast<const T*>(ar.k), qk + tid);
  }
  const float sq = block_sum(q * q, red), sk = block_sum(k * k, red);
  if (tid < ar.dk) {
    qs[tid] = q * (ar.l2norm ? ar.scale / sqrtf(sq + ar.eps) : ar.scale);
    ks[tid] = k * (ar.l2norm ? 1.f / sqrtf(sk + ar.eps) : 1.f);
  }
  __syncthreads();
  const float x = ldf(reinterpret_cast<const T*>(ar.a), row * ar.H + h) + ar.dt_bias[h];
  const float alpha = expf(-expf(ar.A_log[h]) * (x > 20.f ? x : log1pf(expf(x))));
  const float beta = 1.f / (1.f + expf(-ldf(reinterpret_cast<const T*>(ar.b), row * ar.H + h)));
  if (tid >= ar.dv) return;
  const float v = ldf(reinterpret_cast<const T*>(ar.v), (row * ar.H + h) * ar.dv + tid);
  float* S = ar.state + (slot * ar.H + h) * ar.dk * ar.dv + tid;
  float u = 0.f;
  for (int i = 0; i < ar.dk; ++i) u = fmaf(ks[i], S[(int64_t)i * ar.dv], u);
  const float w = beta * (v - alpha * u);  // the row added along k
  float acc = 0.f;
  for (int i = 0; i < ar.dk; ++i) {
    const float s = fmaf(ks[i], w, alpha * S[(int64_t)i * ar.dv]);
    S[(int64_t)i * ar.dv] = s;
    acc = fmaf(qs[i], s, acc);
  }
  stf(o, tid, acc);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool ok16(const void* p) { return p && aligned16(p); }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_step(const gdn_problem* p, int64_t n_slots, const int32_t* slots,
                               const void* q, const void* k, const void* v, const void* a,
                               const void* b, const float* A_log, const float* dt_bias,
                               float* state, void* o, int32_t* status, void* stream) {
  Prob pr;
  gdn_status s = resolve(p, &pr);
  if (s != GDN_OK) return s;
  if (pr.T != 1 || n_slots < 0) return GDN_ERR_INVALID_ARG;
  if (n_slots > 0x7fffffff || pr.B * pr.H > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
  if ((!slots && n_slots < pr.B) || ((uintptr_t)slots & 3u) != 0 ||
      ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  if (pr.B == 0) return GDN_OK;
  if (!ok16(q) || !ok16(k) || !ok16(v) || !ok16(a) || !ok16(b) || !ok16(A_log) ||
      !ok16(dt_bias) || !ok16(o) || (n_slots > 0 && !ok16(state)))
    return GDN_ERR_INVALID_ARG;
  StepArgs ar;
  memset(&ar, 0, sizeof(ar));
  ar.B = pr.B;
  ar.Ts = pr.Ts;
  ar.Hqk = pr.Hqk;
  ar.H = pr.H;
  ar.r = pr.r;
  ar.n_slots = n_slots;
  ar.dk = (int)pr.dk;
  ar.dv = (int)pr.dv;
  ar.l2norm = pr.l2norm;
  ar.eps = pr.eps;
  ar.scale = pr.scale;
  ar.slots = slots;
  ar.q = q;
  ar.k = k;
  ar.v = v;
  ar.a = a;
  ar.b = b;
  ar.A_log = A_log;
  ar.dt_bias = dt_bias;
  ar.state = state;
  ar.o = o;
  ar.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  const unsigned ctas = (unsigned)(pr.B * pr.H);
  if (pr.dtype == GDN_BF16)
    k_step<__nv_bfloat16><<<ctas, ST_NT, 0, st>>>(ar);
  else
    k_step<float><<<ctas, ST_NT, 0, st>>>(ar);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
