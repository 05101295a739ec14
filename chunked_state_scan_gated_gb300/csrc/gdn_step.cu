// gdn_step.cu -- the core for one token per row over a pool of states (serving).  Per row and
// V head, with the row's state S [dk,dv] and the normalised q, k of gdn_fwd:
//   S' = alpha S + beta k (v - alpha u_k)^T,            u_k = S^T k
//   o  = S'^T q = alpha u_q + beta (k.q) (v - alpha u_k),  u_q = S^T q
// so that both sums over S come from one pass and S is read and written once.
//
// Bound by HBM: 8 dk dv bytes per row and head against 8 dk dv operations.  A CTA holds a slice of
// ST_COLS columns (128 bytes, a full line) of one state in registers: 8 lanes x 4 columns,
// 4 warps x 4 rows per access, dk / 16 accesses, all issued before anything waits.  The sums
// over the rows go through shuffles and shared memory once; then the slice is updated in place.
// Small slices keep the whole GPU busy from one row on (32 heads x 4 slices) and cost only
// the repeated q, k (from L2).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using namespace vec;

constexpr int ST_NT = 128;           // 4 warps
constexpr int ST_COLS = 32;          // state columns per CTA
constexpr int ST_LANES = ST_COLS / 4;
constexpr int ST_ROWS = ST_NT / ST_LANES;  // state rows per access
constexpr int ST_ACC = kMaxHeadDim / ST_ROWS;

struct StepArgs {
  int64_t B, Ts, Hqk, H, r, n_slots;
  int dk, dv, l2norm;
  unsigned slices;  // per state
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// FULL: dk = 128 and dv a multiple of ST_COLS (no bounds on the slice)
template <typename T, bool FULL>
__global__ void __launch_bounds__(ST_NT) k_step(StepArgs ar) {
  __shared__ float s_q[ST_NT / 32][kMaxHeadDim], s_k[ST_NT / 32][kMaxHeadDim];
  __shared__ float4 s_u[ST_NT / 32][2][ST_LANES];
  after_previous();
  before_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned head = blockIdx.x / ar.slices;  // row and V head
  const int64_t b = head / (unsigned)ar.H, h = head % (unsigned)ar.H;
  const int64_t row = b * ar.Ts;
  const int dk = FULL ? kMaxHeadDim : ar.dk;
  const int col = (int)(blockIdx.x % ar.slices) * ST_COLS + (lane % ST_LANES) * 4;
  const int i0 = warp * (32 / ST_LANES) + lane / ST_LANES;  // this thread's first state row
  const bool in = FULL || col < ar.dv;
  const int32_t slot = ar.slots ? ar.slots[b] : (int32_t)b;
  const bool here = slot >= 0 && slot < ar.n_slots;
  float4 S[ST_ACC];
  float* Sp = ar.state + ((here ? slot : 0) * ar.H + h) * dk * ar.dv + (int64_t)i0 * ar.dv + col;
#pragma unroll
  for (int i = 0; i < ST_ACC; ++i)
    if (here && in && (FULL || i * ST_ROWS < dk))
      S[i] = __ldcs(reinterpret_cast<const float4*>(Sp + (int64_t)i * ST_ROWS * ar.dv));
    else
      S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  // q, k of the head: 4 elements per lane, every warp its own copy
  const int64_t qk = (row * ar.Hqk + h / ar.r) * dk + lane * 4;
  float q[4] = {}, k[4] = {};
  if (FULL || lane * 4 < dk) {
    ld4(reinterpret_cast<const T*>(ar.q) + qk, q);
    ld4(reinterpret_cast<const T*>(ar.k) + qk, k);
  }
  const int64_t gate = row * ar.H + h, vo = gate * ar.dv + col;
  float v[4] = {};
  if (in) ld4(reinterpret_cast<const T*>(ar.v) + vo, v);
  const float x = ldf(reinterpret_cast<const T*>(ar.a), gate) + ar.dt_bias[h];
  const float bl = ldf(reinterpret_cast<const T*>(ar.b), gate), al = ar.A_log[h];
  // a slot that an earlier row has already is left to that row
  int taken = 0;
  if (ar.slots && here)
    for (int64_t i = tid; i < b; i += ST_NT) taken |= ar.slots[i] == slot;
  float qq = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    qq = fmaf(q[j], q[j], qq);
    kk = fmaf(k[j], k[j], kk);
    kq = fmaf(k[j], q[j], kq);
  }
  qq = warp_sum(qq);
  kk = warp_sum(kk);
  const float fq = ar.l2norm ? ar.scale / sqrtf(qq + ar.eps) : ar.scale;
  const float fk = ar.l2norm ? 1.f / sqrtf(kk + ar.eps) : 1.f;
  kq = warp_sum(kq) * fq * fk;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s_q[warp][lane * 4 + j] = q[j] * fq;
    s_k[warp][lane * 4 + j] = k[j] * fk;
  }
  __syncwarp();
  const float alpha = expf(-expf(al) * (x > 20.f ? x : log1pf(expf(x))));
  const float beta = 1.f / (1.f + expf(-bl));
  float uk[4] = {}, uq[4] = {};
#pragma unroll
  for (int i = 0; i < ST_ACC; ++i) {
    if (!FULL && i * ST_ROWS >= dk) break;
    const float kr = s_k[warp][i0 + i * ST_ROWS], qr = s_q[warp][i0 + i * ST_ROWS];
    uk[0] = fmaf(kr, S[i].x, uk[0]);
    uk[1] = fmaf(kr, S[i].y, uk[1]);
    uk[2] = fmaf(kr, S[i].z, uk[2]);
    uk[3] = fmaf(kr, S[i].w, uk[3]);
    uq[0] = fmaf(qr, S[i].x, uq[0]);
    uq[1] = fmaf(qr, S[i].y, uq[1]);
    uq[2] = fmaf(qr, S[i].z, uq[2]);
    uq[3] = fmaf(qr, S[i].w, uq[3]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int o = ST_LANES; o < 32; o <<= 1) {
      uk[j] += __shfl_xor_sync(0xffffffffu, uk[j], o);
      uq[j] += __shfl_xor_sync(0xffffffffu, uq[j], o);
    }
  if (lane < ST_LANES) {
    s_u[warp][0][lane] = make_float4(uk[0], uk[1], uk[2], uk[3]);
    s_u[warp][1][lane] = make_float4(uq[0], uq[1], uq[2], uq[3]);
  }
  taken = __syncthreads_or(taken);
  const bool live = here && !taken;
  if (!live && slot != -1 && tid == 0 && ar.status) atomicOr(ar.status, kStatusClamped);
  float4 a0 = make_float4(0.f, 0.f, 0.f, 0.f), a1 = a0;
#pragma unroll
  for (int w = 0; w < ST_NT / 32; ++w) {
    const float4 y0 = s_u[w][0][lane % ST_LANES], y1 = s_u[w][1][lane % ST_LANES];
    a0.x += y0.x; a0.y += y0.y; a0.z += y0.z; a0.w += y0.w;
    a1.x += y1.x; a1.y += y1.y; a1.z += y1.z; a1.w += y1.w;
  }
  // the row added along k
  const float w0 = beta * (v[0] - alpha * a0.x), w1 = beta * (v[1] - alpha * a0.y);
  const float w2 = beta * (v[2] - alpha * a0.z), w3 = beta * (v[3] - alpha * a0.w);
  if (tid < ST_LANES && in) {
    float o[4] = {fmaf(kq, w0, alpha * a1.x), fmaf(kq, w1, alpha * a1.y),
                  fmaf(kq, w2, alpha * a1.z), fmaf(kq, w3, alpha * a1.w)};
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = live ? o[j] : 0.f;
    st4(reinterpret_cast<T*>(ar.o) + vo, o);
  }
  if (!live || !in) return;
#pragma unroll
  for (int i = 0; i < ST_ACC; ++i) {
    if (!FULL && i * ST_ROWS >= dk) break;
    const float kr = s_k[warp][i0 + i * ST_ROWS];
    S[i].x = fmaf(kr, w0, alpha * S[i].x);
    S[i].y = fmaf(kr, w1, alpha * S[i].y);
    S[i].z = fmaf(kr, w2, alpha * S[i].z);
    S[i].w = fmaf(kr, w3, alpha * S[i].w);
    __stcs(reinterpret_cast<float4*>(Sp + (int64_t)i * ST_ROWS * ar.dv), S[i]);
  }
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
  if (n_slots > 0x7fffffff || pr.B * pr.H > 0x1fffffff) return GDN_ERR_UNSUPPORTED;
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
  ar.slices = (unsigned)((pr.dv + ST_COLS - 1) / ST_COLS);
  const unsigned ctas = (unsigned)(pr.B * pr.H * ar.slices);
  const cudaError_t e =
      pr.dtype == GDN_BF16  // dk = dv = 128
          ? launch_behind(k_step<__nv_bfloat16, true>, dim3(ctas), ST_NT, 0, st, ar)
          : launch_behind(k_step<float, false>, dim3(ctas), ST_NT, 0, st, ar);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
