// gdn_attn.cu -- attention of one new token per request over a paged key-value cache.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using namespace vec;

constexpr int AT_NT = 128;

struct AttnArgs {
  int64_t B, Hq, Hk, pages, max_blocks, qs;
  int P;
  float scale;
  const void *q, *kc, *vc;
  const int32_t *table, *len;
  void* o;
  float* lse;
  int32_t* status;
};

// one CTA per request and query head; a warp per key, D / 32 elements per lane
template <int D, typename T>
__global__ void __launch_bounds__(AT_NT) k_attn_decode(AttnArgs ar) {
  constexpr int E = D / 32, W = AT_NT / 32;
  __shared__ float s_m[W], s_l[W], s_o[W][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / ar.Hq, h = blockIdx.x % ar.Hq, hk = h / (ar.Hq / ar.Hk);
  const int64_t cap = ar.max_blocks * ar.P;
  int64_t len = ar.len[b];
  bool bad = len < 0 || len > cap;
  len = len < 0 ? 0 : len > cap ? cap : len;
  float q[E], acc[E] = {}, m = -INFINITY, l = 0.f;
  const T* qp = reinterpret_cast<const T*>(ar.q) + b * ar.qs + h * D;
#pragma unroll
  for (int j = 0; j < E; ++j) q[j] = (float)qp[j * 32 + lane] * ar.scale;
  for (int64_t t = warp; t < len; t += W) {
    const int64_t page = ar.table[b * ar.max_blocks + t / ar.P];
    if (page < 0 || page >= ar.pages) {
      bad = true;
      continue;
    }
    const int64_t off = ((page * ar.P + t % ar.P) * ar.Hk + hk) * D;
    const T* kp = reinterpret_cast<const T*>(ar.kc) + off;
    const T* vp = reinterpret_cast<const T*>(ar.vc) + off;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) s = fmaf(q[j], (float)kp[j * 32 + lane], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float f = expf(m - base), p = expf(s - base);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] = acc[j] * f + p * (float)vp[j * 32 + lane];
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) s_o[warp][j * 32 + lane] = acc[j];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < W; ++w) M = fmaxf(M, s_m[w]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < W; ++w) L += s_l[w] * expf(s_m[w] - base);
  for (int e = threadIdx.x; e < D; e += AT_NT) {
    float x = 0.f;
    for (int w = 0; w < W; ++w) x += s_o[w][e] * expf(s_m[w] - base);
    reinterpret_cast<T*>(ar.o)[(b * ar.Hq + h) * D + e] = (T)(L > 0.f ? x / L : x);
  }
  if (threadIdx.x == 0 && ar.lse) ar.lse[b * ar.Hq + h] = base + logf(L);
  if (bad && ar.status) atomicOr(ar.status, kStatusClamped);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool ok16(const void* p, int64_t n) { return n == 0 || (p && aligned16(p)); }
bool ok4(const void* p, int64_t n) { return n == 0 || (p && ((uintptr_t)p & 3u) == 0); }

gdn_status check_problem(const gdn_attn_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (p->B < 0 || p->Hq < 1 || p->Hk < 1 || p->Hq % p->Hk != 0 || p->pages < 0 ||
      p->max_blocks < 0 || p->page_size < 1 || p->D < 1 || p->scale != p->scale)
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

template <typename T>
cudaError_t launch(const AttnArgs& ar, int D, cudaStream_t st) {
  const unsigned ctas = (unsigned)(ar.B * ar.Hq);
  if (D == 64) k_attn_decode<64, T><<<ctas, AT_NT, 0, st>>>(ar);
  else if (D == 128) k_attn_decode<128, T><<<ctas, AT_NT, 0, st>>>(ar);
  else k_attn_decode<256, T><<<ctas, AT_NT, 0, st>>>(ar);
  return cudaGetLastError();
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_attn_decode_workspace_size(const gdn_attn_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  *bytes = 256;
  return GDN_OK;
}

gdn_status gdn_attn_decode(const gdn_attn_problem* p, const void* q, const void* k_cache,
                           const void* v_cache, const int32_t* block_table,
                           const int32_t* seq_len, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, int32_t* status, void* stream) {
  size_t need = 0;
  gdn_status s = gdn_attn_decode_workspace_size(p, &need);
  if (s != GDN_OK) return s;
  if (p->B == 0) return GDN_OK;
  const int64_t rows = p->pages * p->page_size;
  if (!ok16(q, 1) || !ok16(o, 1) || !ok16(k_cache, rows) || !ok16(v_cache, rows) ||
      !ok4(block_table, p->B * p->max_blocks) || !ok4(seq_len, 1) || !aligned16(lse) ||
      ((uintptr_t)workspace & 255u) != 0 || ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
  AttnArgs ar;
  memset(&ar, 0, sizeof(ar));
  ar.B = p->B;
  ar.Hq = p->Hq;
  ar.Hk = p->Hk;
  ar.pages = p->pages;
  ar.max_blocks = p->max_blocks;
  ar.qs = p->q_stride ? p->q_stride : p->Hq * p->D;
  ar.P = p->page_size;
  ar.scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->D);
  ar.q = q;
  ar.kc = k_cache;
  ar.vc = v_cache;
  ar.table = block_table;
  ar.len = seq_len;
  ar.o = o;
  ar.lse = lse;
  ar.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = p->dtype == GDN_BF16 ? launch<__nv_bfloat16>(ar, p->D, st)
                                             : launch<float>(ar, p->D, st);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
