// gdn_attn_seq.cu -- attention of packed sequences and its gradients: the calls, their schedule,
// and the fp32 kernels (the bf16 ones are in gdn_attn_seq_tc.cu).
//
// Forward, per query row: s_j = scale q.k_j, one pass over the keys with the running maximum m and
// sum l of a softmax, o = sum_j exp(s_j - m) v_j / l, lse = m + log l.  Backward, from lse and
// delta = dO.o: p = exp(s - lse), ds = p (dO.v - delta); a CTA owns a tile of keys (dk, dv: all
// queries that see it) or of queries (dq: all keys that they see), so that every gradient row has
// one writer, no atomics, and sums in a fixed order.
//
// fp32: register tiles on CUDA cores, bound by their FMA rate (the split tf32 products of the
// decode call would need two copies of every operand in shared memory).  Operands are transposed
// as they enter shared memory, so that a thread's rows are one or two 16-byte reads per step.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "gdn_attn_seq.cuh"

namespace gdn {
namespace seq {
namespace {

// ------------------------------------------------------------------------------ schedule

constexpr int PL_NT = 1024;
constexpr int PL_BUCKETS = 1024;

struct PlanSide {
  Tile* list;
  int* count;
  int rows, most;
};

// The list of tiles, those with the most work first (in the order of 1024 classes of work; within
// a class in any order, which no result depends on).  CTA 0: query tiles, CTA 1: key tiles.
__global__ void __launch_bounds__(PL_NT) k_attn_plan(SeqArgs a, PlanSide s0, PlanSide s1) {
  __shared__ int s_start[PL_BUCKETS], s_warp[2][32], s_carry[2], s_max;
  __shared__ int s_q0[PL_NT], s_nq[PL_NT], s_k0[PL_NT], s_nk[PL_NT];
  after_previous();
  before_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool keys = blockIdx.x == 1;
  const PlanSide s = keys ? s1 : s0;
  const int32_t* ck = a.cuk ? a.cuk : a.cuq;
  int bad = 0;
  auto work = [&](int nq, int nk, int at) {  // rows of the other side
    const int off = nk - nq;
    if (!a.causal) return keys ? nq : nk;
    return keys ? max(0, nq - max(0, at - off)) : max(0, min(nk, min(at + s.rows, nq) + off));
  };
  if (tid == 0) s_max = 1;
  for (int i = tid; i < PL_BUCKETS; i += PL_NT) s_start[i] = 0;
  // three turns over the sequences: the largest work, the classes' counts, the list
  for (int turn = 0; turn < 3; ++turn) {
    if (tid < 2) s_carry[tid] = 0;
    __syncthreads();
    if (turn == 2) {  // classes begin one behind the other, the largest first
      if (tid < 32) {
        int before = 0;
        for (int i0 = PL_BUCKETS - 32; i0 >= 0; i0 -= 32) {
          const int n = s_start[i0 + 31 - lane];
          int x = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          s_start[i0 + 31 - lane] = before + x - n;
          before += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) *s.count = min(before, s.most);
      }
      __syncthreads();
    }
    const float f = turn > 0 ? (PL_BUCKETS - 1) / (float)s_max : 0.f;
    for (int b0 = 0; b0 < a.n_seqs; b0 += PL_NT) {
      const int b = b0 + tid;
      // offsets as they count: within the rows and not below any one before
      int lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int32_t* cu = side ? ck : a.cuq;
        const int64_t n = side ? a.Nk : a.Nq;
        const int x0 = b < a.n_seqs ? cu[b] : 0, x1 = b < a.n_seqs ? cu[b + 1] : 0;
        int e = max(clamp_row(x0, n), clamp_row(x1, n));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, e, o);
          if (lane >= o) e = max(e, y);
        }
        if (lane == 31) s_warp[side][warp] = e;
        hi[side] = e;
        if (b < a.n_seqs && (x0 < 0 || x1 < x0 || x1 > n)) bad = 1;
        lo[side] = b < a.n_seqs ? clamp_row(x0, n) : 0;
      }
      __syncthreads();
      int before[2];
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        int c = s_carry[side];
        for (int w = 0; w < warp; ++w) c = max(c, s_warp[side][w]);
        const int up = __shfl_up_sync(0xffffffffu, hi[side], 1);
        before[side] = lane > 0 ? max(c, up) : c;
        hi[side] = max(c, hi[side]);
        lo[side] = max(lo[side], before[side]);
      }
      __syncthreads();
      if (tid == PL_NT - 1) {
        s_carry[0] = hi[0];
        s_carry[1] = hi[1];
      }
      s_q0[tid] = lo[0];
      s_nq[tid] = b < a.n_seqs ? hi[0] - lo[0] : 0;
      s_k0[tid] = lo[1];
      s_nk[tid] = b < a.n_seqs ? hi[1] - lo[1] : 0;
      __syncthreads();
      const int n = min(PL_NT, a.n_seqs - b0);
      for (int i = warp; i < n; i += PL_NT / 32) {  // a warp per sequence, a lane per tile
        const Tile t{s_q0[i], s_nq[i], s_k0[i], s_nk[i], 0};
        const int rows = keys ? t.nk : t.nq;
        for (int at = lane * s.rows; at < rows; at += 32 * s.rows) {
          const int w = work(t.nq, t.nk, at);
          if (turn == 0) {
            atomicMax(&s_max, w);
          } else {
            const int at_class = min(PL_BUCKETS - 1, (int)(w * f));
            const int place = atomicAdd(&s_start[at_class], 1);
            if (turn == 2 && place < s.most) {
              Tile x = t;
              x.at = at;
              s.list[place] = x;
            }
          }
        }
      }
      __syncthreads();
    }
  }
  if (bad && a.status) atomicOr(a.status, kStatusClamped);
}

// ------------------------------------------------------------------- backward: row values

// lse2 = lse log2(e), +inf for a row that sees no key (its p is 0), and delta = dO.o, by rows of
// heads: what the other kernels read along the tokens.  Bound by HBM.
template <int D, typename T>
__global__ void __launch_bounds__(256) k_attn_rows(SeqArgs a) {
  constexpr int EL = 16 / (int)sizeof(T), CH = D / EL, LR = CH < 32 ? CH : 32, CPL = CH / LR;
  after_previous();
  before_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) check_single(a);
  const int sub = threadIdx.x % LR;
  const int64_t rows = a.Nq * a.Hq;
  const int64_t r = (int64_t)blockIdx.x * (256 / LR) + threadIdx.x / LR;
  float s = 0.f;
  if (r < rows) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int64_t at = r * D + (sub + c * LR) * EL;
      const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.o) + at);
      const uint4 y = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.dO) + at);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
          s = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), s);
          s = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), s);
        } else {
          s = fmaf(__uint_as_float(xs[i]), __uint_as_float(ys[i]), s);
        }
      }
    }
  }
#pragma unroll
  for (int o = LR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (r < rows && sub == 0) {
    const int64_t n = r / a.Hq, h = r % a.Hq;
    const float l = a.lse[r];
    a.lse2[h * a.Nq + n] = l == -INFINITY ? INFINITY : l * kLog2e;
    a.delta[h * a.Nq + n] = s;
  }
}

// ----------------------------------------------------------------------- fp32, CUDA cores

constexpr int ST = 64;   // rows and columns of a tile
constexpr int LT = 68;   // a transposed operand's row in shared memory: 16-byte aligned
constexpr int F_HALF = 128, F_NT = 2 * F_HALF, F_DC = 32, F_KC = 16;

template <typename T>
__device__ __forceinline__ float4 ld4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
}
template <typename T>
__device__ __forceinline__ void st4(T* p, float x, float y, float z, float w) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x, y), b = __floats2bfloat162_rn(z, w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  }
}

// By NT threads: dst[c][row] = columns [c0, c0 + C) of rows [0, 64) of src (zeros from row n on).
template <int C, int NT, typename T>
__device__ __forceinline__ void load_t(float* dst, const T* src, int64_t stride, int n, int c0) {
  for (int i = threadIdx.x % NT; i < ST * (C / 4); i += NT) {
    const int r = i % ST, c = i / ST * 4;  // a warp's stores fall on different banks
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n) x = ld4(src + (int64_t)r * stride + c0 + c);
    dst[c * LT + r] = x.x;
    dst[(c + 1) * LT + r] = x.y;
    dst[(c + 2) * LT + r] = x.z;
    dst[(c + 3) * LT + r] = x.w;
  }
}
// dst[row][D] = rows [r0, r0 + R) of src (zeros from row n on).
template <int D, int R, int NT, typename T>
__device__ __forceinline__ void load_r(float* dst, const T* src, int64_t stride, int r0, int n) {
  for (int i = threadIdx.x % NT; i < R * (D / 4); i += NT) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < n) x = ld4(src + (int64_t)(r0 + r) * stride + c);
    *reinterpret_cast<float4*>(dst + r * D + c) = x;
  }
}

template <int D>
constexpr int fwd_half() {  // floats of a half's buffers: K's chunk, P, V's chunk
  return F_DC * LT + ST * LT + F_KC * D;
}
template <int D>
constexpr size_t fwd_smem() {
  return (size_t)(D * LT + 2 * fwd_half<D>() + 2 * ST) * 4;
}

// 64 queries of one head.  Two halves of the CTA take the blocks of 64 keys in turn, each with a
// softmax of its own, and are joined at the end: a prompt's last tile, which takes the longest, is
// done in half the time (9 prompts up to 700 tokens, 12 heads of 64: 121 us with one half).  A thread
// has 8 rows x 4 keys of the scores, 8 rows x D/16 columns of o.
template <int D, typename T>
__global__ void __launch_bounds__(F_NT) k_attn_fwd_simt(SeqArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int NV = D / 64;
  const int half = threadIdx.x / F_HALF, tid = threadIdx.x % F_HALF;
  float *Qt = sm, *Kt = Qt + D * LT + half * fwd_half<D>(), *Pt = Kt + F_DC * LT;
  float *Vc = Pt + ST * LT, *ml = sm + D * LT + 2 * fwd_half<D>();
  auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "n"(F_HALF) : "memory"); };
  after_previous();
  before_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) check_single(a);
  const int h = blockIdx.x % a.Hq, hk = h / a.G;
  Tile t;
  if (!tile_of<false>(a, blockIdx.x / a.Hq, &t)) return;
  const int ty = tid / 16, tx = tid % 16;
  const int rows = min(ST, t.nq - t.at), end = keys_seen(a, t, ST), off = t.nk - t.nq;
  const T* q = (const T*)a.q + (int64_t)(t.q0 + t.at) * a.qs + (int64_t)h * D;
  const T* k = (const T*)a.k + (int64_t)t.k0 * a.ks + (int64_t)hk * D;
  const T* v = (const T*)a.v + (int64_t)t.k0 * a.vs + (int64_t)hk * D;
  load_t<D, F_NT>(Qt, q, a.qs, rows, 0);
  float o[8][NV][4], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) o[i][c][0] = o[i][c][1] = o[i][c][2] = o[i][c][3] = 0.f;
  }
  __syncthreads();
  for (int kb = half * ST; kb < end; kb += 2 * ST) {
    float s[8][4] = {};
    for (int dc = 0; dc < D; dc += F_DC) {
      sync();
      load_t<F_DC, F_HALF>(Kt, k + (int64_t)kb * a.ks, a.ks, t.nk - kb, dc);
      sync();
#pragma unroll 8
      for (int d = 0; d < F_DC; ++d) {
        const float4 x0 = *reinterpret_cast<const float4*>(Qt + (dc + d) * LT + ty * 8);
        const float4 x1 = *reinterpret_cast<const float4*>(Qt + (dc + d) * LT + ty * 8 + 4);
        const float4 y = *reinterpret_cast<const float4*>(Kt + d * LT + tx * 4);
        const float xs[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        const float ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = fmaf(xs[i], ys[j], s[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int top = a.causal ? min(t.nk, t.at + ty * 8 + i + off + 1) : t.nk;  // keys seen
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = kb + tx * 4 + j < top ? s[i][j] * a.sl : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float base = mx == -INFINITY ? 0.f : mx, f = ex2(m[i] - base);
      m[i] = mx;
      l[i] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2(s[i][j] - base);
        l[i] += s[i][j];
      }
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][c][j] *= f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float* at = Pt + (tx * 4 + j) * LT + ty * 8;
      *reinterpret_cast<float4*>(at) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
      *reinterpret_cast<float4*>(at + 4) = make_float4(s[4][j], s[5][j], s[6][j], s[7][j]);
    }
    for (int kc = 0; kc < min(ST, end - kb); kc += F_KC) {
      sync();
      load_r<D, F_KC, F_HALF>(Vc, v + (int64_t)kb * a.vs, a.vs, kc, t.nk - kb);
      sync();
#pragma unroll 4
      for (int j = 0; j < F_KC; ++j) {
        const float4 x0 = *reinterpret_cast<const float4*>(Pt + (kc + j) * LT + ty * 8);
        const float4 x1 = *reinterpret_cast<const float4*>(Pt + (kc + j) * LT + ty * 8 + 4);
        const float xs[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const float4 y = *reinterpret_cast<const float4*>(Vc + j * D + c * 64 + tx * 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i][c][0] = fmaf(xs[i], y.x, o[i][c][0]);
            o[i][c][1] = fmaf(xs[i], y.y, o[i][c][1]);
            o[i][c][2] = fmaf(xs[i], y.z, o[i][c][2]);
            o[i][c][3] = fmaf(xs[i], y.w, o[i][c][3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
  // the second half's o goes over Q, its m and l behind the buffers
  __syncthreads();
  if (half == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int c = 0; c < NV; ++c)
        *reinterpret_cast<float4*>(Qt + (ty * 8 + i) * D + c * 64 + tx * 4) =
            make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
      if (tx == 0) {
        ml[ty * 8 + i] = m[i];
        ml[ST + ty * 8 + i] = l[i];
      }
    }
  }
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (ty * 8 + i >= rows) continue;
    const float m1 = ml[ty * 8 + i], l1 = ml[ST + ty * 8 + i], top = fmaxf(m[i], m1);
    const float base = top == -INFINITY ? 0.f : top, f0 = ex2(m[i] - base), f1 = ex2(m1 - base);
    const float sum = l[i] * f0 + l1 * f1, r = sum != 0.f ? 1.f / sum : 0.f;
    const int64_t row = (int64_t)(t.q0 + t.at + ty * 8 + i) * a.Hq + h;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const float4 y = *reinterpret_cast<const float4*>(Qt + (ty * 8 + i) * D + c * 64 + tx * 4);
      st4((T*)a.out + row * D + c * 64 + tx * 4, (o[i][c][0] * f0 + y.x * f1) * r,
          (o[i][c][1] * f0 + y.y * f1) * r, (o[i][c][2] * f0 + y.z * f1) * r,
          (o[i][c][3] * f0 + y.w * f1) * r);
    }
    if (tx == 0 && a.lse) a.lse[row] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
  }
}

constexpr int B_NT = 256, B_DC = 16, B_XC = 8;

template <int D, bool KV>
constexpr size_t bwd_smem() {
  return (size_t)(2 * D * LT + 2 * B_DC * LT + (KV ? 2 : 1) * ST * LT + (KV ? 2 : 1) * B_XC * D) * 4;
}

// KV: 64 keys of one key head, dk and dv over all queries of its query heads; else 64 queries of
// one head, dq over the keys that they see.  A thread has 4 x 4 scores and 4 rows x D/16 columns of
// each gradient.  The own side's two operands (k, v or q, dO) stay in shared memory.
template <int D, typename T, bool KV>
__global__ void __launch_bounds__(B_NT) k_attn_bwd_simt(SeqArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int NV = D / 64, NP = KV ? 2 : 1;
  float *R1 = sm, *R2 = R1 + D * LT, *C1 = R2 + D * LT, *C2 = C1 + B_DC * LT;
  float *dS = C2 + B_DC * LT, *P = dS + ST * LT, *X1 = dS + NP * ST * LT, *X2 = X1 + B_XC * D;
  after_previous();
  before_next();
  const int heads = KV ? a.Hk : a.Hq, hh = blockIdx.x % heads, hk = KV ? hh : hh / a.G;
  Tile t;
  if (!tile_of<KV>(a, blockIdx.x / heads, &t)) return;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, off = t.nk - t.nq;
  const int rows = min(ST, (KV ? t.nk : t.nq) - t.at);
  const int first = KV ? first_query(a, t) / ST * ST : 0, end = KV ? t.nq : keys_seen(a, t, ST);
  const T* kv_k = (const T*)a.k + (int64_t)t.k0 * a.ks + (int64_t)hk * D;
  const T* kv_v = (const T*)a.v + (int64_t)t.k0 * a.vs + (int64_t)hk * D;
  const int64_t os = (int64_t)a.Hq * D;  // between tokens of dO
  auto q_of = [&](int h) { return (const T*)a.q + (int64_t)t.q0 * a.qs + (int64_t)h * D; };
  auto do_of = [&](int h) { return (const T*)a.dO + t.q0 * os + (int64_t)h * D; };
  if (KV) {
    load_t<D, B_NT>(R1, kv_k + (int64_t)t.at * a.ks, a.ks, rows, 0);
    load_t<D, B_NT>(R2, kv_v + (int64_t)t.at * a.vs, a.vs, rows, 0);
  } else {
    load_t<D, B_NT>(R1, q_of(hh) + (int64_t)t.at * a.qs, a.qs, rows, 0);
    load_t<D, B_NT>(R2, do_of(hh) + (int64_t)t.at * os, os, rows, 0);
  }
  float acc[NP][4][NV][4] = {};
  for (int h = KV ? hh * a.G : hh; h < (KV ? (hh + 1) * a.G : hh + 1); ++h) {
    const float* lse2 = a.lse2 + (int64_t)h * a.Nq + t.q0;
    const float* delta = a.delta + (int64_t)h * a.Nq + t.q0;
    const T *x1 = KV ? q_of(h) : kv_k, *x2 = KV ? do_of(h) : kv_v;
    const int64_t s1 = KV ? a.qs : a.ks, s2 = KV ? os : a.vs;
    const int all = KV ? t.nq : t.nk;
    for (int b = first; b < end; b += ST) {
      float s[4][4] = {}, dp[4][4] = {};
      for (int dc = 0; dc < D; dc += B_DC) {
        __syncthreads();
        load_t<B_DC, B_NT>(C1, x1 + (int64_t)b * s1, s1, all - b, dc);
        load_t<B_DC, B_NT>(C2, x2 + (int64_t)b * s2, s2, all - b, dc);
        __syncthreads();
#pragma unroll
        for (int d = 0; d < B_DC; ++d) {
          const float4 r1 = *reinterpret_cast<const float4*>(R1 + (dc + d) * LT + ty * 4);
          const float4 r2 = *reinterpret_cast<const float4*>(R2 + (dc + d) * LT + ty * 4);
          const float4 c1 = *reinterpret_cast<const float4*>(C1 + d * LT + tx * 4);
          const float4 c2 = *reinterpret_cast<const float4*>(C2 + d * LT + tx * 4);
          const float r1s[4] = {r1.x, r1.y, r1.z, r1.w}, r2s[4] = {r2.x, r2.y, r2.z, r2.w};
          const float c1s[4] = {c1.x, c1.y, c1.z, c1.w}, c2s[4] = {c2.x, c2.y, c2.z, c2.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s[i][j] = fmaf(r1s[i], c1s[j], s[i][j]);
              dp[i][j] = fmaf(r2s[i], c2s[j], dp[i][j]);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p[4], ds[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = t.at + ty * 4 + i, col = b + tx * 4 + j;
          const int qi = KV ? col : row, kj = KV ? row : col;
          const bool in = qi < t.nq && kj < t.nk && (!a.causal || kj <= qi + off);
          p[i] = in ? ex2(fmaf(s[i][j], a.sl, -lse2[qi])) : 0.f;
          ds[i] = in ? p[i] * (dp[i][j] - delta[qi]) : 0.f;
        }
        *reinterpret_cast<float4*>(dS + (tx * 4 + j) * LT + ty * 4) =
            make_float4(ds[0], ds[1], ds[2], ds[3]);
        if (KV)
          *reinterpret_cast<float4*>(P + (tx * 4 + j) * LT + ty * 4) =
              make_float4(p[0], p[1], p[2], p[3]);
      }
      for (int xc = 0; xc < min(ST, end - b); xc += B_XC) {
        __syncthreads();
        load_r<D, B_XC, B_NT>(X1, x1 + (int64_t)b * s1, s1, xc, all - b);
        if (KV) load_r<D, B_XC, B_NT>(X2, x2 + (int64_t)b * s2, s2, xc, all - b);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < B_XC; ++j)
#pragma unroll
          for (int z = 0; z < NP; ++z) {
            const float4 w =
                *reinterpret_cast<const float4*>((z ? P : dS) + (xc + j) * LT + ty * 4);
            const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int c = 0; c < NV; ++c) {
              const float4 y =
                  *reinterpret_cast<const float4*>((z ? X2 : X1) + j * D + c * 64 + tx * 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                acc[z][i][c][0] = fmaf(ws[i], y.x, acc[z][i][c][0]);
                acc[z][i][c][1] = fmaf(ws[i], y.y, acc[z][i][c][1]);
                acc[z][i][c][2] = fmaf(ws[i], y.z, acc[z][i][c][2]);
                acc[z][i][c][3] = fmaf(ws[i], y.w, acc[z][i][c][3]);
              }
            }
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (ty * 4 + i >= rows) continue;
    const int64_t row = (int64_t)((KV ? t.k0 : t.q0) + t.at + ty * 4 + i) * heads + hh;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const float* x = acc[0][i][c];
      st4((T*)(KV ? a.dk : a.dq) + row * D + c * 64 + tx * 4, x[0] * a.scale, x[1] * a.scale,
          x[2] * a.scale, x[3] * a.scale);
      if constexpr (KV) {
        const float* y = acc[1][i][c];
        st4((T*)a.dv + row * D + c * 64 + tx * 4, y[0], y[1], y[2], y[3]);
      }
    }
  }
}

// -------------------------------------------------------------------------------- host

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool ok16(const void* p, int64_t n) { return n == 0 || (p && aligned16(p)); }
bool ok4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

gdn_status check_problem(const gdn_attn_seq_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (p->Nq < 0 || p->Nk < 0 || p->Hq < 1 || p->Hk < 1 || p->Hq % p->Hk != 0 || p->D < 1 ||
      p->n_seqs < (p->Nq + p->Nk > 0 ? 1 : 0) || (p->causal != 0 && p->causal != 1) ||
      !isfinite(p->scale) || !isfinite(fmaxf(p->scale, 0.f) * kLog2e))
    return GDN_ERR_INVALID_ARG;
  constexpr int64_t top = 0x7fffffff;
  if (p->Hq > top / 256) return GDN_ERR_UNSUPPORTED;
  const int64_t unit = p->dtype == GDN_BF16 ? 8 : 4;  // elements in 16 bytes
  const int64_t st[3] = {p->q_stride, p->k_stride, p->v_stride};
  for (int i = 0; i < 3; ++i) {
    if (st[i] != 0 && (st[i] < (i ? p->Hk : p->Hq) * p->D || st[i] % unit != 0))
      return GDN_ERR_INVALID_ARG;
    if (st[i] > top) return GDN_ERR_UNSUPPORTED;
  }
  if (p->D != 64 && p->D != 128 && p->D != 256) return GDN_ERR_UNSUPPORTED;
  if (p->Nq > top / p->Hq || p->Nk > top / p->Hk || p->n_seqs > (1 << 20))
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: the lists' counts, the lists, the backward's rows of lse and delta.
struct Layout {
  size_t lq, lk, lse2, delta, part_k, part_v, part_o, part_lse, total;
  int mq, mk;  // upper bounds of the tiles
  int splits;  // parts that a key head's query heads are divided into, for dk and dv
  int parts;   // .. and the keys of the forward
};
Layout layout(const gdn_attn_seq_problem* p, bool bwd, int rq, int rk) {
  Layout y;
  const int64_t n = p->n_seqs;
  const bool lists = n > 1;  // one sequence needs none
  // every sequence ends in one tile that may be partly empty
  y.mq = (int)(p->Nq / rq + (n < p->Nq ? n : p->Nq));
  y.mk = (int)(p->Nk / rk + (n < p->Nk ? n : p->Nk));
  y.lq = lists ? 256 : 0;
  y.lk = lists ? up(y.lq + y.mq * sizeof(Tile)) : 0;
  y.lse2 = lists && bwd ? up(y.lk + y.mk * sizeof(Tile)) : y.lk;
  y.delta = y.lse2 + (bwd ? up((size_t)p->Nq * p->Hq * 4) : 0);
  y.part_k = y.delta + (bwd ? up((size_t)p->Nq * p->Hq * 4) : 0);
  // bf16: a key tile's query heads go to several CTAs where there are fewer tiles than 4 per SM; each
  // writes a part of dk and dv in fp32, which k_attn_sum adds up (16001 tokens, 16 on 2 heads of 256:
  // one part 7.9 ms, 8: see the kernels' file; the parts cost 16 bytes per element and part).
  y.splits = 1;
  const int64_t G = p->Hq / p->Hk, tiles = (int64_t)y.mk * p->Hk * (rk / 128);
  if (bwd && p->dtype == GDN_BF16 && tiles > 0)
    for (int64_t s = 2; s <= G && tiles * y.splits < 608; ++s)
      if (G % s == 0) y.splits = (int)s;
  const size_t part = y.splits > 1 ? up((size_t)y.splits * p->Nk * p->Hk * p->D * 4) : 0;
  y.part_v = y.part_k + part;
  y.part_o = y.part_v + part;
  // bf16 forward: tiles for less than one wave over many keys (a few new tokens behind a long
  // context) leave SMs idle, so the keys of every tile are divided, 512 at least to a part on average;
  // the parts of o are fp32 and k_attn_merge joins them (64 tokens behind 31936, 32 on 8 heads of 128:
  // 338 us without, 80 with; 256 tiles of 9 sequences behind up to 16000 tokens: 308 and 330).
  y.parts = 1;
  const int64_t items = (int64_t)y.mq * (p->Hq / tc_pack(G));
  if (!bwd && p->dtype == GDN_BF16 && items > 0) {
    int64_t s = items < 152 ? (2 * 152 + items - 1) / items : 1;
    const int64_t keys = p->Nk / (n > 0 ? n : 1);
    if (s > keys / 512) s = keys / 512;
    y.parts = (int)(s < 1 ? 1 : s > kMaxParts ? kMaxParts : s);
  }
  const size_t rows = y.parts > 1 ? (size_t)y.parts * p->Nq * p->Hq * 4 : 0;
  y.part_lse = y.part_o + up(rows * p->D);
  y.total = y.part_lse + up(rows);
  return y;
}
Layout layout_of(const gdn_attn_seq_problem* p, bool bwd) {
  if (p->dtype != GDN_BF16) return layout(p, bwd, ST, ST);
  const TcPlan tp = tc_plan(p->D);
  return bwd ? layout(p, true, tp.dq_rows, tp.dkv_rows)
             : layout(p, false, tp.fwd_rows / tc_pack(p->Hq / p->Hk), ST);
}

// Arguments that both calls share, their checks, and the schedule's launch.
gdn_status begin(const gdn_attn_seq_problem* p, bool bwd, const int32_t* cu_q,
                 const int32_t* cu_k, char* ws, int32_t* status, cudaStream_t st, SeqArgs* a) {
  memset(a, 0, sizeof(*a));
  a->Nq = p->Nq;
  a->Nk = p->Nk;
  a->qs = p->q_stride ? p->q_stride : p->Hq * p->D;
  a->ks = p->k_stride ? p->k_stride : p->Hk * p->D;
  a->vs = p->v_stride ? p->v_stride : p->Hk * p->D;
  a->n_seqs = (int)p->n_seqs;
  a->Hq = (int)p->Hq;
  a->Hk = (int)p->Hk;
  a->G = a->Hq / a->Hk;
  a->causal = p->causal;
  a->scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->D);
  a->sl = a->scale * kLog2e;
  a->cuq = cu_q;
  a->cuk = cu_k;
  a->status = status;
  const Layout y = layout_of(p, bwd);
  const bool bf16 = p->dtype == GDN_BF16;
  const TcPlan tp = tc_plan(p->D);
  a->pack = tc_pack(a->G);
  a->tq.rows = bf16 ? (bwd ? tp.dq_rows : tp.fwd_rows / a->pack) : ST;
  a->tk.rows = bf16 ? tp.dkv_rows : ST;
  a->tq.most = y.mq;
  a->tk.most = y.mk;
  a->lse2 = (float*)(ws + y.lse2);
  a->delta = (float*)(ws + y.delta);
  a->part_k = (float*)(ws + y.part_k);
  a->part_v = (float*)(ws + y.part_v);
  a->splits = y.splits;
  a->part_o = (float*)(ws + y.part_o);
  a->part_lse = (float*)(ws + y.part_lse);
  a->parts = y.parts;
  if (cu_q && p->n_seqs > 1) {
    int* count = (int*)ws;
    PlanSide sq{(Tile*)(ws + y.lq), count, a->tq.rows, y.mq};
    PlanSide sk{(Tile*)(ws + y.lk), count + 1, a->tk.rows, y.mk};
    if (launch_behind(k_attn_plan, dim3(bwd ? 2 : 1), PL_NT, 0, st, *a, sq, sk) != cudaSuccess)
      return GDN_ERR_CUDA;
    a->tq.list = sq.list;
    a->tq.count = sq.count;
    a->tk.list = sk.list;
    a->tk.count = sk.count;
  }
  return GDN_OK;
}

gdn_status check_offsets(const gdn_attn_seq_problem* p, const int32_t* cu_q,
                         const int32_t* cu_k) {
  if (!ok4(cu_q) || !ok4(cu_k)) return GDN_ERR_INVALID_ARG;
  if (cu_q) return !cu_k && p->Nk != p->Nq ? GDN_ERR_INVALID_ARG : GDN_OK;
  if (cu_k || (p->n_seqs > 0 && (p->Nq % p->n_seqs != 0 || p->Nk % p->n_seqs != 0)))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

template <typename F>
auto with_dim(int D, F f) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  using D256 = std::integral_constant<int, 256>;
  return D == 64 ? f(D64()) : D == 128 ? f(D128()) : f(D256());
}

template <auto kKernel>
cudaError_t launch_simt(int64_t grid, int threads, size_t smem, cudaStream_t st,
                        const SeqArgs& a) {
  if (grid == 0) return cudaSuccess;
  const cudaError_t e = allow_smem<kKernel>(smem);
  if (e != cudaSuccess) return e;
  return launch_behind(kKernel, dim3((unsigned)grid), threads, smem, st, a);
}

}  // namespace
}  // namespace seq
}  // namespace gdn

using namespace gdn;
using namespace gdn::seq;

extern "C" {

gdn_status gdn_attn_fwd_workspace_size(const gdn_attn_seq_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  const gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  *bytes = layout_of(p, false).total;
  return GDN_OK;
}

gdn_status gdn_attn_fwd(const gdn_attn_seq_problem* p, const void* q, const void* k,
                        const void* v, const int32_t* cu_q, const int32_t* cu_k, void* o,
                        float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                        void* stream) {
  size_t need = 0;
  gdn_status s = gdn_attn_fwd_workspace_size(p, &need);
  if (s != GDN_OK) return s;
  if ((s = check_offsets(p, cu_q, cu_k)) != GDN_OK) return s;
  if (!ok16(q, p->Nq) || !ok16(o, p->Nq) || !ok16(k, p->Nk) || !ok16(v, p->Nk) ||
      !aligned16(lse) || ((uintptr_t)workspace & 255u) != 0 || ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (p->Nq == 0) return GDN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  SeqArgs a;
  if ((s = begin(p, false, cu_q, cu_k, (char*)workspace, status, st, &a)) != GDN_OK) return s;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = o;
  a.lse = lse;
  const cudaError_t e = p->dtype == GDN_BF16 ? launch_fwd_tc(a, p->D, st)
                                             : with_dim(p->D, [&](auto d) {
    return launch_simt<k_attn_fwd_simt<d(), float>>((int64_t)a.tq.most * a.Hq, F_NT,
                                                    fwd_smem<d()>(), st, a);
  });
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_attn_bwd_workspace_size(const gdn_attn_seq_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  const gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  *bytes = layout_of(p, true).total;
  return GDN_OK;
}

gdn_status gdn_attn_bwd(const gdn_attn_seq_problem* p, const void* q, const void* k,
                        const void* v, const void* o, const float* lse, const void* dO,
                        const int32_t* cu_q, const int32_t* cu_k, void* dq, void* dk, void* dv,
                        void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  size_t need = 0;
  gdn_status s = gdn_attn_bwd_workspace_size(p, &need);
  if (s != GDN_OK) return s;
  if ((s = check_offsets(p, cu_q, cu_k)) != GDN_OK) return s;
  if (!ok16(q, p->Nq) || !ok16(o, p->Nq) || !ok16(dO, p->Nq) || !ok16(lse, p->Nq) ||
      !ok16(dq, p->Nq) || !ok16(k, p->Nk) || !ok16(v, p->Nk) || !ok16(dk, p->Nk) ||
      !ok16(dv, p->Nk) || ((uintptr_t)workspace & 255u) != 0 || ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (p->Nq + p->Nk == 0) return GDN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  SeqArgs a;
  if ((s = begin(p, true, cu_q, cu_k, (char*)workspace, status, st, &a)) != GDN_OK) return s;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = const_cast<float*>(lse);
  a.dO = dO;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  const cudaError_t e = with_dim(p->D, [&](auto d) {
    constexpr int D = d();
    const bool bf16 = p->dtype == GDN_BF16;
    const int64_t rows = (int64_t)a.Nq * a.Hq;
    const int lanes = D * (bf16 ? 2 : 4) / 16, per = 256 / (lanes < 32 ? lanes : 32);
    const unsigned grid = (unsigned)((rows + per - 1) / per);
    cudaError_t e = cudaSuccess;
    if (grid > 0)
      e = bf16 ? launch_behind(k_attn_rows<D, __nv_bfloat16>, dim3(grid), 256, 0, st, a)
               : launch_behind(k_attn_rows<D, float>, dim3(grid), 256, 0, st, a);
    if (e != cudaSuccess) return e;
    if (bf16) return launch_bwd_tc(a, D, st);
    e = launch_simt<k_attn_bwd_simt<D, float, true>>((int64_t)a.tk.most * a.Hk, B_NT,
                                                     bwd_smem<D, true>(), st, a);
    if (e != cudaSuccess) return e;
    return launch_simt<k_attn_bwd_simt<D, float, false>>((int64_t)a.tq.most * a.Hq, B_NT,
                                                         bwd_smem<D, false>(), st, a);
  });
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
