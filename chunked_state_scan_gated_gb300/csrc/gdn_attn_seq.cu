// gdn_attn_seq.cu -- attention of packed sequences and its gradients: the calls, their schedule,
// and the fp32 kernels (the bf16 ones, and those that join parts, are in gdn_attn_seq_tc.cu).
//
// Forward, per query row: s_j = scale q.k_j, one pass over the keys with the running maximum m and
// sum l of a softmax, o = sum_j exp(s_j - m) v_j / l, lse = m + log l.  Backward, from lse and
// delta = dO.o: p = exp(s - lse), ds = p (dO.v - delta); a CTA owns a tile of keys (dk, dv: all
// queries that see it) or of queries (dq: all keys that they see), so that every gradient row has
// one writer, no atomics, and sums in a fixed order.
//
// fp32: register tiles on CUDA cores, whose FMA pipes are busy 55 to 64% of the time behind the reads of
// shared memory (below).  Split products on the tensor cores, as in the decode call, would keep two or
// three terms of every operand in shared memory (two of 64 rows of 128: 64 KB); they are not built.
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
// a class in any order, which no result depends on).  CTA 0: query tiles, CTA 1: key tiles.  One CTA
// goes over the offsets three times, 1024 at a time, in front of everything else: 5 to 6 us of a forward
// of 16 x 1000 or 64 x 250 tokens (157 and 96 us; no difference in the gradients), but 110 us for 4096
// sequences and 2.6 ms for 100,000.
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

// lse2 = lse log2(e) (fp32: lse), +inf for a row that sees no key (its p is 0), and delta = dO.o, by
// rows of heads: what the other kernels read along the tokens.  Bound by HBM.
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
    a.lse2[h * a.Nq + n] = l == -INFINITY ? INFINITY : sizeof(T) == 2 ? l * kLog2e : l;
    a.delta[h * a.Nq + n] = s;
  }
}

// ----------------------------------------------------------------------- fp32, CUDA cores

// The other side's operands come as chunks of 18 KB through a ring in shared memory (cp.async), in two
// shapes: columns of 64 rows for the products over D, whole rows for those over tokens.  A barrier
// per chunk empties the warps' pipelines, which is why chunks are large (2048 tokens, 16 on 2 heads of
// 128, forward / gradients: 450 / 1580 us with 9 KB, 387 / 1460 with 18).  A product over D keeps
// two sums, of the even and of the odd columns, one over tokens two rows: either way two numbers to an
// instruction (one number: 494 and 1609 us).  At two
// warps to a scheduler (registers: accumulators of 128 numbers at D = 256) the FMA pipes are busy 55 to
// 64% of the time, the way from shared memory to the registers 45% in the forward and 70 to 77% in the
// backward.
constexpr int ST = 64;  // rows and columns of a tile
constexpr int LT = 68;  // floats between the columns of the weights: 16-byte aligned

typedef unsigned long long f32x2;

__device__ __forceinline__ void fma2(f32x2& c, f32x2 x, f32x2 y) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(x), "l"(y));
}
__device__ __forceinline__ f32x2 pair(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 parts_of(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ float sum_of(f32x2 x) {
  const float2 r = parts_of(x);
  return r.x + r.y;
}
__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");  // zeros where it is not in
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // for all groups but the last N
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// By NT threads: R rows of C floats of src, zeros from row n on.
template <int R, int C, int PITCH, int NT>
__device__ __forceinline__ void copy_rows(float* dst, const float* src, int64_t stride, int n) {
#pragma unroll
  for (int z = 0; z < R * (C / 4) / NT; ++z) {
    const int i = threadIdx.x % NT + z * NT, r = i / (C / 4), c = i % (C / 4) * 4;
    const bool in = r < n;
    copy16(dst + r * PITCH + c, src + (in ? r * stride + c : 0), in);
  }
}

constexpr int F_HALF = 128, F_NT = 2 * F_HALF, F_STAGES = 3;
constexpr int F_KC = 64, F_KP = F_KC + 4;  // columns of a chunk of K, floats between its rows
constexpr int F_SLOT = ST * F_KP;

template <int D>
constexpr int fwd_half() {  // floats of a half's buffers: the ring, P
  return F_STAGES * F_SLOT + ST * LT;
}
template <int D>
constexpr size_t fwd_smem() {
  return (size_t)(ST * (D + 4) + 2 * fwd_half<D>() + 2 * ST) * 4;
}

// 64 queries of one head.  Two halves of the CTA take the blocks of 64 keys in turn, each with a
// softmax of its own, and are joined at the end: a prompt's last tile, which takes the longest, is
// done in half the time (9 prompts up to 700 tokens, 12 heads of 64: 58 us; one token behind 13,972
// keys, 4 heads of 128: 64 us, 16 heads 169).  A thread has 8 rows (ty, ty + 8, ..) x 4 keys (tx, tx + 16, ..) of the
// scores, 8 rows x D/16 columns of o.
template <int D>
__global__ void __launch_bounds__(F_NT) k_attn_fwd_simt(SeqArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int NV = D / 64, QP = D + 4, NK = D / F_KC, VR = ST * F_KC / D;
  const int half = threadIdx.x / F_HALF, tid = threadIdx.x % F_HALF;
  float *Q = sm, *ring = Q + ST * QP + half * fwd_half<D>(), *Pt = ring + F_STAGES * F_SLOT;
  float* ml = sm + ST * QP + 2 * fwd_half<D>();
  after_previous();
  before_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) check_single(a);
  const int part = blockIdx.x % a.parts, item = blockIdx.x / a.parts;
  const int h = item % a.Hq, hk = h / a.G;
  Tile t;
  if (!tile_of<false>(a, item / a.Hq, &t)) return;
  const int ty = tid / 16, tx = tid % 16;
  const int rows = min(ST, t.nq - t.at), off = t.nk - t.nq, seen = keys_seen(a, t, ST);
  // this part's share of the blocks, and this half's of those
  const int64_t blocks = (seen + ST - 1) / ST;
  const int from = (int)(blocks * part / a.parts), to = (int)(blocks * (part + 1) / a.parts);
  const int end = min(seen, to * ST), mine = max(0, (to - from - half + 1) / 2);
  const float* q = (const float*)a.q + (t.q0 + t.at) * a.qs + (int64_t)h * D;
  const float* k = (const float*)a.k + t.k0 * a.ks + (int64_t)hk * D;
  const float* v = (const float*)a.v + t.k0 * a.vs + (int64_t)hk * D;
  auto first_of = [&](int b) { return (from + half + 2 * b) * ST; };
  auto v_chunks = [&](int b) { return (min(ST, end - first_of(b)) + VR - 1) / VR; };
  int fb = 0, fc = 0, fs = 0;  // the next chunk to be fetched, its place in the ring
  auto fetch = [&]() {
    if (fb < mine) {
      const int kb = first_of(fb);
      float* to_ = ring + fs * F_SLOT;
      if (fc < NK) {
        copy_rows<ST, F_KC, F_KP, F_HALF>(to_, k + kb * a.ks + fc * F_KC, a.ks, end - kb);
      } else {
        const int at = kb + (fc - NK) * VR;
        copy_rows<VR, D, D, F_HALF>(to_, v + at * a.vs, a.vs, end - at);
      }
      fs = fs + 1 == F_STAGES ? 0 : fs + 1;
      if (++fc == NK + v_chunks(fb)) {
        fc = 0;
        ++fb;
      }
    }
    copies_end();  // a group without copies past the last one
  };
  int slot = 0;
  auto next = [&]() {  // the next chunk is there; the one before it is no longer read
    copies_wait<F_STAGES - 2>();
    asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "n"(F_HALF) : "memory");
    fetch();
    const float* x = ring + slot * F_SLOT;
    slot = slot + 1 == F_STAGES ? 0 : slot + 1;
    return x;
  };
  copy_rows<ST, D, QP, F_NT>(Q, q, a.qs, rows);
  copies_end();
#pragma unroll
  for (int i = 0; i < F_STAGES - 1; ++i) fetch();
  f32x2 o[4][NV][4];  // rows 2i and 2i + 1 of the thread's
  float m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < NV; ++c) o[i][c][0] = o[i][c][1] = o[i][c][2] = o[i][c][3] = 0;
  copies_wait<F_STAGES - 1>();
  __syncthreads();  // Q is there
  for (int b = 0; b < mine; ++b) {
    const int kb = first_of(b);
    f32x2 s2[8][4] = {};
#pragma unroll 1
    for (int c = 0; c < NK; ++c) {
      const float* K = next();
#pragma unroll 4
      for (int d = 0; d < F_KC; d += 4) {
        ulonglong2 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = *reinterpret_cast<const ulonglong2*>(Q + (ty + 8 * i) * QP + c * F_KC + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(K + (tx + 16 * j) * F_KP + d);
#pragma unroll
          for (int i = 0; i < 8; ++i) fma2(s2[i][j], x[i].x, y.x);
#pragma unroll
          for (int i = 0; i < 8; ++i) fma2(s2[i][j], x[i].y, y.y);
        }
      }
    }
    float f[8], s[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int top = a.causal ? min(end, t.at + ty + 8 * i + off + 1) : end;  // keys seen
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = kb + tx + 16 * j < top ? sum_of(s2[i][j]) * a.sl : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float base = mx == -INFINITY ? 0.f : mx;
      f[i] = ex2(m[i] - base);
      m[i] = mx;
      l[i] *= f[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2(s[i][j] - base);
        l[i] += s[i][j];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = parts_of(o[i][c][j]);
          o[i][c][j] = pair(x.x * f[2 * i], x.y * f[2 * i + 1]);
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float* at = Pt + (tx + 16 * j) * LT + ty * 8;
      *reinterpret_cast<float4*>(at) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
      *reinterpret_cast<float4*>(at + 4) = make_float4(s[4][j], s[5][j], s[6][j], s[7][j]);
    }
    const int nv = v_chunks(b);
#pragma unroll 1
    for (int c = 0; c < nv; ++c) {
      const float* V = next();
      const float* P = Pt + c * VR * LT + ty * 8;
#pragma unroll 4
      for (int j = 0; j < VR; ++j) {
        const ulonglong2 x0 = *reinterpret_cast<const ulonglong2*>(P + j * LT);
        const ulonglong2 x1 = *reinterpret_cast<const ulonglong2*>(P + j * LT + 4);
        const f32x2 x[4] = {x0.x, x0.y, x1.x, x1.y};
#pragma unroll
        for (int w = 0; w < NV; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(V + j * D + w * 64 + tx * 4);
          const f32x2 ys[4] = {pair(y.x, y.x), pair(y.y, y.y), pair(y.z, y.z), pair(y.w, y.w)};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int z = 0; z < 4; ++z) fma2(o[i][w][z], x[i], ys[z]);
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
      for (int c = 0; c < NV; ++c) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = i % 2 ? parts_of(o[i / 2][c][j]).y : parts_of(o[i / 2][c][j]).x;
        *reinterpret_cast<float4*>(Q + (ty + 8 * i) * D + c * 64 + tx * 4) =
            make_float4(x[0], x[1], x[2], x[3]);
      }
      if (tx == 0) {
        ml[ty + 8 * i] = m[i];
        ml[ST + ty + 8 * i] = l[i];
      }
    }
  }
  __syncthreads();
  if (half == 1) return;
  float* out = a.parts > 1 ? a.part_o + part * a.Nq * a.Hq * D : (float*)a.out;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = ty + 8 * i;
    if (at >= rows) continue;
    const float m1 = ml[at], l1 = ml[ST + at], top = fmaxf(m[i], m1);
    const float base = top == -INFINITY ? 0.f : top, f0 = ex2(m[i] - base), f1 = ex2(m1 - base);
    const float sum = l[i] * f0 + l1 * f1, r = sum != 0.f ? 1.f / sum : 0.f;
    const int64_t row = (int64_t)(t.q0 + t.at + at) * a.Hq + h;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const float4 y = *reinterpret_cast<const float4*>(Q + at * D + c * 64 + tx * 4);
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = i % 2 ? parts_of(o[i / 2][c][j]).y : parts_of(o[i / 2][c][j]).x;
      *reinterpret_cast<float4*>(out + row * D + c * 64 + tx * 4) =
          make_float4((x[0] * f0 + y.x * f1) * r, (x[1] * f0 + y.y * f1) * r,
                      (x[2] * f0 + y.z * f1) * r, (x[3] * f0 + y.w * f1) * r);
    }
    if (tx == 0) {
      const float lse2 = sum != 0.f ? top + log2f(sum) : -INFINITY;
      if (a.parts > 1)
        a.part_lse[part * a.Nq * a.Hq + row] = lse2;
      else if (a.lse)
        a.lse[row] = lse2 * kLn2;
    }
  }
}

constexpr int B_NT = 256;
constexpr int B_CC = 32, B_CP = B_CC + 4;  // columns of a chunk, floats between its rows
constexpr int B_SLOT = 2 * ST * B_CP;
constexpr int B_RUN = 16;  // blocks that are summed up at a time

// Chunks on their way or in use.
template <bool KV>
constexpr int bwd_stages() {
  return KV ? 3 : 2;
}
template <int D, bool KV>
constexpr size_t bwd_smem() {
  return (size_t)(2 * ST * (D + 4) + bwd_stages<KV>() * B_SLOT + (KV ? 2 : 1) * ST * LT) * 4;
}
template <int D, bool KV>
constexpr int bwd_ctas() {
  return 2 * (bwd_smem<D, KV>() + 1024) <= 228 * 1024 ? 2 : 1;
}

// KV: 64 keys of one key head, dk and dv over all queries of its query heads; else 64 queries of
// one head, dq over the keys that they see.  A thread has 4 rows x 4 columns (tx, tx + 16, ..) of
// the scores and 4 rows x D/16 columns of each gradient.  The own side's two operands (k, v or q,
// dO) stay in shared memory.  Scores are computed twice, 7 products in place of 5, so that every
// gradient has one writer (3 rows of 8781 tokens, 2 heads of 128, not causal: 19.4 ms, 42 TFLOP/s
// of what is executed).
template <int D, bool KV>
__global__ void __launch_bounds__(B_NT, bwd_ctas<D, KV>()) k_attn_bwd_simt(SeqArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int NV = D / 64, NP = KV ? 2 : 1, RP = D + 4, STAGES = bwd_stages<KV>();
  constexpr int CC = B_CC, CP = B_CP, SLOT = B_SLOT;
  constexpr int C1 = D / CC, XR = 2 * ST * CC / (D * NP);  // chunks of columns; rows of a chunk of rows
  float *R1 = sm, *R2 = R1 + ST * RP, *ring = R2 + ST * RP, *dS = ring + STAGES * SLOT;
  float* P = dS + (KV ? ST * LT : 0);
  if (!a.late) after_previous();
  before_next();
  const int heads = KV ? a.Hk : a.Hq, part = KV ? blockIdx.x % a.splits : 0;
  const int item = KV ? blockIdx.x / a.splits : blockIdx.x, hh = item % heads, hk = KV ? hh : hh / a.G;
  Tile t;
  if (!tile_of<KV>(a, item / heads, &t)) {
    if (a.late) after_previous();
    return;
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, off = t.nk - t.nq;
  const int rows = min(ST, (KV ? t.nk : t.nq) - t.at);
  const int first = KV ? first_query(a, t) : 0, end = KV ? t.nq : keys_seen(a, t, ST);
  const float* kv_k = (const float*)a.k + t.k0 * a.ks + (int64_t)hk * D;
  const float* kv_v = (const float*)a.v + t.k0 * a.vs + (int64_t)hk * D;
  const int64_t os = (int64_t)a.Hq * D;  // between tokens of dO
  auto q_of = [&](int h) { return (const float*)a.q + t.q0 * a.qs + (int64_t)h * D; };
  auto do_of = [&](int h) { return (const float*)a.dO + t.q0 * os + (int64_t)h * D; };
  const int64_t s1 = KV ? a.qs : a.ks, s2 = KV ? os : a.vs;
  const int mine = KV ? a.G / a.splits : 1, h0 = KV ? hh * a.G + part * mine : hh;
  const int h1 = first < end ? h0 + mine : h0;
  auto x_chunks = [&](int b) { return (min(ST, end - b) + XR - 1) / XR; };
  int fh = h0, fb = first, fc = 0, fs = 0;  // the next chunk to be fetched, its place in the ring
  auto fetch = [&]() {
    if (fh < h1) {
      const float *x1 = KV ? q_of(fh) : kv_k, *x2 = KV ? do_of(fh) : kv_v;
      float* to = ring + fs * SLOT;
      if (fc < C1) {
        copy_rows<ST, CC, CP, B_NT>(to, x1 + fb * s1 + fc * CC, s1, end - fb);
        copy_rows<ST, CC, CP, B_NT>(to + ST * CP, x2 + fb * s2 + fc * CC, s2, end - fb);
      } else {
        const int at = fb + (fc - C1) * XR;
        copy_rows<XR, D, D, B_NT>(to, x1 + at * s1, s1, end - at);
        if (KV) copy_rows<XR, D, D, B_NT>(to + XR * D, x2 + at * s2, s2, end - at);
      }
      fs = fs + 1 == STAGES ? 0 : fs + 1;
      if (++fc == C1 + x_chunks(fb)) {
        fc = 0;
        fb += ST;
        if (fb >= end) {
          fb = first;
          ++fh;
        }
      }
    }
    copies_end();  // a group without copies past the last one
  };
  int slot = 0;
  auto next = [&]() {  // the next chunk is there; the one before it is no longer read
    copies_wait<STAGES - 2>();
    __syncthreads();
    fetch();
    const float* x = ring + slot * SLOT;
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    return x;
  };
  copy_rows<ST, D, RP, B_NT>(R1, (KV ? kv_k : q_of(hh)) + t.at * (KV ? a.ks : a.qs),
                             KV ? a.ks : a.qs, rows);
  copy_rows<ST, D, RP, B_NT>(R2, (KV ? kv_v : do_of(hh)) + t.at * (KV ? a.vs : os),
                             KV ? a.vs : os, rows);
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch();  // the first group holds R1 and R2 too
  f32x2 acc[NP][2][NV][4];                       // rows 2i and 2i + 1 of the thread's
  auto zero = [&]() {
#pragma unroll
    for (int z = 0; z < NP; ++z)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NV; ++c)
          acc[z][i][c][0] = acc[z][i][c][1] = acc[z][i][c][2] = acc[z][i][c][3] = 0;
  };
  zero();
  // what has been summed up, to the gradients (or parts of them), in runs of B_RUN blocks: an
  // accumulator's error grows with its terms (1363 tokens, 8 query heads to a key head: dv 1.4e-6 off in
  // one run, 8.3e-7 in runs of 16 blocks, in the same time)
  int blocks = 0;
  bool begun = false;
  auto flush = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ty * 4 + i >= rows) continue;
      const int64_t row = (int64_t)((KV ? t.k0 : t.q0) + t.at + ty * 4 + i) * heads + hh;
#pragma unroll
      for (int z = 0; z < NP; ++z) {
        float* to = (float*)(z ? a.dv : KV ? a.dk : a.dq);
        if (KV && a.splits > 1) to = (z ? a.part_v : a.part_k) + part * a.Nk * a.Hk * D;
        to += row * D + tx * 4;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          if (begun) sum = *reinterpret_cast<const float4*>(to + c * 64);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = parts_of(acc[z][i / 2][c][e]);
            x[e] = (i % 2 ? y.y : y.x) * (z ? 1.f : a.scale);
          }
          *reinterpret_cast<float4*>(to + c * 64) =
              make_float4(sum.x + x[0], sum.y + x[1], sum.z + x[2], sum.w + x[3]);
        }
      }
    }
    zero();
    blocks = 0;
    begun = true;
  };
  for (int h = h0; h < h1; ++h) {
    const float* lse = a.lse2 + (int64_t)h * a.Nq + t.q0;
    const float* delta = a.delta + (int64_t)h * a.Nq + t.q0;
    for (int b = first; b < end; b += ST) {
      float ls[4], de[4];  // of the queries: the thread's columns, or its rows
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int qi = KV ? b + tx + 16 * j : t.at + ty * 4 + j;
        ls[j] = qi < t.nq ? lse[qi] : INFINITY;
        de[j] = qi < t.nq ? delta[qi] : 0.f;
      }
      f32x2 s[4][4] = {}, dp[4][4] = {};
#pragma unroll 1
      for (int c = 0; c < C1; ++c) {
        const float* x = next();
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int d = 0; d < CC; d += 4) {
            const float* own = (z ? R2 : R1) + ty * 4 * RP + c * CC + d;
            ulonglong2 r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              r[i] = *reinterpret_cast<const ulonglong2*>(own + i * RP);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(
                  x + z * ST * CP + (tx + 16 * j) * CP + d);
#pragma unroll
              for (int i = 0; i < 4; ++i) fma2((z ? dp : s)[i][j], r[i].x, y.x);
#pragma unroll
              for (int i = 0; i < 4; ++i) fma2((z ? dp : s)[i][j], r[i].y, y.y);
            }
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p[4], ds[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = t.at + ty * 4 + i, col = b + tx + 16 * j, w = KV ? j : i;
          const int qi = KV ? col : row, kj = KV ? row : col;
          const bool in = qi < t.nq && kj < t.nk && (!a.causal || kj <= qi + off);
          // the exponent is rounded once, where it is small: p is at most 1
          p[i] = in ? ex2(fmaf(sum_of(s[i][j]), a.scale, -ls[w]) * kLog2e) : 0.f;
          ds[i] = in ? p[i] * (sum_of(dp[i][j]) - de[w]) : 0.f;
        }
        *reinterpret_cast<float4*>(dS + (tx + 16 * j) * LT + ty * 4) =
            make_float4(ds[0], ds[1], ds[2], ds[3]);
        if (KV)
          *reinterpret_cast<float4*>(P + (tx + 16 * j) * LT + ty * 4) =
              make_float4(p[0], p[1], p[2], p[3]);
      }
      const int nx = x_chunks(b);
#pragma unroll 1
      for (int c = 0; c < nx; ++c) {
        const float* x = next();
#pragma unroll
        for (int j = 0; j < XR; ++j)
#pragma unroll
          for (int z = 0; z < NP; ++z) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(
                (z ? P : dS) + (c * XR + j) * LT + ty * 4);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const float4 y =
                  *reinterpret_cast<const float4*>(x + (z * XR + j) * D + v * 64 + tx * 4);
              const f32x2 ys[4] = {pair(y.x, y.x), pair(y.y, y.y), pair(y.z, y.z),
                                   pair(y.w, y.w)};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                fma2(acc[z][0][v][e], w.x, ys[e]);
                fma2(acc[z][1][v][e], w.y, ys[e]);
              }
            }
          }
      }
      if (++blocks == B_RUN) flush();
    }
  }
  if (blocks > 0 || !begun) flush();
  if (a.late) after_previous();
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
  // A key tile's query heads go to several CTAs where there are fewer tiles than 4 per SM; each writes a
  // part of dk and dv in fp32, which k_attn_sum adds up (bf16, 16001 tokens, 16 on 2 heads of 256: one
  // part 7.9 ms, 8: 6.0; the parts cost 16 bytes per element and part).
  y.splits = 1;
  const bool bf16 = p->dtype == GDN_BF16;
  const int64_t G = p->Hq / p->Hk, tiles = (int64_t)y.mk * p->Hk * (bf16 ? rk / 128 : 1);
  if (bwd && tiles > 0)
    for (int64_t s = 2; s <= G && tiles * y.splits < 608; ++s)
      if (G % s == 0) y.splits = (int)s;
  const size_t part = y.splits > 1 ? up((size_t)y.splits * p->Nk * p->Hk * p->D * 4) : 0;
  y.part_v = y.part_k + part;
  y.part_o = y.part_v + part;
  // Forward: tiles for less than one wave over many keys (a few new tokens behind a long context)
  // leave SMs idle, so the keys of every tile are divided, 512 (fp32: 256) at least to a part on
  // average; the parts of o are fp32 and k_attn_merge joins them (bf16, 32 on 8 heads of 128: 64 tokens
  // behind 31936 338 us without, 53 with; with more tiles they cost more than they bring: 256 tiles of 9
  // sequences behind up to 16000 tokens 335 without, 348 in two parts, 4096 tokens 104 and 193.  fp32:
  // one token behind 13,972 keys, 16 heads of 128, 1387 and 169; 4 heads 1384 and 64).
  y.parts = 1;
  const int64_t items = (int64_t)y.mq * (p->Hq / (bf16 ? tc_pack(G) : 1));
  if (!bwd && items > 0) {
    int64_t s = items < 152 ? (2 * 152 + items - 1) / items : 1;
    const int64_t keys = p->Nk / (n > 0 ? n : 1), least = bf16 ? 512 : 256;
    if (s > keys / least) s = keys / least;
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
  a->pack = bf16 ? tc_pack(a->G) : 1;
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
    const cudaError_t e = launch_simt<k_attn_fwd_simt<d()>>((int64_t)a.tq.most * a.Hq * a.parts,
                                                            F_NT, fwd_smem<d()>(), st, a);
    return e == cudaSuccess && a.parts > 1 ? launch_merge(a, d(), true, st) : e;
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
    // one CTA at least: it looks at a single sequence's offsets
    const unsigned grid = rows > 0 ? (unsigned)((rows + per - 1) / per) : 1;
    cudaError_t e = bf16 ? launch_behind(k_attn_rows<D, __nv_bfloat16>, dim3(grid), 256, 0, st, a)
                         : launch_behind(k_attn_rows<D, float>, dim3(grid), 256, 0, st, a);
    if (e != cudaSuccess) return e;
    if (bf16) return launch_bwd_tc(a, D, st);
    e = launch_simt<k_attn_bwd_simt<D, true>>((int64_t)a.tk.most * a.Hk * a.splits, B_NT,
                                              bwd_smem<D, true>(), st, a);
    if (e != cudaSuccess) return e;
    a.late = a.tk.most > 0;  // reads nothing of the launch before
    e = launch_simt<k_attn_bwd_simt<D, false>>((int64_t)a.tq.most * a.Hq, B_NT,
                                               bwd_smem<D, false>(), st, a);
    return e == cudaSuccess && a.Nk > 0 && a.splits > 1 ? launch_sum(a, D, true, st) : e;
  });
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
