// gdn_rope.cu -- RMSNorm of every query and key head with the position rotation.  Per head row
// x of D elements at position t, r = 1 / sqrt(mean(x^2) + eps), n = x r w, and for i < R/2 with
// c = rope_scale cos(t inv_freq[i]), s = rope_scale sin(t inv_freq[i]):
//   y1 = n1 c - n2 s,  y2 = n2 c + n1 s      on the pairs (i, i + R/2) or (2i, 2i + 1)
// Backward: dn1 = dy1 c + dy2 s, dn2 = dy2 c - dy1 s (the transposed rotation), g = dn w,
//   dx = r (g - x r mean(g x r)),  dw = sum over rows of dn x r.
// The angle is formed in revolutions: t * (inv_freq / 2 pi) as an exact two-term product, its
// integer part dropped, so positions past 2^20 lose nothing (angle()).
//
// Bound by HBM (2 row accesses forward, 3 backward).  A row is held 8 elements per lane (16 bytes
// of bf16) by LPR = 8, 16 or 32 lanes, so a warp holds 32 / LPR heads at a time; a group is U such
// sets, whose chains of shuffles are independent (32768 tokens of 18 heads of 256: 96 us with U =
// 2, 107 with 1).  The groups of all tokens are divided evenly over one wave of warps, from a
// decode step's few (each warp one group) to a training batch: no tail.  A warp streams its groups
// through a ring of its own in shared memory (16-byte asynchronous copies) with warp barriers
// only; a rotated element's partner in the other half is read from the ring.  The token's R/2
// angles are computed once and folded with the weights:
//   y = r (x (w c) + xp (w_p s)),  xp the partner elements, s with the sign of the pair's side
// and the arithmetic is packed two fp32 numbers at a time (237 instructions per row without
// either, 113 now).  Measured: forward of those 32768 tokens 96 us (6.3 TB/s), backward of 16001
// tokens of 40 heads of 128 81 us (6.1 TB/s); fp32, 16384 and 16001 tokens: 93 and 158 us (6.5 and
// 6.2 TB/s).  Two CTAs of 8 warps per SM with 4 KB in flight per
// warp are the best of 2 to 4 CTAs and 4 to 16 KB (3 CTAs: 108 us; 8 KB: 100 us).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using namespace vec;

constexpr int RO_NT = 256;     // 8 warps
constexpr int RO_W = RO_NT / 32;
constexpr int RO_CTAS = 152 * 2;  // CTAs at most: one wave of 2 per SM of a 152-SM GPU
constexpr int RO_MAXD = 256;   // 8 elements per lane
constexpr int RO_RING = 4096;  // bytes of a warp's ring
constexpr int RO_FU = 2, RO_GU = 1;  // sets of heads per group, forward and backward
constexpr int RO_SMEM = RO_W * (RO_RING + (RO_MAXD + 16) * 4);  // rings, cos and sin

struct RopeArgs {
  int64_t N, T, qs, ks, vs, n_slots;
  int Hq, Hk, D, R, inter;
  int gq, gk, gv;               // groups of a token's query, key and (cache form) value heads
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
// A frequency in revolutions per position, f / (2 pi) = hi + lo, with 1/(2 pi) as the sum of two
// fp32 numbers.
struct Freq {
  float hi, lo;
};
__device__ __forceinline__ Freq freq(float f) {
  constexpr float kHi = 0x1.45f306p-3f, kLo = 0x1.b9391p-28f;  // 1/(2 pi) = kHi + kLo
  const float hi = __fmul_rn(f, kHi);
  return Freq{hi, fmaf(f, kHi, -hi) + f * kLo};
}
// Revolutions of position x (exact in fp32), less whole ones.  The product with hi is exact as
// value and remainder of an fma.
__device__ __forceinline__ float turns(float x, Freq f) {
  const float p = __fmul_rn(x, f.hi);  // not contracted: its remainder is added here
  return (p - rintf(p)) + fmaf(x, f.hi, -p) + x * f.lo;
}
// cos and sin of t * f, t any int32, f fp32: t is split into two parts that are exact in fp32, and
// only the fraction goes into sincospi.  What is left is the rounding of the fraction (2^-24
// revolutions) and, past 2^24 revolutions, of lo and of the remainders (t f 2^-50: 2^-21 at t = 2^29).
__device__ __forceinline__ void angle(int32_t t, Freq f, float* c, float* s) {
  float u = turns((float)(t & 0xffff), f);
  if (t & ~0xffff) u += turns((float)(t & ~0xffff), f);
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

// 8 elements from a ring.
__device__ __forceinline__ void get(const __nv_bfloat16* p, F2 (&v)[4]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
__device__ __forceinline__ void get(const float* p, F2 (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
  v[0] = f2(a.x, a.y);
  v[1] = f2(a.z, a.w);
  v[2] = f2(b.x, b.y);
  v[3] = f2(b.z, b.w);
}
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
// 16 bytes per lane, without waiting; zeros where !in.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void copy8(T* dst, const T* src, bool in) {
  copy16(dst, src, in);
  if constexpr (sizeof(T) == 4) copy16(dst + 4, src + 4, in);
}

// The warp's table of the token's cos and sin, RO_MAXD / 2 of each, followed by 8 ones and 8
// zeros (no rotation).
constexpr int RO_CS = RO_MAXD + 16;
constexpr int RO_Z = RO_MAXD / 2 / 32;  // angles per lane at most
struct Angles {
  Freq f[RO_Z];  // of angles lane, lane + 32, ...
  int32_t t;     // position of the next token to be filled in, read ahead
  __device__ __forceinline__ void fetch(const RopeArgs& ar, int n) {
    t = n >= ar.N ? 0 : ar.pos ? ar.pos[n] : (int32_t)(n % ar.T);
  }
  __device__ __forceinline__ void init(const RopeArgs& ar, int n, float* cs) {
    const int lane = threadIdx.x & 31;
    fetch(ar, n);
#pragma unroll
    for (int z = 0; z < RO_Z; ++z)
      f[z] = freq(lane + 32 * z < ar.R / 2 ? ar.inv_freq[lane + 32 * z] : 0.f);
    if (lane < 16) cs[RO_MAXD + lane] = lane < 8 ? 1.f : 0.f;
  }
  // fills in the token whose position was read before; reads that of `next`
  __device__ __forceinline__ void fill(const RopeArgs& ar, int next, float* cs) {
    const int lane = threadIdx.x & 31;
    const int32_t at = t;
    fetch(ar, next);
    __syncwarp();  // the last token's readers are done
#pragma unroll
    for (int z = 0; z < RO_Z; ++z) {
      const int i = lane + 32 * z;
      if (i < ar.R / 2) {
        float c, s;
        angle(at, f[z], &c, &s);
        cs[i] = c * ar.rscale;
        cs[RO_MAXD / 2 + i] = s * ar.rscale;
      }
    }
    __syncwarp();
  }
};

// A lane's view of the rotation: y_j = x_j c_j + xp_j s_j with xp the partner elements and the
// sign of the pair's side in s (sgn = -1: the transposed rotation); c = 1, s = 0 past R.
template <bool INTER>
__device__ __forceinline__ void turn(const RopeArgs& ar, const float* cs, int e, float sgn,
                                     F2 (&c)[4], F2 (&s)[4]) {
  const bool in = e < ar.R, first = e < ar.R / 2;
  const int at = !in ? RO_MAXD : INTER ? e / 2 : first ? e : e - ar.R / 2;
  const float4* cp = reinterpret_cast<const float4*>(cs + at);
  const float4* sp = reinterpret_cast<const float4*>(cs + (in ? at + RO_MAXD / 2 : at + 8));
  const float4 c0 = cp[0], s0 = sp[0];
  if constexpr (INTER) {  // 4 pairs (c, c), (-s, s)
    const float cc[4] = {c0.x, c0.y, c0.z, c0.w}, ss[4] = {s0.x, s0.y, s0.z, s0.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = f2(cc[j], cc[j]);
      s[j] = f2(-sgn * ss[j], sgn * ss[j]);
    }
  } else {
    const float4 c1 = cp[1], s1 = sp[1];
    const float g = first ? -sgn : sgn;
    c[0] = f2(c0.x, c0.y);
    c[1] = f2(c0.z, c0.w);
    c[2] = f2(c1.x, c1.y);
    c[3] = f2(c1.z, c1.w);
    s[0] = f2(g * s0.x, g * s0.y);
    s[1] = f2(g * s0.z, g * s0.w);
    s[2] = f2(g * s1.x, g * s1.y);
    s[3] = f2(g * s1.z, g * s1.w);
  }
}
// The lane (of LPR) that holds the partner elements: its own past R (where they do not count).
__device__ __forceinline__ int other_lane(const RopeArgs& ar, int e) {
  if (e >= ar.R) return e / 8;
  return (e < ar.R / 2 ? e + ar.R / 2 : e - ar.R / 2) / 8;
}

// A warp's share of the groups: of the N tokens, as many whole rounds of one token per warp as
// there are (neighbouring warps read neighbouring tokens: a stretch of its own for each warp
// took a tenth longer), then an even part of the groups of the tokens that are left, from
// group tail_g of token tail_n.  Tokens fit 31 bits and groups 32 (checked on the host).
struct Share {
  int warps, full, tail_n, tail_g, groups;  // full: tokens in whole rounds
  unsigned todo;                            // groups of this warp
  __device__ __forceinline__ Share(const RopeArgs& ar, int g) {
    const unsigned w = blockIdx.x * RO_W + (threadIdx.x >> 5);
    groups = g;
    warps = (int)(gridDim.x * RO_W);
    const int rounds = (int)(ar.N / warps);
    full = rounds * warps;
    const uint64_t rest = (uint64_t)(ar.N - full) * g;
    const unsigned first = (unsigned)(rest * w / warps);
    todo = rounds * g + (unsigned)(rest * (w + 1) / warps) - first;
    tail_n = full + (int)(first / g);
    tail_g = (int)(first % g);
  }
};

// A run of groups of one token and kind (0 query, 1 key, 2 value).
struct Run {
  int n;
  int g;     // group of the token
  int kind;
  int i;     // group of the kind
  int stop;  // group of the token behind the kind's last
  int left;  // groups of the kind from here on
  __device__ __forceinline__ void set(const RopeArgs& ar) {
    kind = g < ar.gq ? 0 : g < ar.gq + ar.gk ? 1 : 2;
    stop = kind == 0 ? ar.gq : kind == 1 ? ar.gq + ar.gk : ar.gq + ar.gk + ar.gv;
    left = stop - g;
    i = g - (kind == 0 ? 0 : kind == 1 ? ar.gq : ar.gq + ar.gk);
  }
  __device__ __forceinline__ void tail(const Share& sh) {
    n = sh.tail_n;
    g = sh.tail_g;
  }
  __device__ __forceinline__ void start(const RopeArgs& ar, const Share& sh) {
    n = (int)(blockIdx.x * RO_W + (threadIdx.x >> 5));
    g = 0;
    if (n >= sh.full) tail(sh);
    set(ar);
  }
  // the token behind n
  __device__ __forceinline__ int behind(const Share& sh) const {
    if (n >= sh.full) return n + 1;
    return n + sh.warps < sh.full ? n + sh.warps : sh.tail_n;
  }
  // the run behind this one
  __device__ __forceinline__ void next(const RopeArgs& ar, const Share& sh) {
    g = stop;
    if (g >= sh.groups) {
      g = 0;
      if (n >= sh.full) ++n;
      else if ((n += sh.warps) >= sh.full) tail(sh);
    }
    set(ar);
  }
};

// Issues the groups of a warp's share one after another, NP rows (x, and dy backward) a head.
template <int LPR, int U, int NP, int NST, typename T>
struct Loader {
  static constexpr int RPL = 32 / LPR, SE = 32 * 8;
  Run run;
  unsigned todo;
  int h, end, step;   // this lane's first head, heads of the kind (0 past D), elements per set
  const T* p[NP];
  T* ring;            // this lane's place in stage 0
  __device__ __forceinline__ void set(const RopeArgs& ar) {
    const int lane = threadIdx.x & 31, e = (lane & (LPR - 1)) * 8;
    h = run.i * U * RPL + lane / LPR;
    end = e < ar.D ? (run.kind == 0 ? ar.Hq : ar.Hk) : 0;
    const int64_t at = (int64_t)h * ar.D + e;
    const int64_t n = run.n;
    if (run.kind == 0) {
      p[0] = reinterpret_cast<const T*>(ar.q) + n * ar.qs + at;
      if constexpr (NP == 2)
        p[1] = reinterpret_cast<const T*>(ar.dq_out) + n * ar.Hq * ar.D + at;
    } else if (NP == 2 || run.kind == 1) {
      p[0] = reinterpret_cast<const T*>(ar.k) + n * ar.ks + at;
      if constexpr (NP == 2)
        p[1] = reinterpret_cast<const T*>(ar.dk_out) + n * ar.Hk * ar.D + at;
    } else {
      p[0] = reinterpret_cast<const T*>(ar.v) + n * ar.vs + at;
    }
  }
  __device__ __forceinline__ void issue(const RopeArgs& ar, const Share& sh, int stage) {
    if (todo > 0) {
      T* dst = ring + stage * U * NP * SE;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = h + u * RPL < end;
#pragma unroll
        for (int z = 0; z < NP; ++z)
          copy8(dst + (u * NP + z) * SE, in ? p[z] + u * step : p[z], in);
      }
      --todo;
      if (--run.left > 0) {
        h += U * RPL;
#pragma unroll
        for (int z = 0; z < NP; ++z) p[z] += U * step;
      } else if (todo > 0) {
        run.next(ar, sh);
        set(ar);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// CACHE: k and v rows go to the caches
template <bool CACHE, bool INTER, int LPR, typename T>
__global__ void __launch_bounds__(RO_NT, 2) k_qk_norm_rope_fwd(RopeArgs ar) {
  extern __shared__ __align__(16) char smem[];
  after_previous();
  before_next();
  constexpr int U = RO_FU, RPL = 32 / LPR, SE = 32 * 8;
  constexpr int NST = RO_RING / (U * SE * (int)sizeof(T));
  static_assert(NST >= 2, "the stage being read is not the one being filled");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = (lane & (LPR - 1)) * 8;
  T* ring = reinterpret_cast<T*>(smem + warp * RO_RING);
  float* cs = reinterpret_cast<float*>(smem + RO_W * RO_RING) + warp * RO_CS;
  const int groups = ar.gq + ar.gk + (CACHE ? ar.gv : 0);
  const int other = INTER ? 0 : other_lane(ar, e);
  const int mine = lane * 8, theirs = (lane / LPR * LPR + other) * 8;
  const Share sh(ar, groups);
  if (sh.todo == 0) return;
  Loader<LPR, U, 1, NST, T> ld;
  ld.run.start(ar, sh);
  ld.todo = sh.todo;
  ld.step = RPL * ar.D;
  ld.ring = ring + mine;
  ld.set(ar);
  Run run = ld.run;
  for (int i = 0; i < NST - 1; ++i) ld.issue(ar, sh, i);
  Angles an;
  an.init(ar, run.n, cs);
  unsigned left = sh.todo;
  int64_t dst = -1;
  int stage = 0;
  for (int token = -1; left > 0; run.next(ar, sh)) {
    if (run.n != token) {
      token = run.n;
      an.fill(ar, run.behind(sh), cs);
      dst = run.n;
      if constexpr (CACHE) {
        dst = ar.slots[run.n];
        if (dst < 0 || dst >= ar.n_slots) {
          if (dst != -1 && lane == 0 && ar.status) atomicOr(ar.status, kStatusClamped);
          dst = -1;
        }
      }
    }
    const int kind = run.kind;
    const unsigned count = min((unsigned)run.left, left);
    left -= count;
    F2 A[4], B[4];
    if (!CACHE || kind < 2) {
      const float* w = kind == 0 ? ar.wq : ar.wk;
      float wv[8] = {}, wp[8] = {};
      turn<INTER>(ar, cs, e, 1.f, A, B);
      if (e < ar.D) {
        ld8(w + e, wv);
        if constexpr (!INTER) ld8(w + other * 8, wp);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A[j] = mul(A[j], f2(wv[2 * j], wv[2 * j + 1]));
        B[j] = mul(B[j], INTER ? f2(wv[2 * j + 1], wv[2 * j]) : f2(wp[2 * j], wp[2 * j + 1]));
      }
    }
    int h = run.i * U * RPL + lane / LPR;
    int end = e < ar.D ? (kind == 0 ? ar.Hq : ar.Hk) : 0;
    if (CACHE && kind > 0 && dst < 0) end = 0;
    T* out = reinterpret_cast<T*>(kind == 0 ? ar.q_out : kind == 1 ? ar.k_out : ar.v_out) +
             ((kind == 0 ? (int64_t)run.n * ar.Hq : dst * ar.Hk) + h) * ar.D + e;
#pragma unroll 1
    for (unsigned i = 0; i < count; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
      __syncwarp();  // every lane's part has arrived, and the stage before this one is read
      ld.issue(ar, sh, stage == 0 ? NST - 1 : stage - 1);
      const T* in = ring + stage * U * SE;
      stage = stage == NST - 1 ? 0 : stage + 1;
      F2 v[U][4];
      float ss[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        get(in + u * SE + mine, v[u]);
        F2 sq = mul(v[u][0], v[u][0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) sq = fma(v[u][j], v[u][j], sq);
        const float2 s2 = un(sq);
        ss[u] = s2.x + s2.y;
      }
      if (!CACHE || kind < 2) {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          F2 y[4];
          if constexpr (INTER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 a = un(v[u][j]);
              y[j] = f2(a.y, a.x);
            }
          } else {
            get(in + u * SE + theirs, y);
          }
          const float f = rsqrtf(fmaf(ss[u], ar.inv_d, ar.eps));
          const F2 ff = f2(f, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[u][j] = mul(fma(y[j], B[j], mul(v[u][j], A[j])), ff);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * RPL < end) put(out + u * RPL * ar.D, v[u]);
      h += U * RPL;
      out += U * RPL * ar.D;
    }
  }
}

// dx = f w dn - x f^3 sum(dn x w) / D,  dw += f dn x  with dn the turned dy.  The ring's stages
// hold a group's rows of x and dy; a warp keeps its lanes' dwq, dwk in registers.
template <bool INTER, int LPR, typename T>
__global__ void __launch_bounds__(RO_NT, 2) k_qk_norm_rope_bwd(RopeArgs ar) {
  extern __shared__ __align__(16) char smem[];
  constexpr int U = RO_GU, RPL = 32 / LPR, SE = 32 * 8;
  constexpr int NST = RO_RING / (2 * U * SE * (int)sizeof(T));
  static_assert(NST >= 2, "the stage being read is not the one being filled");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
  const int e = (lane & (LPR - 1)) * 8;
  T* ring = reinterpret_cast<T*>(smem + warp * RO_RING);
  float* cs = reinterpret_cast<float*>(smem + RO_W * RO_RING) + warp * RO_CS;
  const int groups = ar.gq + ar.gk;
  const int other = INTER ? 0 : other_lane(ar, e);
  const int mine = lane * 8, theirs = (lane / LPR * LPR + other) * 8;
  // No before_next(): with the sums' CTAs placed early a call of more than about 150 CTAs took 5 us
  // longer (16001 tokens, 32 + 8 heads of 128: 85.2 against 80.3 us); smaller ones take the same.
  after_previous();
  F2 dw[2][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) dw[0][j] = dw[1][j] = f2(0.f, 0.f);
  const Share sh(ar, groups);
  if (sh.todo > 0) {
    Loader<LPR, U, 2, NST, T> ld;
    ld.run.start(ar, sh);
    ld.todo = sh.todo;
    ld.step = RPL * ar.D;
    ld.ring = ring + mine;
    ld.set(ar);
    Run run = ld.run;
    for (int i = 0; i < NST - 1; ++i) ld.issue(ar, sh, i);
    Angles an;
    an.init(ar, run.n, cs);
    unsigned left = sh.todo;
    int stage = 0;
    F2 C[4], S[4];
    for (int token = -1; left > 0; run.next(ar, sh)) {
      if (run.n != token) {
        token = run.n;
        an.fill(ar, run.behind(sh), cs);
        turn<INTER>(ar, cs, e, -1.f, C, S);
      }
      const int kind = run.kind;
      const unsigned count = min((unsigned)run.left, left);
      left -= count;
      float wv[8] = {};
      if (e < ar.D) ld8((kind == 0 ? ar.wq : ar.wk) + e, wv);
      F2 W[4], d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        W[j] = f2(wv[2 * j], wv[2 * j + 1]);
        d[j] = kind == 0 ? dw[0][j] : dw[1][j];
      }
      const int heads = kind == 0 ? ar.Hq : ar.Hk, end = e < ar.D ? heads : 0;
      int h = run.i * U * RPL + sub;
      T* out = reinterpret_cast<T*>(kind == 0 ? ar.q_out : ar.k_out) +
               ((int64_t)run.n * heads + h) * ar.D + e;
#pragma unroll 1
      for (unsigned i = 0; i < count; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
        __syncwarp();
        ld.issue(ar, sh, stage == 0 ? NST - 1 : stage - 1);
        const T* in = ring + stage * 2 * U * SE;
        stage = stage == NST - 1 ? 0 : stage + 1;
        F2 x[U][4], g[U][4], t[U][4];
        float ss[U], dot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          F2 y[4];
          get(in + 2 * u * SE + mine, x[u]);
          get(in + (2 * u + 1) * SE + mine, g[u]);
          if constexpr (INTER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 a = un(g[u][j]);
              y[j] = f2(a.y, a.x);
            }
          } else {
            get(in + (2 * u + 1) * SE + theirs, y);
          }
          F2 sq = f2(0.f, 0.f), dt = sq;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sq = fma(x[u][j], x[u][j], sq);
            g[u][j] = fma(y[j], S[j], mul(g[u][j], C[j]));  // dn
            t[u][j] = mul(g[u][j], x[u][j]);
            g[u][j] = mul(g[u][j], W[j]);
            dt = fma(g[u][j], x[u][j], dt);
          }
          const float2 s2 = un(sq), d2 = un(dt);
          ss[u] = s2.x + s2.y;
          dot[u] = d2.x + d2.y;
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
            dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
          }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // places past the last head hold zeros: 0 for them, not the 1 / 0 of eps = 0
          const float f = h + u * RPL < heads ? rsqrtf(fmaf(ss[u], ar.inv_d, ar.eps)) : 0.f;
          const float m = -(dot[u] * ar.inv_d) * f * f * f;
          const F2 ff = f2(f, f), mm = f2(m, m);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            d[j] = fma(t[u][j], ff, d[j]);  // zero for lanes without a head
            g[u][j] = fma(x[u][j], mm, mul(g[u][j], ff));
          }
          if (h + u * RPL < end) put(out + u * RPL * ar.D, g[u]);
        }
        h += U * RPL;
        out += U * RPL * ar.D;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kind == 0) dw[0][j] = d[j];
        else dw[1][j] = d[j];
      }
    }
  }
  // this CTA's dwq, dwk: lanes of equal elements, then the warps in order (cs is free now)
  float* red = reinterpret_cast<float*>(smem + RO_W * RO_RING);
  for (int z = 0; z < 2; ++z) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 d = un(z ? dw[1][j] : dw[0][j]);
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        d.x += __shfl_xor_sync(0xffffffffu, d.x, o);
        d.y += __shfl_xor_sync(0xffffffffu, d.y, o);
      }
      if (e < ar.D && sub == 0)
        *reinterpret_cast<float2*>(red + warp * RO_MAXD + e + 2 * j) = d;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < ar.D; c += RO_NT) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < RO_W; ++w) s += red[w * RO_MAXD + c];
      ar.part[((int64_t)blockIdx.x * 2 + z) * ar.D + c] = s;
    }
  }
}

// dwq, dwk = sums over the n_part CTA partials in fp64: 8 columns (one sector) per CTA, thread row
// r adds the partials r, r + 32, ... in order (at most 10, read at once), then the 32 rows in a
// fixed tree.
constexpr int RD_COLS = 8, RD_ROWS = RO_NT / RD_COLS;
constexpr int RD_MOST = (RO_CTAS + RD_ROWS - 1) / RD_ROWS;
__global__ void __launch_bounds__(RO_NT) k_qk_norm_rope_dw(int n_part, int D, const float* part,
                                                           float* dwq, float* dwk) {
  __shared__ double acc[RO_W][RD_COLS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = threadIdx.x % RD_COLS, row = threadIdx.x / RD_COLS;
  const int e = blockIdx.x * RD_COLS + col;  // D is a multiple of 8: e < 2 D
  after_previous();
  before_next();
  float x[RD_MOST];
#pragma unroll
  for (int i = 0; i < RD_MOST; ++i) {
    const int p = row + i * RD_ROWS;
    x[i] = p < n_part ? part[(int64_t)p * 2 * D + e] : 0.f;
  }
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < RD_MOST; ++i) s += x[i];
#pragma unroll
  for (int o = RD_COLS; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane < RD_COLS) acc[warp][lane] = s;
  __syncthreads();
  if (row == 0) {
    s = 0.0;
#pragma unroll
    for (int w = 0; w < RO_W; ++w) s += acc[w][col];
    float* out = e < D ? dwq : dwk;
    if (out) out[e < D ? e : e - D] = (float)s;
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

// Groups of a token's heads; CTAs of a call (a warp has at least one group).
void set_groups(RopeArgs* ar, int u, bool cache) {
  const int rpl = (ar->D > 128 ? 1 : ar->D > 64 ? 2 : 4) * u;
  ar->gq = (ar->Hq + rpl - 1) / rpl;
  ar->gk = (ar->Hk + rpl - 1) / rpl;
  ar->gv = cache ? ar->gk : 0;
}
int64_t ctas_of(const RopeArgs& ar) {
  const int64_t n = (ar.N * (ar.gq + ar.gk + ar.gv) + RO_W - 1) / RO_W;
  return n < RO_CTAS ? n : RO_CTAS;
}

static_assert(RO_SMEM <= 48 * 1024, "above this a kernel has to ask for its shared memory");
template <typename K>
cudaError_t launch(K kernel, const RopeArgs& ar, cudaStream_t st) {
  return launch_behind(kernel, dim3((unsigned)ctas_of(ar)), RO_NT, RO_SMEM, st, ar);
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
gdn_status launch_fwd(RopeArgs& ar, int dtype, cudaStream_t st) {
  set_groups(&ar, RO_FU, CACHE);
  cudaError_t e = cudaSuccess;
  with_types(ar, dtype, [&](auto lpr, auto inter, auto t) {
    e = launch(k_qk_norm_rope_fwd<CACHE, inter(), lpr(), decltype(t)>, ar, st);
  });
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
  return launch_fwd<true>(ar, p->dtype, (cudaStream_t)stream);
}

gdn_status gdn_qk_norm_rope_bwd_workspace_size(const gdn_rope_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  RopeArgs ar;
  gdn_status s = check_problem(p, &ar);
  if (s != GDN_OK) return s;
  set_groups(&ar, RO_GU, false);
  *bytes = (size_t)ctas_of(ar) * 2 * (size_t)ar.D * sizeof(float);
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
  set_groups(&ar, RO_GU, false);
  const int64_t ctas = ctas_of(ar);
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
    cudaError_t e = cudaSuccess;
    with_types(ar, p->dtype, [&](auto lpr, auto inter, auto t) {
      e = launch(k_qk_norm_rope_bwd<inter(), lpr(), decltype(t)>, ar, st);
    });
    if (e != cudaSuccess) return GDN_ERR_CUDA;
  }
  const cudaError_t e =
      launch_behind(k_qk_norm_rope_dw, dim3((unsigned)(2 * ar.D / RD_COLS)), RO_NT, 0, st,
                    (int)ctas, ar.D, (const float*)workspace, ar.Hq ? dwq : nullptr,
                    ar.Hk ? dwk : nullptr);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
