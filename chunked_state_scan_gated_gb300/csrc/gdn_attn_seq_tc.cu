// gdn_attn_seq_tc.cu -- the bf16 kernels of gdn_attn_fwd and gdn_attn_bwd, on tcgen05.
//
// Two kernels serve both directions.  A CTA keeps tiles of 128 rows of its own side in shared
// memory (the M of every product) and streams blocks of the other side through a ring by TMA:
//   k_flash: S = R X1^T;  P = f(S);  acc += P X2
//     forward: R = queries, X1 = keys, X2 = values, P = exp2(S sl - m), with the row's running
//     maximum and sum;  dv: R = keys, X1 = queries, X2 = dO, P = exp2(S sl - lse2)
//   k_slope: S = R1 X1^T;  dP = R2 X2^T;  dS = P (dP - delta);  acc += dS X1 (and acc' += P X2)
//     dq: R = queries, dO, X = keys, values;  dk (and dv): R = keys, values, X = queries, dO
// The gradients of a row have one writer: no atomics, the same bits every time.
//
// S, dP and the accumulators are in TMEM; P (dS) goes back as bf16 over the columns of its S and is
// the A operand of the last product from there, so that the weights never pass through shared
// memory.  X1 and X2 are K-major for S and dP and MN-major for the accumulation: one copy serves
// both.  One thread issues all products, one all copies; the other warps do the softmax, a thread
// per row.
//
// Bound by the tensor cores; the weights' bf16 rounding (2^-9 of a weight, as much as o's own
// rounding adds) is what lets the last product run at their full rate.
#include <cuda.h>
#include <cuda_bf16.h>

#include "gdn_attn_tc.cuh"

namespace gdn {

bool tc_make_map_tokens(CUtensorMap* m, const void* ptr, int64_t N, int64_t stride, int64_t heads,
                        int D, int rows);

namespace seq {
namespace {

constexpr int TR = 128;                     // rows of a tile
constexpr int kSmem = 227 * 1024;
constexpr int kHead = 3072;                 // barriers and row values in front of the tiles
constexpr float kLazy = 8.f;                // log2 units

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Rows [from, to) of a streamed block set to zero: rows of another sequence (or of none) whose
// weights are zero, but which may hold NaN.
template <int NT>
__device__ __forceinline__ void zero_rows(uint8_t* block, int atoms, int atom_bytes, int from,
                                          int to, int tid) {
  for (int i = tid; i < (to - from) * 8 * atoms; i += NT) {
    const int c = i & 7, x = i >> 3, r = from + x % (to - from), at = x / (to - from);
    *reinterpret_cast<uint4*>(block + at * atom_bytes + kmaj_chunk(r, c)) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async();
}

// ------------------------------------------------------------------------- forward and dv

// D <= 128: two tiles share every streamed block, each with one buffer of S: while one tile's
// softmax runs, the tensor cores work for the other.  D = 256: the accumulator of one tile leaves
// room for two buffers of S, which alternate.
template <int D>
struct Flash {
  static constexpr int kTiles = D <= 128 ? 2 : 1;
  static constexpr int kCols = D < 128 ? D : 128;            // columns of a ring stage
  static constexpr int kChunks = D / kCols;                  // stages of a block
  static constexpr int kStage = 128 * kCols * 2;             // bytes
  static constexpr int kAtoms = kCols / 64;
  static constexpr int kTile = TR * D * 2;
  static constexpr int kRaw = (kSmem - kHead - kTiles * kTile) / kStage;
  static constexpr int kStages = kRaw < 8 ? kRaw : 8;
  static constexpr int kThreads = kTiles * 128 + 64;
  static constexpr int kBytes = kHead + kTiles * kTile + kStages * kStage;
};

struct Bars {
  uint64_t r_full, full[10], empty[10], s_full[2], p_full[2], pv[2], o_full[2], drained;
  uint32_t tmem;
  int gave_up;
};
static_assert(sizeof(Bars) <= 512, "");

// A CTA that gave up ends only when its copies have landed: the ring's stages up to `stage` were
// filled in this turn, the others in the one before.
__device__ inline void drain(Bars& bar, int stages, int stage, int turn) {
  mbar_wait(&bar.r_full, 0, nullptr, 0);
  for (int i = 0; i < stages; ++i)
    if (i < stage || turn > 0)
      mbar_wait(&bar.full[i], (i < stage ? turn : turn - 1) & 1, nullptr, 0);
}

template <int D, bool FWD>
__global__ void __launch_bounds__(Flash<D>::kThreads, 1)
    k_flash(const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap m1,
            const __grid_constant__ CUtensorMap m2, SeqArgs a) {
  using F = Flash<D>;
  constexpr int NT = F::kTiles, NC = F::kChunks, ST = F::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars& bar = *reinterpret_cast<Bars*>(sm);
  float* row_values = reinterpret_cast<float*>(sm + 512);  // dv: [tile][2][128] lse2
  uint8_t *own = sm + kHead, *ring = own + NT * F::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&bar.r_full, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.pv[i], 1);
      mbar_init(&bar.o_full[i], 1);
    }
    mbar_init(&bar.drained, 1);
    bar.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  after_previous();
  before_next();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  // columns: S 0 and 1 at 0 and 128, then the accumulators
  auto acc_of = [&](int t) { return tmem + 256 + t * D; };
  auto wait = [&](uint64_t* b, uint32_t parity) { wait_for(b, parity, a.status, &bar.gave_up); };

  if (FWD && blockIdx.x == 0 && tid == 0) check_single(a);
  const int heads = FWD ? a.Hq : a.Hk, hh = blockIdx.x % heads, hk = FWD ? hh / a.G : hh;
  Tile t;
  int n = 0, per = 0;            // iterations; of one query head
  int j0 = 0, lo[2] = {0, 0}, hi[2] = {0, 0};  // blocks: the first, and a tile's [lo, hi)
  const bool some = tile_of<!FWD>(a, blockIdx.x / heads, &t);
  if (some) {
    const int side = FWD ? t.nq : t.nk;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      Tile x = t;
      x.at += i * TR;
      if (x.at >= side) continue;
      if (FWD) {
        hi[i] = (keys_seen(a, x, TR) + 127) / 128;
      } else {
        lo[i] = first_query(a, x) / 128;
        hi[i] = (t.nq + 127) / 128;
        if (lo[i] > hi[i]) lo[i] = hi[i];
      }
    }
    j0 = lo[0];
    per = (FWD && NT == 2 ? max(hi[0], hi[1]) : hi[0]) - j0;
    n = FWD ? per : per * a.G;
  }
  const int xrows = FWD ? t.nk : t.nq, xfirst = FWD ? t.k0 : t.q0;  // the streamed side
  // whether tile i takes part in block j (of the sequence's)
  auto takes = [&](int i, int j) { return j >= lo[i] && j < hi[i]; };
  // the place of an iteration's second operand in the ring, in blocks
  auto place2 = [&](int it) { return NT == 2 || it == n - 1 ? 2 * it + 1 : 2 * it + 2; };

  if (warp == NT * 4 && lane == 0 && n > 0) {
    // ---- copies
    const int row0 = (FWD ? t.q0 : t.k0) + t.at;
    mbar_arrive_expect_tx(&bar.r_full, NT * F::kTile);
    for (int i = 0; i < NT; ++i)
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(own + i * F::kTile + c * 16384, &mr, c * 64, hh, row0 + i * TR, &bar.r_full);
    int stage = 0, turn = 0;
    auto block = [&](const CUtensorMap* m, int g, int j) {
      for (int c = 0; c < NC; ++c) {
        if (turn > 0) wait(&bar.empty[stage], (turn - 1) & 1);
        if (bar.gave_up) return;
        mbar_arrive_expect_tx(&bar.full[stage], F::kStage);
        for (int x = 0; x < F::kAtoms; ++x)
          tma_load_3d(ring + stage * F::kStage + x * 16384, m, c * F::kCols + x * 64,
                      FWD ? hk : hh * a.G + g, xfirst + j * 128, &bar.full[stage]);
        if (++stage == ST) stage = 0, ++turn;
      }
    };
    int g1 = 0, j1 = j0, g2 = 0, j2 = j0;
    auto first = [&]() {
      block(&m1, g1, j1);
      if (++j1 == j0 + per) j1 = j0, ++g1;
    };
    auto second = [&]() {
      block(&m2, g2, j2);
      if (++j2 == j0 + per) j2 = j0, ++g2;
    };
    for (int it = 0; it <= n; ++it) {
      if (NT == 2 && it > 0) second();
      if (it < n) first();
      if (NT == 1 && it > 0) second();
    }
    if (bar.gave_up) drain(bar, ST, stage, turn);
  } else if (warp == NT * 4 + 1 && lane == 0 && n > 0) {
    // ---- products
    const uint32_t base = smem_u32(sm);
    const uint64_t kmaj = sdesc(base, 16, 1024), mnmaj = sdesc(base, 16384, 1024);
    auto at = [&](const uint8_t* p) { return (uint64_t)((smem_u32(p) - base) >> 4); };
    int stage = 0, turn = 0;
    auto next = [&]() {
      if (++stage == ST) stage = 0, ++turn;
    };
    wait(&bar.r_full, 0);
    // 16-row steps of block j that hold rows of the sequence
    auto steps = [&](int j) { return min(8, (xrows - j * 128 + 15) / 16); };
    auto scores = [&](int i, int buf, int c, int j) {  // the contraction's columns c kCols ..
      const uint32_t id = idesc_bf16(128, steps(j) * 16, 0, 0);
#pragma unroll
      for (int k = 0; k < F::kCols / 16; ++k)
        mma_bf16(tmem + buf * 128,
                 kmaj + at(own + i * F::kTile + c * F::kAtoms * 16384) +
                     (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                 kmaj + at(ring + stage * F::kStage) + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                 id, c > 0 || k > 0);
    };
    auto weigh = [&](int i, int buf, int c, int j, bool more) {  // output columns c kCols ..
      const int ks = steps(j);
      for (int k = 0; k < ks; ++k)
        mma_bf16_ts(acc_of(i) + c * F::kCols, tmem + buf * 128 + k * 8,
                    mnmaj + at(ring + stage * F::kStage) + ((k * 2048) >> 4),
                    idesc_bf16(128, F::kCols, 0, 1), more || k > 0);
    };
    if constexpr (NT == 2) {
      int ps[2] = {0, 0};  // weights consumed
      int j = j0;          // of iteration it
      int before = j0;     // of iteration it - 1
      for (int it = 0; it <= n; ++it) {
        const int s2 = stage, t2 = turn;
        if (it > 0) next();
        const int s1 = stage, t1 = turn;
        if (it < n) next();
        const int s_end = stage, t_end = turn;
        if (it > 0) wait(&bar.full[s2], t2 & 1);
        for (int i = 0; i < 2; ++i) {
          if (it > 0 && takes(i, before)) {
            wait(&bar.p_full[i], ps[i] & 1);
            tc_fence_after();
            stage = s2;
            weigh(i, i, 0, before, ps[i] > 0);
            ++ps[i];
            const bool last = FWD ? before == hi[i] - 1 : it == n;
            if (last) mma_commit(&bar.o_full[i]);
          }
          if (it < n && takes(i, j)) {
            wait(&bar.full[s1], t1 & 1);
            stage = s1;
            scores(i, i, 0, j);
            mma_commit(&bar.s_full[i]);
          }
        }
        if (it > 0) mma_commit(&bar.empty[s2]);
        if (it < n) mma_commit(&bar.empty[s1]);
        stage = s_end;
        turn = t_end;
        before = j;
        if (++j == j0 + per) j = j0;
      }
    } else {
      int j = j0, before = j0;
      for (int it = 0; it <= n; ++it) {
        if (it < n) {
          for (int c = 0; c < NC; ++c) {
            wait(&bar.full[stage], turn & 1);
            scores(0, it & 1, c, j);
            mma_commit(&bar.empty[stage]);
            next();
          }
          mma_commit(&bar.s_full[it & 1]);
        }
        if (it > 0) {
          const int w = it - 1;
          wait(&bar.p_full[w & 1], (w >> 1) & 1);
          tc_fence_after();
          for (int c = 0; c < NC; ++c) {
            wait(&bar.full[stage], turn & 1);
            weigh(0, w & 1, c, before, w > 0);
            mma_commit(&bar.empty[stage]);
            next();
          }
          mma_commit(it == n ? &bar.o_full[0] : &bar.pv[w & 1]);
        }
        before = j;
        if (++j == j0 + per) j = j0;
      }
    }
    if (bar.gave_up) {  // products in flight end before the TMEM is given back
      mma_commit(&bar.drained);
      mbar_wait(&bar.drained, 0, nullptr, 0);
    }
  } else if (warp < NT * 4 && some) {
    // ---- softmax: a thread per row
    const int i = warp >> 2, r = tid & 127, at = t.at + i * TR;  // tile, row of it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int off = t.nk - t.nq, first_row = at + (warp & 3) * 32, row = at + r;
    float m = -INFINITY, l = 0.f;  // reference (log2 units) and this row's sum
    float ahead = 0.f;             // dv: the next block's lse2 of query r
    int done = 0, g = 0, j = j0;
    auto value = [&](int gg, int jj) {
      const int q = jj * 128 + r;
      return q < t.nq ? a.lse2[(int64_t)(hh * a.G + gg) * a.Nq + t.q0 + q] : INFINITY;
    };
    if (!FWD && n > 0 && lo[i] < hi[i]) ahead = value(0, lo[i]);
    for (int it = 0; it < n; ++it) {
      const int jj = j, gg = g;
      if (++j == j0 + per) j = j0, ++g;
      if (!takes(i, jj)) continue;
      const int buf = NT == 2 ? i : done & 1, kb = jj * 128;
      const uint32_t parity = NT == 2 ? done & 1 : (done >> 1) & 1;
      float* lv = row_values + (i * 2 + (done & 1)) * 128;
      if (!FWD) {
        lv[r] = ahead;
        bar_sync(1 + i, 128);
        if (it + 1 < n) ahead = jj + 1 < hi[i] ? value(gg, jj + 1) : value(gg + 1, lo[i]);
      }
      wait(&bar.s_full[buf], parity);
      tc_fence_after();
      float s[128];
      tmem_ld128(tmem + lanes + buf * 128, s);
      // columns [c0, c1) of the row count
      int c0 = 0, c1 = 128;
      bool whole;
      if (FWD) {
        c1 = (a.causal ? min(t.nk, row + off + 1) : t.nk) - kb;
        whole = kb + 128 <= (a.causal ? min(t.nk, first_row + off + 1) : t.nk);
      } else {
        c1 = t.nq - kb;
        if (a.causal) c0 = row - off - kb;
        whole = kb + 128 <= t.nq && (!a.causal || first_row + 31 - off <= kb);
      }
      if (!whole) {
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = c >= c0 && c < c1 ? s[c] : -INFINITY;
      }
      uint32_t p[64];
      if (FWD) {
        float mx = s[0];
#pragma unroll
        for (int c = 1; c < 128; ++c) mx = fmaxf(mx, s[c]);
        mx *= a.sl;
        // The reference follows the maximum only when a score is above it by kLazy: weights up to
        // 2^kLazy lose nothing, and the accumulator stays where it is for most blocks.
        const bool up = mx > m + kLazy;
        if (__any_sync(0xffffffffu, up)) {
          const float to = up ? mx : m, f = up ? ex2(m - to) : 1.f;
          l *= f;
          m = to;
          if (done > 0) {
            if (NT == 1) wait(&bar.pv[(done - 1) & 1], ((done - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float x[32];
              tmem_ld32(acc_of(i) + lanes + c, x);
              uint32_t y[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(x[e] * f);
              tmem_st32(acc_of(i) + lanes + c, y);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const float x = ex2(fmaf(s[c], a.sl, -base)), y = ex2(fmaf(s[c + 1], a.sl, -base));
          sum0 += x;
          sum1 += y;
          p[c / 2] = bf16x2(x, y);
        }
        l += sum0 + sum1;
      } else {
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          const float4 v = *reinterpret_cast<const float4*>(lv + c);
          const float x = ex2(fmaf(s[c], a.sl, -v.x)), y = ex2(fmaf(s[c + 1], a.sl, -v.y));
          const float z = ex2(fmaf(s[c + 2], a.sl, -v.z)), w = ex2(fmaf(s[c + 3], a.sl, -v.w));
          p[c / 2] = bf16x2(x, y);
          p[c / 2 + 1] = bf16x2(z, w);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = p[h * 32 + e];
        tmem_st32(tmem + lanes + buf * 128 + h * 32, y);
      }
      if (kb + 128 > xrows && (xrows & 15)) {  // rows behind the sequence in its last 16
        const int from = xrows - kb, to = (from + 15) & ~15;
        for (int c = 0; c < NC; ++c) {
          const int x = place2(it) * NC + c;
          wait(&bar.full[x % ST], (x / ST) & 1);
          zero_rows<128>(ring + (x % ST) * F::kStage, F::kAtoms, 16384, from, to, r);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[buf]);
      ++done;
    }
    // ---- the row's result
    if (done > 0) {
      wait(&bar.o_full[i], 0);
      tc_fence_after();
    }
    const int side = FWD ? t.nq : t.nk;
    const int64_t out = (int64_t)((FWD ? t.q0 : t.k0) + row) * heads + hh;
    const float f = FWD ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(FWD ? a.out : a.dv) + out * D;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float x[32];
      if (done > 0) {
        tmem_ld32(acc_of(i) + lanes + c, x);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = 0.f;
      }
      if (row < side)
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4*>(dst + c + e) =
              make_uint4(bf16x2(x[e] * f, x[e + 1] * f), bf16x2(x[e + 2] * f, x[e + 3] * f),
                         bf16x2(x[e + 4] * f, x[e + 5] * f), bf16x2(x[e + 6] * f, x[e + 7] * f));
    }
    if (FWD && a.lse && row < side)
      a.lse[out] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------- dq, dk (and dv)

// Blocks of 128 rows of the streamed side; of 64 with D = 256, whose own tiles take 128 KB.
template <int D>
struct Slope {
  static constexpr int kBlock = D == 256 ? 64 : 128;
  static constexpr int kStage = kBlock * D * 2;
  static constexpr int kAtom = kBlock * 128;  // bytes of 64 columns
  static constexpr int kTile = TR * D * 2;
  static constexpr int kRaw = (kSmem - kHead - 2 * kTile) / kStage;
  static constexpr int kStages = kRaw < 8 ? kRaw : 8;
  // Three stages only (D = 256): two for X1 and one for X2, in place of one ring for both; S is
  // then issued by a thread of its own, as its X1 arrives last.
  static constexpr bool kTight = kStages < 4;
  static constexpr int kThreads = 256 + (kTight ? 96 : 64);
  static constexpr int kBytes = kHead + 2 * kTile + kStages * kStage;
  // stage and parity of operand x (0: X1, 1: X2) of iteration it
  static __device__ __forceinline__ int stage(int x, int it) {
    return kTight ? (x ? 2 : it & 1) : (2 * it + x) % kStages;
  }
  static __device__ __forceinline__ uint32_t parity(int x, int it) {
    return (kTight ? (x ? it : it >> 1) : (2 * it + x) / kStages) & 1;
  }
  // whether the stage held something before
  static __device__ __forceinline__ bool used(int x, int it) {
    return kTight ? it >= 2 - x : 2 * it + x >= kStages;
  }
};

// What a call computes: dq of queries; dk of keys; dk and dv of keys, where TMEM has room for both
// accumulators (D <= 128): one pass of four products in place of 3 + 2.
enum Kind { kDq, kDk, kDkv };

// Order of the products.  dq, dk: S 0, dP 0, S 1, then for every block j, once its dS is there:
// dP j+1, the accumulation of j, S j+2.  S has two buffers, dS goes over its own S, dP has one: the
// exponentials of block j+1 need S j+1 alone and run while the tensor cores work on dP j+1.
// dk and dv: S 0, dP 0, then for every block j: once its P is there (over its S) dv's part and
// S j+1, once its dS is there (over its dP) dk's part and dP j+1.
template <int D, int KIND>
__global__ void __launch_bounds__(Slope<D>::kThreads, 1)
    k_slope(const __grid_constant__ CUtensorMap mr1, const __grid_constant__ CUtensorMap mr2,
            const __grid_constant__ CUtensorMap m1, const __grid_constant__ CUtensorMap m2,
            SeqArgs a) {
  using F = Slope<D>;
  constexpr bool DQ = KIND == kDq, BOTH = KIND == kDkv;
  constexpr int BN = F::kBlock, ST = F::kStages, HN = BN / 2;
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars& bar = *reinterpret_cast<Bars*>(sm);
  float* row_values = reinterpret_cast<float*>(sm + 512);  // dk: [2][lse2, delta][BN]
  uint8_t *own = sm + kHead, *ring = own + 2 * F::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&bar.r_full, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&bar.s_full[i], 1);
    mbar_init(&bar.pv[0], 1);      // dP is there
    mbar_init(&bar.p_full[0], 8);  // dS is there, dP has been read
    mbar_init(&bar.p_full[1], 8);  // dk and dv: P is there
    mbar_init(&bar.o_full[0], 1);
    mbar_init(&bar.drained, F::kTight ? 2 : 1);
    bar.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  after_previous();
  before_next();
  __syncthreads();
  tc_fence_after();
  // columns: S (two buffers, or one), dP, the accumulators
  const uint32_t tmem = bar.tmem, t_dp = tmem + (BOTH ? 1 : 2) * BN, t_acc = t_dp + BN;
  auto wait = [&](uint64_t* b, uint32_t parity) { wait_for(b, parity, a.status, &bar.gave_up); };

  const int heads = DQ ? a.Hq : a.Hk, hh = blockIdx.x % heads, hk = DQ ? hh / a.G : hh;
  Tile t;
  int n = 0, per = 0, j0 = 0;
  const bool some = tile_of<!DQ>(a, blockIdx.x / heads, &t);
  if (some) {
    if (DQ) {
      per = (keys_seen(a, t, TR) + BN - 1) / BN;
    } else {
      j0 = first_query(a, t) / BN;
      per = max(0, (t.nq + BN - 1) / BN - j0);
    }
    n = DQ ? per : per * a.G;
  }
  const int xrows = DQ ? t.nk : t.nq, xfirst = DQ ? t.k0 : t.q0;
  if (warp == 8 && lane == 0 && n > 0) {
    const int row0 = (DQ ? t.q0 : t.k0) + t.at;
    mbar_arrive_expect_tx(&bar.r_full, 2 * F::kTile);
    for (int c = 0; c < D / 64; ++c) {
      tma_load_3d(own + c * 16384, &mr1, c * 64, hh, row0, &bar.r_full);
      tma_load_3d(own + F::kTile + c * 16384, &mr2, c * 64, hh, row0, &bar.r_full);
    }
    int g = 0, j = j0, it = 0;
    for (; it < n && !bar.gave_up; ++it) {
      for (int x = 0; x < 2; ++x) {
        const int stage = F::stage(x, it);
        if (F::used(x, it)) wait(&bar.empty[stage], F::parity(x, it) ^ 1);
        mbar_arrive_expect_tx(&bar.full[stage], F::kStage);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(ring + stage * F::kStage + c * F::kAtom, x ? &m2 : &m1, c * 64,
                      DQ ? hk : hh * a.G + g, xfirst + j * BN, &bar.full[stage]);
      }
      if (++j == j0 + per) j = j0, ++g;
    }
    if (bar.gave_up) {  // the copies have to land before the CTA ends
      mbar_wait(&bar.r_full, 0, nullptr, 0);
      for (int i = max(0, it - ST); i < it; ++i)
        for (int x = 0; x < 2; ++x) mbar_wait(&bar.full[F::stage(x, i)], F::parity(x, i), nullptr, 0);
    }
  } else if ((warp == 9 || warp == 10) && lane == 0 && n > 0) {
    const uint32_t base = smem_u32(sm);
    const uint64_t kmaj = sdesc(base, 16, 1024), mnmaj = sdesc(base, F::kAtom, 1024);
    auto at = [&](const uint8_t* p) { return (uint64_t)((smem_u32(p) - base) >> 4); };
    auto steps = [&](int j) { return min(BN / 16, (xrows - j * BN + 15) / 16); };
    wait(&bar.r_full, 0);
    // S (x = 0) or dP (x = 1) of iteration it: the own tile x with the streamed operand x
    auto scores = [&](uint32_t to, int x, int it, int j) {
      const int stage = F::stage(x, it);
      wait(&bar.full[stage], F::parity(x, it));
      const uint32_t id = idesc_bf16(128, steps(j) * 16, 0, 0);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_bf16(to, kmaj + at(own + x * F::kTile) + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                 kmaj + at(ring + stage * F::kStage) +
                     (((k >> 2) * F::kAtom + (k & 3) * 32) >> 4),
                 id, k > 0);
    };
    // an accumulation: the bf16 weights at `w` with the streamed operand x of iteration it, whose
    // last use it is
    auto weigh = [&](uint32_t to, uint32_t w, int x, int it, int j) {
      const int ks = steps(j), stage = F::stage(x, it);
      for (int k = 0; k < ks; ++k)
        mma_bf16_ts(to, w + k * 8,
                    mnmaj + at(ring + stage * F::kStage) + ((k * 2048) >> 4),
                    idesc_bf16(128, D, 0, 1), it > 0 || k > 0);
      mma_commit(&bar.empty[stage]);
    };
    int j = j0;
    auto after = [&](int j) { return j + 1 == j0 + per ? j0 : j + 1; };
    auto score0 = [&](int it, int j) {  // S, in its buffer
      const int buf = BOTH ? 0 : it & 1;
      scores(tmem + buf * BN, 0, it, j);
      mma_commit(&bar.s_full[buf]);
    };
    auto score1 = [&](int it, int j) {  // dP
      scores(t_dp, 1, it, j);
      mma_commit(&bar.pv[0]);
      if (!BOTH) mma_commit(&bar.empty[F::stage(1, it)]);
    };
    if constexpr (BOTH) {
      if (warp == 9) {
        score0(0, j);
        score1(0, j);
        for (int it = 0; it < n; ++it) {
          const int j1 = after(j);
          wait(&bar.p_full[1], it & 1);
          tc_fence_after();
          weigh(t_acc + D, tmem, 1, it, j);
          if (it + 1 < n) score0(it + 1, j1);
          wait(&bar.p_full[0], it & 1);
          tc_fence_after();
          weigh(t_acc, t_dp, 0, it, j);
          if (it + 1 < n) score1(it + 1, j1);
          else mma_commit(&bar.o_full[0]);
          j = j1;
        }
      }
    } else if (F::kTight && warp == 10) {
      // X1 of iteration it comes into the stage of it - 2 once that one's accumulation has ended,
      // which had read the S buffer that is written here
      for (int it = 0; it < n; ++it, j = after(j)) score0(it, j);
    } else if (warp == 9) {
      if (!F::kTight) score0(0, j);
      score1(0, j);
      if (!F::kTight && n > 1) score0(1, after(j));
      for (int it = 0; it < n; ++it) {
        const int j1 = after(j);
        wait(&bar.p_full[0], it & 1);
        tc_fence_after();
        if (it + 1 < n) score1(it + 1, j1);
        weigh(t_acc, tmem + (it & 1) * BN, 0, it, j);
        if (it + 1 == n) mma_commit(&bar.o_full[0]);
        if (!F::kTight && it + 2 < n) score0(it + 2, after(j1));
        j = j1;
      }
    }
    if (bar.gave_up) {
      mma_commit(&bar.drained);
      mbar_wait(&bar.drained, 0, nullptr, 0);
    }
  } else if (warp < 8 && some) {
    // ---- a thread per row and half of the block's columns
    const int half = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int off = t.nk - t.nq, first_row = t.at + (warp & 3) * 32, row = t.at + r;
    float lse2 = INFINITY, delta = 0.f, ahead = 0.f;
    if (DQ && row < t.nq) {
      lse2 = a.lse2[(int64_t)hh * a.Nq + t.q0 + row];
      delta = a.delta[(int64_t)hh * a.Nq + t.q0 + row];
    }
    // dk: thread tid < 2 BN fetches value tid % BN of lse2 or delta, one block ahead
    auto value = [&](int g, int j) {
      const int q = j * BN + tid % BN;
      const float* src = tid < BN ? a.lse2 : a.delta;
      return tid < 2 * BN && q < t.nq ? src[(int64_t)(hh * a.G + g) * a.Nq + t.q0 + q] : 0.f;
    };
    // the weights of this thread's columns, as bf16 over the columns that the row's two threads
    // have read
    auto put = [&](uint32_t to, const float (&x)[HN]) {
      bar_sync(2 + (warp & 3), 64);
      uint32_t y[HN / 2];
#pragma unroll
      for (int e = 0; e < HN / 2; ++e) y[e] = bf16x2(x[2 * e], x[2 * e + 1]);
      if constexpr (HN == 64) tmem_st32(to + lanes + half * 32, y);
      else tmem_st16(to + lanes + half * 16, y);
    };
    auto tell = [&](uint64_t* b) {
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    int g = 0, j = j0;
    if (!DQ && n > 0) ahead = value(0, j0);
    for (int it = 0; it < n; ++it) {
      const int kb = j * BN;
      if (++j == j0 + per) j = j0, ++g;
      float* lv = row_values + (it & 1) * 2 * BN;
      if (!DQ) {
        if (tid < 2 * BN) lv[tid] = ahead;
        bar_sync(1, 256);
        if (it + 1 < n) ahead = value(g, j);
      }
      int c0 = 0, c1;  // columns [c0, c1) of the row count
      bool whole;
      if (DQ) {
        c1 = (a.causal ? min(t.nk, row + off + 1) : t.nk) - kb;
        whole = kb + BN <= (a.causal ? min(t.nk, first_row + off + 1) : t.nk);
      } else {
        c1 = t.nq - kb;
        if (a.causal) c0 = row - off - kb;
        whole = kb + BN <= t.nq && (!a.causal || first_row + 31 - off <= kb);
      }
      auto mask = [&](float (&x)[HN]) {
        if (whole) return;
#pragma unroll
        for (int c = 0; c < HN; ++c)
          x[c] = half * HN + c >= c0 && half * HN + c < c1 ? x[c] : 0.f;
      };
      // rows of a block behind the sequence, in its last 16
      const bool ragged = kb + BN > xrows && (xrows & 15);
      auto zero = [&](int x) {
        if (!ragged) return;
        const int stage = F::stage(x, it);
        if (x) wait(&bar.full[stage], F::parity(x, it));  // X2: dP may not have read it yet
        zero_rows<256>(ring + stage * F::kStage, D / 64, F::kAtom, xrows - kb,
                       (xrows - kb + 15) & ~15, tid);
      };
      const int buf = BOTH ? 0 : it & 1;
      const uint32_t ts = tmem + buf * BN;
      wait(&bar.s_full[buf], (BOTH ? it : it >> 1) & 1);
      tc_fence_after();
      float s[HN], dp[HN];
      if constexpr (HN == 64) tmem_ld64(ts + lanes + half * HN, s);
      else tmem_ld32(ts + lanes + half * HN, s);
#pragma unroll
      for (int c = 0; c < HN; c += 4) {
        float4 v = make_float4(lse2, lse2, lse2, lse2);
        if (!DQ) v = *reinterpret_cast<const float4*>(lv + half * HN + c);
        s[c] = ex2(fmaf(s[c], a.sl, -v.x));
        s[c + 1] = ex2(fmaf(s[c + 1], a.sl, -v.y));
        s[c + 2] = ex2(fmaf(s[c + 2], a.sl, -v.z));
        s[c + 3] = ex2(fmaf(s[c + 3], a.sl, -v.w));
      }
      if (BOTH) {
        mask(s);
        put(ts, s);
        zero(1);
        tell(&bar.p_full[1]);
      }
      wait(&bar.pv[0], it & 1);
      tc_fence_after();
      if constexpr (HN == 64) tmem_ld64(t_dp + lanes + half * HN, dp);
      else tmem_ld32(t_dp + lanes + half * HN, dp);
#pragma unroll
      for (int c = 0; c < HN; c += 4) {
        float4 v = make_float4(delta, delta, delta, delta);
        if (!DQ) v = *reinterpret_cast<const float4*>(lv + BN + half * HN + c);
        s[c] *= dp[c] - v.x;
        s[c + 1] *= dp[c + 1] - v.y;
        s[c + 2] *= dp[c + 2] - v.z;
        s[c + 3] *= dp[c + 3] - v.w;
      }
      mask(s);
      put(BOTH ? t_dp : ts, s);
      zero(0);
      tell(&bar.p_full[0]);
    }
    if (n > 0) {
      wait(&bar.o_full[0], 0);
      tc_fence_after();
    }
    const int side = DQ ? t.nq : t.nk;
    const int64_t out = ((int64_t)((DQ ? t.q0 : t.k0) + row) * heads + hh) * D;
#pragma unroll 1
    for (int x0 = 0; x0 < (BOTH ? D : D / 2); x0 += 32) {
      const bool second = BOTH && x0 >= D / 2;  // dv
      const int c = half * (D / 2) + x0 % (D / 2);
      float x[32];
      if (n > 0) {
        tmem_ld32(t_acc + lanes + (second ? D : 0) + c, x);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = 0.f;
      }
      const float f = second ? 1.f : a.scale;
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(DQ ? a.dq : second ? a.dv : a.dk) +
                           out + c;
      if (row < side)
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4*>(dst + e) =
              make_uint4(bf16x2(x[e] * f, x[e + 1] * f), bf16x2(x[e + 2] * f, x[e + 3] * f),
                         bf16x2(x[e + 4] * f, x[e + 5] * f), bf16x2(x[e + 6] * f, x[e + 7] * f));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------- host

template <typename K, typename... M>
cudaError_t launch(K kernel, int64_t grid, int threads, int smem, cudaStream_t st, M... maps_args) {
  if (grid == 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  return launch_behind(kernel, dim3((unsigned)grid), threads, smem, st, maps_args...);
}

// Maps of q, k, v (and dO); rows that do not exist are never loaded (a map of one row of another
// tensor stands in).
struct Maps {
  CUtensorMap q, k, v, d;
};
bool make(CUtensorMap* m, const void* p, int64_t n, int64_t stride, int64_t heads, int D,
          int rows) {
  return tc_make_map_tokens(m, p, n, stride, heads, D, rows);
}

template <int D>
cudaError_t fwd(const SeqArgs& a, cudaStream_t st) {
  CUtensorMap q, k, v;
  if (!make(&q, a.q, a.Nq, a.qs, a.Hq, D, 128)) return cudaErrorInvalidValue;
  k = v = q;
  if (a.Nk > 0 && (!make(&k, a.k, a.Nk, a.ks, a.Hk, D, 128) ||
                   !make(&v, a.v, a.Nk, a.vs, a.Hk, D, 128)))
    return cudaErrorInvalidValue;
  return launch(k_flash<D, true>, (int64_t)a.tq.most * a.Hq, Flash<D>::kThreads,
                Flash<D>::kBytes, st, q, k, v, a);
}

template <int D>
cudaError_t bwd(const SeqArgs& a, cudaStream_t st) {
  constexpr int BN = Slope<D>::kBlock;
  const int64_t os = (int64_t)a.Hq * D;
  CUtensorMap q, d, k, v, qb, db, kb, vb;  // boxes of 128 rows, and of the blocks' rows
  if (a.Nq > 0 && (!make(&q, a.q, a.Nq, a.qs, a.Hq, D, 128) ||
                   !make(&d, a.dO, a.Nq, os, a.Hq, D, 128) ||
                   !make(&qb, a.q, a.Nq, a.qs, a.Hq, D, BN) ||
                   !make(&db, a.dO, a.Nq, os, a.Hq, D, BN)))
    return cudaErrorInvalidValue;
  if (a.Nk > 0 && (!make(&k, a.k, a.Nk, a.ks, a.Hk, D, 128) ||
                   !make(&v, a.v, a.Nk, a.vs, a.Hk, D, 128) ||
                   !make(&kb, a.k, a.Nk, a.ks, a.Hk, D, BN) ||
                   !make(&vb, a.v, a.Nk, a.vs, a.Hk, D, BN)))
    return cudaErrorInvalidValue;
  if (a.Nq == 0) q = d = qb = db = k;
  if (a.Nk == 0) k = v = kb = vb = q;
  if (a.Nk > 0) {
    const int64_t ctas = (int64_t)a.tk.most * a.Hk;
    cudaError_t e = launch(k_slope<D, D == 256 ? kDk : kDkv>, ctas, Slope<D>::kThreads,
                           Slope<D>::kBytes, st, k, v, qb, db, a);
    if (e != cudaSuccess) return e;
    if constexpr (D == 256) {
      e = launch(k_flash<D, false>, ctas, Flash<D>::kThreads, Flash<D>::kBytes, st, k, q, d, a);
      if (e != cudaSuccess) return e;
    }
  }
  if (a.Nq == 0) return cudaSuccess;
  return launch(k_slope<D, kDq>, (int64_t)a.tq.most * a.Hq, Slope<D>::kThreads,
                Slope<D>::kBytes, st, q, d, kb, vb, a);
}

}  // namespace

TcPlan tc_plan(int D) {
  const int two = D == 64 ? Flash<64>::kTiles : D == 128 ? Flash<128>::kTiles : Flash<256>::kTiles;
  return TcPlan{two * TR, TR, TR};
}
cudaError_t launch_fwd_tc(const SeqArgs& a, int D, cudaStream_t st) {
  return D == 64 ? fwd<64>(a, st) : D == 128 ? fwd<128>(a, st) : fwd<256>(a, st);
}
cudaError_t launch_bwd_tc(const SeqArgs& a, int D, cudaStream_t st) {
  return D == 64 ? bwd<64>(a, st) : D == 128 ? bwd<128>(a, st) : bwd<256>(a, st);
}

}  // namespace seq
}  // namespace gdn
