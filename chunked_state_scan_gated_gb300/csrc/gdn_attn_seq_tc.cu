// gdn_attn_seq_tc.cu -- the bf16 kernels of gdn_attn_fwd and gdn_attn_bwd, on tcgen05.
//
// A CTA (k_slope_pair: a pair) keeps tiles of 128 rows of its own side in shared memory (the M of every
// product) and streams blocks of 128 rows of the other side through a ring by TMA:
//   k_flash: S = R X1^T;  P = f(S);  acc += P X2
//     forward: R = queries, X1 = keys, X2 = values, P = exp2(S sl - m), with the row's running
//     maximum and sum;  dv (D = 256): R = keys, X1 = queries, X2 = dO, P = exp2(S sl - lse2)
//   k_slope (D <= 128), k_slope_pair (D = 256): S = R1 X1^T;  dP = R2 X2^T;  dS = P (dP - delta);
//     acc += dS X1 (and acc' += P X2)
//     dq: R = queries, dO, X = keys, values;  dk (D <= 128: and dv): R = keys, values, X = queries, dO
// The gradients of a row have one writer: no atomics, the same bits every time.
//
// S, dP and the accumulators are in TMEM; P (dS) goes back as bf16 over the columns of its S and is
// the A operand of the last product from there, so that the weights never pass through shared
// memory.  X1 and X2 are K-major for S and dP and MN-major for the accumulation: one copy serves
// both (the pair's halves differ between the two, so X1 comes twice there).  One thread issues all
// products, one all copies, one warp finds the next items, four write results; eight do the softmax, a
// thread per row or half of one.
//
// Bound by the tensor cores and, in long calls, by the chip's power (16384 tokens, 32 heads on 8 of 128,
// causal: forward 1.30 ms = 1.69 PFLOP/s, backward 4.73 ms; 16 on 2 of 256: 1.27 and 6.00); the weights'
// bf16 rounding (2^-9 of a weight, as much as o's own rounding adds) is what lets the last product run
// at their full rate.
#include <cuda.h>
#include <cuda_bf16.h>

#include "gdn_attn_tc.cuh"

namespace gdn {

bool tc_make_map_tokens(CUtensorMap* m, const void* ptr, int64_t N, int64_t stride, int64_t heads,
                        int D, int rows, int pack);

namespace seq {
namespace {

constexpr int TR = 128;                     // rows of a tile
constexpr int kSmem = 227 * 1024;
constexpr int kHead = 3 * 1024;             // barriers and row values in front of the tiles
constexpr float kLazy = 8.f;                // log2 units

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A shared-memory descriptor as its two words: steps along an operand change the low one only.
struct Desc {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Desc(uint64_t d) : lo((uint32_t)d), hi((uint32_t)(d >> 32)) {}
  __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
    return ((uint64_t)hi << 32) | (lo + (bytes >> 4));
  }
};

// K columns of two K-major operands, whose groups of 64 columns are A and B bytes apart.
template <int K, int A, int B>
__device__ __forceinline__ void mma_rows(uint32_t to, const Desc& a, uint32_t a0, const Desc& b,
                                         uint32_t b0, uint32_t id, bool more, uint32_t issue) {
#pragma unroll
  for (int k = 0; k < K / 16; ++k)
    mma_ss(to, a.at(a0 + (k >> 2) * A + (k & 3) * 32), b.at(b0 + (k >> 2) * B + (k & 3) * 32), id,
           k > 0 || more, issue);
}
// Steps [K0, K1) of 16 rows of an MN-major operand (of `steps` in all), weighed with the weights in
// TMEM.
template <int K0, int K1>
__device__ __forceinline__ void mma_weights(uint32_t to, uint32_t w, const Desc& b, uint32_t b0,
                                            uint32_t id, int steps, bool more, uint32_t issue) {
  if (steps >= K1) {
#pragma unroll
    for (int k = K0; k < K1; ++k) mma_ts(to, w + k * 8, b.at(b0 + k * 2048), id, k > 0 || more, issue);
  } else {
#pragma unroll 1
    for (int k = K0; k < steps; ++k)
      mma_ts(to, w + k * 8, b.at(b0 + k * 2048), id, k > 0 || more, issue);
  }
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

// Items on their way to a CTA's warps: one warp finds them (a list's entry and a few divisions, 1 us)
// while the others work on those before.
constexpr int kItemWords = 16;
constexpr int kTakers = 14;  // warps: 8 softmax, 4 results, copies, products
struct Feed {
  alignas(16) int item[2][kItemWords];
  uint64_t full[2], empty[2];
  __device__ __forceinline__ void init() {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kTakers);
    }
  }
};

struct Bars {
  Feed feed;
  uint64_t r_full, r_empty, full[8], empty[8], s_full[2], p_full[2], p_rest[2], pv[2], o_full[2],
      o_empty[2], l_full[2], l_empty[2], drained;
  uint32_t tmem;
  Alive alive;
};
static_assert(sizeof(Bars) <= 512, "");

// A CTA that gave up ends only when its copies have landed: those of its last own tile, and the
// ring's stages, of which those up to `stage` were filled in this turn, the others in the last.
__device__ inline void drain(Bars& bar, int works, int stages, int stage, int turn) {
  if (works > 0) mbar_wait(&bar.r_full, (works - 1) & 1, nullptr, 0);
  for (int i = 0; i < stages; ++i)
    if (i < stage || turn > 0)
      mbar_wait(&bar.full[i], (i < stage ? turn : turn - 1) & 1, nullptr, 0);
}

__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8]) {  // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// 32 columns of an output row, times f, as bf16 or (a part of o, dk or dv) as fp32.  A thread's row is
// far from its neighbour's, so that a store fills a sector of 32 bytes or half of one: by 32 bytes where
// the output's alignment allows it (64 prompts of 250 tokens, 32 on 8 heads: D = 128 forward 99 and 95
// us, D = 256 backward 666 and 645).  Parts are always aligned to 32.
__device__ __forceinline__ void write_row(__nv_bfloat16* dst, const float (&y)[32], float f) {
#pragma unroll
  for (int e = 0; e < 32; e += 16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = bf16x2(y[e + 2 * i] * f, y[e + 2 * i + 1] * f);
    if (((uintptr_t)dst & 31) == 0) {
      store32(dst + e, w);
    } else {
      *reinterpret_cast<uint4*>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(dst + e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}
__device__ __forceinline__ void write_row(float* dst, const float (&y)[32], float f) {
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(y[e + i] * f);
    store32(dst + e, w);
  }
}
// Columns c .. c + 31 of row `row` (of all key rows) of dk (dv: second), of the query heads from
// `head` on.
template <int D>
__device__ __forceinline__ void write_dkv(const SeqArgs& a, bool second, int64_t row, int hk,
                                          int head, int c, const float (&y)[32]) {
  const float f = second ? 1.f : a.scale;
  const int64_t at = (row * a.Hk + hk) * D + c;
  if (a.splits == 1) {
    write_row(reinterpret_cast<__nv_bfloat16*>(second ? a.dv : a.dk) + at, y, f);
  } else {
    const int part = (head - hk * a.G) / (a.G / a.splits);
    write_row((second ? a.part_v : a.part_k) + (int64_t)part * a.Nk * a.Hk * D + at, y, f);
  }
}

// ------------------------------------------------------------------------- forward and dv

// D <= 128: two tiles share every streamed block, each with one buffer of S: while one tile's
// softmax runs, the tensor cores work for the other.  D = 256: the accumulator of one tile leaves
// room for two buffers of S, which alternate.  Two warpgroups do the softmax (one for each tile, or
// for half of the tile's columns each), one writes results, one issues copies and products.
// setmaxnreg: the registers of a thread, which sum up to no more than the launch's.
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
  static constexpr int kThreads = 512;
  static constexpr int kBytes = kHead + kTiles * kTile + kStages * kStage;
  static constexpr int kSoftRegs = 192, kEndRegs = 64, kIssueRegs = 64;  // of 4 x 128
};
template <int N> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// (x, y) = (x, y) m + c, two at once.
__device__ __forceinline__ void fma2(float& x, float& y, float m, float c) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n"
      " mov.b64 d, {%3, %3};\n fma.rn.f32x2 a, a, b, d;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x), "+f"(y) : "f"(m), "f"(c));
}
__device__ __forceinline__ void fma2(float& x, float& y, float m, float c, float d) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n"
      " mov.b64 d, {%3, %4};\n fma.rn.f32x2 a, a, b, d;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x), "+f"(y) : "f"(m), "f"(c), "f"(d));
}
// (x, y) = (x, y) (a + c, b + d)
__device__ __forceinline__ void mul_sum2(float& x, float& y, float a, float b, float c, float d) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n"
      " mov.b64 r, {%4, %5};\n add.rn.f32x2 q, q, r;\n mul.rn.f32x2 p, p, q;\n"
      " mov.b64 {%0, %1}, p;\n}\n"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b), "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}

// One CTA's share of the work: items of the sorted list, in turns that change direction, so that
// the CTAs end together.
struct Turns {
  int round = -1, total, ctas, cta;
  __device__ __forceinline__ explicit Turns(int n, int per = 1)
      : total(n), ctas(gridDim.x / per), cta(blockIdx.x / per) {}
  __device__ __forceinline__ int next() {  // -1: none left
    while (true) {
      ++round;
      const int64_t first = (int64_t)round * ctas;
      if (first >= total) return -1;
      const int64_t i = first + (round & 1 ? ctas - 1 - cta : cta);
      if (i < total) return (int)i;
    }
  }
};

// The finder's side: every item there is, then one with n = -1.  Where the CTA gave up, that one at
// once: all others see it after the same items, so that their barriers of some warps stay matched.
template <typename ITEM>
__device__ __forceinline__ void feed_items(Feed& f, Turns turns, const SeqArgs& a,
                                           Alive& alive) {
  static_assert(sizeof(ITEM) <= sizeof(f.item[0]), "");
  int turn = 0;
  auto put = [&](const ITEM& x) {
    const int s = turn & 1;
    if (turn >= 2) wait_alone(&f.empty[s], ((turn >> 1) - 1) & 1, alive);
    *reinterpret_cast<ITEM*>(f.item[s]) = x;
    mbar_arrive(&f.full[s]);
    alive.moved = clock64();
    ++turn;
  };
  ITEM x;
  for (int idx; !alive.gave_up && (idx = turns.next()) >= 0;)
    if (x.find(a, idx)) put(x);
  x.n = -1;
  put(x);
}
// The others': the next item; false: there is none.  By whole warps, or (ALONE) by one lane.
template <bool ALONE, typename ITEM>
__device__ __forceinline__ bool take_item(Feed& f, int& turn, ITEM& x, Alive& alive) {
  const int s = turn & 1;
  if (!wait_alone(&f.full[s], (turn >> 1) & 1, alive)) return false;
  ++turn;
  x = *reinterpret_cast<const ITEM*>(f.item[s]);
  if (!ALONE) __syncwarp();
  if (ALONE || (threadIdx.x & 31) == 0) mbar_arrive(&f.empty[s]);
  return x.n >= 0;
}

// An item of k_flash: kTiles tiles of one sequence and head (or key head), the blocks that they
// stream and those [lo, hi) that each tile takes.
template <int D, bool FWD>
struct Item {
  using F = Flash<D>;
  Tile t;
  int head, hk;    // the first query head (FWD), the key head
  int part;        // of the keys (FWD)
  int n, per, j0;  // iterations; of one query head; the first block
  int lo0, lo1, hi0, hi1;
  __device__ __forceinline__ int lo(int i) const { return i ? lo1 : lo0; }
  __device__ __forceinline__ int hi(int i) const { return i ? hi1 : hi0; }
  __device__ __forceinline__ bool find(const SeqArgs& a, int idx) {
    part = 0;
    if (FWD && a.parts > 1) {
      part = idx % a.parts;
      idx /= a.parts;
    }
    const int groups = FWD ? a.Hq / a.pack : a.Hk * a.splits, g = idx % groups;
    const int subs = FWD ? 1 : a.tk.rows / TR, tile = idx / groups;
    if (!tile_of<!FWD>(a, tile / subs, &t)) return false;
    if (!FWD) t.at += tile % subs * TR;  // dv: 128 rows of one of the list's tiles
    head = g * (FWD ? a.pack : a.G / a.splits);
    hk = head / a.G;
    const int side = FWD ? t.nq : t.nk, rows = FWD ? TR / a.pack : TR;
    lo0 = lo1 = hi0 = hi1 = 0;
#pragma unroll
    for (int i = 0; i < F::kTiles; ++i) {
      Tile x = t;
      x.at += i * rows;
      if (x.at >= side) continue;
      int from = 0, to;
      if (FWD) {
        to = (keys_seen(a, x, rows) + 127) / 128;
      } else {
        to = (t.nq + 127) / 128;
        from = min(to, first_query(a, x) / 128);
      }
      (i ? lo1 : lo0) = from;
      (i ? hi1 : hi0) = to;
    }
    if (FWD && a.parts > 1) {  // this part's share of the blocks
      const int all = max(hi0, hi1), from = (int)((int64_t)all * part / a.parts);
      const int to = (int)((int64_t)all * (part + 1) / a.parts);
      lo0 = lo1 = from;
      hi0 = max(from, min(hi0, to));
      hi1 = max(from, min(hi1, to));
    }
    j0 = lo0;
    per = max(hi0, hi1) - j0;
    n = FWD ? per : per * (a.G / a.splits);
    return true;
  }
  __device__ __forceinline__ void make_uniform() {
    for (int* v : {&t.q0, &t.nq, &t.k0, &t.nk, &t.at, &n, &per, &j0, &lo0, &lo1, &hi0, &hi1})
      *v = uniform(*v);
  }
  // whether tile i takes block j (of the sequence's)
  __device__ __forceinline__ bool takes(int i, int j) const { return j >= lo(i) && j < hi(i); }
  __device__ __forceinline__ bool works(int i) const { return lo(i) < hi(i); }
  __device__ __forceinline__ int after(int j) const { return j + 1 == j0 + per ? j0 : j + 1; }
};

template <int D, bool FWD>
__global__ void __launch_bounds__(Flash<D>::kThreads, 1)
    k_flash(const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap m1,
            const __grid_constant__ CUtensorMap m2, SeqArgs a) {
  using F = Flash<D>;
  constexpr int NT = F::kTiles, NC = F::kChunks, ST = F::kStages;
  static_assert(FWD || NT == 1, "row_values");
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars& bar = *reinterpret_cast<Bars*>(sm);
  float* row_values = reinterpret_cast<float*>(sm + 512);  // dv: [2][128] -lse2
  float* row_tops = row_values;                            // forward, D = 256: [2][half][128]
  float* row_factors = reinterpret_cast<float*>(sm + (NT == 1 ? 2560 : 512));  // [tile][128] 1 / l
  uint8_t *own = sm + kHead, *ring = own + NT * F::kTile;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, group = warp >> 2;

  if (tid == 32) {
    prefetch_map(&mr);
    prefetch_map(&m1);
    prefetch_map(&m2);
  }
  if (tid == 0) {
    mbar_init(&bar.r_full, 1);
    mbar_init(&bar.r_empty, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.p_rest[i], 4);
      mbar_init(&bar.pv[i], 1);
      mbar_init(&bar.o_full[i], 1);
      mbar_init(&bar.o_empty[i], 4);
      mbar_init(&bar.l_full[i], 4);
      mbar_init(&bar.l_empty[i], 4);
    }
    mbar_init(&bar.drained, 1);
    bar.feed.init();
    bar.alive.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  if (!a.late) after_previous();
  before_next();
  if (tid == 0) bar.alive.moved = clock64();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(bar.tmem);
  // columns: S 0 and 1 at 0 and 128, then the accumulators
  auto acc_of = [&](int t) { return tmem + 256 + t * D; };
  auto wait = [&](uint64_t* b, uint32_t parity) { wait_for(b, parity, bar.alive); };
  if (FWD && blockIdx.x == 0 && tid == 0) check_single(a);
  const int per_tile =
      FWD ? a.Hq / a.pack * a.parts : a.tk.rows / TR * a.Hk * a.splits;  // items
  Item<D, FWD> x;
  int taken = 0;

  if (group == 3) {
    fewer_registers<F::kIssueRegs>();
    if (warp == 12 && lane == 0) {
      // ---- copies
      int stage = 0, turn = 0, works = 0;
      while (take_item<true>(bar.feed, taken, x, bar.alive)) {
        if (x.n == 0) continue;
        const int rows = FWD ? TR / a.pack : TR;
        if (works > 0) wait(&bar.r_empty, (works - 1) & 1);
        if (bar.alive.gave_up) continue;
        ++works;
        mbar_arrive_expect_tx(&bar.r_full, NT * F::kTile);
        for (int i = 0; i < NT; ++i)
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(own + i * F::kTile + c * 16384, &mr, c * 64, FWD ? x.head : x.hk,
                        (FWD ? x.t.q0 : x.t.k0) + x.t.at + i * rows, &bar.r_full);
        auto block = [&](const CUtensorMap* m, int g, int j) {
          for (int c = 0; c < NC; ++c) {
            if (turn > 0) wait(&bar.empty[stage], (turn - 1) & 1);
            if (bar.alive.gave_up) return;
            mbar_arrive_expect_tx(&bar.full[stage], F::kStage);
            for (int y = 0; y < F::kAtoms; ++y)
              tma_load_3d(ring + stage * F::kStage + y * 16384, m, c * F::kCols + y * 64,
                          FWD ? x.hk : x.head + g, (FWD ? x.t.k0 : x.t.q0) + j * 128,
                          &bar.full[stage]);
            if (++stage == ST) stage = 0, ++turn;
            bar.alive.moved = clock64();
          }
        };
        int g1 = 0, j1 = x.j0, g2 = 0, j2 = x.j0;
        auto first = [&]() {
          block(&m1, g1, j1);
          if ((j1 = x.after(j1)) == x.j0) ++g1;
        };
        auto second = [&]() {
          block(&m2, g2, j2);
          if ((j2 = x.after(j2)) == x.j0) ++g2;
        };
        for (int it = 0; it <= x.n; ++it) {
          if (NT == 2 && it > 0) second();
          if (it < x.n) first();
          if (NT == 1 && it > 0) second();
        }
      }
      if (bar.alive.gave_up) drain(bar, works, ST, stage, turn);
    } else if (warp == 13) {
      // ---- products
      const uint32_t issue = elected();
      const uint32_t base = smem_u32(sm);
      const Desc kmaj(sdesc(base, 16, 1024)), mnmaj(sdesc(base, 16384, 1024));
      constexpr uint32_t kOwn = kHead, kRing = kHead + NT * F::kTile;
      int stage = 0, turn = 0, works = 0;  // works: items that have blocks
      int filled[2] = {0, 0};              // items of which a tile has some
      // tile i's accumulator has been read, if it held something
      auto vacant = [&](int i) {
        if (filled[i] > 0) wait(&bar.o_empty[i], (filled[i] - 1) & 1);
        ++filled[i];
      };
      int weights[2] = {0, 0}, scored = 0;  // parities of a tile's weights; blocks (NT = 1)
      auto next = [&]() {
        if (++stage == ST) stage = 0, ++turn;
      };
      while (take_item<false>(bar.feed, taken, x, bar.alive)) {
        x.make_uniform();
        if (x.n == 0) continue;
        const int xrows = FWD ? x.t.nk : x.t.nq;
        wait(&bar.r_full, works & 1);
        ++works;
        // 16-row steps of block j that hold rows of the sequence
        auto steps = [&](int j) { return min(8, (xrows - j * 128 + 15) / 16); };
        auto scores = [&](int i, int buf, int c, int j) {  // the contraction's columns c kCols ..
          mma_rows<F::kCols, 16384, 16384>(tmem + buf * 128, kmaj,
                                           kOwn + i * F::kTile + c * F::kAtoms * 16384, kmaj,
                                           kRing + stage * F::kStage,
                                           idesc_bf16(128, steps(j) * 16, 0, 0), c > 0, issue);
        };
        // output columns c kCols .., by the first half of the weights or the rest
        constexpr uint32_t kId = idesc_bf16(128, F::kCols, 0, 1);
        auto weigh0 = [&](int i, int buf, int c, int ks, bool more) {
          mma_weights<0, 4>(acc_of(i) + c * F::kCols, tmem + buf * 128, mnmaj,
                            kRing + stage * F::kStage, kId, ks, more, issue);
        };
        auto weigh1 = [&](int i, int buf, int c, int ks) {
          mma_weights<4, 8>(acc_of(i) + c * F::kCols, tmem + buf * 128, mnmaj,
                            kRing + stage * F::kStage, kId, ks, true, issue);
        };
        if constexpr (NT == 2) {
          // forward: tile i takes the first last[i] blocks; the ring holds K 0, V 0, K 1, V 1, ..
          const int last[2] = {x.hi0 - x.j0, x.hi1 - x.j0};
          auto score = [&](int i, int it) {
            scores(i, i, 0, x.j0 + it);
            commit_to(&bar.s_full[i], issue);
          };
          wait(&bar.full[stage], turn & 1);
          if (last[0] > 0) score(0, 0);
          if (last[1] > 0) score(1, 0);
          commit_to(&bar.empty[stage], issue);
          if (x.n == 1) commit_to(&bar.r_empty, issue);
          next();
          if (last[0] > 0) vacant(0);
          if (last[1] > 0) vacant(1);
          for (int it = 0; it < x.n; ++it) {
            const int sv = stage, ks = steps(x.j0 + it);
            wait(&bar.full[sv], turn & 1);
            next();
            const int sk = stage, tk = turn;
            const bool ahead = it + 1 < x.n;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (it >= last[i]) continue;
              wait(&bar.p_full[i], weights[i]);
              tc_fence_after();
              stage = sv;
              weigh0(i, i, 0, ks, it > 0);
              wait(&bar.p_rest[i], weights[i]);
              weights[i] ^= 1;
              tc_fence_after();
              weigh1(i, i, 0, ks);
              if (it + 1 < last[i]) {
                wait(&bar.full[sk], tk & 1);
                stage = sk;
                score(i, it + 1);
              } else {
                commit_to(&bar.o_full[i], issue);
              }
            }
            commit_to(&bar.empty[sv], issue);
            stage = sk;
            if (ahead) {
              commit_to(&bar.empty[sk], issue);
              if (it + 2 == x.n) commit_to(&bar.r_empty, issue);
              next();
            }
          }
        } else {
          // the ring holds X1 0, X1 1, X2 0, X1 2, X2 1, ..
          int ahead = x.j0, j = x.j0;  // blocks of the next S and of the next accumulation
          auto score = [&](int it) {
            const int buf = (scored + it) & 1;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              wait(&bar.full[stage], turn & 1);
              scores(0, buf, c, ahead);
              commit_to(&bar.empty[stage], issue);
              next();
            }
            commit_to(&bar.s_full[buf], issue);
            if (it == x.n - 1) commit_to(&bar.r_empty, issue);
            ahead = x.after(ahead);
          };
          score(0);
          if (x.n > 1) score(1);
          vacant(0);
          for (int it = 0; it < x.n; ++it) {
            const int w = scored + it, buf = w & 1, ks = steps(j);
            wait(&bar.p_full[buf], (w >> 1) & 1);
            wait(&bar.p_rest[buf], (w >> 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              wait(&bar.full[stage], turn & 1);
              mma_weights<0, 8>(acc_of(0) + c * F::kCols, tmem + buf * 128, mnmaj,
                                kRing + stage * F::kStage, kId, ks, it > 0, issue);
              commit_to(&bar.empty[stage], issue);
              next();
            }
            commit_to(&bar.pv[buf], issue);
            if (it == x.n - 1) commit_to(&bar.o_full[0], issue);
            if (it + 2 < x.n) score(it + 2);
            j = x.after(j);
          }
          scored += x.n;
        }
      }
      if (bar.alive.gave_up) {  // products in flight end before the TMEM is given back
        commit_to(&bar.drained, issue);
        mbar_wait(&bar.drained, 0, nullptr, 0);
      }
    } else if (warp == 14 && lane == 0) {
      feed_items<Item<D, FWD>>(bar.feed, Turns(tiles_there<!FWD>(a) * per_tile), a, bar.alive);
    }
  } else if (group == 2) {
    // ---- results: a thread per row
    fewer_registers<F::kEndRegs>();
    const int r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int items = 0, works[2] = {0, 0};
    while (take_item<false>(bar.feed, taken, x, bar.alive)) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int row = FWD ? x.t.at + (i * TR + r) / a.pack : x.t.at + i * TR + r;
        const int side = FWD ? x.t.nq : x.t.nk;
        const int64_t out =
            (int64_t)(x.t.q0 + row) * a.Hq + x.head + (a.pack > 1 ? r % a.pack : 0);  // forward
        float f = 1.f;
        if (FWD) {
          wait(&bar.l_full[i], items & 1);
          f = row_factors[i * 128 + r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.l_empty[i]);
        }
        const bool work = x.works(i);
        if (work) {
          wait(&bar.o_full[i], works[i] & 1);
          ++works[i];
          tc_fence_after();
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float y[32];
          if (work) {
            tmem_ld32(acc_of(i) + lanes + c, y);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0.f;
          }
          if (c == D - 32 && work) {  // read: the next item may accumulate
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_empty[i]);
          }
          if (row < side) {
            if (FWD && a.parts > 1) write_row(a.part_o + (x.part * a.Nq * a.Hq + out) * D + c, y, f);
            else if (FWD) write_row(reinterpret_cast<__nv_bfloat16*>(a.out) + out * D + c, y, f);
            else write_dkv<D>(a, true, x.t.k0 + row, x.hk, x.head, c, y);
          }
        }
      }
      ++items;
    }
  } else {
    // ---- softmax: a thread per row, or per row and half of its columns
    more_registers<F::kSoftRegs>();
    constexpr int N = NT == 2 ? 128 : 64;  // columns of a thread
    const int i = NT == 2 ? group : 0, half = NT == 2 ? 0 : group;
    const int r = tid & 127;  // row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int items = 0, done = 0;  // done: blocks of the tile so far, of all items
    int placed = 0;           // blocks of the ring in front of this item
    while (take_item<false>(bar.feed, taken, x, bar.alive)) {
      const int rows = FWD ? TR / a.pack : TR, at = x.t.at + i * rows, off = x.t.nk - x.t.nq;
      const int w0 = (warp & 3) * 32;  // the warp's rows: tokens first .. last
      const int first = FWD ? at + w0 / a.pack : at + w0;
      const int last = FWD ? at + (w0 + 31) / a.pack : first + 31;
      const int row = FWD ? at + r / a.pack : at + r;
      const int xrows = FWD ? x.t.nk : x.t.nq;
      float m = -INFINITY, l = 0.f;  // reference (log2 units) and the sum of this thread's weights
      float ahead = 0.f;             // dv: the next block's lse2 of query r
      auto value = [&](int g, int j) {
        const int q = j * 128 + r;
        return q < x.t.nq ? a.lse2[(int64_t)(x.head + g) * a.Nq + x.t.q0 + q] : INFINITY;
      };
      if (!FWD && x.n > 0) ahead = value(0, x.lo(i));
      int g = 0, j = x.j0;
      bool begun = false;
      for (int it = 0; it < x.n; ++it) {
        const int jj = j;
        if ((j = x.after(j)) == x.j0) ++g;
        if (!x.takes(i, jj)) continue;
        const int buf = NT == 2 ? i : done & 1, kb = jj * 128;
        const uint32_t parity = NT == 2 ? done & 1 : (done >> 1) & 1;
        const uint32_t ts = tmem + lanes + buf * 128;
        float* lv = row_values + (done & 1) * 128;
        if (!FWD) {
          if (half == 0) lv[r] = -ahead;
          bar_sync(1, 256);
          if (it + 1 < x.n) ahead = value(g, j);
        }
        wait(&bar.s_full[buf], parity);
        tc_fence_after();
        float s[N];
        {
          float s0[64];
          tmem_ld_begin(ts + half * 64, s0);
          if constexpr (N == 128) {
            float s1[64];
            tmem_ld_begin(ts + 64, s1);
            tmem_ld_end(s0);
            tmem_ld_end(s1);
#pragma unroll
            for (int c = 0; c < 64; ++c) s[64 + c] = s1[c];
          } else {
            tmem_ld_end(s0);
          }
#pragma unroll
          for (int c = 0; c < 64; ++c) s[c] = s0[c];
        }
        // columns [c0, c1) of the row count
        int c0 = 0, c1 = 128;
        bool whole;
        if (FWD) {
          c1 = (a.causal ? min(x.t.nk, row + off + 1) : x.t.nk) - kb;
          whole = kb + 128 <= (a.causal ? min(x.t.nk, first + off + 1) : x.t.nk);
        } else {
          c1 = x.t.nq - kb;
          if (a.causal) c0 = row - off - kb;
          whole = kb + 128 <= x.t.nq && (!a.causal || last - off <= kb);
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < N; ++c)
            s[c] = half * 64 + c >= c0 && half * 64 + c < c1 ? s[c] : -INFINITY;
        }
        float base = 0.f, sum0 = 0.f, sum1 = 0.f, sum2 = 0.f, sum3 = 0.f;
        if (FWD) {
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < N - 4; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], s[c + e]), s[c + e + 4]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[N - 4 + e]);
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.sl;
          if constexpr (NT == 1) {  // the other half's; both halves of S have been read then
            float* tops = row_tops + (done & 1) * 256;
            tops[half * 128 + r] = top;
            bar_sync(1 + (warp & 3), 64);
            top = fmaxf(top, tops[(1 - half) * 128 + r]);
          }
          // The reference follows the maximum only when a score is above it by kLazy: weights up
          // to 2^kLazy lose nothing, and the accumulator stays where it is for most blocks.
          const bool up = top > m + kLazy;
          if (__any_sync(0xffffffffu, up)) {
            const float to = up ? top : m, f = up ? ex2(m - to) : 1.f;
            l *= f;
            m = to;
            if (begun) {
              if (NT == 1) wait(&bar.pv[(done - 1) & 1], ((done - 1) >> 1) & 1);
              tc_fence_after();
#pragma unroll 1
              for (int c = half * (D / 2); c < (NT == 1 ? (half + 1) * (D / 2) : D); c += 16) {
                float y[16];
                uint32_t z[16];
                tmem_ld16(acc_of(i) + lanes + c, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(y[e] * f);
                tmem_st16(acc_of(i) + lanes + c, z);
              }
            }
          }
          base = m == -INFINITY ? 0.f : m;
        } else {
          bar_sync(2 + (warp & 3), 64);  // both halves of S have been read
        }
        if (kb + 128 > xrows && (xrows & 15)) {  // rows behind the sequence in its last 16
          const int from = xrows - kb, to = (from + 15) & ~15;
          // D = 256: a stage's wait below is for one turn of the ring, so the turn before has to be
          // over, which it is once the block before has been accumulated (with two tiles that came
          // before this block's scores)
          if (NT == 1 && done > 0) wait(&bar.pv[(done - 1) & 1], ((done - 1) >> 1) & 1);
          const int place = placed + (NT == 2 || it == x.n - 1 ? 2 * it + 1 : 2 * it + 2);
          for (int c = 0; c < NC; ++c) {
            const int y = place * NC + c;
            wait(&bar.full[y % ST], (y / ST) & 1);
            zero_rows<NT == 2 ? 128 : 256>(ring + (y % ST) * F::kStage, F::kAtoms, 16384, from, to,
                                           NT == 2 ? r : tid);
          }
        }
        // the weights, 32 columns at a time; the product begins when the first 64 are there
#pragma unroll
        for (int q = 0; q < N / 32; ++q) {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float* z = s + q * 32 + e;
            if (FWD) {
              fma2(z[0], z[1], a.sl, -base);
              fma2(z[2], z[3], a.sl, -base);
            } else {
              const float4 v = *reinterpret_cast<const float4*>(lv + half * 64 + q * 32 + e);
              fma2(z[0], z[1], a.sl, v.x, v.y);
              fma2(z[2], z[3], a.sl, v.z, v.w);
            }
            z[0] = ex2(z[0]);
            z[1] = ex2(z[1]);
            z[2] = ex2(z[2]);
            z[3] = ex2(z[3]);
            if (FWD) {
              add2(sum0, sum1, z[0], z[1]);
              add2(sum2, sum3, z[2], z[3]);
            }
            y[e / 2] = bf16x2(z[0], z[1]);
            y[e / 2 + 1] = bf16x2(z[2], z[3]);
          }
          tmem_st16(ts + half * 32 + q * 16, y);
          if (q & 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q == 1 && half == 0 ? &bar.p_full[buf] : &bar.p_rest[buf]);
          }
        }
        l += (sum0 + sum1) + (sum2 + sum3);
        begun = true;
        ++done;
      }
      placed += 2 * x.n;
      if (FWD) {
        if constexpr (NT == 1) {  // the other half's sum, with no block left to use the place
          float* tops = row_tops + (done & 1) * 256;
          tops[half * 128 + r] = l;
          bar_sync(1 + (warp & 3), 64);
          l += tops[(1 - half) * 128 + r];
          bar_sync(1 + (warp & 3), 64);
        }
        if (half == 0) {
          if (items > 0) wait(&bar.l_empty[i], (items - 1) & 1);  // the last one's was read
          row_factors[i * 128 + r] = l != 0.f ? 1.f / l : 0.f;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.l_full[i]);
          if (row < x.t.nq) {
            const int64_t out = (int64_t)(x.t.q0 + row) * a.Hq + x.head + r % a.pack;
            const float lse2 = l != 0.f ? m + log2f(l) : -INFINITY;
            if (a.parts > 1) a.part_lse[x.part * a.Nq * a.Hq + out] = lse2;
            else if (a.lse) a.lse[out] = lse2 * kLn2;
          }
        }
      }
      ++items;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && bar.alive.gave_up && a.status) atomicOr(a.status, kStatusTimeout);
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (a.late) after_previous();
}

// ------------------------------------------------------------------------- dq, dk (and dv)

template <int D>
struct Slope {
  static constexpr int kBlock = 128;            // rows of a streamed block
  static constexpr int kStage = kBlock * D * 2;
  static constexpr int kAtom = kBlock * 128;    // bytes of 64 columns
  static constexpr int kTile = TR * D * 2;
  static constexpr int kRaw = (kSmem - kHead - 2 * kTile) / kStage;
  static constexpr int kStages = kRaw < 8 ? kRaw : 8;
  static constexpr int kThreads = 512;
  static constexpr int kBytes = kHead + 2 * kTile + kStages * kStage;
};

// What a launch computes: dq of queries; dk and dv of keys, where TMEM has room for both accumulators
// (D <= 128): one pass of four products in place of 3 + 2; dk of keys.
enum Kind { kDq, kDkv, kDk };

// An item of k_slope: a tile of one sequence and head (or key head), and its iterations.
template <bool DQ, int BN, int ROWS>
struct SlopeItem {
  Tile t;
  int head, hk;    // the (first) query head, the key head
  int n, per, j0;  // iterations; of one query head; the first block
  __device__ __forceinline__ bool find(const SeqArgs& a, int idx) {
    const int groups = DQ ? a.Hq : a.Hk * a.splits, part = idx % groups;
    if (!tile_of<!DQ>(a, idx / groups, &t)) return false;
    head = DQ ? part : part * (a.G / a.splits);
    hk = head / a.G;
    j0 = 0;
    if (DQ) {
      per = (keys_seen(a, t, ROWS) + BN - 1) / BN;
    } else {
      j0 = first_query(a, t) / BN;
      per = max(0, (t.nq + BN - 1) / BN - j0);
    }
    n = DQ ? per : per * (a.G / a.splits);
    return true;
  }
  __device__ __forceinline__ void make_uniform() {
    for (int* v : {&t.q0, &t.nq, &t.k0, &t.nk, &t.at, &n, &per, &j0}) *v = uniform(*v);
  }
  __device__ __forceinline__ int after(int j) const { return j + 1 == j0 + per ? j0 : j + 1; }
};

// A place in the ring: stage and parity.
struct Place {
  int stage;
  uint32_t parity;
  template <int N> __device__ __forceinline__ Place on(int by) const {
    Place p{stage + by, parity};
    if (p.stage >= N) p.stage -= N, p.parity ^= 1;
    return p;
  }
};

// Heads of 64 and 128.  Order of the products.  dq: S 0, dP 0, S 1, then for every block j, once its
// dS is there: dP j+1, the accumulation of j, S j+2.  S has two buffers, dS goes over its own S, dP
// has one: the exponentials of block j+1 need S j+1 alone and run while the tensor cores work on
// dP j+1.  dk and dv: S 0, dP 0, then for every block j: once its P is there (over its S) dv's part
// and S j+1, once its dS is there (over its dP) dk's part and dP j+1.
// The warpgroups are those of k_flash; both softmax ones work on the tile, for half of a block's
// columns each.
template <int D, int KIND>
__global__ void __launch_bounds__(Slope<D>::kThreads, 1)
    k_slope(const __grid_constant__ CUtensorMap mr1, const __grid_constant__ CUtensorMap mr2,
            const __grid_constant__ CUtensorMap m1, const __grid_constant__ CUtensorMap m2,
            SeqArgs a) {
  using F = Slope<D>;
  constexpr bool DQ = KIND == kDq;
  constexpr int BN = F::kBlock, ST = F::kStages, HN = BN / 2;
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars& bar = *reinterpret_cast<Bars*>(sm);
  float* row_values = reinterpret_cast<float*>(sm + 512);  // dk: [2][-lse2, -delta][BN]
  uint8_t *own = sm + kHead, *ring = own + 2 * F::kTile;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, group = warp >> 2;

  if (tid == 32) {
    prefetch_map(&mr1);
    prefetch_map(&mr2);
    prefetch_map(&m1);
    prefetch_map(&m2);
  }
  if (tid == 0) {
    mbar_init(&bar.r_full, 1);
    mbar_init(&bar.r_empty, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&bar.s_full[i], 1);
    mbar_init(&bar.pv[0], 1);      // dP is there
    mbar_init(&bar.p_full[0], 8);  // dS is there, dP has been read
    mbar_init(&bar.p_full[1], 8);  // dk and dv: P is there
    mbar_init(&bar.o_full[0], 1);
    mbar_init(&bar.o_empty[0], 4);
    mbar_init(&bar.drained, 1);
    bar.feed.init();
    bar.alive.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  if (!a.late) after_previous();
  before_next();
  if (tid == 0) bar.alive.moved = clock64();
  __syncthreads();
  tc_fence_after();
  // columns: S (two buffers, or one), dP, the accumulators
  const uint32_t tmem = uniform(bar.tmem), t_dp = tmem + (DQ ? 2 : 1) * BN, t_acc = t_dp + BN;
  auto wait = [&](uint64_t* b, uint32_t parity) { wait_for(b, parity, bar.alive); };
  const int per_tile = DQ ? a.Hq : a.Hk * a.splits;  // items
  SlopeItem<DQ, BN, TR> x;
  int taken = 0;
  // X1 0, X2 0, X1 1, X2 1, .. of all items follow each other in the ring
  auto place = [&](int p) { return Place{p % ST, (uint32_t)(p / ST) & 1}; };

  if (group == 3) {
    fewer_registers<64>();
    if (warp == 12 && lane == 0) {
      // ---- copies
      int works = 0, c = 0;
      Place at{0, 0};
      while (take_item<true>(bar.feed, taken, x, bar.alive)) {
        if (x.n == 0) continue;
        const int row0 = (DQ ? x.t.q0 : x.t.k0) + x.t.at;
        if (works > 0) wait(&bar.r_empty, (works - 1) & 1);
        if (bar.alive.gave_up) continue;
        ++works;
        mbar_arrive_expect_tx(&bar.r_full, 2 * F::kTile);
        for (int i = 0; i < D / 64; ++i) {
          tma_load_3d(own + i * 16384, &mr1, i * 64, DQ ? x.head : x.hk, row0, &bar.r_full);
          tma_load_3d(own + F::kTile + i * 16384, &mr2, i * 64, DQ ? x.head : x.hk, row0,
                      &bar.r_full);
        }
        int g = 0, j = x.j0;
        for (int it = 0; it < x.n && !bar.alive.gave_up; ++it, ++c) {
          for (int y = 0; y < 2; ++y) {
            if (2 * c + y >= ST) wait(&bar.empty[at.stage], at.parity ^ 1);
            mbar_arrive_expect_tx(&bar.full[at.stage], F::kStage);
            for (int i = 0; i < D / 64; ++i)
              tma_load_3d(ring + at.stage * F::kStage + i * F::kAtom, y ? &m2 : &m1, i * 64,
                          DQ ? x.hk : x.head + g, (DQ ? x.t.k0 : x.t.q0) + j * BN,
                          &bar.full[at.stage]);
            at = at.template on<ST>(1);
          }
          bar.alive.moved = clock64();
          if ((j = x.after(j)) == x.j0) ++g;
        }
      }
      if (bar.alive.gave_up) {  // the copies have to land before the CTA ends
        if (works > 0) mbar_wait(&bar.r_full, (works - 1) & 1, nullptr, 0);
        for (int p = max(0, 2 * c - ST); p < 2 * c; ++p)
          mbar_wait(&bar.full[place(p).stage], place(p).parity, nullptr, 0);
      }
    } else if (warp == 13) {
      // ---- products
      const uint32_t issue = elected();
      const uint32_t base = smem_u32(sm);
      const Desc kmaj(sdesc(base, 16, 1024)), mnmaj(sdesc(base, F::kAtom, 1024));
      constexpr uint32_t kOwn = kHead, kRing = kHead + 2 * F::kTile;
      int works = 0, c = 0;
      Place p1{0, 0}, p2{1, 0};  // of X1 and X2 of iteration c
      while (take_item<false>(bar.feed, taken, x, bar.alive)) {
        x.make_uniform();
        if (x.n == 0) continue;
        const int xrows = DQ ? x.t.nk : x.t.nq;
        wait(&bar.r_full, works & 1);
        ++works;
        auto steps = [&](int j) { return min(BN / 16, (xrows - j * BN + 15) / 16); };
        // S (y = 0) or dP (y = 1): the own tile y with the streamed operand at `at`
        auto scores = [&](uint32_t to, int y, const Place& at, int j) {
          wait(&bar.full[at.stage], at.parity);
          mma_rows<D, 16384, F::kAtom>(to, kmaj, kOwn + y * F::kTile, kmaj,
                                       kRing + at.stage * F::kStage,
                                       idesc_bf16(128, steps(j) * 16, 0, 0), false, issue);
        };
        // an accumulation: the bf16 weights at `w` with a streamed operand, whose last use it is
        auto weigh = [&](uint32_t to, uint32_t w, const Place& at, int j, bool more) {
          mma_weights<0, BN / 16>(to, w, mnmaj, kRing + at.stage * F::kStage,
                                  idesc_bf16(128, D, 0, 1), steps(j), more, issue);
          commit_to(&bar.empty[at.stage], issue);
        };
        auto next = [&](const Place& p) { return p.template on<ST>(2); };
        // before an item's first accumulation: that of the one before has been read
        auto vacant = [&](int it) {
          if (it == 0 && works > 1) wait(&bar.o_empty[0], works & 1);
        };
        int j = x.j0;
        if constexpr (!DQ) {
          scores(tmem, 0, p1, j);
          commit_to(&bar.s_full[0], issue);
          scores(t_dp, 1, p2, j);
          commit_to(&bar.pv[0], issue);
          if (x.n == 1) commit_to(&bar.r_empty, issue);
          for (int it = 0; it < x.n; ++it, ++c) {
            const int j1 = x.after(j);
            const bool ahead = it + 1 < x.n;
            const Place n1 = next(p1), n2 = next(p2);
            vacant(it);
            wait(&bar.p_full[1], c & 1);
            tc_fence_after();
            weigh(t_acc + D, tmem, p2, j, it > 0);
            if (ahead) {
              scores(tmem, 0, n1, j1);
              commit_to(&bar.s_full[0], issue);
            }
            wait(&bar.p_full[0], c & 1);
            tc_fence_after();
            weigh(t_acc, t_dp, p1, j, it > 0);
            if (ahead) {
              scores(t_dp, 1, n2, j1);
              commit_to(&bar.pv[0], issue);
              if (it + 2 == x.n) commit_to(&bar.r_empty, issue);
            } else {
              commit_to(&bar.o_full[0], issue);
            }
            p1 = n1;
            p2 = n2;
            j = j1;
          }
        } else {
          auto slope = [&](const Place& at, int j) {
            scores(t_dp, 1, at, j);
            commit_to(&bar.pv[0], issue);
            commit_to(&bar.empty[at.stage], issue);
          };
          auto score = [&](int c, const Place& at, int j) {
            scores(tmem + (c & 1) * BN, 0, at, j);
            commit_to(&bar.s_full[c & 1], issue);
          };
          score(c, p1, j);
          slope(p2, j);
          if (x.n == 1) commit_to(&bar.r_empty, issue);
          if (x.n > 1) score(c + 1, next(p1), x.after(j));
          for (int it = 0; it < x.n; ++it, ++c) {
            const int j1 = x.after(j);
            const Place n1 = next(p1), n2 = next(p2);
            vacant(it);
            wait(&bar.p_full[0], c & 1);
            tc_fence_after();
            if (it + 1 < x.n) {
              slope(n2, j1);
              if (it + 2 == x.n) commit_to(&bar.r_empty, issue);
            }
            weigh(t_acc, tmem + (c & 1) * BN, p1, j, it > 0);
            if (it + 1 == x.n) commit_to(&bar.o_full[0], issue);
            if (it + 2 < x.n) score(c, next(n1), x.after(j1));
            p1 = n1;
            p2 = n2;
            j = j1;
          }
        }
      }
      if (bar.alive.gave_up) {
        commit_to(&bar.drained, issue);
        mbar_wait(&bar.drained, 0, nullptr, 0);
      }
    } else if (warp == 14 && lane == 0) {
      feed_items<SlopeItem<DQ, BN, TR>>(bar.feed, Turns(tiles_there<!DQ>(a) * per_tile), a,
                                        bar.alive);
    }
  } else if (group == 2) {
    // ---- results: a thread per row
    fewer_registers<64>();
    const int r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int works = 0;
    while (take_item<false>(bar.feed, taken, x, bar.alive)) {
      const int row = x.t.at + r, side = DQ ? x.t.nq : x.t.nk;
      if (x.n > 0) {
        wait(&bar.o_full[0], works & 1);
        ++works;
        tc_fence_after();
      }
      constexpr int kAll = DQ ? D : 2 * D;
#pragma unroll 1
      for (int c = 0; c < kAll; c += 32) {
        float y[32];
        if (x.n > 0) {
          tmem_ld32(t_acc + lanes + c, y);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = 0.f;
        }
        if (c == kAll - 32 && x.n > 0) {  // read: the next item may accumulate
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.o_empty[0]);
        }
        if (row < side) {
          if (DQ)
            write_row(reinterpret_cast<__nv_bfloat16*>(a.dq) +
                          ((int64_t)(x.t.q0 + row) * a.Hq + x.head) * D + c, y, a.scale);
          else
            write_dkv<D>(a, c >= D, x.t.k0 + row, x.hk, x.head, c >= D ? c - D : c, y);
        }
      }
    }
  } else {
    // ---- a thread per row and half of the block's columns
    more_registers<192>();
    const int half = group, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // the weights of this thread's columns, as bf16 over the columns that the row's two threads
    // have read
    auto put = [&](uint32_t to, const float (&w)[HN]) {
      bar_sync(2 + (warp & 3), 64);
      uint32_t y[HN / 2];
#pragma unroll
      for (int e = 0; e < HN / 2; ++e) y[e] = bf16x2(w[2 * e], w[2 * e + 1]);
      tmem_st32(to + lanes + half * 32, y);
    };
    auto tell = [&](uint64_t* b) {
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    int c = 0;  // iterations of all items
    while (take_item<false>(bar.feed, taken, x, bar.alive)) {
      const int off = x.t.nk - x.t.nq, first_row = x.t.at + (warp & 3) * 32, row = x.t.at + r;
      const int xrows = DQ ? x.t.nk : x.t.nq;
      float lse2 = INFINITY, delta = 0.f, ahead = 0.f;
      if (DQ && row < x.t.nq) {
        lse2 = a.lse2[(int64_t)x.head * a.Nq + x.t.q0 + row];
        delta = a.delta[(int64_t)x.head * a.Nq + x.t.q0 + row];
      }
      // dk, dv: a thread fetches value tid % BN of lse2 or delta, one block ahead
      auto value = [&](int g, int j) {
        const int q = j * BN + tid % BN;
        const float* src = tid < BN ? a.lse2 : a.delta;
        return q < x.t.nq ? src[(int64_t)(x.head + g) * a.Nq + x.t.q0 + q] : 0.f;
      };
      int g = 0, j = x.j0;
      if (!DQ && x.n > 0) ahead = value(0, x.j0);
      for (int it = 0; it < x.n; ++it, ++c) {
        const int kb = j * BN;
        if ((j = x.after(j)) == x.j0) ++g;
        float* lv = row_values + (c & 1) * 2 * BN;
        if (!DQ) {
          lv[tid] = -ahead;
          bar_sync(1, 256);
          if (it + 1 < x.n) ahead = value(g, j);
        }
        int c0 = 0, c1;  // columns [c0, c1) of the row count
        bool whole;
        if (DQ) {
          c1 = (a.causal ? min(x.t.nk, row + off + 1) : x.t.nk) - kb;
          whole = kb + BN <= (a.causal ? min(x.t.nk, first_row + off + 1) : x.t.nk);
        } else {
          c1 = x.t.nq - kb;
          if (a.causal) c0 = row - off - kb;
          whole = kb + BN <= x.t.nq && (!a.causal || first_row + 31 - off <= kb);
        }
        auto mask = [&](float (&w)[HN]) {
          if (whole) return;
#pragma unroll
          for (int e = 0; e < HN; ++e)
            w[e] = half * HN + e >= c0 && half * HN + e < c1 ? w[e] : 0.f;
        };
        // rows of a block behind the sequence, in its last 16
        const bool ragged = kb + BN > xrows && (xrows & 15);
        auto zero = [&](int y) {
          if (!ragged) return;
          const Place at = place(2 * c + y);
          if (y) wait(&bar.full[at.stage], at.parity);  // X2: dP may not have read it yet
          zero_rows<256>(ring + at.stage * F::kStage, D / 64, F::kAtom, xrows - kb,
                         (xrows - kb + 15) & ~15, tid);
        };
        const int buf = DQ ? c & 1 : 0;
        const uint32_t ts = tmem + buf * BN;
        wait(&bar.s_full[buf], (DQ ? c >> 1 : c) & 1);
        tc_fence_after();
        float s[HN], dp[HN];
        tmem_ld64(ts + lanes + half * HN, s);
#pragma unroll
        for (int e = 0; e < HN; e += 4) {
          if (DQ) {
            fma2(s[e], s[e + 1], a.sl, -lse2);
            fma2(s[e + 2], s[e + 3], a.sl, -lse2);
          } else {
            const float4 v = *reinterpret_cast<const float4*>(lv + half * HN + e);
            fma2(s[e], s[e + 1], a.sl, v.x, v.y);
            fma2(s[e + 2], s[e + 3], a.sl, v.z, v.w);
          }
          s[e] = ex2(s[e]);
          s[e + 1] = ex2(s[e + 1]);
          s[e + 2] = ex2(s[e + 2]);
          s[e + 3] = ex2(s[e + 3]);
        }
        if (!DQ) {
          mask(s);
          put(ts, s);
          zero(1);
          tell(&bar.p_full[1]);
        }
        wait(&bar.pv[0], c & 1);
        tc_fence_after();
        tmem_ld64(t_dp + lanes + half * HN, dp);
#pragma unroll
        for (int e = 0; e < HN; e += 4) {
          float4 v = make_float4(-delta, -delta, -delta, -delta);
          if (!DQ) v = *reinterpret_cast<const float4*>(lv + BN + half * HN + e);
          mul_sum2(s[e], s[e + 1], dp[e], dp[e + 1], v.x, v.y);
          mul_sum2(s[e + 2], s[e + 3], dp[e + 2], dp[e + 3], v.z, v.w);
        }
        mask(s);
        put(DQ ? ts : t_dp, s);
        zero(0);
        tell(&bar.p_full[0]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && bar.alive.gave_up && a.status) atomicOr(a.status, kStatusTimeout);
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (a.late) after_previous();
}

// ----------------------------------------------------------------- dq and dk, heads of 256

// A pair of CTAs takes 256 own rows, 128 each, and products of 256 x 128 x 16: each CTA's shared
// memory holds its own rows of both operands (128 KB), half of a block's 128 rows of X1 and X2 for S
// and dP, and half of X1's columns for the accumulation (32 KB each).  With one CTA alone there is
// room for blocks of 64 rows only, whose products take almost as long as those of 128 (59 of 64
// cycles: the first operand's rows have to be read all the same), and for three of them, which is
// too few to hide the copies.
struct Pair {
  static constexpr int D = 256, kBlock = 128;
  static constexpr int kTile = TR * D * 2;  // own rows, of each operand
  static constexpr int kPart = 32 * 1024;   // of X1 and X2 by rows, of X1 by columns
  static constexpr int kThreads = 512;
  static constexpr int kBytes = kHead + 2 * kTile + 3 * kPart;
};
struct PairBars {
  Feed feed;
  uint64_t r_full, r_empty, full[3], empty[3], s_full, dp_full, o_full;  // of this CTA
  uint64_t peer[4], s_read, ds_full, o_empty;  // of the first CTA: what the other's copies bring
                                               // (full[3], r_full), what both have read or written
  uint64_t drained;
  uint32_t tmem;
  Alive alive;
};
static_assert(sizeof(PairBars) <= 512, "");

// Order of the products: S 0, dP 0, then for every block j: S j+1 once S j has been read, the
// accumulation of j once its dS is there (over its dP), dP j+1.  So the tensor cores have S j+1 to do
// while dS j is worked out, and every copy has the time of two products to arrive.
template <int KIND>
__global__ void __launch_bounds__(Pair::kThreads, 1) __cluster_dims__(2, 1, 1)
    k_slope_pair(const __grid_constant__ CUtensorMap mr1, const __grid_constant__ CUtensorMap mr2,
                 const __grid_constant__ CUtensorMap m1, const __grid_constant__ CUtensorMap m2,
                 const __grid_constant__ CUtensorMap m1c, SeqArgs a) {
  using F = Pair;
  constexpr bool DQ = KIND == kDq;
  constexpr int D = F::D, BN = F::kBlock, HN = 64;
  extern __shared__ __align__(1024) uint8_t sm[];
  PairBars& bar = *reinterpret_cast<PairBars*>(sm);
  float* row_values = reinterpret_cast<float*>(sm + 512);  // dk: [2][-lse2, -delta][BN]
  uint8_t *own = sm + kHead, *parts = own + 2 * F::kTile;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, group = warp >> 2;
  const int rank = uniform(pair_rank());

  if (tid == 32) {
    prefetch_map(&mr1);
    prefetch_map(&mr2);
    prefetch_map(&m1);
    prefetch_map(&m2);
    prefetch_map(&m1c);
  }
  if (tid == 0) {
    for (uint64_t* b : {&bar.r_full, &bar.r_empty, &bar.s_full, &bar.dp_full, &bar.o_full,
                        &bar.drained})
      mbar_init(b, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bar.peer[i], 1);
    mbar_init(&bar.s_read, 16);
    mbar_init(&bar.ds_full, 16);
    mbar_init(&bar.o_empty, 8);
    bar.feed.init();
    bar.alive.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 0) pair_tmem_alloc(&bar.tmem);
  tc_fence_before();
  if (!a.late) after_previous();
  before_next();
  if (tid == 0) bar.alive.moved = clock64();
  __syncthreads();
  pair_sync();
  tc_fence_after();
  const uint32_t tmem = uniform(bar.tmem), t_dp = tmem + BN, t_acc = tmem + 2 * BN;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    wait_for<true>(b, parity, bar.alive);
  };
  const int per_tile = DQ ? a.Hq : a.Hk * a.splits;  // items
  SlopeItem<DQ, BN, 2 * TR> x;
  int taken = 0;

  if (group == 3) {
    fewer_registers<64>();
    if (warp == 12 && lane == 0) {
      // ---- copies: parts 0 X1 by rows, 1 X2 by rows, 2 X1 by columns
      int works = 0, c = 0;
      while (take_item<true>(bar.feed, taken, x, bar.alive)) {
        if (x.n == 0) continue;
        const int row0 = (DQ ? x.t.q0 : x.t.k0) + x.t.at + rank * TR;
        if (works > 0) wait(&bar.r_empty, (works - 1) & 1);
        if (bar.alive.gave_up) continue;
        ++works;
        mbar_arrive_expect_tx(&bar.r_full, 2 * F::kTile);
        for (int i = 0; i < D / 64; ++i) {
          tma_load_3d(own + i * 16384, &mr1, i * 64, DQ ? x.head : x.hk, row0, &bar.r_full);
          tma_load_3d(own + F::kTile + i * 16384, &mr2, i * 64, DQ ? x.head : x.hk, row0,
                      &bar.r_full);
        }
        int g = 0, j = x.j0;
        for (int it = 0; it < x.n && !bar.alive.gave_up; ++it, ++c) {
          const int head = DQ ? x.hk : x.head + g, row = (DQ ? x.t.k0 : x.t.q0) + j * BN;
          for (int y = 0; y < 3; ++y) {
            if (c > 0) wait(&bar.empty[y], (c - 1) & 1);
            mbar_arrive_expect_tx(&bar.full[y], F::kPart);
            uint8_t* to = parts + y * F::kPart;
            if (y < 2) {
              for (int i = 0; i < 4; ++i)
                tma_load_3d(to + i * 8192, y ? &m2 : &m1, i * 64, head, row + rank * 64,
                            &bar.full[y]);
            } else {
              for (int i = 0; i < 2; ++i)
                tma_load_3d(to + i * 16384, &m1c, rank * 128 + i * 64, head, row, &bar.full[y]);
            }
          }
          bar.alive.moved = clock64();
          if ((j = x.after(j)) == x.j0) ++g;
        }
      }
      if (bar.alive.gave_up) {  // the copies have to land before the CTA ends
        if (works > 0) mbar_wait(&bar.r_full, (works - 1) & 1, nullptr, 0);
        if (c > 0)
          for (int y = 0; y < 3; ++y) mbar_wait(&bar.full[y], (c - 1) & 1, nullptr, 0);
      }
    } else if (warp == 13 && rank == 1) {
      // ---- tells the first CTA what has arrived here, in the order in which it is used
      int works = 0, c = 0;
      auto tell = [&](uint64_t* b, uint32_t parity, int to) {
        wait(b, parity);
        if (lane == 0) arrive_first(&bar.peer[to]);
      };
      while (take_item<false>(bar.feed, taken, x, bar.alive)) {
        if (x.n == 0) continue;
        tell(&bar.r_full, works & 1, 3);
        ++works;
        const int n = uniform(x.n);
        tell(&bar.full[0], c & 1, 0);
        tell(&bar.full[1], c & 1, 1);
        for (int it = 0; it < n; ++it, ++c) {
          if (it + 1 < n) tell(&bar.full[0], (c + 1) & 1, 0);
          tell(&bar.full[2], c & 1, 2);
          if (it + 1 < n) tell(&bar.full[1], (c + 1) & 1, 1);
        }
      }
    } else if (warp == 13) {
      // ---- products
      const uint32_t issue = elected();
      const uint32_t base = smem_u32(sm);
      const Desc kmaj(sdesc(base, 16, 1024)), mnmaj(sdesc(base, 16384, 1024));
      constexpr uint32_t kOwn = kHead, kParts = kHead + 2 * F::kTile;
      int works = 0, c = 0;
      while (take_item<false>(bar.feed, taken, x, bar.alive)) {
        x.make_uniform();
        if (x.n == 0) continue;
        const int xrows = DQ ? x.t.nk : x.t.nq;
        wait(&bar.r_full, works & 1);
        wait(&bar.peer[3], works & 1);
        ++works;
        // S (y = 0) or dP (y = 1) of iteration c
        auto scores = [&](uint32_t to, int y, int c) {
          wait(&bar.full[y], c & 1);
          wait(&bar.peer[y], c & 1);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            pair_mma_ss(to, kmaj.at(kOwn + y * F::kTile + (k >> 2) * 16384 + (k & 3) * 32),
                        kmaj.at(kParts + y * F::kPart + (k >> 2) * 8192 + (k & 3) * 32),
                        idesc_bf16(256, BN, 0, 0), k > 0, issue);
          pair_commit(&bar.empty[y], issue);
          pair_commit(y ? &bar.dp_full : &bar.s_full, issue);
        };
        int j = x.j0;
        scores(tmem, 0, c);
        scores(t_dp, 1, c);
        if (x.n == 1) pair_commit(&bar.r_empty, issue);
        for (int it = 0; it < x.n; ++it, ++c) {
          const bool ahead = it + 1 < x.n;
          if (ahead) {
            wait(&bar.s_read, c & 1);
            tc_fence_after();
            scores(tmem, 0, c + 1);
          } else {
            wait(&bar.s_read, c & 1);
          }
          if (it == 0 && works > 1) wait(&bar.o_empty, works & 1);  // the item before was read
          wait(&bar.full[2], c & 1);
          wait(&bar.peer[2], c & 1);
          wait(&bar.ds_full, c & 1);
          tc_fence_after();
          const int steps = min(BN / 16, (xrows - j * BN + 15) / 16);
          if (steps == BN / 16) {
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              pair_mma_ts(t_acc, t_dp + k * 8, mnmaj.at(kParts + 2 * F::kPart + k * 2048),
                          idesc_bf16(256, D, 0, 1), it > 0 || k > 0, issue);
          } else {
#pragma unroll 1
            for (int k = 0; k < steps; ++k)
              pair_mma_ts(t_acc, t_dp + k * 8, mnmaj.at(kParts + 2 * F::kPart + k * 2048),
                          idesc_bf16(256, D, 0, 1), it > 0 || k > 0, issue);
          }
          pair_commit(&bar.empty[2], issue);
          if (ahead) {
            scores(t_dp, 1, c + 1);
            if (it + 2 == x.n) pair_commit(&bar.r_empty, issue);
          } else {
            pair_commit(&bar.o_full, issue);
          }
          j = x.after(j);
        }
      }
      if (bar.alive.gave_up) {
        pair_commit(&bar.drained, issue);
        mbar_wait(&bar.drained, 0, nullptr, 0);
      }
    } else if (warp == 14 && lane == 0) {
      feed_items<SlopeItem<DQ, BN, 2 * TR>>(bar.feed, Turns(tiles_there<!DQ>(a) * per_tile, 2), a,
                                            bar.alive);
    }
  } else if (group == 2) {
    // ---- results: a thread per row
    fewer_registers<64>();
    const int r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int works = 0;
    while (take_item<false>(bar.feed, taken, x, bar.alive)) {
      const int row = x.t.at + rank * TR + r, side = DQ ? x.t.nq : x.t.nk;
      if (x.n > 0) {
        wait(&bar.o_full, works & 1);
        ++works;
        tc_fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float y[32];
        if (x.n > 0) {
          tmem_ld32(t_acc + lanes + c, y);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = 0.f;
        }
        if (c == D - 32 && x.n > 0) {  // read: the next item may accumulate
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_first(&bar.o_empty);
        }
        if (row < side) {
          if (DQ)
            write_row(reinterpret_cast<__nv_bfloat16*>(a.dq) +
                          ((int64_t)(x.t.q0 + row) * a.Hq + x.head) * D + c, y, a.scale);
          else
            write_dkv<D>(a, false, x.t.k0 + row, x.hk, x.head, c, y);
        }
      }
    }
  } else {
    // ---- a thread per row and half of the block's columns
    more_registers<192>();
    const int half = group, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int c = 0;  // iterations of all items
    while (take_item<false>(bar.feed, taken, x, bar.alive)) {
      const int off = x.t.nk - x.t.nq, at = x.t.at + rank * TR;
      const int first_row = at + (warp & 3) * 32, row = at + r;
      const int xrows = DQ ? x.t.nk : x.t.nq;
      float lse2 = INFINITY, delta = 0.f, ahead = 0.f;
      if (DQ && row < x.t.nq) {
        lse2 = a.lse2[(int64_t)x.head * a.Nq + x.t.q0 + row];
        delta = a.delta[(int64_t)x.head * a.Nq + x.t.q0 + row];
      }
      // dk: the first 128 threads fetch lse2 of the next block's queries, the others delta
      auto value = [&](int g, int j) {
        const int q = j * BN + r;
        const float* src = half == 0 ? a.lse2 : a.delta;
        return q < x.t.nq ? src[(int64_t)(x.head + g) * a.Nq + x.t.q0 + q] : 0.f;
      };
      int g = 0, j = x.j0;
      if (!DQ && x.n > 0) ahead = value(0, x.j0);
      for (int it = 0; it < x.n; ++it, ++c) {
        const int kb = j * BN;
        if ((j = x.after(j)) == x.j0) ++g;
        float* lv = row_values + (c & 1) * 2 * BN;
        if (!DQ) {
          lv[tid] = -ahead;
          bar_sync(1, 256);
          if (it + 1 < x.n) ahead = value(g, j);
        }
        int c0 = 0, c1;  // columns [c0, c1) of the row count
        bool whole;
        if (DQ) {
          c1 = (a.causal ? min(x.t.nk, row + off + 1) : x.t.nk) - kb;
          whole = kb + BN <= (a.causal ? min(x.t.nk, first_row + off + 1) : x.t.nk);
        } else {
          c1 = x.t.nq - kb;
          if (a.causal) c0 = row - off - kb;
          whole = kb + BN <= x.t.nq && (!a.causal || first_row + 31 - off <= kb);
        }
        wait(&bar.s_full, c & 1);
        tc_fence_after();
        float s[HN], dp[HN];
        tmem_ld64(tmem + lanes + half * HN, s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&bar.s_read);
#pragma unroll
        for (int e = 0; e < HN; e += 4) {
          if (DQ) {
            fma2(s[e], s[e + 1], a.sl, -lse2);
            fma2(s[e + 2], s[e + 3], a.sl, -lse2);
          } else {
            const float4 v = *reinterpret_cast<const float4*>(lv + half * HN + e);
            fma2(s[e], s[e + 1], a.sl, v.x, v.y);
            fma2(s[e + 2], s[e + 3], a.sl, v.z, v.w);
          }
          s[e] = ex2(s[e]);
          s[e + 1] = ex2(s[e + 1]);
          s[e + 2] = ex2(s[e + 2]);
          s[e + 3] = ex2(s[e + 3]);
        }
        wait(&bar.dp_full, c & 1);
        tc_fence_after();
        tmem_ld64(t_dp + lanes + half * HN, dp);
#pragma unroll
        for (int e = 0; e < HN; e += 4) {
          float4 v = make_float4(-delta, -delta, -delta, -delta);
          if (!DQ) v = *reinterpret_cast<const float4*>(lv + BN + half * HN + e);
          mul_sum2(s[e], s[e + 1], dp[e], dp[e + 1], v.x, v.y);
          mul_sum2(s[e + 2], s[e + 3], dp[e + 2], dp[e + 3], v.z, v.w);
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < HN; ++e)
            s[e] = half * HN + e >= c0 && half * HN + e < c1 ? s[e] : 0.f;
        }
        bar_sync(2 + (warp & 3), 64);  // both halves of dP have been read
        uint32_t y[HN / 2];
#pragma unroll
        for (int e = 0; e < HN / 2; ++e) y[e] = bf16x2(s[2 * e], s[2 * e + 1]);
        tmem_st32(t_dp + lanes + half * 32, y);
        if (kb + BN > xrows && (xrows & 15)) {  // rows behind the sequence in its last 16
          wait(&bar.full[2], c & 1);
          zero_rows<256>(parts + 2 * F::kPart, 2, 16384, xrows - kb, (xrows - kb + 15) & ~15, tid);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&bar.ds_full);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && bar.alive.gave_up && a.status) atomicOr(a.status, kStatusTimeout);
  __syncwarp();
  pair_sync();  // neither CTA's barriers or TMEM are used any more
  if (warp == 0) pair_tmem_dealloc(tmem);
  if (a.late) after_previous();
}

__device__ __forceinline__ void write4(__nv_bfloat16* to, float4 x) {
  *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2(x.x, x.y), bf16x2(x.z, x.w));
}
__device__ __forceinline__ void write4(float* to, float4 x) {
  *reinterpret_cast<float4*>(to) = x;
}

// dk and dv from their parts, which are added in their order: a CTA takes SUM_ROWS rows of a key tile
// and head.  Bound by HBM.
constexpr int SUM_ROWS = 16;
template <int D, typename T>
__global__ void __launch_bounds__(256) k_attn_sum(SeqArgs a) {
  after_previous();
  before_next();
  Tile t;
  const int per = a.tk.rows / SUM_ROWS, hk = blockIdx.x % a.Hk, x = blockIdx.x / a.Hk;
  if (!tile_of<true>(a, x / per, &t)) return;
  t.at += x % per * SUM_ROWS;
  const int rows = min(SUM_ROWS, t.nk - t.at);
  const int64_t step = a.Nk * a.Hk * D;
#pragma unroll 2
  for (int i = threadIdx.x; i < rows * (D / 4); i += 256) {
    const int64_t at = ((int64_t)(t.k0 + t.at + i / (D / 4)) * a.Hk + hk) * D + i % (D / 4) * 4;
    const float *pk = a.part_k + at, *pv = a.part_v + at;
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
#pragma unroll 4
    for (int q = 0; q < a.splits; ++q) {
      const float4 y = *reinterpret_cast<const float4*>(pk + q * step);
      const float4 z = *reinterpret_cast<const float4*>(pv + q * step);
      k.x += y.x;
      k.y += y.y;
      k.z += y.z;
      k.w += y.w;
      v.x += z.x;
      v.y += z.y;
      v.z += z.z;
      v.w += z.w;
    }
    write4(reinterpret_cast<T*>(a.dk) + at, k);
    write4(reinterpret_cast<T*>(a.dv) + at, v);
  }
}

// o and lse from the parts of the keys: a CTA takes SUM_ROWS rows of a tile.  With L_p the part's
// log2-sum and o_p its average: w_p = 2^(L_p - max L), o = sum w_p o_p / sum w_p.  A part without
// keys has L_p = -inf and counts nothing.
template <int D, typename T>
__global__ void __launch_bounds__(256) k_attn_merge(SeqArgs a) {
  constexpr int PER = D / 4;  // threads of a row
  __shared__ float s_w[SUM_ROWS][kMaxParts];
  after_previous();
  before_next();
  Tile t;
  const int groups = a.Hq / a.pack, rows = a.tq.rows * a.pack, per = rows / SUM_ROWS;
  const int head = blockIdx.x % groups * a.pack, y = blockIdx.x / groups;
  if (!tile_of<false>(a, y / per, &t)) return;
  const int r0 = y % per * SUM_ROWS;
  const int64_t step = a.Nq * a.Hq;
  auto row_of = [&](int r, int64_t* at) {  // row r0 + r of the tile: whether it exists, its place
    const int token = t.at + (r0 + r) / a.pack;
    *at = (int64_t)(t.q0 + token) * a.Hq + head + (r0 + r) % a.pack;
    return token < t.nq;
  };
  if (threadIdx.x < SUM_ROWS) {
    int64_t at;
    if (row_of(threadIdx.x, &at)) {
      float m = -INFINITY, l = 0.f;
      for (int p = 0; p < a.parts; ++p) m = fmaxf(m, a.part_lse[p * step + at]);
      const float base = m == -INFINITY ? 0.f : m;
      for (int p = 0; p < a.parts; ++p) {
        const float w = ex2(a.part_lse[p * step + at] - base);
        s_w[threadIdx.x][p] = w;
        l += w;
      }
      for (int p = 0; p < a.parts; ++p) s_w[threadIdx.x][p] = l != 0.f ? s_w[threadIdx.x][p] / l : 0.f;
      if (a.lse) a.lse[at] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < SUM_ROWS * PER; i += 256) {
    int64_t at;
    if (!row_of(i / PER, &at)) continue;
    const float* src = a.part_o + at * D + i % PER * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p) {
      const float4 x = *reinterpret_cast<const float4*>(src + p * step * D);
      const float w = s_w[i / PER][p];
      o.x = fmaf(x.x, w, o.x);
      o.y = fmaf(x.y, w, o.y);
      o.z = fmaf(x.z, w, o.z);
      o.w = fmaf(x.w, w, o.w);
    }
    write4(reinterpret_cast<T*>(a.out) + at * D + i % PER * 4, o);
  }
}

// ---------------------------------------------------------------------------------- host

template <auto kKernel, typename... M>
cudaError_t launch(int64_t grid, int threads, int smem, cudaStream_t st, const M&... args) {
  if (grid == 0) return cudaSuccess;
  const cudaError_t e = allow_smem<kKernel>(smem);
  if (e != cudaSuccess) return e;
  return launch_behind(kKernel, dim3((unsigned)grid), threads, smem, st, args...);
}

// Maps; rows that do not exist are never loaded (a map of another tensor stands in).
bool make(CUtensorMap* m, const void* p, int64_t n, int64_t stride, int64_t heads, int D,
          int rows, int pack = 1) {
  return tc_make_map_tokens(m, p, n, stride, heads, D, rows, pack);
}

// CTAs, one per SM, each of which takes several items.
int64_t ctas_of(int64_t items) {
  const int64_t sms = device_sms();
  return items < sms ? items : sms;
}

// The same in pairs.
int64_t pairs_of(int64_t items) {
  const int64_t sms = device_sms() / 2;
  return 2 * (items < sms ? items : sms);
}

template <int D>
cudaError_t fwd(const SeqArgs& a, cudaStream_t st) {
  CUtensorMap q, k, v;
  if (!make(&q, a.q, a.Nq, a.qs, a.Hq, D, TR / a.pack, a.pack)) return cudaErrorInvalidValue;
  k = v = q;
  if (a.Nk > 0 && (!make(&k, a.k, a.Nk, a.ks, a.Hk, D, 128) ||
                   !make(&v, a.v, a.Nk, a.vs, a.Hk, D, 128)))
    return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)a.tq.most * (a.Hq / a.pack);
  const cudaError_t e = launch<k_flash<D, true>>(ctas_of(tiles * a.parts), Flash<D>::kThreads,
                                                 Flash<D>::kBytes, st, q, k, v, a);
  return e == cudaSuccess && a.parts > 1 ? launch_merge(a, D, false, st) : e;
}

template <int D>
cudaError_t bwd(SeqArgs a, cudaStream_t st) {
  const int64_t os = (int64_t)a.Hq * D;
  CUtensorMap q, d, k, v;  // boxes of 128 rows
  if (a.Nq > 0 && (!make(&q, a.q, a.Nq, a.qs, a.Hq, D, 128) ||
                   !make(&d, a.dO, a.Nq, os, a.Hq, D, 128)))
    return cudaErrorInvalidValue;
  if (a.Nk > 0 && (!make(&k, a.k, a.Nk, a.ks, a.Hk, D, 128) ||
                   !make(&v, a.v, a.Nk, a.vs, a.Hk, D, 128)))
    return cudaErrorInvalidValue;
  if (a.Nq == 0) q = d = k;
  if (a.Nk == 0) k = v = q;
  // The first launch waits for what came before it; the others read nothing that it writes and begin
  // as its CTAs end (late), and wait for it before they end themselves, so that the last one's end is
  // the end of all.
  const int64_t key_items = (int64_t)a.tk.most * a.Hk * a.splits;
  const int64_t query_items = (int64_t)a.tq.most * a.Hq;
  cudaError_t e = cudaSuccess;
  if constexpr (D == 256) {
    CUtensorMap qh, dh, kh, vh;  // boxes of 64 rows
    if (a.Nq > 0 && (!make(&qh, a.q, a.Nq, a.qs, a.Hq, D, 64) ||
                     !make(&dh, a.dO, a.Nq, os, a.Hq, D, 64)))
      return cudaErrorInvalidValue;
    if (a.Nk > 0 && (!make(&kh, a.k, a.Nk, a.ks, a.Hk, D, 64) ||
                     !make(&vh, a.v, a.Nk, a.vs, a.Hk, D, 64)))
      return cudaErrorInvalidValue;
    if (a.Nq == 0) qh = dh = kh;
    if (a.Nk == 0) kh = vh = qh;
    if (a.Nk > 0) {
      e = launch<k_slope_pair<kDk>>(pairs_of(key_items), Pair::kThreads, Pair::kBytes, st, k, v, qh,
                                    dh, q, a);
      if (e != cudaSuccess) return e;
      a.late = 1;
      e = launch<k_flash<D, false>>(ctas_of(2 * key_items), Flash<D>::kThreads, Flash<D>::kBytes, st,
                                    k, q, d, a);
    }
    if (e == cudaSuccess && a.Nq > 0)
      e = launch<k_slope_pair<kDq>>(pairs_of(query_items), Pair::kThreads, Pair::kBytes, st, q, d,
                                    kh, vh, k, a);
  } else {
    if (a.Nk > 0)
      e = launch<k_slope<D, kDkv>>(ctas_of(key_items), Slope<D>::kThreads, Slope<D>::kBytes, st, k,
                                   v, q, d, a);
    a.late = a.Nk > 0;
    if (e == cudaSuccess && a.Nq > 0)
      e = launch<k_slope<D, kDq>>(ctas_of(query_items), Slope<D>::kThreads, Slope<D>::kBytes, st,
                                  q, d, k, v, a);
  }
  return e == cudaSuccess && a.Nk > 0 && a.splits > 1 ? launch_sum(a, D, false, st) : e;
}

}  // namespace

cudaError_t launch_sum(const SeqArgs& a, int D, bool fp32, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.tk.most * a.Hk * (a.tk.rows / SUM_ROWS)));
  auto go = [&](auto kernel) { return launch_behind(kernel, grid, 256, 0, st, a); };
  if (fp32)
    return D == 64    ? go(k_attn_sum<64, float>)
           : D == 128 ? go(k_attn_sum<128, float>)
                      : go(k_attn_sum<256, float>);
  return D == 64    ? go(k_attn_sum<64, __nv_bfloat16>)
         : D == 128 ? go(k_attn_sum<128, __nv_bfloat16>)
                    : go(k_attn_sum<256, __nv_bfloat16>);
}
cudaError_t launch_merge(const SeqArgs& a, int D, bool fp32, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.tq.most * (a.Hq / a.pack) *
                             (a.tq.rows * a.pack / SUM_ROWS)));
  auto go = [&](auto kernel) { return launch_behind(kernel, grid, 256, 0, st, a); };
  if (fp32)
    return D == 64    ? go(k_attn_merge<64, float>)
           : D == 128 ? go(k_attn_merge<128, float>)
                      : go(k_attn_merge<256, float>);
  return D == 64    ? go(k_attn_merge<64, __nv_bfloat16>)
         : D == 128 ? go(k_attn_merge<128, __nv_bfloat16>)
                    : go(k_attn_merge<256, __nv_bfloat16>);
}
TcPlan tc_plan(int D) {
  const int two = D == 64 ? Flash<64>::kTiles : D == 128 ? Flash<128>::kTiles : Flash<256>::kTiles;
  const int own = D == 256 ? 2 * TR : TR;
  return TcPlan{two * TR, own, own};  // fwd: rows, of which `pack` belong to a token
}
cudaError_t launch_fwd_tc(const SeqArgs& a, int D, cudaStream_t st) {
  return D == 64 ? fwd<64>(a, st) : D == 128 ? fwd<128>(a, st) : fwd<256>(a, st);
}
cudaError_t launch_bwd_tc(const SeqArgs& a, int D, cudaStream_t st) {
  return D == 64 ? bwd<64>(a, st) : D == 128 ? bwd<128>(a, st) : bwd<256>(a, st);
}

}  // namespace seq
}  // namespace gdn
