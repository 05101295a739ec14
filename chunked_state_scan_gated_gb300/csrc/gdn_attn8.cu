// gdn_attn8.cu -- attention of one new token per request over a paged cache in 8 bits: e4m3 codes
// with a scale for every 16 tokens and head (gdn_cache8.cu writes it).  Schedule, join and the
// shape of the products are those of the 16- and 32-bit caches (gdn_attn_split.cuh, gdn_attn.cu):
// fragments go from global memory straight into registers, 8 query heads to a product.
//
// Bound by HBM, at 1 byte per element and 4 per 16 D elements.  What differs:
//   - e4m3 turns into f16 exactly, two numbers to an instruction, and the products run in f16.  V's
//     fragments want two keys of one column: their bytes are put together first, then converted.
//   - q has more range than f16: each query row is scaled by a power of two that brings its largest
//     element to [2^13, 2^14); bf16 elements are then exact in f16 (down to 2^-27 of the largest,
//     2^-39 of it is lost below), fp32 ones go as two f16 terms (2^-22).
//   - a score is the product times the row's and the block's factors, in fp32; K's scale is one
//     number per 16-key block, uniform in the warp.
//   - V's scale goes into the weights: w = p vs, held as w 2^7 / R.  R follows the largest w of the head:
//     it shrinks with the weights when the scores' reference rises, and is raised to a tile's largest w
//     when the reference rises or a block's scale is above 16 R (both rare; then the accumulators are
//     rescaled).  Weights are at most 2^4 (the scores' lazy reference), so that f16 holds 2^15 at most;
//     it keeps 2^-11 of a w down to 2^-21 R and 2^-32 R below.  R is never above the largest w: a block
//     counts by its weight, however large its scale.  bf16 q: one f16 term (an eighth of o's own
//     rounding); fp32 q: two (2^-22).
#include <cuda_fp16.h>

#include "gdn_attn_split.cuh"

namespace gdn {
namespace {

// A cache in 8 bits, read with q and o of type TO.
template <typename TO> struct Q8 {};

template <typename TO>
struct Cache<Q8<TO>> {
  using Out = TO;
  template <int D> static constexpr int el() { return D == 64 ? 8 : 16; }
};

// 4 KB of K and of V to a warp's tile (8 KB at D = 256): what is on its way per SM, 64 KB, and the
// work per tile weigh against each other (131001 tokens, 8 heads of 128: 16 keys and 4 CTAs 56.3 us,
// 32 and 3 57.8, 32 and 2 55.0, which is 53.3 with R by head; 812,553 tokens, 2 heads of 256: 16 and 2
// 159, 32 and 2 149, now 144).
template <typename TO> struct Cfg<64, Q8<TO>, 1> : Fit<32, 4, 1> {};
template <typename TO> struct Cfg<128, Q8<TO>, 1> : Fit<32, 2, 1> {};
template <typename TO> struct Cfg<256, Q8<TO>, 1> : Fit<32, 2, 1> {};
template <typename TO> struct Cfg<64, Q8<TO>, 2> : Fit<32, 3, 1> {};
template <typename TO> struct Cfg<128, Q8<TO>, 2> : Fit<32, 2, 1> {};
template <typename TO> struct Cfg<256, Q8<TO>, 2> : Fit<16, 2, 1> {};

constexpr float A8_LAZY = 4.f;   // log2 units
constexpr float A8_UP = 0x1p7f;      // what R is in f16
constexpr float A8_OVER = 16.f;      // how far a scale may be above R
constexpr float A8_MOST = 0x1p100f;  // of A8_UP / R: R is 2^-93 at least

// Q in shared memory as f16 (fp32: the second terms behind the first), rows 16 bytes longer than D
// elements: the 8 lanes of a 16-byte read phase (2 rows x 4 chunks of 32 bytes) fall on different
// banks.  Behind it the rows' factors.
template <int D, typename TO, int NG>
struct Smem<D, Q8<TO>, NG> {
  static constexpr int kTerms = sizeof(TO) == 4 ? 2 : 1;
  static constexpr int kRow = D * 2 + 16;  // bytes
  static constexpr int kTerm = AT_G * NG * kRow;
  static constexpr int kFactors = kTerms * kTerm;
  static constexpr int kQ = kFactors + AT_G * NG * 4;
  static constexpr int kORow = D + 2;      // floats
  static constexpr int kO = AT_W * AT_G * kORow * 4;
  static constexpr int kBytes = kQ > kO ? kQ : kO;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 numbers as f16: the first two in lo.
__device__ __forceinline__ void widen(uint32_t x, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*lo), "=r"(*hi) : "r"(x));
}
__device__ __forceinline__ uint32_t f16x2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x, y as sums hi + lo of f16 numbers.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t* hi, uint32_t* lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = f16x2(x - f.x, y - f.y);
}
// volatile: kept in place (registers)
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int BYTES>
__device__ __forceinline__ void load(uint32_t* dst, const uint8_t* p, bool in) {
  if constexpr (BYTES == 16) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in)
      asm("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
          : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    dst[0] = v.x;
    dst[1] = v.y;
    dst[2] = v.z;
    dst[3] = v.w;
  } else {
    uint2 v = make_uint2(0, 0);
    if (in)
      asm("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    dst[0] = v.x;
    dst[1] = v.y;
  }
}

__device__ __forceinline__ float rcp(float x) {  // 2^-23 off
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The largest of the 8 lanes that hold a head's keys.
__device__ __forceinline__ float over_keys(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// `heads` query rows from q on to shared memory, in f16 with their factors (zeros past them).
template <int D, typename TO, int NG>
__device__ __forceinline__ void stage_q8(char* smem, const TO* q, int heads) {
  using S = Smem<D, Q8<TO>, NG>;
  constexpr int ROWS = AT_G * NG / AT_W, E = D / 32;  // rows of a warp, elements of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float x[ROWS][E];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = warp + i * AT_W;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      float2 v = make_float2(0.f, 0.f);
      if (h < heads) {
        const TO* p = q + (int64_t)h * D + e * 32 + lane * 2;
        if constexpr (sizeof(TO) == 2)
          v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
        else
          v = *reinterpret_cast<const float2*>(p);
      }
      x[i][e] = v.x;
      x[i][e + 1] = v.y;
    }
  }
  __syncthreads();  // other warps may still read what was there
  float* factors = reinterpret_cast<float*>(smem + S::kFactors);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = warp + i * AT_W;
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[i][e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    int ex = (int)(__float_as_uint(top) >> 23) - 127;
    if (ex < -100) ex = ex == -127 && top == 0.f ? 13 : -100;  // a row of zeros: any factor
    if (ex == 128) ex = 13;                                    // not finite: as it is
    const float up = __uint_as_float((uint32_t)(13 - ex + 127) << 23);  // 2^(13 - ex)
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      uint32_t hi, lo;
      split_f16(x[i][e] * up, x[i][e + 1] * up, &hi, &lo);
      char* at = smem + h * S::kRow + (e * 32 + lane * 2) * 2;
      *reinterpret_cast<uint32_t*>(at) = hi;
      if (S::kTerms == 2) *reinterpret_cast<uint32_t*>(at + S::kTerm) = lo;
    }
    if (lane == 0) factors[h] = __uint_as_float((uint32_t)(ex - 13 + 127) << 23);
  }
}

template <int D, typename TO, int NG>
__device__ void run_piece8(const AttnArgs& ar, char* smem, int64_t b, int n, int hk, int hg,
                           int t0, int t1, Acc<D, NG>& a, int* bad) {
  using S = Smem<D, Q8<TO>, NG>;
  constexpr int GP = AT_G * NG, NK = Cfg<D, Q8<TO>, NG>::kKeys / 16, KC = D / 64, VW = D / 32;
  constexpr int VB = D == 64 ? 8 : 16;  // bytes of a load of V
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int heads = min(GP, ar.G - hg * GP);
  const int64_t row = ar.Hk * D;  // bytes between a page's rows
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(ar.kc) + (int64_t)hk * D;
  const uint8_t* vc = reinterpret_cast<const uint8_t*>(ar.vc) + (int64_t)hk * D;
  const float *ksc = ar.ksc + hk, *vsc = ar.vsc + hk;
  const int32_t* table = ar.table + b * ar.max_blocks;
  // A warp's next blocks of 16 keys: number, page of the table and block in the page, moved on
  // by the blocks of a CTA tile without dividing.
  constexpr int STEP = AT_W * NK;
  const int pb = ar.P / 16, end = min((n - 1) / 16 + 1, t1 * STEP);
  const int dpi = STEP / pb, dpo = STEP % pb;
  int blk = t0 * STEP + warp * NK, pi = blk / pb, po = blk % pb;
  int32_t pg[NK];  // pages of the blocks that were looked up, one tile ahead
  int pofs[NK], cnt[NK];
  auto look_up = [&]() {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      int x = po + i, y = pi;  // a page has one block at least
      while (x >= pb) x -= pb, ++y;
      const bool live = blk + i < end;
      pg[i] = live ? table[y] : -1;
      pofs[i] = x;
      cnt[i] = live ? min(16, n - (blk + i) * 16) : 0;
    }
    blk += STEP;
    pi += dpi;
    po += dpo;
    if (po >= pb) {
      po -= pb;
      ++pi;
    }
  };
  // their places as numbers of 16-row blocks of the cache; rows that count
  auto place = [&](int64_t (&at)[NK], int (&rows)[NK]) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      rows[i] = cnt[i];
      if (cnt[i] > 0 && (pg[i] < 0 || pg[i] >= ar.pages)) {
        *bad = 1;
        rows[i] = 0;
      }
      at[i] = rows[i] > 0 ? (int64_t)pg[i] * pb + pofs[i] : 0;
    }
  };
  uint32_t k[NK][2][KC][4], v[NK][4][VW];
  float ks[NK], vs[NK];
  auto load_k = [&](const int64_t (&at)[NK], const int (&rows)[NK]) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const uint8_t* p = kc + at[i] * 16 * row + g * row + t * 16;
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int c = 0; c < KC; ++c)
          load<16>(k[i][z][c], p + z * 8 * row + c * 64, g + 8 * z < rows[i]);
      ks[i] = rows[i] > 0 ? ksc[at[i] * ar.Hk] : 0.f;
    }
  };
  auto load_v = [&](const int64_t (&at)[NK], const int (&rows)[NK]) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int key = 2 * t + (z & 1) + 8 * (z >> 1);
        const uint8_t* p = vc + (at[i] * 16 + key) * row + g * VB;
#pragma unroll
        for (int w = 0; w < VW; w += VB / 4)
          load<VB>(&v[i][z][w], p + (w / 4) * 128, key < rows[i]);
      }
      vs[i] = rows[i] > 0 ? vsc[at[i] * ar.Hk] : 0.f;
    }
  };
  int64_t cur[NK];
  int rows[NK];
  look_up();
  stage_q8<D, TO, NG>(
      smem, reinterpret_cast<const TO*>(ar.q) + b * ar.qs + ((int64_t)hk * ar.G + hg * GP) * D,
      heads);
  place(cur, rows);
  load_k(cur, rows);
  load_v(cur, rows);
#pragma unroll
  for (int q = 0; q < NG; ++q) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      a.o[q][i][0] = a.o[q][i][1] = a.o[q][i][2] = a.o[q][i][3] = 0.f;
    a.m[q][0] = a.m[q][1] = -INFINITY;
    a.l[q][0] = a.l[q][1] = 0.f;
  }
  look_up();
  __syncthreads();  // Q is there
  float qf[NG][2];
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    const float2 f =
        *reinterpret_cast<const float2*>(smem + S::kFactors + (q * AT_G + 2 * t) * 4);
    qf[q][0] = f.x;
    qf[q][1] = f.y;
  }
  float rv[NG][2];  // A8_UP / R of heads 2t, 2t + 1
  float vok = 0.f;  // A8_OVER times the least R of the warp's heads
#pragma unroll
  for (int q = 0; q < NG; ++q) rv[q][0] = rv[q][1] = A8_MOST;
#pragma unroll 1
  for (int tile = t0; tile < t1; ++tile) {
    int64_t nxt[NK];
    int nrows[NK];
    place(nxt, nrows);
    look_up();
    // fp32: the tensor cores cut an accumulator's low bits off at every product, so 64 columns'
    // products, second terms first, have accumulators of their own, which are added with rounding
    // (error against 64 bits at 517 tokens of D = 256: 1.8e-6 without, see the tests' bound)
    float s[NG][NK][4] = {};
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        float x[NK][4] = {};
#pragma unroll
        for (int z = S::kTerms - 1; z >= 0; --z) {
          const char* qs = smem + z * S::kTerm + (q * AT_G + g) * S::kRow + (t + 4 * c) * 32;
          const uint4 lo = *reinterpret_cast<const uint4*>(qs);
          const uint4 hi = *reinterpret_cast<const uint4*>(qs + 16);
          const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t a0, a1, a2, a3;
              widen(k[i][0][c][u], &a0, &a2);
              widen(k[i][1][c][u], &a1, &a3);
              mma_f16(S::kTerms == 2 ? x[i] : s[q][i], a0, a1, a2, a3, w[2 * u], w[2 * u + 1]);
            }
        }
        if constexpr (S::kTerms == 2)
#pragma unroll
          for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[q][i][j] += x[i][j];
      }
    float kf[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) kf[i] = ks[i];
    load_k(nxt, nrows);
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int i = 0; i < NK; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[q][i][j] = g + 8 * (j >> 1) < rows[i] ? s[q][i][j] * (qf[q][j & 1] * kf[i]) : -INFINITY;
    float mx[NG][2];
    bool up = false;
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      mx[q][0] = mx[q][1] = -INFINITY;
#pragma unroll
      for (int i = 0; i < NK; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[q][j & 1] = fmaxf(mx[q][j & 1], s[q][i][j]);
      up = up || mx[q][0] > a.m[q][0] + ar.lazy || mx[q][1] > a.m[q][1] + ar.lazy;
    }
    float vtop = 0.f;
#pragma unroll
    for (int i = 0; i < NK; ++i) vtop = fmaxf(vtop, vs[i]);
    // the scores' reference follows the maximum lazily, as in gdn_attn.cu
    if (vtop > vok || __any_sync(0xffffffffu, up)) {
      float most = 0.f;
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float m = fmaxf(over_keys(mx[q][j]), a.m[q][j]), base = m == -INFINITY ? 0.f : m;
          float w = 0.f;  // the tile's largest
#pragma unroll
          for (int i = 0; i < NK; ++i)
            w = fmaxf(w, ex2((fmaxf(s[q][i][j], s[q][i][j + 2]) - base) * ar.sl) * vs[i]);
          w = over_keys(w);
          const float e = m == a.m[q][j] ? 1.f : ex2((a.m[q][j] - m) * ar.sl);  // 0 from -inf
          a.l[q][j] *= e;
          a.m[q][j] = m;
          const float r = rv[q][j] * rcp(e);  // infinite from 0
          rv[q][j] = fminf(w * r > A8_UP ? A8_UP * rcp(w) : r, A8_MOST);
          f[j] = rv[q][j] * rcp(r);
          most = fmaxf(most, rv[q][j]);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) a.o[q][i][j] *= f[j & 1];
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      vok = A8_OVER * A8_UP * rcp(most);
    }
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float base = a.m[q][j & 1] == -INFINITY ? 0.f : a.m[q][j & 1];
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          const float p = ex2((s[q][i][j] - base) * ar.sl);
          a.l[q][j & 1] += p;
          s[q][i][j] = p * (vs[i] * rv[q][j & 1]);
        }
      }
    // fp32: the tensor cores cut an accumulator's low bits off at every product, so a tile's
    // products have accumulators of their own, which are then added with rounding
    uint32_t ph[NK][NG][2], pl[NK][NG][2];
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          split_f16(s[q][i][2 * z], s[q][i][2 * z + 1], &ph[i][q][z], &pl[i][q][z]);
          ph[i][q][z] = turn8x8(ph[i][q][z]);
          if (S::kTerms == 2) pl[i][q][z] = turn8x8(pl[i][q][z]);
        }
#pragma unroll
    for (int w = 0; w < VW; ++w)
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // columns 2u, 2u + 1 of the word's four
        const uint32_t sel = u ? 0x7362 : 0x5140;
        float x[NG][4] = {};
        uint32_t f[NK][4];
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          widen(__byte_perm(v[i][0][w], v[i][1][w], sel), &f[i][0], &f[i][1]);
          widen(__byte_perm(v[i][2][w], v[i][3][w], sel), &f[i][2], &f[i][3]);
        }
#pragma unroll
        for (int z = S::kTerms - 1; z >= 0; --z)
#pragma unroll
          for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int q = 0; q < NG; ++q)
              mma_f16(S::kTerms == 2 ? x[q] : a.o[q][2 * w + u], f[i][0], f[i][1], f[i][2], f[i][3],
                      (z ? pl : ph)[i][q][0], (z ? pl : ph)[i][q][1]);
        if constexpr (S::kTerms == 2)
#pragma unroll
          for (int q = 0; q < NG; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) a.o[q][2 * w + u][j] += x[q][j];
      }
    load_v(nxt, nrows);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      cur[i] = nxt[i];
      rows[i] = nrows[i];
    }
  }
#pragma unroll
  for (int q = 0; q < NG; ++q) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) a.o[q][i][j] *= rcp(rv[q][j & 1]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        a.l[q][j] += __shfl_xor_sync(0xffffffffu, a.l[q][j], o);
  }
}

template <int D, typename TO, int NG>
struct Piece<D, Q8<TO>, NG> {
  template <typename... A>
  static __device__ __forceinline__ void run(A&&... a) { run_piece8<D, TO, NG>(a...); }
};

// Runs f with the call's head dim and type as template arguments.
template <typename F>
auto with_types(const gdn_attn_problem* p, F f) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  using D256 = std::integral_constant<int, 256>;
  if (p->dtype == GDN_BF16) {
    const Q8<__nv_bfloat16> t{};
    return p->D == 64 ? f(D64(), t) : p->D == 128 ? f(D128(), t) : f(D256(), t);
  }
  const Q8<float> t{};
  return p->D == 64 ? f(D64(), t) : p->D == 128 ? f(D128(), t) : f(D256(), t);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_attn_decode8_workspace_size(const gdn_attn_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  *bytes = with_types(p, [](auto d, auto t) { return workspace_of<d(), decltype(t)>(); });
  return GDN_OK;
}

gdn_status gdn_attn_decode8(const gdn_attn_problem* p, const void* q, const void* k_cache,
                            const void* v_cache, const float* k_scale, const float* v_scale,
                            const int32_t* block_table, const int32_t* seq_len, void* o,
                            float* lse, void* workspace, size_t workspace_bytes,
                            int32_t* status, void* stream) {
  size_t need = 0;
  gdn_status s = gdn_attn_decode8_workspace_size(p, &need);
  if (s != GDN_OK) return s;
  if (p->B == 0) return GDN_OK;
  const int64_t rows = p->pages * p->page_size;
  if (!ok16(q, 1) || !ok16(o, 1) || !ok16(k_cache, rows) || !ok16(v_cache, rows) ||
      !ok16(k_scale, rows) || !ok16(v_scale, rows) || !ok4(block_table, p->B * p->max_blocks) ||
      !ok4(seq_len, 1) || !aligned16(lse) || ((uintptr_t)workspace & 255u) != 0 ||
      ((uintptr_t)status & 255u) != 0)
    return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
  AttnArgs ar = args_of(p, q, k_cache, v_cache, block_table, seq_len, o, lse, status, A8_LAZY);
  ar.ksc = k_scale;
  ar.vsc = v_scale;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = with_types(p, [&](auto d, auto t) {
    // one pass over the cache serves 8 query heads of a key head, or 16
    return ar.G <= AT_G ? launch<d(), decltype(t), 1>(ar, (char*)workspace, st)
                        : launch<d(), decltype(t), 2>(ar, (char*)workspace, st);
  });
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
