// gdn_attn.cu -- attention of one new token per request over a paged key-value cache.  Per
// request and query head, over its n cached tokens:
//   s_j = scale q.k_j,  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  lse = m + log(sum)
// with the running maximum m and sum of a one-pass softmax.
//
// Bound by HBM: every K and V row is read once.  A piece of work is (request, key head, range
// of tokens); the query heads of a key head are the 8 columns of the products
//   S^T [16 keys x 8 heads] = K [16 x D] Q^T,   O^T [D x 8] += V^T [D x 16 keys] P^T
// so a group of 8 query heads fills mma.sync's tile (more than 8 per key head go 16 to a pass over
// the cache, two products per fragment: 131001 tokens with 16 query heads to each of 8 key heads
// of 128: 94 us against 158 in two passes) and K, V need no transposition: both are the products'
// A operand, whose fragments are loaded from global memory straight into registers, 16 bytes per
// lane.  That works because the contraction index of the first product (the head's elements) and
// the output rows of the second may be permuted freely:
//   K: lane (g, t) = (lane / 4, lane % 4) loads 16-byte chunk t + 4c of key rows g and g + 8,
//      and the 4 (2) words of a chunk serve 2 products, Q's fragment being the same chunk;
//   V: the lane loads chunk g + 8c of the rows of the 4 keys of its fragment; the pairs of
//      keys are put together with byte permutes.
// P^T comes out of the first product transposed (keys by heads) and is turned with movmatrix
// (bf16) or shuffles (fp32).  On bf16 the weights go into V's product as two bf16 terms each, so
// that o has no rounding but its own (one term: 2^-9 of a weight, a third more error in o; two
// cost 0 to 4% of the time, the tensor pipe being far from full).  No shared memory, barrier or copy wait is on the path of the
// data: a warp's next K tile is on its way while it does the softmax and V's product, and the
// next V tile during the next K product; 8 to 16 such warps per SM keep 64 to 128 KB in flight.
// fp32 caches use tf32 products of the two-term split x = hi + lo (2^-23 of x; all four products),
// which keeps fp32 accuracy at the same layout.  The split is done with integer and fp32
// instructions at full rate (131001 tokens of 8 heads of 128: 181 us against 234 with conversion
// instructions and a test of every value for infinities; 176 with the accumulators of mma_split).
//
// Split: the unit is a CTA tile of one (request, key head); the units of all requests in a
// row are divided evenly over the CTAs of one wave, whatever the lengths: no tail, and one long
// request uses the whole GPU.  A CTA's first and last pieces may be parts of a request; these
// go to the workspace and k_attn_join adds them up.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "gdn_internal.h"
#include "gdn_launch.cuh"

namespace gdn {
namespace {

constexpr int AT_W = 4;            // warps per CTA
constexpr int AT_NT = 32 * AT_W;
constexpr int AT_G = 8;            // query heads per product
constexpr int AT_SMS = 152;
constexpr float AT_LAZY = 8.f;     // log2 units
constexpr float AT_LOG2E = 1.4426950408889634f;
// What a piece costs beside its tiles, in units (its first loads and its end): without it a CTA
// with many short requests lags (61 ragged requests 128 against 102 us; 2 to 5: the same).
constexpr int AT_START = 1;

// Keys per warp tile, CTAs per SM and parts, for NG groups of AT_G query heads per piece: the K
// and V tiles and the accumulators of D x 8 NG fill most of a CTA's share of the registers.
// kParts > 1: the two tiles do not fit; they go by that many parts of D.
template <int KEYS, int CTAS, int PARTS>
struct Fit {
  static constexpr int kKeys = KEYS, kCtas = CTAS, kParts = PARTS;
};
template <int D, typename T, int NG> struct Cfg;
template <> struct Cfg<64, __nv_bfloat16, 1> : Fit<32, 4, 1> {};
template <> struct Cfg<128, __nv_bfloat16, 1> : Fit<16, 3, 1> {};
template <> struct Cfg<256, __nv_bfloat16, 1> : Fit<16, 2, 1> {};
template <> struct Cfg<64, float, 1> : Fit<16, 3, 1> {};
template <> struct Cfg<128, float, 1> : Fit<16, 2, 1> {};
template <> struct Cfg<256, float, 1> : Fit<16, 2, 2> {};
template <> struct Cfg<64, __nv_bfloat16, 2> : Fit<32, 3, 1> {};
template <> struct Cfg<128, __nv_bfloat16, 2> : Fit<16, 2, 1> {};
template <> struct Cfg<256, __nv_bfloat16, 2> : Fit<16, 2, 2> {};
template <> struct Cfg<64, float, 2> : Fit<16, 2, 1> {};
template <> struct Cfg<128, float, 2> : Fit<16, 2, 2> {};
template <> struct Cfg<256, float, 2> : Fit<16, 2, 4> {};

// Parts of pieces in the workspace: slot 2c of CTA c is the piece that began before it, slot
// 2c + 1 the one that goes on behind it.  Join c tells of the piece that goes on from CTA c to
// CTA c + 1, if one does.
struct __align__(16) Join {
  int32_t b, h;         // request, piece of it
  int32_t first, last;  // CTAs that it begins and ends in (last < 0: none goes on)
};

struct AttnArgs {
  int64_t B, Hq, Hk, pages, max_blocks, qs;
  int P, G, HG;   // tokens per page, query heads per key head, pieces of them
  float sl;       // scale log2(e)
  float lazy;     // AT_LAZY in units of the unscaled scores
  const void *q, *kc, *vc;
  const int32_t *table, *len;
  void* o;
  float* lse;
  Join* join;     // [CTAs]
  float2* ml;     // [CTAs][2][AT_G NG] reference score (unscaled) and sum
  float* acc;     // [CTAs][2][AT_G NG][D]
  int32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 ldg16(const void* p) {
  uint4 v;
  asm("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// volatile: kept in place, or the weights of several blocks are turned early and spill what they
// displace (12 or 16 query heads on 2 of 256: 336 us against 295; 517 tokens 9.5 against 9.0)
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two weights (at least 0, or NaN) as sums hi + lo of bf16 numbers, x in the low halves: hi is cut
// off and lo, what is left, rounded (2^-15 of the weight).  lo is not zero where hi is not, so that
// an infinite v gives the infinity that hi v is, not 0 * inf beside it.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t* hi, uint32_t* lo) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y), h = __byte_perm(a, b, 0x7632);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x - __uint_as_float(a & 0xffff0000u),
                                                 y - __uint_as_float(b & 0xffff0000u));
  *hi = h;
  *lo = __vmaxu2(*reinterpret_cast<const uint32_t*>(&l), __vminu2(h, 0x00010001u));
}
// x = hi + lo with hi, lo in tf32: hi is x rounded to nearest (ties away), lo what is left, rounded
// too (2^-23 of x).  SAFE: an infinite or NaN x goes into lo alone, which mma_split<SAFE> multiplies
// only with the other operand's hi, so that no 0 * inf arises beside the product itself.  CUT: both
// are cut off (2^-21 of x), as rounding could make the largest finite numbers infinite; what is left
// of a cut x has 2 bits too many at most, which adding 0x7ff does not carry out of (131001 tokens,
// 8 heads of 128: 176 us, and 180 without the addition, for the order that the registers then get).
template <bool SAFE, bool CUT = SAFE>
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t* hi, uint32_t* lo) {
  constexpr uint32_t kMask = 0xffffe000u;
  const bool infinite = SAFE && (x & 0x7f800000u) == 0x7f800000u;
  const uint32_t h = (x + (CUT ? 0u : 0x1000u)) & kMask;
  const uint32_t l =
      (__float_as_uint(__uint_as_float(x) - __uint_as_float(h)) + (CUT ? 0x7ffu : 0x1000u)) & kMask;
  *hi = infinite ? 0u : h;
  *lo = infinite ? x : l;
}
__device__ __forceinline__ void split_query(uint32_t x, uint32_t* hi, uint32_t* lo) {
  if ((x & 0x7f800000u) >= 0x7f000000u) split_tf32<true>(x, hi, lo);
  else split_tf32<false>(x, hi, lo);
}
// acc += 4 v: not finite once any value is not, or is as large as 2^126 (a sum that overflows
// only takes the SAFE form without need)
__device__ __forceinline__ void probe(const uint4& v, uint64_t* acc) {
  asm("{\n\t.reg .b64 a, b, f;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "mov.b64 f, 0x4080000040800000;\n\tfma.rn.f32x2 %0, a, f, %0;\n\t"
      "fma.rn.f32x2 %0, b, f, %0;\n\t}"
      : "+l"(*acc) : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
}
__device__ __forceinline__ bool plain(uint64_t acc) {  // for every lane of the warp
  const float x = __uint_as_float((uint32_t)acc), y = __uint_as_float((uint32_t)(acc >> 32));
  return !__any_sync(0xffffffffu, !(fabsf(x) + fabsf(y) < INFINITY));
}
// hi + lo += A B with A and B given as split values; lo lo is left out where a value is in lo alone
// (with an infinity there the other's lo could only add to or spoil what its hi gives).  The
// tensor cores cut an accumulator's low bits off at every product, so the small products have an
// accumulator of their own, and both are kept for a few products only and then added up with
// rounded fp32 additions (one accumulator throughout: 2.6e-6 off at D = 256, 3.1e-7 now).
template <bool SAFE>
__device__ __forceinline__ void mma_split(float (&hi)[4], float (&lo)[4], const uint32_t (&ah)[4],
                                          const uint32_t (&al)[4], const uint32_t (&bh)[2],
                                          const uint32_t (&bl)[2]) {
  if constexpr (!SAFE) mma_tf32(lo, al, bl[0], bl[1]);
  mma_tf32(lo, al, bh[0], bh[1]);
  mma_tf32(lo, ah, bl[0], bl[1]);
  mma_tf32(hi, ah, bh[0], bh[1]);
}

// Q of the piece in shared memory: AT_G NG rows (zeros past the piece's heads); rows are 64 bytes
// longer than D elements, so that the 8 lanes of a 16-byte read phase (2 rows x 4 chunks)
// fall on different banks.  fp32: hi rows, then lo rows.
template <int D, typename T, int NG> struct Smem {
  static constexpr int kRow = D * (int)sizeof(T) + 64;  // bytes
  static constexpr int kQ = AT_G * NG * kRow * (sizeof(T) == 4 ? 2 : 1);
  static constexpr int kORow = D + 2;                   // floats
  static constexpr int kO = AT_W * AT_G * kORow * 4;
  static constexpr int kBytes = kQ > kO ? kQ : kO;      // Q and O take turns
};

// What a warp keeps of its piece.
template <int D, int NG> struct Acc {
  float o[NG][D / 16][4];    // O^T tiles
  float m[NG][2], l[NG][2];  // heads 2t, 2t + 1: reference score (unscaled), this lane's sum
};

// NK blocks of 16 keys by DP elements.
template <int DP, typename T, int NK>
struct Tile {
  static constexpr int EL = 16 / (int)sizeof(T);
  uint4 r[NK][4][DP / (8 * EL)];  // K: rows g, g + 8 of even, then odd chunks; V: 4 keys
};

template <int DP, int NK>
__device__ __forceinline__ bool plain(const Tile<DP, float, NK>& x) {
  uint64_t acc = 0;
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int z = 0; z < 4; ++z)
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) probe(x.r[i][z][c], &acc);
  return plain(acc);
}

// One 16-key block's place in the cache: rows kept, and the block's first row.
struct Block {
  int64_t off;  // element offset of its first row
  int n;        // rows that count (0..16)
};

// s += the scores of NK blocks over one part of D, for heads 2t, 2t + 1 of the lane's rows g and
// g + 8; qs points at the part in Q's rows.
template <int D, int DP, int NK, int NG>
__device__ __forceinline__ void scores(const Tile<DP, __nv_bfloat16, NK>& k, const char* qs,
                                       bool /*qplain*/, float (&s)[NG][NK][4]) {
  constexpr int kRow = Smem<D, __nv_bfloat16, NG>::kRow;
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int c = 0; c < DP / 32; ++c)
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      const uint4 b =
          *reinterpret_cast<const uint4*>(qs + (q * AT_G + g) * kRow + (t + 4 * c) * 16);
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint4 a0 = k.r[i][(c & 1) * 2][c >> 1], a1 = k.r[i][(c & 1) * 2 + 1][c >> 1];
        mma_bf16(s[q][i], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
        mma_bf16(s[q][i], a0.z, a1.z, a0.w, a1.w, b.z, b.w);
      }
    }
}
template <bool SAFE, int D, int DP, int NK, int NG>
__device__ __forceinline__ void scores_split(const Tile<DP, float, NK>& k, const char* qs,
                                             float (&s)[NG][NK][4]) {
  constexpr int kRow = Smem<D, float, NG>::kRow;
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int c0 = 0; c0 < DP / 16; c0 += 4) {  // 64 elements: 8 products of hi
    float hi[NG][NK][4] = {}, lo[NG][NK][4] = {};
#pragma unroll
    for (int c = c0; c < c0 + 4; ++c) {
      uint4 bh[NG], bl[NG];
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        const char* at = qs + (q * AT_G + g) * kRow + (t + 4 * c) * 16;
        bh[q] = *reinterpret_cast<const uint4*>(at);
        bl[q] = *reinterpret_cast<const uint4*>(at + AT_G * NG * kRow);
      }
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint4 a0 = k.r[i][(c & 1) * 2][c >> 1], a1 = k.r[i][(c & 1) * 2 + 1][c >> 1];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t ah[4], al[4];
          split_tf32<SAFE>(word(a0, 2 * u), &ah[0], &al[0]);
          split_tf32<SAFE>(word(a1, 2 * u), &ah[1], &al[1]);
          split_tf32<SAFE>(word(a0, 2 * u + 1), &ah[2], &al[2]);
          split_tf32<SAFE>(word(a1, 2 * u + 1), &ah[3], &al[3]);
#pragma unroll
          for (int q = 0; q < NG; ++q) {
            const uint32_t h[2] = {word(bh[q], 2 * u), word(bh[q], 2 * u + 1)};
            const uint32_t l[2] = {word(bl[q], 2 * u), word(bl[q], 2 * u + 1)};
            mma_split<SAFE>(hi[q][i], lo[q][i], ah, al, h, l);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int i = 0; i < NK; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[q][i][j] += hi[q][i][j] + lo[q][i][j];
  }
}

template <int D, int DP, int NK, int NG>
__device__ __forceinline__ void scores(const Tile<DP, float, NK>& k, const char* qs, bool qplain,
                                       float (&s)[NG][NK][4]) {
  if (plain(k) && qplain) scores_split<false, D>(k, qs, s);
  else scores_split<true, D>(k, qs, s);
}

// O^T += V^T P^T over part `part` of D; p holds the weights in the scores' layout.
template <int D, int DP, int NK, int NG>
__device__ __forceinline__ void weigh(const Tile<DP, __nv_bfloat16, NK>& v,
                                      const float (&p)[NG][NK][4], Acc<D, NG>& a, int part) {
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    uint32_t h0[NG], h1[NG], l0[NG], l1[NG];
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      split_bf16(p[q][i][0], p[q][i][1], &h0[q], &l0[q]);
      split_bf16(p[q][i][2], p[q][i][3], &h1[q], &l1[q]);
      h0[q] = transpose8x8(h0[q]);
      h1[q] = transpose8x8(h1[q]);
      l0[q] = transpose8x8(l0[q]);
      l1[q] = transpose8x8(l1[q]);
    }
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x0 = word(v.r[i][0][c], w), x1 = word(v.r[i][1][c], w);
        const uint32_t x2 = word(v.r[i][2][c], w), x3 = word(v.r[i][3][c], w);
        const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
        const uint32_t a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          mma_bf16(a.o[q][part * (DP / 16) + c * 4 + w], a0, a1, a2, a3, l0[q], l1[q]);
          mma_bf16(a.o[q][part * (DP / 16) + c * 4 + w], a0, a1, a2, a3, h0[q], h1[q]);
        }
      }
  }
}
template <bool SAFE, int D, int DP, int NK, int NG>
__device__ __forceinline__ void weigh_split(const Tile<DP, float, NK>& v,
                                            const float (&p)[NG][NK][4], Acc<D, NG>& a, int part) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    uint32_t bh[2][NG][2], bl[2][NG][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)  // keys 8u .. 8u + 7
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // P[key 8u + t + 4z][head g] from lane (t + 4z, g / 2)
          const int src = (t + 4 * z) * 4 + (g >> 1);
          const float e = __shfl_sync(0xffffffffu, p[q][i][2 * u], src);
          const float f = __shfl_sync(0xffffffffu, p[q][i][2 * u + 1], src);
          split_tf32<true, false>(__float_as_uint(g & 1 ? f : e), &bh[u][q][z], &bl[u][q][z]);
        }
#pragma unroll
    for (int c = 0; c < DP / 32; ++c)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float hi[NG][4] = {}, lo[NG][4] = {};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t ah[4], al[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            split_tf32<SAFE>(word(v.r[i][2 * u + (z >> 1)][c], 2 * w + (z & 1)), &ah[z],
                             &al[z]);
#pragma unroll
          for (int q = 0; q < NG; ++q) mma_split<SAFE>(hi[q], lo[q], ah, al, bh[u][q], bl[u][q]);
        }
#pragma unroll
        for (int q = 0; q < NG; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            a.o[q][part * (DP / 16) + c * 2 + w][j] += hi[q][j] + lo[q][j];
      }
  }
}
template <int D, int DP, int NK, int NG>
__device__ __forceinline__ void weigh(const Tile<DP, float, NK>& v, const float (&p)[NG][NK][4],
                                      Acc<D, NG>& a, int part) {
  if (plain(v)) weigh_split<false>(v, p, a, part);
  else weigh_split<true>(v, p, a, part);
}

// FULL: every row counts.
template <bool FULL, int DP, typename T, int NK>
__device__ __forceinline__ void load_k(Tile<DP, T, NK>& k, const T* base, const Block (&blk)[NK],
                                       int64_t row) {
  constexpr int EL = 16 / (int)sizeof(T);
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const T* p = base + blk[i].off + g * row + t * EL;
    const bool in0 = FULL || g < blk[i].n, in1 = FULL || g + 8 < blk[i].n;
#pragma unroll
    for (int c = 0; c < DP / (4 * EL); ++c) {
      const uint4 z = make_uint4(0, 0, 0, 0);
      k.r[i][(c & 1) * 2][c >> 1] = in0 ? ldg16(p + c * 4 * EL) : z;
      k.r[i][(c & 1) * 2 + 1][c >> 1] = in1 ? ldg16(p + 8 * row + c * 4 * EL) : z;
    }
  }
}
template <bool FULL, int DP, typename T, int NK>
__device__ __forceinline__ void load_v(Tile<DP, T, NK>& v, const T* base, const Block (&blk)[NK],
                                       int64_t row) {
  constexpr int EL = 16 / (int)sizeof(T);
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      // the fragment's keys: 2t, 2t + 1, 2t + 8, 2t + 9 (bf16), t, t + 4, t + 8, t + 12 (fp32)
      const int key = sizeof(T) == 2 ? 2 * t + (z & 1) + 8 * (z >> 1) : t + 4 * z;
      const T* p = base + blk[i].off + key * row + g * EL;
      const bool in = FULL || key < blk[i].n;
#pragma unroll
      for (int c = 0; c < DP / (8 * EL); ++c)
        v.r[i][z][c] = in ? ldg16(p + c * 8 * EL) : make_uint4(0, 0, 0, 0);
    }
}
template <int DP, typename T, int NK>
__device__ __forceinline__ void load_k(Tile<DP, T, NK>& k, const T* base, const Block (&blk)[NK],
                                       int64_t row, bool full) {
  if (full) load_k<true>(k, base, blk, row);
  else load_k<false>(k, base, blk, row);
}
template <int DP, typename T, int NK>
__device__ __forceinline__ void load_v(Tile<DP, T, NK>& v, const T* base, const Block (&blk)[NK],
                                       int64_t row, bool full) {
  if (full) load_v<true>(v, base, blk, row);
  else load_v<false>(v, base, blk, row);
}

// Q of `heads` query heads from q on, to shared memory (fp32: split).  Returns the sum of probe()s.
template <int D, typename T, int NG>
__device__ __forceinline__ uint64_t stage_q(char* smem, const T* q, int heads) {
  constexpr int EL = 16 / (int)sizeof(T), ROW = D / EL, N = AT_G * NG * ROW;  // 16-byte chunks
  constexpr int kRow = Smem<D, T, NG>::kRow;
  uint64_t acc = 0;
  if constexpr (sizeof(T) == 2 && NG == 1) {
    constexpr int PER = (N + AT_NT - 1) / AT_NT;  // all loads at once, before the barrier
    uint4 x[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + j * AT_NT;
      x[j] = make_uint4(0, 0, 0, 0);
      if (i / ROW < heads) x[j] = *reinterpret_cast<const uint4*>(q + (int64_t)i * EL);
    }
    __syncthreads();  // other warps may still read what was there
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + j * AT_NT;
      if (i < N) *reinterpret_cast<uint4*>(smem + i / ROW * kRow + i % ROW * 16) = x[j];
    }
  } else {
    __syncthreads();
    for (int i = threadIdx.x; i < N; i += AT_NT) {
      uint4 x = make_uint4(0, 0, 0, 0), hi, lo;
      if (i / ROW < heads) x = *reinterpret_cast<const uint4*>(q + (int64_t)i * EL);
      char* dst = smem + i / ROW * kRow + i % ROW * 16;
      if constexpr (sizeof(T) == 4) {
        probe(x, &acc);
        split_query(x.x, &hi.x, &lo.x);
        split_query(x.y, &hi.y, &lo.y);
        split_query(x.z, &hi.z, &lo.z);
        split_query(x.w, &hi.w, &lo.w);
        *reinterpret_cast<uint4*>(dst) = hi;
        *reinterpret_cast<uint4*>(dst + AT_G * NG * kRow) = lo;
      } else {
        *reinterpret_cast<uint4*>(dst) = x;
      }
    }
  }
  return acc;
}

// Tokens [0, n) of request b, units [t0, t1) of CTA tiles.
template <int D, typename T, int NG>
__device__ void piece(const AttnArgs& ar, char* smem, int64_t b, int n, int hk, int hg, int t0,
                      int t1, Acc<D, NG>& a, int* bad) {
  constexpr int GP = AT_G * NG, KT = Cfg<D, T, NG>::kKeys, NK = KT / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
  const int heads = min(GP, ar.G - hg * GP);
  // Q goes to shared memory with the numbers of the first pages on their way where the registers
  // allow it (517 tokens, 16 on 2 heads of 256: 8.5 us against 9.0; 400 requests of 50 to 150: 31.1
  // against 33.1; the others spill), in front of everything else where not.  Its address is worked
  // out there and not before: kept meanwhile, it costs D = 128 a twentieth.
  constexpr bool kEarly = sizeof(T) == 2 && NG == 1;
  auto queries = [&]() {
    return reinterpret_cast<const T*>(ar.q) + b * ar.qs + ((int64_t)hk * ar.G + hg * GP) * D;
  };
  uint64_t qacc = 0;
  if constexpr (!kEarly) qacc = stage_q<D, T, NG>(smem, queries(), heads);
  constexpr int kParts = Cfg<D, T, NG>::kParts, DP = D / kParts;
  const int64_t row = ar.Hk * D;  // elements between a page's rows
  const T* kc = reinterpret_cast<const T*>(ar.kc) + (int64_t)hk * D;
  const T* vc = reinterpret_cast<const T*>(ar.vc) + (int64_t)hk * D;
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
      const bool wrap = po + i >= pb;
      const bool live = blk + i < end;
      pg[i] = live ? table[pi + wrap] : -1;
      pofs[i] = (po + i - (wrap ? pb : 0)) * 16;
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
  // their places; whether all 16 rows of all of them count
  auto place = [&](Block (&x)[NK]) {
    bool full = true;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      x[i].n = cnt[i];
      if (cnt[i] > 0 && (pg[i] < 0 || pg[i] >= ar.pages)) {
        *bad = 1;
        x[i].n = 0;
      }
      x[i].off = x[i].n > 0 ? ((int64_t)pg[i] * ar.P + pofs[i]) * row : 0;
      full = full && x[i].n == 16;
    }
    return full;
  };
  // kParts = 1: k and v in turn; else the parts K 0, 1, .., V 0, 1, .. of a tile alternate between
  // the two buffers, each loaded one step ahead
  Tile<DP, T, NK> k, v;
  Block cur[NK];
  look_up();
  if constexpr (kEarly) stage_q<D, T, NG>(smem, queries(), heads);
  bool full = place(cur);
  load_k(k, kc, cur, row, full);
  if constexpr (kParts == 1) load_v(v, vc, cur, row, full);
#pragma unroll
  for (int q = 0; q < NG; ++q) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      a.o[q][i][0] = a.o[q][i][1] = a.o[q][i][2] = a.o[q][i][3] = 0.f;
    a.m[q][0] = a.m[q][1] = -INFINITY;
    a.l[q][0] = a.l[q][1] = 0.f;
  }
  look_up();
  // Q is there; fp32: whether all of it is finite
  const bool qplain = __syncthreads_and(sizeof(T) == 2 || plain(qacc));
#pragma unroll 1
  for (int tile = t0; tile < t1; ++tile) {
    Block nxt[NK];
    const bool nfull = place(nxt);
    look_up();
    float s[NG][NK][4] = {};
    if constexpr (kParts == 1) {
      scores<D>(k, smem, qplain, s);
      load_k(k, kc, nxt, row, nfull);
    } else {
#pragma unroll
      for (int z = 0; z < kParts; ++z) {
        Tile<DP, T, NK>&x = z & 1 ? v : k, &y = z & 1 ? k : v;
        if (z + 1 < kParts) load_k(y, kc + (z + 1) * DP, cur, row, full);
        else load_v(y, vc, cur, row, full);
        scores<D>(x, smem + z * DP * sizeof(T), qplain, s);
      }
    }
    if (!full)
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (g + 8 * (j >> 1) >= cur[i].n) s[q][i][j] = -INFINITY;
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
    // The reference value m of a head follows the maximum only when a score is above it by
    // AT_LAZY: weights up to 2^AT_LAZY lose nothing in fp32 sums or in bf16's relative rounding,
    // and most tiles need one vote in place of six shuffles and a pass over the accumulators.
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = mx[q][j];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          m = fmaxf(m, a.m[q][j]);
          f[j] = m == a.m[q][j] ? 1.f : ex2((a.m[q][j] - m) * ar.sl);  // 0 from -inf
          a.l[q][j] *= f[j];
          a.m[q][j] = m;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) a.o[q][i][j] *= f[j & 1];
      }
    }
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float base = a.m[q][j & 1] == -INFINITY ? 0.f : a.m[q][j & 1];
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          // the difference first: equal scores weigh the same whatever their size
          s[q][i][j] = ex2((s[q][i][j] - base) * ar.sl);
          a.l[q][j & 1] += s[q][i][j];
        }
      }
    if constexpr (kParts == 1) {
      weigh(v, s, a, 0);
      load_v(v, vc, nxt, row, nfull);
    } else {
      static_assert(kParts == 1 || kParts % 2 == 0, "V's first part goes where K's does");
#pragma unroll
      for (int z = 0; z < kParts; ++z) {
        Tile<DP, T, NK>&x = z & 1 ? v : k, &y = z & 1 ? k : v;
        if (z + 1 < kParts) load_v(y, vc + (z + 1) * DP, cur, row, full);
        else load_k(y, kc, nxt, row, nfull);
        weigh(x, s, a, z);
      }
    }
#pragma unroll
    for (int i = 0; i < NK; ++i) cur[i] = nxt[i];
    full = nfull;
  }
#pragma unroll
  for (int q = 0; q < NG; ++q)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        a.l[q][j] += __shfl_xor_sync(0xffffffffu, a.l[q][j], o);
}

// The 4 warps' results joined, AT_G heads at a time: to o and lse (slot < 0), or as the partial
// piece `slot`.
template <int D, typename T, int NG>
__device__ void finish(const AttnArgs& ar, char* smem, float2 (*ml)[AT_G], int64_t b, int h0,
                       int heads, const Acc<D, NG>& a, int64_t slot) {
  constexpr int kORow = Smem<D, T, NG>::kORow, EL = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  float* so = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    __syncthreads();  // every warp is done with Q, or with the heads before these
    if (g == 0) {
      ml[warp][2 * t] = make_float2(a.m[q][0], a.l[q][0]);
      ml[warp][2 * t + 1] = make_float2(a.m[q][1], a.l[q][1]);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int d = EL * (g + 8 * (i / (EL / 2))) + 2 * (i % (EL / 2));
      *reinterpret_cast<float2*>(so + (warp * AT_G + 2 * t) * kORow + d) =
          make_float2(a.o[q][i][0], a.o[q][i][2]);
      *reinterpret_cast<float2*>(so + (warp * AT_G + 2 * t + 1) * kORow + d) =
          make_float2(a.o[q][i][1], a.o[q][i][3]);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < min(AT_G, heads - q * AT_G) * (D / 2); x += AT_NT) {
      const int h = x / (D / 2), d = (x % (D / 2)) * 2, hp = q * AT_G + h;
      float m = -INFINITY, l = 0.f;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < AT_W; ++w) m = fmaxf(m, ml[w][h].x);
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < AT_W; ++w) {
        const float f = ex2((ml[w][h].x - base) * ar.sl);
        const float2 y = *reinterpret_cast<const float2*>(so + (w * AT_G + h) * kORow + d);
        l = fmaf(ml[w][h].y, f, l);
        o.x = fmaf(y.x, f, o.x);
        o.y = fmaf(y.y, f, o.y);
      }
      if (slot >= 0) {
        const int64_t at = slot * (AT_G * NG) + hp;
        *reinterpret_cast<float2*>(ar.acc + at * D + d) = o;
        if (d == 0) ar.ml[at] = make_float2(m, l);
        continue;
      }
      const float r = l != 0.f ? 1.f / l : 0.f;  // nothing counted: zero, not 0 / 0
      const int64_t row = b * ar.Hq + h0 + hp;
      T* out = reinterpret_cast<T*>(ar.o) + row * D + d;
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(o.x * r, o.y * r);
      else
        *reinterpret_cast<float2*>(out) = make_float2(o.x * r, o.y * r);
      if (d == 0 && ar.lse)
        ar.lse[row] = (base * ar.sl + log2f(l)) * 0.69314718055994531f;
    }
  }
}

// How the work is divided.  The units of request b are those of its
// pieces (key head x AT_G NG query heads) in a row, each its CTA tiles behind AT_START; the
// W units of all requests are divided over C CTAs, CTA c taking [W c / C, W (c + 1) / C).
// Each warp finds its way by itself: a lane sums up a run of requests, one scan over the lanes.
// AHEAD: read past the first-level cache, for a caller that has not waited for the kernel before
// it (the lengths were written before that one began).
template <int D, typename T, int NG, bool AHEAD>
struct Schedule {
  static constexpr int TK = Cfg<D, T, NG>::kKeys * AT_W;  // keys per CTA tile
  const AttnArgs& ar;
  int64_t W, incl, excl;  // all units; up to and before this lane's run
  int C, run, per;        // CTAs with work, requests per run, pieces per request

  __device__ __forceinline__ int length(int64_t b) const {
    const int32_t n = AHEAD ? __ldcg(ar.len + b) : ar.len[b];
    const int64_t cap = ar.max_blocks * ar.P;
    return (int)(n < 0 ? 0 : n > cap ? cap : n);
  }
  static __device__ __forceinline__ int tiles(int n) { return n > 0 ? (n - 1) / TK + 1 : 0; }
  __device__ __forceinline__ int64_t units(int64_t b) const {
    const int n = tiles(length(b));
    return n > 0 ? (int64_t)(n + AT_START) * per : 0;
  }
  static __device__ __forceinline__ int64_t scan(int64_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
  __device__ __forceinline__ Schedule(const AttnArgs& a, int ctas) : ar(a) {
    const int lane = threadIdx.x & 31;
    per = (int)ar.Hk * ar.HG;
    run = (int)((ar.B + 31) / 32);
    const int64_t b0 = (int64_t)lane * run, b1 = min(ar.B, b0 + run);
    int64_t sum = 0;
#pragma unroll 4
    for (int64_t b = b0; b < b1; ++b) sum += units(b);
    incl = scan(sum);
    excl = incl - sum;
    W = __shfl_sync(0xffffffffu, incl, 31);
    C = (int)(W < ctas ? W : ctas);
  }
  __device__ __forceinline__ int64_t first(int c) const { return W * c / C; }
  // the CTA of unit u: the last c with first(c) <= u
  __device__ __forceinline__ int cta_of(int64_t u) const { return (int)(((u + 1) * C - 1) / W); }
  // the request of unit u (0 <= u < W) and the unit's number in it
  __device__ __forceinline__ void find(int64_t u, int64_t* b, int64_t* r) const {
    const int lane = threadIdx.x & 31;
    const int own = __ffs(__ballot_sync(0xffffffffu, incl > u)) - 1;
    int64_t at = __shfl_sync(0xffffffffu, excl, own), b0 = (int64_t)own * run;
    if (run > 1) {
      const int64_t end = min(ar.B, b0 + run);
      for (;; b0 += 32) {
        const int64_t n = b0 + lane < end ? units(b0 + lane) : 0, x = scan(n);
        const unsigned over = __ballot_sync(0xffffffffu, at + x > u);
        if (over) {
          const int i = __ffs(over) - 1;
          at += __shfl_sync(0xffffffffu, x - n, i);
          b0 += i;
          break;
        }
        at += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    *b = b0;
    *r = u - at;
  }
};

template <int D, typename T, int NG>
__global__ void __launch_bounds__(AT_NT, Cfg<D, T, NG>::kCtas) k_attn_decode(AttnArgs ar) {
  constexpr int GP = AT_G * NG;
  extern __shared__ __align__(16) char smem[];
  __shared__ float2 ml[AT_W][AT_G];
  after_previous();
  before_next();
  const int tid = threadIdx.x, c = blockIdx.x;
  const Schedule<D, T, NG, false> sc(ar, gridDim.x);
  int bad = 0;
  if (c == 0)
    for (int64_t b = tid; b < ar.B; b += AT_NT) bad |= sc.length(b) != ar.len[b];
  // requests without tokens
  for (int64_t b = c; b < ar.B; b += gridDim.x)
    if (sc.length(b) == 0) {
      T* o = reinterpret_cast<T*>(ar.o) + b * ar.Hq * D;
      for (int64_t i = tid; i < ar.Hq * D; i += AT_NT) o[i] = (T)0.f;
      if (ar.lse)
        for (int64_t i = tid; i < ar.Hq; i += AT_NT) ar.lse[b * ar.Hq + i] = -INFINITY;
    }
  Join goes_on{0, 0, 0, -1};
  if (c < sc.C) {
    int64_t u = sc.first(c), b, r;
    const int64_t u1 = sc.first(c + 1);
    sc.find(u, &b, &r);
    int n = sc.length(b), nt = sc.tiles(n), w = nt + AT_START;
    int h = (int)(r / w), r0 = (int)(r % w);  // piece of the request, unit in it
    while (u < u1) {
      const int r1 = (int)(u1 - u < w - r0 ? r0 + (u1 - u) : w);
      const int t0 = max(0, r0 - AT_START), t1 = max(0, r1 - AT_START);
      if (t0 < t1) {
        const int hk = h / ar.HG, hg = h % ar.HG, heads = min(GP, ar.G - hg * GP);
        Acc<D, NG> a;
        piece<D, T, NG>(ar, smem, b, n, hk, hg, t0, t1, a, &bad);
        const int64_t slot = t0 == 0 && t1 == nt ? -1 : t0 == 0 ? 2 * c + 1 : 2 * c;
        finish<D, T, NG>(ar, smem, ml, b, hk * ar.G + hg * GP, heads, a, slot);
        if (t1 < nt) {  // the share ends in this piece, whose tile 0 is unit u - r0 + AT_START
          const int64_t tile0 = u - r0 + AT_START;
          goes_on = Join{(int32_t)b, h, sc.cta_of(tile0), sc.cta_of(tile0 + nt - 1)};
        }
      }
      u += r1 - r0;
      r0 = 0;
      if (u < u1 && ++h == sc.per) {
        h = 0;
        do n = sc.length(++b); while (n == 0);
        nt = sc.tiles(n);
        w = nt + AT_START;
      }
    }
  }
  if (tid == 0) ar.join[c] = goes_on;
  if (bad && ar.status) atomicOr(ar.status, kStatusClamped);
}

constexpr int AJ_NT = 32 * AT_G;  // a warp per query head
constexpr int AJ_FEW = 8;        // parts that one warp adds up by itself
constexpr int AJ_DC = 64;         // columns per item of a CTA

template <typename T>
__device__ __forceinline__ void store_o(T* o, float4 x, float r) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x * r, x.y * r);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x.z * r, x.w * r);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(o) = make_float4(x.x * r, x.y * r, x.z * r, x.w * r);
  }
}
__device__ __forceinline__ void add_scaled(float4& a, const float4& x, float f) {
  a.x = fmaf(x.x, f, a.x);
  a.y = fmaf(x.y, f, a.y);
  a.z = fmaf(x.z, f, a.z);
  a.w = fmaf(x.w, f, a.w);
}

// Adds up the parts of the pieces that were split.  CTA x serves the piece that goes on from CTA
// x of the pass above to CTA x + 1: a piece of n parts has n - 1 CTAs.  They share its items (a
// query head and AJ_DC columns), 16 parts at a time; or, with up to AJ_FEW parts (a batch: hundreds
// of pieces of 2 or 3), or up to 32 where the CTAs would have to take several items each, the
// first of them does it alone, a warp per query head (517 tokens, 9 parts, 32 items: 9.4 us for
// the whole call against 12.7 shared; 10 parts of 3 items: 13.4 shared, 14.3 alone).  Which piece
// it is, a CTA works out from the lengths while the pass still runs where one load per warp tells
// them (the kernels in front of the pass wrote them; 8 requests of 1000 tokens 11.9 against 12.8
// us); with more requests all CTAs together would wait for the same few lines of L2 (400 requests
// of 100 tokens 102 us), and it reads what the pass wrote down (44 us).
template <int D, typename T, int NG>
__global__ void __launch_bounds__(AJ_NT) k_attn_join(AttnArgs ar) {
  constexpr int GP = AT_G * NG, NW = AJ_NT / 32, MAXC = AT_SMS * Cfg<D, T, NG>::kCtas;
  __shared__ float s_w[MAXC], s_red[NW][2];
  __shared__ float4 s_o[AJ_NT / 16][AJ_DC / 4];
  const int x = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Join j{0, 0, 0, -1};
  if (ar.B <= 32) {
    const Schedule<D, T, NG, true> sc(ar, gridDim.x);
    if (x < sc.C) {
      int64_t b, r;
      const int64_t u = sc.first(x + 1) - 1;  // CTA x's last unit, in piece [start, start + w)
      sc.find(u, &b, &r);
      const int w = sc.tiles(sc.length(b)) + AT_START;
      const int64_t tile0 = u - r % w + AT_START;
      j = Join{(int32_t)b, (int32_t)(r / w), sc.cta_of(tile0), sc.cta_of(tile0 + w - AT_START - 1)};
    }
    after_previous();
    if (x < j.first || x >= j.last) return;
  } else {
    after_previous();
    j = ar.join[x];
    if (j.last < 0) return;
  }
  before_next();
  const int c = j.first, n = j.last - c + 1;
  const int hk = j.h / ar.HG, hg = j.h % ar.HG, heads = min(GP, ar.G - hg * GP);
  const int64_t row0 = (int64_t)j.b * ar.Hq + hk * ar.G + hg * GP;
  // parts: slot 2c + 1 of the piece's first CTA c, slot 2i of the CTAs behind it
  if (n <= AJ_FEW || (n <= 32 && heads * (D / AJ_DC) > n - 1)) {
    if (x > c) return;
    for (int g = warp; g < heads; g += NW) {
      auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * GP + g; };
      const float2 ml = lane < n ? ar.ml[slot(lane)] : make_float2(-INFINITY, 0.f);
      float m = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.f : m, f = ex2((ml.x - base) * ar.sl);
      float l = ml.y * f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      constexpr int V = D >= 128 ? D / 128 : 1;  // columns 4 lane + 128 v
      const bool in = D >= 128 || lane * 4 < D;
      float4 a[V];
#pragma unroll
      for (int v = 0; v < V; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < n; i0 += AJ_FEW)
#pragma unroll
        for (int j = 0; j < AJ_FEW; ++j) {
          const int i = i0 + j;
          const float fi = __shfl_sync(0xffffffffu, f, i);
          const float* part = ar.acc + slot(i) * D + lane * 4;
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (i < n && in) add_scaled(a[v], *reinterpret_cast<const float4*>(part + v * 128), fi);
        }
      const float q = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (in) store_o(reinterpret_cast<T*>(ar.o) + (row0 + g) * D + lane * 4 + v * 128, a[v], q);
      if (lane == 0 && ar.lse) ar.lse[row0 + g] = (base * ar.sl + log2f(l)) * 0.69314718055994531f;
    }
    return;
  }
  for (int item = x - c; item < heads * (D / AJ_DC); item += n - 1) {
    const int g = item % heads, d0 = item / heads * AJ_DC, col = tid % 16, first = tid / 16;
    auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * GP + g; };
    float m = -INFINITY, l = 0.f;
    for (int i = tid; i < n; i += AJ_NT) m = fmaxf(m, ar.ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();  // the last item's readers are done
    if (lane == 0) s_red[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, s_red[w][0]);
    const float base = m == -INFINITY ? 0.f : m;
    for (int i = tid; i < n; i += AJ_NT) {
      const float2 y = ar.ml[slot(i)];
      const float f = ex2((y.x - base) * ar.sl);
      s_w[i] = f;
      l = fmaf(y.y, f, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) s_red[warp][1] = l;
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = first; i < n; i += AJ_NT / 16)
      add_scaled(a, *reinterpret_cast<const float4*>(ar.acc + slot(i) * D + d0 + col * 4), s_w[i]);
    s_o[first][col] = a;
    __syncthreads();
    if (tid < AJ_DC / 4) {
      a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < AJ_NT / 16; ++i) add_scaled(a, s_o[i][tid], 1.f);
      l = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) l += s_red[w][1];
      store_o(reinterpret_cast<T*>(ar.o) + (row0 + g) * D + d0 + tid * 4, a,
              l != 0.f ? 1.f / l : 0.f);
      if (tid == 0 && d0 == 0 && ar.lse)
        ar.lse[row0 + g] = (base * ar.sl + log2f(l)) * 0.69314718055994531f;
    }
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool ok16(const void* p, int64_t n) { return n == 0 || (p && aligned16(p)); }
bool ok4(const void* p, int64_t n) { return n == 0 || (p && ((uintptr_t)p & 3u) == 0); }

gdn_status check_problem(const gdn_attn_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (p->B < 0 || p->Hq < 1 || p->Hk < 1 || p->Hq % p->Hk != 0 || p->pages < 0 ||
      p->max_blocks < 0 || p->page_size < 1 || p->D < 1 || !isfinite(p->scale) ||
      !isfinite(fmaxf(p->scale, 0.f) * AT_LOG2E))
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

// CTAs of the pass and the workspace's parts (a fixed count per kind, so that results do not
// depend on the device).
struct Plan {
  int ctas;
  size_t ml, acc, total;
};
template <int D, typename T, int NG>
Plan plan_of() {
  Plan pl;
  pl.ctas = AT_SMS * Cfg<D, T, NG>::kCtas;
  const size_t parts = (size_t)pl.ctas * 2 * AT_G * NG;
  pl.ml = (pl.ctas * sizeof(Join) + 255) & ~(size_t)255;
  pl.acc = pl.ml + ((parts * sizeof(float2) + 255) & ~(size_t)255);
  pl.total = pl.acc + parts * D * sizeof(float);
  return pl;
}
template <int D, typename T>
size_t workspace_of() {
  const size_t a = plan_of<D, T, 1>().total, b = plan_of<D, T, 2>().total;
  return a > b ? a : b;
}

// Runs f with the call's head dim and type as template arguments.
template <typename F>
auto with_types(const gdn_attn_problem* p, F f) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  using D256 = std::integral_constant<int, 256>;
  if (p->dtype == GDN_BF16) {
    const __nv_bfloat16 t{};
    return p->D == 64 ? f(D64(), t) : p->D == 128 ? f(D128(), t) : f(D256(), t);
  }
  return p->D == 64 ? f(D64(), 0.f) : p->D == 128 ? f(D128(), 0.f) : f(D256(), 0.f);
}

template <int D, typename T, int NG>
cudaError_t launch(AttnArgs ar, char* ws, cudaStream_t st) {
  const Plan pl = plan_of<D, T, NG>();
  ar.HG = (ar.G + AT_G * NG - 1) / (AT_G * NG);
  ar.join = (Join*)ws;
  ar.ml = (float2*)(ws + pl.ml);
  ar.acc = (float*)(ws + pl.acc);
  const cudaError_t e = launch_behind(k_attn_decode<D, T, NG>, dim3(pl.ctas), AT_NT,
                                      Smem<D, T, NG>::kBytes, st, ar);
  if (e != cudaSuccess) return e;
  return launch_behind(k_attn_join<D, T, NG>, dim3(pl.ctas), AJ_NT, 0, st, ar);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_attn_decode_workspace_size(const gdn_attn_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  *bytes = with_types(p, [](auto d, auto t) { return workspace_of<d(), decltype(t)>(); });
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
  ar.G = (int)(p->Hq / p->Hk);
  ar.sl = (p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->D)) * AT_LOG2E;
  ar.lazy = fminf(AT_LAZY / ar.sl, 1e30f);
  ar.q = q;
  ar.kc = k_cache;
  ar.vc = v_cache;
  ar.table = block_table;
  ar.len = seq_len;
  ar.o = o;
  ar.lse = lse;
  ar.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = with_types(p, [&](auto d, auto t) {
    // one pass over the cache serves 8 query heads of a key head, or 16
    return ar.G <= AT_G ? launch<d(), decltype(t), 1>(ar, (char*)workspace, st)
                        : launch<d(), decltype(t), 2>(ar, (char*)workspace, st);
  });
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
