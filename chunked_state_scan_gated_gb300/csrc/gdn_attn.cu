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
#include "gdn_attn_split.cuh"

namespace gdn {
namespace {

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
template <int D, typename T, int NG>
struct Smem {
  static constexpr int kRow = D * (int)sizeof(T) + 64;  // bytes
  static constexpr int kQ = AT_G * NG * kRow * (sizeof(T) == 4 ? 2 : 1);
  static constexpr int kORow = D + 2;                   // floats
  static constexpr int kO = AT_W * AT_G * kORow * 4;
  static constexpr int kBytes = kQ > kO ? kQ : kO;      // Q and O take turns
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
__device__ void run_piece(const AttnArgs& ar, char* smem, int64_t b, int n, int hk, int hg, int t0,
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

template <int D, typename T, int NG>
struct Piece {
  template <typename... A>
  static __device__ __forceinline__ void run(A&&... a) { run_piece<D, T, NG>(a...); }
};

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
  const AttnArgs ar =
      args_of(p, q, k_cache, v_cache, block_table, seq_len, o, lse, status, AT_LAZY);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = with_types(p, [&](auto d, auto t) {
    // one pass over the cache serves 8 query heads of a key head, or 16
    return ar.G <= AT_G ? launch<d(), decltype(t), 1>(ar, (char*)workspace, st)
                        : launch<d(), decltype(t), 2>(ar, (char*)workspace, st);
  });
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
