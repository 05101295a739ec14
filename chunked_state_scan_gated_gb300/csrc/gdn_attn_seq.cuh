// gdn_attn_seq.cuh -- what the kernels of gdn_attn_fwd and gdn_attn_bwd share: the call's
// arguments and the way from a CTA's number to its tile of a packed sequence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.h"
#include "gdn_launch.cuh"

namespace gdn {
namespace seq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// A tile of rows (queries or keys) of one sequence.
struct Tile {
  int q0, nq;  // the sequence's query rows
  int k0, nk;  // its key rows
  int at;      // the tile's first row in the sequence
};

// The tiles of one side, in the order in which CTAs take them: those with the most work first, so
// that the last to begin are the shortest.
struct Tiles {
  const Tile* list;  // null: one sequence, or sequences of one length
  const int* count;  // of the list
  int rows;          // per tile
  int most;          // upper bound of the count, known on the host
};

struct SeqArgs {
  int64_t Nq, Nk, qs, ks, vs;  // rows; elements between tokens
  int n_seqs, Hq, Hk, G, causal;
  int pack;  // bf16 forward: query heads of a key head that share a tile, a row per token and head
  float scale, sl;  // of the scores; times log2(e)
  const void *q, *k, *v, *o, *dO;
  const int32_t *cuq, *cuk;
  void *out, *dq, *dk, *dv;
  float* lse;          // forward: written (nullable); backward: read
  float *lse2, *delta; // [Hq][Nq]: lse log2(e) (+inf where no key is seen), dO.o
  Tiles tq, tk;
  float *part_k, *part_v;  // [splits][Nk][Hk][D]: dk, dv of a part of a key head's query heads
  int splits;              // 1: none, dk and dv are written themselves
  float *part_o, *part_lse;  // [parts][Nq][Hq](D): o and log2-sum over a part of the keys
  int parts;               // 1: none, o and lse are written themselves
  int late;                // 1: the kernel waits for the one before it at its end, not first
  int32_t* status;
};

constexpr int kMaxParts = 32;

__device__ __forceinline__ int clamp_row(int64_t x, int64_t n) {
  return (int)(x < 0 ? 0 : x > n ? n : x);
}

// The tiles that there are, at most `most`.
template <bool KEYS>
__device__ __forceinline__ int tiles_there(const SeqArgs& a) {
  const Tiles& ts = KEYS ? a.tk : a.tq;
  if (ts.list) return *ts.count;
  int rows = (int)((KEYS ? a.Nk : a.Nq) / a.n_seqs);
  if (a.cuq) {
    const int32_t* cu = KEYS && a.cuk ? a.cuk : a.cuq;
    const int64_t n = KEYS ? a.Nk : a.Nq;
    rows = max(0, clamp_row(cu[1], n) - clamp_row(cu[0], n));
  }
  return (rows + ts.rows - 1) / ts.rows * a.n_seqs;
}

// The idx-th tile; false: there is none.  KEYS: tiles of the key side.
template <bool KEYS>
__device__ __forceinline__ bool tile_of(const SeqArgs& a, int idx, Tile* t) {
  const Tiles& ts = KEYS ? a.tk : a.tq;
  if (ts.list) {
    if (idx >= *ts.count) return false;
    *t = ts.list[idx];
    return true;
  }
  int b = 0, i = idx;
  if (a.cuq) {
    t->q0 = clamp_row(a.cuq[0], a.Nq);
    t->nq = max(0, clamp_row(a.cuq[1], a.Nq) - t->q0);
    const int32_t* ck = a.cuk ? a.cuk : a.cuq;
    t->k0 = clamp_row(ck[0], a.Nk);
    t->nk = max(0, clamp_row(ck[1], a.Nk) - t->k0);
  } else {
    b = idx % a.n_seqs;
    i = idx / a.n_seqs;
    t->nq = (int)(a.Nq / a.n_seqs);
    t->nk = (int)(a.Nk / a.n_seqs);
    t->q0 = b * t->nq;
    t->k0 = b * t->nk;
  }
  const int n = KEYS ? t->nk : t->nq, tiles = (n + ts.rows - 1) / ts.rows;
  if (i >= tiles) return false;
  // causal: late queries see the most keys, early keys are seen by the most queries
  t->at = (KEYS ? i : tiles - 1 - i) * ts.rows;
  return true;
}

// Keys that the queries [at, at + n) of the tile see between them: [0, result).
__device__ __forceinline__ int keys_seen(const SeqArgs& a, const Tile& t, int n) {
  if (!a.causal) return t.nk;
  return max(0, min(t.nk, min(t.at + n, t.nq) + t.nk - t.nq));
}
// The first query that sees a key of a tile that begins at key t.at (t.nq: none).
__device__ __forceinline__ int first_query(const SeqArgs& a, const Tile& t) {
  if (!a.causal) return 0;
  return min(t.nq, max(0, t.at - (t.nk - t.nq)));
}

// One sequence by its offsets: they are checked where there is no list to be made.
__device__ __forceinline__ void check_single(const SeqArgs& a) {
  if (!a.cuq || a.n_seqs != 1 || !a.status) return;
  const int32_t* ck = a.cuk ? a.cuk : a.cuq;
  if (a.cuq[0] < 0 || a.cuq[1] < a.cuq[0] || a.cuq[1] > a.Nq || ck[0] < 0 || ck[1] < ck[0] ||
      ck[1] > a.Nk)
    atomicOr(a.status, kStatusClamped);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- kernels of gdn_attn_seq_tc.cu (bf16) ----
struct TcPlan {
  int fwd_rows, dq_rows, dkv_rows;  // rows per tile
};
// Query heads that share a tile of the forward: the largest power of two, up to 16, in the group.
inline int tc_pack(int64_t G) { return G % 16 == 0 ? 16 : G % 8 == 0 ? 8 : G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1; }
TcPlan tc_plan(int D);
cudaError_t launch_fwd_tc(const SeqArgs& a, int D, cudaStream_t st);
cudaError_t launch_bwd_tc(const SeqArgs& a, int D, cudaStream_t st);
// dk and dv from their parts, o and lse from the parts of the keys, in either type.
cudaError_t launch_sum(const SeqArgs& a, int D, bool fp32, cudaStream_t st);
cudaError_t launch_merge(const SeqArgs& a, int D, bool fp32, cudaStream_t st);

}  // namespace seq
}  // namespace gdn
