// block_internal.cuh -- sparse attention over selected blocks (block_select.cu,
// block_attn.cu, block_bwd.cu, block_mma.cu): sizes, the plan, shared device code.
//
// Keys are cut into blocks of `block` consecutive positions.  The query at
// position p (the last Tq of the sequence's keys) has a list of blocks; it
// attends, by softmax, to the keys at positions <= p of the listed blocks.  The
// heads of a group share keys, values and lists.
#pragma once

#include "seq_internal.cuh"

namespace sdm {

struct BlkArgs {
  int B, H, G, R;       // R = H / G heads per group
  int Tq, Tk, d, bs, n_sel;
  int nb;               // blocks, the last one possibly partial
  float scale;
  sdm_strides sq, sk, sv, so;
  const int32_t* lengths;
};

// Position of query 0 of batch b (negative: that many queries have no key).
__device__ __forceinline__ int blk_pos0(const BlkArgs& a, int b) {
  return seq_len(a.lengths, b, a.Tk) - a.Tq;
}

// Keys that a query at position p sees of block j of its list; 0 for an entry
// that is no block or lies wholly behind p.
__device__ __forceinline__ int blk_keys(const BlkArgs& a, int j, int p) {
  if (j < 0 || j >= a.nb) return 0;
  const int n = p - j * a.bs + 1;
  return n < 0 ? 0 : (n > a.bs ? a.bs : n);
}

// The plan: for every (b, group), the (query, list slot) pairs of each block in
// query order, as entry = query * n_sel + slot.
struct BlkPlan {
  int seg, nseg;         // queries per counting segment, segments
  int* hist;             // [BG][nseg][nb] counts, then first positions
  int* first;            // [BG][nb + 1] first entry of each block
  int* entry;            // [BG][Tq * n_sel]
  size_t bytes;
};
BlkPlan blk_plan(const sdm_block_dims* d, void* base);
cudaError_t launch_blk_plan(const BlkArgs& a, const BlkPlan& p, const int32_t* idx, cudaStream_t s);

int blk_check(const sdm_block_dims* d);
BlkArgs blk_args(const sdm_block_dims* d, const sdm_block_views* v, const int32_t* lengths);
int blk_views_ok(const sdm_block_views* v);

}  // namespace sdm
