// block_internal.cuh -- sparse attention over selected blocks (block_select.cu,
// block_attn.cu, block_bwd.cu, block_mma.cu, block_bwd_mma.cu,
// block_step.cu): sizes, the plan, shared device code.
//
// Keys are cut into blocks of `block` consecutive positions.  The query at
// position p (the last Tq of the sequence's keys) has a list of blocks; it
// attends, by softmax, to the keys at positions <= p of the listed blocks.  The
// heads of a group share keys, values and lists.
#pragma once

#include "seq_internal.cuh"

namespace sdm {

// Division of 0 <= n < 2^31 by a fixed positive number: a multiply-high, an add and a
// shift (with s = ceil(log2 d) and m = ceil(2^(32 + s) / d) - 2^32 it is exact).
struct FastDiv {
  uint32_t m, s, d;
  __device__ __forceinline__ int div(int n) const {
    return int((__umulhi(uint32_t(n), m) + uint32_t(n)) >> s);
  }
};
inline FastDiv fast_div(int d) {
  FastDiv f;
  f.d = uint32_t(d);
  f.s = 0;
  while ((1ull << f.s) < f.d) ++f.s;
  f.m = uint32_t(((1ull << (32 + f.s)) + f.d - 1) / f.d - (1ull << 32));
  return f;
}

struct BlkArgs {
  int B, H, G, R;       // R = H / G heads per group
  int Tq, Tk, d, bs, n_sel;
  int nb;               // blocks, the last one possibly partial
  int q0, nq;           // queries of this pass: [q0, q0 + nq) of Tq
  float scale;
  FastDiv by_R, by_sel;
  sdm_strides sq, sk, sv, so;
  const int32_t* lengths;
};

// Position of query 0 of batch b, counted from the call's first query (negative:
// that many queries have no key).
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

// The plan of a pass over nq queries: for every (b, group), the (query, list slot)
// pairs of each block in query order, as entry = (query - q0) * n_sel + slot, and the
// blocks' rows (pair, head of the group) cut into items of at most `rows` rows.
struct BlkPlan {
  int seg, nseg;         // queries per counting segment, segments
  int rows;              // rows per item
  int most;              // items per (b, group), at most
  int* hist;             // [BG][nseg][nb] counts, then first positions
  int* first;            // [BG][nb + 1] first entry of each block
  int* item;             // [BG][nb + 1] first item of each block
  int* entry;            // [BG][nq * n_sel]
  size_t bytes;
};
BlkPlan blk_plan(const sdm_block_dims* d, int nq, int rows, void* base);

// The block of an item (binary search in the items' first numbers), -1 behind the last.
__device__ __forceinline__ int blk_of_item(const int* item, int nb, int it) {
  if (it >= item[nb]) return -1;
  int lo = 0, hi = nb - 1;  // item[lo] <= it < item[hi + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (item[mid] <= it) lo = mid; else hi = mid - 1;
  }
  return lo;
}
cudaError_t launch_blk_plan(const BlkArgs& a, const BlkPlan& p, const int32_t* idx, cudaStream_t s);

// Tensor-core forward pass (block_mma.cu): block by block over the lists' pairs,
// partial results per (query, slot, head), then a join.
struct BlkFwdWs {
  BlkPlan plan;
  float2* ml;      // [BG][nq][n_sel][R] log-sum-exp (base 2) and scale of each partial row
  void* part;      // [BG][nq][n_sel][R][d] half
  size_t bytes;
};
BlkFwdWs blk_fwd_ws(const sdm_block_dims* d, int nq, void* base);
cudaError_t launch_blk_tc(const BlkArgs& a, const BlkFwdWs& w, unsigned grid, const void* q, const void* k,
                          const void* v, cudaStream_t s);  // the tiles (block_tc.cu)
int blk_chunk(const sdm_block_dims* d);        // queries per pass
bool blk_tiles_pay(const sdm_block_dims* d);   // whether the tensor-core pass is taken
cudaError_t launch_blk_fwd_mma(const sdm_block_dims* d, BlkArgs a, const void* q, const void* k,
                               const void* v, const int32_t* idx, void* o, float* lse,
                               void* workspace, cudaStream_t s);

// Query by query on the tensor cores (block_step.cu); bf16, views in 16-byte pieces.
cudaError_t launch_blk_step(const BlkArgs& a, const void* q, const void* k, const void* v,
                            const int32_t* idx, void* o, float* lse, cudaStream_t s);

// Tensor-core backward pass (block_bwd_mma.cu).
struct BlkBwdWs {
  float* delta;    // [B][H][Tq] do.o
  float* sum;      // [2][BG][Tk][d] dk, dv so far, where there is more than one pass
  BlkPlan plan;
  float4* mul;     // [BG][nq][n_sel][R][block / keys] scales of each part of dq and of sum P k, sum of dS
  void* part;      // [BG][nq][n_sel][R][block / keys][d] half: dq
  void* kpart;     // [BG][nq][n_sel][R][block / keys][d] e4m3: sum P k
  float* kv;       // [BG][items][block / keys][2][keys][d] parts of dk, dv
  size_t bytes;
};
BlkBwdWs blk_bwd_ws(const sdm_block_dims* d, int nq, void* base);
bool blk_bwd_tiles_pay(const sdm_block_dims* d);
int blk_bwd_chunk(const sdm_block_dims* d);
// dk, dv from the items' parts w.kv of kt keys each (with begin and end: of one pass).
cudaError_t launch_blk_dkv(const BlkArgs& a, const BlkBwdWs& w, bool bf16, void* dk, void* dv,
                           const sdm_strides& sdk, const sdm_strides& sdv, int kt, bool begin, bool end,
                           cudaStream_t s);
cudaError_t launch_blk_bwd_mma(const sdm_block_dims* d, BlkArgs a, const void* q, const void* k,
                               const void* v, const int32_t* idx, const void* o, const float* lse,
                               const void* d_o, void* dq, void* dk, void* dv,
                               const sdm_block_views* gv, void* workspace, cudaStream_t s);

int blk_check(const sdm_block_dims* d);
BlkArgs blk_args(const sdm_block_dims* d, const sdm_block_views* v, const int32_t* lengths);
int blk_views_ok(const sdm_block_views* v);

}  // namespace sdm
