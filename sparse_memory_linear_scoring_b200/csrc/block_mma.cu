// block_mma.cu -- block-selected attention on the tensor cores (bf16), forward.
//
// Each query picks its own blocks, so a tile of neighbouring queries shares few of
// them, and a query alone has too few rows (the heads of its group) for a tensor-core
// tile.  The other way round every tile is full: a CTA takes one block of keys and
// the list of (query, slot) pairs that name it (the plan of block_select.cu), and its
// rows are those pairs times the heads of the group.  Keys and values are read once
// per item of 512 to 1024 rows; a row has one block of scores, so its softmax needs no
// running maximum.  What this costs is a partial result per (query, slot, head) --
// d halves, a log-sum-exp and a scale, written here and read once by the join:
//     o = sum_s exp(lse_s - lse) o_s,   lse = log sum_s exp(lse_s).
// Partials are halves scaled by the row's largest element to 2^15: 11 significant bits
// for elements down to 2^-29 of it, an error of 2^-12 beside the 2^-9 of the weights' and
// the result's bf16; float32 partials would double the bytes that bound this path.
#include <cuda_fp16.h>

#include "block_internal.cuh"

namespace sdm {

// Rows of an item.  Its keys' load and the CTA's start cost as much as a tile of 128 rows
// and a half; longer items share that among more, shorter ones keep three CTAs an SM busy
// to the end: as long as there are four rounds of them, up to 1024 (8192 tokens, 16 heads
// of 128: 445 us with 512, 422 with 1024, 434 with 2048).
static int item_rows(const sdm_block_dims* d, int nq) {
  const long long rows = (long long)d->B * d->H * nq * d->n_sel;
  long long n = rows / (4 * 3 * 148);
  n = n < 512 ? 512 : n > 1024 ? 1024 : n;
  return int(n / 128 * 128);
}

// A row of o from its partials: D / 8 lanes a row.  A lane first takes every LN-th slot
// of the list for the maximum and the sum, then each of LN slots at a time for its
// weight, which the others get by shuffles, with 4 partial rows' loads in flight.  The
// (query, slot) pairs without keys have no partial and are skipped by the same test
// that left them out.
template <int D>
__global__ void __launch_bounds__(64)
k_blk_join(BlkArgs a, BlkFwdWs w, const int32_t* __restrict__ idx, __nv_bfloat16* __restrict__ o,
           float* __restrict__ lse) {
  wait_for_previous();
  constexpr int LN = D / 8;
  const long long i = ((long long)blockIdx.x * 64 + threadIdx.x) / LN;
  const int ln = threadIdx.x % LN, c = ln * 8;
  const bool in = i < (long long)a.B * a.G * a.nq * a.R;
  const long long i0 = in ? i : 0;
  const long long bt = i0 / a.R;
  const int r = int(i0 - bt * a.R);
  const int bg = int(bt / a.nq), t = int(bt - (long long)bg * a.nq), b = bg / a.G, h = (bg - b * a.G) * a.R + r;
  const int32_t* list = idx + ((size_t)bg * a.Tq + a.q0 + t) * a.n_sel;
  const int p = blk_pos0(a, b) + a.q0 + t;
  const float2* ml = w.ml + (size_t)bt * a.n_sel * a.R + r;
  const __half* part = static_cast<const __half*>(w.part) + ((size_t)bt * a.n_sel * a.R + r) * D + c;
  float m = -INFINITY;
  for (int s = ln; s < a.n_sel; s += LN)
    if (blk_keys(a, list[s], p) > 0) {
      const float x = ml[(size_t)s * a.R].x;
      m = fmaxf(m, x);
    }
#pragma unroll
  for (int z = 1; z < LN; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < a.n_sel; s0 += LN) {
    const int s = s0 + ln;
    float f = -1.f;  // no partial
    if (s < a.n_sel && blk_keys(a, list[s], p) > 0) {
      const float2 u = ml[(size_t)s * a.R];
      const float e = exp2f(u.x - base);
      l += e;
      f = e * u.y;
    }
#pragma unroll
    for (int z0 = 0; z0 < LN; z0 += 4) {
      uint4 x[4];
      float fz[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        fz[z] = __shfl_sync(0xffffffffu, f, z0 + z, LN);
        x[z] = make_uint4(0u, 0u, 0u, 0u);
        if (fz[z] != -1.f) x[z] = __ldcs(reinterpret_cast<const uint4*>(part + (size_t)(s0 + z0 + z) * a.R * D));
      }
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const __half2* hx = reinterpret_cast<const __half2*>(&x[z]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 y = __half22float2(hx[u]);
          acc[2 * u] = fmaf(fz[z], y.x, acc[2 * u]);
          acc[2 * u + 1] = fmaf(fz[z], y.y, acc[2 * u + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int z = 1; z < LN; z <<= 1) l += __shfl_xor_sync(0xffffffffu, l, z);
  if (!in) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int z = 0; z < 8; ++z) acc[z] *= inv;
  Vec<__nv_bfloat16, 8>::store(o + row_off(a.so, b, h, a.q0 + t) + c, acc);
  if (lse && c == 0)
    lse[((size_t)b * a.H + h) * a.Tq + a.q0 + t] = l == 0.f ? -INFINITY : (base + log2f(l)) / kLog2e;
}

// ---------------------------------------------------------------- host side
// Query by query the listed keys and values are read anew for each query (and 16 heads),
// at about 4 TB/s; block by block the plan, the tiles and the join take about 33 us
// before the work counts, and short calls have few queries a block anyway.  d = 128,
// 16 blocks of 64, one sequence, 4 groups: 64 queries (134 MB) 33 us query by query, 39
// block by block; 128 queries 64 and 44; 16 groups, 32 queries 64 and 56.
bool blk_tiles_pay(const sdm_block_dims* d) {
  const long long hc = (d->H / d->G + 15) / 16;
  return d->in_dtype == SDM_DTYPE_BF16 && d->Tq >= 32 &&
         hc * d->B * d->G * d->Tq * d->n_sel * d->block * d->d * 4 > (128LL << 20);
}

// Queries per pass: as many as keep the partials within 2 GiB (at least 128).
int blk_chunk(const sdm_block_dims* d) {
  const long long per = (long long)d->B * d->H * d->n_sel * (d->d * 2 + 8);
  long long n = (2LL << 30) / per;
  if (n < 128) n = 128;
  if (n > d->Tq) n = d->Tq;
  const long long passes = (d->Tq + n - 1) / n;  // even passes
  return int((d->Tq + passes - 1) / passes);
}

BlkFwdWs blk_fwd_ws(const sdm_block_dims* d, int nq, void* base) {
  BlkFwdWs w;
  w.plan = blk_plan(d, nq, item_rows(d, nq), base);
  const size_t rows = size_t(d->B) * d->H * nq * d->n_sel;
  char* b = static_cast<char*>(base);
  size_t o = w.plan.bytes;
  w.ml = reinterpret_cast<float2*>(b + o);
  o = (o + rows * 8 + 255) & ~size_t(255);
  w.part = b + o;
  w.bytes = o + rows * d->d * 2;
  return w;
}

template <int D>
static cudaError_t launch_fwd(const sdm_block_dims* d, BlkArgs a, const void* q, const void* k,
                              const void* v, const int32_t* idx, void* o, float* lse,
                              void* workspace, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const int chunk = blk_chunk(d);
  for (int q0 = 0; q0 < d->Tq; q0 += chunk) {
    a.q0 = q0;
    a.nq = d->Tq - q0 < chunk ? d->Tq - q0 : chunk;
    const BlkFwdWs w = blk_fwd_ws(d, a.nq, workspace);
    cudaError_t e = launch_blk_plan(a, w.plan, idx, s);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)a.B * a.G * w.plan.most;
    if (grid >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    e = launch_blk_tc(a, w, unsigned(grid), q, k, v, s);
    if (e != cudaSuccess) return e;
    const long long n = (long long)a.B * a.H * a.nq * (D / 8);
    launch_after(k_blk_join<D>, unsigned((n + 63) / 64), 64, 0, s, a, w, idx, (bf*)o, lse);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_blk_fwd_mma(const sdm_block_dims* d, BlkArgs a, const void* q, const void* k,
                               const void* v, const int32_t* idx, void* o, float* lse,
                               void* workspace, cudaStream_t s) {
  if (a.d == 32) return launch_fwd<32>(d, a, q, k, v, idx, o, lse, workspace, s);
  if (a.d == 64) return launch_fwd<64>(d, a, q, k, v, idx, o, lse, workspace, s);
  return launch_fwd<128>(d, a, q, k, v, idx, o, lse, workspace, s);
}

}  // namespace sdm
