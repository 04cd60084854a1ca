// block_select.cu -- block means, the selection of blocks by them, and the plan
// that turns the queries' lists into the blocks' lists.
//
// Mean of block j: kc_j = (1 / block) sum of its keys, in the keys' type, for
// complete blocks.  Score of block j for a query of group g: the sum over the
// group's heads of q_h . kc_j = (sum_h q_h) . kc_j.  The list of a query at
// position p: its own block c = p / block, then the best n_sel - 1 of the blocks
// before it, higher score first and lower index at a tie, then -1.
#include "block_internal.cuh"

namespace sdm {

// ---------------------------------------------------------------- means
// A CTA per block: a thread sums a share of the rows of one 4-column piece.  The sums
// are double: exact for bf16 keys whatever the order, so the means (and with
// them the lists) do not depend on how the rows are shared out.
template <typename Tin>
__global__ void __launch_bounds__(128)
k_blk_pool(BlkArgs a, sdm_strides skc, const Tin* __restrict__ k, Tin* __restrict__ kc, int first,
           int count, int vec) {
  __shared__ double red[128][4];
  const int bg = blockIdx.x / count, j = first + blockIdx.x - bg * count;
  const int b = bg / a.G, g = bg - b * a.G;
  const int nc = a.d >> 2, sub = threadIdx.x / nc, nsub = 128 / nc, c = (threadIdx.x % nc) * 4;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const Tin* p = k + row_off(a.sk, b, g, j * a.bs) + c;
  for (int r = sub; r < a.bs; r += nsub) {
    float f[4];
    if (vec) {
      Vec<Tin, 4>::load(p + (long long)r * a.sk.t, f);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = to_f32(p[(long long)r * a.sk.t + e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += double(f[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[threadIdx.x][e] = s[e];
  __syncthreads();
  if (sub == 0) {
    Tin* o = kc + row_off(skc, b, g, j) + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      for (int q = 1; q < nsub; ++q) s[e] += red[threadIdx.x + q * nc][e];
      o[e] = from_f32<Tin>(float(s[e] / a.bs));
    }
  }
}

// ---------------------------------------------------------------- selection
// Scores in double on CUDA cores: a rounding difference at a list's boundary
// would change the list, and float sums differ from one order to the next by
// more than neighbouring scores do about once in 10^5 rows.
constexpr int kSelQ = 32;   // queries per CTA
constexpr int kSelJ = 32;   // blocks per tile
constexpr int kSelMost = 64;

__host__ __device__ inline size_t blk_select_smem(int d) {
  // qs, kt [32][d + 1] double, scores [32][33] double, lists [32][64] (double, int)
  return size_t(8) * (2 * 32 * (d + 1) + 32 * 33 + 32 * kSelMost) + size_t(4) * 32 * kSelMost;
}

// Insert (s, j) into a descending list of m entries held in shared memory, all
// lanes of the warp together; ls[m-1] < s on entry.
__device__ __forceinline__ void list_insert(double* ls, int* li, int m, double s, int j) {
  const int lane = threadIdx.x & 31;
  const double a0 = lane < m ? ls[lane] : 0.0, a1 = lane + 32 < m ? ls[lane + 32] : 0.0;
  const int i0 = lane < m ? li[lane] : 0, i1 = lane + 32 < m ? li[lane + 32] : 0;
  const unsigned b0 = __ballot_sync(0xffffffffu, lane < m && a0 >= s);
  const unsigned b1 = __ballot_sync(0xffffffffu, lane + 32 < m && a1 >= s);
  const int pos = __popc(b0) + __popc(b1);
  __syncwarp();
  if (lane >= pos && lane + 1 < m) { ls[lane + 1] = a0; li[lane + 1] = i0; }
  if (lane + 32 >= pos && lane + 33 < m) { ls[lane + 33] = a1; li[lane + 33] = i1; }
  if (lane == 0) { ls[pos] = s; li[pos] = j; }
  __syncwarp();
}

template <typename Tin>
__global__ void __launch_bounds__(256)
k_blk_select(BlkArgs a, sdm_strides skc, const Tin* __restrict__ q, const Tin* __restrict__ kc,
             int nkc, int32_t* __restrict__ idx) {
  extern __shared__ __align__(16) double sd[];
  const int d = a.d, dp = d + 1, m = a.n_sel - 1;
  double* qs = sd;
  double* kt = qs + kSelQ * dp;
  double* sc = kt + kSelJ * dp;
  double* ls = sc + kSelQ * 33;
  int* li = reinterpret_cast<int*>(ls + kSelQ * kSelMost);
  const int nqt = (a.Tq + kSelQ - 1) / kSelQ;
  const int bg = blockIdx.x / nqt, q0 = (blockIdx.x - bg * nqt) * kSelQ;
  const int b = bg / a.G, g = bg - b * a.G;
  const int nq = min(kSelQ, a.Tq - q0), tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int p0 = blk_pos0(a, b) + q0;
  for (int i = tid; i < kSelQ * d; i += 256) {
    const int t = i / d, e = i - t * d;
    double s = 0.0;
    if (t < nq)
      for (int r = 0; r < a.R; ++r) s += double(to_f32(q[row_off(a.sq, b, g * a.R + r, q0 + t) + e]));
    qs[t * dp + e] = s;
  }
  for (int i = tid; i < kSelQ * kSelMost; i += 256) {
    ls[i] = -INFINITY;
    li[i] = -1;
  }
  // blocks before the last query's own
  const int last = p0 + nq - 1;
  const int nj = m > 0 && last >= 0 ? min(last / a.bs, nkc) : 0;
  for (int j0 = 0; j0 < nj; j0 += kSelJ) {
    __syncthreads();
    for (int i = tid; i < kSelJ * d; i += 256) {
      const int j = i / d, e = i - j * d;
      kt[j * dp + e] = j0 + j < nj ? double(to_f32(kc[row_off(skc, b, g, j0 + j) + e])) : 0.0;
    }
    __syncthreads();
    {
      const int t = (tid >> 4) * 2, j = tid & 15;
      double s00 = 0, s01 = 0, s10 = 0, s11 = 0;
      for (int e = 0; e < d; ++e) {
        const double a0 = qs[t * dp + e], a1 = qs[(t + 1) * dp + e];
        const double b0 = kt[j * dp + e], b1 = kt[(j + 16) * dp + e];
        s00 = fma(a0, b0, s00); s01 = fma(a0, b1, s01);
        s10 = fma(a1, b0, s10); s11 = fma(a1, b1, s11);
      }
      sc[t * 33 + j] = s00; sc[t * 33 + j + 16] = s01;
      sc[(t + 1) * 33 + j] = s10; sc[(t + 1) * 33 + j + 16] = s11;
    }
    __syncthreads();
    for (int t = wp; t < nq; t += 8) {
      const int p = p0 + t;
      const int cur = p >= 0 ? p / a.bs : 0;
      const double s = sc[t * 33 + lane];
      double* l = ls + t * kSelMost;
      int* x = li + t * kSelMost;
      // NaN compares false: such a block is never listed
      unsigned todo = __ballot_sync(0xffffffffu, j0 + lane < min(cur, nj) && s > l[m - 1]);
      while (todo) {
        const int w = __ffs(todo) - 1;
        todo &= todo - 1;
        const double sw = __shfl_sync(0xffffffffu, s, w);
        if (sw > l[m - 1]) list_insert(l, x, m, sw, j0 + w);
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < nq * a.n_sel; i += 256) {
    const int t = i / a.n_sel, r = i - t * a.n_sel, p = p0 + t;
    const int v = p < 0 ? -1 : (r == 0 ? p / a.bs : li[t * kSelMost + r - 1]);
    idx[((size_t)bg * a.Tq + q0) * a.n_sel + i] = v;
  }
}

// ---------------------------------------------------------------- plan
// Counting sort by block.  Each segment of queries counts its pairs per block;
// one CTA per (b, group) turns the counts into first positions, block by block and
// segment by segment; then each segment places its pairs, one warp walking them in
// order, so the lists come out in query order whatever runs first.
__global__ void __launch_bounds__(256)
k_blk_count(BlkArgs a, BlkPlan p, const int32_t* __restrict__ idx) {
  extern __shared__ int cnt[];
  const int sg = blockIdx.x % p.nseg, bg = blockIdx.x / p.nseg;
  for (int j = threadIdx.x; j < a.nb; j += 256) cnt[j] = 0;
  __syncthreads();
  const int pos0 = blk_pos0(a, bg / a.G);
  const int q0 = sg * p.seg, n = min(p.seg, a.nq - q0) * a.n_sel;
  const int32_t* ip = idx + ((size_t)bg * a.Tq + a.q0 + q0) * a.n_sel;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int j = ip[i];
    if (blk_keys(a, j, pos0 + a.q0 + q0 + i / a.n_sel) > 0) atomicAdd(&cnt[j], 1);
  }
  __syncthreads();
  int* o = p.hist + (size_t)blockIdx.x * a.nb;
  for (int j = threadIdx.x; j < a.nb; j += 256) o[j] = cnt[j];
}

__global__ void __launch_bounds__(1024)
k_blk_offsets(BlkArgs a, BlkPlan p) {
  __shared__ int2 wsum[32];
  const int bg = blockIdx.x, tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  int* hist = p.hist + (size_t)bg * p.nseg * a.nb;
  int* first = p.first + (size_t)bg * (a.nb + 1);
  int* item = p.item + (size_t)bg * (a.nb + 1);
  // inclusive scan of (pairs, items) over the CTA; `total` gets the sums
  auto scan = [&](int2 v, int2* total) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
      if (lane >= o) { v.x += x; v.y += y; }
    }
    __syncthreads();
    if (lane == 31) wsum[wp] = v;
    __syncthreads();
    int2 before = make_int2(0, 0), all = before;
    for (int w = 0; w < 32; ++w) {
      if (w < wp) { before.x += wsum[w].x; before.y += wsum[w].y; }
      all.x += wsum[w].x; all.y += wsum[w].y;
    }
    *total = all;
    return make_int2(v.x + before.x, v.y + before.y);
  };
  int2 carry = make_int2(0, 0);
  for (int j0 = 0; j0 < a.nb; j0 += 1024) {
    const int j = j0 + tid;
    int tot = 0;
    if (j < a.nb)
#pragma unroll 8
      for (int s = 0; s < p.nseg; ++s) tot += hist[(size_t)s * a.nb + j];
    const int its = int(((long long)tot * a.R + p.rows - 1) / p.rows);
    int2 sum;
    const int2 inc = scan(make_int2(tot, its), &sum);
    if (j < a.nb) {
      int at = carry.x + inc.x - tot;
      first[j] = at;
      item[j] = carry.y + inc.y - its;
      for (int s = 0; s < p.nseg; ++s) {
        const int n = hist[(size_t)s * a.nb + j];
        hist[(size_t)s * a.nb + j] = at;
        at += n;
      }
    }
    carry.x += sum.x;
    carry.y += sum.y;
  }
  if (tid == 0) {
    first[a.nb] = carry.x;
    item[a.nb] = carry.y;
  }
}

__global__ void __launch_bounds__(32)
k_blk_place(BlkArgs a, BlkPlan p, const int32_t* __restrict__ idx) {
  extern __shared__ int at[];
  const int sg = blockIdx.x % p.nseg, bg = blockIdx.x / p.nseg, lane = threadIdx.x;
  const int* h = p.hist + (size_t)blockIdx.x * a.nb;
  for (int j = lane; j < a.nb; j += 32) at[j] = h[j];
  __syncwarp();
  const int pos0 = blk_pos0(a, bg / a.G);
  const int q0 = sg * p.seg, n = min(p.seg, a.nq - q0) * a.n_sel;
  const int32_t* ip = idx + ((size_t)bg * a.Tq + a.q0 + q0) * a.n_sel;
  int* out = p.entry + (size_t)bg * a.nq * a.n_sel;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    int j = -1;
    if (i < n) {
      j = ip[i];
      if (blk_keys(a, j, pos0 + a.q0 + q0 + i / a.n_sel) == 0) j = -1;
    }
    const unsigned same = __match_any_sync(0xffffffffu, j);
    const int rank = __popc(same & ((1u << lane) - 1));
    int base = 0;
    if (j >= 0) base = at[j];
    __syncwarp();
    if (j >= 0) {
      out[base + rank] = q0 * a.n_sel + i;
      if (rank == 0) at[j] = base + __popc(same);
    }
    __syncwarp();
  }
}

BlkPlan blk_plan(const sdm_block_dims* d, int nq, int rows, void* base) {
  BlkPlan p;
  memset(&p, 0, sizeof(p));
  const size_t BG = size_t(d->B) * d->G;
  const int nb = (d->Tk + d->block - 1) / d->block;
  // segments of 128 queries, longer ones past 256 segments (the counts are
  // nseg x nb per group)
  p.seg = 128;
  while ((nq + (long long)p.seg - 1) / p.seg > 256) p.seg <<= 1;
  p.nseg = (nq + p.seg - 1) / p.seg;
  p.rows = rows;
  p.most = int((long long)nq * d->n_sel * (d->H / d->G) / rows) + nb;
  char* b = static_cast<char*>(base);
  size_t o = 0;
  auto take = [&](size_t n) {
    int* q = reinterpret_cast<int*>(b + o);
    o = (o + n * 4 + 255) & ~size_t(255);
    return q;
  };
  // room for the most segments that so many queries or fewer can have
  p.hist = take(BG * (nq > 128 * 256 ? 256 : (nq + 127) / 128) * nb);
  p.first = take(BG * (nb + 1));
  p.item = take(BG * (nb + 1));
  p.entry = take(BG * nq * d->n_sel);
  p.bytes = o;
  return p;
}

cudaError_t launch_blk_plan(const BlkArgs& a, const BlkPlan& p, const int32_t* idx, cudaStream_t s) {
  const int smem = a.nb * 4;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_blk_count, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(k_blk_place, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
    return e;
  const unsigned grid = unsigned(a.B * a.G) * unsigned(p.nseg);
  k_blk_count<<<grid, 256, smem, s>>>(a, p, idx);
  k_blk_offsets<<<a.B * a.G, 1024, 0, s>>>(a, p);
  k_blk_place<<<grid, 32, smem, s>>>(a, p, idx);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- host side
int blk_check(const sdm_block_dims* d) {
  if (!d) return SDM_ERR_NULL;
  if (d->B < 1 || d->H < 1 || d->G < 1 || d->H % d->G != 0 || d->Tq < 0 || d->Tk < 0 ||
      d->Tq > d->Tk || d->Tk > (1 << 28) || d->d < 1 || d->block < 1 || d->n_sel < 1 ||
      (d->in_dtype != SDM_DTYPE_F32 && d->in_dtype != SDM_DTYPE_BF16) ||
      !(d->scale == d->scale && d->scale - d->scale == 0.f))
    return SDM_ERR_DIMS;
  if ((long long)d->B * d->H > (1 << 20) || (long long)d->B * d->H * d->Tq >= (1LL << 31) ||
      (long long)d->Tq * d->n_sel * (d->H / d->G) >= (1LL << 31))
    return SDM_ERR_DIMS;
  if ((d->d != 32 && d->d != 64 && d->d != 128) ||
      (d->block != 32 && d->block != 64 && d->block != 128) || d->n_sel > kSelMost ||
      (d->Tk + d->block - 1) / d->block > 49152)
    return SDM_ERR_UNSUPPORTED;
  return SDM_OK;
}

int blk_views_ok(const sdm_block_views* v) {
  if (!v) return SDM_ERR_NULL;
  for (const sdm_strides* p : {&v->q, &v->k, &v->v, &v->o, &v->kc})
    if (!strides_ok(p)) return SDM_ERR_DIMS;
  return SDM_OK;
}

BlkArgs blk_args(const sdm_block_dims* d, const sdm_block_views* v, const int32_t* lengths) {
  BlkArgs a;
  memset(&a, 0, sizeof(a));
  a.B = d->B; a.H = d->H; a.G = d->G; a.R = d->H / d->G;
  a.Tq = d->Tq; a.Tk = d->Tk; a.d = d->d; a.bs = d->block; a.n_sel = d->n_sel;
  a.nb = (d->Tk + d->block - 1) / d->block;
  a.q0 = 0; a.nq = d->Tq;
  a.scale = d->scale;
  a.sq = v->q; a.sk = v->k; a.sv = v->v; a.so = v->o;
  a.lengths = lengths;
  return a;
}

}  // namespace sdm

using namespace sdm;

extern "C" int sdm_block_pool(const void* k, void* kc, int32_t first, const sdm_block_dims* dims,
                              const sdm_block_views* views, void* stream) {
  int rc = blk_check(dims);
  if (rc != SDM_OK) return rc;
  if ((rc = blk_views_ok(views)) != SDM_OK) return rc;
  const int n = dims->Tk / dims->block;
  if (first < 0 || first > n) return SDM_ERR_DIMS;
  if (first == n) return SDM_OK;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  if ((rc = need_ptr(k, es)) != SDM_OK || (rc = need_ptr(kc, es)) != SDM_OK) return rc;
  const BlkArgs a = blk_args(dims, views, nullptr);
  const long long grid = (long long)a.B * a.G * (n - first);
  if (grid >= (1LL << 31)) return SDM_ERR_DIMS;
  const int vec = view_aligned(k, a.sk, int(es), 4 * es);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->in_dtype == SDM_DTYPE_BF16)
    k_blk_pool<__nv_bfloat16><<<unsigned(grid), 128, 0, s>>>(a, views->kc, (const __nv_bfloat16*)k,
                                                             (__nv_bfloat16*)kc, first, n - first, vec);
  else
    k_blk_pool<float><<<unsigned(grid), 128, 0, s>>>(a, views->kc, (const float*)k, (float*)kc,
                                                     first, n - first, vec);
  return cudaGetLastError() == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

template <typename Tin>
static cudaError_t launch_select(const BlkArgs& a, const sdm_strides& skc, const void* q,
                                 const void* kc, int nkc, int32_t* idx, cudaStream_t s) {
  const int smem = int(blk_select_smem(a.d));
  cudaError_t e = cudaFuncSetAttribute(k_blk_select<Tin>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(a.B * a.G) * unsigned((a.Tq + kSelQ - 1) / kSelQ);
  k_blk_select<Tin><<<grid, 256, smem, s>>>(a, skc, (const Tin*)q, (const Tin*)kc, nkc, idx);
  return cudaGetLastError();
}

extern "C" int sdm_block_select(const void* q, const void* kc, int32_t n_means,
                                const int32_t* lengths, int32_t* idx, const sdm_block_dims* dims,
                                const sdm_block_views* views, void* stream) {
  int rc = blk_check(dims);
  if (rc != SDM_OK) return rc;
  if ((rc = blk_views_ok(views)) != SDM_OK) return rc;
  // every block that lies before some query needs its mean
  if (n_means < 0 || (dims->Tk > 0 && n_means < (dims->Tk - 1) / dims->block)) return SDM_ERR_DIMS;
  if (dims->Tq == 0) return SDM_OK;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  if ((rc = need_ptr(q, es)) != SDM_OK || (rc = need_ptr(idx, 4)) != SDM_OK) return rc;
  if (n_means > 0 && (rc = need_ptr(kc, es)) != SDM_OK) return rc;
  if (!aligned_to(lengths, 4)) return SDM_ERR_ALIGN;
  const BlkArgs a = blk_args(dims, views, lengths);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dims->in_dtype == SDM_DTYPE_BF16
          ? launch_select<__nv_bfloat16>(a, views->kc, q, kc, n_means, idx, s)
          : launch_select<float>(a, views->kc, q, kc, n_means, idx, s);
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
