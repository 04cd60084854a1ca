// block_select.cu -- block means, the selection of blocks by them, and the plan
// that turns the queries' lists into the blocks' lists.
//
// Mean of block j: kc_j = (1 / block) sum of its keys, in the keys' type, for
// complete blocks.  Score of block j for a query of group g: the sum over the
// group's heads of q_h . kc_j = (sum_h q_h) . kc_j.  The list of a query at
// position p: its own block c = p / block, then the best n_sel - 1 of the blocks
// before it, higher score first and lower index at a tie, then -1.
#include <limits.h>

#include "block_internal.cuh"

namespace sdm {

// ---------------------------------------------------------------- means
// A CTA per block: a thread sums a share of the rows of one 4-column piece.  The sums
// are double: exact for bf16 keys whose exponents in a column lie within 2^38 of one another
// (8 bits each, 7 more for 128 rows), so there the means (and with them the lists) do not
// depend on how the rows are shared out.  The mean is rounded to float32 and then to the
// keys' type.
template <typename Tin>
__global__ void __launch_bounds__(128)
k_blk_pool(BlkArgs a, sdm_strides skc, const Tin* __restrict__ k, Tin* __restrict__ kc, int first,
           int count, int vec) {
  wait_for_previous();
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
// Scores in double: a rounding difference at a list's boundary would change the list,
// and float sums differ from one order to the next by more than neighbouring
// scores do about once in 10^5 rows.  The products run on the double-precision tensor
// instruction, which has the vector units' rate but takes a 16 x 8 x 16 product from 12
// operands a lane, where a 2 x 2 tile of scalar products waits for shared memory
// (8192 queries, 4 groups of d = 128, up to 128 blocks: 463 us that way, 2 batches).
// A CTA takes 32 queries; its 8 warps score 16 queries x 32 blocks each, then a
// warp per query extracts the best of its list and the 128 new scores, one at a
// time: scores become ordered 64-bit integers, a lane keeps its own in descending
// order, and the winner is the lane with the largest head.
constexpr int kSelQ = 32;    // queries per CTA
constexpr int kSelJ = 128;   // blocks per tile
constexpr int kSelMost = 64;
constexpr int kSelThreads = 256;

__host__ __device__ inline size_t blk_select_smem(int d) {
  // qs [32][d + 2] double, scores [32][129] double, lists [32][64] (64-bit key, int)
  return size_t(8) * (kSelQ * (d + 2) + kSelQ * (kSelJ + 1) + kSelQ * kSelMost) + size_t(4) * kSelQ * kSelMost;
}

// c += a b, 16 x 8 x 16.  With g = lane / 4, q = lane % 4: a[2 i + r] is row g + 8 r and
// b[i] column g of inner index q + 4 i (any inner order, the same for both); c[0], c[1]
// row g, columns 2 q, 2 q + 1, c[2], c[3] row g + 8.
__device__ __forceinline__ void mma_f64(double (&c)[4], const double (&a)[8], const double (&b)[4]) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f64.f64.f64.f64 {%0,%1,%2,%3}, "
               "{%4,%5,%6,%7,%8,%9,%10,%11}, {%12,%13,%14,%15}, {%0,%1,%2,%3};"
               : "+d"(c[0]), "+d"(c[1]), "+d"(c[2]), "+d"(c[3])
               : "d"(a[0]), "d"(a[1]), "d"(a[2]), "d"(a[3]), "d"(a[4]), "d"(a[5]), "d"(a[6]), "d"(a[7]),
                 "d"(b[0]), "d"(b[1]), "d"(b[2]), "d"(b[3]));
}

// Order of scores as integers; 0 for -inf and NaN, which are never listed.
__device__ __forceinline__ unsigned long long score_key(double s) {
  s += 0.0;  // -0 ties with 0
  if (!(s > -INFINITY)) return 0ull;
  const unsigned long long u = __double_as_longlong(s);
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// Best m of the warp's candidates: NS keys a lane, with their blocks.  Writes them to
// lk, li in order (lower block first at ties), the rest of the m places empty.
template <int NS>
__device__ __forceinline__ void extract_best(unsigned long long (&v)[NS], int (&id)[NS], int m,
                                             unsigned long long* lk, int* li) {
  const int lane = threadIdx.x & 31;
  // descending, lower block first at ties (odd-even transposition: NS rounds)
#pragma unroll
  for (int r = 0; r < NS; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < NS; i += 2) {
      const bool sw = v[i] < v[i + 1] || (v[i] == v[i + 1] && id[i] > id[i + 1]);
      const unsigned long long a = sw ? v[i + 1] : v[i], b = sw ? v[i] : v[i + 1];
      const int x = sw ? id[i + 1] : id[i], y = sw ? id[i] : id[i + 1];
      v[i] = a; v[i + 1] = b;
      id[i] = x; id[i + 1] = y;
    }
  int r = 0;
  for (; r < m; ++r) {
    const unsigned hi = unsigned(v[0] >> 32);
    const unsigned top = __reduce_max_sync(0xffffffffu, hi);
    if (top == 0) break;  // keys that are scores have a non-zero upper half
    unsigned win = __ballot_sync(0xffffffffu, hi == top);
    if (win & (win - 1)) {
      const unsigned lo = hi == top ? unsigned(v[0]) : 0u;
      const unsigned tl = __reduce_max_sync(0xffffffffu, lo);
      const int j = hi == top && lo == tl ? id[0] : INT_MAX;
      win = __ballot_sync(0xffffffffu, j == __reduce_min_sync(0xffffffffu, j));
    }
    if (win >> lane & 1) {
      lk[r] = v[0];
      li[r] = id[0];
#pragma unroll
      for (int i = 0; i + 1 < NS; ++i) {
        v[i] = v[i + 1];
        id[i] = id[i + 1];
      }
      v[NS - 1] = 0ull;
    }
  }
  for (int e = r + lane; e < m; e += 32) {
    lk[e] = 0ull;
    li[e] = -1;
  }
  __syncwarp();
}

// ONE: a single query a CTA, its scores on the vector units (a 16-row product would be one row and
// its latency: 64 sequences 7.8 us for 6.6 here, one of 131072 keys 56).
template <typename Tin, bool ONE>
__global__ void __launch_bounds__(kSelThreads)
k_blk_select(BlkArgs a, sdm_strides skc, const Tin* __restrict__ q, const Tin* __restrict__ kc,
             int nkc, int32_t* __restrict__ idx, int vec) {
  wait_for_previous();
  extern __shared__ __align__(16) double sd[];
  const int d = a.d, dp = d + 2, m = a.n_sel - 1;  // pitch: 16-byte reads of 8 rows without conflicts
  double* qs = sd;
  double* sc = qs + kSelQ * dp;
  unsigned long long* lk = reinterpret_cast<unsigned long long*>(sc + kSelQ * (kSelJ + 1));
  int* li = reinterpret_cast<int*>(lk + kSelQ * kSelMost);
  const int nqt = (a.Tq + kSelQ - 1) / kSelQ;
  const int bg = blockIdx.x / nqt, q0 = (blockIdx.x - bg * nqt) * kSelQ;
  const int b = bg / a.G, g = bg - b * a.G;
  const int nq = min(kSelQ, a.Tq - q0), tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int p0 = blk_pos0(a, b) + q0;
  for (int i = tid; i < kSelQ * (d / 4); i += kSelThreads) {
    const int t = i / (d / 4), e = (i - t * (d / 4)) * 4;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (t < nq)
#pragma unroll 4
      for (int r = 0; r < a.R; ++r) {
        const Tin* p = q + row_off(a.sq, b, g * a.R + r, q0 + t) + e;
        float f[4];
        if (vec & 1) {
          Vec<Tin, 4>::load(p, f);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) f[u] = to_f32(p[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] += double(f[u]);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u) qs[t * dp + e + u] = s[u];
  }
  // blocks before the last query's own
  const int last = p0 + nq - 1;
  const int nj = m > 0 && last >= 0 ? min(last / a.bs, nkc) : 0;
  const int qt = (wp & 1) * 16, jt = (wp >> 1) * 32, gr = lane >> 2, qd = lane & 3;
  for (int i = tid; i < kSelQ * kSelMost && nj == 0; i += kSelThreads) li[i] = -1;
  for (int j0 = 0; j0 < nj; j0 += kSelJ) {
    __syncthreads();  // the queries are in place; the last tile's scores have been read
    if constexpr (ONE) {
      const int j = j0 + (tid >> 1), e0 = (tid & 1) * (d / 2);
      double s[2] = {0.0, 0.0};
      if (j < nj) {
        const Tin* kr = kc + row_off(skc, b, g, j) + e0;
#pragma unroll 4
        for (int e = 0; e < d / 2; e += 4) {
          float f[4];
          if (vec & 2) {
            Vec<Tin, 4>::load(kr + e, f);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) f[u] = to_f32(kr[e + u]);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) s[u & 1] = fma(qs[e0 + e + u], double(f[u]), s[u & 1]);
        }
      }
      s[0] += s[1];
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
      if ((tid & 1) == 0) sc[tid >> 1] = s[0];
    } else if (qt < nq && j0 + jt < nj) {
      double acc[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0;
      const Tin* kp[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)  // columns behind the last block repeat it and are not read back
        kp[n] = kc + row_off(skc, b, g, min(j0 + jt + 8 * n + gr, nj - 1)) + 4 * qd;
      float nx[4][4];  // the next 16 columns are on their way while these are multiplied
      auto fetch = [&](int k) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (vec & 2) {
            Vec<Tin, 4>::load(kp[n] + k, nx[n]);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) nx[n][u] = to_f32(kp[n][k + u]);
          }
        }
      };
      fetch(0);
      for (int k = 0; k < d; k += 16) {
        float f[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int u = 0; u < 4; ++u) f[n][u] = nx[n][u];
        if (k + 16 < d) fetch(k + 16);
        double af[8];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const double2* p = reinterpret_cast<const double2*>(qs + (qt + gr + 8 * r) * dp + k + 4 * qd);
          const double2 x = p[0], y = p[1];
          af[r] = x.x; af[2 + r] = x.y; af[4 + r] = y.x; af[6 + r] = y.y;
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const double bf[4] = {double(f[n][0]), double(f[n][1]), double(f[n][2]), double(f[n][3])};
          mma_f64(acc[n], af, bf);
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        double* o = sc + (qt + gr) * (kSelJ + 1) + jt + 8 * n + 2 * qd;
        o[0] = acc[n][0]; o[1] = acc[n][1];
        o[8 * (kSelJ + 1)] = acc[n][2]; o[8 * (kSelJ + 1) + 1] = acc[n][3];
      }
    }
    __syncthreads();
    for (int t = wp; t < nq; t += kSelThreads / 32) {
      const int p = p0 + t;
      const int end = min(p >= 0 ? p / a.bs : 0, nj);  // blocks before the query's own
      unsigned long long* l = lk + t * kSelMost;
      int* x = li + t * kSelMost;
      unsigned long long v[4];
      int id[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        id[c] = j0 + 32 * c + lane;
        v[c] = id[c] < end ? score_key(sc[t * (kSelJ + 1) + 32 * c + lane]) : 0ull;
      }
      if (j0 == 0) {
        extract_best<4>(v, id, m, l, x);
      } else {
        const unsigned long long worst = l[m - 1];  // a new block beats it or stays out
        bool any = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) any |= v[c] > worst;
        if (!__any_sync(0xffffffffu, any)) continue;
        unsigned long long w[6];
        int y[6];
#pragma unroll
        for (int c = 0; c < 4; ++c) { w[c] = v[c]; y[c] = id[c]; }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int e = 32 * c + lane;
          w[4 + c] = e < m ? l[e] : 0ull;
          y[4 + c] = e < m ? x[e] : 0;
        }
        __syncwarp();
        extract_best<6>(w, y, m, l, x);
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < nq * a.n_sel; i += kSelThreads) {
    const int t = i / a.n_sel, r = i - t * a.n_sel, p = p0 + t;
    const int v = p < 0 ? -1 : (r == 0 ? p / a.bs : li[t * kSelMost + r - 1]);
    idx[((size_t)bg * a.Tq + q0) * a.n_sel + i] = v;
  }
}

// ---------------------------------------------------------------- plan
// Counting sort by block.  Each segment of queries counts its pairs per block;
// one CTA per (b, group) turns the counts into first positions, block by block and
// segment by segment; then each segment places its pairs, its warps walking their
// shares in order, so the lists come out in query order whatever runs first.
__global__ void __launch_bounds__(256)
k_blk_count(BlkArgs a, BlkPlan p, const int32_t* __restrict__ idx) {
  wait_for_previous();
  extern __shared__ int cnt[];
  const int sg = blockIdx.x % p.nseg, bg = blockIdx.x / p.nseg;
  for (int j = threadIdx.x; j < a.nb; j += 256) cnt[j] = 0;
  __syncthreads();
  const int pos0 = blk_pos0(a, bg / a.G);
  const int q0 = sg * p.seg, n = min(p.seg, a.nq - q0) * a.n_sel;
  const int32_t* ip = idx + ((size_t)bg * a.Tq + a.q0 + q0) * a.n_sel;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int j = ip[i];
    if (blk_keys(a, j, pos0 + a.q0 + q0 + a.by_sel.div(i)) > 0) atomicAdd(&cnt[j], 1);
  }
  __syncthreads();
  int* o = p.hist + (size_t)blockIdx.x * a.nb;
  for (int j = threadIdx.x; j < a.nb; j += 256) o[j] = cnt[j];
}

__global__ void __launch_bounds__(1024)
k_blk_offsets(BlkArgs a, BlkPlan p) {
  wait_for_previous();
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

// W warps share a segment: each counts its part of the pairs, the counts become
// first positions warp by warp, and each places its part.
__global__ void __launch_bounds__(256)
k_blk_place(BlkArgs a, BlkPlan p, const int32_t* __restrict__ idx, int W) {
  wait_for_previous();
  extern __shared__ int at[];  // [W][nb]
  const int sg = blockIdx.x % p.nseg, bg = blockIdx.x / p.nseg;
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, nt = 32 * W;
  const int* h = p.hist + (size_t)blockIdx.x * a.nb;
  for (int i = threadIdx.x; i < W * a.nb; i += nt) at[i] = 0;
  __syncthreads();
  const int pos0 = blk_pos0(a, bg / a.G);
  const int q0 = sg * p.seg, n = min(p.seg, a.nq - q0) * a.n_sel;
  const int32_t* ip = idx + ((size_t)bg * a.Tq + a.q0 + q0) * a.n_sel;
  int* out = p.entry + (size_t)bg * a.nq * a.n_sel;
  const int each = ((n + W - 1) / W + 31) & ~31;
  const int i1 = min(n, (wp + 1) * each);
  int* mine = at + (size_t)wp * a.nb;
  auto block_of = [&](int i) {
    if (i >= i1) return -1;
    const int j = ip[i];
    return blk_keys(a, j, pos0 + a.q0 + q0 + a.by_sel.div(i)) > 0 ? j : -1;
  };
  if (W > 1) {
    for (int i = wp * each + lane; i < i1; i += 32) {
      const int j = block_of(i);
      if (j >= 0) atomicAdd(&mine[j], 1);
    }
    __syncthreads();
  }
  for (int j = threadIdx.x; j < a.nb; j += nt) {
    int x = h[j];
    for (int w = 0; w < W; ++w) {
      const int c = at[(size_t)w * a.nb + j];
      at[(size_t)w * a.nb + j] = x;
      x += c;
    }
  }
  __syncthreads();
  for (int i0 = wp * each; i0 < i1; i0 += 32) {
    const int i = i0 + lane;
    const int j = block_of(i);
    const unsigned same = __match_any_sync(0xffffffffu, j);
    const int rank = __popc(same & ((1u << lane) - 1));
    int base = 0;
    if (j >= 0) base = mine[j];
    __syncwarp();
    if (j >= 0) {
      out[base + rank] = q0 * a.n_sel + i;
      if (rank == 0) mine[j] = base + __popc(same);
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
  int W = 8;  // warps of a segment, as many as its counts leave room for
  while (W > 1 && (W * smem > 64 * 1024)) W >>= 1;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_blk_count, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(k_blk_place, cudaFuncAttributeMaxDynamicSharedMemorySize, W * smem)) != cudaSuccess)
    return e;
  const unsigned grid = unsigned(a.B * a.G) * unsigned(p.nseg);
  launch_after(k_blk_count, grid, 256, smem, s, a, p, idx);
  launch_after(k_blk_offsets, a.B * a.G, 1024, 0, s, a, p);
  launch_after(k_blk_place, grid, 32 * W, W * smem, s, a, p, idx, W);
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
  a.by_R = fast_div(a.R);
  a.by_sel = fast_div(a.n_sel);
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
    launch_after(k_blk_pool<__nv_bfloat16>, unsigned(grid), 128, 0, s, a, views->kc, (const __nv_bfloat16*)k,
                                                             (__nv_bfloat16*)kc, first, n - first, vec);
  else
    launch_after(k_blk_pool<float>, unsigned(grid), 128, 0, s, a, views->kc, (const float*)k, (float*)kc,
                                                     first, n - first, vec);
  return cudaGetLastError() == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

template <typename Tin>
static cudaError_t launch_select(const BlkArgs& a, const sdm_strides& skc, const void* q,
                                 const void* kc, int nkc, int32_t* idx, cudaStream_t s) {
  const int smem = int(blk_select_smem(a.d)), es = int(sizeof(Tin));
  const unsigned grid = unsigned(a.B * a.G) * unsigned((a.Tq + kSelQ - 1) / kSelQ);
  const int vec = (view_aligned(q, a.sq, es, 4 * es) ? 1 : 0) | (view_aligned(kc, skc, es, 4 * es) ? 2 : 0);
  auto go = [&](auto kernel) -> cudaError_t {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    launch_after(kernel, grid, kSelThreads, smem, s, a, skc, (const Tin*)q, (const Tin*)kc, nkc, idx, vec);
    return cudaGetLastError();
  };
  return a.Tq == 1 ? go(k_blk_select<Tin, true>) : go(k_blk_select<Tin, false>);
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
