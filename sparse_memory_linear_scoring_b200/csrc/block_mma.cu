// block_mma.cu -- block-selected attention on the tensor cores (bf16), forward.
//
// Each query picks its own blocks, so a tile of neighbouring queries shares few of
// them, and a query alone has too few rows (the heads of its group) for a tensor-core
// tile.  The other way round every tile is full: a CTA takes one block of keys and
// the list of (query, slot) pairs that name it (the plan of block_select.cu), and its
// rows are those pairs times the heads of the group.  Keys and values are read once
// per item of kItemRows rows; a row has one block of scores, so its softmax needs no
// running maximum.  What this costs is a partial result per (query, slot, head) --
// d halves, a log-sum-exp and a scale, written here and read once by the join:
//     o = sum_s exp(lse_s - lse) o_s,   lse = log sum_s exp(lse_s).
// Partials are halves scaled by the row's largest element: 11 significant bits, an
// error of 2^-12 beside the 2^-9 of the weights' and the result's bf16; float32
// partials would double the bytes that bound this path.
#include <cuda_fp16.h>

#include "block_internal.cuh"
#include "mma_dev.cuh"

namespace sdm {

constexpr int kItemRows = 512;
constexpr int kTileWarps = 4;                  // 16 rows each
constexpr int kTileRows = 16 * kTileWarps;

template <int D, int BS>
struct BlkTile {
  static constexpr int LD = D + 8;
  static constexpr int KV = BS * LD;            // one of K, V
  static constexpr int QW = 16 * LD;            // a warp's rows
  static constexpr size_t smem = size_t(2) * (2 * KV + 2 * kTileWarps * QW) + 16;
};

template <int D, int BS>
__global__ void __launch_bounds__(kTileWarps * 32)
k_blk_tile(BlkArgs a, BlkFwdWs w, const __nv_bfloat16* __restrict__ q,
           const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v) {
  using L = BlkTile<D, BS>;
  extern __shared__ __align__(16) unsigned char raw[];
  __nv_bfloat16* Ks = reinterpret_cast<__nv_bfloat16*>(raw);
  __nv_bfloat16* Vs = Ks + L::KV;
  __nv_bfloat16* Qs = Vs + L::KV;
  uint32_t* odd = reinterpret_cast<uint32_t*>(Qs + 2 * kTileWarps * L::QW);  // keys with inf or NaN values
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int g = lane >> 2, qd = lane & 3;
  const int bg = blockIdx.x / w.plan.most, it = blockIdx.x - bg * w.plan.most;
  const int b = bg / a.G, grp = bg - b * a.G;
  const int* item = w.plan.item + (size_t)bg * (a.nb + 1);
  const int j = blk_of_item(item, a.nb, it);
  if (j < 0) return;
  const int* first = w.plan.first + (size_t)bg * (a.nb + 1);
  const int e0 = first[j], rows = (first[j + 1] - e0) * a.R;
  const int r0 = (it - item[j]) * kItemRows, r1 = min(r0 + kItemRows, rows);
  const int* entry = w.plan.entry + (size_t)bg * a.nq * a.n_sel + e0;
  const int pos0 = blk_pos0(a, b);
  const int k0 = j * BS, len = pos0 + a.Tq;  // keys at or past len are not read

  if (tid < 4) odd[tid] = 0;
  for (int i = tid; i < BS * (D / 8); i += kTileWarps * 32) {
    const int kk = i / (D / 8), c = (i % (D / 8)) * 8;
    const bool in = k0 + kk < len;
    const int at = in ? k0 + kk : 0;
    cp_async16(smem_u32(Ks + kk * L::LD + c), k + row_off(a.sk, b, grp, at) + c, in);
    cp_async16(smem_u32(Vs + kk * L::LD + c), v + row_off(a.sv, b, grp, at) + c, in);
  }
  // rows of a tile: 16 per warp; lanes l and l + 16 know row l's keys (those it sees) and
  // the place of its partial result
  auto fetch = [&](int base, int st, int& keys, size_t& place) {
    __nv_bfloat16* dst = Qs + (st * kTileWarps + wp) * L::QW;
    const int row = base + 16 * wp + (lane & 15);
    const bool in = row < r1;
    const int en = in ? a.by_R.div(row) : 0, r = in ? row - en * a.R : 0;
    const int e = in ? entry[en] : 0;
    const int t = a.q0 + a.by_sel.div(e);
    keys = in ? min(BS, pos0 + t - k0 + 1) : 0;
    place = ((size_t)bg * a.nq * a.n_sel + e) * a.R + r;
    const unsigned long long src =
        reinterpret_cast<unsigned long long>(q + row_off(a.sq, b, grp * a.R + r, t));
    // consecutive lanes take consecutive pieces of a row
#pragma unroll
    for (int i = lane; i < 16 * (D / 8); i += 32) {
      const int rr = i / (D / 8), c = (i % (D / 8)) * 8;
      const __nv_bfloat16* p =
          reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, src, rr));
      cp_async16(smem_u32(dst + rr * L::LD + c), p + c, base + 16 * wp + rr < r1);
    }
  };
  int keys, nkeys = 0;
  size_t place, nplace = 0;
  fetch(r0, 0, keys, place);
  cp_async_commit();
  cp_async_wait<0>();
  __syncthreads();
  // A masked weight is 0, but 0 times an infinite or NaN value is not: such values are
  // taken out of the tile and added, by hand, to the rows that see their key.
  for (int i = tid; i < BS * (D / 8); i += kTileWarps * 32) {
    const int kk = i / (D / 8);
    const uint4 u = *reinterpret_cast<const uint4*>(Vs + kk * L::LD + (i % (D / 8)) * 8);
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    bool bad = false;
#pragma unroll
    for (int z = 0; z < 4; ++z)
      bad |= (x[z] & 0x7f80u) == 0x7f80u || (x[z] & 0x7f800000u) == 0x7f800000u;
    if (bad) atomicOr(&odd[kk >> 5], 1u << (kk & 31));
  }
  __syncthreads();
  uint32_t anyodd = 0;
#pragma unroll
  for (int z = 0; z < BS / 32; ++z) anyodd |= odd[z];
  __half* part = static_cast<__half*>(w.part);
  const float c2 = fabsf(a.scale) * kLog2e;
  const uint32_t ak = smem_u32(Ks), av = smem_u32(Vs);

  for (int base = r0, st = 0; base < r1; base += kTileRows, st ^= 1, keys = nkeys, place = nplace) {
    if (base + kTileRows < r1) fetch(base + kTileRows, st ^ 1, nkeys, nplace);
    cp_async_commit();
    __nv_bfloat16* mine = Qs + (st * kTileWarps + wp) * L::QW;
    const uint32_t aq = smem_u32(mine);
    const int ra = base + 16 * wp + g, rb = ra + 8;
    const int na = __shfl_sync(0xffffffffu, keys, g), nb = __shfl_sync(0xffffffffu, keys, g + 8);
    cp_async_wait<1>();
    __syncwarp();
    float sc[BS / 8][4];
#pragma unroll
    for (int n = 0; n < BS / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D; kk += 16) {
      uint32_t af[4];
      ldsm4(af, aq + 2 * frag_a(lane, 0, kk, L::LD));
#pragma unroll
      for (int n = 0; n < BS / 16; ++n) {
        uint32_t bf[4];
        ldsm4(bf, ak + 2 * frag_b(lane, 16 * n, kk, L::LD));
        mma_bf16(sc[2 * n], af, bf[0], bf[1]);
        mma_bf16(sc[2 * n + 1], af, bf[2], bf[3]);
      }
    }
    if (a.scale < 0.f) {
#pragma unroll
      for (int n = 0; n < BS / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = -sc[n][i];
    }
    if (__any_sync(0xffffffffu, keys < BS)) {  // rows of the block's own queries, or none
#pragma unroll
      for (int n = 0; n < BS / 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = 8 * n + 2 * qd + i;
          if (col >= na) sc[n][i] = -INFINITY;
          if (col >= nb) sc[n][2 + i] = -INFINITY;
        }
    }
    float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
    for (int n = 0; n < BS / 8; ++n) {
      ma = fmaxf(ma, fmaxf(sc[n][0], sc[n][1]));
      mb = fmaxf(mb, fmaxf(sc[n][2], sc[n][3]));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    }
    const float ba = ma == -INFINITY ? 0.f : ma * c2, bb = mb == -INFINITY ? 0.f : mb * c2;
    float la = 0.f, lb = 0.f;
    uint32_t pf[BS / 16][4];
#pragma unroll
    for (int n = 0; n < BS / 8; ++n) {
      const float x0 = ex2(fmaf(sc[n][0], c2, -ba)), x1 = ex2(fmaf(sc[n][1], c2, -ba));
      const float x2 = ex2(fmaf(sc[n][2], c2, -bb)), x3 = ex2(fmaf(sc[n][3], c2, -bb));
      la += x0 + x1;
      lb += x2 + x3;
      pf[n >> 1][(n & 1) * 2] = pack_bf16(x0, x1);
      pf[n >> 1][(n & 1) * 2 + 1] = pack_bf16(x2, x3);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      la += __shfl_xor_sync(0xffffffffu, la, o);
      lb += __shfl_xor_sync(0xffffffffu, lb, o);
    }
    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    if (anyodd == 0) {
#pragma unroll
      for (int kk = 0; kk < BS / 16; ++kk)
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t vf[4];
          ldsm4t(vf, av + 2 * frag_bt(lane, 16 * n, 16 * kk, L::LD));
          mma_bf16(acc[2 * n], pf[kk], vf[0], vf[1]);
          mma_bf16(acc[2 * n + 1], pf[kk], vf[2], vf[3]);
        }
    } else {
#pragma unroll
      for (int kk = 0; kk < BS / 16; ++kk) {
        // the weights of this lane's rows at 16 keys, one key at a time
        for (int y = 0; y < 16; ++y) {
          const int src = (lane & ~3) | ((y >> 1) & 3);
          const uint32_t wa = __shfl_sync(0xffffffffu, y < 8 ? pf[kk][0] : pf[kk][2], src);
          const uint32_t wb = __shfl_sync(0xffffffffu, y < 8 ? pf[kk][1] : pf[kk][3], src);
          const float xa = (y & 1) ? bf16_hi(wa) : bf16_lo(wa), xb = (y & 1) ? bf16_hi(wb) : bf16_lo(wb);
          const int key = 16 * kk + y;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const uint32_t u = *reinterpret_cast<const uint32_t*>(Vs + key * L::LD + 8 * n + 2 * qd);
            if (key < na) {
              acc[n][0] = fmaf(xa, bf16_lo(u), acc[n][0]);
              acc[n][1] = fmaf(xa, bf16_hi(u), acc[n][1]);
            }
            if (key < nb) {
              acc[n][2] = fmaf(xb, bf16_lo(u), acc[n][2]);
              acc[n][3] = fmaf(xb, bf16_hi(u), acc[n][3]);
            }
          }
        }
      }
    }
    // acc / la, scaled by the row's largest finite element, to halves
    float xa = 0.f, xb = 0.f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      xa = fmaxf(xa, fmaxf(fabsf(acc[n][0]), fabsf(acc[n][1])));
      xb = fmaxf(xb, fmaxf(fabsf(acc[n][2]), fabsf(acc[n][3])));
    }
    if (__any_sync(0xffffffffu, xa == INFINITY || xb == INFINITY)) {
      xa = xb = 0.f;
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (fabsf(acc[n][i]) < INFINITY) xa = fmaxf(xa, fabsf(acc[n][i]));
          if (fabsf(acc[n][2 + i]) < INFINITY) xb = fmaxf(xb, fabsf(acc[n][2 + i]));
        }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, o));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, o));
    }
    xa = fmaxf(xa, 2.3509887e-38f);  // 2^-125: its reciprocal is still finite
    xb = fmaxf(xb, 2.3509887e-38f);
    const float va = 1.f / xa, vb = 1.f / xb;
    __half* stage = reinterpret_cast<__half*>(mine);
    __syncwarp();  // the warp has read its queries
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      *reinterpret_cast<__half2*>(stage + g * L::LD + 8 * n + 2 * qd) =
          __floats2half2_rn(acc[n][0] * va, acc[n][1] * va);
      *reinterpret_cast<__half2*>(stage + (g + 8) * L::LD + 8 * n + 2 * qd) =
          __floats2half2_rn(acc[n][2] * vb, acc[n][3] * vb);
    }
    const size_t oa = __shfl_sync(0xffffffffu, place, g), ob = __shfl_sync(0xffffffffu, place, g + 8);
    if (qd == 0) {
      if (ra < r1) w.ml[oa] = la == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(ba + log2f(la), xa / la);
      if (rb < r1) w.ml[ob] = lb == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(bb + log2f(lb), xb / lb);
    }
    __syncwarp();
#pragma unroll
    for (int i = lane; i < 16 * (D / 8); i += 32) {
      const int r = i / (D / 8), c = (i % (D / 8)) * 8;
      const size_t o = __shfl_sync(0xffffffffu, place, r);
      if (base + 16 * wp + r < r1)
        *reinterpret_cast<uint4*>(part + o * D + c) = *reinterpret_cast<const uint4*>(stage + r * L::LD + c);
    }
    __syncwarp();  // before the next fetch into these rows
  }
  cp_async_wait<0>();
}

// A row of o from its partials: D / 8 lanes a row.  A lane first takes every LN-th slot
// of the list for the maximum and the sum, then each of LN slots at a time for its
// weight, which the others get by shuffles, with 4 partial rows' loads in flight.  The
// (query, slot) pairs without keys have no partial and are skipped by the same test
// that left them out.
template <int D>
__global__ void __launch_bounds__(256)
k_blk_join(BlkArgs a, BlkFwdWs w, const int32_t* __restrict__ idx, __nv_bfloat16* __restrict__ o,
           float* __restrict__ lse) {
  constexpr int LN = D / 8;
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) / LN;
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
        if (fz[z] != -1.f) x[z] = *reinterpret_cast<const uint4*>(part + (size_t)(s0 + z0 + z) * a.R * D);
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
  w.plan = blk_plan(d, nq, kItemRows, base);
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
    auto go = [&](auto bs) -> cudaError_t {
      constexpr int BS = decltype(bs)::value;
      const int sm = int(BlkTile<D, BS>::smem);
      cudaError_t r = cudaFuncSetAttribute(k_blk_tile<D, BS>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
      if (r != cudaSuccess) return r;
      k_blk_tile<D, BS><<<unsigned(grid), kTileWarps * 32, sm, s>>>(a, w, (const bf*)q, (const bf*)k, (const bf*)v);
      return cudaGetLastError();
    };
    e = a.bs == 32 ? go(std::integral_constant<int, 32>())
                   : a.bs == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
    if (e != cudaSuccess) return e;
    const long long n = (long long)a.B * a.H * a.nq * (D / 8);
    k_blk_join<D><<<unsigned((n + 255) / 256), 256, 0, s>>>(a, w, idx, (bf*)o, lse);
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
