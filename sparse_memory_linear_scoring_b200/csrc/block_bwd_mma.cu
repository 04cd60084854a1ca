// block_bwd_mma.cu -- gradients of block-selected attention on the tensor cores (bf16).
//
// As in block_mma.cu a CTA takes one block of keys (64 at most) and up to kGradRows of
// the rows (pair, head of the group) that list it, so that K and V stay in shared
// memory and dK and dV in registers while the rows stream past, 64 at a time:
//     P = exp(scale Q K^T - lse),  dS = P (dO V^T - delta) scale,
//     dV += P^T dO,  dK += dS^T Q,  dQ part = dS K.
// P is rounded to bf16 once for dV (2^-9 of a term, as the result itself: dV is 0.0023 of its
// norm off, where the result's rounding alone makes 0.0017).  dQ and dK take
// dS in two bf16 parts (2^-17): a row of dS sums to zero, so what its keys (for dK: a key's
// queries) have in common drops out, while rounding errors times it do not (0.0026 of dQ's
// norm; the result's own rounding is 0.0017).  Each warp owns 16 rows for P, dS and dQ, and
// 16 keys (or 16 keys and half the columns) for dK and dV, whose operands it takes
// transposed from shared memory.  A row's dQ is a sum over its list: parts are halves
// scaled by their largest element to 2^15 (2^-12 beside the result's 2^-9, down to 2^-29 of
// that element), joined in list order.
// dK and dV of one item are float32 parts, joined in item order: no atomics, equal calls
// give equal bits.
// delta = do.o comes from o as the forward wrote it, in bf16, and what that is off, e, is
// off in dQ by e sum_k P_k k_k: the largest error there would be (0.0022 of the norm).  But
// sum_k dS_k over a row's list is e scale instead of 0, so each part also leaves its sum
// of dS and its sum P_k k_k (8-bit floats scaled by their largest element: a factor of an
// error), and the join takes their product off again.
// Without the parts a row's dQ would need a second walk over its list, which reads K and
// V once more per query and recomputes P and dS, about half of all products.
// 4 x 2048 tokens, 8 heads of 64 on 2, 8 blocks of 64: 157 us here, 23 for the join of dQ.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "block_internal.cuh"
#include "mma_dev.cuh"

namespace sdm {

constexpr int kGradRows = 512;   // rows per item
constexpr int kGradTile = 64;    // rows per tile, 16 a warp
constexpr int kGradThreads = 128;

template <int D, int KT>
struct GradTile {
  static constexpr int ST = D <= 64 ? 2 : 1;   // row tiles in flight; at 128 a second CTA an SM does more
  static constexpr int LD = D + 8, LP = KT + 8;
  static constexpr int KV = KT * LD, RW = kGradTile * LD, PS = kGradTile * LP;
  static constexpr size_t smem = size_t(2) * (2 * KV + ST * 2 * RW + 3 * PS) + 32;
};

template <int D, int KT>
__global__ void __launch_bounds__(kGradThreads)
k_blk_grad(BlkArgs a, BlkBwdWs w, const __nv_bfloat16* __restrict__ q,
           const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
           const float* __restrict__ lse, const __nv_bfloat16* __restrict__ d_o, sdm_strides sdo) {
  wait_for_previous();
  using L = GradTile<D, KT>;
  extern __shared__ __align__(16) unsigned char raw[];
  __nv_bfloat16* Ks = reinterpret_cast<__nv_bfloat16*>(raw);
  __nv_bfloat16* Vs = Ks + L::KV;
  __nv_bfloat16* Rs = Vs + L::KV;                  // [ST][Q, dO][64][LD]
  __nv_bfloat16* Ps = Rs + L::ST * 2 * L::RW;      // [64][LP]
  __nv_bfloat16* Ds = Ps + L::PS;
  __nv_bfloat16* Es = Ds + L::PS;                  // second part of dS
  uint32_t* odd = reinterpret_cast<uint32_t*>(Es + L::PS);  // keys with inf or NaN in K
  uint32_t* rowodd = odd + 4;  // [4]: by warp, its rows with inf or NaN in Q or dO and masked keys
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int g = lane >> 2, qd = lane & 3;
  const int per = a.bs / KT, sub = blockIdx.x % per;
  const int ii = blockIdx.x / per;
  const int bg = ii / w.plan.most, it = ii - bg * w.plan.most;
  const int b = bg / a.G, grp = bg - b * a.G;
  const int* item = w.plan.item + (size_t)bg * (a.nb + 1);
  const int j = blk_of_item(item, a.nb, it);
  if (j < 0) return;
  const int* first = w.plan.first + (size_t)bg * (a.nb + 1);
  const int e0 = first[j], rows = (first[j + 1] - e0) * a.R;
  const int r0 = (it - item[j]) * kGradRows, r1 = min(r0 + kGradRows, rows);
  const int* entry = w.plan.entry + (size_t)bg * a.nq * a.n_sel + e0;
  const int pos0 = blk_pos0(a, b);
  const int k0 = j * a.bs + sub * KT, len = pos0 + a.Tq;  // keys at or past len are not read

  if (tid < 2) odd[tid] = 0;
  for (int i = tid; i < KT * (D / 8); i += kGradThreads) {
    const int kk = i / (D / 8), c = (i % (D / 8)) * 8;
    const bool in = k0 + kk < len;
    const int at = in ? k0 + kk : 0;
    cp_async16(smem_u32(Ks + kk * L::LD + c), k + row_off(a.sk, b, grp, at) + c, in);
    cp_async16(smem_u32(Vs + kk * L::LD + c), v + row_off(a.sv, b, grp, at) + c, in);
  }
  // the warp's own 16 rows of Q and dO; lanes l and l + 16 know row l: the keys it sees,
  // the place of its part of dq, log2 of its softmax sum and its delta
  struct Row { int keys; size_t place; float l2, dl; };
  auto fetch = [&](int base, int st, Row& me) {
    __nv_bfloat16* dq_ = Rs + st * 2 * L::RW + wp * 16 * L::LD;
    const int row = base + 16 * wp + (lane & 15);
    const bool in = row < r1;
    const int en = in ? a.by_R.div(row) : 0, r = in ? row - en * a.R : 0;
    const int e = in ? entry[en] : 0;
    const int h = grp * a.R + r, t = a.q0 + a.by_sel.div(e);
    me.keys = in ? max(0, min(KT, pos0 + t - k0 + 1)) : 0;
    me.place = (((size_t)bg * a.nq * a.n_sel + e) * a.R + r) * per + sub;
    const size_t at = ((size_t)b * a.H + h) * a.Tq + t;
    const float x = in ? lse[at] : -INFINITY;
    me.l2 = x == -INFINITY ? INFINITY : x * kLog2e;
    me.dl = in ? w.delta[at] : 0.f;
    const unsigned long long sq = reinterpret_cast<unsigned long long>(q + row_off(a.sq, b, h, t));
    const unsigned long long so = reinterpret_cast<unsigned long long>(d_o + row_off(sdo, b, h, t));
#pragma unroll
    for (int i = lane; i < 16 * (D / 8); i += 32) {
      const int rr = i / (D / 8), c = (i % (D / 8)) * 8;
      const __nv_bfloat16* pq = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, sq, rr));
      const __nv_bfloat16* po = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, so, rr));
      const bool ok = base + 16 * wp + rr < r1;
      cp_async16(smem_u32(dq_ + rr * L::LD + c), pq + c, ok);
      cp_async16(smem_u32(dq_ + L::RW + rr * L::LD + c), po + c, ok);
    }
  };
  Row me, next = {0, 0, INFINITY, 0.f};
  fetch(r0, 0, me);
  cp_async_commit();
  cp_async_wait<0>();
  __syncthreads();
  for (int i = tid; i < KT * (D / 8); i += kGradThreads) {
    const int kk = i / (D / 8);
    const uint4 u = *reinterpret_cast<const uint4*>(Ks + kk * L::LD + (i % (D / 8)) * 8);
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    bool bad = false;
#pragma unroll
    for (int z = 0; z < 4; ++z)
      bad |= (x[z] & 0x7f80u) == 0x7f80u || (x[z] & 0x7f800000u) == 0x7f800000u;
    if (bad) atomicOr(&odd[kk >> 5], 1u << (kk & 31));
  }
  __syncthreads();
  const bool anyodd = (odd[0] | odd[KT / 32 - 1]) != 0;
  const float c2 = a.scale * kLog2e;
  const uint32_t ak = smem_u32(Ks), av = smem_u32(Vs), ap = smem_u32(Ps), ad = smem_u32(Ds), ae = smem_u32(Es);
  // dK, dV: keys 16 ks.., columns cp DP..
  constexpr int NK = KT / 16, DP = D * NK / 4;
  const int ks = wp % NK, cp = (wp / NK) * DP;
  float gk[DP / 8][4], gv[DP / 8][4];
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) gk[n][i] = gv[n][i] = 0.f;

  for (int base = r0, st = 0; base < r1; base += kGradTile, st ^= L::ST - 1, me = next) {
    if (L::ST == 2 && base + kGradTile < r1) fetch(base + kGradTile, st ^ 1, next);
    cp_async_commit();
    const int ra = base + 16 * wp + g, rb = ra + 8;
    const int na = __shfl_sync(0xffffffffu, me.keys, g), nb = __shfl_sync(0xffffffffu, me.keys, g + 8);
    const float la = __shfl_sync(0xffffffffu, me.l2, g), lb = __shfl_sync(0xffffffffu, me.l2, g + 8);
    const float da = __shfl_sync(0xffffffffu, me.dl, g), db = __shfl_sync(0xffffffffu, me.dl, g + 8);
    const bool masked = __any_sync(0xffffffffu, me.keys < KT);  // rows of the block's own queries, or none
    if (L::ST == 2) cp_async_wait<1>(); else cp_async_wait<0>();
    __syncwarp();
    const __nv_bfloat16* Qs = Rs + st * 2 * L::RW;
    const uint32_t aq = smem_u32(Qs), ao = aq + 2 * L::RW;
    float ea = 0.f, eb = 0.f;  // the rows' sums of dS
    {
      float sc[KT / 8][4], dp[KT / 8][4];
#pragma unroll
      for (int n = 0; n < KT / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = dp[n][i] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D; kk += 16) {
        uint32_t af[4], of[4];
        ldsm4(af, aq + 2 * frag_a(lane, 16 * wp, kk, L::LD));
        ldsm4(of, ao + 2 * frag_a(lane, 16 * wp, kk, L::LD));
#pragma unroll
        for (int n = 0; n < KT / 16; ++n) {
          uint32_t bf[4];
          ldsm4(bf, ak + 2 * frag_b(lane, 16 * n, kk, L::LD));
          mma_bf16(sc[2 * n], af, bf[0], bf[1]);
          mma_bf16(sc[2 * n + 1], af, bf[2], bf[3]);
          ldsm4(bf, av + 2 * frag_b(lane, 16 * n, kk, L::LD));
          mma_bf16(dp[2 * n], of, bf[0], bf[1]);
          mma_bf16(dp[2 * n + 1], of, bf[2], bf[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < KT / 8; ++n) {
        float p[4], s[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = 8 * n + 2 * qd + i;
          p[i] = ex2(fmaf(sc[n][i], c2, -la));
          p[2 + i] = ex2(fmaf(sc[n][2 + i], c2, -lb));
          s[i] = p[i] * ((dp[n][i] - da) * a.scale);
          s[2 + i] = p[2 + i] * ((dp[n][2 + i] - db) * a.scale);
          if (masked && col >= na) p[i] = s[i] = 0.f;
          if (masked && col >= nb) p[2 + i] = s[2 + i] = 0.f;
        }
        const int at = (16 * wp + g) * L::LP + 8 * n + 2 * qd;
        ea += s[0] + s[1];
        eb += s[2] + s[3];
        uint32_t s0[2], s1[2];
        split_bf16<2>(s[0], s[1], s0);
        split_bf16<2>(s[2], s[3], s1);
        *reinterpret_cast<uint32_t*>(Ps + at) = pack_bf16(p[0], p[1]);
        *reinterpret_cast<uint32_t*>(Ps + at + 8 * L::LP) = pack_bf16(p[2], p[3]);
        *reinterpret_cast<uint32_t*>(Ds + at) = s0[0];
        *reinterpret_cast<uint32_t*>(Ds + at + 8 * L::LP) = s1[0];
        *reinterpret_cast<uint32_t*>(Es + at) = s0[1];
        *reinterpret_cast<uint32_t*>(Es + at + 8 * L::LP) = s1[1];
      }
    }
    // A masked weight is 0, but 0 times an infinite or NaN query or gradient is not: such
    // elements are taken out of the rows and added, by hand, to the keys that their row sees.
    uint32_t mine = 0;
    if (masked) {
      __nv_bfloat16* rows_ = Rs + st * 2 * L::RW + wp * 16 * L::LD;
#pragma unroll
      for (int i = lane; i < 16 * (D / 8); i += 32) {
        const int rr = i / (D / 8), c = (i % (D / 8)) * 8;
        OddBf16 z;
        z.add(rows_ + rr * L::LD + c);
        z.add(rows_ + L::RW + rr * L::LD + c);
        if (z.any()) mine |= 1u << rr;
      }
      mine = __reduce_or_sync(0xffffffffu, mine) & __ballot_sync(0xffffffffu, me.keys < KT) & 0xffffu;
      if (mine) {
        for (int i = lane; i < 16 * D; i += 32) {
          const int rr = i / D, at = rr * L::LD + i % D;
          if (!(mine >> rr & 1)) continue;
          if (!(fabsf(__bfloat162float(rows_[at])) < INFINITY)) rows_[at] = __float2bfloat16_rn(0.f);
          if (!(fabsf(__bfloat162float(rows_[L::RW + at])) < INFINITY)) rows_[L::RW + at] = __float2bfloat16_rn(0.f);
        }
      }
    }
    if (lane == 0) rowodd[wp] = mine;
    __syncthreads();  // all rows' Q, dO, P and dS are in place
#pragma unroll
    for (int kk = 0; kk < kGradTile; kk += 16) {
      uint32_t pf[4], sf[4], tf[4];
      ldsm4t(pf, ap + 2 * frag_at(lane, 16 * ks, kk, L::LP));
      ldsm4t(sf, ad + 2 * frag_at(lane, 16 * ks, kk, L::LP));
      ldsm4t(tf, ae + 2 * frag_at(lane, 16 * ks, kk, L::LP));
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t bf[4];
        ldsm4t(bf, ao + 2 * frag_bt(lane, cp + 16 * n, kk, L::LD));
        mma_bf16(gv[2 * n], pf, bf[0], bf[1]);
        mma_bf16(gv[2 * n + 1], pf, bf[2], bf[3]);
        ldsm4t(bf, aq + 2 * frag_bt(lane, cp + 16 * n, kk, L::LD));
        mma_bf16(gk[2 * n], tf, bf[0], bf[1]);
        mma_bf16(gk[2 * n + 1], tf, bf[2], bf[3]);
        mma_bf16(gk[2 * n], sf, bf[0], bf[1]);
        mma_bf16(gk[2 * n + 1], sf, bf[2], bf[3]);
      }
    }
    if (rowodd[0] | rowodd[1] | rowodd[2] | rowodd[3]) {
#pragma unroll 1
      for (int rr = 0; rr < kGradTile; ++rr) {
        if (!(rowodd[rr >> 4] >> (rr & 15) & 1)) continue;
        const int row = base + rr, en = a.by_R.div(row), h = grp * a.R + row - en * a.R;
        const int t = a.q0 + a.by_sel.div(entry[en]), n = pos0 + t - k0 + 1;  // keys it sees
        const __nv_bfloat16 *qr = q + row_off(a.sq, b, h, t) + cp, *dr = d_o + row_off(sdo, b, h, t) + cp;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = 16 * ks + g + 8 * u, at = rr * L::LP + key;
          if (key >= n) continue;
          const float pk = __bfloat162float(Ps[at]), sk = __bfloat162float(Ds[at]) + __bfloat162float(Es[at]);
#pragma unroll
          for (int m = 0; m < DP / 8; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = __bfloat162float(qr[8 * m + 2 * qd + i]), y = __bfloat162float(dr[8 * m + 2 * qd + i]);
              if (!(fabsf(x) < INFINITY)) gk[m][2 * u + i] = fmaf(sk, x, gk[m][2 * u + i]);
              if (!(fabsf(y) < INFINITY)) gv[m][2 * u + i] = fmaf(pk, y, gv[m][2 * u + i]);
            }
        }
      }
    }
    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    // acc += (A, and A2 beside it) K; `clean` leaves out what is not finite in K, since 0
    // times that is not 0
    auto times_keys = [&](auto clean, auto two, uint32_t a1, uint32_t a2) {
#pragma unroll
      for (int kk = 0; kk < KT / 16; ++kk) {
        uint32_t df[4], ef[4];
        ldsm4(df, a1 + 2 * frag_a(lane, 16 * wp, 16 * kk, L::LP));
        if constexpr (decltype(two)::value) ldsm4(ef, a2 + 2 * frag_a(lane, 16 * wp, 16 * kk, L::LP));
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t bf[4];
          ldsm4t(bf, ak + 2 * frag_bt(lane, 16 * n, 16 * kk, L::LD));
          if constexpr (decltype(clean)::value) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if ((bf[i] & 0x7f80u) == 0x7f80u) bf[i] &= 0xffff0000u;
              if ((bf[i] & 0x7f800000u) == 0x7f800000u) bf[i] &= 0x0000ffffu;
            }
          }
          if constexpr (decltype(two)::value) {
            mma_bf16(acc[2 * n], ef, bf[0], bf[1]);
            mma_bf16(acc[2 * n + 1], ef, bf[2], bf[3]);
          }
          mma_bf16(acc[2 * n], df, bf[0], bf[1]);
          mma_bf16(acc[2 * n + 1], df, bf[2], bf[3]);
        }
      }
    };
    if (D == 128 || anyodd) times_keys(std::true_type(), std::true_type(), ad, ae);  // one copy: registers
    else times_keys(std::false_type(), std::true_type(), ad, ae);
    if (anyodd) {  // the rest of the keys that are not finite, for the rows that see them
      for (int key = 0; key < KT; ++key) {
        if (!(odd[key >> 5] >> (key & 31) & 1)) continue;
        const int pa = (16 * wp + g) * L::LP + key, pb = pa + 8 * L::LP;
        const float xa = __bfloat162float(Ds[pa]), xb = __bfloat162float(Ds[pb]);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(Ks + key * L::LD + 8 * n + 2 * qd);
          const bool lo = (u & 0x7f80u) == 0x7f80u, hi = (u & 0x7f800000u) == 0x7f800000u;
          if (lo && key < na) acc[n][0] = fmaf(xa, bf16_lo(u), acc[n][0]);
          if (hi && key < na) acc[n][1] = fmaf(xa, bf16_hi(u), acc[n][1]);
          if (lo && key < nb) acc[n][2] = fmaf(xb, bf16_lo(u), acc[n][2]);
          if (hi && key < nb) acc[n][3] = fmaf(xb, bf16_hi(u), acc[n][3]);
        }
      }
    }
    float xa = 0.f, xb = 0.f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      xa = fmaxf(xa, fmaxf(fabsf(acc[n][0]), fabsf(acc[n][1])));
      xb = fmaxf(xb, fmaxf(fabsf(acc[n][2]), fabsf(acc[n][3])));
    }
    if (__any_sync(0xffffffffu, xa == INFINITY || xb == INFINITY)) {  // the largest finite one
      xa = xb = 0.f;
#pragma unroll
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
    xa = fmaxf(xa, 7.7037198e-34f);  // 2^-110: the factor stays finite
    xb = fmaxf(xb, 7.7037198e-34f);
    const float va = 32768.f / xa, vb = 32768.f / xb;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ea += __shfl_xor_sync(0xffffffffu, ea, o);
      eb += __shfl_xor_sync(0xffffffffu, eb, o);
    }
    __syncthreads();  // everyone has read this tile's rows, P and dS
    __half* stage = reinterpret_cast<__half*>(Rs + st * 2 * L::RW + wp * 16 * L::LD);
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      *reinterpret_cast<__half2*>(stage + g * L::LD + 8 * n + 2 * qd) =
          __floats2half2_rn(acc[n][0] * va, acc[n][1] * va);
      *reinterpret_cast<__half2*>(stage + (g + 8) * L::LD + 8 * n + 2 * qd) =
          __floats2half2_rn(acc[n][2] * vb, acc[n][3] * vb);
    }
    __syncwarp();
    __half* part = static_cast<__half*>(w.part);
#pragma unroll
    for (int i = lane; i < 16 * (D / 8); i += 32) {
      const int r = i / (D / 8), c = (i % (D / 8)) * 8;
      const size_t u = __shfl_sync(0xffffffffu, me.place, r);
      if (base + 16 * wp + r < r1)
        *reinterpret_cast<uint4*>(part + u * D + c) = *reinterpret_cast<const uint4*>(stage + r * L::LD + c);
    }
    // sum P_k k_k, as above, over what is finite (a row that sees more has no finite dQ)
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    if (D == 128 || anyodd) times_keys(std::true_type(), std::false_type(), ap, ap);
    else times_keys(std::false_type(), std::false_type(), ap, ap);
    float ka = 0.f, kb = 0.f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      ka = fmaxf(ka, fmaxf(fabsf(acc[n][0]), fabsf(acc[n][1])));
      kb = fmaxf(kb, fmaxf(fabsf(acc[n][2]), fabsf(acc[n][3])));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
      kb = fmaxf(kb, __shfl_xor_sync(0xffffffffu, kb, o));
    }
    ka = fminf(fmaxf(ka, 7.7037198e-34f), 1.7e38f);
    kb = fminf(fmaxf(kb, 7.7037198e-34f), 1.7e38f);
    const float fa = 256.f / ka, fb = 256.f / kb;  // 8-bit floats reach 448
    const size_t oa = __shfl_sync(0xffffffffu, me.place, g), ob = __shfl_sync(0xffffffffu, me.place, g + 8);
    if (qd == 0) {
      if (ra < r1) w.mul[oa] = make_float4(xa * (1.f / 32768.f), ka * (1.f / 256.f), ea, 0.f);
      if (rb < r1) w.mul[ob] = make_float4(xb * (1.f / 32768.f), kb * (1.f / 256.f), eb, 0.f);
    }
    __syncwarp();  // the warp has sent its parts of dQ
    unsigned short* bytes = reinterpret_cast<unsigned short*>(stage);  // rows of LD halves again
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      bytes[g * L::LD + 4 * n + qd] =
          __nv_cvt_float2_to_fp8x2(make_float2(acc[n][0] * fa, acc[n][1] * fa), __NV_SATFINITE, __NV_E4M3);
      bytes[(g + 8) * L::LD + 4 * n + qd] =
          __nv_cvt_float2_to_fp8x2(make_float2(acc[n][2] * fb, acc[n][3] * fb), __NV_SATFINITE, __NV_E4M3);
    }
    __syncwarp();
    unsigned char* kpart = static_cast<unsigned char*>(w.kpart);
#pragma unroll
    for (int i = lane; i < 16 * (D / 16); i += 32) {
      const int r = i / (D / 16), c = (i % (D / 16)) * 16;
      const size_t u = __shfl_sync(0xffffffffu, me.place, r);
      if (base + 16 * wp + r < r1)
        *reinterpret_cast<uint4*>(kpart + u * D + c) = *reinterpret_cast<const uint4*>(bytes + r * L::LD + c / 2);
    }
    __syncwarp();  // before the next fetch into these rows
    if (L::ST == 1 && base + kGradTile < r1) fetch(base + kGradTile, 0, next);
  }
  cp_async_wait<0>();
  float* kp = w.kv + (size_t)blockIdx.x * 2 * KT * D;
#pragma unroll
  for (int n = 0; n < DP / 8; ++n) {
    float* o = kp + (16 * ks + g) * D + cp + 8 * n + 2 * qd;
    *reinterpret_cast<float2*>(o) = make_float2(gk[n][0], gk[n][1]);
    *reinterpret_cast<float2*>(o + 8 * D) = make_float2(gk[n][2], gk[n][3]);
    *reinterpret_cast<float2*>(o + KT * D) = make_float2(gv[n][0], gv[n][1]);
    *reinterpret_cast<float2*>(o + (KT + 8) * D) = make_float2(gv[n][2], gv[n][3]);
  }
}

// delta = do.o, D / 8 lanes a row.
template <int D>
__global__ void __launch_bounds__(256)
k_blk_delta(BlkArgs a, const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ d_o,
            sdm_strides sdo, float* __restrict__ delta) {
  wait_for_previous();
  constexpr int LN = D / 8;
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) / LN;
  const int c = (threadIdx.x % LN) * 8;
  const bool in = i < (long long)a.B * a.H * a.Tq;
  float s = 0.f;
  if (in) {
    const int t = int(i % a.Tq), bh = int(i / a.Tq), b = bh / a.H, h = bh - b * a.H;
    float x[8], y[8];
    Vec<__nv_bfloat16, 8>::load(o + row_off(a.so, b, h, t) + c, x);
    Vec<__nv_bfloat16, 8>::load(d_o + row_off(sdo, b, h, t) + c, y);
#pragma unroll
    for (int z = 0; z < 8; ++z) s = fmaf(x[z], y[z], s);
  }
#pragma unroll
  for (int w = LN / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
  if (in && c == 0) delta[i] = s;
}

// A row of dq from its parts, in list order; pairs without keys have none.  As in the
// forward's join a lane looks up every LN-th part; two rows' loads are in flight (four
// take registers that more warps use better).
template <int D>
__global__ void __launch_bounds__(128, 10)
k_blk_dq(BlkArgs a, BlkBwdWs w, const int32_t* __restrict__ idx, __nv_bfloat16* __restrict__ dq,
         sdm_strides sdq, int kt) {
  wait_for_previous();
  constexpr int LN = D / 8;
  const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) / LN;
  const int ln = threadIdx.x % LN, c = ln * 8;
  const bool in = i < (long long)a.B * a.G * a.nq * a.R;
  const long long i0 = in ? i : 0, bt = i0 / a.R;
  const int r = int(i0 - bt * a.R), per = a.bs / kt;  // per: 1 or 2 parts a pair
  const int bg = int(bt / a.nq), t = int(bt - (long long)bg * a.nq), b = bg / a.G, h = (bg - b * a.G) * a.R + r;
  const int32_t* list = idx + ((size_t)bg * a.Tq + a.q0 + t) * a.n_sel;
  const int p = blk_pos0(a, b) + a.q0 + t, parts = a.n_sel * per;
  // part y: slot y / per, keys (y % per) kt .. of its block
  auto place = [&](int y) { return per == 2 ? (y >> 1) * 2 * a.R + (y & 1) : y * a.R; };
  const size_t first = ((size_t)bt * a.n_sel * a.R + r) * per;
  const __half* part = static_cast<const __half*>(w.part) + first * D + c;
  const unsigned char* kpart = static_cast<const unsigned char*>(w.kpart) + first * D + c;
  const float4* mul = w.mul + first;
  auto there = [&](int y) {
    return y < parts && blk_keys(a, list[per == 2 ? y >> 1 : y], p) > (per == 2 && (y & 1) ? kt : 0);
  };
  float e = 0.f;
  for (int y = ln; y < parts; y += LN)
    if (there(y)) e += mul[place(y)].z;
#pragma unroll
  for (int z = 1; z < LN; z <<= 1) e += __shfl_xor_sync(0xffffffffu, e, z);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int y0 = 0; y0 < parts; y0 += LN) {
    float f = -1.f, fk = 0.f;  // no part
    if (there(y0 + ln)) {
      const float4 u = mul[place(y0 + ln)];
      f = u.x;
      fk = -e * u.y;
    }
#pragma unroll
    for (int z0 = 0; z0 < LN; z0 += 2) {
      uint4 x[2];
      uint2 kx[2];
      float fz[2], kz[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        fz[z] = __shfl_sync(0xffffffffu, f, z0 + z, LN);
        kz[z] = __shfl_sync(0xffffffffu, fk, z0 + z, LN);
        x[z] = make_uint4(0u, 0u, 0u, 0u);
        kx[z] = make_uint2(0u, 0u);
        if (fz[z] != -1.f) {
          const size_t at = (size_t)place(y0 + z0 + z) * D;
          x[z] = __ldcs(reinterpret_cast<const uint4*>(part + at));
          if (kz[z] != 0.f) kx[z] = __ldcs(reinterpret_cast<const uint2*>(kpart + at));
        }
      }
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const __half2* hx = reinterpret_cast<const __half2*>(&x[z]);
        const unsigned short* k8 = reinterpret_cast<const unsigned short*>(&kx[z]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 v = __half22float2(hx[u]);
          const __half2_raw kr = __nv_cvt_fp8x2_to_halfraw2(k8[u], __NV_E4M3);
          const float2 kv = __half22float2(__half2(kr));
          acc[2 * u] = fmaf(kz[z], kv.x, fmaf(fz[z], v.x, acc[2 * u]));
          acc[2 * u + 1] = fmaf(kz[z], kv.y, fmaf(fz[z], v.y, acc[2 * u + 1]));
        }
      }
    }
  }
  if (in) Vec<__nv_bfloat16, 8>::store(dq + row_off(sdq, b, h, a.q0 + t) + c, acc);
}

// dk, dv of 4 columns of a key: the items of its block in order.  With several passes
// over the queries, sum [2][BG][Tk][D] carries the total from pass to pass.
template <typename Tin, int D>
__global__ void __launch_bounds__(256)
k_blk_dkv(BlkArgs a, BlkBwdWs w, Tin* __restrict__ dk, Tin* __restrict__ dv,
          sdm_strides sdk, sdm_strides sdv, int kt, int begin, int end, int vec) {
  wait_for_previous();
  constexpr int LN = D / 4;
  long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int c = int(i % LN) * 4;
  i /= LN;
  if (i >= (long long)a.B * a.G * a.Tk) return;
  const int key = int(i % a.Tk), bg = int(i / a.Tk), which = blockIdx.y;
  const int j = key / a.bs, in = key - j * a.bs, sub = in / kt, per = a.bs / kt;
  const int* item = w.plan.item + (size_t)bg * (a.nb + 1);
  const int i0 = item[j], i1 = item[j + 1];
  float* sum = w.sum + (((size_t)which * a.B * a.G + bg) * a.Tk + key) * D + c;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!begin) s = *reinterpret_cast<const float4*>(sum);
  const float* p = w.kv + ((((size_t)bg * w.plan.most + i0) * per + sub) * 2 + which) * kt * D +
                   (size_t)(in - sub * kt) * D + c;
  const size_t step = (size_t)per * 2 * kt * D;
#pragma unroll 4
  for (int u = i0; u < i1; ++u, p += step) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  if (!end) {
    *reinterpret_cast<float4*>(sum) = s;
  } else {
    const float f[4] = {s.x, s.y, s.z, s.w};
    const int b = bg / a.G, g = bg - b * a.G;
    Tin* o = which ? dv + row_off(sdv, b, g, key) : dk + row_off(sdk, b, g, key);
    if (vec) {
      Vec<Tin, 4>::store(o + c, f);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c + e] = from_f32<Tin>(f[e]);
    }
  }
}

cudaError_t launch_blk_dkv(const BlkArgs& a, const BlkBwdWs& w, bool bf16, void* dk, void* dv,
                           const sdm_strides& sdk, const sdm_strides& sdv, int kt, bool begin, bool end,
                           cudaStream_t s) {
  const long long n = (long long)a.B * a.G * a.Tk * (a.d / 4);
  const dim3 grid(unsigned((n + 255) / 256), 2);
  const int es = bf16 ? 2 : 4;
  const int vec = view_aligned(dk, sdk, es, 4 * es) && view_aligned(dv, sdv, es, 4 * es);
  auto go = [&](auto dd) {
    constexpr int D = decltype(dd)::value;
    if (bf16)
      launch_after(k_blk_dkv<__nv_bfloat16, D>, grid, 256, 0, s, a, w, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, sdk, sdv,
                                                       kt, begin, end, vec);
    else
      launch_after(k_blk_dkv<float, D>, grid, 256, 0, s, a, w, (float*)dk, (float*)dv, sdk, sdv, kt, begin, end, vec);
    return cudaGetLastError();
  };
  return a.d == 32 ? go(std::integral_constant<int, 32>())
                   : a.d == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
}

// ---------------------------------------------------------------- host side
static int grad_keys(const sdm_block_dims* d) { return d->block < 64 ? 32 : 64; }

// Fewer queries than half a tile leave it mostly empty, and the query-by-query kernels
// have none of the plan's launches.
bool blk_bwd_tiles_pay(const sdm_block_dims* d) { return d->in_dtype == SDM_DTYPE_BF16 && d->Tq >= 32; }

// Queries per pass: as many as keep the parts of dq within 2 GiB (at least 128).
int blk_bwd_chunk(const sdm_block_dims* d) {
  const long long per = (long long)d->B * d->H * d->n_sel * (d->block / grad_keys(d)) * (d->d * 3 + 16);
  long long n = (2LL << 30) / per;
  if (n < 128) n = 128;
  if (n > d->Tq) n = d->Tq;
  if (n < 1) n = 1;
  const long long passes = (d->Tq + n - 1) / n;  // even passes
  return passes > 0 ? int((d->Tq + passes - 1) / passes) : 1;
}

BlkBwdWs blk_bwd_ws(const sdm_block_dims* d, int nq, void* base) {
  BlkBwdWs w;
  memset(&w, 0, sizeof(w));
  const size_t BG = size_t(d->B) * d->G, per = size_t(d->block / grad_keys(d));
  const size_t rows = size_t(d->B) * d->H * nq * d->n_sel * per;
  char* b = static_cast<char*>(base);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* p = b + o;
    o = (o + bytes + 255) & ~size_t(255);
    return p;
  };
  // what does not depend on the pass comes first
  w.delta = reinterpret_cast<float*>(take(size_t(d->B) * d->H * d->Tq * 4));
  w.sum = reinterpret_cast<float*>(take(blk_bwd_chunk(d) < d->Tq ? 2 * BG * d->Tk * d->d * 4 : 0));
  w.plan = blk_plan(d, nq, kGradRows, b + o);
  take(w.plan.bytes);
  w.mul = reinterpret_cast<float4*>(take(rows * 16));
  w.part = take(rows * d->d * 2);
  w.kpart = take(rows * d->d);
  w.kv = reinterpret_cast<float*>(take(BG * w.plan.most * d->block * 2 * d->d * 4));
  w.bytes = o;
  return w;
}

template <int D>
static cudaError_t launch_grad(const sdm_block_dims* d, BlkArgs a, const void* q, const void* k,
                               const void* v, const int32_t* idx, const void* o, const float* lse,
                               const void* d_o, void* dq, void* dk, void* dv,
                               const sdm_block_views* gv, void* workspace, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const int chunk = blk_bwd_chunk(d), kt = grad_keys(d);
  cudaError_t e;
  for (int q0 = 0; q0 < d->Tq; q0 += chunk) {
    a.q0 = q0;
    a.nq = d->Tq - q0 < chunk ? d->Tq - q0 : chunk;
    const BlkBwdWs w = blk_bwd_ws(d, a.nq, workspace);
    if (q0 == 0) {
      const long long n = (long long)a.B * a.H * a.Tq * (D / 8);
      launch_after(k_blk_delta<D>, unsigned((n + 255) / 256), 256, 0, s, a, (const bf*)o, (const bf*)d_o, gv->o, w.delta);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if ((e = launch_blk_plan(a, w.plan, idx, s)) != cudaSuccess) return e;
    const long long grid = (long long)a.B * a.G * w.plan.most * (a.bs / kt);
    if (grid >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    auto go = [&](auto key) -> cudaError_t {
      constexpr int KT = decltype(key)::value;
      const int sm = int(GradTile<D, KT>::smem);
      cudaError_t r = cudaFuncSetAttribute(k_blk_grad<D, KT>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
      if (r != cudaSuccess) return r;
      launch_after(k_blk_grad<D, KT>, unsigned(grid), kGradThreads, sm, s, a, w, (const bf*)q, (const bf*)k,
                                                                 (const bf*)v, lse, (const bf*)d_o, gv->o);
      return cudaGetLastError();
    };
    e = kt == 32 ? go(std::integral_constant<int, 32>()) : go(std::integral_constant<int, 64>());
    if (e != cudaSuccess) return e;
    const long long nr = (long long)a.B * a.H * a.nq * (D / 8);
    launch_after(k_blk_dq<D>, unsigned((nr + 127) / 128), 128, 0, s, a, w, idx, (bf*)dq, gv->q, kt);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_blk_dkv(a, w, true, dk, dv, gv->k, gv->v, kt, q0 == 0, q0 + a.nq == d->Tq, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_blk_bwd_mma(const sdm_block_dims* d, BlkArgs a, const void* q, const void* k,
                               const void* v, const int32_t* idx, const void* o, const float* lse,
                               const void* d_o, void* dq, void* dk, void* dv,
                               const sdm_block_views* gv, void* workspace, cudaStream_t s) {
  if (a.d == 32) return launch_grad<32>(d, a, q, k, v, idx, o, lse, d_o, dq, dk, dv, gv, workspace, s);
  if (a.d == 64) return launch_grad<64>(d, a, q, k, v, idx, o, lse, d_o, dq, dk, dv, gv, workspace, s);
  return launch_grad<128>(d, a, q, k, v, idx, o, lse, d_o, dq, dk, dv, gv, workspace, s);
}

}  // namespace sdm
