// ssm_bwd_mma.cu -- gradients of the selective scan on the tensor cores (bf16 inputs,
// widths 64 and 128), in chunks of 64 steps.  ssm_bwd.cu has the formulas and passes.
//
// Two kernels over all (head, chunk) pairs: each chunk's own contribution to the states
// and to their gradients, and, after the carries, the gradients.  What ends in float32
// (states, ddt, dA, dD, dS0) keeps float32 accuracy: products of bf16 inputs are exact,
// and a float32 operand beside a bf16 one is split into three bf16 parts (rest below
// 2^-24).  W G, whose product ends in dx, is rounded once, and dx takes the first of dSin's
// parts alone: one rounding in each term (dx is 0.0020 of its norm off, where the result's
// rounding alone makes 0.0017).  W dt R is two parts: in
// a short call it makes most of dB and dC, and one part's error (0.0021 of their norm) would
// add to the results' own (0.0017).  Per chunk and head 14 products of 64 x 64 x 64 at
// widths of 64, eight of them for the splits; the tiles of x, dy, B, C and the two float32
// states that a CTA reads (72 KB) bound it.  4 x 2048 steps, 8 heads of 64 x 64: 18 us the
// contributions, 52 the gradients (CUDA cores: 98 and 258).
#include <type_traits>

#include "mma_dev.cuh"
#include "ssm_internal.cuh"

namespace sdm {

constexpr int kGQ = kSsmQT;  // 64

// Rows of a [B][H][T][W] view into a tile of pitch ld; rows at or past n are zero.
template <int W, int NT>
__device__ __forceinline__ void tile_rows(uint32_t dst, int ld, const __nv_bfloat16* src,
                                          const sdm_strides& s, int b, int h, int t0, int n) {
#pragma unroll
  for (int i = threadIdx.x; i < kGQ * (W / 8); i += NT) {
    const int t = i / (W / 8), e = (i % (W / 8)) * 8;
    const bool in = t < n;
    cp_async16(dst + 2 * (t * ld + e), src + row_off(s, b, h, in ? t0 + t : 0) + e, in);
  }
}

// Adds the thread's own pieces of such a tile (they have arrived) to a check for inf and NaN.
template <int W, int NT>
__device__ __forceinline__ void check_rows(OddBf16& z, const __nv_bfloat16* tile, int ld) {
#pragma unroll
  for (int i = threadIdx.x; i < kGQ * (W / 8); i += NT) z.add(tile + i / (W / 8) * ld + (i % (W / 8)) * 8);
}

// dec: hi, lo, dt, exp(g_t), exp(g_Q - g_t), each [64]; by one warp.
__device__ __forceinline__ void chunk_weights(float* dec, const float* dt, const sdm_strides& s, int b,
                                              int h, int t0, int n, float A) {
  float *hi = dec, *lo = dec + kGQ, *dts = dec + 2 * kGQ, *eg = dec + 3 * kGQ, *ej = dec + 4 * kGQ;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 2 * lane + i;
    dts[t] = t < n ? dt[row_off(s, b, h, t0 + t)] : 0.f;
  }
  __syncwarp();
  chunk_decay<2>(dts, A, hi, lo);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 2 * lane + i;
    eg[t] = ex2(hi[t] + lo[t]);
    ej[t] = decay_between(hi[kGQ - 1], lo[kGQ - 1], hi[t], lo[t]);
  }
}

template <int P, int N>
struct LocalTile {
  static constexpr int LX = P + 8, LN = N + 8, NT = 2 * P;
  static constexpr size_t smem = size_t(2) * 2 * kGQ * (LX + LN) + 4 * 5 * kGQ;
};

// fS = sum_j e_j dt_j x_j B_j^T, gS = sum_t exp(g_t) dy_t C_t^T; warp w owns rows 16 w...
template <int P, int N>
__global__ void __launch_bounds__(2 * P)
k_ssm_local_tile(SsmArgs a, const __nv_bfloat16* __restrict__ x, const float* __restrict__ dt,
                 const float* __restrict__ A, const __nv_bfloat16* __restrict__ Bm,
                 const __nv_bfloat16* __restrict__ Cm, const __nv_bfloat16* __restrict__ dy,
                 float* __restrict__ fS, float* __restrict__ gS, float* __restrict__ lg) {
  wait_for_previous();
  using L = LocalTile<P, N>;
  extern __shared__ __align__(16) unsigned char raw[];
  __nv_bfloat16* t_ = reinterpret_cast<__nv_bfloat16*>(raw);
  const uint32_t ax = smem_u32(t_), ay = ax + 2 * kGQ * L::LX, ab = ay + 2 * kGQ * L::LX,
                 ac = ab + 2 * kGQ * L::LN;
  float* dec = reinterpret_cast<float*>(t_ + 2 * kGQ * (L::LX + L::LN));
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int c = blockIdx.x % a.nch, bh = blockIdx.x / a.nch;
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  const int t0 = c * kGQ, n = min(kGQ, a.T - t0);
  tile_rows<P, L::NT>(ax, L::LX, x, a.sx, b, h, t0, n);
  tile_rows<N, L::NT>(ab, L::LN, Bm, a.sB, b, gr, t0, n);
  cp_async_commit();
  tile_rows<P, L::NT>(ay, L::LX, dy, a.sy, b, h, t0, n);
  tile_rows<N, L::NT>(ac, L::LN, Cm, a.sC, b, gr, t0, n);
  cp_async_commit();
  if (wp == 0) chunk_weights(dec, dt, a.sdt, b, h, t0, n, A[h]);
  const float *hi = dec, *lo = dec + kGQ, *dts = dec + 2 * kGQ, *eg = dec + 3 * kGQ, *ej = dec + 4 * kGQ;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (side == 0) cp_async_wait<1>(); else cp_async_wait<0>();
    __syncthreads();
    const uint32_t ar = side == 0 ? ax : ay, am = side == 0 ? ab : ac;
    uint32_t xw[4][3][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t xf[4];
      ldsm4t(xf, ar + 2 * frag_at(lane, 16 * wp, 16 * k, L::LX));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * k + (i >> 1) * 8 + 2 * q;
        float2 w;
        if (side == 0) {
          const float2 u = *reinterpret_cast<const float2*>(ej + t), v = *reinterpret_cast<const float2*>(dts + t);
          w = make_float2(u.x * v.x, u.y * v.y);
        } else {
          w = *reinterpret_cast<const float2*>(eg + t);
        }
        uint32_t u[3];
        split_bf16<3>(bf16_lo(xf[i]) * w.x, bf16_hi(xf[i]) * w.y, u);
        xw[k][0][i] = u[0]; xw[k][1][i] = u[1]; xw[k][2][i] = u[2];
      }
    }
    float* out = (side == 0 ? fS : gS) + size_t(blockIdx.x) * P * N + (16 * wp + g) * N + 2 * q;
    float all[4] = {0.f, 0.f, 0.f, 0.f};  // not finite if some result is not
#pragma unroll
    for (int m = 0; m < N / 16; ++m) {
      float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t bf[4];
        ldsm4t(bf, am + 2 * frag_bt(lane, 16 * m, 16 * k, L::LN));
#pragma unroll
        for (int i = 2; i >= 0; --i) {  // small parts first
          mma_bf16(d0, xw[k][i], bf[0], bf[1]);
          mma_bf16(d1, xw[k][i], bf[2], bf[3]);
        }
      }
      *reinterpret_cast<float2*>(out + 16 * m) = make_float2(d0[0], d0[1]);
      *reinterpret_cast<float2*>(out + 16 * m + 8 * N) = make_float2(d0[2], d0[3]);
      *reinterpret_cast<float2*>(out + 16 * m + 8) = make_float2(d1[0], d1[1]);
      *reinterpret_cast<float2*>(out + 16 * m + 8 * N + 8) = make_float2(d1[2], d1[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) all[i] += d0[i] + d1[i];
    }
    if (!(fabsf(all[0] + all[1]) + fabsf(all[2] + all[3]) < INFINITY)) {
      // inf or NaN, which parts do not add up to: step by step
      const __nv_bfloat16 *rt = t_ + side * kGQ * L::LX, *mt = t_ + 2 * kGQ * L::LX + side * kGQ * L::LN;
      const float Ah = A[h];
#pragma unroll 1
      for (int m = 0; m < N / 8; ++m) {
        float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int t = side == 0 ? i : n - 1 - i;
          const float at = expf(dts[t] * Ah), f = side == 0 ? dts[t] : 1.f;
          const float ua = f * __bfloat162float(rt[t * L::LX + 16 * wp + g]);
          const float ub = f * __bfloat162float(rt[t * L::LX + 16 * wp + g + 8]);
          const uint32_t w = *reinterpret_cast<const uint32_t*>(mt + t * L::LN + 8 * m + 2 * q);
          const float c[4] = {ua * bf16_lo(w), ua * bf16_hi(w), ub * bf16_lo(w), ub * bf16_hi(w)};
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] = side == 0 ? fmaf(at, r[e], c[e]) : at * (r[e] + c[e]);
        }
        *reinterpret_cast<float2*>(out + 8 * m) = make_float2(r[0], r[1]);
        *reinterpret_cast<float2*>(out + 8 * m + 8 * N) = make_float2(r[2], r[3]);
      }
    }
  }
  if (threadIdx.x == 0) lg[blockIdx.x] = hi[kGQ - 1] + lo[kGQ - 1];
}

constexpr int kGradWarps = 8;

template <int P, int N>
struct SsmGradTile {
  static constexpr int LX = P + 8, LN = N + 8, LM = kGQ + 8;
  static constexpr int SP = P * LN;  // one part of a state
  // x, dy, B, C; three parts of one state at a time; the weights W G, W dt R in two parts
  static constexpr int elems = 2 * kGQ * (LX + LN) + 3 * SP + 3 * kGQ * LM;
  // decays [5][64], row sums of E and dots with C, B [2][3][64], column sums [4][64],
  // boundary [8], R_tt [64]
  static constexpr int floats = 5 * kGQ + 6 * kGQ + 4 * kGQ + kGQ + 2 * 8;
  static constexpr size_t smem = size_t(2) * elems + 4 * floats;
};

// A state's three bf16 parts from float32, [P][LN] each.
template <int P, int N>
__device__ __forceinline__ void split_state(__nv_bfloat16* S, const float* __restrict__ src) {
  using L = SsmGradTile<P, N>;
#pragma unroll 4
  for (int i = threadIdx.x; i < P * N / 4; i += kGradWarps * 32) {
    const int p = i / (N / 4), e = (i % (N / 4)) * 4;
    const float4 v = *reinterpret_cast<const float4*>(src + 4 * (size_t)i);
    uint32_t u[3], w[3];
    split_bf16<3>(v.x, v.y, u);
    split_bf16<3>(v.z, v.w, w);
#pragma unroll
    for (int z = 0; z < 3; ++z)
      *reinterpret_cast<uint2*>(S + z * L::SP + p * L::LN + e) = make_uint2(u[z], w[z]);
  }
}

// Warp (rt, ch): rows 16 rt .. of every output, the ch-th half of its columns.
template <int P, int N>
__global__ void __launch_bounds__(kGradWarps * 32)
k_ssm_grad(SsmBwdArgs ba, const __nv_bfloat16* __restrict__ x, const float* __restrict__ dt,
           const float* __restrict__ A, const __nv_bfloat16* __restrict__ Bm,
           const __nv_bfloat16* __restrict__ Cm, const float* __restrict__ D,
           const __nv_bfloat16* __restrict__ dy, SsmBwdWs w, __nv_bfloat16* __restrict__ dx,
           float* __restrict__ ddt, __nv_bfloat16* __restrict__ dB, __nv_bfloat16* __restrict__ dC) {
  wait_for_previous();
  using L = SsmGradTile<P, N>;
  constexpr int NT = kGradWarps * 32;
  extern __shared__ __align__(16) unsigned char raw[];
  const SsmArgs& a = ba.a;
  __nv_bfloat16* xs = reinterpret_cast<__nv_bfloat16*>(raw);
  __nv_bfloat16* ys = xs + kGQ * L::LX;
  __nv_bfloat16* Bs = ys + kGQ * L::LX;
  __nv_bfloat16* Cs = Bs + kGQ * L::LN;
  __nv_bfloat16* Ss = Cs + kGQ * L::LN;
  __nv_bfloat16* MG = Ss + 3 * L::SP;
  __nv_bfloat16* MR = MG + kGQ * L::LM;
  __nv_bfloat16* M2 = MR + kGQ * L::LM;
  float* dec = reinterpret_cast<float*>(M2 + kGQ * L::LM);
  const float *hi = dec, *lo = dec + kGQ, *dts = dec + 2 * kGQ, *eg = dec + 3 * kGQ, *ej = dec + 4 * kGQ;
  float* rowE = dec + 5 * kGQ;   // [2][64]
  float* dotC = rowE + 2 * kGQ;  // [2][64] C_t.I1_t
  float* dotB = dotC + 2 * kGQ;  // [2][64] B_j.I2_j
  float* colE = dotB + 2 * kGQ;  // [4][64]
  float* dg = colE + 4 * kGQ;    // [64] R_tt
  double* red = reinterpret_cast<double*>(dg + kGQ);  // [8]
  const uint32_t ax = smem_u32(xs), ay = smem_u32(ys), ab = smem_u32(Bs), ac = smem_u32(Cs),
                 as = smem_u32(Ss), ag = smem_u32(MG), ar = smem_u32(MR), a2 = smem_u32(M2);
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int rt = wp & 3, ch = wp >> 2;
  const int c = blockIdx.x % a.nch, bh = blockIdx.x / a.nch;
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  const int t0 = c * kGQ, n = min(kGQ, a.T - t0);
  const size_t PN = size_t(P) * N;
  const float* S0 = w.fS + size_t(blockIdx.x) * PN;
  const float* dSin = w.gS + size_t(blockIdx.x) * PN;
  const float* Send = c + 1 < a.nch ? S0 + PN : w.ST + size_t(bh) * PN;
  tile_rows<P, NT>(ax, L::LX, x, a.sx, b, h, t0, n);
  tile_rows<P, NT>(ay, L::LX, dy, a.sy, b, h, t0, n);
  tile_rows<N, NT>(ab, L::LN, Bm, a.sB, b, gr, t0, n);
  tile_rows<N, NT>(ac, L::LN, Cm, a.sC, b, gr, t0, n);
  cp_async_commit();
  if (wp == 0) chunk_weights(dec, dt, a.sdt, b, h, t0, n, A[h]);
  split_state<P, N>(Ss, S0);
  cp_async_wait<0>();
  OddBf16 z;
  check_rows<P, NT>(z, ys, L::LX);
  check_rows<N, NT>(z, Bs, L::LN);
  check_rows<N, NT>(z, Cs, L::LN);
  const bool careful = __syncthreads_or(z.any());  // inf or NaN in the operands of masked weights

  const int ta = 16 * rt + g, tb = ta + 8;  // the lane's rows
  {  // weights and E = W G R for rows t, columns j in [32 ch, 32 ch + 32)
    float gg[4][4], rr[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) gg[m][i] = rr[m][i] = 0.f;
#pragma unroll
    for (int k = 0; k < N; k += 16) {
      uint32_t af[4];
      ldsm4(af, ac + 2 * frag_a(lane, 16 * rt, k, L::LN));
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (2 * ch + m <= rt) {
          uint32_t bf[4];
          ldsm4(bf, ab + 2 * frag_b(lane, 32 * ch + 16 * m, k, L::LN));
          mma_bf16(gg[2 * m], af, bf[0], bf[1]);
          mma_bf16(gg[2 * m + 1], af, bf[2], bf[3]);
        }
    }
#pragma unroll
    for (int k = 0; k < P; k += 16) {
      uint32_t af[4];
      ldsm4(af, ay + 2 * frag_a(lane, 16 * rt, k, L::LX));
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (2 * ch + m <= rt) {
          uint32_t bf[4];
          ldsm4(bf, ax + 2 * frag_b(lane, 32 * ch + 16 * m, k, L::LX));
          mma_bf16(rr[2 * m], af, bf[0], bf[1]);
          mma_bf16(rr[2 * m + 1], af, bf[2], bf[3]);
        }
    }
    float ea = 0.f, eb = 0.f;
    const float ha = hi[ta], la = lo[ta], hb = hi[tb], lb = lo[tb];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int j = 32 * ch + 8 * m + 2 * q;
      float mg[4], mr[4], ce[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float hj = hi[j + i], lj = lo[j + i], dj = dts[j + i];
        // chosen, not multiplied by 0: a later step may hold a NaN
        const bool ia = j + i <= ta, ib = j + i <= tb;
        const float wa = decay_between(ha, la, hj, lj), wb = decay_between(hb, lb, hj, lj);
        mg[i] = ia ? wa * gg[m][i] : 0.f; mg[2 + i] = ib ? wb * gg[m][2 + i] : 0.f;
        mr[i] = ia ? wa * dj * rr[m][i] : 0.f; mr[2 + i] = ib ? wb * dj * rr[m][2 + i] : 0.f;
        const float xa = ia ? mg[i] * rr[m][i] : 0.f, xb = ib ? mg[2 + i] * rr[m][2 + i] : 0.f;
        ea = fmaf(xa, dj, ea);
        eb = fmaf(xb, dj, eb);
        ce[i] = xa + xb;
        if (j + i == ta) dg[ta] = rr[m][i];
        if (j + i == tb) dg[tb] = rr[m][2 + i];
      }
      *reinterpret_cast<uint32_t*>(MG + ta * L::LM + j) = pack_bf16(mg[0], mg[1]);
      *reinterpret_cast<uint32_t*>(MG + tb * L::LM + j) = pack_bf16(mg[2], mg[3]);
      uint32_t ra[2], rb[2];
      split_bf16<2>(mr[0], mr[1], ra);
      split_bf16<2>(mr[2], mr[3], rb);
      *reinterpret_cast<uint32_t*>(MR + ta * L::LM + j) = ra[0];
      *reinterpret_cast<uint32_t*>(MR + tb * L::LM + j) = rb[0];
      *reinterpret_cast<uint32_t*>(M2 + ta * L::LM + j) = ra[1];
      *reinterpret_cast<uint32_t*>(M2 + tb * L::LM + j) = rb[1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) ce[i] += __shfl_xor_sync(0xffffffffu, ce[i], o);
        if (g == 0) colE[rt * kGQ + j + i] = ce[i];
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ea += __shfl_xor_sync(0xffffffffu, ea, o);
      eb += __shfl_xor_sync(0xffffffffu, eb, o);
    }
    if (q == 0) {
      rowE[ch * kGQ + ta] = ea;
      rowE[ch * kGQ + tb] = eb;
    }
  }
  __syncthreads();  // MG, MR

  constexpr int NH = N / 2, PH = P / 2;
  // rows of x or dy times the state's three parts: columns n0 .. n0 + NH
  const int n0 = ch * NH, p0 = ch * PH;
  auto times_state = [&](float (&acc)[NH / 8][4], uint32_t rows) {
#pragma unroll
    for (int m = 0; m < NH / 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
#pragma unroll
    for (int k = 0; k < P; k += 16) {
      uint32_t af[4];
      ldsm4(af, rows + 2 * frag_a(lane, 16 * rt, k, L::LX));
#pragma unroll
      for (int m = 0; m < NH / 16; ++m)
#pragma unroll
        for (int z = 2; z >= 0; --z) {
          uint32_t bf[4];
          ldsm4t(bf, as + 2 * (z * L::SP + frag_bt(lane, n0 + 16 * m, k, L::LN)));
          mma_bf16(acc[2 * m], af, bf[0], bf[1]);
          mma_bf16(acc[2 * m + 1], af, bf[2], bf[3]);
        }
    }
  };
  // dots of acc's rows with the tile's, then acc's rows times fa, fb
  auto dot_scale = [&](float (&acc)[NH / 8][4], const __nv_bfloat16* tile, float* dst, float fa, float fb) {
    float sa = 0.f, sb = 0.f;
#pragma unroll
    for (int m = 0; m < NH / 8; ++m) {
      const uint32_t ua = *reinterpret_cast<const uint32_t*>(tile + ta * L::LN + n0 + 8 * m + 2 * q);
      const uint32_t ub = *reinterpret_cast<const uint32_t*>(tile + tb * L::LN + n0 + 8 * m + 2 * q);
      sa = fmaf(acc[m][0], bf16_lo(ua), fmaf(acc[m][1], bf16_hi(ua), sa));
      sb = fmaf(acc[m][2], bf16_lo(ub), fmaf(acc[m][3], bf16_hi(ub), sb));
      acc[m][0] *= fa; acc[m][1] *= fa;
      acc[m][2] *= fb; acc[m][3] *= fb;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sa += __shfl_xor_sync(0xffffffffu, sa, o);
      sb += __shfl_xor_sync(0xffffffffu, sb, o);
    }
    if (q == 0) {
      dst[ch * kGQ + ta] = sa;
      dst[ch * kGQ + tb] = sb;
    }
  };
  // a group's gradient: the result itself, or one head's part of it
  auto put = [&](float (&acc)[NH / 8][4], __nv_bfloat16* out, const sdm_strides& so, float* part) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = r ? tb : ta;
      if (t >= n) continue;
      if (a.hg == 1) {
        __nv_bfloat16* o = out + row_off(so, b, gr, t0 + t) + n0 + 2 * q;
#pragma unroll
        for (int m = 0; m < NH / 8; ++m)
          *reinterpret_cast<uint32_t*>(o + 8 * m) = pack_bf16(acc[m][2 * r], acc[m][2 * r + 1]);
      } else {
        float* o = part + (size_t(bh) * a.T + t0 + t) * N + n0 + 2 * q;
#pragma unroll
        for (int m = 0; m < NH / 8; ++m)
          *reinterpret_cast<float2*>(o + 8 * m) = make_float2(acc[m][2 * r], acc[m][2 * r + 1]);
      }
    }
  };
  // The diagonal tile of a product with masked weights M (m2: their second part), without
  // the masked ones: rows t of M, or with T its columns, times the rows of `tile`.
  auto diagonal = [&](auto& acc, auto transposed, const __nv_bfloat16* m1, const __nv_bfloat16* m2,
                      const __nv_bfloat16* tile, int ld) {
    constexpr bool T = decltype(transposed)::value;
    constexpr int W = int(sizeof(acc) / sizeof(acc[0]));
#pragma unroll 1
    for (int z = 0; z < 16; ++z) {
      const int r = 16 * rt + z;
      const int oa = T ? r * L::LM + ta : ta * L::LM + r, ob = T ? r * L::LM + tb : tb * L::LM + r;
      const float ma = __bfloat162float(m1[oa]) + (m2 ? __bfloat162float(m2[oa]) : 0.f);
      const float mb = __bfloat162float(m1[ob]) + (m2 ? __bfloat162float(m2[ob]) : 0.f);
      const bool ia = T ? z >= g : z <= g, ib = T ? z >= g + 8 : z <= g + 8;
#pragma unroll
      for (int m = 0; m < W; ++m) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(tile + r * ld + 8 * m + 2 * q);
        if (ia) {
          acc[m][0] = fmaf(ma, bf16_lo(u), acc[m][0]);
          acc[m][1] = fmaf(ma, bf16_hi(u), acc[m][1]);
        }
        if (ib) {
          acc[m][2] = fmaf(mb, bf16_lo(u), acc[m][2]);
          acc[m][3] = fmaf(mb, bf16_hi(u), acc[m][3]);
        }
      }
    }
  };
  {  // dC_t = exp(g_t) I1_t + sum_j MR_tj B_j
    float acc[NH / 8][4];
    times_state(acc, ay);
    dot_scale(acc, Cs, dotC, eg[ta], eg[tb]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < rt || (k == rt && !careful)) {
        uint32_t af[4], cf[4];
        ldsm4(af, ar + 2 * frag_a(lane, 16 * rt, 16 * k, L::LM));
        ldsm4(cf, a2 + 2 * frag_a(lane, 16 * rt, 16 * k, L::LM));
#pragma unroll
        for (int m = 0; m < NH / 16; ++m) {
          uint32_t bf[4];
          ldsm4t(bf, ab + 2 * frag_bt(lane, n0 + 16 * m, 16 * k, L::LN));
          mma_bf16(acc[2 * m], cf, bf[0], bf[1]);
          mma_bf16(acc[2 * m + 1], cf, bf[2], bf[3]);
          mma_bf16(acc[2 * m], af, bf[0], bf[1]);
          mma_bf16(acc[2 * m + 1], af, bf[2], bf[3]);
        }
      }
    if (careful) diagonal(acc, std::false_type(), MR, M2, Bs + n0, L::LN);
    put(acc, dC, ba.sdC, w.pC);
  }
  __syncthreads();  // everyone is done with S_0
  split_state<P, N>(Ss, dSin);
  {  // <dSin, S_Q>, in double: it enters every q of the chunk, and dA sums them over all steps
    double s = 0.0;
#pragma unroll 4
    for (int i = tid; i < int(PN) / 4; i += NT) {
      const float4 u = *reinterpret_cast<const float4*>(dSin + 4 * i), v = *reinterpret_cast<const float4*>(Send + 4 * i);
      s = fma(double(u.x), double(v.x), fma(double(u.y), double(v.y), s));
      s = fma(double(u.z), double(v.z), fma(double(u.w), double(v.w), s));
    }
    s = warp_sum(s);
    if (lane == 0) red[wp] = s;
  }
  __syncthreads();
  {  // dB_j = dt_j e_j I2_j + sum_t MR_tj C_t
    float acc[NH / 8][4];
    times_state(acc, ax);
    dot_scale(acc, Bs, dotB, dts[ta] * ej[ta], dts[tb] * ej[tb]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k > rt || (k == rt && !careful)) {
        uint32_t af[4], cf[4];
        ldsm4t(af, ar + 2 * frag_at(lane, 16 * rt, 16 * k, L::LM));
        ldsm4t(cf, a2 + 2 * frag_at(lane, 16 * rt, 16 * k, L::LM));
#pragma unroll
        for (int m = 0; m < NH / 16; ++m) {
          uint32_t bf[4];
          ldsm4t(bf, ac + 2 * frag_bt(lane, n0 + 16 * m, 16 * k, L::LN));
          mma_bf16(acc[2 * m], cf, bf[0], bf[1]);
          mma_bf16(acc[2 * m + 1], cf, bf[2], bf[3]);
          mma_bf16(acc[2 * m], af, bf[0], bf[1]);
          mma_bf16(acc[2 * m + 1], af, bf[2], bf[3]);
        }
      }
    if (careful) diagonal(acc, std::true_type(), MR, M2, Cs + n0, L::LN);
    put(acc, dB, ba.sdB, w.pB);
  }
  {  // dx_j = dt_j (e_j dSin B_j + sum_t MG_tj dy_t) + D dy_j
    float acc[PH / 8][4];
#pragma unroll
    for (int m = 0; m < PH / 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
#pragma unroll
    for (int k = 0; k < N; k += 16) {
      uint32_t af[4];
      ldsm4(af, ab + 2 * frag_a(lane, 16 * rt, k, L::LN));
#pragma unroll
      for (int m = 0; m < PH / 16; ++m) {
        uint32_t bf[4];
        ldsm4(bf, as + 2 * frag_b(lane, p0 + 16 * m, k, L::LN));
        mma_bf16(acc[2 * m], af, bf[0], bf[1]);
        mma_bf16(acc[2 * m + 1], af, bf[2], bf[3]);
      }
    }
#pragma unroll
    for (int m = 0; m < PH / 8; ++m) {
      acc[m][0] *= ej[ta]; acc[m][1] *= ej[ta];
      acc[m][2] *= ej[tb]; acc[m][3] *= ej[tb];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k > rt || (k == rt && !careful)) {
        uint32_t af[4];
        ldsm4t(af, ag + 2 * frag_at(lane, 16 * rt, 16 * k, L::LM));
#pragma unroll
        for (int m = 0; m < PH / 16; ++m) {
          uint32_t bf[4];
          ldsm4t(bf, ay + 2 * frag_bt(lane, p0 + 16 * m, 16 * k, L::LX));
          mma_bf16(acc[2 * m], af, bf[0], bf[1]);
          mma_bf16(acc[2 * m + 1], af, bf[2], bf[3]);
        }
      }
    if (careful) diagonal(acc, std::true_type(), MG, static_cast<const __nv_bfloat16*>(nullptr), ys + p0, L::LX);
    const float Dh = D ? D[h] : 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = r ? tb : ta;
      if (t >= n) continue;
      const float d = dts[t];
      __nv_bfloat16* o = dx + row_off(ba.sdx, b, h, t0 + t) + p0 + 2 * q;
#pragma unroll
      for (int m = 0; m < PH / 8; ++m) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(ys + t * L::LX + p0 + 8 * m + 2 * q);
        *reinterpret_cast<uint32_t*>(o + 8 * m) =
            pack_bf16(fmaf(d, acc[m][2 * r], Dh * bf16_lo(u)), fmaf(d, acc[m][2 * r + 1], Dh * bf16_hi(u)));
      }
    }
  }
  __syncthreads();
  if (wp == 0) {
    float xu[2];
    double v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const double yd = double(rowE[t]) + rowE[kGQ + t] + double(eg[t]) * (dotC[t] + dotC[kGQ + t]);
      double ce = 0.0;
#pragma unroll
      for (int r = 0; r < 4; ++r) ce += colE[r * kGQ + t];
      ce += double(ej[t]) * (dotB[t] + dotB[kGQ + t]);
      xu[i] = float(ce);
      v[i] = yd - dts[t] * ce;
    }
    const double s = v[0] + v[1];
    double suf = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // suffix sum over the lanes
      const double u = __shfl_down_sync(0xffffffffu, suf, o);
      if (lane + o < 32) suf += u;
    }
    double end = 0.0;
#pragma unroll
    for (int k = 0; k < kGradWarps; ++k) end += red[k];
    const double after = __shfl_down_sync(0xffffffffu, suf, 1);
    double q1 = (lane == 31 ? 0.0 : after) + v[1] + end, q0 = suf + end;
    if (!isfinite(end)) {  // a state that is not finite at the chunk's end: from its start
      double qs = 0.0, before = s;
      for (int i = lane; i < int(PN); i += 32) qs = fma(double(dSin[i]), double(S0[i]), qs);
      double cd = 0.0;
#pragma unroll
      for (int i = 0; i < 2; ++i) cd += double(eg[2 * lane + i]) * (dotC[2 * lane + i] + dotC[kGQ + 2 * lane + i]);
      qs = exp2(double(hi[kGQ - 1]) + lo[kGQ - 1]) * warp_sum(qs) + warp_sum(cd);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += u;
      }
      before = __shfl_up_sync(0xffffffffu, before, 1);
      if (lane == 0) before = 0.0;
      if (!isfinite(q0)) q0 = qs - before;
      if (!isfinite(q1)) q1 = qs - before - v[0];
    }
    const float Ah = A[h];
    double sA = 0.0, sD = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const double qt = i ? q1 : q0;
      if (t < n) {
        ddt[row_off(ba.sddt, b, h, t0 + t)] = float(Ah * qt + xu[i]);
        sD += dg[t];
      }
      sA = fma(double(dts[t]), qt, sA);
    }
    sA = warp_sum(sA);
    sD = warp_sum(sD);
    if (lane == 0) {
      w.dAD[size_t(blockIdx.x) * 2] = sA;
      w.dAD[size_t(blockIdx.x) * 2 + 1] = sD;
    }
  }
}

template <int P, int N>
static cudaError_t launch_grad(const SsmBwdArgs& ba, const void* x, const float* dt, const float* A,
                               const void* Bm, const void* Cm, const float* D, const float* S0,
                               const void* dy, const float* dST, const SsmBwdWs& w, void* dx, float* ddt,
                               void* dB, void* dC, float* dS0, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const SsmArgs& a = ba.a;
  const unsigned grid = unsigned(a.B * a.H) * unsigned(a.nch);
  const int s1 = int(LocalTile<P, N>::smem), s2 = int(SsmGradTile<P, N>::smem);
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_ssm_local_tile<P, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, s1)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(k_ssm_grad<P, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, s2)) != cudaSuccess)
    return e;
  launch_after(k_ssm_local_tile<P, N>, grid, 2 * P, s1, s, a, (const bf*)x, dt, A, (const bf*)Bm, (const bf*)Cm,
                                                (const bf*)dy, w.fS, w.gS, w.lg);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_ssm_carries(w.fS, w.gS, w.lg, S0, w.ST, dST, dS0, a.B * a.H, a.nch, P * N, s)) != cudaSuccess)
    return e;
  launch_after(k_ssm_grad<P, N>, grid, kGradWarps * 32, s2, s, ba, (const bf*)x, dt, A, (const bf*)Bm, (const bf*)Cm,
                                                    D, (const bf*)dy, w, (bf*)dx, ddt, (bf*)dB, (bf*)dC);
  return cudaGetLastError();
}

cudaError_t launch_ssm_bwd_mma(const SsmBwdArgs& ba, const void* x, const float* dt, const float* A,
                               const void* Bm, const void* Cm, const float* D, const float* S0,
                               const void* dy, const float* dST, const SsmBwdWs& w, void* dx, float* ddt,
                               void* dB, void* dC, float* dS0, cudaStream_t s) {
  const SsmArgs& a = ba.a;
  if (a.P == 64)
    return a.N == 64 ? launch_grad<64, 64>(ba, x, dt, A, Bm, Cm, D, S0, dy, dST, w, dx, ddt, dB, dC, dS0, s)
                     : launch_grad<64, 128>(ba, x, dt, A, Bm, Cm, D, S0, dy, dST, w, dx, ddt, dB, dC, dS0, s);
  return a.N == 64 ? launch_grad<128, 64>(ba, x, dt, A, Bm, Cm, D, S0, dy, dST, w, dx, ddt, dB, dC, dS0, s)
                   : launch_grad<128, 128>(ba, x, dt, A, Bm, Cm, D, S0, dy, dST, w, dx, ddt, dB, dC, dS0, s);
}

}  // namespace sdm
