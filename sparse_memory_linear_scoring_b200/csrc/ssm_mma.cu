// ssm_mma.cu -- the selective scan's chunk walk on the tensor cores (bf16 inputs,
// widths 64 and 128).  ssm_internal.cuh has the chunk formulas, ssm.cu the
// segments.
//
// A CTA walks one segment of 64 rows of one head's S in chunks of 64 steps (the rows of S
// do not meet; at d_v = 128 the two halves share only the scores, a tenth of the
// products, and two CTAs of 4 warps an SM, each at its own barriers, keep the tensor
// cores busier than one of 8).  Warp w owns rows 16 w .. 16 w + 15, which stay in its
// registers as float32 accumulators from chunk to chunk; the chunk's x, B and C tiles
// arrive by cp.async one chunk ahead.
// Per chunk:
//   scores G = C B^T, weights M = mask exp(g_t - g_j) dt_j G (bf16 for the next
//   product: one rounding of a weight, below that of y itself),
//   y = M x + exp(g_t) (C S^T) + D x   (S rounded to bf16 for this product only),
//   S = exp(g_Q) S + (w x)^T B with w_j = exp(g_Q - g_j) dt_j.
// S itself is an output in float32 and is carried over thousands of steps, so where it
// becomes one (a segment's own contribution; a walk of one segment) w x is split into
// three bf16 parts (what is left is below 2^-24) against the exact B.  In the second walk
// of several segments S only makes y, whose product takes it rounded to bf16: there two
// parts do (2^-16 of a term beside 2^-9), a fifth fewer products at 128 x 128.  The last
// state then comes from the carry.
// (With the two roundings of y's operands y is 0.0019 to 0.0023 of its norm off, where the
// result's rounding alone makes 0.0017.)
// A chunk whose x holds an infinity or NaN is found as its tiles arrive, by 0 times its
// elements, and a state that is not finite when the segment ends; both are rare and slow.
// 65536 steps of 8 heads of 128 x 128: 307 us the outputs (300 without that check).  Warp-level products (about 0.4
// of the 0.83 a ns and SM they reach) and the instructions around them bound it: the
// weights' exponentials with denormal results alone were worth 47 us; factors of rows and
// columns in place of most of the exponentials took 13 us more.  The first walk took 178 us
// this way at d_k = 128, where ssm_tc.cu now takes it.
#include "mma_dev.cuh"
#include "ssm_internal.cuh"

namespace sdm {

constexpr int kTQ = kSsmQT;  // 64

template <int N, bool OUT>
struct SsmTile {
  static constexpr int P = 64;                     // rows of S
  static constexpr int LX = P + 8, LN = N + 8;     // pitches: ldmatrix without bank conflicts
  static constexpr int X = kTQ * LX, BC = kTQ * LN;
  static constexpr int STAGE = X + (OUT ? 2 : 1) * BC;   // bf16 elements
  static constexpr int SB = OUT ? P * LN : 0;            // S rounded to bf16
  static constexpr int DEC = 5 * kTQ;                    // hi, lo, dt, exp(g), w
  static constexpr size_t smem = size_t(2) * (2 * STAGE + SB) + size_t(4) * 2 * DEC + 16;  // flags at the end
};

// Warp 0: decays of one chunk from its steps 2 lane, 2 lane + 1.
__device__ __forceinline__ void tile_decay(float* dec, float d0, float d1, float A) {
  float *hi = dec, *lo = dec + kTQ, *dts = dec + 2 * kTQ, *eg = dec + 3 * kTQ, *w = dec + 4 * kTQ;
  const int lane = threadIdx.x & 31;
  dts[2 * lane] = d0;
  dts[2 * lane + 1] = d1;
  __syncwarp();
  chunk_decay<2>(dts, A, hi, lo);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 2 * lane + i;
    eg[t] = ex2(hi[t] + lo[t]);
    w[t] = decay_between(hi[kTQ - 1], lo[kTQ - 1], hi[t], lo[t]) * dts[t];
  }
}

template <int N, bool OUT, int PARTS>
__global__ void __launch_bounds__(128)
k_ssm_tile(SsmArgs a, const __nv_bfloat16* __restrict__ x, const float* __restrict__ dt,
           const float* __restrict__ A, const __nv_bfloat16* __restrict__ Bm,
           const __nv_bfloat16* __restrict__ Cm, const float* __restrict__ D, float* __restrict__ S,
           const int32_t* __restrict__ lengths, __nv_bfloat16* __restrict__ y,
           float* __restrict__ segS, float* __restrict__ segG) {
  wait_for_previous();
  using L = SsmTile<N, OUT>;
  constexpr int P = L::P;
  extern __shared__ __align__(16) unsigned char raw[];
  __nv_bfloat16* st = reinterpret_cast<__nv_bfloat16*>(raw);
  __nv_bfloat16* Sb = st + 2 * L::STAGE;
  float* dec = reinterpret_cast<float*>(Sb + L::SB);
  volatile int* odd = reinterpret_cast<volatile int*>(dec + 2 * L::DEC);  // [2]: last chunk + 1 with inf or NaN in x
  constexpr int NT = 128;
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int seg = blockIdx.x % a.nseg, halves = a.P / P;
  const int bp = blockIdx.x / a.nseg, bh = bp / halves, pr = (bp - bh * halves) * P;  // first row of S
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  x += pr;
  y += pr;
  const int T = seq_len(lengths, b, a.T);
  const float Ah = A[h], Dh = OUT && D ? D[h] : 0.f;
  const int c0 = seg * a.cps, c1 = min(c0 + a.cps, a.nch);

  auto load = [&](int c) {
    __nv_bfloat16* s = st + (c & 1) * L::STAGE;
    const int t0 = c * kTQ;
    const uint32_t sx = smem_u32(s), sb = sx + 2 * L::X, sc = sb + 2 * L::BC;
    for (int i = tid; i < kTQ * (P / 8); i += NT) {
      const int t = i / (P / 8), e = (i % (P / 8)) * 8;
      const bool in = t0 + t < T;
      cp_async16(sx + 2 * (t * L::LX + e), x + row_off(a.sx, b, h, in ? t0 + t : 0) + e, in);
    }
    for (int i = tid; i < kTQ * (N / 8); i += NT) {
      const int t = i / (N / 8), e = (i % (N / 8)) * 8;
      const bool in = t0 + t < T;
      const int tt = in ? t0 + t : 0;
      cp_async16(sb + 2 * (t * L::LN + e), Bm + row_off(a.sB, b, gr, tt) + e, in);
      if (OUT) cp_async16(sc + 2 * (t * L::LN + e), Cm + row_off(a.sC, b, gr, tt) + e, in);
    }
  };
  // whether the thread's own pieces of x, which have arrived, hold an infinity or NaN
  auto own_odd = [&](const __nv_bfloat16* s) {
    OddBf16 z;
#pragma unroll
    for (int i = 0; i < kTQ * (P / 8) / NT; ++i) {
      const int e = tid + i * NT;
      z.add(s + e / (P / 8) * L::LX + (e % (P / 8)) * 8);
    }
    return z.any();
  };
  auto dt_at = [&](int c, int i) {
    const int t = c * kTQ + 2 * lane + i;
    return c < c1 && t < T ? dt[row_off(a.sdt, b, h, t)] : 0.f;
  };

  // S rows 16 wp + g, + 8; columns 8 n + 2 q, + 1
  const int g = lane >> 2, q = lane & 3;
  float s[N / 8][4];
  const size_t PN = size_t(a.P) * N;
  float* slot = (a.nseg > 1 ? segS + (size_t(bh) * a.nseg + seg) * PN : S + size_t(bh) * PN) + size_t(pr) * N;
#pragma unroll
  for (int n = 0; n < N / 8; ++n) {
    const float* p0 = slot + (16 * wp + g) * N + 8 * n + 2 * q;
    float2 u = make_float2(0.f, 0.f), v = u;
    if (OUT) {
      u = *reinterpret_cast<const float2*>(p0);
      v = *reinterpret_cast<const float2*>(p0 + 8 * N);
    }
    s[n][0] = u.x; s[n][1] = u.y; s[n][2] = v.x; s[n][3] = v.y;
  }
  auto put_state = [&]() {
#pragma unroll
    for (int n = 0; n < N / 8; ++n) {
      __nv_bfloat16* p0 = Sb + (16 * wp + g) * L::LN + 8 * n + 2 * q;
      *reinterpret_cast<uint32_t*>(p0) = pack_bf16(s[n][0], s[n][1]);
      *reinterpret_cast<uint32_t*>(p0 + 8 * L::LN) = pack_bf16(s[n][2], s[n][3]);
    }
  };
  if (OUT) {
    put_state();
    if (tid < 2) odd[tid] = 0;
    __syncthreads();
  }
  load(c0);
  cp_async_commit();
  if (c0 + 1 < c1) load(c0 + 1);
  cp_async_commit();
  if (wp == 0) tile_decay(dec + (c0 & 1) * L::DEC, dt_at(c0, 0), dt_at(c0, 1), Ah);
  float tot = 0.f;

  for (int c = c0; c < c1; ++c) {
    cp_async_wait<1>();
    const __nv_bfloat16* xs = st + (c & 1) * L::STAGE;
    if (OUT && own_odd(xs)) odd[c & 1] = c + 1;
    __syncthreads();  // chunk c's tiles, decays and bf16 state are in place
    const bool careful = OUT && odd[c & 1] == c + 1;  // x holds inf or NaN
    __nv_bfloat16* yw = st + (c & 1) * L::STAGE + L::X + L::BC + wp * 16 * L::LN;  // C rows of the warp
    const uint32_t ax = smem_u32(xs), ab = ax + 2 * L::X, ac = ab + 2 * L::BC;
    const float* dc = dec + (c & 1) * L::DEC;
    const float *hi = dc, *lo = dc + kTQ, *dts = dc + 2 * kTQ, *eg = dc + 3 * kTQ, *wj = dc + 4 * kTQ;
    float nd0 = 0.f, nd1 = 0.f;
    if (wp == 0) {  // next chunk's steps, read ahead
      nd0 = dt_at(c + 1, 0);
      nd1 = dt_at(c + 1, 1);
    }
    const int t0 = c * kTQ, live = T - t0;
    if (OUT) {
      const int rt = wp;  // rows 16 rt.. of y
      float acc[8][4];
      if (live > 16 * rt) {
        float sc[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = sc[n][i] = 0.f;
#pragma unroll
        for (int k = 0; k < N; k += 16) {
          uint32_t af[4];
          ldsm4(af, ac + 2 * frag_a(lane, 16 * rt, k, L::LN));
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            if (n <= rt) {
              uint32_t bf[4];
              ldsm4(bf, ab + 2 * frag_b(lane, 16 * n, k, L::LN));
              mma_bf16(sc[2 * n], af, bf[0], bf[1]);
              mma_bf16(sc[2 * n + 1], af, bf[2], bf[3]);
            }
            uint32_t sf[4];
            ldsm4(sf, smem_u32(Sb) + 2 * frag_b(lane, 16 * n, k, L::LN));
            mma_bf16(acc[2 * n], af, sf[0], sf[1]);
            mma_bf16(acc[2 * n + 1], af, sf[2], sf[3]);
          }
        }
        const int ta = 16 * rt + g, tb = ta + 8;
        const float ea = eg[ta], eb = eg[tb], ha = hi[ta], hb = hi[tb], la = lo[ta], lb = lo[tb];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          acc[n][0] *= ea; acc[n][1] *= ea;
          acc[n][2] *= eb; acc[n][3] *= eb;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k <= rt) {
            uint32_t mf[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int j = 16 * k + 8 * u + 2 * q;
              const float2 hj = *reinterpret_cast<const float2*>(hi + j);
              const float2 lj = *reinterpret_cast<const float2*>(lo + j);
              const float2 dj = *reinterpret_cast<const float2*>(dts + j);
              float* v = sc[2 * k + u];
              const float m0 = j <= ta ? decay_between(ha, la, hj.x, lj.x) * dj.x * v[0] : 0.f;
              const float m1 = j + 1 <= ta ? decay_between(ha, la, hj.y, lj.y) * dj.y * v[1] : 0.f;
              const float m2 = j <= tb ? decay_between(hb, lb, hj.x, lj.x) * dj.x * v[2] : 0.f;
              const float m3 = j + 1 <= tb ? decay_between(hb, lb, hj.y, lj.y) * dj.y * v[3] : 0.f;
              mf[2 * u] = pack_bf16(m0, m1);
              mf[2 * u + 1] = pack_bf16(m2, m3);
            }
            if (careful && k == rt) {  // the diagonal without the masked products
#pragma unroll 1
              for (int z = 0; z < 16; ++z) {  // column 16 k + z of M: lane z % 8 / 2 of the row's four
                const int from = (lane & ~3) | ((z & 7) >> 1);
                const uint32_t wa = __shfl_sync(0xffffffffu, z < 8 ? mf[0] : mf[2], from);
                const uint32_t wb = __shfl_sync(0xffffffffu, z < 8 ? mf[1] : mf[3], from);
                const float ma = z & 1 ? bf16_hi(wa) : bf16_lo(wa), mb = z & 1 ? bf16_hi(wb) : bf16_lo(wb);
                const __nv_bfloat16* xr = xs + (16 * k + z) * L::LX + 2 * q;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                  const uint32_t u = *reinterpret_cast<const uint32_t*>(xr + 8 * n);
                  if (z <= g) {
                    acc[n][0] = fmaf(ma, bf16_lo(u), acc[n][0]);
                    acc[n][1] = fmaf(ma, bf16_hi(u), acc[n][1]);
                  }
                  if (z <= g + 8) {
                    acc[n][2] = fmaf(mb, bf16_lo(u), acc[n][2]);
                    acc[n][3] = fmaf(mb, bf16_hi(u), acc[n][3]);
                  }
                }
              }
            } else {
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                uint32_t xf[4];
                ldsm4t(xf, ax + 2 * frag_bt(lane, 16 * n, 16 * k, L::LX));
                mma_bf16(acc[2 * n], mf, xf[0], xf[1]);
                mma_bf16(acc[2 * n + 1], mf, xf[2], xf[3]);
              }
            }
          }
        }
        // + D x, rows at or past the end are 0; through shared memory to 16-byte stores, in
        // the place of the warp's own rows of C, which no other warp reads
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int e = 8 * n + 2 * q;
          const uint32_t xa = *reinterpret_cast<const uint32_t*>(xs + ta * L::LX + e);
          const uint32_t xb = *reinterpret_cast<const uint32_t*>(xs + tb * L::LX + e);
          *reinterpret_cast<uint32_t*>(yw + g * L::LN + e) =
              ta < live ? pack_bf16(fmaf(Dh, bf16_lo(xa), acc[n][0]), fmaf(Dh, bf16_hi(xa), acc[n][1])) : 0u;
          *reinterpret_cast<uint32_t*>(yw + (g + 8) * L::LN + e) =
              tb < live ? pack_bf16(fmaf(Dh, bf16_lo(xb), acc[n][2]), fmaf(Dh, bf16_hi(xb), acc[n][3])) : 0u;
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 3) + 4 * i, t = t0 + 16 * rt + r;
        if (t < a.T) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (live > 16 * rt) v = *reinterpret_cast<const uint4*>(yw + r * L::LN + (lane & 7) * 8);
          *reinterpret_cast<uint4*>(y + row_off(a.sy, b, h, t) + (lane & 7) * 8) = v;
        }
      }
    }
    const float gq = hi[kTQ - 1] + lo[kTQ - 1];
    tot += gq;
    if (live > 0) {
      // (w x)^T as A fragments in parts, all 64 steps
      uint32_t xw[4][PARTS][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t xf[4];
        ldsm4t(xf, ax + 2 * frag_at(lane, 16 * wp, 16 * k, L::LX));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 w = *reinterpret_cast<const float2*>(wj + 16 * k + (i >> 1) * 8 + 2 * q);
          uint32_t u[PARTS];
          split_bf16<PARTS>(bf16_lo(xf[i]) * w.x, bf16_hi(xf[i]) * w.y, u);
#pragma unroll
          for (int z = 0; z < PARTS; ++z) xw[k][z][i] = u[z];
        }
      }
      const float eq = ex2(gq);
#pragma unroll
      for (int n = 0; n < N / 16; ++n) {
        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t bf[4];
          ldsm4t(bf, ab + 2 * frag_bt(lane, 16 * n, 16 * k, L::LN));
#pragma unroll
          for (int i = PARTS - 1; i >= 0; --i) {  // small parts first
            mma_bf16(d0, xw[k][i], bf[0], bf[1]);
            mma_bf16(d1, xw[k][i], bf[2], bf[3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[2 * n][i] = fmaf(eq, s[2 * n][i], d0[i]);
          s[2 * n + 1][i] = fmaf(eq, s[2 * n + 1][i], d1[i]);
        }
      }
    }
    if (wp == 0 && c + 1 < c1) tile_decay(dec + ((c + 1) & 1) * L::DEC, nd0, nd1, Ah);
    __syncthreads();  // everyone is done with chunk c's tiles and state
    if (OUT) put_state();
    if (c + 2 < c1) load(c + 2);
    cp_async_commit();
  }
  cp_async_wait<0>();
  float* out = OUT ? S + size_t(bh) * PN + size_t(pr) * N : slot;
  if (!OUT || a.nseg == 1) {
    bool bad = false;
#pragma unroll
    for (int n = 0; n < N / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) bad |= !(fabsf(s[n][i]) < INFINITY);
    if (bad) {  // inf or NaN in S, x or B, which parts do not add up to: the recurrence itself
#pragma unroll
      for (int n = 0; n < N / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[n][i] = OUT ? slot[(16 * wp + g + (i >> 1) * 8) * N + 8 * n + 2 * q + (i & 1)] : 0.f;
#pragma unroll 1
      for (int t = c0 * kTQ; t < min(c1 * kTQ, T); ++t) {
        const float d = dt[row_off(a.sdt, b, h, t)], at = expf(d * Ah);
        const __nv_bfloat16* xr = x + row_off(a.sx, b, h, t) + 16 * wp + g;
        const __nv_bfloat16* br = Bm + row_off(a.sB, b, gr, t) + 2 * q;
        const float ua = d * __bfloat162float(xr[0]), ub = d * __bfloat162float(xr[8]);
#pragma unroll
        for (int n = 0; n < N / 8; ++n) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(br + 8 * n);
          s[n][0] = fmaf(at, s[n][0], ua * bf16_lo(u));
          s[n][1] = fmaf(at, s[n][1], ua * bf16_hi(u));
          s[n][2] = fmaf(at, s[n][2], ub * bf16_lo(u));
          s[n][3] = fmaf(at, s[n][3], ub * bf16_hi(u));
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N / 8; ++n) {
      float* p0 = out + (16 * wp + g) * N + 8 * n + 2 * q;
      *reinterpret_cast<float2*>(p0) = make_float2(s[n][0], s[n][1]);
      *reinterpret_cast<float2*>(p0 + 8 * N) = make_float2(s[n][2], s[n][3]);
    }
  }
  if (!OUT && tid == 0 && pr == 0) segG[size_t(bh) * a.nseg + seg] = tot;
}

template <int N>
static cudaError_t launch_tile(const SsmArgs& a, const void* x, const float* dt, const float* A,
                               const void* Bm, const void* Cm, const float* D, float* S,
                               const int32_t* lengths, void* y, float* segS, float* segG,
                               cudaStream_t s) {
  using bf = __nv_bfloat16;
  const unsigned grid = unsigned(a.B * a.H) * unsigned(a.P / 64) * unsigned(a.nseg);
  const int s1 = int(SsmTile<N, true>::smem);
  auto go = [&](auto kernel, int sm) -> cudaError_t {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    if (r != cudaSuccess) return r;
    launch_after(kernel, grid, 128, sm, s, a, (const bf*)x, dt, A, (const bf*)Bm, (const bf*)Cm, D, S, lengths, (bf*)y,
                                 segS, segG);
    return cudaGetLastError();
  };
  if (a.nseg == 1) return go(k_ssm_tile<N, true, 3>, s1);
  cudaError_t e;
  if constexpr (N == 128) e = launch_ssm_seg(a, x, dt, A, Bm, lengths, segS, segG, s);
  else e = go(k_ssm_tile<N, false, 3>, int(SsmTile<N, false>::smem));
  if (e == cudaSuccess) e = launch_ssm_carry(segS, segG, S, S, a.B * a.H, a.nseg, a.P * N, s);
  return e == cudaSuccess ? go(k_ssm_tile<N, true, 2>, s1) : e;
}

cudaError_t launch_ssm_fwd_mma(const SsmArgs& a, const void* x, const float* dt, const float* A,
                               const void* Bm, const void* Cm, const float* D, float* S,
                               const int32_t* lengths, void* y, float* segS, float* segG,
                               cudaStream_t s) {
  return a.N == 64 ? launch_tile<64>(a, x, dt, A, Bm, Cm, D, S, lengths, y, segS, segG, s)
                   : launch_tile<128>(a, x, dt, A, Bm, Cm, D, S, lengths, y, segS, segG, s);
}

}  // namespace sdm
