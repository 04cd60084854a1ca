// ssm_bwd.cu -- gradients of the selective state space scan.
//
// With dS_t the gradient of S_t, dS_t = dy_t C_t^T + a_{t+1} dS_{t+1}.  Inside a
// chunk with W_tj = exp(g_t - g_j), G_tj = C_t.B_j, R_tj = dy_t.x_j, the state S_0
// before it and the gradient dSin that arrives at its end, e_j = exp(g_Q - g_j),
// I1_t = S_0^T dy_t and I2_j = dSin^T x_j:
//     du_j = sum_{t>=j} W_tj G_tj dy_t + e_j dSin B_j,      dx_j = dt_j du_j + D dy_j,
//     dB_j = dt_j (sum_{t>=j} W_tj R_tj C_t + e_j I2_j),
//     dC_t = sum_{j<=t} W_tj dt_j R_tj B_j + exp(g_t) I1_t,
//     dS_0 = exp(g_Q) dSin + sum_t exp(g_t) dy_t C_t^T.
// The gradient of dt_t A is q_t = <dS_t, a_t S_{t-1}>.  It never needs a state
// inside the chunk: <dS_t, S_t> = dy_t.(S_t C_t) + q_{t+1}, so
//     q_t = q_{t+1} + dy_t.(S_t C_t) - dt_t x_t.du_t,   q_{Q+1} = <dSin, S_Q>,
// and both dots come from sums over W G R and from C_t.I1_t, B_j.I2_j, which are
// at hand.  Starting the sum anew at each chunk's end keeps its rounding from
// piling up along the sequence.  Where S_Q is not finite (a NaN in x or B of some step),
// the steps before that take it from the chunk's start instead, which is
//     q_1 = exp(g_Q) <dSin, S_0> + sum_t exp(g_t) C_t.I1_t.  ddt_t = x_t.du_t + A q_t, dA = sum dt_t q_t,
// dD = sum x_t.dy_t.
//
// Passes: k_ssm_local (each chunk's own contribution to the states and to their
// gradients), two carries, then k_ssm_bwd over all (head, chunk) pairs at once;
// gradients of shared B and C are summed over the group's heads in order.
#include <utility>

#include "ssm_internal.cuh"

namespace sdm {

constexpr int kBwdThreads = 256;

static SsmBwdWs ssm_bwd_ws(const sdm_ssm_dims* d, int Q, void* base) {
  SsmBwdWs w;
  memset(&w, 0, sizeof(w));
  const size_t BH = size_t(d->B) * d->H, PN = size_t(d->d_v) * d->d_k;
  const size_t nch = size_t((d->T + Q - 1) / Q);
  char* b = static_cast<char*>(base);
  size_t o = 0;
  auto take = [&](size_t floats) {
    float* p = reinterpret_cast<float*>(b + o);
    o = (o + floats * 4 + 255) & ~size_t(255);
    return p;
  };
  w.fS = take(BH * nch * PN);
  w.gS = take(BH * nch * PN);
  w.ST = take(BH * PN);
  w.lg = take(BH * nch);
  w.dAD = reinterpret_cast<double*>(take(BH * nch * 4));
  if (d->H != d->G) {
    w.pB = take(BH * d->T * d->d_k);
    w.pC = take(BH * d->T * d->d_k);
  }
  w.total = o;
  return w;
}

// Loads of a chunk's rows as float32; rows past n are zero.
template <typename Tin>
__device__ __forceinline__ void load_rows(float* dst, int ld, const Tin* src, const sdm_strides& s,
                                          int b, int h, int t0, int n, int Q, int W) {
  for (int i = threadIdx.x; i < Q * W; i += kBwdThreads) {
    const int t = i / W, e = i - t * W;
    dst[t * ld + e] = t < n ? to_f32(src[row_off(s, b, h, t0 + t) + e]) : 0.f;
  }
}

template <typename Tin>
__global__ void __launch_bounds__(kBwdThreads)
k_ssm_local(SsmArgs a, const Tin* __restrict__ x, const float* __restrict__ dt,
            const float* __restrict__ A, const Tin* __restrict__ Bm, const Tin* __restrict__ Cm,
            const Tin* __restrict__ dy, float* __restrict__ fS, float* __restrict__ gS,
            float* __restrict__ lg) {
  wait_for_previous();
  extern __shared__ __align__(16) float sm[];
  constexpr int Q = kSsmQ;
  const int P = a.P, N = a.N;
  float* xs = sm;             // [Q][P] x scaled by exp(g_Q - g_j) dt_j
  float* ys = xs + Q * P;     // [Q][P] dy scaled by exp(g_t)
  float* Bs = ys + Q * P;     // [Q][N]
  float* Cs = Bs + Q * N;
  float* dts = Cs + Q * N;
  float* hi = dts + Q;
  float* lo = hi + Q;
  const int c = blockIdx.x % a.nch, bh = blockIdx.x / a.nch;
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  const int t0 = c * Q, n = min(Q, a.T - t0), tid = threadIdx.x;
  if (tid < Q) dts[tid] = tid < n ? dt[row_off(a.sdt, b, h, t0 + tid)] : 0.f;
  load_rows(Bs, N, Bm, a.sB, b, gr, t0, n, Q, N);
  load_rows(Cs, N, Cm, a.sC, b, gr, t0, n, Q, N);
  __syncthreads();
  if (tid < 32) chunk_decay<1>(dts, A[h], hi, lo);
  __syncthreads();
  for (int i = tid; i < Q * P; i += kBwdThreads) {
    const int t = i / P, p = i - t * P;
    const bool in = t < n;
    xs[i] = in ? to_f32(x[row_off(a.sx, b, h, t0 + t) + p]) * dts[t] *
                     decay_between(hi[Q - 1], lo[Q - 1], hi[t], lo[t])
               : 0.f;
    ys[i] = in ? to_f32(dy[row_off(a.sy, b, h, t0 + t) + p]) * ex2(hi[t] + lo[t]) : 0.f;
  }
  __syncthreads();
  const size_t o = size_t(blockIdx.x) * P * N;
  const int nn4 = N >> 2;
  for (int tile = tid; tile < (P >> 2) * nn4; tile += kBwdThreads) {
    const int p = (tile / nn4) * 4, e = (tile % nn4) * 4;
    float s[4][4] = {}, g[4][4] = {};
    for (int j = 0; j < n; ++j) {
      const float4 xv = *reinterpret_cast<const float4*>(xs + j * P + p);
      const float4 yv = *reinterpret_cast<const float4*>(ys + j * P + p);
      const float4 bv = *reinterpret_cast<const float4*>(Bs + j * N + e);
      const float4 cv = *reinterpret_cast<const float4*>(Cs + j * N + e);
      const float xa[4] = {xv.x, xv.y, xv.z, xv.w}, ya[4] = {yv.x, yv.y, yv.z, yv.w};
      const float ba[4] = {bv.x, bv.y, bv.z, bv.w}, ca[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          s[u][v] = fmaf(xa[u], ba[v], s[u][v]);
          g[u][v] = fmaf(ya[u], ca[v], g[u][v]);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const size_t at = o + size_t(p + u) * N + e;
      *reinterpret_cast<float4*>(fS + at) = make_float4(s[u][0], s[u][1], s[u][2], s[u][3]);
      *reinterpret_cast<float4*>(gS + at) = make_float4(g[u][0], g[u][1], g[u][2], g[u][3]);
    }
  }
  if (tid == 0) lg[blockIdx.x] = hi[Q - 1] + lo[Q - 1];
}

__host__ __device__ inline size_t ssm_bwd_smem(int P, int N) {
  constexpr int Q = kSsmQ;
  return size_t(4) * (2 * Q * (P + 1) + 2 * Q * (N + 1) + 3 * Q * (Q + 1) + Q * 33 * 2 + 6 * Q + 32);
}

template <typename Tin>
__global__ void __launch_bounds__(kBwdThreads)
k_ssm_bwd(SsmBwdArgs ba, const Tin* __restrict__ x, const float* __restrict__ dt,
          const float* __restrict__ A, const Tin* __restrict__ Bm, const Tin* __restrict__ Cm,
          const float* __restrict__ D, const Tin* __restrict__ dy, SsmBwdWs w, Tin* __restrict__ dx,
          float* __restrict__ ddt, Tin* __restrict__ dB, Tin* __restrict__ dC) {
  wait_for_previous();
  extern __shared__ __align__(16) float sm[];
  const SsmArgs& a = ba.a;
  constexpr int Q = kSsmQ, Qp = Q + 1;
  const int P = a.P, N = a.N, Pp = P + 1, Np = N + 1;
  float* xs = sm;
  float* ys = xs + Q * Pp;
  float* Bs = ys + Q * Pp;
  float* Cs = Bs + Q * Np;
  float* MG = Cs + Q * Np;   // W G
  float* MR = MG + Q * Qp;   // W dt_j R
  float* E = MR + Q * Qp;    // W G R
  float* pc = E + Q * Qp;    // parts of C_t.I1_t
  float* pb = pc + Q * 33;   // parts of B_j.I2_j
  float* dts = pb + Q * 33;
  float* hi = dts + Q;
  float* lo = hi + Q;
  float* rowE = lo + Q;
  float* colE = rowE + Q;
  float* dg = colE + Q;      // R_tt
  // 8-byte aligned: an even number of floats lies before it
  double* red = reinterpret_cast<double*>(dg + Q);
  const int c = blockIdx.x % a.nch, bh = blockIdx.x / a.nch;
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  const int t0 = c * Q, n = min(Q, a.T - t0), tid = threadIdx.x;
  const size_t PN = size_t(P) * N;
  const float* S0 = w.fS + size_t(blockIdx.x) * PN;
  const float* dSin = w.gS + size_t(blockIdx.x) * PN;
  const float* Send = c + 1 < a.nch ? S0 + PN : w.ST + size_t(bh) * PN;
  if (tid < Q) dts[tid] = tid < n ? dt[row_off(a.sdt, b, h, t0 + tid)] : 0.f;
  load_rows(xs, Pp, x, a.sx, b, h, t0, n, Q, P);
  load_rows(ys, Pp, dy, a.sy, b, h, t0, n, Q, P);
  load_rows(Bs, Np, Bm, a.sB, b, gr, t0, n, Q, N);
  load_rows(Cs, Np, Cm, a.sC, b, gr, t0, n, Q, N);
  __syncthreads();
  if (tid < 32) chunk_decay<1>(dts, A[h], hi, lo);
  // <dSin, S_Q>, in double: it enters every q of the chunk, and dA sums them over all steps
  double bnd = 0.0;
  for (size_t i = tid; i < PN; i += kBwdThreads) bnd = fma(double(dSin[i]), double(Send[i]), bnd);
  bnd = warp_sum(bnd);
  if ((tid & 31) == 0) red[tid >> 5] = bnd;
  __syncthreads();
  {
    const int t = (tid >> 4) * 2, j = (tid & 15) * 2;
    float g[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, r[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    if (j <= t + 1) {
      for (int e = 0; e < N; ++e)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) g[u][v] = fmaf(Cs[(t + u) * Np + e], Bs[(j + v) * Np + e], g[u][v]);
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) r[u][v] = fmaf(ys[(t + u) * Pp + p], xs[(j + v) * Pp + p], r[u][v]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int tt = t + u, jj = j + v;
        // chosen, not multiplied by 0: a later step may hold a NaN
        const bool in = jj <= tt;
        const float W = in ? decay_between(hi[tt], lo[tt], hi[jj], lo[jj]) : 0.f;
        MG[tt * Qp + jj] = in ? W * g[u][v] : 0.f;
        MR[tt * Qp + jj] = in ? W * dts[jj] * r[u][v] : 0.f;
        E[tt * Qp + jj] = in ? W * g[u][v] * r[u][v] : 0.f;
        if (tt == jj) dg[tt] = r[u][v];
      }
  }
  __syncthreads();
  if (tid < Q) {
    float s = 0.f;
    for (int j = 0; j <= tid; ++j) s = fmaf(E[tid * Qp + j], dts[j], s);
    rowE[tid] = s;
  } else if (tid < 2 * Q) {
    const int j = tid - Q;
    float s = 0.f;
    for (int t = j; t < Q; ++t) s += E[t * Qp + j];
    colE[j] = s;
  }
  const int nn4 = N >> 2, np4 = P >> 2;
  for (int tile = tid; tile < 2 * (Q >> 2) * nn4; tile += kBwdThreads) {
    // tiles of dC first, then of dB
    const bool forC = tile < (Q >> 2) * nn4;
    const int tl = forC ? tile : tile - (Q >> 2) * nn4;
    const int t = (tl / nn4) * 4, e = (tl % nn4) * 4;
    const float* rows = forC ? ys : xs;
    const float* mat = forC ? S0 : dSin;
    float acc[4][4] = {};
    for (int p = 0; p < P; ++p) {
      const float4 m4 = *reinterpret_cast<const float4*>(mat + size_t(p) * N + e);
      const float mv[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float rv = rows[(t + u) * Pp + p];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(rv, mv[v], acc[u][v]);
      }
    }
    const float* dot = forC ? Cs : Bs;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < 4; ++v) s = fmaf(acc[u][v], dot[(t + u) * Np + e + v], s);
      (forC ? pc : pb)[(t + u) * 33 + (e >> 2)] = s;
      const float f = forC ? ex2(hi[t + u] + lo[t + u])
                           : dts[t + u] * decay_between(hi[Q - 1], lo[Q - 1], hi[t + u], lo[t + u]);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[u][v] *= f;
    }
    // (the diagonal by itself, for the same reason)
    if (forC) {
      for (int j = 0; j < t; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float m = MR[(t + u) * Qp + j];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(m, Bs[j * Np + e + v], acc[u][v]);
        }
#pragma unroll
      for (int z = 0; z < 4; ++z)
#pragma unroll
        for (int u = z; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[u][v] = fmaf(MR[(t + u) * Qp + t + z], Bs[(t + z) * Np + e + v], acc[u][v]);
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z)
#pragma unroll
        for (int u = 0; u <= z; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[u][v] = fmaf(MR[(t + z) * Qp + t + u], Cs[(t + z) * Np + e + v], acc[u][v]);
      for (int s = t + 4; s < Q; ++s)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float m = MR[s * Qp + t + u];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(m, Cs[s * Np + e + v], acc[u][v]);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (t + u >= n) break;
      if (a.hg == 1) {
        Tin* o = forC ? dC + row_off(ba.sdC, b, gr, t0 + t + u) + e
                      : dB + row_off(ba.sdB, b, gr, t0 + t + u) + e;
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = from_f32<Tin>(acc[u][v]);
      } else {
        float* o = (forC ? w.pC : w.pB) + (size_t(bh) * a.T + t0 + t + u) * N + e;
        *reinterpret_cast<float4*>(o) = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
      }
    }
  }
  for (int tile = tid; tile < (Q >> 2) * np4; tile += kBwdThreads) {
    const int t = (tile / np4) * 4, p = (tile % np4) * 4;
    float acc[4][4] = {};
    for (int e = 0; e < N; e += 4) {
      float4 m[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) m[v] = *reinterpret_cast<const float4*>(dSin + size_t(p + v) * N + e);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float* bp = Bs + (t + u) * Np + e;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[u][v] = fmaf(bp[0], m[v].x, fmaf(bp[1], m[v].y, fmaf(bp[2], m[v].z, fmaf(bp[3], m[v].w, acc[u][v]))));
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = decay_between(hi[Q - 1], lo[Q - 1], hi[t + u], lo[t + u]);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[u][v] *= f;
    }
#pragma unroll
    for (int z = 0; z < 4; ++z)
#pragma unroll
      for (int u = 0; u <= z; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[u][v] = fmaf(MG[(t + z) * Qp + t + u], ys[(t + z) * Pp + p + v], acc[u][v]);
    for (int s = t + 4; s < Q; ++s)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float m = MG[s * Qp + t + u];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(m, ys[s * Pp + p + v], acc[u][v]);
      }
    const float Dh = D ? D[h] : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (t + u >= n) break;
      Tin* o = dx + row_off(ba.sdx, b, h, t0 + t + u) + p;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        o[v] = from_f32<Tin>(fmaf(dts[t + u], acc[u][v], Dh * ys[(t + u) * Pp + p + v]));
    }
  }
  __syncthreads();
  if (tid < 32) {
    float ci = 0.f, bi = 0.f;
    for (int k = 0; k < nn4; ++k) {
      ci += pc[tid * 33 + k];
      bi += pb[tid * 33 + k];
    }
    const double yd = double(rowE[tid]) + double(ex2(hi[tid] + lo[tid])) * ci;
    const double xu = double(colE[tid]) + double(decay_between(hi[Q - 1], lo[Q - 1], hi[tid], lo[tid])) * bi;
    const double v = yd - dts[tid] * xu;
    double q = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // suffix sum
      const double u = __shfl_down_sync(0xffffffffu, q, o);
      if (tid + o < 32) q += u;
    }
    double end = 0.0;
    for (int k = 0; k < kBwdThreads / 32; ++k) end += red[k];
    q += end;
    if (!isfinite(end)) {  // a state that is not finite at the chunk's end: from its start
      double q1 = 0.0, before = v;
      for (size_t i = tid; i < PN; i += 32) q1 = fma(double(dSin[i]), double(S0[i]), q1);
      q1 = exp2(double(hi[Q - 1]) + lo[Q - 1]) * warp_sum(q1) + warp_sum(double(ex2(hi[tid] + lo[tid])) * ci);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(0xffffffffu, before, o);
        if (tid >= o) before += u;
      }
      before = __shfl_up_sync(0xffffffffu, before, 1);
      if (!isfinite(q)) q = q1 - (tid == 0 ? 0.0 : before);
    }
    if (tid < n) ddt[row_off(ba.sddt, b, h, t0 + tid)] = float(A[h] * q + xu);
    const double sA = warp_sum(double(dts[tid]) * q), sD = warp_sum(tid < n ? double(dg[tid]) : 0.0);
    if (tid == 0) {
      w.dAD[size_t(blockIdx.x) * 2] = sA;
      w.dAD[size_t(blockIdx.x) * 2 + 1] = sD;
    }
  }
}

// dB, dC [B][G][T][N] from the per-head parts, heads in order; 4 columns a thread.
template <typename Tin>
__global__ void __launch_bounds__(256)
k_ssm_fold(SsmBwdArgs ba, const float* __restrict__ pB, const float* __restrict__ pC,
           Tin* __restrict__ dB, Tin* __restrict__ dC) {
  wait_for_previous();
  const SsmArgs& a = ba.a;
  const int nn4 = a.N >> 2;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)a.B * a.G * a.T * nn4) return;
  const int e = int(i % nn4) * 4;
  const long long r = i / nn4;
  const int t = int(r % a.T);
  const int bg = int(r / a.T), b = bg / a.G, g = bg - b * a.G;
  const float* src = blockIdx.y ? pC : pB;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < a.hg; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(
        src + ((size_t(b) * a.H + g * a.hg + k) * a.T + t) * a.N + e);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  Tin* o = blockIdx.y ? dC + row_off(ba.sdC, b, g, t) + e : dB + row_off(ba.sdB, b, g, t) + e;
  o[0] = from_f32<Tin>(s.x); o[1] = from_f32<Tin>(s.y);
  o[2] = from_f32<Tin>(s.z); o[3] = from_f32<Tin>(s.w);
}

// dA, dD: a CTA per head sums its batches' and chunks' parts in a fixed order.
__global__ void __launch_bounds__(256)
k_ssm_dAD(const double* __restrict__ part, int B, int H, int nch, float* __restrict__ dA,
          float* __restrict__ dD) {
  wait_for_previous();
  __shared__ double rA[8], rD[8];
  const int h = blockIdx.x, n = B * nch;
  double sA = 0.0, sD = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int b = i / nch, c = i - b * nch;
    const double2 v = *reinterpret_cast<const double2*>(part + ((size_t(b) * H + h) * nch + c) * 2);
    sA += v.x;
    sD += v.y;
  }
  sA = warp_sum(sA);
  sD = warp_sum(sD);
  if ((threadIdx.x & 31) == 0) {
    rA[threadIdx.x >> 5] = sA;
    rD[threadIdx.x >> 5] = sD;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 8; ++k) {
      sA += rA[k];
      sD += rD[k];
    }
    dA[h] = float(sA);
    if (dD) dD[h] = float(sD);
  }
}

template <typename Tin>
static cudaError_t launch_ssm_bwd_simt(const SsmBwdArgs& ba, const void* x, const float* dt,
                                       const float* A, const void* Bm, const void* Cm,
                                       const float* D, const float* S0, const void* dy,
                                       const float* dST, const SsmBwdWs& w, void* dx, float* ddt,
                                       void* dB, void* dC, float* dS0, cudaStream_t s) {
  const SsmArgs& a = ba.a;
  const unsigned grid = unsigned(a.B * a.H) * unsigned(a.nch);
  const int s1 = int(4 * (2 * kSsmQ * a.P + 2 * kSsmQ * a.N + 3 * kSsmQ));
  const int s2 = int(ssm_bwd_smem(a.P, a.N));
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_ssm_local<Tin>, cudaFuncAttributeMaxDynamicSharedMemorySize, s1)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(k_ssm_bwd<Tin>, cudaFuncAttributeMaxDynamicSharedMemorySize, s2)) != cudaSuccess)
    return e;
  launch_after(k_ssm_local<Tin>, grid, kBwdThreads, s1, s, a, (const Tin*)x, dt, A, (const Tin*)Bm,
                                                 (const Tin*)Cm, (const Tin*)dy, w.fS, w.gS, w.lg);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int BH = a.B * a.H, PN = a.P * a.N;
  if ((e = launch_ssm_carries(w.fS, w.gS, w.lg, S0, w.ST, dST, dS0, BH, a.nch, PN, s)) != cudaSuccess) return e;
  launch_after(k_ssm_bwd<Tin>, grid, kBwdThreads, s2, s, ba, (const Tin*)x, dt, A, (const Tin*)Bm,
                                               (const Tin*)Cm, D, (const Tin*)dy, w, (Tin*)dx, ddt,
                                               (Tin*)dB, (Tin*)dC);
  return cudaGetLastError();
}

template <typename Tin>
static cudaError_t launch_ssm_fold(const SsmBwdArgs& ba, const SsmBwdWs& w, void* dB, void* dC,
                                   cudaStream_t s) {
  const SsmArgs& a = ba.a;
  if (a.hg == 1) return cudaSuccess;
  const long long n = (long long)a.B * a.G * a.T * (a.N / 4);
  launch_after(k_ssm_fold<Tin>, dim3(unsigned((n + 255) / 256), 2), 256, 0, s, ba, w.pB, w.pC, (Tin*)dB, (Tin*)dC);
  return cudaGetLastError();
}

}  // namespace sdm

using namespace sdm;

static long long ssm_bwd_grid(const sdm_ssm_dims* d) {
  return (long long)d->B * d->H * ((d->T + kSsmQ - 1) / kSsmQ);
}

extern "C" size_t sdm_ssm_backward_workspace_bytes(const sdm_ssm_dims* dims) {
  if (ssm_check(dims) != SDM_OK || ssm_bwd_grid(dims) >= (1LL << 31)) return 0;
  size_t n = ssm_bwd_ws(dims, kSsmQ, nullptr).total;  // the shorter chunks need more
  return n > 0 ? n : 16;
}

extern "C" int sdm_ssm_backward(const void* x, const float* dt, const float* A, const void* Bm,
                                const void* Cm, const float* D, const float* S0, const void* dy,
                                const float* dS_T, void* dx, float* ddt, float* dA, void* dB,
                                void* dC, float* dD, float* dS0, const sdm_ssm_dims* dims,
                                const sdm_ssm_views* views, const sdm_ssm_views* grad_views,
                                void* workspace, size_t ws_bytes, void* stream) {
  int rc = ssm_check(dims);
  if (rc != SDM_OK) return rc;
  if (dims->T == 0) return SDM_ERR_DIMS;  // there is no step to differentiate
  if (ssm_bwd_grid(dims) >= (1LL << 31)) return SDM_ERR_UNSUPPORTED;
  if ((rc = ssm_views_ok(views)) != SDM_OK || (rc = ssm_views_ok(grad_views)) != SDM_OK) return rc;
  if ((rc = ssm_ptrs(dims, x, dt, A, Bm, Cm, D)) != SDM_OK) return rc;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  for (const void* p : {dy, static_cast<const void*>(dx), static_cast<const void*>(dB), static_cast<const void*>(dC)})
    if ((rc = need_ptr(p, es)) != SDM_OK) return rc;
  for (const void* p : {static_cast<const void*>(ddt), static_cast<const void*>(dA)})
    if ((rc = need_ptr(p, 4)) != SDM_OK) return rc;
  if (!aligned_to(dD, 4) || !aligned_to(S0, 16) || !aligned_to(dS_T, 16) || !aligned_to(dS0, 16))
    return SDM_ERR_ALIGN;
  if (!workspace || ws_bytes < sdm_ssm_backward_workspace_bytes(dims)) return SDM_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return SDM_ERR_ALIGN;
  SsmBwdArgs ba;
  ba.a = ssm_args(dims, views);
  ba.sdx = grad_views->x; ba.sddt = grad_views->dt; ba.sdB = grad_views->B; ba.sdC = grad_views->C;
  const bool bf = dims->in_dtype == SDM_DTYPE_BF16;
  const bool mma = ssm_tensor_sizes(dims) && view_aligned(x, ba.a.sx, 2, 16) &&
                   view_aligned(Bm, ba.a.sB, 2, 16) && view_aligned(Cm, ba.a.sC, 2, 16) &&
                   view_aligned(dy, ba.a.sy, 2, 16) && view_aligned(dx, ba.sdx, 2, 4) &&
                   view_aligned(dB, ba.sdB, 2, 4) && view_aligned(dC, ba.sdC, 2, 4);
  ba.a.Q = mma ? kSsmQT : kSsmQ;
  ba.a.nch = (dims->T + ba.a.Q - 1) / ba.a.Q;
  const SsmBwdWs w = ssm_bwd_ws(dims, ba.a.Q, workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = mma ? launch_ssm_bwd_mma(ba, x, dt, A, Bm, Cm, D, S0, dy, dS_T, w, dx, ddt, dB, dC, dS0, s)
                : bf ? launch_ssm_bwd_simt<__nv_bfloat16>(ba, x, dt, A, Bm, Cm, D, S0, dy, dS_T, w, dx, ddt, dB, dC, dS0, s)
                     : launch_ssm_bwd_simt<float>(ba, x, dt, A, Bm, Cm, D, S0, dy, dS_T, w, dx, ddt, dB, dC, dS0, s);
  if (e == cudaSuccess)
    e = bf ? launch_ssm_fold<__nv_bfloat16>(ba, w, dB, dC, s) : launch_ssm_fold<float>(ba, w, dB, dC, s);
  if (e == cudaSuccess) {
    launch_after(k_ssm_dAD, dims->H, 256, 0, s, w.dAD, dims->B, dims->H, ba.a.nch, dA, dD);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
