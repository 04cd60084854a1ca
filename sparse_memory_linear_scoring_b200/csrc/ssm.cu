// ssm.cu -- the selective state space scan: CUDA-core chunk kernels, the
// single-token kernel, the carry between segments, and the C ABI of the forward
// pass.  ssm_internal.cuh has the formulas.
//
// The chunks of a head follow one another, so a call with few heads would leave
// most SMs idle.  The time axis is cut into segments of whole chunks: a first
// pass gets each segment's own contribution to the state (k_ssm_walk without
// outputs), k_ssm_carry chains them, and the second pass walks all segments at
// once from their true states.  With enough heads to fill the card there is one
// segment and one pass.
#include <utility>

#include "ssm_internal.cuh"

namespace sdm {

// ---------------------------------------------------------------- carry
// Forward: segS[i] := state before segment i, S_end := the last state.
// Reverse: segS[i] := gradient arriving at the end of segment i (from S0, the
// gradient of the last state, or 0), S_end := gradient of the first state.
struct Carry {
  float* segS;
  const float* S0;
  float* S_end;
  int reverse;
};

__global__ void __launch_bounds__(128)
k_ssm_carry(Carry c0, Carry c1, const float* __restrict__ segG, int nseg, int PN) {
  wait_for_previous();
  const Carry c = blockIdx.z ? c1 : c0;
  const int bh = blockIdx.y;
  const int e = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (e >= PN) return;
  float4 S = c.S0 ? *reinterpret_cast<const float4*>(c.S0 + (size_t)bh * PN + e)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
  float* p = c.segS + (size_t)bh * nseg * PN + e;
  const float* g = segG + (size_t)bh * nseg;
  constexpr int U = 8;  // segments whose loads are in flight together
  for (int i0 = 0; i0 < nseg; i0 += U) {
    float4 v[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u < nseg) {
        const int i = c.reverse ? nseg - 1 - (i0 + u) : i0 + u;
        v[u] = *reinterpret_cast<const float4*>(p + (size_t)i * PN);
        d[u] = g[i];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u < nseg) {
        const int i = c.reverse ? nseg - 1 - (i0 + u) : i0 + u;
        *reinterpret_cast<float4*>(p + (size_t)i * PN) = S;
        const float a = exp2f(d[u]);
        S.x = fmaf(a, S.x, v[u].x); S.y = fmaf(a, S.y, v[u].y);
        S.z = fmaf(a, S.z, v[u].z); S.w = fmaf(a, S.w, v[u].w);
      }
    }
  }
  if (c.S_end) *reinterpret_cast<float4*>(c.S_end + (size_t)bh * PN + e) = S;
}

static cudaError_t launch_carry(const Carry& c0, const Carry& c1, int both, const float* segG, int BH,
                                int nseg, int PN, cudaStream_t s) {
  for (int b0 = 0; b0 < BH; b0 += 65535) {  // the grid's y axis ends at 65535
    const int n = BH - b0 < 65535 ? BH - b0 : 65535;
    const size_t o = size_t(b0) * PN;
    auto at = [&](const Carry& c) {
      return Carry{c.segS + o * nseg, c.S0 ? c.S0 + o : nullptr, c.S_end ? c.S_end + o : nullptr, c.reverse};
    };
    launch_after(k_ssm_carry, dim3((PN / 4 + 127) / 128, n, both ? 2 : 1), 128, 0, s,
        at(c0), at(c1), segG + size_t(b0) * nseg, nseg, PN);
  }
  return cudaGetLastError();
}

cudaError_t launch_ssm_carry(float* segS, const float* segG, const float* S0, float* S_end, int BH,
                             int nseg, int PN, cudaStream_t s) {
  const Carry c = {segS, S0, S_end, 0};
  return launch_carry(c, c, 0, segG, BH, nseg, PN, s);
}

cudaError_t launch_ssm_carries(float* fS, float* gS, const float* lg, const float* S0, float* ST,
                               const float* dST, float* dS0, int BH, int nch, int PN, cudaStream_t s) {
  return launch_carry({fS, S0, ST, 0}, {gS, dST, dS0, 1}, 1, lg, BH, nch, PN, s);
}

// ---------------------------------------------------------------- CUDA-core walk
// A CTA walks one segment of one head, S in shared memory; float32 throughout
// (fused multiply-adds on 4 x 4 register tiles).  It serves float32 inputs, where
// three-way splits on the tensor cores would cost as much, and bf16 sizes or
// alignments the tensor-core walk does not take.
constexpr int kWalkThreads = 256;

__host__ __device__ inline size_t ssm_walk_smem(int P, int N) {
  // x [Q][P], B, C [Q][N + 1], M [Q][Q + 1], S [P][N + 1], dt, hi, lo, w [Q]
  return size_t(4) * (kSsmQ * P + 2 * kSsmQ * (N + 1) + kSsmQ * (kSsmQ + 1) + P * (N + 1) + 4 * kSsmQ);
}

template <typename Tin, bool OUT>
__global__ void __launch_bounds__(kWalkThreads)
k_ssm_walk(SsmArgs a, const Tin* __restrict__ x, const float* __restrict__ dt,
           const float* __restrict__ A, const Tin* __restrict__ Bm, const Tin* __restrict__ Cm,
           const float* __restrict__ D, float* __restrict__ S, const int32_t* __restrict__ lengths,
           Tin* __restrict__ y, float* __restrict__ segS, float* __restrict__ segG) {
  wait_for_previous();
  extern __shared__ __align__(16) float sm[];
  constexpr int Q = kSsmQ;
  const int P = a.P, N = a.N, Np = N + 1, Qp = Q + 1;
  float* xs = sm;
  float* Bs = xs + Q * P;
  float* Cs = Bs + Q * Np;
  float* Ms = Cs + Q * Np;
  float* Ss = Ms + Q * Qp;
  float* dts = Ss + P * Np;
  float* hi = dts + Q;
  float* lo = hi + Q;
  float* wj = lo + Q;
  const int tid = threadIdx.x;
  const int seg = blockIdx.x % a.nseg, bh = blockIdx.x / a.nseg;
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  const int L = seq_len(lengths, b, a.T);
  const float Ah = A[h], Dh = D ? D[h] : 0.f;
  const size_t PN = size_t(P) * N;
  float* slot = a.nseg > 1 ? segS + size_t(blockIdx.x) * PN : S + size_t(bh) * PN;
  for (int i = tid; i < P * N; i += kWalkThreads) Ss[(i / N) * Np + i % N] = OUT ? slot[i] : 0.f;
  const int c0 = seg * a.cps, c1 = min(c0 + a.cps, a.nch);
  float tot = 0.f;
  const int np4 = P >> 2, nn4 = N >> 2;
  for (int c = c0; c < c1; ++c) {
    const int t0 = c * Q;
    const int n = max(0, min(Q, L - t0));  // live steps; the rest count as dt = 0
    __syncthreads();
    for (int i = tid; i < Q * P; i += kWalkThreads) {
      const int t = i / P, p = i - t * P;
      xs[i] = t < n ? to_f32(x[row_off(a.sx, b, h, t0 + t) + p]) : 0.f;
    }
    for (int i = tid; i < Q * N; i += kWalkThreads) {
      const int t = i / N, e = i - t * N;
      Bs[t * Np + e] = t < n ? to_f32(Bm[row_off(a.sB, b, gr, t0 + t) + e]) : 0.f;
      if (OUT) Cs[t * Np + e] = t < n ? to_f32(Cm[row_off(a.sC, b, gr, t0 + t) + e]) : 0.f;
    }
    if (tid < Q) dts[tid] = tid < n ? dt[row_off(a.sdt, b, h, t0 + tid)] : 0.f;
    __syncthreads();
    if (tid < 32) {
      chunk_decay<1>(dts, Ah, hi, lo);
      __syncwarp();
      wj[tid] = decay_between(hi[Q - 1], lo[Q - 1], hi[tid], lo[tid]) * dts[tid];
    }
    __syncthreads();
    const float gq = hi[Q - 1] + lo[Q - 1];
    tot += gq;
    if (OUT) {
      // M_tj = exp(g_t - g_j) dt_j (C_t . B_j), one 2 x 2 tile a thread
      {
        const int t = (tid >> 4) * 2, j = (tid & 15) * 2;
        float s[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
        if (j <= t + 1)
          for (int e = 0; e < N; ++e) {
            const float c0_ = Cs[t * Np + e], c1_ = Cs[(t + 1) * Np + e];
            const float b0_ = Bs[j * Np + e], b1_ = Bs[(j + 1) * Np + e];
            s[0][0] = fmaf(c0_, b0_, s[0][0]); s[0][1] = fmaf(c0_, b1_, s[0][1]);
            s[1][0] = fmaf(c1_, b0_, s[1][0]); s[1][1] = fmaf(c1_, b1_, s[1][1]);
          }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            Ms[(t + u) * Qp + j + v] =
                j + v <= t + u ? decay_between(hi[t + u], lo[t + u], hi[j + v], lo[j + v]) *
                                     dts[j + v] * s[u][v]
                               : 0.f;
      }
      __syncthreads();
      for (int tile = tid; tile < (Q >> 2) * np4; tile += kWalkThreads) {
        const int t = (tile / np4) * 4, p = (tile % np4) * 4;
        float acc[4][4] = {};
        for (int e = 0; e < N; ++e) {
          float cv[4], sv[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            cv[u] = Cs[(t + u) * Np + e];
            sv[u] = Ss[(p + u) * Np + e];
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(cv[u], sv[v], acc[u][v]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float eg = ex2(hi[t + u] + lo[t + u]);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[u][v] *= eg;
        }
        for (int j = 0; j < t; ++j) {
          float mv[4], xv[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            mv[u] = Ms[(t + u) * Qp + j];
            xv[u] = xs[j * P + p + u];
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(mv[u], xv[v], acc[u][v]);
        }
#pragma unroll
        for (int z = 0; z < 4; ++z)  // the diagonal: a later x may be NaN, and 0 NaN is not 0
#pragma unroll
          for (int u = z; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[u][v] = fmaf(Ms[(t + u) * Qp + t + z], xs[(t + z) * P + p + v], acc[u][v]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (t0 + t + u >= a.T) break;
          Tin* yp = y + row_off(a.sy, b, h, t0 + t + u) + p;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            yp[v] = from_f32<Tin>(t + u < n ? fmaf(Dh, xs[(t + u) * P + p + v], acc[u][v]) : 0.f);
        }
      }
      __syncthreads();
    }
    const float eq = ex2(gq);
    for (int tile = tid; tile < np4 * nn4; tile += kWalkThreads) {
      const int p = (tile / nn4) * 4, e = (tile % nn4) * 4;
      float acc[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = eq * Ss[(p + u) * Np + e + v];
      for (int j = 0; j < n; ++j) {
        const float w = wj[j];
        float xv[4], bv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          xv[u] = w * xs[j * P + p + u];
          bv[u] = Bs[j * Np + e + u];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(xv[u], bv[v], acc[u][v]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) Ss[(p + u) * Np + e + v] = acc[u][v];
    }
  }
  __syncthreads();
  if (!OUT) {
    for (int i = tid; i < P * N; i += kWalkThreads) slot[i] = Ss[(i / N) * Np + i % N];
    if (tid == 0) segG[blockIdx.x] = tot;
  } else if (seg == a.nseg - 1) {
    for (int i = tid; i < P * N; i += kWalkThreads) S[size_t(bh) * PN + i] = Ss[(i / N) * Np + i % N];
  }
}

// ---------------------------------------------------------------- single tokens
// S is read and written once: 8 P N bytes a head against 5 P N flops.  A row of S
// lies across N / 4 lanes as float4; a thread holds R rows of its columns, so 4
// 16-byte loads are in flight, and walks the call's few steps with them.
constexpr int kStepRows = 4;
constexpr int kStepThreads = 128;

template <typename Tin>
__global__ void __launch_bounds__(kStepThreads)
k_ssm_step(SsmArgs a, const Tin* __restrict__ x, const float* __restrict__ dt,
           const float* __restrict__ A, const Tin* __restrict__ Bm, const Tin* __restrict__ Cm,
           const float* __restrict__ D, float* __restrict__ S, Tin* __restrict__ y, int tiles) {
  wait_for_previous();
  const int bh = blockIdx.x / tiles, tile = blockIdx.x - bh * tiles;
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  const int ln = a.N >> 2;  // lanes per row (4..32)
  const int lane = threadIdx.x % ln, grp = threadIdx.x / ln;
  const int r0 = (tile * (kStepThreads / ln) + grp) * kStepRows;
  float4 s[kStepRows];
  float* Sp = S + (size_t(bh) * a.P + r0) * a.N + lane * 4;
#pragma unroll
  for (int r = 0; r < kStepRows; ++r)
    s[r] = r0 + r < a.P ? *reinterpret_cast<const float4*>(Sp + r * a.N)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  const float Ah = A[h], Dh = D ? D[h] : 0.f;
  for (int t = 0; t < a.T; ++t) {
    const float d = dt[row_off(a.sdt, b, h, t)];
    const float g = d * Ah, e = expf(g);
    const float da = e == 0.f ? 0.f : fmaf(e, fmaf(d, Ah, -g), e);  // exp of the unrounded product
    const Tin* bp = Bm + row_off(a.sB, b, gr, t) + lane * 4;
    const Tin* cp = Cm + row_off(a.sC, b, gr, t) + lane * 4;
    float bv[4], cv[4], xv[kStepRows];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bv[e] = to_f32(bp[e]);
      cv[e] = to_f32(cp[e]);
    }
    const Tin* xp = x + row_off(a.sx, b, h, t) + r0;
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) xv[r] = r0 + r < a.P ? to_f32(xp[r]) : 0.f;
    float o[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
      const float u = d * xv[r];
      s[r].x = fmaf(da, s[r].x, u * bv[0]); s[r].y = fmaf(da, s[r].y, u * bv[1]);
      s[r].z = fmaf(da, s[r].z, u * bv[2]); s[r].w = fmaf(da, s[r].w, u * bv[3]);
      o[r] = fmaf(s[r].x, cv[0], s[r].y * cv[1]) + fmaf(s[r].z, cv[2], s[r].w * cv[3]);
    }
    for (int q = ln >> 1; q > 0; q >>= 1)
#pragma unroll
      for (int r = 0; r < kStepRows; ++r) o[r] += __shfl_xor_sync(0xffffffffu, o[r], q);
    if (lane == 0) {
      Tin* yp = y + row_off(a.sy, b, h, t) + r0;
#pragma unroll
      for (int r = 0; r < kStepRows; ++r)
        if (r0 + r < a.P) yp[r] = from_f32<Tin>(fmaf(Dh, xv[r], o[r]));
    }
  }
#pragma unroll
  for (int r = 0; r < kStepRows; ++r)
    if (r0 + r < a.P) *reinterpret_cast<float4*>(Sp + r * a.N) = s[r];
}

// ---------------------------------------------------------------- host side
int ssm_check(const sdm_ssm_dims* d) {
  if (!d) return SDM_ERR_NULL;
  if (d->B < 1 || d->H < 1 || d->G < 1 || d->H % d->G != 0 || d->T < 0 || d->T > (1 << 30) ||
      d->d_v < 1 || d->d_k < 1 ||
      (d->in_dtype != SDM_DTYPE_F32 && d->in_dtype != SDM_DTYPE_BF16))
    return SDM_ERR_DIMS;
  if ((long long)d->B * d->H > (1 << 24) || (long long)d->B * d->H * (long long)d->T > (1LL << 40))
    return SDM_ERR_DIMS;
  auto ok = [](int x) { return x == 16 || x == 32 || x == 64 || x == 128; };
  if (!ok(d->d_v) || !ok(d->d_k)) return SDM_ERR_UNSUPPORTED;
  return SDM_OK;
}

// Segments: enough that (head, segment) pairs fill the card twice over, but few enough
// that the carry, about 0.1 us a segment of a head, stays below the two walks of 2 to 5 us
// a chunk: 2 c nch / nseg + 0.1 nseg is least near nseg = 8 sqrt(nch).  (At least 4 chunks
// a segment, as a rule on the states' bytes would have it, cost 777 steps of 3 float32
// heads 57 us in the walks instead of 16.)
static void ssm_segments(const sdm_ssm_dims* d, int Q, SsmArgs* a) {
  a->Q = Q;
  a->nch = (d->T + Q - 1) / Q;
  const long long BH = (long long)d->B * d->H * (Q == kSsmQT ? (d->d_v + 63) / 64 : 1);  // walks of a segment
  long long nseg = 2 * 148 / BH;
  while (nseg > 1 && nseg * nseg > 64LL * a->nch) --nseg;
  if (nseg > a->nch) nseg = a->nch;
  if (nseg < 1) nseg = 1;
  a->cps = int((a->nch + nseg - 1) / nseg);
  if (a->cps < 1) a->cps = 1;
  a->nseg = (a->nch + a->cps - 1) / a->cps;
  if (a->nseg < 1) a->nseg = 1;
}

SsmArgs ssm_args(const sdm_ssm_dims* d, const sdm_ssm_views* v) {
  SsmArgs a;
  memset(&a, 0, sizeof(a));
  a.B = d->B; a.H = d->H; a.G = d->G; a.T = d->T; a.P = d->d_v; a.N = d->d_k;
  a.hg = d->H / d->G;
  a.sx = v->x; a.sdt = v->dt; a.sB = v->B; a.sC = v->C; a.sy = v->y;
  return a;
}

int ssm_views_ok(const sdm_ssm_views* v) {
  if (!v) return SDM_ERR_NULL;
  for (const sdm_strides* p : {&v->x, &v->dt, &v->B, &v->C, &v->y})
    if (!strides_ok(p)) return SDM_ERR_DIMS;
  return SDM_OK;
}

template <typename Tin>
static cudaError_t launch_ssm_fwd_simt(const SsmArgs& a, const void* x, const float* dt,
                                       const float* A, const void* Bm, const void* Cm,
                                       const float* D, float* S, const int32_t* lengths, void* y,
                                       float* segS, float* segG, cudaStream_t s) {
  const int smem = int(ssm_walk_smem(a.P, a.N));
  const unsigned grid = unsigned(a.B * a.H) * unsigned(a.nseg);
  cudaError_t e;
  if (a.nseg > 1) {
    if ((e = cudaFuncSetAttribute(k_ssm_walk<Tin, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  smem)) != cudaSuccess)
      return e;
    launch_after(k_ssm_walk<Tin, false>, grid, kWalkThreads, smem, s,
        a, (const Tin*)x, dt, A, (const Tin*)Bm, (const Tin*)Cm, D, S, lengths, (Tin*)y, segS, segG);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_ssm_carry(segS, segG, S, nullptr, a.B * a.H, a.nseg, a.P * a.N, s)) !=
        cudaSuccess)
      return e;
  }
  if ((e = cudaFuncSetAttribute(k_ssm_walk<Tin, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem)) != cudaSuccess)
    return e;
  launch_after(k_ssm_walk<Tin, true>, grid, kWalkThreads, smem, s,
      a, (const Tin*)x, dt, A, (const Tin*)Bm, (const Tin*)Cm, D, S, lengths, (Tin*)y, segS, segG);
  return cudaGetLastError();
}

}  // namespace sdm

using namespace sdm;

int sdm::ssm_ptrs(const sdm_ssm_dims* d, const void* x, const float* dt, const float* A,
                    const void* Bm, const void* Cm, const float* D) {
  const size_t es = d->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  int rc;
  for (const void* p : {x, Bm, Cm})
    if ((rc = need_ptr(p, es)) != SDM_OK) return rc;
  for (const float* p : {dt, A})
    if ((rc = need_ptr(p, 4)) != SDM_OK) return rc;
  return aligned_to(D, 4) ? SDM_OK : SDM_ERR_ALIGN;
}

extern "C" size_t sdm_ssm_workspace_bytes(const sdm_ssm_dims* dims) {
  if (ssm_check(dims) != SDM_OK) return 0;
  size_t most = 16;
  for (int Q : {kSsmQ, kSsmQT}) {  // either chunk length may be taken
    SsmArgs a;
    ssm_segments(dims, Q, &a);
    if (a.nseg > 1) {
      const size_t n = size_t(dims->B) * dims->H * a.nseg *
                       (size_t(dims->d_v) * dims->d_k + 4) * 4;
      if (n > most) most = n;
    }
  }
  return most;
}

extern "C" int sdm_ssm_forward(const void* x, const float* dt, const float* A, const void* Bm,
                               const void* Cm, const float* D, float* S_inout,
                               const int32_t* lengths, void* y, const sdm_ssm_dims* dims,
                               const sdm_ssm_views* views, void* workspace, size_t ws_bytes,
                               void* stream) {
  int rc = ssm_check(dims);
  if (rc != SDM_OK) return rc;
  if (dims->T == 0) return SDM_OK;
  if ((rc = ssm_views_ok(views)) != SDM_OK) return rc;
  if ((rc = ssm_ptrs(dims, x, dt, A, Bm, Cm, D)) != SDM_OK) return rc;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  if ((rc = need_ptr(S_inout, 16)) != SDM_OK || (rc = need_ptr(y, es)) != SDM_OK) return rc;
  if (!aligned_to(lengths, 4)) return SDM_ERR_ALIGN;
  if (!workspace || ws_bytes < sdm_ssm_workspace_bytes(dims)) return SDM_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return SDM_ERR_ALIGN;
  SsmArgs a = ssm_args(dims, views);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool mma = ssm_tensor_sizes(dims) && view_aligned(x, a.sx, 2, 16) &&
                   view_aligned(Bm, a.sB, 2, 16) && view_aligned(Cm, a.sC, 2, 16) &&
                   view_aligned(y, a.sy, 2, 16);
  ssm_segments(dims, mma ? kSsmQT : kSsmQ, &a);
  float* segS = static_cast<float*>(workspace);
  float* segG = segS + size_t(a.B) * a.H * a.nseg * a.P * a.N;
  cudaError_t e;
  if (mma)
    e = launch_ssm_fwd_mma(a, x, dt, A, Bm, Cm, D, S_inout, lengths, y, segS, segG, s);
  else if (dims->in_dtype == SDM_DTYPE_BF16)
    e = launch_ssm_fwd_simt<__nv_bfloat16>(a, x, dt, A, Bm, Cm, D, S_inout, lengths, y, segS, segG, s);
  else
    e = launch_ssm_fwd_simt<float>(a, x, dt, A, Bm, Cm, D, S_inout, lengths, y, segS, segG, s);
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" int sdm_ssm_step(const void* x, const float* dt, const float* A, const void* Bm,
                            const void* Cm, const float* D, float* S_inout, void* y,
                            const sdm_ssm_dims* dims, const sdm_ssm_views* views, void* stream) {
  int rc = ssm_check(dims);
  if (rc != SDM_OK) return rc;
  if (dims->T == 0) return SDM_OK;
  if ((rc = ssm_views_ok(views)) != SDM_OK) return rc;
  if ((rc = ssm_ptrs(dims, x, dt, A, Bm, Cm, D)) != SDM_OK) return rc;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  if ((rc = need_ptr(S_inout, 16)) != SDM_OK || (rc = need_ptr(y, es)) != SDM_OK) return rc;
  const SsmArgs a = ssm_args(dims, views);
  const int rows = kStepThreads / (a.N / 4) * kStepRows;
  const int tiles = (a.P + rows - 1) / rows;
  const unsigned grid = unsigned(a.B * a.H) * unsigned(tiles);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->in_dtype == SDM_DTYPE_BF16)
    launch_after(k_ssm_step<__nv_bfloat16>, grid, kStepThreads, 0, s,
        a, (const __nv_bfloat16*)x, dt, A, (const __nv_bfloat16*)Bm, (const __nv_bfloat16*)Cm, D,
        S_inout, (__nv_bfloat16*)y, tiles);
  else
    launch_after(k_ssm_step<float>, grid, kStepThreads, 0, s, a, (const float*)x, dt, A, (const float*)Bm,
                                                    (const float*)Cm, D, S_inout, (float*)y, tiles);
  return cudaGetLastError() == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
