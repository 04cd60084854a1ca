// conv.cu -- short causal convolution along the sequence, one filter per channel,
// with SiLU or without, the last K - 1 inputs carried as state.
//
//   p_t = bias + sum_{i<K} w_i x_{t-K+1+i},   y = p  or  p sigmoid(p),
//   dp = dy silu'(p),  dx_t = sum_i w_i dp_{t+K-1-i},  dw_i = sum_t dp_t x_{t-K+1+i}.
//
// Both directions move bytes and little else, but not by much: 2K + 5 flops and two
// special functions an element against 4 bytes in bf16, so a plain division (about 10
// instructions) for the sigmoid would bound them.  A thread keeps the window of the
// last K - 1 inputs of 4 neighbouring channels (2 in the float32 backward, where the
// filter, its gradient and two windows share the registers) and walks a tile of steps,
// the next rows (8 forward, 4 backward) on their way while one group is computed, two
// multiply-adds to an instruction.  Every input is read once from DRAM, plus K - 1 rows a
// tile that its neighbour has brought into L2.  65536 steps of 1280 bf16 channels: forward
// 70 us (336 MB, 4.8 TB/s), backward 143 us (503 MB, 3.5 TB/s).  Memory latency bounds both:
// 14 to 17 warps an SM, which their registers leave, mostly wait for loads, with issue slots
// 47% and DRAM 55% and 43% busy.  float32: 109 us forward (6.1 TB/s), 350 both directions.
// 16-byte threads without rows ahead and with plain divisions took 208 and 660 (bf16).
#include "seq_internal.cuh"

namespace sdm {

struct ConvArgs {
  int B, H, T, d, tt, ntile, wvec;
  sdm_strides sx, sy;
};

// s = 1 / (1 + exp(-p)) and c = 1 - s on the special function unit; s is 0 below
// p = -87.3, where it is less than 2^-126.  The rounding of p log2 e moves exp by |p| 2^-24
// of itself, which beside bf16 results (2^-9) does not count.  For float32 its remainder is
// carried into exp (2^-21 of s wherever p lies), and c is exp(-p) s where 1 - s would
// keep only s's last bits.
template <typename T>
__device__ __forceinline__ void sigmoid(float p, float& s, float& c) {
  const float x = p * -kLog2e;
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  if (sizeof(T) == 4 && fabsf(p) < 128.f) {
    const float rest = fmaf(p, -kLog2e, -x) + p * -1.9259629911e-8f;  // log2 e is kLog2e + 1.93e-8
    e = fmaf(e, rest * 0.69314718056f, e);
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  c = sizeof(T) == 4 && p > 0.f ? e * s : 1.f - s;
}

// acc += a * b over V channels, two to an instruction.
template <int V>
__device__ __forceinline__ void fma_row(float (&acc)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int c = 0; c < V; c += 2)
      asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
          "mov.b64 z, {%0, %1};\n\tfma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
          : "+f"(acc[c]), "+f"(acc[c + 1]) : "f"(a[c]), "f"(a[c + 1]), "f"(b[c]), "f"(b[c + 1]));
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = fmaf(a[c], b[c], acc[c]);
  }
}

// V elements as they lie in memory.
template <typename T, int V>
struct Raw {
  uint32_t u[(V * sizeof(T) + 3) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V * sizeof(T) == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
    } else if constexpr (V * sizeof(T) == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      u[0] = v.x; u[1] = v.y;
    } else if constexpr (V * sizeof(T) == 4) {
      u[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      u[0] = *reinterpret_cast<const unsigned short*>(p);
    }
  }
  __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if constexpr (sizeof(T) == 4) f[c] = __uint_as_float(u[c]);
      else f[c] = __uint_as_float((c & 1) ? u[c / 2] & 0xffff0000u : u[c / 2] << 16);
    }
  }
};

// The filters of V neighbouring channels: V * K consecutive elements.
template <typename T, int V, int K>
__device__ __forceinline__ void load_taps(const T* wp, bool vec, float (&wf)[K][V]) {
  float f[K * V];
  if (vec) {
#pragma unroll
    for (int k = 0; k < K; ++k) Vec<T, V>::load(wp + k * V, f + k * V);
  } else {
#pragma unroll
    for (int i = 0; i < K * V; ++i) f[i] = to_f32(wp[i]);
  }
#pragma unroll
  for (int c = 0; c < V; ++c)
#pragma unroll
    for (int k = 0; k < K; ++k) wf[k][c] = f[c * K + k];
}

// One thread: V channels, tt steps.  The thread of tile 0 alone reads and then
// replaces the state of its channels, so the update in place has no race.
template <typename T, int V, int K, bool SILU>
__global__ void __launch_bounds__(128)
k_conv_fwd(ConvArgs a, const T* __restrict__ x, const T* __restrict__ w, const T* __restrict__ bias,
           T* state, const int32_t* __restrict__ lengths, T* __restrict__ y) {
  wait_for_previous();
  const int nv = a.d / V;
  long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long per_b = (long long)a.ntile * a.H * nv;
  if (i >= per_b * a.B) return;
  const int b = int(i / per_b);
  i -= b * per_b;
  const int tile = int(i / (a.H * nv));
  const int hv = int(i - (long long)tile * (a.H * nv));
  const int h = hv / nv, c0 = (hv - h * nv) * V;
  const int L = seq_len(lengths, b, a.T);
  const int t0 = tile * a.tt, t1 = min(t0 + a.tt, a.T);
  constexpr int U = 8;  // rows whose loads are in flight together
  float wf[K][V], bf[V], win[K - 1 + U][V];
  load_taps<T, V, K>(w + ((long long)h * a.d + c0) * K, a.wvec, wf);
#pragma unroll
  for (int c = 0; c < V; ++c) bf[c] = bias ? to_f32(bias[(long long)h * a.d + c0 + c]) : 0.f;
  const T* xp = x + row_off(a.sx, b, h, 0) + c0;
  T* yp = y + row_off(a.sy, b, h, 0) + c0;
  T* sp = state ? state + (((long long)b * a.H + h) * (K - 1)) * a.d + c0 : nullptr;
#pragma unroll
  for (int k = 0; k < K - 1; ++k) {
    const int t = t0 - (K - 1) + k;
    if (t >= 0 && t < L) {
      Vec<T, V>::load(xp + t * a.sx.t, win[k]);
    } else if (t < 0 && sp) {
      Vec<T, V>::load(sp + (long long)(t + K - 1) * a.d, win[k]);
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) win[k][c] = 0.f;
    }
  }
  const int te = min(t1, L);
  auto step = [&](int u, T* to) {  // win[u + K - 1] is the step's own input
    float p[V];
#pragma unroll
    for (int c = 0; c < V; ++c) p[c] = bf[c];
#pragma unroll
    for (int k = 0; k < K; ++k) fma_row<V>(p, wf[k], win[u + k]);
    if (SILU) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float sg, rest;
        sigmoid<T>(p[c], sg, rest);
        p[c] *= sg;
      }
    }
    Vec<T, V>::store(to, p);
  };
  auto shift = [&](int n) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
#pragma unroll
      for (int c = 0; c < V; ++c) win[k][c] = win[k + n][c];
  };
  int t = t0;
  const int groups = te > t0 ? (te - t0) / U : 0;
  if (groups > 0) {  // the next group's rows are on their way while one is computed
    Raw<T, V> nx[U];
    const T* xr = xp + t0 * a.sx.t;
    T* yr = yp + t0 * a.sy.t;
    auto fetch = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u, xr += a.sx.t) nx[u].load(xr);
    };
    fetch();
#pragma unroll 1
    for (int n = 0; n < groups; ++n) {
#pragma unroll
      for (int u = 0; u < U; ++u) nx[u].unpack(win[K - 1 + u]);
      if (n + 1 < groups) fetch();
#pragma unroll
      for (int u = 0; u < U; ++u, yr += a.sy.t) step(u, yr);
      shift(U);
    }
    t += groups * U;
  }
  for (; t < te; ++t) {
    Vec<T, V>::load(xp + t * a.sx.t, win[K - 1]);
    step(0, yp + t * a.sy.t);
    shift(1);
  }
  if (te < t1) {  // steps behind the sequence's end
    float z[V];
#pragma unroll
    for (int c = 0; c < V; ++c) z[c] = 0.f;
    for (int t = max(te, t0); t < t1; ++t) Vec<T, V>::store(yp + t * a.sy.t, z);
  }
  if (sp && tile == 0) {
    // row r := input L - (K - 1) + r; rows still from the old state move down in order
    for (int r = 0; r < K - 1; ++r) {
      const int t = L - (K - 1) + r;
      float v[V];
      if (t >= 0) Vec<T, V>::load(xp + t * a.sx.t, v);
      else Vec<T, V>::load(sp + (long long)(t + K - 1) * a.d, v);
      Vec<T, V>::store(sp + (long long)r * a.d, v);
    }
  }
}

struct ConvBwdArgs {
  int B, H, T, d, tt, ntile;  // ntile: CTA tiles of kConvSub * tt steps
  int C;                      // H * d
  int wvec;                   // filters can be read in pieces of V
  sdm_strides sx, sdy, sdx;
};
constexpr int kConvSub = 4;  // step sub-tiles of a CTA, summed in shared memory

// A CTA: 32 lanes of V channels x kConvSub sub-tiles of tt steps.  Each thread
// recomputes p of its steps and of the K - 1 after them (their dp reaches back
// into its tile).  part[b * ntile + tile][K + 1][C] gets the CTA's sums of dw, db.
template <typename T, int V, int K, bool SILU>
__global__ void __launch_bounds__(32 * kConvSub, K > 4 ? 1 : 4)
k_conv_bwd(ConvBwdArgs a, const T* __restrict__ x, const T* __restrict__ w,
           const T* __restrict__ bias, const T* __restrict__ state0, const T* __restrict__ dy,
           const float* __restrict__ dstate, T* __restrict__ dx, float* __restrict__ dstate0,
           float* __restrict__ part) {
  wait_for_previous();
  __shared__ float red[kConvSub][32][V];
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int nv = a.d / V;
  const int hv = blockIdx.x * 32 + lane;
  const int tile = blockIdx.y % a.ntile, b = blockIdx.y / a.ntile;
  const bool live = hv < a.H * nv;
  const int h = live ? hv / nv : 0, c0 = live ? (hv - h * nv) * V : 0;
  const int t0 = (tile * kConvSub + sub) * a.tt;
  constexpr int U = 4;  // rows whose loads are in flight together
  float wf[K][V], bf[V], win[K][V], dpw[K][V], dw[K][V], db[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
#pragma unroll
    for (int k = 0; k < K; ++k) wf[k][c] = dw[k][c] = dpw[k][c] = win[k][c] = 0.f;
    bf[c] = bias && live ? to_f32(bias[(long long)h * a.d + c0 + c]) : 0.f;
    db[c] = 0.f;
  }
  if (live && t0 < a.T) {
    load_taps<T, V, K>(w + ((long long)h * a.d + c0) * K, a.wvec, wf);
    const T* xp = x + row_off(a.sx, b, h, 0) + c0;
    const T* yp = dy + row_off(a.sdy, b, h, 0) + c0;
    T* op = dx + row_off(a.sdx, b, h, 0) + c0;
    const long long st = ((long long)b * a.H + h) * (K - 1);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      const int t = t0 - (K - 1) + k;
      if (t >= 0) Vec<T, V>::load(xp + t * a.sx.t, win[k + 1]);
      else if (state0) Vec<T, V>::load(state0 + (st + t + K - 1) * a.d + c0, win[k + 1]);
    }
    const int own = min(t0 + a.tt, a.T);   // steps [t0, own) are this thread's
    const int end = own + K - 1;
    // one step: input xi, gradient gi; `mine` counts in dw and db.  out: the gradient of
    // input t - K + 1
    auto step = [&](const float* xi, const float* gi, bool mine, float (&out)[V]) {
      float dp[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
          win[k][c] = win[k + 1][c];
          dpw[k][c] = dpw[k + 1][c];
        }
        win[K - 1][c] = xi[c];
        dp[c] = gi[c];
      }
      if (SILU) {
        float p[V];
#pragma unroll
        for (int c = 0; c < V; ++c) p[c] = bf[c];
#pragma unroll
        for (int k = 0; k < K; ++k) fma_row<V>(p, wf[k], win[k]);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          float sg, rest;
          sigmoid<T>(p[c], sg, rest);
          dp[c] *= fmaf(p[c] * sg, rest, sg);
        }
      }
      if (mine) {
#pragma unroll
        for (int c = 0; c < V; ++c) db[c] += dp[c];
#pragma unroll
        for (int k = 0; k < K; ++k) fma_row<V>(dw[k], dp, win[k]);
      }
#pragma unroll
      for (int c = 0; c < V; ++c) {
        dpw[K - 1][c] = dp[c];
        out[c] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < K; ++k) fma_row<V>(out, wf[k], dpw[K - 1 - k]);
    };
    auto edge = [&](int t) {  // any step: range checks, states at both ends
      float in[V], g[V], out[V];
#pragma unroll
      for (int c = 0; c < V; ++c) in[c] = g[c] = 0.f;
      if (t < a.T) {
        Vec<T, V>::load(xp + t * a.sx.t, in);
        Vec<T, V>::load(yp + t * a.sdy.t, g);
      }
      step(in, g, t < own, out);
      if (t >= a.T)  // behind the end dp is 0 whatever p is
#pragma unroll
        for (int c = 0; c < V; ++c) {
          dpw[K - 1][c] = 0.f;
          out[c] = 0.f;
#pragma unroll
          for (int k = 1; k < K; ++k) out[c] = fmaf(wf[k][c], dpw[K - 1 - k][c], out[c]);
        }
      const int si = t - (K - 1);
      if (si >= t0 || t0 == 0) {
        const int r = si - a.T + K - 1;  // its row in the final state
        if (dstate && r >= 0)
#pragma unroll
          for (int c = 0; c < V; ++c) out[c] += dstate[(st + r) * a.d + c0 + c];
        if (si >= 0) Vec<T, V>::store(op + si * a.sdx.t, out);
        else if (dstate0)
#pragma unroll
          for (int c = 0; c < V; ++c) dstate0[(st + si + K - 1) * a.d + c0 + c] = out[c];
      }
    };
    int t = t0;
    for (; t < min(t0 + K - 1, end); ++t) edge(t);
    // steps whose input gradient is this thread's and meets neither end; the next group's
    // rows are on their way while one is computed
    const int groups = t < own ? (own - t) / U : 0;
    if (groups > 0) {
      Raw<T, V> nx[U], ng[U];
      const T* xr = xp + t * a.sx.t;
      const T* yr = yp + t * a.sdy.t;
      T* orow = op + (t - (K - 1)) * a.sdx.t;
      auto fetch = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u, xr += a.sx.t, yr += a.sdy.t) {
          nx[u].load(xr);
          ng[u].load(yr);
        }
      };
      fetch();
#pragma unroll 1
      for (int n = 0; n < groups; ++n) {
        float in[U][V], g[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          nx[u].unpack(in[u]);
          ng[u].unpack(g[u]);
        }
        if (n + 1 < groups) fetch();
#pragma unroll
        for (int u = 0; u < U; ++u, orow += a.sdx.t) {
          float out[V];
          step(in[u], g[u], true, out);
          Vec<T, V>::store(orow, out);
        }
      }
      t += groups * U;
    }
    for (; t < end; ++t) edge(t);
  }
  // sums over the CTA's sub-tiles, in order
  float* po = part + (size_t)blockIdx.y * (K + 1) * a.C;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
#pragma unroll
    for (int c = 0; c < V; ++c) red[sub][lane][c] = k < K ? dw[k < K ? k : 0][c] : db[c];
    __syncthreads();
    for (int j = threadIdx.x; j < 32 * V; j += 32 * kConvSub) {
      const int l = j / V, c = j - l * V;
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < kConvSub; ++q) s += red[q][l][c];
      const int col = (blockIdx.x * 32 + l) * V + c;
      if (col < a.C) po[(size_t)k * a.C + col] = s;
    }
    __syncthreads();
  }
}

// dw [C][K] and db [C] from the partial sums [rows][K + 1][C]: a CTA takes 32
// columns of one of the K + 1 rows, its 8 warps every 8th partial.
__global__ void __launch_bounds__(256)
k_conv_reduce(const float* __restrict__ part, int rows, int K, int C, float* __restrict__ dw,
              float* __restrict__ db) {
  wait_for_previous();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, k = blockIdx.y;
  float s = 0.f;
  if (col < C)
#pragma unroll 8
    for (int r = wp; r < rows; r += 8) s += part[((size_t)r * (K + 1) + k) * C + col];
  red[wp][lane] = s;
  __syncthreads();
  if (wp == 0 && col < C) {
    for (int q = 1; q < 8; ++q) s += red[q][lane];
    if (k < K) dw[(size_t)col * K + k] = s;
    else if (db) db[col] = s;
  }
}

static int conv_check(const sdm_conv_dims* d) {
  if (!d) return SDM_ERR_NULL;
  if (d->B < 1 || d->H < 1 || d->T < 0 || d->T > (1 << 30) || d->d < 1 || d->K < 1 ||
      (d->in_dtype != SDM_DTYPE_F32 && d->in_dtype != SDM_DTYPE_BF16))
    return SDM_ERR_DIMS;
  if ((long long)d->H * d->d > (1LL << 24) || (long long)d->B * d->H > (1LL << 24) ||
      (long long)d->B * d->H * d->d * (d->T > 0 ? d->T : 1) > (1LL << 45))
    return SDM_ERR_DIMS;
  if (d->K < 2 || d->K > 8) return SDM_ERR_UNSUPPORTED;
  return SDM_OK;
}

// Steps a thread walks.  Longer tiles re-read fewer halo rows (K - 1 a tile, from L2)
// and load the filter less often; shorter ones keep the card full.  The longest that
// still gives every SM 768 threads.
static int conv_tile(const sdm_conv_dims* d, int V, int lo, int hi, int sub) {
  int tt = hi;
  const long long vecs = (long long)d->B * d->H * ((d->d + V - 1) / V);
  while (tt > lo && vecs * (((long long)d->T + tt * sub - 1) / (tt * sub)) * sub < 148LL * 768) tt >>= 1;
  return tt;
}

template <typename T, int V, int K>
static cudaError_t launch_conv_fwd(const ConvArgs& a, bool silu, const void* x, const void* w,
                                   const void* bias, void* state, const int32_t* lengths, void* y,
                                   cudaStream_t s) {
  const long long n = (long long)a.B * a.ntile * a.H * (a.d / V);
  const unsigned grid = unsigned((n + 127) / 128);
  if (silu)
    launch_after(k_conv_fwd<T, V, K, true>, grid, 128, 0, s, a, (const T*)x, (const T*)w, (const T*)bias,
                                                   (T*)state, lengths, (T*)y);
  else
    launch_after(k_conv_fwd<T, V, K, false>, grid, 128, 0, s, a, (const T*)x, (const T*)w, (const T*)bias,
                                                    (T*)state, lengths, (T*)y);
  return cudaGetLastError();
}

template <typename T, int V, int K>
static cudaError_t launch_conv_bwd(const ConvBwdArgs& a, bool silu, const void* x, const void* w,
                                   const void* bias, const void* state0, const void* dy,
                                   const float* dstate, void* dx, float* dw, float* db,
                                   float* dstate0, float* part, cudaStream_t s) {
  const dim3 grid((a.H * (a.d / V) + 31) / 32, a.B * a.ntile);
  if (silu)
    launch_after(k_conv_bwd<T, V, K, true>, grid, 32 * kConvSub, 0, s, a, (const T*)x, (const T*)w, (const T*)bias,
                                                   (const T*)state0, (const T*)dy, dstate, (T*)dx,
                                                   dstate0, part);
  else
    launch_after(k_conv_bwd<T, V, K, false>, grid, 32 * kConvSub, 0, s, a, (const T*)x, (const T*)w, (const T*)bias,
                                                    (const T*)state0, (const T*)dy, dstate,
                                                    (T*)dx, dstate0, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  launch_after(k_conv_reduce, dim3((a.C + 31) / 32, K + 1), 256, 0, s, part, a.B * a.ntile, K, a.C, dw, db);
  return cudaGetLastError();
}

// Steps of a backward CTA's thread; the tile count of the grid's y axis stays
// below its limit of 65535.
static int conv_bwd_tiles(const sdm_conv_dims* d, int* tt) {
  *tt = conv_tile(d, d->in_dtype == SDM_DTYPE_BF16 ? 4 : 2, 8, 64, kConvSub);
  long long n;
  while ((n = ((long long)d->T + *tt * kConvSub - 1) / (*tt * kConvSub)) * d->B > 65535 &&
         *tt < (1 << 26))
    *tt <<= 1;
  return int(n);
}

template <typename F>
static cudaError_t conv_k(int K, F f) {
  switch (K) {
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return f(std::integral_constant<int, 8>());
  }
}

}  // namespace sdm

using namespace sdm;

extern "C" int sdm_conv_forward(const void* x, const void* w, const void* bias, void* state_inout,
                                const int32_t* lengths, void* y, const sdm_conv_dims* dims,
                                const sdm_strides* sx, const sdm_strides* sy, void* stream) {
  int rc = conv_check(dims);
  if (rc != SDM_OK) return rc;
  if (dims->T == 0) return SDM_OK;
  if (!strides_ok(sx) || !strides_ok(sy)) return SDM_ERR_DIMS;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  for (const void* p : {x, w, static_cast<const void*>(y)})
    if ((rc = need_ptr(p, es)) != SDM_OK) return rc;
  if (!aligned_to(bias, es) || !aligned_to(state_inout, es) || !aligned_to(lengths, 4))
    return SDM_ERR_ALIGN;
  const int V = 4;
  const size_t vb = V * es;
  const bool vec = dims->d % V == 0 && view_aligned(x, *sx, es, vb) && view_aligned(y, *sy, es, vb) &&
                   aligned_to(state_inout, vb);
  ConvArgs a{dims->B, dims->H, dims->T, dims->d, 0, 0, aligned_to(w, vb), *sx, *sy};
  a.tt = conv_tile(dims, vec ? V : 1, 8, 32, 1);
  a.ntile = (dims->T + a.tt - 1) / a.tt;
  if (((long long)a.B * a.ntile * a.H * (a.d / (vec ? V : 1)) + 127) / 128 >= (1LL << 31))
    return SDM_ERR_DIMS;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool silu = dims->silu != 0, bf = dims->in_dtype == SDM_DTYPE_BF16;
  const cudaError_t e = conv_k(dims->K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (bf)
      return vec ? launch_conv_fwd<__nv_bfloat16, 4, K>(a, silu, x, w, bias, state_inout, lengths, y, s)
                 : launch_conv_fwd<__nv_bfloat16, 1, K>(a, silu, x, w, bias, state_inout, lengths, y, s);
    return vec ? launch_conv_fwd<float, 4, K>(a, silu, x, w, bias, state_inout, lengths, y, s)
               : launch_conv_fwd<float, 1, K>(a, silu, x, w, bias, state_inout, lengths, y, s);
  });
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" size_t sdm_conv_backward_workspace_bytes(const sdm_conv_dims* dims) {
  if (conv_check(dims) != SDM_OK) return 0;
  int tt;
  const int n = conv_bwd_tiles(dims, &tt);
  const size_t b = size_t(dims->B) * n * (dims->K + 1) * dims->H * dims->d * 4;
  return b > 0 ? b : 16;
}

extern "C" int sdm_conv_backward(const void* x, const void* w, const void* bias,
                                 const void* state0, const void* dy, const float* dstate,
                                 void* dx, float* dw, float* dbias, float* dstate0,
                                 const sdm_conv_dims* dims, const sdm_strides* sx,
                                 const sdm_strides* sdy, const sdm_strides* sdx, void* workspace,
                                 size_t ws_bytes, void* stream) {
  int rc = conv_check(dims);
  if (rc != SDM_OK) return rc;
  if (dims->T == 0) return SDM_ERR_DIMS;  // there is no step to differentiate
  if (!strides_ok(sx) || !strides_ok(sdy) || !strides_ok(sdx)) return SDM_ERR_DIMS;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  for (const void* p : {x, w, dy, static_cast<const void*>(dx)})
    if ((rc = need_ptr(p, es)) != SDM_OK) return rc;
  if ((rc = need_ptr(dw, 4)) != SDM_OK) return rc;
  if (!aligned_to(bias, es) || !aligned_to(state0, es) || !aligned_to(dstate, 4) ||
      !aligned_to(dbias, 4) || !aligned_to(dstate0, 4))
    return SDM_ERR_ALIGN;
  if (!workspace || ws_bytes < sdm_conv_backward_workspace_bytes(dims)) return SDM_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return SDM_ERR_ALIGN;
  const int V = es == 2 ? 4 : 2;
  const size_t vb = V * es;
  const bool vec = dims->d % V == 0 && view_aligned(x, *sx, es, vb) &&
                   view_aligned(dy, *sdy, es, vb) && view_aligned(dx, *sdx, es, vb) &&
                   aligned_to(state0, vb);
  ConvBwdArgs a{dims->B, dims->H, dims->T, dims->d, 0, 0, dims->H * dims->d,
                aligned_to(w, vb), *sx, *sdy, *sdx};
  a.ntile = conv_bwd_tiles(dims, &a.tt);
  if ((long long)a.B * a.ntile > 65535) return SDM_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool silu = dims->silu != 0, bf = dims->in_dtype == SDM_DTYPE_BF16;
  float* part = static_cast<float*>(workspace);
  const cudaError_t e = conv_k(dims->K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (bf)
      return vec ? launch_conv_bwd<__nv_bfloat16, 4, K>(a, silu, x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0, part, s)
                 : launch_conv_bwd<__nv_bfloat16, 1, K>(a, silu, x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0, part, s);
    return vec ? launch_conv_bwd<float, 2, K>(a, silu, x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0, part, s)
               : launch_conv_bwd<float, 1, K>(a, silu, x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0, part, s);
  });
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
