// ssm_internal.cuh -- the selective state space scan (ssm.cu, ssm_mma.cu,
// ssm_bwd.cu, ssm_bwd_mma.cu): sizes of a call, its workspace, and what the kernels share.
//
// Per (b,h) head, S in R^{P x N} (P = d_v rows, N = d_k columns as in gdn.cu):
//     a_t = exp(dt_t A_h);  S_t = a_t S_{t-1} + dt_t x_t B_t^T;  y_t = S_t C_t + D_h x_t,
// B and C shared by the heads of a group.  With g_t = sum_{s<=t} dt_s A from a
// chunk's first step and S_0 the state before it,
//     y_t = sum_{j<=t} exp(g_t - g_j) dt_j (C_t.B_j) x_j + exp(g_t) S_0 C_t + D x_t,
//     S_Q = exp(g_Q) S_0 + sum_j exp(g_Q - g_j) dt_j x_j B_j^T.
// Every exponent is a difference with the later step first, so nothing overflows
// for A <= 0.  g is summed in double and held, times log2 e, as a float pair:
// near steps far into a strongly decaying chunk keep exact differences, which a
// single float loses (g = -60 would cost 4e-6 of a weight).
//
// A value that is not finite stays out of what does not depend on it: a masked weight is
// left out of a sum where 0 times that value would enter it, and the chunks' products that
// split an operand into bf16 parts, where an infinity would become inf - inf, are taken
// step by step for a chunk that holds such a value.
#pragma once

#include "seq_internal.cuh"

namespace sdm {

struct SsmArgs {
  int B, H, G, T, P, N;
  int Q;      // steps per chunk
  int nch;    // chunks
  int cps;    // chunks per segment
  int nseg;   // segments walked in parallel per head
  int hg;     // heads per group
  sdm_strides sx, sdt, sB, sC, sy;
};

// Steps per chunk of the CUDA-core kernels (ssm.cu, ssm_bwd.cu) and of the
// tensor-core ones.
constexpr int kSsmQ = 32;
constexpr int kSsmQT = 64;

// Running sum of dt A log2(e) over a chunk's steps, in double, by one warp: step t
// (t < 32 * R) of the chunk gets the pair hi[t] + lo[t].
template <int R>
__device__ __forceinline__ void chunk_decay(const float* dts, float A, float* hi, float* lo) {
  const int lane = threadIdx.x & 31;
  const double al = double(A) * 1.4426950408889634074;
  double v[R], s = 0.0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    s += double(dts[R * lane + i]) * al;
    v[i] = s;
  }
  double inc = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  double ex = __shfl_up_sync(0xffffffffu, inc, 1);  // steps before the lane's: not inc - s, which
  if (lane == 0) ex = 0.0;                          // a NaN among the lane's own would enter
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const double g = ex + v[i];
    const float h = float(g);
    hi[R * lane + i] = h;
    lo[R * lane + i] = float(g - double(h));
  }
}

// exp(g_t - g_j) of the pairs above.
__device__ __forceinline__ float decay_between(float hi_t, float lo_t, float hi_j, float lo_j) {
  return ex2((hi_t - hi_j) + (lo_t - lo_j));  // below 2^-126: 0
}

// Launchers.  The states kernel writes, per (head, segment), the segment's own
// contribution to the state and its total log2 decay; the carry kernel turns the
// former into the state before each segment.
// S_end (may be S0 itself, or NULL) gets the last state.
cudaError_t launch_ssm_carry(float* segS, const float* segG, const float* S0, float* S_end, int BH,
                             int nseg, int PN, cudaStream_t s);

// The tensor-core walk takes bf16 inputs of widths 64 and 128 whose views allow
// 16-byte pieces.
cudaError_t launch_ssm_fwd_mma(const SsmArgs& a, const void* x, const float* dt, const float* A,
                               const void* Bm, const void* Cm, const float* D, float* S,
                               const int32_t* lengths, void* y, float* segS, float* segG,
                               cudaStream_t s);
// Each segment's own contribution and decay on tcgen05 (ssm_tc.cu), d_k = 128.
cudaError_t launch_ssm_seg(const SsmArgs& a, const void* x, const float* dt, const float* A, const void* Bm,
                           const int32_t* lengths, float* segS, float* segG, cudaStream_t s);
inline bool ssm_tensor_sizes(const sdm_ssm_dims* d) {
  return d->in_dtype == SDM_DTYPE_BF16 && d->d_v >= 64 && d->d_k >= 64;
}

// Backward pass (ssm_bwd.cu, ssm_bwd_mma.cu).
struct SsmBwdArgs {
  SsmArgs a;  // sy: strides of dy
  sdm_strides sdx, sddt, sdB, sdC;
};

struct SsmBwdWs {
  float* fS;    // [BH][nch][P][N] state before each chunk
  float* gS;    // [BH][nch][P][N] gradient arriving at each chunk's end
  float* ST;    // [BH][P][N] last state
  float* lg;    // [BH][nch] log2 decay of each chunk
  double* dAD;  // [BH][nch][2] parts of dA and dD
  float* pB;    // [BH][T][N] per-head dB, dC where heads share them
  float* pC;
  size_t total;
};

// Both carries of the backward pass in one launch: states before the chunks and last
// states from S0, gradients at the chunks' ends and of S0 from dST.
cudaError_t launch_ssm_carries(float* fS, float* gS, const float* lg, const float* S0, float* ST,
                               const float* dST, float* dS0, int BH, int nch, int PN, cudaStream_t s);
cudaError_t launch_ssm_bwd_mma(const SsmBwdArgs& ba, const void* x, const float* dt, const float* A,
                               const void* Bm, const void* Cm, const float* D, const float* S0,
                               const void* dy, const float* dST, const SsmBwdWs& w, void* dx, float* ddt,
                               void* dB, void* dC, float* dS0, cudaStream_t s);

// Argument checks and sizes shared by the entry points.
SsmArgs ssm_args(const sdm_ssm_dims* d, const sdm_ssm_views* v);
int ssm_views_ok(const sdm_ssm_views* v);
int ssm_ptrs(const sdm_ssm_dims* d, const void* x, const float* dt, const float* A, const void* Bm,
             const void* Cm, const float* D);
int ssm_check(const sdm_ssm_dims* d);

}  // namespace sdm
