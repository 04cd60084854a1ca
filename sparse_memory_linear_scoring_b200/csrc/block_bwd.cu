// block_bwd.cu -- gradients of keys and values of block-selected attention on CUDA
// cores, and the C ABI of the backward pass.  block_attn.cu has the formulas;
// here dv_k = sum P_k do, dk_k = sum ds_k q over the queries that list k's block.
//
// A CTA owns 32 keys of a block and walks the block's list of (query, slot) pairs
// in query order, 8 rows (query, head of the group) at a time, so the sums over
// queries and over the heads that share the keys stay in registers, need no
// atomics and come out the same on every run.
#include "block_internal.cuh"

namespace sdm {

cudaError_t launch_blk_row_bwd(const BlkArgs& a, bool bf16, const void* q, const void* k,
                               const void* v, const int32_t* idx, const void* o, const float* lse,
                               const void* d_o, float* delta, void* dq, const sdm_strides& sdo,
                               const sdm_strides& sdq, cudaStream_t s);

constexpr int kKvThreads = 256;
constexpr int kKvRows = 8;

__host__ __device__ inline size_t blk_kv_smem(int d) {
  return size_t(4) * (2 * 32 * (d + 1) + 2 * kKvRows * d + 2 * kKvRows * 33 + 4 * kKvRows);
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kKvThreads)
k_blk_kv(BlkArgs a, BlkPlan pl, const Tin* __restrict__ q, const Tin* __restrict__ k,
         const Tin* __restrict__ v, const float* __restrict__ lse, const Tin* __restrict__ d_o,
         const float* __restrict__ delta, Tin* __restrict__ dk, Tin* __restrict__ dv,
         sdm_strides sdo, sdm_strides sdk, sdm_strides sdv) {
  extern __shared__ __align__(16) float sm[];
  constexpr int Dp = D + 1;
  float* Ks = sm;
  float* Vs = Ks + 32 * Dp;
  float* qs = Vs + 32 * Dp;        // [8][D]
  float* gs = qs + kKvRows * D;    // [8][D] do
  float* ps = gs + kKvRows * D;    // [8][33]
  float* ds = ps + kKvRows * 33;   // [8][33]
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int per = a.bs / 32;
  const int sub = blockIdx.x % per;
  const int j = int((blockIdx.x / per) % a.nb), bg = blockIdx.x / per / a.nb;
  const int b = bg / a.G, g = bg - b * a.G;
  const int k0 = j * a.bs + sub * 32;
  const int nk = min(32, a.Tk - k0);  // keys of this CTA
  if (nk <= 0) return;
  const int pos0 = blk_pos0(a, b);
  const int len = pos0 + a.Tq;  // keys at or behind it belong to no query and are not read
  for (int e = tid; e < 32 * D; e += kKvThreads) {
    const int kk = e / D, c = e - kk * D;
    const bool in = kk < nk && k0 + kk < len;
    Ks[kk * Dp + c] = in ? to_f32(k[row_off(a.sk, b, g, k0 + kk) + c]) : 0.f;
    Vs[kk * Dp + c] = in ? to_f32(v[row_off(a.sv, b, g, k0 + kk) + c]) : 0.f;
  }
  constexpr int KS = kKvThreads / D, NA = 32 / KS;  // a thread: column c of NA keys
  const int c = tid % D, ks = tid / D;
  float ak[NA], av[NA];
#pragma unroll
  for (int u = 0; u < NA; ++u) ak[u] = av[u] = 0.f;
  const int* first = pl.first + (size_t)bg * (a.nb + 1);
  const int e0 = first[j], e1 = first[j + 1];
  const int* entry = pl.entry + (size_t)bg * a.Tq * a.n_sel;
  const long long rows = (long long)(e1 - e0) * a.R;
  for (long long w0 = 0; w0 < rows; w0 += kKvRows) {
    __syncthreads();
    for (int e = tid; e < kKvRows * D; e += kKvThreads) {
      const int r = e / D, cc = e - r * D;
      float x = 0.f, y = 0.f;
      if (w0 + r < rows) {
        const int t = entry[e0 + int((w0 + r) / a.R)] / a.n_sel, h = g * a.R + int((w0 + r) % a.R);
        x = to_f32(q[row_off(a.sq, b, h, t) + cc]);
        y = to_f32(d_o[row_off(sdo, b, h, t) + cc]);
      }
      qs[e] = x;
      gs[e] = y;
    }
    __syncthreads();
    {  // warp wp takes row wp, lane takes a key
      float s = 0.f, dp = 0.f, P = 0.f, dS = 0.f;
#pragma unroll 8
      for (int e = 0; e < D; ++e) {
        s = fmaf(qs[wp * D + e], Ks[lane * Dp + e], s);
        dp = fmaf(gs[wp * D + e], Vs[lane * Dp + e], dp);
      }
      if (w0 + wp < rows) {
        const int t = entry[e0 + int((w0 + wp) / a.R)] / a.n_sel, h = g * a.R + int((w0 + wp) % a.R);
        const size_t at = ((size_t)b * a.H + h) * a.Tq + t;
        const float ls = lse[at];
        if (lane < nk && k0 + lane <= pos0 + t && ls != -INFINITY) {
          P = expf(s * a.scale - ls);
          dS = P * (dp - delta[at]) * a.scale;
        }
      }
      ps[wp * 33 + lane] = P;
      ds[wp * 33 + lane] = dS;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kKvRows; ++r) {
      const float x = qs[r * D + c], y = gs[r * D + c];
#pragma unroll
      for (int u = 0; u < NA; ++u) {
        ak[u] = fmaf(ds[r * 33 + ks + u * KS], x, ak[u]);
        av[u] = fmaf(ps[r * 33 + ks + u * KS], y, av[u]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < NA; ++u) {
    const int kk = ks + u * KS;
    if (kk >= nk) continue;
    dk[row_off(sdk, b, g, k0 + kk) + c] = from_f32<Tin>(ak[u]);
    dv[row_off(sdv, b, g, k0 + kk) + c] = from_f32<Tin>(av[u]);
  }
}

template <typename Tin>
static cudaError_t launch_kv(const BlkArgs& a, const BlkPlan& pl, const void* q, const void* k,
                             const void* v, const float* lse, const void* d_o, const float* delta,
                             void* dk, void* dv, const sdm_strides& sdo, const sdm_strides& sdk,
                             const sdm_strides& sdv, cudaStream_t s) {
  const long long grid = (long long)a.B * a.G * a.nb * (a.bs / 32);
  if (grid >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const int smem = int(blk_kv_smem(a.d));
  auto go = [&](auto dd) -> cudaError_t {
    constexpr int D = decltype(dd)::value;
    cudaError_t e = cudaFuncSetAttribute(k_blk_kv<Tin, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_blk_kv<Tin, D><<<unsigned(grid), kKvThreads, smem, s>>>(
        a, pl, (const Tin*)q, (const Tin*)k, (const Tin*)v, lse, (const Tin*)d_o, delta, (Tin*)dk,
        (Tin*)dv, sdo, sdk, sdv);
    return cudaGetLastError();
  };
  if (a.d == 32) return go(std::integral_constant<int, 32>());
  if (a.d == 64) return go(std::integral_constant<int, 64>());
  return go(std::integral_constant<int, 128>());
}

}  // namespace sdm

using namespace sdm;

static size_t blk_delta_bytes(const sdm_block_dims* d) {
  return (size_t(d->B) * d->H * d->Tq * 4 + 255) & ~size_t(255);
}

extern "C" size_t sdm_block_backward_workspace_bytes(const sdm_block_dims* dims) {
  if (blk_check(dims) != SDM_OK) return 0;
  size_t n = blk_delta_bytes(dims) + blk_plan(dims, dims->Tq, 512, nullptr).bytes;
  if (blk_bwd_tiles_pay(dims)) {  // views that are not aligned still take the other path
    const size_t t = blk_bwd_ws(dims, blk_bwd_chunk(dims), nullptr).bytes;
    if (t > n) n = t;
  }
  return n > 0 ? n : 16;
}

extern "C" int sdm_block_backward(const void* q, const void* k, const void* v, const int32_t* idx,
                                  const int32_t* lengths, const void* o, const float* lse,
                                  const void* d_o, void* dq, void* dk, void* dv,
                                  const sdm_block_dims* dims, const sdm_block_views* views,
                                  const sdm_block_views* grad_views, void* workspace,
                                  size_t ws_bytes, void* stream) {
  int rc = blk_check(dims);
  if (rc != SDM_OK) return rc;
  if ((rc = blk_views_ok(views)) != SDM_OK || (rc = blk_views_ok(grad_views)) != SDM_OK) return rc;
  if (dims->Tq == 0) return SDM_ERR_DIMS;  // there is no query to differentiate
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  for (const void* p : {q, k, v, o, d_o, static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if ((rc = need_ptr(p, es)) != SDM_OK) return rc;
  if ((rc = need_ptr(idx, 4)) != SDM_OK || (rc = need_ptr(lse, 4)) != SDM_OK) return rc;
  if (!aligned_to(lengths, 4)) return SDM_ERR_ALIGN;
  if (!workspace || ws_bytes < sdm_block_backward_workspace_bytes(dims)) return SDM_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return SDM_ERR_ALIGN;
  const BlkArgs a = blk_args(dims, views, lengths);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const sdm_block_views* gv = grad_views;
  if (blk_bwd_tiles_pay(dims) && view_aligned(q, a.sq, 2, 16) && view_aligned(k, a.sk, 2, 16) &&
      view_aligned(v, a.sv, 2, 16) && view_aligned(o, a.so, 2, 16) && view_aligned(d_o, gv->o, 2, 16) &&
      view_aligned(dq, gv->q, 2, 16) && view_aligned(dk, gv->k, 2, 16) && view_aligned(dv, gv->v, 2, 16))
    return launch_blk_bwd_mma(dims, a, q, k, v, idx, o, lse, d_o, dq, dk, dv, gv, workspace, s) == cudaSuccess
               ? SDM_OK : SDM_ERR_CUDA;
  float* delta = static_cast<float*>(workspace);
  const BlkPlan pl = blk_plan(dims, dims->Tq, 512, static_cast<char*>(workspace) + blk_delta_bytes(dims));
  const bool bf = dims->in_dtype == SDM_DTYPE_BF16;
  cudaError_t e = launch_blk_row_bwd(a, bf, q, k, v, idx, o, lse, d_o, delta, dq, grad_views->o, grad_views->q, s);
  if (e == cudaSuccess) e = launch_blk_plan(a, pl, idx, s);
  if (e == cudaSuccess)
    e = bf ? launch_kv<__nv_bfloat16>(a, pl, q, k, v, lse, d_o, delta, dk, dv, grad_views->o, grad_views->k, grad_views->v, s)
           : launch_kv<float>(a, pl, q, k, v, lse, d_o, delta, dk, dv, grad_views->o, grad_views->k, grad_views->v, s);
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
