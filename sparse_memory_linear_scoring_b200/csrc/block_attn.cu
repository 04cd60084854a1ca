// block_attn.cu -- attention over listed blocks, a CTA per query and group: the
// CUDA-core path (float32 inputs, single tokens, short calls), forward and the
// query's gradient; and the C ABI of the forward pass.
//
//   s_k = scale q.k over the listed keys at positions <= p;  o = sum softmax(s)_k v_k;
//   lse = log sum exp(s_k);  no key: o = 0, lse = -inf.
//   backward: P_k = exp(s_k - lse), dP_k = do.v_k, ds_k = P_k (dP_k - do.o) scale,
//   dq = sum ds_k k_k.
// One pass over the keys with the running maximum and sum, 32 keys at a time, for
// up to 8 heads of the group at once, which then share the tile.
#include "block_internal.cuh"

namespace sdm {

constexpr int kRowThreads = 128;
constexpr int kRowHeads = 8;   // heads of a group a CTA takes
constexpr int kRowKeys = 32;   // keys per tile

__host__ __device__ inline size_t blk_row_smem(int d, bool bwd) {
  // q (and do) [8][d], K, V [32][d + 1], p [8][33], rescale, m, l, (lse, delta) [8]
  return size_t(4) * ((bwd ? 2 : 1) * kRowHeads * d + 2 * kRowKeys * (d + 1) + kRowHeads * 33 + 5 * kRowHeads);
}

template <typename Tin, int D, bool BWD>
__global__ void __launch_bounds__(kRowThreads)
k_blk_row(BlkArgs a, const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
          const int32_t* __restrict__ idx, Tin* __restrict__ o, float* __restrict__ lse,
          const Tin* __restrict__ d_o, float* __restrict__ delta, Tin* __restrict__ dq,
          sdm_strides sdo, sdm_strides sdq, int hc) {
  extern __shared__ __align__(16) float sm[];
  constexpr int Dp = D + 1;
  float* qs = sm;
  float* gs = qs + kRowHeads * D;             // do, backward only
  float* Ks = qs + (BWD ? 2 : 1) * kRowHeads * D;
  float* Vs = Ks + kRowKeys * Dp;
  float* ps = Vs + kRowKeys * Dp;             // [8][33]
  float* fs = ps + kRowHeads * 33;            // rescale factors, then 1 / l
  float* ms = fs + kRowHeads;
  float* dl = ms + kRowHeads;                 // do.o
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  long long i = blockIdx.x;
  const int ch = int(i % hc); i /= hc;
  const int t = int(i % a.Tq);
  const int bg = int(i / a.Tq), b = bg / a.G, g = bg - b * a.G;
  const int r0 = ch * kRowHeads, nh = min(kRowHeads, a.R - r0), h0 = g * a.R + r0;
  const int p = blk_pos0(a, b) + t;
  for (int e = tid; e < kRowHeads * D; e += kRowThreads) {
    const int r = e / D, c = e - r * D;
    qs[e] = r < nh ? to_f32(q[row_off(a.sq, b, h0 + r, t) + c]) * a.scale : 0.f;
    if (BWD) gs[e] = r < nh ? to_f32(d_o[row_off(sdo, b, h0 + r, t) + c]) : 0.f;
  }
  // a thread owns column c of heads hs, hs + HS, ...
  constexpr int HS = kRowThreads / D > 0 ? kRowThreads / D : 1, NA = kRowHeads / HS;
  const int c = tid % D, hs = tid / D;
  float acc[NA];
#pragma unroll
  for (int u = 0; u < NA; ++u) acc[u] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2 wp, 2 wp + 1
  if (BWD) {
    // delta = do.o, and the saved log-sum-exp in place of the running maximum
    for (int r = wp; r < kRowHeads; r += 4) {
      float s = 0.f;
      if (r < nh)
        for (int e = lane; e < D; e += 32)
          s = fmaf(to_f32(d_o[row_off(sdo, b, h0 + r, t) + e]), to_f32(o[row_off(a.so, b, h0 + r, t) + e]), s);
      s = warp_sum(s);
      if (lane == 0) {
        dl[r] = s;
        ms[r] = r < nh ? lse[((size_t)b * a.H + h0 + r) * a.Tq + t] : -INFINITY;
        if (r < nh) delta[((size_t)b * a.H + h0 + r) * a.Tq + t] = s;
      }
    }
  }
  const int32_t* list = idx + ((size_t)bg * a.Tq + t) * a.n_sel;
  for (int sl = 0; sl < a.n_sel; ++sl) {
    const int j = list[sl];
    const int n = blk_keys(a, j, p);
    for (int k0 = 0; k0 < n; k0 += kRowKeys) {
      const int nk = min(kRowKeys, n - k0);
      __syncthreads();
      for (int e = tid; e < kRowKeys * D; e += kRowThreads) {
        const int kk = e / D, cc = e - kk * D;
        const bool in = kk < nk;  // keys behind the query are not read
        const int at = j * a.bs + k0 + kk;
        Ks[kk * Dp + cc] = in ? to_f32(k[row_off(a.sk, b, g, at) + cc]) : 0.f;
        Vs[kk * Dp + cc] = in ? to_f32(v[row_off(a.sv, b, g, at) + cc]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = 2 * wp + u;
        float s = 0.f;
#pragma unroll 8
        for (int e = 0; e < D; ++e) s = fmaf(qs[r * D + e], Ks[lane * Dp + e], s);
        if (lane >= nk) s = -INFINITY;
        if (!BWD) {
          float mx = s;
#pragma unroll
          for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          mx = fmaxf(mx, m[u]);
          const float base = mx == -INFINITY ? 0.f : mx;
          const float e = lane < nk ? expf(s - base) : 0.f;
          const float f = expf(m[u] - base);  // 0 from the empty start
          l[u] = fmaf(l[u], f, warp_sum(e));
          m[u] = mx;
          ps[r * 33 + lane] = e;
          if (lane == 0) fs[r] = f;
        } else {
          float dp = 0.f;
#pragma unroll 8
          for (int e = 0; e < D; ++e) dp = fmaf(gs[r * D + e], Vs[lane * Dp + e], dp);
          const float pr = lane < nk && ms[r] != -INFINITY ? expf(s - ms[r]) : 0.f;
          ps[r * 33 + lane] = pr * (dp - dl[r]) * a.scale;
        }
      }
      __syncthreads();
      if (hs < HS) {
#pragma unroll
        for (int u = 0; u < NA; ++u) {
          const int r = hs + u * HS;
          float x = BWD ? acc[u] : acc[u] * fs[r];
          const float* M = BWD ? Ks : Vs;
          for (int kk = 0; kk < nk; ++kk) x = fmaf(ps[r * 33 + kk], M[kk * Dp + c], x);
          acc[u] = x;
        }
      }
    }
  }
  __syncthreads();
  if (!BWD) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 2 * wp + u;
      if (lane == 0) {
        fs[r] = l[u] == 0.f ? 0.f : 1.f / l[u];
        if (lse && r < nh)
          lse[((size_t)b * a.H + h0 + r) * a.Tq + t] = l[u] == 0.f ? -INFINITY : m[u] + logf(l[u]);
      }
    }
    __syncthreads();
  }
  if (hs < HS) {
#pragma unroll
    for (int u = 0; u < NA; ++u) {
      const int r = hs + u * HS;
      if (r >= nh) continue;
      if (BWD) dq[row_off(sdq, b, h0 + r, t) + c] = from_f32<Tin>(acc[u]);
      else o[row_off(a.so, b, h0 + r, t) + c] = from_f32<Tin>(acc[u] * fs[r]);
    }
  }
}

template <typename Tin, bool BWD>
static cudaError_t launch_row(const BlkArgs& a, const void* q, const void* k, const void* v,
                              const int32_t* idx, void* o, float* lse, const void* d_o,
                              float* delta, void* dq, const sdm_strides& sdo,
                              const sdm_strides& sdq, cudaStream_t s) {
  const int hc = (a.R + kRowHeads - 1) / kRowHeads;
  const long long grid = (long long)a.B * a.G * a.Tq * hc;
  if (grid >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const int smem = int(blk_row_smem(a.d, BWD));
  auto go = [&](auto dd) -> cudaError_t {
    constexpr int D = decltype(dd)::value;
    cudaError_t e = cudaFuncSetAttribute(k_blk_row<Tin, D, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_blk_row<Tin, D, BWD><<<unsigned(grid), kRowThreads, smem, s>>>(
        a, (const Tin*)q, (const Tin*)k, (const Tin*)v, idx, (Tin*)o, lse, (const Tin*)d_o, delta,
        (Tin*)dq, sdo, sdq, hc);
    return cudaGetLastError();
  };
  if (a.d == 32) return go(std::integral_constant<int, 32>());
  if (a.d == 64) return go(std::integral_constant<int, 64>());
  return go(std::integral_constant<int, 128>());
}

cudaError_t launch_blk_row_fwd(const BlkArgs& a, bool bf16, const void* q, const void* k,
                               const void* v, const int32_t* idx, void* o, float* lse,
                               cudaStream_t s) {
  const sdm_strides z = {0, 0, 0};
  return bf16 ? launch_row<__nv_bfloat16, false>(a, q, k, v, idx, o, lse, nullptr, nullptr, nullptr, z, z, s)
              : launch_row<float, false>(a, q, k, v, idx, o, lse, nullptr, nullptr, nullptr, z, z, s);
}

cudaError_t launch_blk_row_bwd(const BlkArgs& a, bool bf16, const void* q, const void* k,
                               const void* v, const int32_t* idx, const void* o, const float* lse,
                               const void* d_o, float* delta, void* dq, const sdm_strides& sdo,
                               const sdm_strides& sdq, cudaStream_t s) {
  void* om = const_cast<void*>(o);
  float* lm = const_cast<float*>(lse);
  return bf16 ? launch_row<__nv_bfloat16, true>(a, q, k, v, idx, om, lm, d_o, delta, dq, sdo, sdq, s)
              : launch_row<float, true>(a, q, k, v, idx, om, lm, d_o, delta, dq, sdo, sdq, s);
}

}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_block_workspace_bytes(const sdm_block_dims* dims) {
  if (blk_check(dims) != SDM_OK) return 0;
  return blk_tiles_pay(dims) ? blk_fwd_ws(dims, blk_chunk(dims), nullptr).bytes : 16;
}

extern "C" int sdm_block_forward(const void* q, const void* k, const void* v, const int32_t* idx,
                                 const int32_t* lengths, void* o, float* lse,
                                 const sdm_block_dims* dims, const sdm_block_views* views,
                                 void* workspace, size_t ws_bytes, void* stream) {
  int rc = blk_check(dims);
  if (rc != SDM_OK) return rc;
  if ((rc = blk_views_ok(views)) != SDM_OK) return rc;
  if (dims->Tq == 0) return SDM_OK;
  const size_t es = dims->in_dtype == SDM_DTYPE_BF16 ? 2 : 4;
  for (const void* p : {q, k, v, static_cast<const void*>(o)})
    if ((rc = need_ptr(p, es)) != SDM_OK) return rc;
  if ((rc = need_ptr(idx, 4)) != SDM_OK) return rc;
  if (!aligned_to(lengths, 4) || !aligned_to(lse, 4)) return SDM_ERR_ALIGN;
  if (!workspace || ws_bytes < sdm_block_workspace_bytes(dims)) return SDM_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return SDM_ERR_ALIGN;
  const BlkArgs a = blk_args(dims, views, lengths);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool tiles = blk_tiles_pay(dims) && view_aligned(q, a.sq, 2, 16) && view_aligned(k, a.sk, 2, 16) &&
                     view_aligned(v, a.sv, 2, 16) && view_aligned(o, a.so, 2, 16);
  const cudaError_t e = tiles ? launch_blk_fwd_mma(dims, a, q, k, v, idx, o, lse, workspace, s)
                              : launch_blk_row_fwd(a, dims->in_dtype == SDM_DTYPE_BF16, q, k, v, idx, o, lse, s);
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
