// block_bwd.cu -- gradients of keys and values of block-selected attention on CUDA
// cores, and the C ABI of the backward pass.  block_attn.cu has the formulas;
// here dv_k = sum P_k do, dk_k = sum ds_k q over the queries that list k's block.
//
// A CTA owns 32 keys of a block and an item of the block's list of (query, slot) pairs,
// which it walks in query order, 32 rows (query, head of the group) at a time, so the sums
// over queries and over the heads that share the keys stay in registers.  An item leaves
// a float32 part; the parts are summed in item order: no atomics, equal calls give equal
// bits.  (One CTA for all of a block's rows left most of the card idle: 1760 float32
// tokens, 4 heads of 32, lists of 16 took 0.6 ms in this kernel.)
#include "block_internal.cuh"

namespace sdm {

cudaError_t launch_blk_row_bwd(const BlkArgs& a, bool bf16, const void* q, const void* k,
                               const void* v, const int32_t* idx, const void* o, const float* lse,
                               const void* d_o, float* delta, void* dq, const sdm_strides& sdo,
                               const sdm_strides& sdq, cudaStream_t s);

constexpr int kKvThreads = 256;
constexpr int kKvRows = 32;

__host__ __device__ inline size_t blk_kv_smem(int d) {
  // K, V [32][d + 4], q, do [32][d], P, dS [32][36], rows' facts [32][4]
  return size_t(4) * (2 * 32 * (d + 4) + 2 * kKvRows * d + 2 * kKvRows * 36 + 4 * kKvRows);
}

// Both halves read shared memory in 16-byte pieces and share them among 4 rows (scores,
// lane = key) or 4 columns x 32 / (256 / (D / 4)) keys (sums): about 2 and 2.7 multiply-adds
// a read; single elements gave 0.5 and 0.9, which bound the kernel.
template <typename Tin, int D>
__global__ void __launch_bounds__(kKvThreads)
k_blk_kv(BlkArgs a, BlkPlan pl, const Tin* __restrict__ q, const Tin* __restrict__ k,
         const Tin* __restrict__ v, const float* __restrict__ lse, const Tin* __restrict__ d_o,
         const float* __restrict__ delta, float* __restrict__ part, sdm_strides sdo, int vec) {
  wait_for_previous();
  extern __shared__ __align__(16) float sm[];
  constexpr int Dp = D + 4;
  float* Ks = sm;
  float* Vs = Ks + 32 * Dp;
  float* qs = Vs + 32 * Dp;        // [32][D]
  float* gs = qs + kKvRows * D;    // [32][D] do
  float* ps = gs + kKvRows * D;    // [32][36]
  float* ds = ps + kKvRows * 36;   // [32][36]
  int* rt = reinterpret_cast<int*>(ds + kKvRows * 36);
  int* rh = rt + kKvRows;
  float* rl = reinterpret_cast<float*>(rh + kKvRows);
  float* rd = rl + kKvRows;
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int per = a.bs / 32;
  const int sub = blockIdx.x % per;
  const int ii = blockIdx.x / per, bg = ii / pl.most, it = ii - bg * pl.most;
  const int b = bg / a.G, g = bg - b * a.G;
  const int* item = pl.item + (size_t)bg * (a.nb + 1);
  const int j = blk_of_item(item, a.nb, it);
  if (j < 0) return;
  const int k0 = j * a.bs + sub * 32;
  const int nk = max(0, min(32, a.Tk - k0));  // keys of this CTA
  const int pos0 = blk_pos0(a, b);
  const int len = pos0 + a.Tq;  // keys at or behind it belong to no query and are not read
  auto four = [&](const Tin* p, bool in, float* dst) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (in) {
      if (vec) {
        Vec<Tin, 4>::load(p, f);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = to_f32(p[e]);
      }
    }
    *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
    return !(fabsf(f[0]) + fabsf(f[1]) + fabsf(f[2]) + fabsf(f[3]) < INFINITY);
  };
  for (int i = tid; i < 32 * (D / 4); i += kKvThreads) {
    const int kk = i / (D / 4), c = (i % (D / 4)) * 4;
    const bool in = kk < nk && k0 + kk < len;
    const int at = in ? k0 + kk : 0;
    four(k + row_off(a.sk, b, g, at) + c, in, Ks + kk * Dp + c);
    four(v + row_off(a.sv, b, g, at) + c, in, Vs + kk * Dp + c);
  }
  // sums: a thread owns columns c .. c + 3 of NA keys
  constexpr int KS = kKvThreads / (D / 4), NA = 32 / KS;
  const int c = (tid % (D / 4)) * 4, ks = tid / (D / 4) * NA;
  float ak[NA][4], av[NA][4];
#pragma unroll
  for (int u = 0; u < NA; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) ak[u][e] = av[u][e] = 0.f;
  const int* first = pl.first + (size_t)bg * (a.nb + 1);
  const int e0 = first[j], e1 = first[j + 1];
  const int* entry = pl.entry + (size_t)bg * a.Tq * a.n_sel + e0;
  const int all = (e1 - e0) * a.R;  // below 2^31
  const int r0 = (it - item[j]) * pl.rows, rows = all - r0 < pl.rows ? all : r0 + pl.rows;
  for (int w0 = r0; w0 < rows; w0 += kKvRows) {
    __syncthreads();
    if (tid < kKvRows) {
      const bool in = w0 + tid < rows;
      const int en = in ? a.by_R.div(w0 + tid) : 0;
      const int t = in ? a.by_sel.div(entry[en]) : 0, h = g * a.R + (in ? w0 + tid - en * a.R : 0);
      const size_t at = ((size_t)b * a.H + h) * a.Tq + t;
      rt[tid] = in ? t : -1;
      rh[tid] = h;
      rl[tid] = in ? lse[at] : -INFINITY;
      rd[tid] = in ? delta[at] : 0.f;
    }
    __syncthreads();
    bool odd = false;
#pragma unroll 4
    for (int i = tid; i < kKvRows * (D / 4); i += kKvThreads) {
      const int r = i / (D / 4), cc = (i % (D / 4)) * 4;
      const bool in = rt[r] >= 0;
      const int t = in ? rt[r] : 0;
      odd |= four(q + row_off(a.sq, b, rh[r], t) + cc, in, qs + r * D + cc);
      odd |= four(d_o + row_off(sdo, b, rh[r], t) + cc, in, gs + r * D + cc);
    }
    // rows with inf or NaN: 0 times them is not 0, so they leave out the keys they do not see
    const bool careful = __syncthreads_or(odd);
    {  // warp wp takes rows 4 wp .. 4 wp + 3, lane takes a key
      float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int e = 0; e < D; e += 4) {
        const float4 kv = *reinterpret_cast<const float4*>(Ks + lane * Dp + e);
        const float4 vv = *reinterpret_cast<const float4*>(Vs + lane * Dp + e);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 x = *reinterpret_cast<const float4*>(qs + (4 * wp + r) * D + e);
          const float4 y = *reinterpret_cast<const float4*>(gs + (4 * wp + r) * D + e);
          s[r] = fmaf(x.x, kv.x, fmaf(x.y, kv.y, fmaf(x.z, kv.z, fmaf(x.w, kv.w, s[r]))));
          dp[r] = fmaf(y.x, vv.x, fmaf(y.y, vv.y, fmaf(y.z, vv.z, fmaf(y.w, vv.w, dp[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 4 * wp + r;
        float P = 0.f, dS = 0.f;
        if (rt[row] >= 0 && lane < nk && k0 + lane <= pos0 + rt[row] && rl[row] != -INFINITY) {
          P = expf(s[r] * a.scale - rl[row]);
          dS = P * (dp[r] - rd[row]) * a.scale;
        }
        ps[row * 36 + lane] = P;
        ds[row * 36 + lane] = dS;
      }
    }
    __syncthreads();
#pragma unroll 4
    for (int r = 0; r < kKvRows; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(qs + r * D + c);
      const float4 y = *reinterpret_cast<const float4*>(gs + r * D + c);
#pragma unroll
      for (int u = 0; u < NA; ++u) {
        if (careful && k0 + ks + u > pos0 + rt[r]) continue;
        const float w = ds[r * 36 + ks + u], z = ps[r * 36 + ks + u];
        ak[u][0] = fmaf(w, x.x, ak[u][0]); ak[u][1] = fmaf(w, x.y, ak[u][1]);
        ak[u][2] = fmaf(w, x.z, ak[u][2]); ak[u][3] = fmaf(w, x.w, ak[u][3]);
        av[u][0] = fmaf(z, y.x, av[u][0]); av[u][1] = fmaf(z, y.y, av[u][1]);
        av[u][2] = fmaf(z, y.z, av[u][2]); av[u][3] = fmaf(z, y.w, av[u][3]);
      }
    }
  }
  float* o = part + (size_t)blockIdx.x * 2 * 32 * D + c;
#pragma unroll
  for (int u = 0; u < NA; ++u) {
    *reinterpret_cast<float4*>(o + (ks + u) * D) = make_float4(ak[u][0], ak[u][1], ak[u][2], ak[u][3]);
    *reinterpret_cast<float4*>(o + (32 + ks + u) * D) = make_float4(av[u][0], av[u][1], av[u][2], av[u][3]);
  }
}

template <typename Tin>
static cudaError_t launch_kv(const BlkArgs& a, const BlkPlan& pl, const void* q, const void* k,
                             const void* v, const float* lse, const void* d_o, const float* delta,
                             float* part, const sdm_strides& sdo, cudaStream_t s) {
  const long long grid = (long long)a.B * a.G * pl.most * (a.bs / 32);
  if (grid >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const int smem = int(blk_kv_smem(a.d)), es = int(sizeof(Tin));
  const int vec = view_aligned(q, a.sq, es, 4 * es) && view_aligned(k, a.sk, es, 4 * es) &&
                  view_aligned(v, a.sv, es, 4 * es) && view_aligned(d_o, sdo, es, 4 * es);
  auto go = [&](auto dd) -> cudaError_t {
    constexpr int D = decltype(dd)::value;
    cudaError_t e = cudaFuncSetAttribute(k_blk_kv<Tin, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    launch_after(k_blk_kv<Tin, D>, unsigned(grid), kKvThreads, smem, s,
        a, pl, (const Tin*)q, (const Tin*)k, (const Tin*)v, lse, (const Tin*)d_o, delta, part, sdo, vec);
    return cudaGetLastError();
  };
  if (a.d == 32) return go(std::integral_constant<int, 32>());
  if (a.d == 64) return go(std::integral_constant<int, 64>());
  return go(std::integral_constant<int, 128>());
}

// Workspace: do.o, the plan, the items' parts.  Items of 64 rows while there are few,
// longer ones past 4096 of them, so that the parts stay below 256 MB or so.
static BlkBwdWs blk_simt_ws(const sdm_block_dims* d, void* base) {
  BlkBwdWs w;
  memset(&w, 0, sizeof(w));
  long long rows = (long long)d->B * d->H * d->Tq * d->n_sel / 4096;
  rows = rows < 64 ? 64 : rows > (1 << 20) ? (1 << 20) : (rows + 7) / 8 * 8;
  char* b = static_cast<char*>(base);
  size_t o = (size_t(d->B) * d->H * d->Tq * 4 + 255) & ~size_t(255);
  w.delta = reinterpret_cast<float*>(b);
  w.plan = blk_plan(d, d->Tq, int(rows), b + o);
  o += w.plan.bytes;
  w.kv = reinterpret_cast<float*>(b + o);
  w.bytes = o + size_t(d->B) * d->G * w.plan.most * d->block * 2 * d->d * 4;
  return w;
}

}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_block_backward_workspace_bytes(const sdm_block_dims* dims) {
  if (blk_check(dims) != SDM_OK) return 0;
  size_t n = blk_simt_ws(dims, nullptr).bytes;
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
  const BlkBwdWs w = blk_simt_ws(dims, workspace);
  const bool bf = dims->in_dtype == SDM_DTYPE_BF16;
  cudaError_t e = launch_blk_row_bwd(a, bf, q, k, v, idx, o, lse, d_o, w.delta, dq, gv->o, gv->q, s);
  if (e == cudaSuccess) e = launch_blk_plan(a, w.plan, idx, s);
  if (e == cudaSuccess)
    e = bf ? launch_kv<__nv_bfloat16>(a, w.plan, q, k, v, lse, d_o, w.delta, w.kv, gv->o, s)
           : launch_kv<float>(a, w.plan, q, k, v, lse, d_o, w.delta, w.kv, gv->o, s);
  if (e == cudaSuccess) e = launch_blk_dkv(a, w, bf, dk, dv, gv->k, gv->v, 32, true, true, s);
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
