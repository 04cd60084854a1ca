// block_step.cu -- attention over listed blocks for single tokens and short calls (bf16),
// query by query on the tensor cores.
//
// The up to 16 heads of a group that share a query's list are the rows of one
// 16-row tile, so that a piece of 32 listed keys costs two products of 16 x 32 x d
// however many heads there are, and K and V are read once for all of them: 2 d bytes a
// key each way is what bounds it.  A warp takes pieces of its own, the next one on its
// way (cp.async) while one is computed, with a running maximum and sum; the warps of up
// to 8 CTAs of a cluster share a query and join through distributed shared memory, so
// one launch without a workspace fills the card from few sequences.
// P is rounded to bf16 for its product as in block_tc.cu.
// block_attn.cu has the formulas, and the CUDA-core kernel for views that cannot be read
// in 16-byte pieces; per head and key that one needs about 100 instructions where a tile
// needs 200 a piece in all (64 sequences of up to 4096 keys, 16 heads of 64 on 4: 35 us
// there, 14 here, 4.8 TB/s).
#include <cooperative_groups.h>

#include "block_internal.cuh"
#include "mma_dev.cuh"

namespace sdm {

namespace cg = cooperative_groups;

constexpr int kStepWarps = 4;
constexpr int kStepCluster = 8;
constexpr int kPiece = 32;  // keys

template <int D>
struct StepTile {
  static constexpr int LD = D + 8;
  static constexpr int STAGE = 2 * kPiece * LD;          // K, V
  static constexpr size_t warp = size_t(2) * 2 * STAGE;  // bytes, two stages
  static_assert(warp >= size_t(16) * D * 4 + 128, "a warp's rows and its maxima and sums reuse its stages");
  static constexpr size_t smem = kStepWarps * warp;
};

template <int D>
__global__ void __launch_bounds__(kStepWarps * 32)
k_blk_step(BlkArgs a, const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
           const __nv_bfloat16* __restrict__ v, const int32_t* __restrict__ idx,
           __nv_bfloat16* __restrict__ o, float* __restrict__ lse, int hc, int cs) {
  wait_for_previous();
  using L = StepTile<D>;
  extern __shared__ __align__(16) unsigned char raw[];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, g = lane >> 2, qd = lane & 3;
  __nv_bfloat16* st = reinterpret_cast<__nv_bfloat16*>(raw + wp * L::warp);
  const uint32_t ast = smem_u32(st);
  const int rank = blockIdx.x % cs;
  long long it = blockIdx.x / cs;
  const int ch = int(it % hc); it /= hc;
  const int t = int(it % a.Tq);
  const int bg = int(it / a.Tq), b = bg / a.G, gr = bg - b * a.G;
  const int r0 = ch * 16, nh = min(16, a.R - r0), h0 = gr * a.R + r0;
  const int p = blk_pos0(a, b) + t;
  const int32_t* list = idx + ((size_t)bg * a.Tq + t) * a.n_sel;
  const int per = a.bs / kPiece, pieces = a.n_sel * per, step = cs * kStepWarps;
  const __nv_bfloat16* kb = k + row_off(a.sk, b, gr, 0);
  const __nv_bfloat16* vb = v + row_off(a.sv, b, gr, 0);
  int pc = rank * kStepWarps + wp;
  // the next piece with keys from pc on: its load into a stage, and its keys (0: none left)
  auto fetch = [&](int stage) {
    int n = 0, j = 0, sub = 0;
    for (; pc < pieces && n <= 0; pc += step) {
      const int s = pc / per;
      sub = pc - s * per;
      j = list[s];
      n = min(kPiece, blk_keys(a, j, p) - sub * kPiece);
    }
    if (n > 0) {
      const long long key0 = (long long)j * a.bs + sub * kPiece;
#pragma unroll
      for (int i = lane; i < kPiece * (D / 8); i += 32) {
        const int kk = i / (D / 8), c = (i % (D / 8)) * 8;
        const long long at = kk < n ? key0 + kk : key0;  // keys behind the query are not read
        const uint32_t dst = ast + 2 * (stage * L::STAGE + kk * L::LD + c);
        cp_async16(dst, kb + at * a.sk.t + c, kk < n);
        cp_async16(dst + 2 * kPiece * L::LD, vb + at * a.sv.t + c, kk < n);
      }
    }
    cp_async_commit();
    return max(n, 0);
  };
  int n = fetch(0);
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = g + (i & 1) * 8;
      qf[kk][i] = r < nh ? *reinterpret_cast<const uint32_t*>(
                               q + row_off(a.sq, b, h0 + r, t) + 16 * kk + (i >> 1) * 8 + 2 * qd) : 0u;
    }
  const float c2 = a.scale * kLog2e;
  float acc[D / 8][4], ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
#pragma unroll
  for (int m = 0; m < D / 8; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
  for (int stage = 0; n > 0; stage ^= 1) {
    const int next = fetch(stage ^ 1);
    cp_async_wait<1>();
    __syncwarp();
    const uint32_t ak = ast + 2 * stage * L::STAGE, av = ak + 2 * kPiece * L::LD;
    float sc[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[m][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t bf[4];
        ldsm4(bf, ak + 2 * frag_b(lane, 16 * m, 16 * kk, L::LD));
        mma_bf16(sc[2 * m], qf[kk], bf[0], bf[1]);
        mma_bf16(sc[2 * m + 1], qf[kk], bf[2], bf[3]);
      }
    float xa = ma, xb = mb;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = 8 * m + 2 * qd + i < n;
        sc[m][i] = in ? sc[m][i] * c2 : -INFINITY;
        sc[m][2 + i] = in ? sc[m][2 + i] * c2 : -INFINITY;
        xa = fmaxf(xa, sc[m][i]);
        xb = fmaxf(xb, sc[m][2 + i]);
      }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, w));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, w));
    }
    const float ba = xa == -INFINITY ? 0.f : xa, bb = xb == -INFINITY ? 0.f : xb;
    const float fa = ex2(ma - ba), fb = ex2(mb - bb);  // 0 from the empty start
    ma = xa;
    mb = xb;
    la *= fa;
    lb *= fb;
    uint32_t pf[2][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float x0 = ex2(sc[m][0] - ba), x1 = ex2(sc[m][1] - ba);
      const float x2 = ex2(sc[m][2] - bb), x3 = ex2(sc[m][3] - bb);
      la += x0 + x1;
      lb += x2 + x3;
      pf[m >> 1][(m & 1) * 2] = pack_bf16(x0, x1);
      pf[m >> 1][(m & 1) * 2 + 1] = pack_bf16(x2, x3);
    }
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        acc[2 * m + u][0] *= fa; acc[2 * m + u][1] *= fa;
        acc[2 * m + u][2] *= fb; acc[2 * m + u][3] *= fb;
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t bf[4];
        ldsm4t(bf, av + 2 * frag_bt(lane, 16 * m, 16 * kk, L::LD));
        mma_bf16(acc[2 * m], pf[kk], bf[0], bf[1]);
        mma_bf16(acc[2 * m + 1], pf[kk], bf[2], bf[3]);
      }
    }
    __syncwarp();  // the stage has been read
    n = next;
  }
  cp_async_wait<0>();
  __syncwarp();
  // the warp's rows, maxima and sums over its stages: [16][D], m[16], l[16]
  float* part = reinterpret_cast<float*>(raw + wp * L::warp);
#pragma unroll
  for (int w = 1; w < 4; w <<= 1) {
    la += __shfl_xor_sync(0xffffffffu, la, w);
    lb += __shfl_xor_sync(0xffffffffu, lb, w);
  }
#pragma unroll
  for (int m = 0; m < D / 8; ++m) {
    *reinterpret_cast<float2*>(part + g * D + 8 * m + 2 * qd) = make_float2(acc[m][0], acc[m][1]);
    *reinterpret_cast<float2*>(part + (g + 8) * D + 8 * m + 2 * qd) = make_float2(acc[m][2], acc[m][3]);
  }
  if (qd == 0) {
    part[16 * D + g] = ma;
    part[16 * D + g + 8] = mb;
    part[16 * D + 16 + g] = la;
    part[16 * D + 24 + g] = lb;
  }
  cg::cluster_group cl = cg::this_cluster();
  if (cs > 1) cl.sync(); else __syncthreads();
  // a warp finishes 64 or 128 columns of a row at a time: D / 32 a lane
  constexpr int VC = D / 32;
  for (int r = rank * kStepWarps + wp; r < nh; r += step) {
    float mx = -INFINITY;
    for (int w = 0; w < step; ++w) {
      const float* x = reinterpret_cast<const float*>(raw + (w % kStepWarps) * L::warp);
      if (cs > 1) x = cl.map_shared_rank(x, w / kStepWarps);
      mx = fmaxf(mx, x[16 * D + r]);
    }
    if (mx == -INFINITY) mx = 0.f;
    float sum = 0.f, y[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) y[e] = 0.f;
    for (int w = 0; w < step; ++w) {
      const float* x = reinterpret_cast<const float*>(raw + (w % kStepWarps) * L::warp);
      if (cs > 1) x = cl.map_shared_rank(x, w / kStepWarps);
      const float f = ex2(x[16 * D + r] - mx);
      sum = fmaf(f, x[16 * D + 16 + r], sum);
#pragma unroll
      for (int e = 0; e < VC; ++e) y[e] = fmaf(f, x[r * D + lane * VC + e], y[e]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat16* op = o + row_off(a.so, b, h0 + r, t) + lane * VC;
#pragma unroll
    for (int e = 0; e < VC; ++e) op[e] = __float2bfloat16_rn(y[e] * inv);
    if (lse && lane == 0)
      lse[((size_t)b * a.H + h0 + r) * a.Tq + t] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) / kLog2e;
  }
  if (cs > 1) cl.sync();  // the others may still be reading this CTA's rows
}

// CTAs that share a query: more than one only while they all fit the card at one an SM
// and a warp has two pieces, since launching and joining a cluster costs more than it
// saves elsewhere.  16 blocks of 64, d = 64, 4 groups, clusters of 1 / 2 / 4 / 8:
// 1 sequence 10.3 / 8.0 / 6.7 / 6.9 us, 16 sequences 10.5 / 8.3 / 8.8 / 16.3,
// 64 sequences 14.0 / 20.5 / 25.7 / 47.2; 4 sequences with 64 blocks 33 / 20 / 13 / 11.
template <int D>
static cudaError_t launch_step(const BlkArgs& a, const void* q, const void* k, const void* v,
                               const int32_t* idx, void* o, float* lse, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const int hc = (a.R + 15) / 16, pieces = a.n_sel * (a.bs / kPiece);
  const long long items = (long long)a.B * a.G * a.Tq * hc;
  int cs = 1;
  while (cs < kStepCluster && 2 * items * cs <= 148 && 4 * cs * kStepWarps <= pieces) cs *= 2;
  if (items * cs >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const int sm = int(StepTile<D>::smem);
  cudaError_t e = cudaFuncSetAttribute(k_blk_step<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c;
  memset(&c, 0, sizeof(c));
  cudaLaunchAttribute at[2];
  memset(at, 0, sizeof(at));
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(cs);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_after()
  at[1].val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = dim3(unsigned(items * cs));
  c.blockDim = dim3(kStepWarps * 32);
  c.dynamicSmemBytes = size_t(sm);
  c.stream = s;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, k_blk_step<D>, a, (const bf*)q, (const bf*)k, (const bf*)v, idx, (bf*)o, lse,
                            hc, cs);
}

cudaError_t launch_blk_step(const BlkArgs& a, const void* q, const void* k, const void* v,
                            const int32_t* idx, void* o, float* lse, cudaStream_t s) {
  if (a.d == 32) return launch_step<32>(a, q, k, v, idx, o, lse, s);
  if (a.d == 64) return launch_step<64>(a, q, k, v, idx, o, lse, s);
  return launch_step<128>(a, q, k, v, idx, o, lse, s);
}

}  // namespace sdm
