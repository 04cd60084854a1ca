// ssm_tc.cu -- the selective scan's first walk on the fifth-generation tensor cores (bf16,
// d_k = 128): each segment's own contribution to the state,
//     F = sum_j w_j x_j B_j^T,   w_j = dt_j exp(sum of dt A over the segment's later steps).
//
// F^T [n][p] is a sum of products B^T (w x): the chunk's B, as it lies, is the MN-major A
// operand of 128 rows, and w x, split by the threads into three bf16 parts (F is a float32
// result; what is left is below 2^-24), the MN-major B operand.  The chunks are taken from
// the last to the first, so that w needs no decay of F, only a running sum.  Twelve products
// of 128 x d_v x 16 a chunk go to one of two TMEM buffers, and the other is drained into
// float32 registers meanwhile: sums over chunks there round to nearest, where hundreds of
// accumulations in the tensor core would truncate one way.  65536 steps of 8 heads of
// 128 x 128: 96 us (warp-level products: 178), 3200 cycles a chunk, of which the products
// need about 770; the threads' split (65 instructions for 8 elements), the single
// thread's 12 issues and the drain follow one another.  Loads two chunks ahead (101 us) or
// 512 threads (103) do not help.
#include "mma_dev.cuh"
#include "ssm_internal.cuh"
#include "tc_dev.cuh"

namespace sdm {

constexpr int kSegThreads = 256;
constexpr uint32_t kAMajorMN = 1u << 15;  // instruction descriptor: A is MN-major

template <int P>
struct SegTile {
  static constexpr uint32_t BB = 2 * kSsmQT * 128;               // B: two panels of 64 columns
  static constexpr uint32_t XB = uint32_t(P / 64) * kSsmQT * 128;  // one part of w x
  static constexpr uint32_t STAGE = BB + 3 * XB;
  static constexpr uint32_t smem = 2 * STAGE + 2 * kSsmQT * 4 + 64 + 1024;
  static constexpr int COLS = 2 * P;                             // two buffers of F^T
};

__device__ __forceinline__ void tmem_cols16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <int P>
__global__ void __launch_bounds__(kSegThreads)
k_ssm_seg(SsmArgs a, const __nv_bfloat16* __restrict__ x, const float* __restrict__ dt,
          const float* __restrict__ A, const __nv_bfloat16* __restrict__ Bm,
          const int32_t* __restrict__ lengths, float* __restrict__ segS, float* __restrict__ segG) {
  wait_for_previous();
  using L = SegTile<P>;
  constexpr int N = 128, Q = kSsmQT;
  extern __shared__ unsigned char raw0[];
  unsigned char* raw = raw0 + ((1024 - (smem_u32(raw0) & 1023)) & 1023);
  float* wj = reinterpret_cast<float*>(raw + 2 * L::STAGE);        // [2][64]
  uint64_t* bars = reinterpret_cast<uint64_t*>(wj + 2 * Q);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 2);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tslot + 1);
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, quad = wp & 3, half = wp >> 2;
  const int seg = blockIdx.x % a.nseg, bh = blockIdx.x / a.nseg;
  const int b = bh / a.H, h = bh - b * a.H, gr = h / a.hg;
  const int T = seq_len(lengths, b, a.T);
  const int c0 = seg * a.cps, c1 = min(c0 + a.cps, a.nch);
  if (tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (wp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                 "n"(L::COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the chunk's pieces of 8 elements, one chunk ahead: NX of x and 4 of B a thread
  constexpr int NX = Q * (P / 8) / kSegThreads, NB = Q * (N / 8) / kSegThreads;
  uint4 px[NX], pb[NB];
  auto ahead = [&](int c) {
    const int t0 = c * Q;
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int e = tid + i * kSegThreads, t = e / (P / 8), col = (e % (P / 8)) * 8;
      px[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c >= c0 && t0 + t < T) px[i] = *reinterpret_cast<const uint4*>(x + row_off(a.sx, b, h, t0 + t) + col);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int e = tid + i * kSegThreads, t = e / (N / 8), col = (e % (N / 8)) * 8;
      pb[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c >= c0 && t0 + t < T) pb[i] = *reinterpret_cast<const uint4*>(Bm + row_off(a.sB, b, gr, t0 + t) + col);
    }
  };
  // weights of a chunk, by warp 0: steps 2 lane, 2 lane + 1; `later`: log2 decay behind it
  const double al = double(A[h]) * 1.4426950408889634074;
  double later = 0.0;
  float d0 = 0.f, d1 = 0.f;
  auto steps = [&](int c) {
    const int t = c * Q + 2 * lane;
    d0 = c >= c0 && t < T ? dt[row_off(a.sdt, b, h, t)] : 0.f;
    d1 = c >= c0 && t + 1 < T ? dt[row_off(a.sdt, b, h, t + 1)] : 0.f;
  };
  auto weights = [&](float* w) {
    const double v0 = double(d0) * al, v1 = double(d1) * al;
    double inc = v0 + v1;  // suffix sums over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double u = __shfl_down_sync(0xffffffffu, inc, o);
      if (lane + o < 32) inc += u;
    }
    const double ex = inc - (v0 + v1);  // behind step 2 lane + 1
    w[2 * lane] = d0 * ex2(float(later + ex + v1));
    w[2 * lane + 1] = d1 * ex2(float(later + ex));
    later += __shfl_sync(0xffffffffu, inc, 0);
  };
  ahead(c1 - 1);
  if (wp == 0) {
    steps(c1 - 1);
    weights(wj);
    steps(c1 - 2);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  constexpr uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | kAMajorMN | kBMajorMN | (uint32_t(P >> 3) << 17) |
                          (uint32_t(N >> 4) << 24);
  constexpr int PH = P / 2;  // columns p of the thread, row n = 32 quad + lane
  float F[PH];
#pragma unroll
  for (int e = 0; e < PH; ++e) F[e] = 0.f;
  auto drain = [&](int s, uint32_t parity) {
    mbar_wait(&bars[s], parity, gave_up);
    tc_fence_after();
#pragma unroll
    for (int e = 0; e < PH; e += 16) {
      uint32_t r[16];
      tmem_cols16(tmem + (uint32_t(32 * quad) << 16) + s * P + half * PH + e, r);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int u = 0; u < 16; ++u) F[e + u] += __uint_as_float(r[u]);
    }
    tc_fence_before();
  };

  const int n = c1 - c0;
  for (int i = 0; i < n; ++i) {  // chunk c1 - 1 - i; its stage was last read by chunk i - 2, drained
    const int s = i & 1;
    const uint32_t st = smem_u32(raw) + s * L::STAGE;
    unsigned char* sp = raw + s * L::STAGE;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int e = tid + k * kSegThreads, t = e / (N / 8), col = e % (N / 8);
      *reinterpret_cast<uint4*>(sp + (col >> 3) * (Q * 128) + t * 128 + (((col & 7) ^ (t & 7)) << 4)) = pb[k];
    }
#pragma unroll
    for (int k = 0; k < NX; ++k) {
      const int e = tid + k * kSegThreads, t = e / (P / 8), col = e % (P / 8);
      const float w = wj[s * Q + t];
      const uint32_t u[4] = {px[k].x, px[k].y, px[k].z, px[k].w};
      uint32_t o[3][4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t z[3];
        split_bf16<3>(bf16_lo(u[y]) * w, bf16_hi(u[y]) * w, z);
        o[0][y] = z[0]; o[1][y] = z[1]; o[2][y] = z[2];
      }
      unsigned char* to = sp + L::BB + (col >> 3) * (Q * 128) + t * 128 + (((col & 7) ^ (t & 7)) << 4);
#pragma unroll
      for (int z = 0; z < 3; ++z)
        *reinterpret_cast<uint4*>(to + z * L::XB) = make_uint4(o[z][0], o[z][1], o[z][2], o[z][3]);
    }
    if (i + 1 < n) {
      ahead(c1 - 2 - i);
      if (wp == 0) {
        weights(wj + (s ^ 1) * Q);
        steps(c1 - 3 - i);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();  // the stage is filled, buffer s has been drained
    if (tid == 0) {
      tc_fence_after();
#pragma unroll
      for (int z = 2; z >= 0; --z)  // small parts first
#pragma unroll
        for (int kk = 0; kk < Q / 16; ++kk)
          umma_bf16(tmem + s * P, sdesc_mn(st + kk * 2048, Q * 128),
                    sdesc_mn(st + L::BB + z * L::XB + kk * 2048, Q * 128), id, z < 2 || kk > 0 ? 1u : 0u);
      umma_commit(&bars[s]);
    }
    if (i > 0) drain(s ^ 1, ((i - 1) >> 1) & 1);
  }
  if (n > 0) drain((n - 1) & 1, ((n - 1) >> 1) & 1);
  float* slot = segS + (size_t(bh) * a.nseg + seg) * P * N + 32 * quad + lane;
  const float bad = *gave_up ? NAN : 0.f;  // a wait that ran out poisons the state
  bool odd = false;
#pragma unroll
  for (int e = 0; e < PH; ++e) odd |= !(fabsf(F[e]) < INFINITY);
  if (odd) {  // inf or NaN among the inputs: the recurrence itself
#pragma unroll
    for (int e = 0; e < PH; ++e) F[e] = 0.f;
    const float Ah = A[h];
#pragma unroll 1
    for (int t = c0 * Q; t < min(c1 * Q, T); ++t) {
      const float d = dt[row_off(a.sdt, b, h, t)], at = expf(d * Ah);
      const float u = d * __bfloat162float(Bm[row_off(a.sB, b, gr, t) + 32 * quad + lane]);
      const __nv_bfloat16* xr = x + row_off(a.sx, b, h, t) + half * PH;
#pragma unroll
      for (int e = 0; e < PH; ++e) F[e] = fmaf(at, F[e], u * __bfloat162float(xr[e]));
    }
  }
#pragma unroll
  for (int e = 0; e < PH; ++e) slot[size_t(half * PH + e) * N] = F[e] + bad;
  if (tid == 0) segG[blockIdx.x] = float(later);
  tc_fence_before();
  __syncthreads();
  if (wp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::COLS) : "memory");
  }
}

cudaError_t launch_ssm_seg(const SsmArgs& a, const void* x, const float* dt, const float* A, const void* Bm,
                           const int32_t* lengths, float* segS, float* segG, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const unsigned grid = unsigned(a.B * a.H) * unsigned(a.nseg);
  auto go = [&](auto kernel, int sm) -> cudaError_t {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    if (r != cudaSuccess) return r;
    launch_after(kernel, grid, kSegThreads, sm, s, a, (const bf*)x, dt, A, (const bf*)Bm, lengths, segS, segG);
    return cudaGetLastError();
  };
  return a.P == 64 ? go(k_ssm_seg<64>, int(SegTile<64>::smem)) : go(k_ssm_seg<128>, int(SegTile<128>::smem));
}

}  // namespace sdm
