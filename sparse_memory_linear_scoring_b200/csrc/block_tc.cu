// block_tc.cu -- the tiles of block-selected attention's forward pass on the
// fifth-generation tensor cores (bf16).  block_mma.cu has the plan, the parts and the join.
//
// A CTA holds one block's keys and values and takes an item of the rows (query that
// lists the block, head of the group), 128 at a time, one row to a thread:
//   gather the rows' queries (cp.async into the 128-byte swizzle),
//   S = Q K^T (tcgen05.mma, 128 x BS in TMEM),
//   softmax of the thread's own row from TMEM, P as bf16 over the queries' place,
//   O = P V (tcgen05.mma; V is MN-major as it lies, so nothing is transposed),
//   O over the row's largest element as halves, through shared memory to the parts.
// P is rounded to bf16 for its product, the sum that divides it is of the unrounded weights in
// float32: o is 0.0021 of its norm off, where the result's rounding alone makes 0.0017.
// The products take a few percent of the time.  What bounds a tile is the softmax, the
// conversion of O, the gather and the way out, 47 warp instructions a row (warp-level
// fragments, where four lanes share each row's maxima and sums and every operand goes
// through registers, took 65), and a chain of four waits: 3 CTAs an SM (at d = 128, by
// shared memory) run side by side instead of one with more stages, so the queries' place
// serves P and the outgoing rows, and S and O share TMEM columns.
// 8192 tokens, 2 sequences, 16 heads of 128 on 4, 16 blocks of 64: 397 us, of which the
// 1.1 GB of parts take about 80; two threads a row (24 warps an SM for 12) took 486, a bulk
// copy for each outgoing row 444, paired float32 instructions 465 (register moves).
#include <cuda_fp16.h>

#include "block_internal.cuh"
#include "mma_dev.cuh"
#include "tc_dev.cuh"

namespace sdm {

constexpr int kTcRows = 128;

template <int D, int BS>
struct TcTile {
  static constexpr int PD = (D + 63) / 64;              // panels of 64 columns of Q, K, V
  static constexpr int PB = (BS + 63) / 64;             // panels of P
  static constexpr uint32_t KV = uint32_t(PD) * BS * 128;  // bytes of K, of V
  static constexpr uint32_t OP = 2 * D + 16;            // pitch of an outgoing row
  static constexpr uint32_t q_bytes = uint32_t(PD) * kTcRows * 128;
  static constexpr uint32_t p_bytes = uint32_t(PB) * kTcRows * 128;
  static constexpr uint32_t o_bytes = kTcRows * OP;
  static constexpr uint32_t W0 = q_bytes > p_bytes ? q_bytes : p_bytes;
  static constexpr uint32_t WORK = ((W0 > o_bytes ? W0 : o_bytes) + 1023) & ~1023u;
  static constexpr uint32_t smem = 2 * KV + WORK + 64 + 1024;  // barriers, flags; base aligned to 1024
  static constexpr int COLS = (D > BS ? D : BS) <= 32 ? 32 : (D > BS ? D : BS) <= 64 ? 64 : 128;  // of TMEM
};

// tcgen05.ld of 32 columns of the thread's row, without waiting.
__device__ __forceinline__ void tmem_row32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Byte offset of 16-byte piece c of row r in panels of `rows` rows (128-byte swizzle).
__device__ __forceinline__ uint32_t swz(int r, int c, int rows) {
  return uint32_t((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int D, int BS>
__global__ void __launch_bounds__(kTcRows, D == 128 ? (BS == 128 ? 2 : 3) : (BS == 128 ? 3 : 4))
k_blk_tc(BlkArgs a, BlkFwdWs w, const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
         const __nv_bfloat16* __restrict__ v) {
  wait_for_previous();
  using L = TcTile<D, BS>;
  extern __shared__ unsigned char raw0[];
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int bg = blockIdx.x / w.plan.most, it = blockIdx.x - bg * w.plan.most;
  const int b = bg / a.G, grp = bg - b * a.G;
  const int* item = w.plan.item + (size_t)bg * (a.nb + 1);
  const int j = blk_of_item(item, a.nb, it);
  if (j < 0) return;
  unsigned char* raw = raw0 + ((1024 - (smem_u32(raw0) & 1023)) & 1023);
  unsigned char* work = raw + 2 * L::KV;  // queries, then P, then outgoing rows
  uint64_t* bars = reinterpret_cast<uint64_t*>(work + L::WORK);  // S done, O done
  uint32_t* odd = reinterpret_cast<uint32_t*>(bars + 2);         // [4] keys with inf or NaN values
  uint32_t* tslot = odd + 4;
  volatile int* gave_up = reinterpret_cast<volatile int*>(tslot + 1);
  const uint32_t aK = smem_u32(raw), aV = aK + L::KV, aW = aV + L::KV;
  const int* first = w.plan.first + (size_t)bg * (a.nb + 1);
  const int e0 = first[j], rows = (first[j + 1] - e0) * a.R;
  const int r0 = (it - item[j]) * w.plan.rows, r1 = min(r0 + w.plan.rows, rows);
  const int* entry = w.plan.entry + (size_t)bg * a.nq * a.n_sel + e0;
  const int pos0 = blk_pos0(a, b);
  const int k0 = j * BS, len = pos0 + a.Tq;  // keys at or past len are not read

  if (tid < 4) odd[tid] = 0;
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
#pragma unroll 4
  for (int i = tid; i < BS * (D / 8); i += kTcRows) {
    const int kk = i / (D / 8), c = i % (D / 8);
    const bool in = k0 + kk < len;
    const int at = in ? k0 + kk : 0;
    const uint32_t o = swz(kk, c, BS);
    cp_async16(aK + o, k + row_off(a.sk, b, grp, at) + 8 * c, in);
    cp_async16(aV + o, v + row_off(a.sv, b, grp, at) + 8 * c, in);
  }
  // the thread's row of a tile: the keys it sees, its part's place, its query.  peek sends
  // for the row's list entry, look makes something of it when it has arrived.
  int keys, en, ee = 0;
  size_t place;
  unsigned long long src;
  auto peek = [&](int row) {
    en = row < r1 ? a.by_R.div(row) : -1;
    if (en >= 0) ee = entry[en];
  };
  auto look = [&](int row) {
    const bool in = en >= 0;
    const int r = in ? row - en * a.R : 0, e = in ? ee : 0;
    const int t = a.q0 + a.by_sel.div(e);
    keys = in ? min(BS, pos0 + t - k0 + 1) : 0;
    place = ((size_t)bg * a.nq * a.n_sel + e) * a.R + r;
    src = reinterpret_cast<unsigned long long>(q + row_off(a.sq, b, grp * a.R + r, t));
  };
  auto gather = [&](int base) {  // consecutive lanes take consecutive pieces of a row
#pragma unroll
    for (int i = lane; i < 32 * (D / 8); i += 32) {
      const int rr = i / (D / 8), c = i % (D / 8);
      const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, src, rr));
      cp_async16(aW + swz(32 * wp + rr, c, kTcRows), p + 8 * c, base + 32 * wp + rr < r1);
    }
    cp_async_commit();
  };
  peek(r0 + tid);
  look(r0 + tid);
  gather(r0);
  cp_async_wait<0>();
  __syncthreads();
  // A masked weight is 0, but 0 times an infinite or NaN value is not: such values are
  // taken out of the tile and added, by hand, to the rows that see their key.
  for (int i = tid; i < BS * (D / 8); i += kTcRows) {
    const int kk = i / (D / 8);
    uint4* pv = reinterpret_cast<uint4*>(raw + L::KV + swz(kk, i % (D / 8), BS));
    uint4 u = *pv;
    uint32_t* x = reinterpret_cast<uint32_t*>(&u);
    bool bad = false;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const bool lo = (x[z] & 0x7f80u) == 0x7f80u, hi = (x[z] & 0x7f800000u) == 0x7f800000u;
      bad |= lo || hi;
      if (lo) x[z] &= 0xffff0000u;
      if (hi) x[z] &= 0x0000ffffu;
    }
    if (bad) {
      *pv = u;
      atomicOr(&odd[kk >> 5], 1u << (kk & 31));
    }
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t trow = tmem + (uint32_t(32 * wp) << 16);
  const uint32_t anyodd = odd[0] | odd[1] | odd[2] | odd[3];
  __half* part = static_cast<__half*>(w.part);
  const float c2 = fmaxf(fabsf(a.scale) * kLog2e, 1.1754944e-38f);  // masked scores stay -inf at scale 0
  constexpr uint32_t idS = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(BS >> 3) << 17) | (uint32_t(kTcRows >> 4) << 24);
  constexpr uint32_t idO = (1u << 4) | (1u << 7) | (1u << 10) | kBMajorMN | (uint32_t(D >> 3) << 17) |
                           (uint32_t(kTcRows >> 4) << 24);

  uint32_t parity = 0;
  for (int base = r0; base < r1; base += kTcRows, parity ^= 1) {
    if (tid == 0) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16(tmem, sdesc(aW + (kk >> 2) * (kTcRows * 128) + (kk & 3) * 32),
                  sdesc(aK + (kk >> 2) * (BS * 128) + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
      umma_commit(&bars[0]);
    }
    if (base + kTcRows < r1) peek(base + kTcRows + tid);  // the next tile's rows
    mbar_wait(&bars[0], parity, gave_up);
    tc_fence_after();
    float l = 0.f, m = -INFINITY;
    {
      float sc[BS];
#pragma unroll
      for (int c = 0; c < BS; c += 32) tmem_row32(trow + c, sc + c);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      if (a.scale < 0.f) {
#pragma unroll
        for (int c = 0; c < BS; ++c) sc[c] = -sc[c];
      }
      if (__any_sync(0xffffffffu, keys < BS)) {  // rows of the block's own queries, or none
#pragma unroll
        for (int c = 0; c < BS; ++c)
          if (c >= keys) sc[c] = -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < BS; c += 2) m = fmaxf(m, fmaxf(sc[c], sc[c + 1]));
      m = m == -INFINITY ? 0.f : m * c2;
#pragma unroll
      for (int c = 0; c < BS; c += 8) {
        uint32_t u[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float x = ex2(fmaf(sc[c + 2 * z], c2, -m)), y = ex2(fmaf(sc[c + 2 * z + 1], c2, -m));
          l += x + y;
          u[z] = pack_bf16(x, y);
        }
        *reinterpret_cast<uint4*>(work + swz(tid, c >> 3, kTcRows)) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();  // P is in place, S has been read
    if (tid == 0) {
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < BS / 16; ++kk)
        umma_bf16(tmem, sdesc(aW + (kk >> 2) * (kTcRows * 128) + (kk & 3) * 32),
                  sdesc_mn(aV + kk * 2048, BS * 128), idO, kk > 0 ? 1u : 0u);
      umma_commit(&bars[1]);
    }
    mbar_wait(&bars[1], parity, gave_up);
    tc_fence_after();
    float acc[D];
#pragma unroll
    for (int c = 0; c < D; c += 32) tmem_row32(trow + c, acc + c);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    if (anyodd) {
      // P lies where the outgoing rows go: the thread's own row only is read and written
#pragma unroll 1
      for (int z = 0; z < BS / 32; ++z) {
        uint32_t todo = odd[z];
        while (todo) {
          const int key = 32 * z + __ffs(todo) - 1;
          todo &= todo - 1;
          if (key >= keys) continue;
          const float p = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
              work + swz(tid, key >> 3, kTcRows) + (key & 7) * 2));
          const __nv_bfloat16* vr = v + row_off(a.sv, b, grp, k0 + key);
#pragma unroll
          for (int c = 0; c < D; c += 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(vr + c);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              if ((x[y] & 0x7f80u) == 0x7f80u) acc[c + 2 * y] = fmaf(p, bf16_lo(x[y]), acc[c + 2 * y]);
              if ((x[y] & 0x7f800000u) == 0x7f800000u) acc[c + 2 * y + 1] = fmaf(p, bf16_hi(x[y]), acc[c + 2 * y + 1]);
            }
          }
        }
      }
      __syncthreads();  // every row of P has been read
    }
    float xm = 0.f;
#pragma unroll
    for (int c = 0; c < D; c += 2) xm = fmaxf(xm, fmaxf(fabsf(acc[c]), fabsf(acc[c + 1])));
    if (xm == INFINITY) {  // the largest finite one
      xm = 0.f;
#pragma unroll
      for (int c = 0; c < D; ++c)
        if (fabsf(acc[c]) < INFINITY) xm = fmaxf(xm, fabsf(acc[c]));
    }
    xm = fmaxf(xm, 7.7037198e-34f);  // 2^-110: the factor stays finite
    // the largest becomes 2^15: halves keep all their bits down to 2^-29 of it
    const float f = 32768.f / xm;
    unsigned char* orow = work + tid * L::OP;
#pragma unroll
    for (int c = 0; c < D; c += 8) {
      uint32_t u[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const __half2 hh = __floats2half2_rn(acc[c + 2 * z] * f, acc[c + 2 * z + 1] * f);
        u[z] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      *reinterpret_cast<uint4*>(orow + 2 * c) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    if (base + tid < r1) {
      // a wait that ran out poisons the row
      float2 ml = l == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(m + log2f(l), xm * (1.f / 32768.f) / l);
      if (*gave_up) ml = make_float2(NAN, NAN);
      w.ml[place] = ml;
    }
    __syncwarp();
    // the warp's rows go out with consecutive lanes on consecutive pieces (a bulk copy a row
    // took 2200 cycles a tile, 64 a copy)
    constexpr int NW = 4;  // pieces read together (one: 423 us at the case above, four 397, eight 423)
#pragma unroll
    for (int i0 = 0; i0 < D / 8; i0 += NW) {
      uint4 u[NW];
#pragma unroll
      for (int z = 0; z < NW; ++z) {
        const int i = lane + 32 * (i0 + z), rr = i / (D / 8), c = i % (D / 8);
        u[z] = *reinterpret_cast<const uint4*>(work + (32 * wp + rr) * L::OP + 16 * c);
      }
#pragma unroll
      for (int z = 0; z < NW; ++z) {
        const int i = lane + 32 * (i0 + z), rr = i / (D / 8), c = i % (D / 8);
        const size_t to = __shfl_sync(0xffffffffu, place, rr);
        if (base + 32 * wp + rr < r1) *reinterpret_cast<uint4*>(part + to * D + 8 * c) = u[z];
      }
    }
    if (base + kTcRows < r1) {
      look(base + kTcRows + tid);
      tc_fence_before();
      __syncthreads();  // the outgoing rows and O have been read
      gather(base + kTcRows);
      cp_async_wait<0>();
      fence_async_smem();
      __syncthreads();  // the queries are in place
      tc_fence_after();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (wp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::COLS) : "memory");
  }
}

template <int D, int BS>
static cudaError_t launch_tc(const BlkArgs& a, const BlkFwdWs& w, unsigned grid, const void* q, const void* k,
                             const void* v, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const int sm = int(TcTile<D, BS>::smem);
  const cudaError_t e = cudaFuncSetAttribute(k_blk_tc<D, BS>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
  if (e != cudaSuccess) return e;
  launch_after(k_blk_tc<D, BS>, grid, kTcRows, sm, s, a, w, (const bf*)q, (const bf*)k, (const bf*)v);
  return cudaGetLastError();
}

cudaError_t launch_blk_tc(const BlkArgs& a, const BlkFwdWs& w, unsigned grid, const void* q, const void* k,
                          const void* v, cudaStream_t s) {
#define SDM_BLK_TC(D_, BS_) if (a.d == D_ && a.bs == BS_) return launch_tc<D_, BS_>(a, w, grid, q, k, v, s)
  SDM_BLK_TC(32, 32); SDM_BLK_TC(32, 64); SDM_BLK_TC(32, 128);
  SDM_BLK_TC(64, 32); SDM_BLK_TC(64, 64); SDM_BLK_TC(64, 128);
  SDM_BLK_TC(128, 32); SDM_BLK_TC(128, 64); SDM_BLK_TC(128, 128);
#undef SDM_BLK_TC
  return cudaErrorInvalidValue;
}

}  // namespace sdm
