// mma_dev.cuh -- warp-level tensor-core helpers of the sequence operators:
// m16n8k16 products of bf16 with float32 sums, ldmatrix, cp.async, and splits of
// float32 values into bf16 parts.
//
// Fragments of a 16 x 8 x 16 product in lane l (g = l / 4, q = l % 4):
//   A (4 registers): rows g, g + 8; columns 2q, 2q + 1 and 8 + 2q, 8 + 2q + 1
//     (a0: row g low columns, a1: row g + 8 low, a2: row g high, a3: row g + 8 high);
//   B (2 registers): column g; rows 2q, 2q + 1 and 8 + 2q, 8 + 2q + 1;
//   C (4 floats): c0, c1 row g, columns 2q, 2q + 1; c2, c3 row g + 8.
#pragma once

#include "seq_internal.cuh"

namespace sdm {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
               "{%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Addresses of ldsm4 / ldsm4t lanes inside a bf16 tile with row pitch ld (elements):
// A of rows r0.. and columns c0.. stored as rows (ldsm4),
__device__ __forceinline__ int frag_a(int lane, int r0, int c0, int ld) {
  return (r0 + (lane & 15)) * ld + c0 + (lane >> 4) * 8;
}
// A stored transposed, tile[column][row] (ldsm4t),
__device__ __forceinline__ int frag_at(int lane, int r0, int c0, int ld) {
  return (c0 + ((lane >> 4) << 3) + (lane & 7)) * ld + r0 + ((lane >> 3) & 1) * 8;
}
// B of two neighbouring column tiles n0, n0 + 8 and rows k0.. stored as
// tile[column][row] (ldsm4): registers 0, 1 the first tile, 2, 3 the second,
__device__ __forceinline__ int frag_b(int lane, int n0, int k0, int ld) {
  return (n0 + ((lane >> 4) << 3) + (lane & 7)) * ld + k0 + ((lane >> 3) & 1) * 8;
}
// and stored as tile[row][column] (ldsm4t).
__device__ __forceinline__ int frag_bt(int lane, int n0, int k0, int ld) {
  return (k0 + (lane & 15)) * ld + n0 + (lane >> 4) * 8;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// x = part 0 + part 1 (+ part 2) + rest, each part the bf16 nearest to what the parts
// before it left, so the rest is at most 2^-8 of x per part (2: 2^-16, 3: 2^-24).
template <int PARTS>
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t (&u)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    u[i] = pack_bf16(a, b);
    a -= bf16_lo(u[i]);
    b -= bf16_hi(u[i]);
  }
}

// Whether bf16 pieces of 16 bytes in shared memory hold an infinity or NaN: 0 times them is
// added up, in four sums that stay 0 otherwise.
struct OddBf16 {
  __nv_bfloat162 z[4];
  __device__ __forceinline__ OddBf16() {
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = __float2bfloat162_rn(0.f);
  }
  __device__ __forceinline__ void add(const __nv_bfloat16* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z[i] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), __float2bfloat162_rn(0.f), z[i]);
  }
  __device__ __forceinline__ bool any() const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(z);
    return (u[0] | u[1] | u[2] | u[3]) != 0u;
  }
};

// 16 bytes global -> shared; `in` false writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace sdm
