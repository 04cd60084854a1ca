// seq_internal.cuh -- shared pieces of the sequence operators (conv.cu, ssm.cu,
// ssm_bwd.cu, block_*.cu): strided [B][H][T][d] views, argument checks, and the
// warp-level tensor-core helpers.
#pragma once

#include <string.h>

#include <initializer_list>

#include "sdm_internal.cuh"

namespace sdm {

constexpr float kLog2e = 1.4426950408889634f;

// Offset of row (b, h, t) of a strided view (elements, 64 bits throughout).
__host__ __device__ __forceinline__ long long row_off(const sdm_strides& s, int b, int h, int t) {
  return (long long)b * s.b + (long long)h * s.h + (long long)t * s.t;
}

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// V consecutive elements as floats / back (V * sizeof(T) <= 16 bytes, aligned to it).
template <typename T, int V>
struct Vec {
  static __device__ __forceinline__ void load(const T* p, float* f) {
    if constexpr (V == 1) {
      f[0] = to_f32(*p);
    } else if constexpr (V == 2 && sizeof(T) == 4) {
      const float2 v = *reinterpret_cast<const float2*>(p);
      f[0] = v.x; f[1] = v.y;
    } else if constexpr (V == 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
      f[0] = __uint_as_float(u << 16); f[1] = __uint_as_float(u & 0xffff0000u);
    } else if constexpr (sizeof(T) == 4) {
      static_assert(sizeof(T) != 4 || V == 4, "float vectors are 2 or 4 wide");
      const float4 v = *reinterpret_cast<const float4*>(p);
      f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else if constexpr (V == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
      f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float* f) {
    if constexpr (V == 1) {
      *p = from_f32<T>(f[0]);
    } else if constexpr (V == 2 && sizeof(T) == 4) {
      *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
      uint32_t u[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
      else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
      else *reinterpret_cast<uint32_t*>(p) = u[0];
    }
  }
};

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether a view can be read in `bytes`-wide pieces along its last axis.
inline bool view_aligned(const void* p, const sdm_strides& s, int esize, size_t bytes) {
  const long long m = (long long)(bytes / esize);
  return aligned_to(p, bytes) && s.b % m == 0 && s.h % m == 0 && s.t % m == 0;
}

// A pointer that has to be there, aligned to its element.
inline int need_ptr(const void* p, size_t a) {
  if (!p) return SDM_ERR_NULL;
  return aligned_to(p, a) ? SDM_OK : SDM_ERR_ALIGN;
}

// Strides of an input view: an axis may be broadcast (stride 0) or reversed in
// nothing; outputs need rows that cannot overlap, which the caller vouches for.
inline bool strides_ok(const sdm_strides* s) {
  return s && s->b >= 0 && s->h >= 0 && s->t >= 0 && s->b < (1LL << 45) && s->h < (1LL << 45) &&
         s->t < (1LL << 45);
}

__device__ __forceinline__ int seq_len(const int32_t* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// Kernels that follow one another closely are launched while the one before them ends
// (programmatic stream serialization) and wait for it here, as their first statement,
// until it is complete and its writes are visible: about 1 us less a launch, 27 -> 20 us
// for the selection and attention of 64 single tokens.  No kernel lets the next one in
// before it ends: CTAs that wait beside a running kernel cost it 1% to 15%.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c;
  memset(&c, 0, sizeof(c));
  cudaLaunchAttribute at;
  memset(&at, 0, sizeof(at));
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = grid;
  c.blockDim = dim3(unsigned(threads));
  c.dynamicSmemBytes = size_t(smem);
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// 2^x on the special function unit; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

}  // namespace sdm
