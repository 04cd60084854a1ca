// block_attn.cu -- attention over listed blocks, query by query on CUDA cores: single
// tokens and short calls whose views block_step.cu does not take, float32 inputs,
// forward and the query's gradient; and the C ABI of the forward pass.
//
//   s_k = scale q.k over the listed keys at positions <= p;  o = sum softmax(s)_k v_k;
//   lse = log sum exp(s_k);  no key: o = 0, lse = -inf.
//   backward: P_k = exp(s_k - lse), dP_k = do.v_k, ds_k = P_k (dP_k - do.o) scale,
//   dq = sum ds_k k_k.
// With o rounded to bf16, do.o is off by some e, and dq by e sum P_k k_k: so sum P_k k_k and
// e = sum_k P_k (dP_k - do.o), which would be 0, are summed too and their product taken off,
// and the delta that is left for dk and dv gets e.
//
// A query reads n_sel blocks of keys and values once for up to 4 heads that share
// them, which is 2 flops a byte and head: loads bound it.  So there are no shared
// tiles and no barriers in the walk: a warp takes 32 listed keys at a time, each row in
// 16-byte pieces over D * size / 16 lanes, straight into registers, with up to 8 row
// loads a lane in flight; partial dots are summed by a transposing butterfly (LN - 1
// exchanges for 32 keys instead of 5 a key), which leaves lane l the score of key
// (l % LN) * (32 / LN) + l / LN.  The warps of up to 8 CTAs of a cluster share a
// query's list, so that a few queries fill the card, and join their running maxima,
// sums and rows through distributed shared memory: one launch, no workspace.
#include <cooperative_groups.h>

#include "block_internal.cuh"

namespace sdm {

namespace cg = cooperative_groups;

constexpr int kRowWarps = 4;
constexpr int kRowCluster = 8;

// 16 bytes of a row, and the same as floats.
template <typename Tin>
__device__ __forceinline__ uint4 row_piece(const Tin* p, bool in, bool vec) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  if (in) {
    if (vec) {
      u = *reinterpret_cast<const uint4*>(p);
    } else if constexpr (sizeof(Tin) == 4) {
      u = make_uint4(__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]), __float_as_uint(p[3]));
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
      u = make_uint4(h[0] | uint32_t(h[1]) << 16, h[2] | uint32_t(h[3]) << 16,
                     h[4] | uint32_t(h[5]) << 16, h[6] | uint32_t(h[7]) << 16);
    }
  }
  return u;
}
template <typename Tin>
__device__ __forceinline__ void piece_f32(const uint4& u, float* f) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(Tin) == 4) {
      f[i] = __uint_as_float(x[i]);
    } else {
      f[2 * i] = __uint_as_float(x[i] << 16);
      f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    }
  }
}

// Sums v[0 .. 2 * O - 1] over lanes that differ in the bits below 2 * O; the lane keeps
// the one whose number is its low bits (in v[0]).
template <int O>
__device__ __forceinline__ void fold_lanes(float* v) {
  const bool up = threadIdx.x & O;
#pragma unroll
  for (int i = 0; i < O; ++i) {
    const float keep = up ? v[i + O] : v[i], give = up ? v[i] : v[i + O];
    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, O);
  }
  if constexpr (O > 1) fold_lanes<O / 2>(v);
}

template <typename Tin, int D, int RH, bool BWD>
__global__ void __launch_bounds__(kRowWarps * 32)
k_blk_row(BlkArgs a, const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
          const int32_t* __restrict__ idx, Tin* __restrict__ o, float* __restrict__ lse,
          const Tin* __restrict__ d_o, float* __restrict__ delta, Tin* __restrict__ dq,
          sdm_strides sdo, sdm_strides sdq, int hc, int cs, int vec) {
  wait_for_previous();
  constexpr int V = 16 / int(sizeof(Tin)), LN = D / V, KP = 32 / LN;
  constexpr int NB = LN < 8 ? LN : 8, NG = LN / NB;  // rows loaded together, such groups
  constexpr bool FIX = BWD && sizeof(Tin) == 2;  // o is rounded: e comes off again
  __shared__ float part[kRowWarps][RH][D], pk[FIX ? kRowWarps : 1][RH][FIX ? D : 1];
  __shared__ float pm[kRowWarps][RH], pl[kRowWarps][RH], pd[RH];  // backward: pl for e, pd for do.o
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int rank = blockIdx.x % cs;
  long long i = blockIdx.x / cs;
  const int ch = int(i % hc); i /= hc;
  const int t = int(i % a.Tq);
  const int bg = int(i / a.Tq), b = bg / a.G, g = bg - b * a.G;
  const int r0 = ch * RH, nh = min(RH, a.R - r0), h0 = g * a.R + r0;
  const int p = blk_pos0(a, b) + t;
  const int c = (lane % LN) * V, sub = lane / LN;  // columns of the lane, its row among KP
  const float qscale = a.scale * kLog2e;
  float qf[RH][V], gf[BWD ? RH : 1][V], ls[RH], dl[RH];
#pragma unroll
  for (int r = 0; r < RH; ++r) {
    const bool in = r < nh;
    const uint4 u = row_piece(q + row_off(a.sq, b, h0 + (in ? r : 0), t) + c, in, vec & 1);
    piece_f32<Tin>(u, qf[r]);
#pragma unroll
    for (int e = 0; e < V; ++e) qf[r][e] *= qscale;
    if constexpr (BWD) {
      float of[V];
      piece_f32<Tin>(row_piece(d_o + row_off(sdo, b, h0 + (in ? r : 0), t) + c, in, vec & 2), gf[r]);
      piece_f32<Tin>(row_piece(o + row_off(a.so, b, h0 + (in ? r : 0), t) + c, in, vec & 2), of);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) s = fmaf(gf[r][e], of[e], s);
#pragma unroll
      for (int w = LN / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      dl[r] = s;
      const size_t at = ((size_t)b * a.H + h0 + (in ? r : 0)) * a.Tq + t;
      const float x = in ? lse[at] : -INFINITY;
      ls[r] = x == -INFINITY ? INFINITY : x * kLog2e;  // weights of a row without keys are 0
      if (FIX) {
        if (threadIdx.x == 0) pd[r] = s;
      } else if (rank == 0 && threadIdx.x == 0 && in) {
        delta[at] = s;
      }
    }
  }
  float acc[RH][V], m[RH], l[RH], ak[FIX ? RH : 1][V];
#pragma unroll
  for (int r = 0; r < RH; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[r][e] = ak[FIX ? r : 0][e] = 0.f;
  }
  const int32_t* list = idx + ((size_t)bg * a.Tq + t) * a.n_sel;
  const int per = a.bs / 32, pieces = a.n_sel * per;
  for (int pc = rank * kRowWarps + wp; pc < pieces; pc += cs * kRowWarps) {
    const int j = list[pc / per], k0 = (pc % per) * 32;
    const int n = min(32, blk_keys(a, j, p) - k0);  // keys behind the query are not read
    if (n <= 0) continue;
    const long long key0 = (long long)j * a.bs + k0;
    const Tin* kp = k + row_off(a.sk, b, g, 0) + key0 * a.sk.t + c;
    const Tin* vp = v + row_off(a.sv, b, g, 0) + key0 * a.sv.t + c;
    float s[RH], dp[BWD ? RH : 1], w[FIX ? RH : 1];
    // scores (and do.v): each group of NB row loads leaves one value a lane
    auto dots = [&](const Tin* base, long long st, const float (&x)[RH][V], int on, float (&out)[RH]) {
      float gsum[RH][NG];
#pragma unroll
      for (int u = 0; u < NG; ++u) {
        uint4 raw[NB];
#pragma unroll
        for (int z = 0; z < NB; ++z) {
          const int kk = (u * NB + z) * KP + sub;
          raw[z] = row_piece(base + kk * st, kk < n, on);
        }
        float w[RH][NB];
#pragma unroll
        for (int z = 0; z < NB; ++z) {
          float f[V];
          piece_f32<Tin>(raw[z], f);
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            w[r][z] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) w[r][z] = fmaf(x[r][e], f[e], w[r][z]);
          }
        }
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          fold_lanes<NB / 2>(w[r]);
          gsum[r][u] = w[r][0];
        }
      }
#pragma unroll
      for (int r = 0; r < RH; ++r) {
        if constexpr (NG == 2) {
          const bool up = lane & 8;
          const float keep = up ? gsum[r][1] : gsum[r][0], give = up ? gsum[r][0] : gsum[r][1];
          out[r] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
        } else if constexpr (NG == 4) {
          const bool up = lane & 16, mid = lane & 8;
          float y[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float keep = up ? gsum[r][z + 2] : gsum[r][z], give = up ? gsum[r][z] : gsum[r][z + 2];
            y[z] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
          }
          const float keep = mid ? y[1] : y[0], give = mid ? y[0] : y[1];
          out[r] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
        } else {
          out[r] = gsum[r][0];
        }
      }
    };
    dots(kp, a.sk.t, qf, vec & 4, s);
    const bool mine = (lane % LN) * KP + sub < n;  // the lane's own key
    if constexpr (BWD) {
      dots(vp, a.sv.t, gf, vec & 8, dp);
#pragma unroll
      for (int r = 0; r < RH; ++r) {
        const float P = mine ? exp2f(s[r] - ls[r]) : 0.f, x = mine ? P * (dp[r] - dl[r]) : 0.f;
        s[r] = x * a.scale;
        if constexpr (FIX) {
          w[r] = P;
          l[r] += x;
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < RH; ++r) {
        if (!mine) s[r] = -INFINITY;
        float mx = s[r];
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        mx = fmaxf(mx, m[r]);
        const float base = mx == -INFINITY ? 0.f : mx;
        s[r] = mine ? exp2f(s[r] - base) : 0.f;
        const float f = exp2f(m[r] - base);  // 0 from the empty start
        l[r] = fmaf(l[r], f, s[r]);
        m[r] = mx;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[r][e] *= f;
      }
    }
    const Tin* mp = BWD ? kp : vp;
    const long long ms = BWD ? a.sk.t : a.sv.t;
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      uint4 raw[NB];
#pragma unroll
      for (int z = 0; z < NB; ++z) {
        const int kk = (u * NB + z) * KP + sub;
        raw[z] = row_piece(mp + kk * ms, kk < n, vec & (BWD ? 4 : 8));
      }
#pragma unroll
      for (int z = 0; z < NB; ++z) {
        float f[V];
        piece_f32<Tin>(raw[z], f);
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          const int from = (lane & ~(LN - 1)) | (u * NB + z);
          const float y = __shfl_sync(0xffffffffu, s[r], from);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[r][e] = fmaf(y, f[e], acc[r][e]);
          if constexpr (FIX) {
            const float P = __shfl_sync(0xffffffffu, w[r], from);
#pragma unroll
            for (int e = 0; e < V; ++e) ak[r][e] = fmaf(P, f[e], ak[r][e]);
          }
        }
      }
    }
  }
  // the warp's rows, then the join over the cluster's warps
#pragma unroll
  for (int r = 0; r < RH; ++r) {
#pragma unroll
    for (int w = LN; w < 32; w <<= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        acc[r][e] += __shfl_xor_sync(0xffffffffu, acc[r][e], w);
        if constexpr (FIX) ak[r][e] += __shfl_xor_sync(0xffffffffu, ak[r][e], w);
      }
    if (sub == 0)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        part[wp][r][c + e] = acc[r][e];
        if constexpr (FIX) pk[wp][r][c + e] = ak[r][e];
      }
    if constexpr (!BWD || FIX) {
      l[r] = warp_sum(l[r]);
      if (lane == 0) {
        pm[wp][r] = m[r];
        pl[wp][r] = l[r];
      }
    }
  }
  cg::cluster_group cl = cg::this_cluster();
  if (cs > 1) cl.sync(); else __syncthreads();
  for (int e = rank * kRowWarps * 32 + threadIdx.x; e < nh * D; e += cs * kRowWarps * 32) {
    const int r = e / D, col = e % D;
    float mx = -INFINITY, x = 0.f, sum = 0.f, sk = 0.f;
    if constexpr (!BWD) {
      for (int w = 0; w < cs; ++w) {
        const float* om = cs > 1 ? cl.map_shared_rank(&pm[0][0], w) : &pm[0][0];
#pragma unroll
        for (int y = 0; y < kRowWarps; ++y) mx = fmaxf(mx, om[y * RH + r]);
      }
      if (mx == -INFINITY) mx = 0.f;
    }
    for (int w = 0; w < cs; ++w) {
      const float* op = cs > 1 ? cl.map_shared_rank(&part[0][0][0], w) : &part[0][0][0];
      const float* om = cs > 1 ? cl.map_shared_rank(&pm[0][0], w) : &pm[0][0];
      const float* ol = cs > 1 ? cl.map_shared_rank(&pl[0][0], w) : &pl[0][0];
#pragma unroll
      for (int y = 0; y < kRowWarps; ++y) {
        const float z = op[(y * RH + r) * D + col];
        if constexpr (FIX) {
          const float* ok = cs > 1 ? cl.map_shared_rank(&pk[0][0][0], w) : &pk[0][0][0];
          x += z;
          sk += ok[(y * RH + r) * D + col];
          sum += ol[y * RH + r];
        } else if constexpr (BWD) {
          x += z;
        } else {
          const float f = exp2f(om[y * RH + r] - mx);
          x = fmaf(f, z, x);
          sum = fmaf(f, ol[y * RH + r], sum);
        }
      }
    }
    if constexpr (BWD) {
      if constexpr (FIX) {
        x -= sum * a.scale * sk;
        if (col == 0) delta[((size_t)b * a.H + h0 + r) * a.Tq + t] = pd[r] + sum;
      }
      dq[row_off(sdq, b, h0 + r, t) + col] = from_f32<Tin>(x);
    } else {
      o[row_off(a.so, b, h0 + r, t) + col] = from_f32<Tin>(sum == 0.f ? 0.f : x / sum);
      if (lse && col == 0)
        lse[((size_t)b * a.H + h0 + r) * a.Tq + t] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) / kLog2e;
    }
  }
  if (cs > 1) cl.sync();  // the others may still be reading this CTA's rows
}

// CTAs that share a query: more than one while they all fit the card at 4 an SM and a
// warp has a piece of 32 keys.  float32, 16 blocks of 64, d = 64, 4 groups of 4 heads,
// clusters of 1 / 2 / 4 / 8: 1 sequence 26 / 16 / 10 / 8 us, 32 sequences
// 29 / 20 / 16 / 22, 64 sequences 41 / 30 / 35 / 46.
template <typename Tin, int D, int RH, bool BWD>
static cudaError_t launch_row(const BlkArgs& a, const void* q, const void* k, const void* v,
                              const int32_t* idx, void* o, float* lse, const void* d_o,
                              float* delta, void* dq, const sdm_strides& sdo,
                              const sdm_strides& sdq, cudaStream_t s) {
  const int es = int(sizeof(Tin)), hc = (a.R + RH - 1) / RH, pieces = a.n_sel * (a.bs / 32);
  const long long items = (long long)a.B * a.G * a.Tq * hc;
  int cs = 1;
  while (cs < kRowCluster && 2 * items * cs <= 4 * 148 && 2 * cs * kRowWarps <= pieces) cs *= 2;
  if (items * cs >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  int vec = view_aligned(q, a.sq, es, 16) ? 1 : 0;
  if (BWD && view_aligned(d_o, sdo, es, 16) && view_aligned(o, a.so, es, 16)) vec |= 2;
  if (view_aligned(k, a.sk, es, 16)) vec |= 4;
  if (view_aligned(v, a.sv, es, 16)) vec |= 8;
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
  c.blockDim = dim3(kRowWarps * 32);
  c.stream = s;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, k_blk_row<Tin, D, RH, BWD>, a, (const Tin*)q, (const Tin*)k,
                            (const Tin*)v, idx, (Tin*)o, lse, (const Tin*)d_o, delta, (Tin*)dq, sdo,
                            sdq, hc, cs, vec);
}

template <typename Tin, bool BWD>
static cudaError_t launch_row_any(const BlkArgs& a, const void* q, const void* k, const void* v,
                                  const int32_t* idx, void* o, float* lse, const void* d_o,
                                  float* delta, void* dq, const sdm_strides& sdo,
                                  const sdm_strides& sdq, cudaStream_t s) {
  auto go = [&](auto dd) -> cudaError_t {
    constexpr int D = decltype(dd)::value;
    if (a.R == 1) return launch_row<Tin, D, 1, BWD>(a, q, k, v, idx, o, lse, d_o, delta, dq, sdo, sdq, s);
    if (a.R == 2) return launch_row<Tin, D, 2, BWD>(a, q, k, v, idx, o, lse, d_o, delta, dq, sdo, sdq, s);
    return launch_row<Tin, D, 4, BWD>(a, q, k, v, idx, o, lse, d_o, delta, dq, sdo, sdq, s);
  };
  if (a.d == 32) return go(std::integral_constant<int, 32>());
  if (a.d == 64) return go(std::integral_constant<int, 64>());
  return go(std::integral_constant<int, 128>());
}

cudaError_t launch_blk_row_fwd(const BlkArgs& a, bool bf16, const void* q, const void* k,
                               const void* v, const int32_t* idx, void* o, float* lse,
                               cudaStream_t s) {
  const sdm_strides z = {0, 0, 0};
  return bf16 ? launch_row_any<__nv_bfloat16, false>(a, q, k, v, idx, o, lse, nullptr, nullptr, nullptr, z, z, s)
              : launch_row_any<float, false>(a, q, k, v, idx, o, lse, nullptr, nullptr, nullptr, z, z, s);
}

cudaError_t launch_blk_row_bwd(const BlkArgs& a, bool bf16, const void* q, const void* k,
                               const void* v, const int32_t* idx, const void* o, const float* lse,
                               const void* d_o, float* delta, void* dq, const sdm_strides& sdo,
                               const sdm_strides& sdq, cudaStream_t s) {
  void* om = const_cast<void*>(o);
  float* lm = const_cast<float*>(lse);
  return bf16 ? launch_row_any<__nv_bfloat16, true>(a, q, k, v, idx, om, lm, d_o, delta, dq, sdo, sdq, s)
              : launch_row_any<float, true>(a, q, k, v, idx, om, lm, d_o, delta, dq, sdo, sdq, s);
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
  const bool pieces = dims->in_dtype == SDM_DTYPE_BF16 && view_aligned(q, a.sq, 2, 16) &&
                      view_aligned(k, a.sk, 2, 16) && view_aligned(v, a.sv, 2, 16) && view_aligned(o, a.so, 2, 16);
  const cudaError_t e = !pieces ? launch_blk_row_fwd(a, dims->in_dtype == SDM_DTYPE_BF16, q, k, v, idx, o, lse, s)
                        : blk_tiles_pay(dims) ? launch_blk_fwd_mma(dims, a, q, k, v, idx, o, lse, workspace, s)
                                              : launch_blk_step(a, q, k, v, idx, o, lse, s);
  return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
