// Root-mean-square norm of hidden rows with the residual's addition, and the FP8 rows that the
// projections after it read:
//     s = x + residual          (residual_out = s rounded to x's type)
//     y = s * rsqrt(mean(s^2) + eps) * weight
//     scale = absmax(y) / 448 per row or per 128 values (1 where all are zero), codes = E4M3(y / scale)
// Everything between the loads and the stores is fp32: the norm and the codes are taken from the
// unrounded sum, so the only roundings are the stored residual's, the codes' and (where asked for)
// the bf16 copy's.  The quotient y / scale is a product with the correctly rounded reciprocal, within
// one fp32 ulp of it.
//
// Bound by HBM: each input is read and each output written once (7 bytes a value for bf16 with a
// residual).  One CTA per row keeps the row in registers between the two reductions.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kVec = 8;                       // values per thread and step: 16 bytes of bf16

// Eight values as they lie in memory
template <bool F32>
struct Raw {
  uint4 u[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const void* p, int64_t elem) {
  Raw<F32> r;
  const uint4* u = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + elem * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.u[i] = u[i];
  return r;
}

template <bool F32>
__device__ __forceinline__ void widen(const Raw<F32>& r, float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const uint32_t w[4] = {r.u[i].x, r.u[i].y, r.u[i].z, r.u[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (F32) {
        v[4 * i + j] = __uint_as_float(w[j]);
      } else {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}

__device__ __forceinline__ uint4 bf16x8(const float (&v)[kVec]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t elem, const float (&v)[kVec]) {
  if constexpr (F32) {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + elem);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + elem) = bf16x8(v);
  }
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Sum (or maximum) of v over the CTA; every thread gets it.  `part` holds one value per warp.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  v = static_cast<int>(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;   // sums of squares and |y| are >= 0
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  return v;
}

// One CTA per row; vector i * blockDim + tid of the row is a thread's i-th.  blockDim is a
// multiple of 32, so a group of 128 values is 16 neighbouring lanes.
template <bool F32, int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormArgs a) {
  __shared__ float part_sum[32], part_max[32];
  grid_dependency_wait();
  launch_dependents();
  const int64_t row = blockIdx.x;
  const int nvec = a.d / kVec, tid = threadIdx.x;
  // every load of the row before the first store, which might be to the same memory
  Raw<F32> rx[VPT], rr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + tid;
    if (v < nvec) {
      rx[i] = load8<F32>(a.x, row * a.x_stride + v * kVec);
      if (a.residual) rr[i] = load8<F32>(a.residual, row * a.d + v * kVec);
    }
  }
  float s[VPT][kVec];
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + tid;
#pragma unroll
    for (int e = 0; e < kVec; ++e) s[i][e] = 0.f;
    if (v < nvec) {
      widen<F32>(rx[i], s[i]);
      if (a.residual) {
        float r[kVec];
        widen<F32>(rr[i], r);
#pragma unroll
        for (int e = 0; e < kVec; ++e) s[i][e] += r[e];
        store8<F32>(a.residual_out, row * a.d + v * kVec, s[i]);
      }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) sq += s[i][e] * s[i][e];
  }
  const float inv = 1.0f / sqrtf(block_reduce<false>(sq, part_sum) / static_cast<float>(a.d) + a.eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + tid;
    float group_max = 0.f;
    if (v < nvec) {
      float w[kVec];
      if (a.w_f32) widen<true>(load8<true>(a.weight, v * kVec), w);
      else widen<false>(load8<false>(a.weight, v * kVec), w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        s[i][e] = s[i][e] * inv * w[e];
        group_max = fmaxf(group_max, fabsf(s[i][e]));
      }
      if (a.normed) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.normed) + row * a.d + v * kVec) = bf16x8(s[i]);
    }
    if (a.group) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) group_max = fmaxf(group_max, __shfl_xor_sync(0xffffffffu, group_max, o));
      const float sc = group_max > 0.f ? __fdiv_rn(group_max, 448.0f) : 1.0f;
      const float q = __frcp_rn(sc);
      if (v < nvec) {
        const int groups = (a.d + 127) / 128;
        if (v % 16 == 0) a.scale[row * groups + v / 16] = sc;
        *reinterpret_cast<uint2*>(a.codes + row * a.d + v * kVec) =
            make_uint2(e4m3x4(s[i][0] * q, s[i][1] * q, s[i][2] * q, s[i][3] * q),
                       e4m3x4(s[i][4] * q, s[i][5] * q, s[i][6] * q, s[i][7] * q));
      }
    } else {
      amax = fmaxf(amax, group_max);
    }
  }
  if (!a.group) {
    amax = block_reduce<true>(amax, part_max);
    const float sc = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    const float q = __frcp_rn(sc);
    if (tid == 0) a.scale[row] = sc;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * blockDim.x + tid;
      if (v < nvec)
        *reinterpret_cast<uint2*>(a.codes + row * a.d + v * kVec) =
            make_uint2(e4m3x4(s[i][0] * q, s[i][1] * q, s[i][2] * q, s[i][3] * q),
                       e4m3x4(s[i][4] * q, s[i][5] * q, s[i][6] * q, s[i][7] * q));
    }
  }
}

template <bool F32>
cudaError_t launch_typed(const NormArgs& a, cudaStream_t stream) {
  const int nvec = a.d / kVec;
  int vpt = 1;
  while (vpt < 4 && (nvec + vpt - 1) / vpt > 256) vpt <<= 1;
  int threads = (nvec + vpt - 1) / vpt;
  threads = (threads + 31) / 32 * 32;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (vpt) {
    case 1: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<F32, 1>, a);
    case 2: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<F32, 2>, a);
    default: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<F32, 4>, a);
  }
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const NormArgs& a, cudaStream_t stream) {
  return a.x_f32 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
}

}  // namespace dsa
