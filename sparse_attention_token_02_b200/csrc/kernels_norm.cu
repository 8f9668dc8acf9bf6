// Root-mean-square norm of hidden rows with the residual's addition, and the FP8 rows that the
// projections after it read:
//     s = x + residual          (residual_out = s rounded to x's type)
//     y = s * rsqrt(mean(s^2) + eps) * weight
//     scale = absmax(y) / 448 per row or per 128 values (1 where all are zero), codes = E4M3(y / scale)
// Everything between the loads and the stores is fp32: the norm and the codes are taken from the
// unrounded sum, so the only roundings to fewer bits are the stored residual's, the codes' and (where asked for)
// the bf16 copy's.
//
// With t = s * weight, y is inv * t: products and maxima are made before the row's sum is known, y / scale is
// t * (448 / max|t|), and the sum enters the scale alone: of 73 million codes 1149 are not those of the exact y and scale,
// where y / scale from a rounded y and scale leaves 1667.  The reciprocal square root is within two fp32 ulps, the product
// with 1 / 448 within one more.
//
// Bound by HBM: each input is read and each output written once (7 bytes a value for bf16 with a residual); 16384 x 7168
// rows back to back in a graph take 129 us (98 % of the measured copy rate), without a residual 91 to 94 us (59 %: there the
// instructions, some 20 a value, weigh as much).  A CTA keeps a row in registers between the sum and the codes and has
// its next row's loads under way meanwhile: one CTA a row and weights applied after the sum took 133 and 107 us, and
// 17 us for 16384 rows of 128 values that take 6 now.  A ring of rows in shared memory (155 us) cost more than it hid.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kVec = 8;                       // values per thread and step: 16 bytes of bf16
constexpr float kTiny = 0x1p-100f, kLift = 0x1p64f;
// Values so large that squares, or products with a weight, might overflow are held down by kDown, for any weight below 2^70.
// A row whose sum of squares passes kLarge is done again from its values times kDown, after the CTA's others; the squares of
// smaller ones overflow nothing.  Where there is nothing to start again from (the rounded sum may have replaced a bf16
// residual), eight values whose squares pass kLarge are held down at once and their row is finished apart, which costs
// rows of 1536 with a residual 8 % (31 -> 33.3 us for 16384); a CTA of one row, of more than 8192 values, does the same,
// where the second pass would make registers spill (107 us for 8192 rows of 16384, 125 with it).
constexpr float kLarge = 0x1p96f, kDown = 0x1p-72f;

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

// The same for rows, which are read once: bf16 ones leave the first-level cache to the weights (2048 rows of 7168 17.5 ->
// 16.3 us; fp32 rows lost, 100 -> 108 us for 16384).
template <bool F32>
__device__ __forceinline__ Raw<F32> load8_once(const void* p, int64_t elem) {
  Raw<F32> r;
  const uint8_t* u = static_cast<const uint8_t*>(p) + elem * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i)
    if constexpr (F32) {
      r.u[i] = reinterpret_cast<const uint4*>(u)[i];
    } else {
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.u[i].x), "=r"(r.u[i].y), "=r"(r.u[i].z), "=r"(r.u[i].w)
                   : "l"(u)
                   : "memory");
    }
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

// The rest of a row with values held down, given the warps' sums.  A group (or row) with one such value has all of them held
// down: what that takes from others lies 2^100 below its maximum.
template <int VPT, int QUADS>
__device__ __forceinline__ void finish_wild_row(const NormArgs& a, int64_t row, float (&t)[VPT][kVec], uint32_t low,
                                                float4 (&part)[3][QUADS], int nvec) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* const sums = reinterpret_cast<const float*>(part[0]);
  float* const maxima = reinterpret_cast<float*>(part[1]);
  const float* const large = reinterpret_cast<const float*>(part[2]);
  float sum = 0.f, down = 0.f;
  for (int i = 0; i < 4 * QUADS; ++i) {
    sum += sums[i];
    down += large[i];
  }
  const float per_value = 1.0f / static_cast<float>(a.d);
  const float inv_low = rsqrtf((down + sum * (kDown * kDown)) * per_value + a.eps * (kDown * kDown)), inv = inv_low * kDown;
  const int64_t at = row * a.d;
  float top[VPT], most = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + tid;
    const bool held = low >> i & 1;
    if (a.normed && v < nvec) {
      float y[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) y[e] = t[i][e] * (held ? inv_low : inv);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.normed) + at + v * kVec) = bf16x8(y);
    }
    const uint32_t lanes = __ballot_sync(0xffffffffu, held);
    const bool follow = !a.group || (lanes >> (lane & 16) & 0xFFFFu);
    if (follow && !held) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) t[i][e] *= kDown;
    }
    if (follow) low |= 1u << i;
    top[i] = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) top[i] = fmaxf(top[i], fabsf(t[i][e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < 16 || !a.group) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    most = fmaxf(most, top[i]);
  }
  if (!a.group) {
    if (lane == 0) maxima[warp] = most;
    __syncthreads();
    for (int i = 0; i < 4 * QUADS; ++i) most = fmaxf(most, maxima[i]);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + tid;
    if (v >= nvec) continue;
    const float its = low >> i & 1 ? inv_low : inv, amax = a.group ? top[i] : most;
    const float lift = amax < kTiny ? kLift : 1.0f, peak = amax * its;
    const float sc = peak > 0.f ? peak * (1.0f / 448.0f) : 1.0f;
    if (a.group ? (v & 15) == 0 : v == 0) a.scale[a.group ? row * ((a.d + 127) / 128) + v / 16 : row] = sc;
    const float up = peak > 0.f ? lift : 1.0f, f = peak > 0.f ? __fdiv_rn(448.0f, amax * lift) : its;
    *reinterpret_cast<uint2*>(a.codes + at + v * kVec) =
        make_uint2(e4m3x4(t[i][0] * up * f, t[i][1] * up * f, t[i][2] * up * f, t[i][3] * up * f),
                   e4m3x4(t[i][4] * up * f, t[i][5] * up * f, t[i][6] * up * f, t[i][7] * up * f));
  }
}

// A CTA takes every gridDim-th row; vector i * blockDim + tid of a row is a thread's i-th.  blockDim is a
// multiple of 32, so a group of 128 values is 16 neighbouring lanes.  With one or two vectors a thread the next row
// is under way while this one is summed and written; with four (rows of more than 8192 values) a CTA has one row.
template <bool F32, int VPT, bool RES>
__global__ void __launch_bounds__(VPT <= 2 ? 512 : 1024, VPT <= 2 ? 2 : 1) rmsnorm_kernel(NormArgs a) {
  constexpr bool kAhead = VPT <= 2;
  constexpr int kWarps = kAhead ? 16 : 32;
  __shared__ float4 part[2][3][kWarps / 4];              // two rows in turn: every warp's sum, maximum and sum of large squares
  constexpr bool kAtOnce = VPT == 4 || (RES && !F32);
  __shared__ uint8_t held[kAtOnce ? kWarps * 32 : 1];    // a thread's vectors held down: rare, so not in a register
  const int nvec = a.d / kVec, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (kAtOnce) held[tid] = 0;
  for (int i = tid; i < 6 * kWarps; i += blockDim.x) reinterpret_cast<float*>(part)[i] = 0.f;   // warps that are not there
  __syncthreads();
  grid_dependency_wait();
  launch_dependents();
  int turn = 0;
  bool again = false;
  auto pass = [&](auto done) {                           // over the CTA's rows; over those done once whose values have to be held down
    constexpr bool kDone = decltype(done)::value;
    // every load of a row before the first store, which might be to the same memory
    Raw<F32> rx[VPT], rr[RES ? VPT : 1];
    auto load = [&](int64_t row) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * blockDim.x + tid;
        if (v < nvec) {
          // an fp32 residual_out holds the sum as it is
          rx[i] = kDone && RES ? load8_once<F32>(a.residual_out, row * a.d + v * kVec) : load8_once<F32>(a.x, row * a.x_stride + v * kVec);
          if (RES && !kDone) rr[i] = load8_once<F32>(a.residual, row * a.d + v * kVec);
        }
      }
    };
    const float per_value = 1.0f / static_cast<float>(a.d);
    int64_t row = blockIdx.x;
    load(row);
    for (; row < a.rows; row += gridDim.x, turn ^= 1) {
      // t = s * weight: what is left of y is the row's factor, known after the sum
      float t[VPT][kVec], top[VPT];
      float sq = 0.f, large = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * blockDim.x + tid;
        top[i] = 0.f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) t[i][e] = 0.f;
        if (v < nvec) {
          widen<F32>(rx[i], t[i]);
          if (kDone) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) t[i][e] *= kDown;
          } else if (RES) {
            float r[kVec];
            widen<F32>(rr[i], r);
#pragma unroll
            for (int e = 0; e < kVec; ++e) t[i][e] += r[e];
            store8<F32>(a.residual_out, row * a.d + v * kVec, t[i]);
          }
          float w[kVec];
          if (a.w_f32) widen<true>(load8<true>(a.weight, v * kVec), w);
          else widen<false>(load8<false>(a.weight, v * kVec), w);
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < kVec; ++e) q += t[i][e] * t[i][e];
          if (kAtOnce && q > kLarge) {
            held[tid] |= 1u << i;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
              t[i][e] *= kDown;
              large += t[i][e] * t[i][e];
            }
          } else {
            sq += q;
          }
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            t[i][e] *= w[e];
            top[i] = fmaxf(top[i], fabsf(t[i][e]));
          }
        }
      }
      if (kAhead && row + gridDim.x < a.rows) load(row + gridDim.x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      if (a.group) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
      } else {
#pragma unroll
        for (int i = 1; i < VPT; ++i) top[0] = fmaxf(top[0], top[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
      }
      const bool any = kAtOnce && __any_sync(0xffffffffu, large != 0.f);
      if (kAtOnce && any) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) large += __shfl_xor_sync(0xffffffffu, large, o);
      }
      if (lane == 0) {
        reinterpret_cast<float*>(part[turn][0])[warp] = sq;
        reinterpret_cast<float*>(part[turn][1])[warp] = top[0];
        if (kAtOnce) reinterpret_cast<float*>(part[turn][2])[warp] = large;
      }
      const int64_t at = row * a.d;
      if constexpr (kAtOnce) {
        if (__syncthreads_or(any)) {
          finish_wild_row<VPT>(a, row, t, held[tid], part[turn], nvec);
          held[tid] = 0;
          if (!kAhead) break;
          continue;
        }
      } else {
        __syncthreads();
      }
      float sum = 0.f, most = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps / 4; ++i) {
        const float4 p = part[turn][0][i];
        sum += (p.x + p.y) + (p.z + p.w);
      }
      if (!a.group) {
#pragma unroll
        for (int i = 0; i < kWarps / 4; ++i) {
          const float4 p = part[turn][1][i];
          most = fmaxf(fmaxf(most, fmaxf(p.x, p.y)), fmaxf(p.z, p.w));
        }
      }
      if (!kAtOnce && !kDone) again = again || sum > kLarge;   // the same for every thread
      if (kDone && !(sum > 4.0f * kLarge * (kDown * kDown))) {   // it was right before, by a rounding or far
        if (!kAhead) break;
        continue;
      }
      const float inv = rsqrtf(sum * per_value + (kDone ? a.eps * (kDown * kDown) : a.eps));
      if (a.normed) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int v = i * blockDim.x + tid;
          if (v < nvec) {
            float y[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) y[e] = t[i][e] * inv;
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.normed) + at + v * kVec) = bf16x8(y);
          }
        }
      }
      // A group's scale is worked out once for the thread's VPT groups: by every VPT-th part of its 16 lanes.
      constexpr int kShift = VPT == 4 ? 2 : VPT == 2 ? 3 : 4;
      const int mine = (lane >> kShift) & (VPT - 1);
      float amax = most;
      if (a.group) {
        amax = top[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i)
          if (mine == i) amax = top[i];
      }
      // y / scale = t * 448 / max|t|.  Values so small that the quotient could overflow go up by 2^64 first.
      const float lift = amax < kTiny ? kLift : 1.0f;
      const float peak = amax * inv;                         // 0 or NaN: the scale is 1, the codes are those of y
      const float sc = peak > 0.f ? peak * (1.0f / 448.0f) : 1.0f;
      const float factor = peak > 0.f ? __fdiv_rn(448.0f, amax * lift) : inv;
      if (a.group) {
        const int first = (mine * blockDim.x + tid) & ~15;    // the group's first vector
        if ((lane & ((1 << kShift) - 1)) == 0 && first < nvec) a.scale[row * ((a.d + 127) / 128) + first / 16] = sc;
      } else if (tid == 0) {
        a.scale[row] = sc;
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * blockDim.x + tid;
        const int from = (lane & 16) | i << kShift;
        const float k = VPT == 1 || !a.group ? factor : __shfl_sync(0xffffffffu, factor, from);
        const float largest = a.group ? top[i] : most;
        if (largest < kTiny && largest * inv > 0.f) {
#pragma unroll
          for (int e = 0; e < kVec; ++e) t[i][e] *= kLift;
        }
        if (v < nvec)
          *reinterpret_cast<uint2*>(a.codes + at + v * kVec) =
              make_uint2(e4m3x4(t[i][0] * k, t[i][1] * k, t[i][2] * k, t[i][3] * k),
                         e4m3x4(t[i][4] * k, t[i][5] * k, t[i][6] * k, t[i][7] * k));
      }
      if (!kAhead) break;
    }
  };
  pass(std::false_type{});
  if (!kAtOnce && again) {
    __syncthreads();
    if constexpr (!kAtOnce) pass(std::true_type{});
  }
}

template <bool F32, int VPT, bool RES>
cudaError_t launch_vpt(const NormArgs& a, int threads, cudaStream_t stream) {
  const auto kernel = rmsnorm_kernel<F32, VPT, RES>;
  int64_t grid = a.rows;
  if (VPT <= 2) {                                        // as many CTAs as stay resident
    int device = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return e;
    if (a.rows > sms) {
      thread_local int blocks[17] = {};                  // an SM holds, per number of warps
      int& n = blocks[threads / 32];
      if (n == 0 && (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0)) != cudaSuccess) return e;
      grid = std::min<int64_t>(grid, int64_t(sms) * std::max(1, n));
    }
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool F32, bool RES>
cudaError_t launch_typed(const NormArgs& a, cudaStream_t stream) {
  // Two vectors a thread from 2048 values on: with one, 16384 x 4096 bf16 rows take 87 us for 77.  Rows of fp32 with a
  // residual keep to one, whose registers do not spill (150 us for 139).
  const int nvec = a.d / kVec;
  int vpt = 1;
  while (vpt < 4 && (nvec + vpt - 1) / vpt > (vpt == 1 && !(F32 && RES) ? 256 : 512)) vpt <<= 1;
  int threads = (nvec + vpt - 1) / vpt;
  threads = (threads + 31) / 32 * 32;
  switch (vpt) {
    case 1: return launch_vpt<F32, 1, RES>(a, threads, stream);
    case 2: return launch_vpt<F32, 2, RES>(a, threads, stream);
    default: return launch_vpt<F32, 4, RES>(a, threads, stream);
  }
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const NormArgs& a, cudaStream_t stream) {
  if (a.residual) return a.x_f32 ? launch_typed<true, true>(a, stream) : launch_typed<false, true>(a, stream);
  return a.x_f32 ? launch_typed<true, false>(a, stream) : launch_typed<false, false>(a, stream);
}

}  // namespace dsa
