// Append to the paged latent cache: one token's latent (512 values, which attention reads as its
// values and as most of its key) and the token's rotated key part (64 values), written to the row
// that the page table gives for the token's position.
//     row = pages[seq, p / page_size] * page_size + p % page_size
//     rope[row] = rotate(kr_new, p)                     (bf16)
//     latent[row] = c_new in bf16, or E4M3 codes with one scale
// The FP8 scale is the smallest power of two with absmax <= 448 * scale (at least 2^-100; 1 for a row of
// zeros): E4M3 is a floating format, so a power of two costs no relative precision, and the codes
// times it are exact in bf16, which attention multiplies in.
//
// A pair turns by p * f of a full turn, f = base^(-2 i / rope_dim) / (2 pi).  f is held in 64 bits, so that one integer
// product gives the angle's fraction of a turn at any position (within p * 2^-53, as in fp64, and 2^-31), and sine and
// cosine of a fraction of a turn need no reduction.
// Bound by HBM (about 1.2 KB read and 0.7 to 1.2 KB written a token); one warp per token with all its loads issued
// before the first use, even of the token's sequence.  16384 tokens to FP8, back to back in a graph over four sets of
// tensors: 12.5 us with fp64 angles and the sequence awaited first, 8.0 now (3.7 TB/s, 8.3 over more sets; 5.8 to 6.2 where up
// to three sets, 30 MB each, stay in the L2); the frequencies go through shared memory because a warp whose lanes read
// different parameters is served lane by lane (9.9 us).  32 tokens: 1.6 us.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kAppendWarps = 4;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// e of the smallest power of two 2^e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), at least -100
__device__ __forceinline__ int pow2_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -100 ? -100 : e;
}

// One rotated or passed-through value of the key part
template <bool F32>
__device__ __forceinline__ float kr_value(const void* p, int64_t elem) {
  return F32 ? static_cast<const float*>(p)[elem] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[elem]);
}

struct Turns {
  int32_t rope_dim, interleaved;
  uint64_t f[kLatentRope / 2];                           // turns per position, modulo one, times 2^64
};

template <bool F32>
__global__ void __launch_bounds__(kAppendWarps * 32) latent_append_kernel(LatentAppendArgs a, Turns turns) {
  // Lanes that read different parameters are served one by one: one warp does so for the block.
  __shared__ uint64_t per_position[kLatentRope / 2];
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < kLatentRope / 2) per_position[lane] = turns.f[lane];
  __syncthreads();
  grid_dependency_wait();
  launch_dependents();
  const int32_t t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= a.n) return;                                  // whole warps leave together
  const int32_t seq = a.seq_ids[t], pos = a.positions[t];
  // lane's latent values: 16 lane .. 16 lane + 15
  uint4 raw[F32 ? 4 : 2];
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c_new) + (t * a.c_stride + lane * 16) * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 2); ++i) raw[i] = src[i];
  // lane's two key values: pair `lane` while that rotates, else the next two that pass through
  const int npairs = turns.rope_dim / 2;
  const bool rotates = lane < npairs;
  const int i0 = turns.interleaved || !rotates ? 2 * lane : lane;
  const int i1 = turns.interleaved || !rotates ? 2 * lane + 1 : lane + npairs;
  float x0 = 0.f, x1 = 0.f;
  if (a.kv.rope) {
    x0 = kr_value<F32>(a.kr_new, t * a.kr_stride + i0);
    x1 = kr_value<F32>(a.kr_new, t * a.kr_stride + i1);
  }
  if (seq < 0) return;                                   // a padding token
  const int32_t slot = pos < 0 ? -1 : a.kv.page_shift >= 0 ? pos >> a.kv.page_shift : pos / a.kv.page_size;
  int32_t page = -1;
  if (seq < a.kv.num_seqs && slot >= 0 && slot < a.kv.max_pages) page = a.kv.pages[static_cast<int64_t>(seq) * a.kv.max_pages + slot];
  if (page < 0 || page >= a.kv.num_pages) {              // no such page: nothing is written
    if (lane == 0) record_error(a.err, DSA_DEVERR_PAGE, t);
    return;
  }
  const int64_t row = static_cast<int64_t>(page) * a.kv.page_size + (pos - slot * a.kv.page_size);
  if (a.kv.rope) {
    if (rotates) {
      const uint64_t turned = per_position[lane] * static_cast<uint32_t>(pos);
      float sine, cosine;                                // of the upper half, a signed fraction of half a turn
      sincospif(static_cast<float>(static_cast<int32_t>(turned >> 32)) * 0x1p-31f, &sine, &cosine);
      const float u = x0 * cosine - x1 * sine;
      x1 = x0 * sine + x1 * cosine;
      x0 = u;
    }
    __nv_bfloat16* kr = static_cast<__nv_bfloat16*>(a.kv.rope) + row * kLatentRope;
    if (i1 == i0 + 1 && (i0 & 1) == 0) {
      *reinterpret_cast<uint32_t*>(kr + i0) = pack_bf16(x0, x1);
    } else {
      kr[i0] = __float2bfloat16_rn(x0);
      kr[i1] = __float2bfloat16_rn(x1);
    }
  }
  float v[16];
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 2); ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (F32) {
        v[4 * i + j] = __uint_as_float(w[j]);
      } else {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
  if (a.kv.fp8) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = amax > 0.f ? pow2_exponent(amax) : 0;
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    if (lane == 0) a.kv.scale[row] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    uint4 c;
    c.x = codes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    c.y = codes4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    c.z = codes4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv);
    c.w = codes4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.kv.latent) + row * kLatentDim + lane * 16) = c;
  } else {
    uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.kv.latent) + row * kLatentDim + lane * 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      o[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                        pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
  }
}

// The last rotation's fractions of a turn are kept: 32 of them a call would cost as much as the launch.
const Turns& turns_of(const RopeParams& r) {
  thread_local Turns t{};
  thread_local double base = 0.0;
  if (t.rope_dim != r.rope_dim || base != r.base) {
    for (int i = 0; i < kLatentRope / 2; ++i) {
      const double f = r.inv_freq[i] * 0.15915494309189533576888376337251;     // 1 / (2 pi)
      const double part = std::ldexp(f - std::floor(f), 64);
      t.f[i] = part < 0x1p64 ? static_cast<uint64_t>(part) : 0;
    }
    t.rope_dim = r.rope_dim;
    base = r.base;
  }
  t.interleaved = r.interleaved;
  return t;
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, const RopeParams& r, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.n + kAppendWarps - 1) / kAppendWarps));
  cfg.blockDim = dim3(kAppendWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a.src_f32 ? latent_append_kernel<true> : latent_append_kernel<false>, a, turns_of(r));
}

}  // namespace dsa
