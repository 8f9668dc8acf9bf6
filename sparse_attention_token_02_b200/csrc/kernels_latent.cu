// Append to the paged latent cache: one token's latent (512 values, which attention reads as its
// values and as most of its key) and the token's rotated key part (64 values), written to the row
// that the page table gives for the token's position.
//     row = pages[seq, p / page_size] * page_size + p % page_size
//     rope[row] = rotate(kr_new, p)                     (bf16; the indexer's rotation, fp64 angles)
//     latent[row] = c_new in bf16, or E4M3 codes with one scale
// The FP8 scale is the smallest power of two with absmax <= 448 * scale (at least 2^-100; 1 for a row of
// zeros): E4M3 is a floating format, so a power of two costs no relative precision, and the codes
// times it are exact in bf16, which attention multiplies in.
//
// Bound by HBM (about 1.2 KB read and 0.7 to 1.2 KB written a token); one warp per token with all
// its loads issued before the first use.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace dsa {

namespace {

constexpr int kAppendWarps = 8;

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
__device__ __forceinline__ float kr_value(const void* p, int f32, int64_t elem) {
  return f32 ? static_cast<const float*>(p)[elem] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[elem]);
}

__global__ void __launch_bounds__(kAppendWarps * 32) latent_append_kernel(LatentAppendArgs a, RopeParams rp) {
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x & 31;
  const int32_t t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= a.n) return;                                  // whole warps leave together
  const int32_t seq = a.seq_ids[t], pos = a.positions[t];
  if (seq < 0) return;                                   // a padding token
  // lane's latent values: 16 lane .. 16 lane + 15
  float v[16];
  if (a.src_f32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(a.c_new) + t * a.c_stride + lane * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = f[i];
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
  } else {
    const uint4* u = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.c_new) + t * a.c_stride + lane * 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 x = u[i];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
  // lane's two key values: pair `lane` while that rotates, else the next two that pass through
  const int npairs = rp.rope_dim / 2;
  const bool rotates = lane < npairs;
  const int i0 = rp.interleaved || !rotates ? 2 * lane : lane;
  const int i1 = rp.interleaved || !rotates ? 2 * lane + 1 : lane + npairs;
  float x0 = 0.f, x1 = 0.f;
  if (a.kv.rope) {
    x0 = kr_value(a.kr_new, a.src_f32, t * a.kr_stride + i0);
    x1 = kr_value(a.kr_new, a.src_f32, t * a.kr_stride + i1);
  }
  const int32_t slot = pos >= 0 ? pos / a.kv.page_size : -1;
  int32_t page = -1;
  if (seq < a.kv.num_seqs && slot >= 0 && slot < a.kv.max_pages) page = a.kv.pages[static_cast<int64_t>(seq) * a.kv.max_pages + slot];
  if (page < 0 || page >= a.kv.num_pages) {              // no such page: nothing is written
    if (lane == 0) record_error(a.err, DSA_DEVERR_PAGE, t);
    return;
  }
  const int64_t row = static_cast<int64_t>(page) * a.kv.page_size + pos % a.kv.page_size;
  if (a.kv.rope) {
    if (rotates) {
      const float2 cs = pair_cos_sin(lane, pos, rp);
      const float u = x0 * cs.x - x1 * cs.y;
      x1 = x0 * cs.y + x1 * cs.x;
      x0 = u;
    }
    __nv_bfloat16* kr = static_cast<__nv_bfloat16*>(a.kv.rope) + row * kLatentRope;
    kr[i0] = __float2bfloat16_rn(x0);
    kr[i1] = __float2bfloat16_rn(x1);
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
  return cudaLaunchKernelEx(&cfg, latent_append_kernel, a, r);
}

}  // namespace dsa
