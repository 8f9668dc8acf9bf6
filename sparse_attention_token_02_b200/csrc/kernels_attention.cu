// Attention over the paged latent cache.  Row (t, h), keys j (the selected positions, or every position
// below the token's length):
//     s_j = scale * (q_latent[t, h] . c_j + q_rope[t, h] . r_j)
//     out[t, h] = sum_j exp(s_j - m) c_j / sum_j exp(s_j - m),   lse[t, h] = m + log sum_j exp(s_j - m)
// in one pass over the keys with a running maximum m.  Keys are cut into chunks; a row's parts (one per
// chunk, each with its own m and sum) are joined by the second kernel.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;

// Cache row of position p of sequence seq, or -1 (reported) where the page table has no page for it.
__device__ __forceinline__ int64_t cache_row(const LatentView& kv, int32_t seq, int32_t p, int* err, int info) {
  const int32_t slot = p / kv.page_size;
  int32_t page = -1;
  if (slot < kv.max_pages) page = kv.pages[static_cast<int64_t>(seq) * kv.max_pages + slot];
  if (page < 0 || page >= kv.num_pages) {
    record_error(err, DSA_DEVERR_PAGE, info);
    return -1;
  }
  return static_cast<int64_t>(page) * kv.page_size + (p - slot * kv.page_size);
}

// Sequence of token t: -1 for a padding token and (reported) for one outside the page table.
__device__ __forceinline__ int32_t token_seq(const AttnArgs& a, int32_t t) {
  const int32_t s = a.seq_ids[t];
  if (s >= a.kv.num_seqs) {
    record_error(a.err, DSA_DEVERR_PAGE, t);
    return -1;
  }
  return s;
}

// Positions that token t may read: a prefix of its sequence.
__device__ __forceinline__ int32_t token_limit(const AttnArgs& a, int32_t t, int32_t seq) {
  if (seq < 0) return 0;
  const int32_t n = a.key_lens[t];
  if (n > a.max_keys) {
    record_error(a.err, DSA_DEVERR_PAGE, t);
    return a.max_keys;
  }
  return n;
}

// One warp per row at a time: the plain form of the pass, no tiles.
__global__ void __launch_bounds__(kThreads) attention_kernel(AttnArgs a, AttnPlan p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_shared = p.shared_groups * p.shared_slots;
  int item = blockIdx.x;
  int64_t row0, rows;
  int slot, token = -1;
  int32_t k0, k1;
  if (item < n_shared) {
    row0 = static_cast<int64_t>(item % p.shared_groups) * kAttnRows;
    rows = min(static_cast<int64_t>(kAttnRows), static_cast<int64_t>(a.T) * a.H - row0);
    slot = item / p.shared_groups;
    k0 = slot * p.shared_chunk;
    k1 = min(k0 + p.shared_chunk, a.shared_len);
  } else {
    item -= n_shared;
    const int g = item % p.own_groups;
    item /= p.own_groups;
    token = item % a.T;
    row0 = static_cast<int64_t>(token) * a.H + g * kAttnRows;
    rows = min(kAttnRows, a.H - g * kAttnRows);
    const int own_slot = item / a.T;
    slot = p.shared_slots + own_slot;
    const int32_t base = a.idx ? 0 : a.shared_len;
    k0 = base + own_slot * p.own_chunk;
    k1 = min(k0 + p.own_chunk, a.idx ? a.top_k : a.max_keys);
  }
  for (int64_t i = warp; i < rows; i += kThreads / 32) {
    const int64_t r = row0 + i;
    const int32_t t = static_cast<int32_t>(r / a.H), h = static_cast<int32_t>(r % a.H);
    const int32_t seq = token_seq(a, t);
    const int32_t limit = a.idx ? (seq < 0 ? 0 : a.top_k) : token_limit(a, t, seq);
    const int32_t end = min(k1, limit);
    const __nv_bfloat16* ql = static_cast<const __nv_bfloat16*>(a.q_latent) + t * a.ql_t + h * a.ql_h + lane * 16;
    float q[16], o[16], q0 = 0.f, q1 = 0.f;
    for (int e = 0; e < 16; ++e) {
      q[e] = __bfloat162float(ql[e]);
      o[e] = 0.f;
    }
    if (a.kv.rope) {
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q_rope) + t * a.qr_t + h * a.qr_h + lane * 2;
      q0 = __bfloat162float(qr[0]);
      q1 = __bfloat162float(qr[1]);
    }
    float m = -INFINITY, l = 0.f;
    for (int32_t k = k0; k < end; ++k) {
      const int32_t pos = a.idx ? a.idx[static_cast<int64_t>(t) * a.top_k + k] : k;
      if (pos < 0) continue;
      const int64_t row = cache_row(a.kv, token < 0 ? a.shared_seq : seq, pos, a.err, t);
      if (row < 0) continue;
      float c[16], s = 0.f;
      for (int e = 0; e < 16; ++e) {
        const int64_t at = row * kLatentDim + lane * 16 + e;
        if (a.kv.fp8) {
          __nv_fp8_e4m3 f;
          f.__x = static_cast<const uint8_t*>(a.kv.latent)[at];
          c[e] = static_cast<float>(f) * a.kv.scale[row];
        } else {
          c[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.kv.latent)[at]);
        }
        s += q[e] * c[e];
      }
      if (a.kv.rope) {
        const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(a.kv.rope) + row * kLatentRope + lane * 2;
        s += q0 * __bfloat162float(kr[0]) + q1 * __bfloat162float(kr[1]);
      }
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= a.scale_log2;
      const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - ref), w = exp2f(s - ref);
      l = l * f + w;
      for (int e = 0; e < 16; ++e) o[e] = o[e] * f + w * c[e];
      m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
    if (p.slots() == 1) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + r * kLatentDim + lane * 16;
      for (int e = 0; e < 16; ++e) out[e] = __float2bfloat16_rn(o[e] * inv);
      if (a.lse && lane == 0) a.lse[r] = lse2 * kLn2;
    } else {
      const int64_t pr = static_cast<int64_t>(slot) * a.T * a.H + r;
      for (int e = 0; e < 16; ++e) a.part_o[pr * kLatentDim + lane * 16 + e] = o[e] * inv;
      if (lane == 0) a.part_lse[pr] = lse2;
    }
  }
}

// Joins the parts of one row: weights 2^(lse_i - max) over their sum.  128 threads, 4 values each.
__global__ void __launch_bounds__(128) attention_join_kernel(AttnArgs a, int slots) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t r = blockIdx.x, R = static_cast<int64_t>(a.T) * a.H;
  float m = -INFINITY;
  for (int s = 0; s < slots; ++s) m = fmaxf(m, a.part_lse[s * R + r]);
  const float ref = m == -INFINITY ? 0.f : m;
  float total = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < slots; ++s) {
    const float lse = a.part_lse[s * R + r];
    if (lse == -INFINITY) continue;                      // nothing was written for it
    const float w = exp2f(lse - ref);
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + (s * R + r) * kLatentDim + threadIdx.x * 4);
    total += w;
    o.x += w * x.x; o.y += w * x.y; o.z += w * x.z; o.w += w * x.w;
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + r * kLatentDim + threadIdx.x * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (a.lse && threadIdx.x == 0) a.lse[r] = total == 0.f ? -INFINITY : (m + log2f(total)) * kLn2;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

AttnPlan plan_attention(int64_t T, int32_t H, int64_t shared_keys, int64_t own_keys, int sms) {
  const int64_t R = T * H, shared_tiles = ceil_div(shared_keys, kAttnTile);
  // a call with no keys at all still writes its empty rows
  const int64_t own_tiles = own_keys > 0 || shared_keys == 0 ? std::max<int64_t>(1, ceil_div(own_keys, kAttnTile)) : 0;
  const int64_t longest = std::max(shared_tiles, own_tiles);
  AttnPlan best{};
  double best_cost = 0.0;
  for (int64_t k = 1; k <= std::min<int64_t>(longest, 160); ++k) {
    const int64_t chunk = ceil_div(longest, k);
    AttnPlan p{};
    p.shared_groups = static_cast<int32_t>(ceil_div(R, kAttnRows));
    p.own_groups = static_cast<int32_t>(ceil_div(H, kAttnRows));
    p.shared_slots = static_cast<int32_t>(ceil_div(shared_tiles, chunk));
    p.own_slots = static_cast<int32_t>(ceil_div(own_tiles, chunk));
    p.shared_chunk = p.own_chunk = static_cast<int32_t>(std::min<int64_t>(chunk, longest) * kAttnTile);
    const int64_t items = int64_t(p.shared_groups) * p.shared_slots + T * p.own_groups * p.own_slots;
    const double cost = ceil_div(items, sms) * (chunk + 4.0) + (p.slots() > 1 ? 3.0 + p.slots() * R * 0.0006 : 0.0);
    if (k == 1 || cost < best_cost) {
      best = p;
      best_cost = cost;
    }
  }
  return best;
}

size_t attention_workspace(const AttnPlan& p, int64_t T, int32_t H) {
  return p.slots() > 1 ? size_t(p.slots()) * T * H * (kLatentDim + 1) * sizeof(float) : 0;
}

cudaError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int* launched, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(int64_t(p.shared_groups) * p.shared_slots + int64_t(a.T) * p.own_groups * p.own_slots));
  cfg.blockDim = dim3(kThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, attention_kernel, a, p);
  if (e != cudaSuccess) return e;
  ++*launched;
  if (p.slots() > 1) {
    cfg.gridDim = dim3(static_cast<unsigned>(int64_t(a.T) * a.H));
    cfg.blockDim = dim3(128);
    e = cudaLaunchKernelEx(&cfg, attention_join_kernel, a, static_cast<int>(p.slots()));
    if (e != cudaSuccess) return e;
    ++*launched;
  }
  return cudaSuccess;
}

}  // namespace dsa
