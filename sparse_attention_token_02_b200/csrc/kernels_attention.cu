// Attention over the paged latent cache.  Row (t, h), keys j (the selected positions, or every position
// below the token's length):
//     s_j = scale * (q_latent[t, h] . c_j + q_rope[t, h] . r_j)
//     out[t, h] = sum_j exp(s_j - m) c_j / sum_j exp(s_j - m),   lse[t, h] = m + log sum_j exp(s_j - m)
// in one pass over the keys with a running maximum m.  Keys are cut into chunks; a row's parts (one per
// chunk, each with its own m and sum) are joined by the second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

// The page table's entry for position p (>= 0) of sequence seq: -1 past its columns.
__device__ __forceinline__ int32_t page_entry(const LatentView& kv, int32_t seq, int32_t p) {
  const int32_t slot = kv.page_shift >= 0 ? p >> kv.page_shift : p / kv.page_size;
  return slot < kv.max_pages ? __ldg(kv.pages + static_cast<int64_t>(seq) * kv.max_pages + slot) : -1;
}

// Cache row of position p on that page, or -1 (reported) where there is no such page.
__device__ __forceinline__ int32_t page_row(const LatentView& kv, int32_t page, int32_t p, int* err, int info) {
  if (page < 0 || page >= kv.num_pages) {
    record_error(err, DSA_DEVERR_PAGE, info);
    return -1;
  }
  const int32_t in_page = kv.page_shift >= 0 ? p & (kv.page_size - 1) : p % kv.page_size;
  return page * kv.page_size + in_page;                  // fewer than 2^31 rows
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

// ------------------------------------------------------------------------------------------------ the pass

// Shared memory of a CTA: operand blocks of 64 rows x 64 values (128-byte rows, 128-byte swizzle): the
// rotated part of the queries, then three stages of keys.  A tile's weights take the place of its keys' rotated
// part, which only the first product reads.
constexpr uint32_t kBlock = 64 * 128;
constexpr int kLatentBlocks = kLatentDim / 64;               // 8; the rotated part is a ninth
constexpr int kHalf = kLatentBlocks / 2;                     // blocks per half: values 0 .. 255, 256 .. 511
constexpr uint32_t kStage = (kLatentBlocks + 1) * kBlock;
constexpr uint32_t kRotated = kLatentBlocks * kBlock;        // within a stage
constexpr int kStages = 3;
constexpr uint32_t kOffK = kBlock;
constexpr uint32_t kSmemBytes = kOffK + kStages * kStage;
// the result on its way out, over the keys' stages: rows of 512 fp32 or bf16 values, padded to spread the banks
constexpr uint32_t kOutRow32 = kLatentDim * 4 + 16, kOutRow16 = kLatentDim * 2 + 16;
static_assert(64 * kOutRow32 <= kStages * kStage, "the result must fit");

// Tensor memory.  A 64-row accumulator fills 16 of every 32 lanes, and a product's A operand in tensor memory
// sits in the lanes of its result, so the values 0 .. 255 live in the lower 16 lanes and 256 .. 511 in
// the upper 16: the queries (128 columns of bf16 pairs), two tiles of scores (64 columns each, one sum for
// either half of the values, added when they are read) and the output (256 columns).  Keeping the queries here
// leaves the shared memory's bandwidth, which bounds a 64 x 64 product with both operands in it, to the
// keys, and its room to a third stage.
// All 512 columns are taken, so the allocation starts at column 0, a constant for the issuing thread.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;
constexpr uint32_t kTmemS = 256;
constexpr uint32_t kTmemQ = 384;
constexpr uint32_t kUpperLanes = 16u << 16;

constexpr int kSoftmaxWarps = 4;
constexpr int kFirstWarp = 4, kSecondWarp = 5;                // issue the first and the second products
constexpr int kLoadWarp0 = 6;
constexpr int kLoadWarps = 8;
constexpr int kThreads = (kLoadWarp0 + kLoadWarps) * 32;

// The running maximum may lag behind the true one by this much (base 2) before the sums are rescaled:
// fp32 sums and bf16 weights lose nothing by weights of up to 2^8.
constexpr float kLag = 8.0f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two E4M3 codes (the low 16 bits) times a power of two, exact in bf16.  The two conversions and the products
// spread over the ALU and FMA pipes; moving the bits by hand (a byte permutation, a shift, two logic instructions
// and one product for a pair, and a look for NaN codes) kept the ALU pipe busy for longer.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes, float scale) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(codes));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return bf16x2(f.x * scale, f.y * scale);
}

__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void st_shared_f32(uint32_t dst, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(v) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t src) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(src) : "memory");
  return v;
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}

// Zeroes what is not finite in `bytes` of bf16 values from `base`, by the 128 threads of the softmax warps.  A key that a row
// may not read has weight 0 there, but 0 * NaN would still reach the row's output; rows that do read it have a score,
// and with it every weight, that is not finite already.  (Minus infinity aside: that key then has weight 0 for them.)
__device__ __forceinline__ void keep_finite(uint32_t base, uint32_t bytes, int thread) {
#pragma unroll 1
  for (uint32_t at = base + thread * 16; at < base + bytes; at += 128 * 16) {
    const uint4 u = ld_shared16(at);
    uint32_t w[4] = {u.x, u.y, u.z, u.w}, any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t wild = __vcmpeq2(w[i] & 0x7F807F80u, 0x7F807F80u);   // an exponent of ones, in either half
      w[i] &= ~wild;
      any |= wild;
    }
    if (any) st_shared16(at, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

struct __align__(8) Shared {
  uint64_t full[kStages][2];    // a half of a tile's keys is in shared memory (the second half with the rotated part)
  uint64_t listed[kStages];     // `valid` of a tile is written
  uint64_t empty[kStages][2];   // a half of the tile's second product is done
  uint64_t scores[2];           // a score tile is complete
  uint64_t taken[2];            // and read
  uint64_t weights[2];          // the weights of a tile are in shared memory, the output is rescaled
  uint64_t queries;             // the queries are in tensor memory
  uint64_t drained[2];          // every first, every second product of the CTA is done
  uint32_t tmem;
  int abort;
  int32_t key_end;
  int32_t first_limit;          // the smallest limit of a row that has keys here, where rows of several tokens meet
  int32_t limit[kAttnRows];     // keys at or past a row's limit are not its own
  float inv[kAttnRows];         // 1 / the row's sum (0 for a row without keys)
  float lse2[kAttnRows];        // the base-2 log of the row's sum
  alignas(8) uint8_t valid[kStages][kLoadWarps];   // keys of a tile that exist, one bit each
};

// One CTA per work item: 64 rows against the keys [k0, key_end) in tiles of 64.
//   8 warps bring each key's row into shared memory (gathered by 16-byte copies; FP8 rows are expanded to
//   bf16 on the way), one thread each issues the products S = Q K^T (64 x 64 x 576) and O += P V (64 x 512
//   x 64; V is the same tile read with its values contiguous), 4 warps turn S into weights P.
// The scores of tile i + 1 are computed while the weights of tile i are made.  Tiles go in and out in halves
// of 256 values, so that the loads of one half run under the products of the other.
// The roles' loops are kept small: together they have to fit the instruction cache.
template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(AttnArgs a, AttnPlan p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem = smem_addr(smem_raw);             // a constant, and the operands' addresses with it

  // the item
  const int n_shared = p.shared_groups * p.shared_slots;
  int item = blockIdx.x + a.first_item;
  int row0;                      // first of the item's rows in the packed [T, H]
  int rows, slot, token = -1;
  if (p.cluster > 1) {
    slot = item % p.cluster;
    item /= p.cluster;
    const int g = item % p.own_groups;
    token = item / p.own_groups;
    row0 = token * a.H + g * p.own_rows;
    rows = min(p.own_rows, a.H - g * p.own_rows);
  } else if (item < n_shared) {
    row0 = item % p.shared_groups * kAttnRows;
    rows = min(kAttnRows, a.T * a.H - row0);
    slot = item / p.shared_groups;
  } else {
    item -= n_shared;
    const int g = item % p.own_groups;
    item /= p.own_groups;
    token = item % a.T;
    row0 = token * a.H + g * p.own_rows;
    rows = min(p.own_rows, a.H - g * p.own_rows);
    slot = p.shared_slots + item / a.T;
  }
  int32_t k0, k1;                // its keys, before lengths are known
  if (token < 0) {
    k0 = slot * p.shared_chunk;
    k1 = min(k0 + p.shared_chunk, a.shared_len);
  } else {
    k0 = (p.shared_slots ? a.shared_len : 0) + (slot - p.shared_slots) * p.own_chunk;
    k1 = min(k0 + p.own_chunk, a.idx ? a.top_k : a.max_keys);
  }
  const LatentView& kv = token < 0 ? a.shared : a.kv;
  const bool fp8 = FP8 && (token >= 0 || !p.expand);
  const int stages = fp8 ? kStages - 1 : kStages;
  const bool rotated = a.kv.rope != nullptr;

  if (warp == kFirstWarp) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        for (int h = 0; h < 2; ++h) {
          mbar_init(&sh.full[i][h], fp8 ? kLoadWarps : kLoadWarps * 32);   // a warp's stores, or each thread's copies
          mbar_init(&sh.empty[i][h], 1);
        }
        mbar_init(&sh.listed[i], kLoadWarps);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.scores[i], 1);
        mbar_init(&sh.taken[i], kSoftmaxWarps);
        mbar_init(&sh.weights[i], kSoftmaxWarps);
        mbar_init(&sh.drained[i], 1);
      }
      mbar_init(&sh.queries, kSoftmaxWarps);
      sh.abort = 0;
      sh.key_end = 0;
      sh.first_limit = 0x7FFFFFFF;
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(&sh.tmem, kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  grid_dependency_wait();

  const int32_t* idx = a.idx ? a.idx + static_cast<int64_t>(token) * a.top_k : nullptr;
  const int32_t shared_seq = p.expand ? 0 : a.shared_seq;
  int32_t seq = shared_seq;
  if (token < 0) {
    if (tid < kAttnRows) {
      int32_t n = 0;
      if (tid < rows) {
        const int32_t t = (row0 + tid) / a.H;
        n = token_limit(a, t, token_seq(a, t));
      }
      sh.limit[tid] = n;
      atomicMax(&sh.key_end, min(n, k1));
      if (n > k0) atomicMin(&sh.first_limit, n);
    }
  } else {
    seq = token_seq(a, token);
    if (idx == nullptr) {
      const int32_t n = token_limit(a, token, seq);
      if (tid < kAttnRows) sh.limit[tid] = n;
      if (tid == 0) sh.key_end = min(n, k1);
    } else {
      // entries behind the last valid one (short histories are padded) are not visited
      if (tid < kAttnRows) sh.limit[tid] = 0x7FFFFFFF;
      int32_t last = 0;
      for (int32_t k = k0 + tid; k < k1; k += 8 * kThreads) {
        int32_t e[8];                                    // loads side by side
#pragma unroll
        for (int x = 0; x < 8; ++x) e[x] = k + x * kThreads < k1 ? __ldg(idx + k + x * kThreads) : -1;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (e[x] >= 0) last = k + x * kThreads + 1;
      }
      last = __reduce_max_sync(0xffffffffu, seq < 0 ? 0 : last);
      if (lane == 0 && last > 0) atomicMax(&sh.key_end, last);
    }
  }
  __syncthreads();
  const int32_t key_end = sh.key_end, first_limit = sh.first_limit;
  const int tiles = key_end > k0 ? (key_end - k0 + kAttnTile - 1) / kAttnTile : 0;
  tc_fence_after();

  if (warp >= kLoadWarp0) {
    // ---------------------------------------------------------------- loads
    const int lw = warp - kLoadWarp0;                    // rows 8 lw .. 8 lw + 7 of every block
    const int sub = lane >> 3, col = lane & 7;           // a lane's 16-byte column, rows sub and sub + 4
    if (rotated && tiles > 0) {
#pragma unroll 1
      for (int r = lw * 8 + sub; r < lw * 8 + 8; r += 4) {   // the queries' rotated part, wanted with the first tile's
        const int qr = row0 + (r < rows ? r : 0);
        const int t = qr / a.H, h = qr - t * a.H;
        cp_async16(smem + r * 128 + ((col ^ (r & 7)) << 4),
                   static_cast<const __nv_bfloat16*>(a.q_rope) + t * a.qr_t + h * a.qr_h + col * 8, r < rows);
      }
    }
    // This warp's key `col` of a tile, the same in the lanes of one column: its position (-1: none) is read two tiles
    // ahead, its page one, so that neither load is waited for.
    int32_t pos2 = -1, pos1 = -1, page1 = -1, row = -1;
    auto advance = [&](int n) {
      row = pos1 < 0 ? -1 : page_row(kv, page1, pos1, a.err, token < 0 ? row0 / a.H : token);
      // shared positions are read through the one sequence whichever item reads them
      page1 = pos2 < 0 ? -1 : page_entry(kv, pos2 < a.shared_len ? shared_seq : seq, pos2);
      pos1 = pos2;
      const int32_t k = k0 + n * kAttnTile + lw * 8 + col;
      pos2 = k < key_end ? (idx ? __ldg(idx + k) : k) : -1;
    };
    int st = 0;
    uint32_t phase = 1;                                  // the stages start free
    auto place = [&](int h) {                            // whether half h of the stage is free, for the warp as one
      const bool ok = mbar_wait<true>(&sh.empty[st][h], phase, &sh.abort);
      return __all_sync(0xffffffffu, ok);
    };
    auto list = [&](uint32_t valid) {
      if (lane == 0) {
        sh.valid[st][lw] = static_cast<uint8_t>(valid);
        mbar_arrive(&sh.listed[st]);
      }
    };
    auto next_stage = [&] {
      if (++st == stages) {
        st = 0;
        phase ^= 1;
      }
    };
    if (!fp8) {
      for (int n = 0; n < tiles + 2; ++n) {
        advance(n);                                      // the rows of tile n - 2
        if (n < 2) continue;
        const uint32_t valid = __ballot_sync(0xffffffffu, row >= 0) & 0xFFu;
        const uint32_t stage = smem + kOffK + st * kStage + lw * 8 * 128;
        const int32_t ra = __shfl_sync(0xffffffffu, row, sub), rb = __shfl_sync(0xffffffffu, row, sub + 4);
        const __nv_bfloat16* sa = static_cast<const __nv_bfloat16*>(kv.latent) + static_cast<int64_t>(max(ra, 0)) * kLatentDim + col * 8;
        const __nv_bfloat16* sb = static_cast<const __nv_bfloat16*>(kv.latent) + static_cast<int64_t>(max(rb, 0)) * kLatentDim + col * 8;
        const uint32_t da = stage + sub * 128 + ((col ^ sub) << 4), db = stage + (sub + 4) * 128 + ((col ^ (sub + 4)) << 4);
        bool ok = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = place(h);
          if (!ok) break;
          if (h == 1) list(valid);
#pragma unroll
          for (int c = h * kHalf; c < h * kHalf + kHalf; ++c) {
            cp_async16(da + c * kBlock, sa + c * 64, ra >= 0);
            cp_async16(db + c * kBlock, sb + c * 64, rb >= 0);
          }
          if (h == 1 && rotated) {
            const __nv_bfloat16* rope = static_cast<const __nv_bfloat16*>(kv.rope) + col * 8;
            cp_async16(da + kRotated, rope + static_cast<int64_t>(max(ra, 0)) * kLatentRope, ra >= 0);
            cp_async16(db + kRotated, rope + static_cast<int64_t>(max(rb, 0)) * kLatentRope, rb >= 0);
          }
          cp_async_arrive(&sh.full[st][h]);              // when this thread's copies so far have landed
        }
        if (!ok) break;
        next_stage();
      }
    } else {
      // FP8 rows come through the place of the third stage, two tiles ahead: every warp copies its own eight rows there
      // (512 bytes each) and expands them from there.  The 16 codes vec of row 2 j + pair are a lane's: eight
      // neighbouring lanes hold four vectors of an even and of an odd row, whose places in an operand block fall on
      // different banks, and so do theirs in the codes' (an odd row's vectors sit four places on).
      const int pair = (lane >> 2) & 1, vec = (lane & 3) + 4 * (lane >> 3);
      const uint32_t ring = smem + kOffK + (kStages - 1) * kStage + lw * 4096;
      // scales, existing keys and rotated parts of the tiles n - 3 and n - 4 (their rows sub and sub + 4, column col)
      float scale1 = 0.f, scale2 = 0.f;
      uint32_t valid1 = 0, valid2 = 0;
      uint4 turned1[2], turned2[2];
      for (int n = 0; n < tiles + 4; ++n) {
        advance(n);                                      // the rows of tile n - 2
        const uint32_t codes = ring + (n & 1) * 32768;
        if (n >= 4) {
          const uint32_t stage = smem + kOffK + st * kStage + lw * 8 * 128;
          cp_async_wait<1>();                            // all but the latest tile's codes
          __syncwarp();
          uint4 u[2][4];                                 // together: what follows waits for each of them
          float s[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r8 = 2 * j + pair;
            s[j] = __shfl_sync(0xffffffffu, scale2, r8);
#pragma unroll
            for (int h = 0; h < 2; ++h) u[h][j] = ld_shared16(codes + r8 * 512 + (((h * 16 + vec) ^ (pair << 2)) << 4));
          }
          bool ok = true;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = place(h);
            if (!ok) break;
            if (h == 1) {
              list(valid2);
              if (rotated) {
                st_shared16(stage + kRotated + sub * 128 + ((col ^ sub) << 4), turned2[0]);
                st_shared16(stage + kRotated + (sub + 4) * 128 + ((col ^ (sub + 4)) << 4), turned2[1]);
              }
            }
            // two 16-byte columns of block vec / 4
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r8 = 2 * j + pair;
              const uint32_t w[4] = {u[h][j].x, u[h][j].y, u[h][j].z, u[h][j].w};
              const uint32_t base = stage + (h * kHalf + (vec >> 2)) * kBlock + r8 * 128;
#pragma unroll
              for (int x = 0; x < 2; ++x)
                st_shared16(base + ((((vec & 3) * 2 + x) ^ r8) << 4),
                            make_uint4(e4m3x2_to_bf16x2(w[2 * x] & 0xFFFFu, s[j]), e4m3x2_to_bf16x2(w[2 * x] >> 16, s[j]),
                                       e4m3x2_to_bf16x2(w[2 * x + 1] & 0xFFFFu, s[j]), e4m3x2_to_bf16x2(w[2 * x + 1] >> 16, s[j])));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full[st][h]);
          }
          if (!ok) break;
          next_stage();
        }
        scale2 = scale1;
        valid2 = valid1;
        scale1 = row >= 0 ? __ldg(kv.scale + row) : 0.f;
        valid1 = __ballot_sync(0xffffffffu, row >= 0) & 0xFFu;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int32_t rj = __shfl_sync(0xffffffffu, row, sub + 4 * j);
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(kv.rope) + static_cast<int64_t>(rj) * kLatentRope) + col;
          turned2[j] = turned1[j];
          turned1[j] = rotated && rj >= 0 ? __ldg(src) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int32_t rj = __shfl_sync(0xffffffffu, row, j);
          cp_async16(codes + j * 512 + ((lane ^ ((j & 1) << 2)) << 4),
                     static_cast<const uint8_t*>(kv.latent) + static_cast<int64_t>(max(rj, 0)) * kLatentDim + lane * 16, rj >= 0);
        }
        cp_async_commit();
      }
    }
    cp_async_wait_all();
  } else if (warp == kFirstWarp) {
    // ---------------------------------------------------------------- scores = Q K^T
    // Two warps issue, one per product: the tensor cores take either's next while the other's issuer waits or
    // reads a barrier (300 cycles between two batches of one issuer stood idle otherwise).
    if (elect_one()) {
      constexpr uint32_t idesc = make_idesc(1, kAttnRows, kAttnTile);
      bool ok = tiles == 0 || mbar_wait<true>(&sh.queries, 0, &sh.abort);
      int st = 0;
      uint32_t phase = 0;
      for (int i = 0; i < tiles && ok; ++i) {
        const uint32_t stage = smem + kOffK + st * kStage;
        const uint32_t d = kTmemS + (i & 1) * kAttnTile;
        if (i >= 2) ok = mbar_wait<true>(&sh.taken[i & 1], ((i >> 1) - 1) & 1, &sh.abort);
        ok = ok && mbar_wait<true>(&sh.full[st][0], phase, &sh.abort);
        if (!ok) break;
        fence_proxy_async_smem();                        // the copies that the barrier reported
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kHalf; ++c)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_ts(d, kTmemQ + (c * 4 + ks) * 8, sdesc_kmajor_sw128(stage + c * kBlock + ks * 32), idesc, c > 0 || ks > 0);
        ok = mbar_wait<true>(&sh.full[st][1], phase, &sh.abort);
        if (!ok) break;
        fence_proxy_async_smem();
#pragma unroll
        for (int c = 0; c < kHalf; ++c)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_ts(d + kUpperLanes, kTmemQ + (c * 4 + ks) * 8 + kUpperLanes,
                        sdesc_kmajor_sw128(stage + (kHalf + c) * kBlock + ks * 32), idesc, c > 0 || ks > 0);
        if (rotated) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16(d + kUpperLanes, sdesc_kmajor_sw128(smem + ks * 32), sdesc_kmajor_sw128(stage + kRotated + ks * 32), idesc, 1);
        }
        umma_commit(&sh.scores[i & 1]);
        if (++st == stages) {
          st = 0;
          phase ^= 1;
        }
      }
      umma_commit(&sh.drained[0]);
      int alone = 0;                                     // also after an abort: nothing may run on freed tensor memory
      mbar_wait<true>(&sh.drained[0], 0, &alone);
    }
    __syncwarp();
  } else if (warp == kSecondWarp) {
    // ---------------------------------------------------------------- output += P V
    if (elect_one()) {
      constexpr uint32_t idesc = make_idesc(1, kAttnRows, 256) | kIdescBMnMajor;
      int st = 0;
      for (int i = 0; i < tiles; ++i) {
        // the weights came from scores of the same keys, so those are in shared memory
        if (!mbar_wait<true>(&sh.weights[i & 1], (i >> 1) & 1, &sh.abort)) break;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t stage = smem + kOffK + st * kStage;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int ks = 0; ks < kAttnTile / 16; ++ks)
            umma_f16(kTmemO + h * kUpperLanes, sdesc_kmajor_sw128(stage + kRotated + ks * 32),
                     sdesc_mnmajor_sw128(stage + h * kHalf * kBlock + ks * 2048, kBlock), idesc, i > 0 || ks > 0);
          umma_commit(&sh.empty[st][h]);
        }
        if (++st == stages) st = 0;
      }
      umma_commit(&sh.drained[1]);
      int alone = 0;
      mbar_wait<true>(&sh.drained[1], 0, &alone);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- weights
    // The thread's two rows of the score tile: lane / 4 and lane / 4 + 8 of the warp's 16, 16 columns of each.
    const int fr = lane >> 2;
    const int32_t limit[2] = {sh.limit[warp * 16 + fr], sh.limit[warp * 16 + fr + 8]};
    const uint32_t quadrant = static_cast<uint32_t>(warp * 32) << 16;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool ok = true;
    if (tiles > 0) {
      // the queries: a lane brings 256 values of the row lane % 16
      const int r = warp * 16 + (lane & 15);
      const int qr = row0 + (r < rows ? r : 0);
      const int t = qr / a.H, h = qr - t * a.H;
      const uint4* ql = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_latent) + t * a.ql_t + h * a.ql_h + (lane >> 4) * 256);
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        uint4 x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = r < rows ? __ldg(ql + c / 4 + e) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t v[32];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[4 * e] = x[8 * y + e].x; v[4 * e + 1] = x[8 * y + e].y; v[4 * e + 2] = x[8 * y + e].z; v[4 * e + 3] = x[8 * y + e].w;
          }
          tmem_st_32x32b_x32(quadrant + kTmemQ + c + 32 * y, v);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.queries);
    }
    int st = 0;
    uint32_t phase = 0;
    for (int i = 0; i < tiles; ++i) {
      ok = mbar_wait<true>(&sh.scores[i & 1], (i >> 1) & 1, &sh.abort);
      ok = ok && mbar_wait<true>(&sh.listed[st], phase, &sh.abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tile = quadrant + kTmemS + (i & 1) * kAttnTile;
      uint32_t raw[32], raw2[32];                        // the scores over either half of the values
      tmem_ld_16x256b_x8(tile, raw);
      tmem_ld_16x256b_x8(tile + kUpperLanes, raw2);
      const uint64_t present = *reinterpret_cast<const uint64_t*>(sh.valid[st]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.taken[i & 1]);
      float x[2][16];
      const int32_t kb = k0 + i * kAttnTile;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            x[r][2 * j + e] = __uint_as_float(raw[4 * j + 2 * r + e]) + __uint_as_float(raw2[4 * j + 2 * r + e]);
      const bool whole = present == ~0ull && limit[0] - kb >= kAttnTile && limit[1] - kb >= kAttnTile;
      if (!__all_sync(0xffffffffu, whole)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int32_t n = limit[r] - kb;               // the row's keys of this tile
          uint64_t mine = n >= kAttnTile ? present : n <= 0 ? 0ull : present & ((1ull << n) - 1);
          mine >>= 2 * (lane & 3);
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((mine >> (8 * j + e)) & 1)) x[r][2 * j + e] = -INFINITY;
        }
      }
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = x[r][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) mx[r] = fmaxf(mx[r], x[r][e]);
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2)) * a.scale_log2;   // the scale is positive
      }
      const bool rescale = __any_sync(0xffffffffu, mx[0] > m[0] + kLag || mx[1] > m[1] + kLag);
      float factor[2] = {1.f, 1.f};
      if (rescale) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mn = fmaxf(m[r], mx[r]);
          factor[r] = mn == -INFINITY ? 1.f : exp2_fast(m[r] - mn);
          l[r] *= factor[r];
          m[r] = mn;
        }
      }
      const uint32_t place = smem + kOffK + st * kStage + kRotated + (warp * 16 + fr) * 128 + (lane & 3) * 4;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float lo = exp2_fast(fmaf(x[r][2 * j], a.scale_log2, -ref)), hi = exp2_fast(fmaf(x[r][2 * j + 1], a.scale_log2, -ref));
          l[r] += lo + hi;                               // the sum keeps fp32; the product's operand is bf16
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(place + r * 1024 + ((j ^ fr) << 4)), "r"(bf16x2(lo, hi)) : "memory");
        }
      }
      if (rescale && i > 0) {
        // the output of the tiles before this one, complete, times the factor
        const int before = st == 0 ? stages - 1 : st - 1;
        ok = mbar_wait<true>(&sh.empty[before][1], st == 0 ? phase ^ 1 : phase, &sh.abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // an output lane's row is lane % 16: its factor sits with the lanes 4 (row % 8) of the score layout
        const float f0 = __shfl_sync(0xffffffffu, factor[0], (lane & 7) * 4);
        const float f1 = __shfl_sync(0xffffffffu, factor[1], (lane & 7) * 4);
        const float f = lane & 8 ? f1 : f0;
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(quadrant + kTmemO + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st_32x32b_x32(quadrant + kTmemO + c, o);
        }
        tmem_st_wait();
      }
      if (first_limit < min(kb + kAttnTile, key_end)) {  // a row that ended before the tile's last key
        ok = mbar_wait<true>(&sh.full[st][0], phase, &sh.abort) && mbar_wait<true>(&sh.full[st][1], phase, &sh.abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        keep_finite(smem + kOffK + st * kStage, kLatentBlocks * kBlock, tid);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.weights[i & 1]);
      if (++st == stages) {
        st = 0;
        phase ^= 1;
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int at = warp * 16 + fr + 8 * r;
      if ((lane & 3) == 0 && ok) {
        sh.inv[at] = l[r] == 0.f ? 0.f : 1.f / l[r];
        const float lse2 = l[r] == 0.f ? -INFINITY : m[r] + log2f(l[r]);
        sh.lse2[at] = lse2;
        if (at < rows && p.cluster == 1) {
          if (p.parts()) a.part_lse[static_cast<int64_t>(slot) * a.T * a.H + row0 + at] = lse2;
          else if (a.lse) a.lse[row0 + at] = lse2 * kLn2;
        }
      }
    }
  }

  // ---------------------------------------------------------------- the result
  // Every product is done and every copy has landed; the keys' place takes the result, whose rows then go out whole.
  launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool wide = p.cluster > 1 || p.parts();          // parts are fp32
  const bool given_up = *const_cast<volatile int*>(&sh.abort) != 0;
  if (given_up) {
    if (tid == 0) record_error(a.err, DSA_DEVERR_TIMEOUT, static_cast<int>(blockIdx.x));
  } else if (tiles > 0 || !wide) {
    const uint32_t stride = wide ? kOutRow32 : kOutRow16;
    if (warp < 12) {                                     // three warps for each of the tensor memory's quarters
      const int r = (warp & 3) * 16 + (lane & 15);
      const float inv = sh.inv[r];
      const uint32_t mem = smem + kOffK + r * stride + (lane >> 4) * (wide ? 1024 : 512);
#pragma unroll 1
      for (int c = (warp >> 2) * 16; c < 256; c += 48) {
        uint32_t o[16];
        tmem_ld_32x32b_x16((static_cast<uint32_t>((warp & 3) * 32) << 16) + kTmemO + c, o);
        tmem_ld_wait();
        // a row without keys is zero whatever its weights' products with foreign keys (or nothing at all) left
        float val[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) val[e] = inv == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
        if (wide) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            st_shared16(mem + (c + e) * 4, make_uint4(__float_as_uint(val[e]), __float_as_uint(val[e + 1]),
                                                      __float_as_uint(val[e + 2]), __float_as_uint(val[e + 3])));
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            st_shared16(mem + (c + e) * 2, make_uint4(bf16x2(val[e], val[e + 1]), bf16x2(val[e + 2], val[e + 3]),
                                                      bf16x2(val[e + 4], val[e + 5]), bf16x2(val[e + 6], val[e + 7])));
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    if (p.cluster == 1) {
      const int shift = wide ? 7 : 6;                    // 16-byte vectors of a row: 512 fp32 or bf16 values
      uint4* out = wide ? reinterpret_cast<uint4*>(a.part_o) + ((static_cast<int64_t>(slot) * a.T * a.H + row0) << shift)
                        : static_cast<uint4*>(a.out) + (static_cast<int64_t>(row0) << shift);
#pragma unroll 2
      for (int v = tid; v < rows << shift; v += kThreads)
        out[v] = ld_shared16(smem + kOffK + (v >> shift) * stride + (v & ((1 << shift) - 1)) * 16);
    }
  }
  if (p.cluster > 1) {
    // The cluster's CTAs hold the parts of the same rows: each joins a share of the rows, four values a thread, from
    // everyone's shared memory, with weights 2^(lse_i - max) over their sum.
    cluster_arrive();
    cluster_wait();
    const int r0 = rows * slot / p.cluster, r1 = rows * (slot + 1) / p.cluster;
    const uint32_t table = smem;                         // [r1 - r0][16] weights, where the queries' rotated part was
    if (tid < r1 - r0) {
      const uint32_t at = smem_addr(&sh.lse2[r0 + tid]);
      float w[kMaxCluster], top = -INFINITY, total = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) w[i] = i < p.cluster ? ld_cluster_f32(cluster_addr(at, i)) : -INFINITY;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) top = fmaxf(top, w[i]);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) total += w[i] = exp2f(w[i] - ref);
      const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) st_shared_f32(table + (tid * kMaxCluster + i) * 4, w[i] * inv);
      if (a.lse) a.lse[row0 + r0 + tid] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
    }
    __syncthreads();
    for (int v = tid; v < (r1 - r0) * 128; v += kThreads) {
      const int r = v >> 7, c = v & 127;
      const uint32_t val = smem + kOffK + (r0 + r) * kOutRow32 + c * 16;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int i = 0; i < p.cluster; i += 8) {           // eight loads under way: a neighbour's memory is far
        float4 x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + e < p.cluster) x[e] = ld_cluster_f32x4(cluster_addr(val, i + e));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = i + e < p.cluster ? ld_shared_f32(table + (r * kMaxCluster + i + e) * 4) : 0.f;
          if (w != 0.f) {                                // else there may be nothing, or anything, in its place
            o.x += w * x[e].x; o.y += w * x[e].y; o.z += w * x[e].z; o.w += w * x[e].w;
          }
        }
      }
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<int64_t>(row0 + r0 + r) * kLatentDim + c * 4) =
          make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
    }
    cluster_arrive();                                    // nobody leaves while its shared memory is read
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kFirstWarp) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------------------------------------ the pass, in pairs
//
// Two CTAs (a cluster) take 128 rows, 64 each, against the same keys: products of 128 rows over a pair of SMs run at the
// tensor cores' full rate, where 64 rows on one run at half.  For the scores a CTA holds half of a tile's keys (32 rows
// of 576 values), for the second product half of the values of all its keys (64 rows of 256).  Keys and values have
// their own stages: a tile's keys are free after its scores, its values after the second product.  CTA 0 issues; CTA 1's
// two idle warps tell it when their CTA's keys and values have landed.  (64 x 128 heads over 2048 selected keys 69 us with
// one CTA per 64 rows, 55 in pairs; 1024 tokens 805 and 687 to 700.)  With the keys in L2 a tile takes about 1800 cycles: 1280 of
// products, about 1500 of shared memory (operands 860, copies in 540, weights 100); neither is busy throughout, and the
// rest goes to the hand-overs between loads, products and weights.  Copying the values of a CTA's own keys from its keys' stage, which spares a quarter
// of the reads of L2, cost 743 us for the 703 of then; a third stage of keys for one of values changed nothing.
constexpr uint32_t kPairKeys = (kLatentBlocks + 1) * 4096u;  // 32 rows x 9 blocks
constexpr uint32_t kPairValues = 4 * kBlock;                 // 64 rows x 4 blocks
constexpr int kKeyStages = 2, kValueStages = 3;
constexpr int kPairQBlocks = 3;                              // the queries' values 384 .. 511 and rotated part
constexpr uint32_t kPairP = kPairQBlocks * kBlock;           // two tiles' weights
constexpr uint32_t kPairK = kPairP + 2 * kBlock;
constexpr uint32_t kPairV = kPairK + kKeyStages * kPairKeys;
constexpr uint32_t kPairSmem = kPairV + kValueStages * kPairValues;
static_assert(64 * kOutRow32 <= kPairSmem - kPairK, "the result must fit");
// tensor memory: the output (two products of 256 values, 128 columns each), two score tiles, the queries' values 0 .. 383
constexpr uint32_t kPairTmemS = 256;
constexpr uint32_t kPairTmemQ = 320;

struct __align__(8) SharedPair {
  uint64_t keys[kKeyStages], values[kValueStages];           // this CTA's copies have landed
  uint64_t peer_keys[kKeyStages], peer_values[kValueStages]; // CTA 0's: and CTA 1's
  uint64_t scores[2];           // a score tile is complete, its keys' stage free
  uint64_t used[kValueStages];  // the tile's second product is done
  uint64_t taken[2], weights[2];   // CTA 0's: both CTAs have read the scores, have written the weights
  uint64_t listed[kValueStages];
  uint64_t queries;             // CTA 0's: both CTAs' queries are in tensor memory
  uint64_t moved;               // the last stage of values no longer holds queries
  uint64_t drained[2];
  uint32_t tmem;
  int abort;
  int32_t key_end, first_limit;
  int32_t limit[kAttnRows];
  float inv[kAttnRows];
  float top[2][2][kAttnRows];   // a tile's maxima over either half of its keys, two tiles in turn
  alignas(8) uint8_t valid[kValueStages][2][kLoadWarps];   // keys that exist, four bits a warp and half
};

__global__ void __launch_bounds__(kThreads, 1) attention_pair_kernel(AttnArgs a, AttnPlan p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ SharedPair sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem = smem_addr(smem_raw);
  const int rank = static_cast<int>(cluster_rank());

  // the item: the same keys for both CTAs
  const int pairs = (p.shared_groups + 1) / 2;
  int item = blockIdx.x >> 1;
  int pair0, row0, rows, slot, token = -1;   // first row of the pair's, of this CTA's rows
  int32_t k0, k1;
  if (item < pairs * p.shared_slots) {
    pair0 = item % pairs * 2 * kAttnRows;
    row0 = pair0 + rank * kAttnRows;
    rows = max(0, min(kAttnRows, a.T * a.H - row0));
    slot = item / pairs;
    k0 = slot * p.shared_chunk;
    k1 = min(k0 + p.shared_chunk, a.shared_len);
  } else {
    item -= pairs * p.shared_slots;
    token = item % a.T;
    slot = p.shared_slots + item / a.T;
    pair0 = token * a.H;
    row0 = pair0 + rank * kAttnRows;
    rows = max(0, min(kAttnRows, a.H - rank * kAttnRows));
    k0 = (p.shared_slots ? a.shared_len : 0) + (slot - p.shared_slots) * p.own_chunk;
    k1 = min(k0 + p.own_chunk, a.idx ? a.top_k : a.max_keys);
  }
  const LatentView& kv = token < 0 ? a.shared : a.kv;
  const bool rotated = a.kv.rope != nullptr;

  if (warp == kFirstWarp) {
    if (lane == 0) {
      for (int i = 0; i < kKeyStages; ++i) {
        mbar_init(&sh.keys[i], kLoadWarps * 32);
        mbar_init(&sh.peer_keys[i], 1);
      }
      for (int i = 0; i < kValueStages; ++i) {
        mbar_init(&sh.values[i], kLoadWarps * 32);
        mbar_init(&sh.peer_values[i], 1);
        mbar_init(&sh.used[i], 1);
        mbar_init(&sh.listed[i], kLoadWarps);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.scores[i], 1);
        mbar_init(&sh.taken[i], 2 * kSoftmaxWarps);
        mbar_init(&sh.weights[i], 2 * kSoftmaxWarps);
        mbar_init(&sh.drained[i], 1);
      }
      mbar_init(&sh.queries, 2 * kSoftmaxWarps);
      mbar_init(&sh.moved, kSoftmaxWarps);
      sh.abort = 0;
      sh.key_end = 0;
      sh.first_limit = 0x7FFFFFFF;
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc_pair(&sh.tmem, kTmemCols);
  }
  __syncthreads();
  cluster_arrive();                                      // either's barriers stand before the other arrives there
  cluster_wait();
  grid_dependency_wait();

  const int32_t* idx = a.idx ? a.idx + static_cast<int64_t>(token) * a.top_k : nullptr;
  const int32_t shared_seq = p.expand ? 0 : a.shared_seq;
  int32_t seq = shared_seq;
  if (token < 0) {
    if (tid < 2 * kAttnRows) {                           // both CTAs' rows: they stop at the same key
      int32_t n = 0;
      if (pair0 + tid < a.T * a.H) {
        const int32_t t = (pair0 + tid) / a.H;
        n = token_limit(a, t, token_seq(a, t));
      }
      if (tid / kAttnRows == rank) sh.limit[tid % kAttnRows] = n;
      atomicMax(&sh.key_end, min(n, k1));
      if (n > k0) atomicMin(&sh.first_limit, n);
    }
  } else {
    seq = token_seq(a, token);
    if (idx == nullptr) {
      const int32_t n = token_limit(a, token, seq);
      if (tid < kAttnRows) sh.limit[tid] = n;
      if (tid == 0) sh.key_end = min(n, k1);
    } else {
      if (tid < kAttnRows) sh.limit[tid] = 0x7FFFFFFF;
      int32_t last = 0;
      for (int32_t k = k0 + tid; k < k1; k += 8 * kThreads) {
        int32_t e[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) e[x] = k + x * kThreads < k1 ? __ldg(idx + k + x * kThreads) : -1;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (e[x] >= 0) last = k + x * kThreads + 1;
      }
      last = __reduce_max_sync(0xffffffffu, seq < 0 ? 0 : last);
      if (lane == 0 && last > 0) atomicMax(&sh.key_end, last);
    }
  }
  __syncthreads();
  const int32_t key_end = sh.key_end, first_limit = sh.first_limit;
  const int tiles = key_end > k0 ? (key_end - k0 + kAttnTile - 1) / kAttnTile : 0;
  tc_fence_after();

  if (warp >= kLoadWarp0) {
    // ---------------------------------------------------------------- loads
    const int lw = warp - kLoadWarp0;
    const int sub = lane >> 3, col = lane & 7;
    if (tiles > 0) {
#pragma unroll 1
      for (int r = lw * 8 + sub; r < lw * 8 + 8; r += 4) {   // the queries' share of shared memory, wanted with the first keys
        const int qr = row0 + (r < rows ? r : 0);
        const int t = rows > 0 ? qr / a.H : 0, h = rows > 0 ? qr - t * a.H : 0;
        const uint32_t dst = smem + r * 128 + ((col ^ (r & 7)) << 4);
        const __nv_bfloat16* ql = static_cast<const __nv_bfloat16*>(a.q_latent) + t * a.ql_t + h * a.ql_h + 384 + col * 8;
        cp_async16(dst, ql, r < rows);
        cp_async16(dst + kBlock, ql + 64, r < rows);
        if (rotated)
          cp_async16(dst + 2 * kBlock, static_cast<const __nv_bfloat16*>(a.q_rope) + t * a.qr_t + h * a.qr_h + col * 8, r < rows);
      }
    }
    // The warp's eight keys of a tile: four of this CTA's half (columns 0 .. 3) and four of the other's.
    const int key = (col < 4 ? rank : 1 - rank) * 32 + lw * 4 + (col & 3);
    int32_t pos2 = -1, pos1 = -1, page1 = -1, row = -1;
    auto advance = [&](int n) {
      row = pos1 < 0 ? -1 : page_row(kv, page1, pos1, a.err, token < 0 ? row0 / a.H : token);
      page1 = pos2 < 0 ? -1 : page_entry(kv, pos2 < a.shared_len ? shared_seq : seq, pos2);
      pos1 = pos2;
      const int32_t k = k0 + n * kAttnTile + key;
      pos2 = k < key_end ? (idx ? __ldg(idx + k) : k) : -1;
    };
    int ks = 0, vs = 0;
    uint32_t kphase = 1, vphase = 1;                     // the stages start free
    for (int n = 0; n < tiles + 2; ++n) {
      advance(n);                                        // the rows of tile n - 2
      if (n < 2) continue;
      const uint32_t valid = __ballot_sync(0xffffffffu, row >= 0);
      // keys: row lw * 4 + sub of this CTA's 32
      bool ok = mbar_wait_cluster(&sh.scores[ks], kphase, &sh.abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int32_t rk = __shfl_sync(0xffffffffu, row, sub);
      const __nv_bfloat16* sk = static_cast<const __nv_bfloat16*>(kv.latent) + static_cast<int64_t>(max(rk, 0)) * kLatentDim + col * 8;
      const int r32 = lw * 4 + sub;
      const uint32_t dk = smem + kPairK + ks * kPairKeys + r32 * 128 + ((col ^ (r32 & 7)) << 4);
#pragma unroll
      for (int c = 0; c < kLatentBlocks; ++c) cp_async16(dk + c * 4096, sk + c * 64, rk >= 0);
      if (rotated)
        cp_async16(dk + kLatentBlocks * 4096, static_cast<const __nv_bfloat16*>(kv.rope) + static_cast<int64_t>(max(rk, 0)) * kLatentRope + col * 8, rk >= 0);
      cp_async_arrive(&sh.keys[ks]);
      // values: the rows of the warp's eight keys, this CTA's half of the values
      ok = mbar_wait_cluster(&sh.used[vs], vphase, &sh.abort) && (n != kValueStages + 1 || mbar_wait<true>(&sh.moved, 0, &sh.abort));
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        sh.valid[vs][rank][lw] = valid & 15;
        sh.valid[vs][1 - rank][lw] = (valid >> 4) & 15;
        mbar_arrive(&sh.listed[vs]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int32_t rv = __shfl_sync(0xffffffffu, row, sub + 4 * j);
        const int r64 = (j == 0 ? rank : 1 - rank) * 32 + lw * 4 + sub;
        const __nv_bfloat16* sv = static_cast<const __nv_bfloat16*>(kv.latent) + static_cast<int64_t>(max(rv, 0)) * kLatentDim + rank * 256 + col * 8;
        const uint32_t dv = smem + kPairV + vs * kPairValues + r64 * 128 + ((col ^ (r64 & 7)) << 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) cp_async16(dv + c * kBlock, sv + c * 64, rv >= 0);
      }
      cp_async_arrive(&sh.values[vs]);
      if (++ks == kKeyStages) {
        ks = 0;
        kphase ^= 1;
      }
      if (++vs == kValueStages) {
        vs = 0;
        vphase ^= 1;
      }
    }
    cp_async_wait_all();
  } else if (warp == kFirstWarp) {
    if (elect_one()) {
      bool ok = true;
      if (rank == 0) {
        // ---------------------------------------------------------------- scores = Q K^T
        constexpr uint32_t idesc = make_idesc(1, 2 * kAttnRows, kAttnTile);
        ok = tiles == 0 || mbar_wait_cluster(&sh.queries, 0, &sh.abort);
        for (int i = 0; i < tiles && ok; ++i) {
          const int st = i & 1;
          const uint32_t phase = (i >> 1) & 1;
          if (i >= 2) ok = mbar_wait_cluster(&sh.taken[st], phase ^ 1, &sh.abort);
          ok = ok && mbar_wait<true>(&sh.keys[st], phase, &sh.abort) && mbar_wait_cluster(&sh.peer_keys[st], phase, &sh.abort);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t keys = smem + kPairK + st * kPairKeys;
          const uint32_t d = kPairTmemS + st * 32;
#pragma unroll
          for (int ks = 0; ks < 24; ++ks)
            umma_pair_f16_ts(d, kPairTmemQ + ks * 8, sdesc_kmajor_sw128(keys + (ks >> 2) * 4096 + (ks & 3) * 32), idesc, ks > 0);
#pragma unroll
          for (int ks = 24; ks < 32; ++ks)
            umma_pair_f16(d, sdesc_kmajor_sw128(smem + ((ks - 24) >> 2) * kBlock + (ks & 3) * 32),
                          sdesc_kmajor_sw128(keys + (ks >> 2) * 4096 + (ks & 3) * 32), idesc, 1);
          if (rotated) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_pair_f16(d, sdesc_kmajor_sw128(smem + 2 * kBlock + ks * 32),
                            sdesc_kmajor_sw128(keys + kLatentBlocks * 4096 + ks * 32), idesc, 1);
          }
          umma_pair_commit(&sh.scores[st]);
        }
        umma_pair_commit(&sh.drained[0]);
      } else {
        for (int i = 0; i < tiles && ok; ++i) {
          ok = mbar_wait<true>(&sh.keys[i & 1], (i >> 1) & 1, &sh.abort);
          if (!ok) break;
          fence_proxy_async_smem();                      // the copies that the barrier reported
          mbar_arrive_cluster(&sh.peer_keys[i & 1], 0);
        }
      }
      int alone = 0;
      mbar_wait_cluster(&sh.drained[0], 0, &alone);
    }
    __syncwarp();
  } else if (warp == kSecondWarp) {
    if (elect_one()) {
      bool ok = true;
      int st = 0;
      uint32_t phase = 0;
      if (rank == 0) {
        // ---------------------------------------------------------------- output += P V
        constexpr uint32_t idesc = make_idesc(1, 2 * kAttnRows, 256) | kIdescBMnMajor;
        for (int i = 0; i < tiles; ++i) {
          ok = mbar_wait<true>(&sh.values[st], phase, &sh.abort) && mbar_wait_cluster(&sh.peer_values[st], phase, &sh.abort) &&
               mbar_wait_cluster(&sh.weights[i & 1], (i >> 1) & 1, &sh.abort);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t values = smem + kPairV + st * kPairValues, w = smem + kPairP + (i & 1) * kBlock;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int ks = 0; ks < kAttnTile / 16; ++ks)
              umma_pair_f16(kTmemO + j * 128, sdesc_kmajor_sw128(w + ks * 32),
                            sdesc_mnmajor_sw128(values + j * 2 * kBlock + ks * 2048, kBlock), idesc, i > 0 || ks > 0);
          umma_pair_commit(&sh.used[st]);
          if (++st == kValueStages) {
            st = 0;
            phase ^= 1;
          }
        }
        umma_pair_commit(&sh.drained[1]);
      } else {
        for (int i = 0; i < tiles; ++i) {
          ok = mbar_wait<true>(&sh.values[st], phase, &sh.abort);
          if (!ok) break;
          fence_proxy_async_smem();
          mbar_arrive_cluster(&sh.peer_values[st], 0);
          if (++st == kValueStages) {
            st = 0;
            phase ^= 1;
          }
        }
      }
      int alone = 0;
      mbar_wait_cluster(&sh.drained[1], 0, &alone);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- weights
    // A thread's row and half of the tile's keys; the warp two further on has the rows' other half.
    const int r = tid & 63, half = tid >> 6;
    const int32_t limit = sh.limit[r];
    const uint32_t quadrant = static_cast<uint32_t>(warp * 32) << 16;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (tiles > 0) {
      // the queries' values 0 .. 383 pass through the weights' place and the last stage of values: read there by lines,
      // they are read back by rows
      auto block = [&](int c) { return smem + (c < 2 ? kPairP + c * kBlock : kPairV + kPairValues * (kValueStages - 1) + (c - 2) * kBlock); };
      const int col = lane & 7;
#pragma unroll 1
      for (int y = warp * 16 + (lane >> 3); y < warp * 16 + 16; y += 4) {
        const int qr = row0 + (y < rows ? y : 0);
        const int t = rows > 0 ? qr / a.H : 0, h = rows > 0 ? qr - t * a.H : 0;
        const __nv_bfloat16* ql = static_cast<const __nv_bfloat16*>(a.q_latent) + t * a.ql_t + h * a.ql_h + col * 8;
#pragma unroll
        for (int c = 0; c < 6; ++c) cp_async16(block(c) + y * 128 + ((col ^ (y & 7)) << 4), ql + c * 64, y < rows);
      }
      cp_async_wait_all();
      named_barrier(3, kSoftmaxWarps * 32);
#pragma unroll
      for (int c = 0; c < 6; ++c) {
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 x = ld_shared16(block(c) + r * 128 + ((e ^ (r & 7)) << 4));
          v[4 * e] = x.x; v[4 * e + 1] = x.y; v[4 * e + 2] = x.z; v[4 * e + 3] = x.w;
        }
        tmem_st_32x32b_x32(quadrant + kPairTmemQ + 32 * c, v);
      }
      tmem_st_wait();
      tc_fence_before();
      fence_proxy_async_smem();
      named_barrier(3, kSoftmaxWarps * 32);                // the weights may take their place
      if (lane == 0) {
        mbar_arrive(&sh.moved);
        mbar_arrive_cluster(&sh.queries, 0);
      }
    }
    int st = 0;
    uint32_t phase = 0;
    for (int i = 0; i < tiles; ++i) {
      const int b = i & 1;
      ok = ok && mbar_wait_cluster(&sh.scores[b], (i >> 1) & 1, &sh.abort) && mbar_wait<true>(&sh.listed[st], phase, &sh.abort);
      // the weights' place: the second product of the tile before last
      if (ok && i >= 2) ok = mbar_wait_cluster(&sh.used[(i - 2) % kValueStages], ((i - 2) / kValueStages) & 1, &sh.abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {                                         // the partner may be waiting: the barrier of every tile is kept
        named_barrier(1 + (warp & 1), 64);
        continue;
      }
      tc_fence_after();
      uint32_t raw[32];
      tmem_ld_32x32b_x32(quadrant + kPairTmemS + b * 32, raw);
      uint64_t present = *reinterpret_cast<const uint64_t*>(sh.valid[st][half]);
      present = (present | present >> 4) & 0x00FF00FF00FF00FFull;         // four bits of every byte, together
      present = (present | present >> 8) & 0x0000FFFF0000FFFFull;
      uint32_t mine = static_cast<uint32_t>(present | present >> 16);
      const int32_t n = limit - (k0 + i * kAttnTile + half * 32);          // the row's keys of this half
      if (n < 32) mine = n <= 0 ? 0u : mine & ((1u << n) - 1);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(&sh.taken[b], 0);
      float x[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(raw[e]);
      if (!__all_sync(0xffffffffu, mine == 0xFFFFFFFFu)) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!((mine >> e) & 1)) x[e] = -INFINITY;
      }
      float mx = x[0];
#pragma unroll
      for (int e = 1; e < 32; ++e) mx = fmaxf(mx, x[e]);
      sh.top[b][half][r] = mx;
      named_barrier(1 + (warp & 1), 64);
      mx = fmaxf(mx, sh.top[b][1 - half][r]) * a.scale_log2;
      // both warps of a row see the same numbers and decide alike
      const bool rescale = __any_sync(0xffffffffu, mx > m + kLag);
      float factor = 1.f;
      if (rescale) {
        const float mn = fmaxf(m, mx);
        factor = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
        l *= factor;
        m = mn;
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const uint32_t place = smem + kPairP + b * kBlock + r * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = exp2_fast(fmaf(x[8 * c + 2 * e], a.scale_log2, -ref)), hi = exp2_fast(fmaf(x[8 * c + 2 * e + 1], a.scale_log2, -ref));
          l += lo + hi;                                  // the sum keeps fp32; the product's operand is bf16
          w[e] = bf16x2(lo, hi);
        }
        st_shared16(place + (((half * 4 + c) ^ (r & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
      }
      if (rescale && i > 0) {
        ok = mbar_wait_cluster(&sh.used[(i - 1) % kValueStages], ((i - 1) / kValueStages) & 1, &sh.abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(quadrant + kTmemO + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
          tmem_st_32x32b_x32(quadrant + kTmemO + c, o);
        }
        tmem_st_wait();
      }
      if (first_limit < min(k0 + (i + 1) * kAttnTile, key_end)) {   // a row of either CTA that ended before the tile's last key
        ok = mbar_wait<true>(&sh.values[st], phase, &sh.abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        keep_finite(smem + kPairV + st * kPairValues, kPairValues, tid);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(&sh.weights[b], 0);
      if (++st == kValueStages) {
        st = 0;
        phase ^= 1;
      }
    }
    // the two halves' sums
    named_barrier(1 + (warp & 1), 64);                   // the last maxima have been read
    sh.top[0][half][r] = l;
    named_barrier(1 + (warp & 1), 64);
    l += sh.top[0][1 - half][r];
    if (half == 0 && ok) {
      sh.inv[r] = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
      if (r < rows) {
        if (p.parts()) a.part_lse[static_cast<int64_t>(slot) * a.T * a.H + row0 + r] = lse2;
        else if (a.lse) a.lse[row0 + r] = lse2 * kLn2;
      }
    }
  }

  // ---------------------------------------------------------------- the result
  launch_dependents();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();                                      // both CTAs' copies and products are done
  cluster_wait();
  tc_fence_after();
  const bool wide = p.parts();
  if (*const_cast<volatile int*>(&sh.abort) != 0) {
    if (tid == 0) record_error(a.err, DSA_DEVERR_TIMEOUT, static_cast<int>(blockIdx.x));
  } else if (tiles > 0 || !wide) {
    const uint32_t stride = wide ? kOutRow32 : kOutRow16;
    if (warp < 12) {
      const int r = (warp & 1) * 32 + lane, half = (warp >> 1) & 1;
      const float inv = sh.inv[r];
      const uint32_t mem = smem + kPairK + r * stride + half * (wide ? 1024 : 512);
#pragma unroll 1
      for (int c = (warp >> 2) * 16; c < 256; c += 48) {
        uint32_t o[16];
        tmem_ld_32x32b_x16((static_cast<uint32_t>((warp & 3) * 32) << 16) + kTmemO + c, o);
        tmem_ld_wait();
        float val[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) val[e] = inv == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
        if (wide) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            st_shared16(mem + (c + e) * 4, make_uint4(__float_as_uint(val[e]), __float_as_uint(val[e + 1]),
                                                      __float_as_uint(val[e + 2]), __float_as_uint(val[e + 3])));
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            st_shared16(mem + (c + e) * 2, make_uint4(bf16x2(val[e], val[e + 1]), bf16x2(val[e + 2], val[e + 3]),
                                                      bf16x2(val[e + 4], val[e + 5]), bf16x2(val[e + 6], val[e + 7])));
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    const int shift = wide ? 7 : 6;
    uint4* out = wide ? reinterpret_cast<uint4*>(a.part_o) + ((static_cast<int64_t>(slot) * a.T * a.H + row0) << shift)
                      : static_cast<uint4*>(a.out) + (static_cast<int64_t>(row0) << shift);
#pragma unroll 2
    for (int v = tid; v < rows << shift; v += kThreads)
      out[v] = ld_shared16(smem + kPairK + (v >> shift) * stride + (v & ((1 << shift) - 1)) * 16);
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();                                      // the pair gives its tensor memory back together
  cluster_wait();
  if (warp == kFirstWarp) {
    tc_fence_after();
    tmem_dealloc_pair(sh.tmem, kTmemCols);
  }
}

// The shared prefix of an FP8 cache in bf16, one row per position, for the many groups of rows that read it: map[p] is p,
// or -1 where the page table has no page.  One warp per position.
__global__ void __launch_bounds__(256) expand_kernel(LatentView kv, int32_t seq, int32_t n, __nv_bfloat16* latent,
                                                     __nv_bfloat16* rope, int32_t* map) {
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x & 31;
  const int32_t p = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (p >= n) return;
  const int32_t row = page_row(kv, page_entry(kv, seq, p), p, nullptr, 0);
  if (lane == 0) map[p] = row < 0 ? -1 : p;
  if (row < 0) return;
  const float s = __ldg(kv.scale + row);
  const uint4 c = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv.latent) + static_cast<int64_t>(row) * kLatentDim) + lane);
  uint4* out = reinterpret_cast<uint4*>(latent + static_cast<int64_t>(p) * kLatentDim) + 2 * lane;
  out[0] = make_uint4(e4m3x2_to_bf16x2(c.x & 0xFFFFu, s), e4m3x2_to_bf16x2(c.x >> 16, s), e4m3x2_to_bf16x2(c.y & 0xFFFFu, s),
                      e4m3x2_to_bf16x2(c.y >> 16, s));
  out[1] = make_uint4(e4m3x2_to_bf16x2(c.z & 0xFFFFu, s), e4m3x2_to_bf16x2(c.z >> 16, s), e4m3x2_to_bf16x2(c.w & 0xFFFFu, s),
                      e4m3x2_to_bf16x2(c.w >> 16, s));
  if (kv.rope && lane < 8)
    reinterpret_cast<uint4*>(rope + static_cast<int64_t>(p) * kLatentRope)[lane] =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(kv.rope) + static_cast<int64_t>(row) * kLatentRope) + lane);
}

// Joins the parts of one row: weights 2^(lse_i - max) over their sum, made by a lane per part; then 128 threads add up
// four values each, eight parts' loads at a time.  Bound by the latency of those loads: rows of many parts get two or
// four such groups of threads (128 rows of 74 parts took 14 us with one).  Blocks of four find no room beside the first
// kernel's, those of two do: attention of 384 rows in 11 parts 17.9 us with four and 16.4 with two, of 256 rows in 16
// parts, few enough blocks, 13.8 and 14.6; of 512 rows in 16 parts 24.6 with one and 22.9 with two.
template <int GROUPS>
__global__ void __launch_bounds__(GROUPS * 128) attention_join_kernel(AttnArgs a, int slots) {
  __shared__ float weight[kMaxSlots];
  __shared__ float part[4 * GROUPS];
  __shared__ float4 sums[GROUPS][128];
  grid_dependency_wait();
  launch_dependents();
  const int64_t r = blockIdx.x, R = static_cast<int64_t>(a.T) * a.H;
  const int tid = threadIdx.x, c = tid & 127, group = tid >> 7;
  float top = -INFINITY;
  for (int s = tid; s < slots; s += GROUPS * 128) top = fmaxf(top, weight[s] = a.part_lse[s * R + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) part[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4 * GROUPS; ++i) top = fmaxf(top, part[i]);
  const float ref = top == -INFINITY ? 0.f : top;
  const float4* v = reinterpret_cast<const float4*>(a.part_o + r * kLatentDim) + c;
  float total = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = group * 8; s0 < slots; s0 += GROUPS * 8) {
    float4 x[8];
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {                        // 0 past the last part, and where nothing was written
      w[e] = s0 + e < slots ? exp2f(weight[s0 + e] - ref) : 0.f;
      x[e] = w[e] != 0.f ? v[(s0 + e) * R * (kLatentDim / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      total += w[e];
      o.x += w[e] * x[e].x; o.y += w[e] * x[e].y; o.z += w[e] * x[e].z; o.w += w[e] * x[e].w;
    }
  }
  if constexpr (GROUPS > 1) {
    __syncthreads();                                     // every weight has been read
    sums[group][c] = o;
    if (c == 0) weight[group] = total;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) {
      const float4 x = sums[g][c];
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
      total += weight[g];
    }
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + r * kLatentDim + c * 4) =
      make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
  if (a.lse && c == 0) a.lse[r] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
}

}  // namespace

// Sets a kernel up for a launch on the current device, once for each device: the attributes stay with its context.
cudaError_t set_up(bool fp8) {
  static std::atomic<uint64_t> ready[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (e != cudaSuccess || (ready[fp8].load(std::memory_order_relaxed) & bit)) return e;
  auto kernel = fp8 ? attention_kernel<true> : attention_kernel<false>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(attention_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e == cudaSuccess) ready[fp8].fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// CTAs that run at once in clusters of a size (2, 4, 8, 16): a cluster's SMs belong to one GPC, so that is fewer than
// there are SMs; 0 where not even one fits.  Without a device (a workspace query on a host that has none): an estimate.
// Where the device does not answer: 0, and *answered false.
int cluster_room(int cluster, int sms, bool* answered) {
  static std::atomic<int> known[64][5];                  // room + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return sms / 18 * 16;
  const int i = __builtin_ctz(cluster);
  int room = known[dev][i].load(std::memory_order_relaxed) - 1;
  if (room < 0) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (set_up(false) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, attention_kernel<false>, &cfg) != cudaSuccess) {
      cudaGetLastError();                                // asked again next time; clusters stay unused until it answers
      *answered = false;
      return 0;
    }
    room = n * cluster;
    known[dev][i].store(room + 1, std::memory_order_relaxed);
  }
  return room;
}

namespace {

size_t part_bytes(const AttnPlan& p, int64_t T, int32_t H) {
  const size_t b = p.parts() ? size_t(p.slots()) * T * H * (kLatentDim + 1) * sizeof(float) : 0;
  return (b + 255) / 256 * 256;
}

}  // namespace

size_t attention_workspace(const AttnPlan& p, int64_t T, int32_t H, int64_t shared_keys) {
  return part_bytes(p, T, H) + (p.expand ? size_t(shared_keys) * (2 * (kLatentDim + kLatentRope) + 4) : 0);
}

cudaError_t launch_attention(const AttnArgs& args, const AttnPlan& p, int* launched, cudaStream_t stream) {
  AttnArgs a = args;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  a.shared = a.kv;
  if (p.expand) {
    __nv_bfloat16* latent = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(a.workspace) + part_bytes(p, a.T, a.H));
    __nv_bfloat16* rope = latent + int64_t(a.shared_len) * kLatentDim;
    int32_t* map = reinterpret_cast<int32_t*>(rope + int64_t(a.shared_len) * kLatentRope);
    cfg.gridDim = dim3(static_cast<unsigned>((a.shared_len + 7) / 8));
    cfg.blockDim = dim3(256);
    cudaError_t e = cudaLaunchKernelEx(&cfg, expand_kernel, a.kv, a.shared_seq, a.shared_len, latent, rope, map);
    if (e != cudaSuccess) return e;
    ++*launched;
    // a cache of one-row pages whose only sequence is the prefix
    a.shared = LatentView{latent, nullptr, a.kv.rope ? rope : nullptr, a.shared_len, 1, 0, 0, map, 1, a.shared_len};
  }
  a.part_o = static_cast<float*>(a.workspace);
  a.part_lse = a.part_o ? a.part_o + size_t(p.slots()) * a.T * a.H * kLatentDim : nullptr;
  cudaError_t e = set_up(a.kv.fp8);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kThreads);
  const int64_t shared_items = int64_t(p.shared_groups) * p.shared_slots, own_items = int64_t(a.T) * p.own_groups * p.own_slots;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.pair ? 2 : p.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  if (p.pair) {
    const int64_t items = int64_t(p.shared_groups + 1) / 2 * p.shared_slots + (a.kv.fp8 ? 0 : int64_t(a.T) * p.own_slots);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * items));
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, attention_pair_kernel, a, p);
    if (e != cudaSuccess) return e;
    ++*launched;
    a.first_item = static_cast<int32_t>(shared_items);   // what is left to the single kernel: an FP8 cache's own items
  }
  if (!p.pair || (a.kv.fp8 && own_items > 0)) {
    cfg.gridDim = dim3(static_cast<unsigned>(shared_items + own_items - a.first_item));
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, a.kv.fp8 ? attention_kernel<true> : attention_kernel<false>, a, p);
    if (e != cudaSuccess) return e;
    ++*launched;
  }
  if (p.parts()) {
    const int64_t R = int64_t(a.T) * a.H;
    cfg.gridDim = dim3(static_cast<unsigned>(R));
    const int join = p.slots() > (R <= 256 ? 8 : 32) ? 4 : p.slots() > 8 ? 2 : 1;      // groups of threads
    cfg.blockDim = dim3(128 * join);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join == 4 ? attention_join_kernel<4> : join == 2 ? attention_join_kernel<2> : attention_join_kernel<1>, a,
                           static_cast<int>(p.slots()));
    if (e != cudaSuccess) return e;
    ++*launched;
  }
  return cudaSuccess;
}

}  // namespace dsa
