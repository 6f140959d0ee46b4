// update_key_bounds: per (physical block, KV head), the channel-wise largest
// and smallest key over the block's valid slots,
//   bounds[b][h][0][d] = max_t K[b][h][t][d],  bounds[b][h][1][d] = min_t ...,
// for the blocks of each sequence that hold one of its newest tokens. A block
// is recomputed whole from the pool, so the result does not depend on what the
// bounds held before (a reused block, a copy-on-write copy).
//
// Bound by HBM (a block's keys are read once, 2/block_size of that is
// written). A warp takes heads_per_warp neighbouring heads of one block, whose
// tiles are one contiguous run, so the chain of length, table entry and keys is
// paid once per run; a tile is read with 16 bytes per lane and 4 loads in flight,
// so that enough warps fit an SM. 32 contexts of 16,384 to 32,768 tokens x 8 heads
// (1.8 GB): 266 us, 6.8 TB/s; one head per warp 340, loads that bypass L1 284, 8 in
// flight 267 (and 7.1 instead of 6.0 us for one block of 256 x 40 heads).
#pragma once

#include "common.cuh"

namespace kvp {
namespace dev {

struct BoundsArgs {
  const void* k_cache;
  void* bounds;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* new_tokens;  // NULL: every token is new
  int32_t num_seqs, num_kv_heads, num_blocks, max_blocks_per_seq;
  int32_t max_context_len, max_new_tokens;
  int32_t blocks_per_seq;  // most touched blocks of one sequence
  int32_t heads_per_warp, head_groups;  // head_groups = ceil(heads / heads_per_warp)
  int32_t log2_bs;
};

constexpr int kBoundsWarps = 8;

// NaN in a valid slot makes the channel's bounds NaN.
template <typename T>
struct MinMax2;
template <>
struct MinMax2<__half> {
  static __device__ __forceinline__ uint32_t max(uint32_t x, uint32_t y) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ uint32_t min(uint32_t x, uint32_t y) {
    const __half2 r = __hmin2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static constexpr uint32_t kInf2 = 0x7c007c00u;
};
template <>
struct MinMax2<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t max(uint32_t x, uint32_t y) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&x),
                                         *reinterpret_cast<__nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ uint32_t min(uint32_t x, uint32_t y) {
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&x),
                                         *reinterpret_cast<__nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static constexpr uint32_t kInf2 = 0x7f807f80u;
};

// T: the bounds' type (the cache's, or fp16 over E4M3 codes, whose values it
// holds exactly); a row of D channels is read by LPR lanes of 16 bytes.
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32) key_bounds_kernel(const BoundsArgs a) {
  constexpr int LPR = D * (FP8 ? 1 : 2) / 16;  // lanes per row
  constexpr int RPL = 32 / LPR;                // rows per load
  constexpr int W = FP8 ? 8 : 4;               // packed words a lane keeps
  const uint32_t warp = blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t per_seq = uint32_t(a.blocks_per_seq) * a.head_groups;
  const uint32_t s = warp / per_seq;
  if (s >= uint32_t(a.num_seqs)) return;
  const uint32_t rest = warp - s * per_seq;
  const int i = rest / a.head_groups;
  const int g0 = (rest - i * a.head_groups) * a.heads_per_warp;
  const int bs = 1 << a.log2_bs;

  int ctx = __ldg(a.context_lens + s);
  if (ctx < 0 || ctx > a.max_context_len) {
    if (rest == 0 && lane == 0) record_error(KVP_DEVERR_CTX, s);
    ctx = ctx < 0 ? 0 : a.max_context_len;
  }
  int fresh = a.new_tokens ? __ldg(a.new_tokens + s) : ctx;
  if (fresh < 0 || fresh > a.max_new_tokens) {
    if (rest == 0 && lane == 0) record_error(KVP_DEVERR_CTX, s);
    fresh = fresh < 0 ? 0 : a.max_new_tokens;
  }
  if (fresh == 0) return;
  const int first = fresh < ctx ? (ctx - fresh) >> a.log2_bs : 0;
  const int lb = first + i;
  if (int64_t(lb) * bs >= ctx) return;
  const int32_t b = __ldg(a.block_tables + int64_t(s) * a.max_blocks_per_seq + lb);
  if (b < 0 || b >= a.num_blocks) {
    if (g0 == 0 && lane == 0) record_error(KVP_DEVERR_BLOCK_ID, (uint64_t(s) << 32) | uint32_t(lb));
    return;
  }
  const int rows = min(bs, ctx - lb * bs);

  const int g1 = min(a.num_kv_heads, g0 + a.heads_per_warp);
  for (int g = g0; g < g1; ++g) {
    const int64_t head = int64_t(b) * a.num_kv_heads + g;
    const uint4* tile = static_cast<const uint4*>(a.k_cache) + (head << a.log2_bs) * LPR + lane % LPR;
    uint32_t hi[W], lo[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      hi[w] = MinMax2<T>::kInf2 | 0x80008000u;
      lo[w] = MinMax2<T>::kInf2;
    }
    constexpr int U = 4;  // loads in flight per lane
    for (int r0 = lane / LPR; r0 < rows; r0 += U * RPL) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r0 + u * RPL < rows) x[u] = __ldg(tile + (r0 + u * RPL) * LPR);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + u * RPL >= rows) continue;
        const uint32_t p[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t e;
          if constexpr (FP8) e = e4m3x2_to_x2<__half>((p[w / 2] >> (16 * (w & 1))) & 0xffffu);
          else e = p[w];
          hi[w] = MinMax2<T>::max(hi[w], e);
          lo[w] = MinMax2<T>::min(lo[w], e);
        }
      }
    }
#pragma unroll
    for (int m = LPR; m < 32; m <<= 1) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        hi[w] = MinMax2<T>::max(hi[w], __shfl_xor_sync(0xffffffffu, hi[w], m));
        lo[w] = MinMax2<T>::min(lo[w], __shfl_xor_sync(0xffffffffu, lo[w], m));
      }
    }
    // lanes of row group 0 write the largest, those of group 1 the smallest
    if (lane < 2 * LPR) {
      const bool low = lane >= LPR;
      uint4* dst = static_cast<uint4*>(a.bounds) + (head * 2 + (low ? 1 : 0)) * (D / 8) +
                   (lane % LPR) * (W / 4);
#pragma unroll
      for (int w = 0; w < W; w += 4)
        dst[w / 4] = low ? make_uint4(lo[w], lo[w + 1], lo[w + 2], lo[w + 3])
                         : make_uint4(hi[w], hi[w + 1], hi[w + 2], hi[w + 3]);
    }
  }
}

}  // namespace dev
}  // namespace kvp
