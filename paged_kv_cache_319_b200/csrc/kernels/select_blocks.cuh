// select_blocks: for every (sequence, KV head), the blocks of its context that
// the group's new queries need most, by an upper bound on their logits.
//
// With M, m the block's channel-wise largest and smallest key,
//   score(b) = sum_d Q+[d] M[d] + Q-[d] m[d],
//   Q+ = sum_g max(q[g], 0),  Q- = sum_g min(q[g], 0),
// which is sum_g sum_d max(q[g][d] M[d], q[g][d] m[d]) and so no smaller than
// the sum over the group of any of the block's logits. A score costs 2 D
// multiply-adds whatever the group's size. Sums are fp64: 16-bit products are exact there and
// so, for all practical data, are the sums, which makes the choice independent
// of the summation order.
//
// One cluster of up to 8 CTAs serves a (sequence, KV head). Each CTA scores a
// contiguous range of blocks (a warp reads a block's 4 D bytes of bounds at 16
// bytes per lane) and keeps the scores as order-preserving 64-bit keys in
// shared memory. The threshold is found by zooming: a 1024-bin histogram of
// the active key range, merged over the cluster through distributed shared
// memory, names the bin that holds the last kept key; that bin is the next
// range. Then the CTAs write their kept blocks in ascending order at offsets
// from a prefix sum over warps and CTAs.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace kvp {
namespace dev {

struct SelectArgs {
  const void* q;
  const void* bounds;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t* out;
  int32_t num_seqs, num_q_heads, num_kv_heads, num_blocks, max_blocks_per_seq;
  int32_t max_context_len;
  int32_t log2_bs;
  int32_t keep, sink, recent;
};

constexpr int kSelWarps = 16;
constexpr int kSelThreads = kSelWarps * 32;
constexpr int kSelBins = 1024;
constexpr int kSelLog2Bins = 10;

// Order-preserving map of fp64 to uint64; NaN above everything, -0 equal to 0.
__device__ __forceinline__ uint64_t score_key(double x) {
  if (x != x) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// TQ: the queries' type, TB: the bounds' type.
template <typename TQ, typename TB, int D>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectArgs a) {
  namespace cg = cooperative_groups;
  constexpr int LPB = D / 4;      // lanes per block: 2 D elements, 8 per lane
  constexpr int BPL = 32 / LPB;   // blocks per warp load
  constexpr int U = 8 / BPL;      // loads in flight: 8 blocks per warp step
  extern __shared__ uint64_t keys[];
  __shared__ uint32_t hist[2][kSelBins];
  __shared__ uint64_t range_lo[kSelWarps], range_hi[kSelWarps];
  __shared__ uint64_t cta_lo, cta_hi;
  __shared__ uint32_t warp_sum[kSelWarps];
  __shared__ uint32_t found[3];  // bin, keys above it, keys in it
  __shared__ uint32_t take[2][kSelWarps + 1];  // kept / tied keys per warp, and of the CTA

  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t nranks = cluster.num_blocks(), rank = cluster.block_rank();
  const uint32_t unit = blockIdx.x / nranks;
  const uint32_t s = unit / a.num_kv_heads, g = unit - s * a.num_kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int ctx = __ldg(a.context_lens + s);
  if (ctx < 0 || ctx > a.max_context_len) {
    if (g == 0 && rank == 0 && tid == 0) record_error(KVP_DEVERR_CTX, s);
    ctx = ctx < 0 ? 0 : a.max_context_len;
  }
  const int n = (ctx + (1 << a.log2_bs) - 1) >> a.log2_bs;
  int32_t* out = a.out + int64_t(unit) * a.keep;
  if (n <= a.keep) {  // every block is kept (uniform over the cluster)
    if (rank == 0)
      for (int i = tid; i < a.keep; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  // n > keep >= sink + recent: candidates [sink, n - recent)
  const int cand = n - a.sink - a.recent;
  uint32_t need = a.keep - a.sink - a.recent;
  if (rank == 0) {
    for (int i = tid; i < a.sink; i += kSelThreads) out[i] = i;
    for (int i = tid; i < a.recent; i += kSelThreads) out[a.keep - a.recent + i] = n - a.recent + i;
  }
  if (need == 0) return;
  const int per = (cand + nranks - 1) / nranks;
  const int first = min(cand, int(rank) * per), count = min(cand, first + per) - first;

  // ---- scores -----------------------------------------------------------------
  const int G = a.num_q_heads / a.num_kv_heads;
  const int sub = lane % LPB;           // lane within its block
  const bool low = sub >= LPB / 2;      // the smallest keys' half
  double w[8];
  {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0.0;
    const uint4* q = static_cast<const uint4*>(a.q) +
                     (int64_t(s) * a.num_q_heads + int64_t(g) * G) * (D / 8) + sub % (LPB / 2);
    for (int h = 0; h < G; ++h) {
      const uint4 x = __ldg(q + h * (D / 8));
      const uint32_t p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Elem<TQ>::to_float2(p[e]);
        // comparisons that keep a NaN query
        w[2 * e] += double(low ? (f.x > 0.f ? 0.f : f.x) : (f.x < 0.f ? 0.f : f.x));
        w[2 * e + 1] += double(low ? (f.y > 0.f ? 0.f : f.y) : (f.y < 0.f ? 0.f : f.y));
      }
    }
  }
  const int32_t* table = a.block_tables + int64_t(s) * a.max_blocks_per_seq + a.sink + first;
  uint64_t my_lo = ~0ull, my_hi = 0;
  for (int c0 = warp * 8; c0 < count; c0 += kSelWarps * 8) {
    int32_t id = -1;
    if (lane < 8 && c0 + lane < count) {
      id = __ldg(table + c0 + lane);
      if (id < 0 || id >= a.num_blocks) {
        if (g == 0)
          record_error(KVP_DEVERR_BLOCK_ID,
                       (uint64_t(s) << 32) | uint32_t(a.sink + first + c0 + lane));
        id = -1;
      }
    }
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t b = __shfl_sync(0xffffffffu, id, u * BPL + lane / LPB);
      x[u] = make_uint4(0, 0, 0, 0);
      if (b >= 0)
        x[u] = __ldg(static_cast<const uint4*>(a.bounds) +
                     (int64_t(b) * a.num_kv_heads + g) * LPB + sub);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t p[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      double sum = 0.0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Elem<TB>::to_float2(p[e]);
        sum = fma(w[2 * e], double(f.x), sum);
        sum = fma(w[2 * e + 1], double(f.y), sum);
      }
#pragma unroll
      for (int m = 1; m < LPB; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      const int c = c0 + u * BPL + lane / LPB;
      const int32_t b = __shfl_sync(0xffffffffu, id, u * BPL + lane / LPB);
      if (sub == 0 && c < count) {
        const uint64_t key = b >= 0 ? score_key(sum) : 0ull;
        keys[c] = key;
        my_lo = min(my_lo, key);
        my_hi = max(my_hi, key);
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    my_lo = min(my_lo, __shfl_xor_sync(0xffffffffu, my_lo, m));
    my_hi = max(my_hi, __shfl_xor_sync(0xffffffffu, my_hi, m));
  }
  if (lane == 0) range_lo[warp] = my_lo, range_hi[warp] = my_hi;
  for (int i = tid; i < kSelBins; i += kSelThreads) hist[0][i] = 0;
  __syncthreads();
  if (tid == 0) {
    uint64_t l = ~0ull, h = 0;
    for (int i = 0; i < kSelWarps; ++i) l = min(l, range_lo[i]), h = max(h, range_hi[i]);
    cta_lo = l, cta_hi = h;
  }
  cluster.sync();
  uint64_t lo = ~0ull, hi = 0;  // the active keys lie in [lo, hi]
  for (uint32_t r = 0; r < nranks; ++r) {
    lo = min(lo, *cluster.map_shared_rank(&cta_lo, r));
    hi = max(hi, *cluster.map_shared_rank(&cta_hi, r));
  }

  // ---- threshold: keys above `hi` are kept, and the first `need` of those in
  // [lo, hi], which are all of them or all equal. `found` is written again only
  // after the next cluster.sync.
  int phase = 0;
  while (lo < hi) {
    const uint64_t span = hi - lo;
    const int bits = 64 - __clzll(static_cast<long long>(span));
    const int shift = bits > kSelLog2Bins ? bits - kSelLog2Bins : 0;
    uint32_t* mine = hist[phase];
    for (int i = tid; i < count; i += kSelThreads) {
      const uint64_t k = keys[i];
      if (k >= lo && k <= hi) atomicAdd(&mine[uint32_t((k - lo) >> shift)], 1u);
    }
    cluster.sync();
    // each thread: two neighbouring bins of the merged histogram, highest first
    constexpr int PER = kSelBins / kSelThreads;
    uint32_t bin[PER], total = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      bin[j] = 0;
      const int b = kSelBins - 1 - (tid * PER + j);
      for (uint32_t r = 0; r < nranks; ++r) bin[j] += cluster.map_shared_rank(mine, r)[b];
      total += bin[j];
    }
    uint32_t incl = total;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    // the other buffer was last read before this iteration's cluster.sync
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[phase ^ 1][i] = 0;
    __syncthreads();
    uint32_t above = incl - total;
    for (int i = 0; i < warp; ++i) above += warp_sum[i];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (above < need && above + bin[j] >= need)
        found[0] = kSelBins - 1 - (tid * PER + j), found[1] = above, found[2] = bin[j];
      above += bin[j];
    }
    __syncthreads();
    const uint64_t base = lo + (uint64_t(found[0]) << shift);
    need -= found[1];
    lo = base;
    const uint64_t width = (uint64_t(1) << shift) - 1;
    if (width < hi - base) hi = base + width;
    phase ^= 1;
    if (found[2] == need) break;  // the whole bin is kept
  }

  // ---- kept blocks in ascending order ----
  const int chunk = ((count + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int from = min(count, warp * chunk), to = min(count, from + chunk);
  uint32_t n_gt = 0, n_eq = 0;
  for (int i = from + lane; i < from + chunk && i - lane < to; i += 32) {
    const uint64_t k = i < to ? keys[i] : 0ull;
    n_gt += __popc(__ballot_sync(0xffffffffu, i < to && k > hi));
    n_eq += __popc(__ballot_sync(0xffffffffu, i < to && k >= lo && k <= hi));
  }
  if (lane == 0) take[0][warp] = n_gt, take[1][warp] = n_eq;
  __syncthreads();
  if (tid < 2) {
    uint32_t sum = 0;
    for (int i = 0; i < kSelWarps; ++i) {
      const uint32_t v = take[tid][i];
      take[tid][i] = sum;
      sum += v;
    }
    take[tid][kSelWarps] = sum;
  }
  cluster.sync();
  uint32_t gt = take[0][warp], eq = take[1][warp];
  for (uint32_t r = 0; r < rank; ++r) {
    gt += cluster.map_shared_rank(&take[0][0], r)[kSelWarps];
    eq += cluster.map_shared_rank(&take[1][0], r)[kSelWarps];
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
  for (int i = from + lane; i < from + chunk && i - lane < to; i += 32) {
    const uint64_t k = i < to ? keys[i] : 0ull;
    const uint32_t b_gt = __ballot_sync(0xffffffffu, i < to && k > hi);
    const uint32_t b_eq = __ballot_sync(0xffffffffu, i < to && k >= lo && k <= hi);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t my_eq = eq + __popc(b_eq & below);
    const uint32_t at = a.sink + gt + __popc(b_gt & below) + min(my_eq, need);
    if (((b_gt >> lane) & 1u) || (((b_eq >> lane) & 1u) && my_eq < need))
      out[at] = a.sink + first + i;
    gt += __popc(b_gt);
    eq += __popc(b_eq);
  }
}

}  // namespace dev
}  // namespace kvp
