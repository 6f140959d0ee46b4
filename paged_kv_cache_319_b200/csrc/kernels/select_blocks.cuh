// select_blocks: for every (sequence, KV head), the blocks of its context that
// the group's new queries need most, by an upper bound on their logits.
//
// With M, m the block's channel-wise largest and smallest key,
//   score(b) = sum_d Q+[d] M[d] + Q-[d] m[d],
//   Q+ = sum_g max(q[g], 0),  Q- = sum_g min(q[g], 0),
// which is sum_g sum_d max(q[g][d] M[d], q[g][d] m[d]) and so no smaller than
// the sum over the group of any of the block's logits. A score costs 2 D
// multiply-adds whatever the group's size. The order is that of fp64 sums:
// 16-bit products are exact there and so, for all practical data, are the sums,
// which makes the choice independent of the summation order.
//
// Bound by HBM (the context's bounds are read once) if the scores cost little:
// in fp64 a block's 2 D conversions and multiply-adds and the reduction over the
// lanes took 4.4 times as long as its bytes (137 us for 32 x 8 rows of 1,500
// blocks and D = 128; now 46, of them about 8 after the last byte). So the scores
// are first taken on the tensor cores in fp32, 16 blocks (A rows) against the
// weights split into three 16-bit parts (columns 0 to 2 of B), with a bound E on
// their error; only blocks whose fp32 score lies within 2 E of the cut, usually a
// handful, are scored in fp64. Where many lie there (equal blocks, a zero query) or
// a fp32 sum could overflow, every block is; and so are all at once where there are only a
// few (up to 64: 4 sequences x 4 heads of 38 blocks 7.2 -> 4.3 us).
//
// E: the weights are scaled by a power of two to at most 2^15, so three parts
// leave 2^-24 of a weight or less; the MMAs' fp32 sums of 2 D products in steps
// of 16 are off by at most 2^-16 of the sum of the products' sizes even if each
// addend is cut to 24 bits; S = max |bound| * sum |weight| is no less than that
// sum, and E = 2^-15 S covers it twice, with 2^-126 sum |weight| + 2^-117 for bounds
// and products below fp32's normal range. No partial sum exceeds S either, so E below
// 2^111 (S below 2^126) keeps them all finite; bf16 bounds from 2^103 (many equal
// weights) or 2^112 (one) on are scored in fp64.
//
// One cluster of up to 8 CTAs serves a (sequence, KV head); each CTA scores a
// contiguous range of blocks. The scores, as order-preserving keys, go straight to
// the first CTA's shared memory, which selects alone: after the scores, what
// counts is the latency of the steps, and a step over the cluster takes 2 to 4 us
// (a barrier and remote reads) where one CTA takes under 1. Only a context with
// more blocks than one CTA holds is selected by the cluster together. The cut is
// found by zooming: a 1024-bin histogram of the active key range names the bin
// that holds the last kept key. The kept blocks are written in ascending order at
// offsets from a prefix sum over warps (and CTAs).
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "mma_sync.cuh"

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

constexpr int kSelMaxWarps = 16;
constexpr int kSelBins = 1024;
constexpr int kSelLog2Bins = 10;
constexpr int kSelNear = 64;  // most blocks near the cut that are scored again

// Order-preserving maps to unsigned integers. fp64: NaN above everything, -0 equal
// to 0. 0 is below the key of every number.
__device__ __forceinline__ uint64_t score_key(double x) {
  if (x != x) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ uint32_t approx_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float approx_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k ^ 0x80000000u) : ~k);
}

// Most CTAs of a cluster, and most keys of one CTA (8 bytes each).
constexpr int kSelMaxRanks = 8;
constexpr int kSelMaxKeys = 26 * 1024;

// The shared state of one selection.
struct SelectShared {
  uint32_t hist[2][kSelBins];
  // of the keys of each warp of the CTAs that select together: range, and the
  // largest |bound| (16-bit pattern)
  uint32_t range_lo[kSelMaxRanks * kSelMaxWarps], range_hi[kSelMaxRanks * kSelMaxWarps];
  uint32_t biggest[kSelMaxRanks * kSelMaxWarps];
  uint64_t warp_lo[kSelMaxWarps], warp_hi[kSelMaxWarps], cta_lo, cta_hi;  // of the fp64 keys
  uint32_t warp_sum[kSelMaxWarps];
  float weight_max[kSelMaxWarps], weight_sum[kSelMaxWarps];
  uint32_t found[3];             // bin, keys above it, keys in it
  uint32_t take[2][kSelMaxWarps + 1];  // kept / tied keys per warp, and of the CTA
  uint32_t above, near;          // this CTA's keys past the near ones, near ones
  uint32_t near_at[kSelNear];    // their places, and fp64 keys
  uint64_t near_key[kSelNear];
  uint32_t all_at[kSelNear];     // all ranks', gathered
  uint64_t all_key[kSelNear];
  uint32_t near_kept[kSelMaxRanks];  // kept near keys of each rank
};

// The CTAs that select together: one (n = 1), or the whole cluster.
struct SelectRanks {
  cooperative_groups::cluster_group cluster;
  uint32_t n;
  __device__ __forceinline__ void sync() {
    if (n == 1)
      __syncthreads();
    else
      cluster.sync();
  }
  template <typename X>
  __device__ __forceinline__ X* at(X* p, uint32_t r) {
    return n == 1 ? p : cluster.map_shared_rank(p, r);
  }
};

// f(i, keys[i]) for this thread's i of [0, count), eight reads in flight.
template <int WARPS, typename Key, typename F>
__device__ __forceinline__ void for_each_key(const Key* keys, int count, F f) {
  constexpr int U = 8, kThreads = WARPS * 32;
  for (int i0 = threadIdx.x; i0 < count; i0 += U * kThreads) {
    Key k[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kThreads < count) k[u] = keys[i0 + u * kThreads];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kThreads < count) f(i0 + u * kThreads, k[u]);
  }
}

// One zoom: the bin of keys[0, count) within [lo, hi] (over the ranks) that holds
// the need-th largest, in found; hist[phase] is used, hist[phase ^ 1] is cleared
// for the next. `found` is written again only after the next ranks.sync.
template <int WARPS, typename Key>
__device__ __forceinline__ int zoom(SelectShared& sh, SelectRanks& ranks, const Key* keys,
                                    int count, Key lo, Key hi, uint32_t need, int phase) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bits = 64 - __clzll(static_cast<long long>(hi - lo));
  const int shift = bits > kSelLog2Bins ? bits - kSelLog2Bins : 0;
  uint32_t* mine = sh.hist[phase];
  for_each_key<WARPS>(keys, count, [&](int, Key k) {
    if (k >= lo && k <= hi) atomicAdd(&mine[uint32_t((k - lo) >> shift)], 1u);
  });
  ranks.sync();
  // each thread: neighbouring bins of the merged histogram, highest first
  constexpr int PER = kSelBins / (WARPS * 32);
  uint32_t bin[PER], total = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) bin[j] = 0;
  for (uint32_t r = 0; r < ranks.n; ++r) {
    const uint32_t* theirs = ranks.at(mine, r);
#pragma unroll
    for (int j = 0; j < PER; ++j) bin[j] += theirs[kSelBins - 1 - (tid * PER + j)];
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) total += bin[j];
  uint32_t incl = total;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += v;
  }
  if (lane == 31) sh.warp_sum[warp] = incl;
  // the other buffer was last read before this call's ranks.sync
  for (int i = tid; i < kSelBins; i += WARPS * 32) sh.hist[phase ^ 1][i] = 0;
  __syncthreads();
  uint32_t above = incl - total + __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0u);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (above < need && above + bin[j] >= need)
      sh.found[0] = kSelBins - 1 - (tid * PER + j), sh.found[1] = above, sh.found[2] = bin[j];
    above += bin[j];
  }
  __syncthreads();
  return shift;
}

// The fp64 keys of blocks table[at[0..U)] (by a warp; every lane has them). at < 0:
// no block, key 0 like a block id outside the pool.
template <typename TB, int D, int U>
__device__ __forceinline__ void exact_keys(const SelectArgs& a, const double* weight,
                                           const int32_t* table, const int (&at)[U], uint32_t g,
                                           uint64_t (&key)[U]) {
  constexpr int W = D / 32;  // 2-element words per lane
  const int lane = threadIdx.x & 31;
  int32_t b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) b[u] = at[u] >= 0 ? __ldg(table + at[u]) : -1;
  uint32_t x[U][W];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (b[u] >= a.num_blocks) b[u] = -1;
    const uint32_t* src = static_cast<const uint32_t*>(a.bounds) +
                          (int64_t(b[u]) * a.num_kv_heads + g) * D + lane;
#pragma unroll
    for (int i = 0; i < W; ++i) x[u][i] = b[u] >= 0 ? __ldg(src + i * 32) : 0u;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 f = Elem<TB>::to_float2(x[u][i]);
      const double2 w = *reinterpret_cast<const double2*>(weight + (i * 32 + lane) * 2);
      sum = fma(w.x, double(f.x), sum);
      sum = fma(w.y, double(f.y), sum);
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    key[u] = b[u] >= 0 ? score_key(sum) : 0ull;
  }
}

// TQ: the queries' type, TB: the bounds' type, WARPS: per CTA.
template <typename TQ, typename TB, int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
    select_blocks_kernel(const SelectArgs a) {
  namespace cg = cooperative_groups;
  constexpr int kThreads = WARPS * 32;
  extern __shared__ uint64_t keys[];
  uint32_t* keys32 = reinterpret_cast<uint32_t*>(keys);
  __shared__ SelectShared sh;
  __shared__ __align__(16) double weight[2 * D];    // Q+, then Q-
  __shared__ __align__(16) uint16_t part[3][2 * D]; // their scaled 16-bit parts

  SelectRanks ranks{cg::this_cluster(), 1};
  const uint32_t nranks = ranks.cluster.num_blocks();
  uint32_t rank = ranks.cluster.block_rank();
  const uint32_t unit = blockIdx.x / nranks;
  const uint32_t s = unit / a.num_kv_heads, g = unit - s * a.num_kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int ctx = __ldg(a.context_lens + s);
  if (ctx < 0 || ctx > a.max_context_len) {
    if (g == 0 && rank == 0 && tid == 0) record_error(KVP_DEVERR_CTX, s);
    ctx = ctx < 0 ? 0 : a.max_context_len;
  }
  const int n = int((ctx + (int64_t(1) << a.log2_bs) - 1) >> a.log2_bs);
  int32_t* out = a.out + int64_t(unit) * a.keep;
  if (n <= a.keep) {  // every block is kept (uniform over the cluster)
    if (rank == 0)
      for (int i = tid; i < a.keep; i += kThreads) out[i] = i < n ? i : -1;
    return;
  }
  // n > keep >= sink + recent: candidates [sink, n - recent)
  const int cand = n - a.sink - a.recent;
  uint32_t need = a.keep - a.sink - a.recent;
  if (rank == 0) {
    for (int i = tid; i < a.sink; i += kThreads) out[i] = i;
    for (int i = tid; i < a.recent; i += kThreads) out[a.keep - a.recent + i] = n - a.recent + i;
  }
  if (need == 0) return;
  const int per = (cand + nranks - 1) / nranks;
  int first = min(cand, int(rank) * per), count = min(cand, first + per) - first;
  const int32_t* table = a.block_tables + int64_t(s) * a.max_blocks_per_seq + a.sink + first;
  const bool gather = cand <= kSelMaxKeys;  // the first CTA selects alone

  const int G = a.num_q_heads / a.num_kv_heads;
  // the sum of a channel's weights over the group; comparisons that keep a NaN query
  auto channel_weight = [&](int e) {
    const bool low = e >= D;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) +
                        (int64_t(s) * a.num_q_heads + int64_t(g) * G) * D + (low ? e - D : e);
    double w = 0.0;
    for (int h = 0; h < G; ++h) {
      const float f = Elem<TQ>::to_float2(__ldg(q + int64_t(h) * D)).x;
      w += double(low ? (f > 0.f ? 0.f : f) : (f < 0.f ? 0.f : f));
    }
    return w;
  };

  // A few blocks: their fp64 scores at once, and every one's place by counting.
  if (cand <= kSelNear) {
    if (rank != 0) return;
    for (int e = tid; e < 2 * D; e += kThreads) weight[e] = channel_weight(e);
    __syncthreads();
    constexpr int U = kSelNear / WARPS;
    int at[U];
    uint64_t k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = u * WARPS + warp < cand ? u * WARPS + warp : -1;
    exact_keys<TB, D, U>(a, weight, table, at, g, k);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (lane == 0) sh.near_key[u * WARPS + warp] = k[u];
    if (tid < cand) {
      const int32_t b = __ldg(table + tid);
      if ((b < 0 || b >= a.num_blocks) && g == 0)
        record_error(KVP_DEVERR_BLOCK_ID, (uint64_t(s) << 32) | uint32_t(a.sink + tid));
    }
    __syncthreads();
    bool kept = false;
    if (tid < cand) {
      const uint64_t mine = sh.near_key[tid];
      uint32_t better = 0;
      for (int i = 0; i < cand; ++i)
        better += sh.near_key[i] > mine || (sh.near_key[i] == mine && i < tid);
      kept = better < need;
    }
    if (tid < kSelNear) {
      const uint32_t m = __ballot_sync(0xffffffffu, kept);
      if (lane == 0) sh.take[0][warp] = m;
    }
    __syncthreads();
    if (kept) {
      uint32_t pos = a.sink + __popc(sh.take[0][warp] & ((1u << lane) - 1u));
      for (int i = 0; i < warp; ++i) pos += __popc(sh.take[0][i]);
      if (pos < uint32_t(a.keep)) out[pos] = a.sink + tid;
    }
    return;
  }

  // the other CTAs' shared memory may be written once they have all started
  if (nranks > 1) ranks.cluster.barrier_arrive();

  // ---- the first loads of the scores, started beside the weights ----
  // 16 blocks per warp and step: lane l holds rows r = l/4 and r + 8 of A and
  // column r of B; of a row it reads 16 bytes at a time, whose words are the k
  // positions of two MMA steps.
  constexpr int ROW = 2 * D * 2;  // bytes of a block's bounds of one head
  constexpr int L = ROW / 64;     // 16-byte loads per row and lane
  const int r = lane >> 2, p = lane & 3;
  auto locate = [&](int c0) {
    int32_t id = -1;
    const int c = c0 + (lane & 15);
    if (c < count) {
      id = __ldg(table + c);
      if (id < 0 || id >= a.num_blocks) {
        if (g == 0 && lane < 16)
          record_error(KVP_DEVERR_BLOCK_ID, (uint64_t(s) << 32) | uint32_t(a.sink + first + c));
        id = -1;
      }
    }
    return id;
  };
  // a step's rows are loaded in two halves, each as soon as its registers are
  // free, so that half of the bytes are always on the way
  uint4 x[2][2][L / 2];
  auto load = [&](int half, int32_t ids) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int32_t b = __shfl_sync(0xffffffffu, ids, r + 8 * y);
      const char* src = static_cast<const char*>(a.bounds) +
                        (int64_t(b) * a.num_kv_heads + g) * ROW + half * (ROW / 2) + p * 16;
#pragma unroll
      for (int j = 0; j < L / 2; ++j) {
        x[half][y][j] = make_uint4(0, 0, 0, 0);
        if (b >= 0) x[half][y][j] = ld_stream(src + j * 64);
      }
    }
  };
  int32_t id = locate(warp * 16), next = locate((warp + WARPS) * 16);

  // ---- weights: fp64 sums, and their three 16-bit parts ----
  float wmax = 0.f, wsum = 0.f;
  for (int e = tid; e < 2 * D; e += kThreads) {
    const double w = channel_weight(e);
    weight[e] = w;
    wmax = fmaxf(wmax, fabsf(float(w)));
  }
  load(0, id);
  load(1, id);
  for (int m = 1; m < 32; m <<= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, m));
  if (lane == 0) sh.weight_max[warp] = wmax;
  for (int i = tid; i < kSelBins; i += kThreads) sh.hist[0][i] = 0;
  __syncthreads();
  for (int i = 0; i < WARPS; ++i) wmax = fmaxf(wmax, sh.weight_max[i]);
  const int wexp = int(__float_as_uint(wmax) >> 23) - 127;
  const double up = wmax > 0.f ? __hiloint2double((1023 + 14 - wexp) << 20, 0) : 1.0;
  for (int e = tid; e < 2 * D; e += kThreads) {
    double w = weight[e] * up;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t x = Elem<TB>::from_float(float(w));
      part[i][e] = uint16_t(x);
      w -= double(Elem<TB>::to_float2(x).x);
    }
    wsum += float(fabs(weight[e] * up));
  }
  for (int m = 1; m < 32; m <<= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, m);
  if (lane == 0) sh.weight_sum[warp] = wsum;
  __syncthreads();
  wsum = 0.f;
  for (int i = 0; i < WARPS; ++i) wsum += sh.weight_sum[i];

  if (nranks > 1) ranks.cluster.barrier_wait();

  // ---- fp32 scores ----
  {
    uint4 w[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      w[j] = make_uint4(0, 0, 0, 0);
      if (r < 3) w[j] = *reinterpret_cast<const uint4*>(&part[r][j * 32 + p * 8]);
    }
    uint32_t big = 0, my_lo = ~0u, my_hi = 0;
    uint32_t* dst = gather ? ranks.cluster.map_shared_rank(keys32, 0) + first : keys32;
    for (int c0 = warp * 16; c0 < count; c0 += WARPS * 16) {
      const int32_t after = locate(c0 + 2 * WARPS * 16);
      float z[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) z[0][e] = z[1][e] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int j = 0; j < L / 2; ++j) {
          const uint4 u = x[half][0][j], v = x[half][1][j], wj = w[half * (L / 2) + j];
          const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
          mma16816<TB>(z[0], a0, wj.x, wj.y);
          mma16816<TB>(z[1], a1, wj.z, wj.w);
          big = __vmaxu2(big, u.x & 0x7fff7fffu);
          big = __vmaxu2(big, u.y & 0x7fff7fffu);
          big = __vmaxu2(big, u.z & 0x7fff7fffu);
          big = __vmaxu2(big, u.w & 0x7fff7fffu);
          big = __vmaxu2(big, v.x & 0x7fff7fffu);
          big = __vmaxu2(big, v.y & 0x7fff7fffu);
          big = __vmaxu2(big, v.z & 0x7fff7fffu);
          big = __vmaxu2(big, v.w & 0x7fff7fffu);
        }
        load(half, next);
      }
      // columns 0 and 1 are in the lanes of p = 0, column 2 in those of p = 1
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float c01 = (z[0][2 * y] + z[1][2 * y]) + (z[0][2 * y + 1] + z[1][2 * y + 1]);
        const float c2 = __shfl_down_sync(0xffffffffu, z[0][2 * y] + z[1][2 * y], 1);
        const bool valid = __shfl_sync(0xffffffffu, id, r + 8 * y) >= 0;
        const int c = c0 + y * 8 + r;
        if (p == 0 && c < count) {
          const uint32_t k = valid ? approx_key(c01 + c2) : 0u;
          dst[c] = k;
          my_lo = min(my_lo, k);
          my_hi = max(my_hi, k);
        }
      }
      id = next;
      next = after;
    }
    big = max(big >> 16, big & 0xffffu);
    big = __reduce_max_sync(0xffffffffu, big);
    my_lo = __reduce_min_sync(0xffffffffu, my_lo);
    my_hi = __reduce_max_sync(0xffffffffu, my_hi);
    // to the first CTA, or to every one
    if (lane == 0)
      for (uint32_t o = 0; o < (gather ? 1 : nranks); ++o) {
        SelectShared* to = ranks.cluster.map_shared_rank(&sh, o);
        const int at = rank * WARPS + warp;
        to->range_lo[at] = my_lo, to->range_hi[at] = my_hi, to->biggest[at] = big;
      }
  }
  if (nranks > 1)
    ranks.cluster.sync();
  else
    __syncthreads();
  if (gather) {
    if (rank != 0) return;  // nothing of this CTA's is read any more
    count = cand;
  } else {
    ranks.n = nranks;
  }
  uint32_t lo32 = ~0u, hi32 = 0, big = 0;  // the active keys lie in [lo32, hi32]
  for (int i = lane; i < int(nranks) * WARPS; i += 32) {
    lo32 = min(lo32, sh.range_lo[i]);
    hi32 = max(hi32, sh.range_hi[i]);
    big = max(big, sh.biggest[i]);
  }
  lo32 = __reduce_min_sync(0xffffffffu, lo32);
  hi32 = __reduce_max_sync(0xffffffffu, hi32);
  big = __reduce_max_sync(0xffffffffu, big);
  const float err = (Elem<TB>::to_float2(big).x * 0x1p-15f + 0x1p-126f) * wsum + 0x1p-117f;
  const bool finite = big < (std::is_same<TB, __half>::value ? 0x7c00u : 0x7f80u) &&
                      err < 0x1p111f && (wmax == 0.f || wmax >= 0x1p-126f) &&
                      wmax < __int_as_float(0x7f800000);  // else a scaled part may be infinite

  // ---- the cut: keys above near_hi are kept, those below near_lo are not ----
  int phase = 0;
  bool exact = !finite;  // score every block in fp64
  uint32_t near_lo = 0, near_hi = ~0u, active = need;
  while (!exact) {
    if (lo32 < hi32) {
      const int shift = zoom<WARPS>(sh, ranks, keys32, count, lo32, hi32, active, phase);
      phase ^= 1;
      const uint32_t base = lo32 + (sh.found[0] << shift), width = (1u << shift) - 1u;
      active -= sh.found[1];
      lo32 = base;
      if (width < hi32 - base) hi32 = base + width;
    }
    // the need-th largest fp32 score lies in [f_lo, f_hi]; the need-th largest
    // score within err of it
    const float f_lo = approx_value(lo32), f_hi = approx_value(hi32);
    near_lo = lo32 ? approx_key(__fsub_rd(f_lo, 2.f * err)) : 0u;
    near_hi = hi32 ? approx_key(__fadd_ru(f_hi, 2.f * err)) : 0u;
    if (tid == 0) sh.above = sh.near = 0;
    __syncthreads();
    uint32_t n_above = 0;
    for_each_key<WARPS>(keys32, count, [&](int i, uint32_t k) {
      n_above += k > near_hi;
      if (k >= near_lo && k <= near_hi) {
        const uint32_t at = atomicAdd(&sh.near, 1u);
        if (at < kSelNear) sh.near_at[at] = i;
      }
    });
    n_above = __reduce_add_sync(0xffffffffu, n_above);
    if (lane == 0 && n_above) atomicAdd(&sh.above, n_above);
    ranks.sync();
    uint32_t near = 0, above = 0;
    for (uint32_t r = 0; r < ranks.n; ++r) {
      const SelectShared* o = ranks.at(&sh, r);
      near += o->near, above += o->above;
    }
    if (near <= kSelNear || near + above == need) {
      need -= above;
      break;
    }
    // a range no wider than the doubt around it will not get better
    exact = lo32 == hi32 || f_hi - f_lo <= err;
    ranks.sync();  // above and near are written again
  }

  uint64_t lo = 0, hi = 0;       // of the fp64 keys: those above hi are kept, and
                                 // the first `need` of those in [lo, hi]
  uint32_t cut = 0;              // of the fp32 keys: the least kept one
  uint32_t base_gt = 0, base_eq = 0;  // kept / tied keys of the ranks before this one
  if (!exact) {
    uint32_t near = 0, before = 0, mine = sh.near;
    for (uint32_t r = 0; r < ranks.n; ++r) {
      const uint32_t o = ranks.at(&sh, r)->near;
      if (r < rank) before += o;
      near += o;
    }
    if (near == need) {  // every near block is kept
      cut = near_lo;
      if (tid < int(ranks.n)) sh.near_kept[tid] = ranks.at(&sh, tid)->near;
      __syncthreads();
    } else {
      cut = near_hi + 1u;
      for (uint32_t i = warp; i < mine; i += WARPS) {
        const int at[1] = {int(sh.near_at[i])};
        uint64_t k[1];
        exact_keys<TB, D, 1>(a, weight, table, at, g, k);
        if (lane == 0) sh.near_key[i] = k[0];
      }
      if (tid < kSelMaxRanks) sh.near_kept[tid] = 0;
      ranks.sync();
      // each rank gathers all near keys and ranks them; position: rank, then place
      uint32_t owner = 0, j = tid;
      if (tid < int(near)) {
        while (true) {
          const uint32_t o = ranks.at(&sh, owner)->near;
          if (j < o) break;
          j -= o, ++owner;
        }
        const SelectShared* o = ranks.at(&sh, owner);
        sh.all_key[tid] = o->near_key[j];
        sh.all_at[tid] = owner * uint32_t(per) + o->near_at[j];
      }
      __syncthreads();
      if (tid < int(near)) {
        const uint64_t k = sh.all_key[tid];
        const uint32_t at = sh.all_at[tid];
        uint32_t better = 0;
        for (uint32_t i = 0; i < near; ++i)
          better += sh.all_key[i] > k || (sh.all_key[i] == k && sh.all_at[i] < at);
        if (better < need) atomicAdd(&sh.near_kept[owner], 1u);
        if (owner == rank) keys32[sh.near_at[j]] = better < need ? ~0u : 0u;
      }
      __syncthreads();
    }
    for (uint32_t r = 0; r < rank; ++r)
      base_gt += ranks.at(&sh, r)->above + sh.near_kept[r];
  } else {
    ranks.sync();  // the scores and their range are written again
    uint64_t my_lo = ~0ull, my_hi = 0;
    constexpr int U = 8;  // blocks in flight per warp
    for (int c0 = warp * U; c0 < count; c0 += WARPS * U) {
      int at[U];
      uint64_t k[U];
#pragma unroll
      for (int u = 0; u < U; ++u) at[u] = c0 + u < count ? c0 + u : -1;
      exact_keys<TB, D, U>(a, weight, table, at, g, k);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c0 + u >= count) continue;
        if (lane == 0) keys[c0 + u] = k[u];
        my_lo = min(my_lo, k[u]);
        my_hi = max(my_hi, k[u]);
      }
    }
    if (lane == 0) sh.warp_lo[warp] = my_lo, sh.warp_hi[warp] = my_hi;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < WARPS; ++i)
        my_lo = min(my_lo, sh.warp_lo[i]), my_hi = max(my_hi, sh.warp_hi[i]);
      sh.cta_lo = my_lo, sh.cta_hi = my_hi;
    }
    ranks.sync();
    lo = ~0ull, hi = 0;
    for (uint32_t r = 0; r < ranks.n; ++r) {
      const SelectShared* o = ranks.at(&sh, r);
      lo = min(lo, o->cta_lo);
      hi = max(hi, o->cta_hi);
    }
    while (lo < hi) {
      const int shift = zoom<WARPS>(sh, ranks, keys, count, lo, hi, need, phase);
      phase ^= 1;
      need -= sh.found[1];
      lo += uint64_t(sh.found[0]) << shift;
      const uint64_t width = (uint64_t(1) << shift) - 1;
      if (width < hi - lo) hi = lo + width;
      if (sh.found[2] == need) break;  // the whole bin is kept
    }
  }

  // ---- kept blocks in ascending order ----
  if (!exact) {
    // a warp takes runs of 1024 keys in turn: lane i keeps the mask of the run's
    // i-th 32 keys, so two scans (lanes, warps) give every mask its offset
    ranks.sync();  // no CTA leaves, or reuses it, while another reads its memory
    uint32_t at = a.sink + base_gt;
    for (int c0 = 0; c0 < count; c0 += WARPS * 1024) {
      const int from = c0 + warp * 1024;
      uint32_t mask = 0;
      const int masks = min(32, (count - from + 31) >> 5);
#pragma unroll 8
      for (int i = 0; i < masks; ++i) {
        const int c = from + i * 32 + lane;
        const uint32_t m = __ballot_sync(0xffffffffu, c < count && keys32[c] >= cut);
        if (lane == i) mask = m;
      }
      uint32_t incl = __popc(mask);
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += v;
      }
      if (lane == 31) sh.warp_sum[warp] = incl;
      __syncthreads();
      const uint32_t sums = lane < WARPS ? sh.warp_sum[lane] : 0u;
      uint32_t pos = at + incl - __popc(mask) + __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0u);
      at += __reduce_add_sync(0xffffffffu, sums);
      for (; mask; mask &= mask - 1, ++pos)
        if (pos < uint32_t(a.keep)) out[pos] = a.sink + first + from + lane * 32 + __ffs(mask) - 1;
      __syncthreads();  // warp_sum is written again
    }
    return;
  }
  auto look = [&](int i, bool& gt, bool& eq) {
    const uint64_t k = i < count ? keys[i] : 0ull;
    gt = i < count && k > hi;
    eq = i < count && k >= lo && k <= hi;
  };
  const int chunk = ((count + WARPS - 1) / WARPS + 31) & ~31;
  const int from = warp * chunk, to = min(count, from + chunk);
  uint32_t n_gt = 0, n_eq = 0;
  for (int i = from; i < to; i += 32) {
    bool gt, eq;
    look(i + lane, gt, eq);
    n_gt += __popc(__ballot_sync(0xffffffffu, gt));
    n_eq += __popc(__ballot_sync(0xffffffffu, eq));
  }
  if (lane == 0) sh.take[0][warp] = n_gt, sh.take[1][warp] = n_eq;
  __syncthreads();
  if (tid < 2) {
    uint32_t sum = 0;
    for (int i = 0; i < WARPS; ++i) {
      const uint32_t v = sh.take[tid][i];
      sh.take[tid][i] = sum;
      sum += v;
    }
    sh.take[tid][WARPS] = sum;
  }
  ranks.sync();
  for (uint32_t r = 0; r < rank; ++r) {
    const SelectShared* o = ranks.at(&sh, r);
    base_gt += o->take[0][WARPS];
    base_eq += o->take[1][WARPS];
  }
  ranks.sync();  // no CTA leaves while another reads its shared memory
  uint32_t gt = base_gt + sh.take[0][warp], eq = base_eq + sh.take[1][warp];
  for (int i = from; i < to; i += 32) {
    bool is_gt, is_eq;
    look(i + lane, is_gt, is_eq);
    const uint32_t b_gt = __ballot_sync(0xffffffffu, is_gt);
    const uint32_t b_eq = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t my_eq = eq + __popc(b_eq & below);
    const uint32_t at = a.sink + gt + __popc(b_gt & below) + min(my_eq, need);
    if ((is_gt || (is_eq && my_eq < need)) && at < uint32_t(a.keep)) out[at] = a.sink + first + i + lane;
    gt += __popc(b_gt);
    eq += __popc(b_eq);
  }
}

}  // namespace dev
}  // namespace kvp
