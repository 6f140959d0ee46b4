// paged_attention_decode_sparse: decode attention over the blocks a list names,
// one list per (sequence, KV head).
//
//   out[s][h] = sum_j softmax_j(scale * q[s][h] . key j) * value j
// over the tokens j < ctx of the listed blocks. An online softmax (running
// maximum m, sum l, unnormalised output, all fp32, log2 domain) is kept per
// warp; warps, then the CTAs of a cluster, are merged by the log-sum-exp
// identity at the end, in a fixed order, so there is no workspace, no second
// kernel and no atomic.
//
// Bound by HBM: a listed block's keys and values are read once per KV head and
// serve the whole group. Every warp works alone on tiles of 16 tokens (two
// half tiles of 8, so blocks of 8, 16 and 32 tokens are alike): TMA fills a ring of
// stages of its own, and mma.sync multiplies from there. Keys and values are
// the A operand (16 tokens, or 16 channels, by 16) and up to 8 query heads per
// column tile the B operand: at the 2 to 32 FLOP per byte of this operator the
// legacy tensor-core path is nowhere near its limit (15 to 22% busy), and a tcgen05
// tile would need 128 rows staged in shared memory first. What bounds a warp is
// the latency of its chain of instructions per tile, so the softmax takes one
// vote per tile and no reduction (32 sequences x 32 heads x 4096 tokens, bf16, on
// 1,024 CTAs: 125 us with a reduction and a rescaling per tile, 105 without), and
// the tiles are swizzled, so that no read has a bank conflict (on 256 CTAs 92 us
// with unswizzled bulk copies, 84 swizzled; 64 x 40 heads x 512 tokens, fp16: 97
// and 87 us, 6.7 TB/s).
//
// Operand layout. In m16n8k16, lane l holds rows l/4 and l/4 + 8 of A and, of
// each row, the k positions 2p, 2p+1, 2p+8, 2p+9 (p = l % 4). A contraction may
// take its k positions in any order if both operands agree:
//  - logits (k = channels): lane l reads 16 contiguous bytes of its token rows,
//    so a 16-byte read feeds two (E4M3: four) k steps; queries are loaded alike.
//  - output (rows = channels, k = tokens): lane l reads 16 bytes of channels
//    of tokens 2p, 2p+1, 2p+8, 2p+9 and pairs neighbouring tokens' values with
//    byte permutes; row l/4 of the row tiles stands for the lane's channels.
// The probabilities come out of the first product as [token][head] and enter
// the second as [token][head] with rows and columns swapped over the lanes: one
// 8x8 transpose (movmatrix) each.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "mma_sync.cuh"

namespace kvp {
namespace dev {
namespace sparse {

// Kind of the error word (beside DevErr's): listed block past the context.
constexpr uint32_t KVP_DEVERR_SELECTED = 7;

struct SparseArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* selected;
  void* out;
  int32_t num_seqs, num_q_heads, num_kv_heads, num_blocks, max_blocks_per_seq;
  int32_t max_context_len;
  int32_t log2_bs;
  int32_t num_selected;
  int32_t head_tiles;  // units per (sequence, KV head): ceil(G / (8 NT))
  uint32_t num_units;  // served by a CTA, a cluster of them, or (SOLO) a warp each
  float scale_log2;
};

// The pools as TMA maps: [rows][D] in boxes of min(block_size, 16) rows, 128-byte
// swizzled, a 256-byte row as two segments ([segment][row][128 bytes]).
struct SparseMaps {
  CUtensorMap k, v;
};

constexpr int kChunk = 512;  // tiles located per pass over the list

// Shared memory: the K/V stages, shared out among the warps (later the merge area),
// then the located rows and valid tokens of kChunk tiles' halves, then the barriers.
// A warp has two stages of 8 KiB (D = 128, 16-bit) or of 4 KiB. Many rows: 64 KiB of
// stages, so that a CTA's start and merge are covered by its neighbours' loads (64
// sequences x 40 heads x 512 tokens before the swizzle, two stages in three CTAs per
// SM: 108 us; three stages in two CTAs 124, six in one 182). Few rows (WIDE): one CTA
// per SM with twice the stages and warps, because a warp's chain per tile takes about
// 1 us (3 sequences x 8 KV heads x 16,000 E4M3 tokens: 31 and 27 us).
template <bool WIDE>
constexpr int kStageBytes = (WIDE ? 128 : 64) * 1024;
template <bool WIDE>
constexpr int kSmemBytes = kStageBytes<WIDE> + kChunk * 10 + 16 * 16 * 8;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(addr));
  return x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t word(const uint4& x, int i) {
  return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
}

// Warps per CTA. The 16-head tiles' merge area leaves room for four.
template <bool FP8, int D, int NT, bool WIDE>
constexpr int kSparseWarps = ((FP8 || D == 64) && NT == 1 ? 8 : 4) * (WIDE ? 2 : 1);

// How the rows are spread: a CTA or a cluster per unit; the same with wide CTAs; or a
// warp per unit, for many rows of short lists: no merge, and a quarter of the CTAs.
enum Spread { CTA, WIDE_CTA, SOLO };

// CTAs per SM that the registers should allow.
template <bool FP8, int D, int NT, Spread SPREAD>
constexpr int kSparseCtas =
    SPREAD == WIDE_CTA ? 1 : NT == 1 && kSparseWarps<FP8, D, NT, false> == 4 ? 3 : 2;

// T: queries, output and products; FP8: E4M3 cache (D = 128); NT: tiles of 8 heads.
template <typename T, bool FP8, int D, int NT, Spread SPREAD>
__global__ void __launch_bounds__(kSparseWarps<FP8, D, NT, SPREAD == WIDE_CTA> * 32,
                                  kSparseCtas<FP8, D, NT, SPREAD>)
    decode_sparse_kernel(const __grid_constant__ SparseMaps maps, const SparseArgs a) {
  namespace cg = cooperative_groups;
  constexpr bool WIDE = SPREAD == WIDE_CTA, ALONE = SPREAD == SOLO;
  constexpr int ROW = D * (FP8 ? 1 : 2);  // bytes of a cached row
  constexpr int KL = ROW / 64;            // 16-byte key loads per token row and lane
  constexpr int VL = ROW / 128;           // 16-byte value loads per token and lane
  constexpr int MT = D / 16;              // 16-channel row tiles of the output
  constexpr int QW = D / 8;               // query words per lane and head tile
  constexpr int HEADS = NT * 8;
  // type of the products: E4M3 values are fp16 values, so an E4M3 cache takes fp16
  // products (bf16 queries scaled by a power of two into its range)
  using M = typename std::conditional<FP8, __half, T>::type;
  // The weights are 2^kLift at their reference and 2^(kLift + 8) at most, so fp16 parts
  // reach down to 2^-(24 + kLift) of it; without the lift a long tail of weights below
  // 2^-25 would vanish from the second product but not from the sum. bf16 has fp32's
  // range. The factor is in the sums as well and cancels.
  constexpr float kLift = std::is_same<M, __half>::value ? 7.f : 0.f;
  constexpr bool kScaleQ = FP8 && !std::is_same<T, __half>::value;
  static_assert(!FP8 || D == 128, "E4M3 caches have head_dim 128");

  constexpr int TILE = 16 * ROW;                    // bytes of a tile's keys
  constexpr int kWarps = kSparseWarps<FP8, D, NT, WIDE>, kThreads = kWarps * 32;
  constexpr int RING = kStageBytes<WIDE> / kWarps;  // bytes of a warp's stages
  constexpr int STAGES = RING / (2 * TILE);
  static_assert(STAGES <= 16 && kStageBytes<WIDE> >= (kWarps * HEADS * (D + 2) + 2 * HEADS) * 4,
                "the merge area lies over the stages");

  extern __shared__ __align__(1024) unsigned char smem[];
  float* sm_acc = reinterpret_cast<float*>(smem);     // [kWarps][HEADS][D]
  float* sm_m = sm_acc + kWarps * HEADS * D;          // [kWarps][HEADS]
  float* sm_l = sm_m + kWarps * HEADS;
  float* part_m = sm_l + kWarps * HEADS;              // [HEADS], this CTA's merged partial
  float* part_l = part_m + HEADS;
  uint2* rows = reinterpret_cast<uint2*>(smem + kStageBytes<WIDE>);  // [kChunk], a row per half
  uint16_t* valid = reinterpret_cast<uint16_t*>(rows + kChunk);         // [kChunk], a byte per half
  uint64_t* bars = reinterpret_cast<uint64_t*>(valid + kChunk);         // [kWarps][16]

  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const uint32_t nranks = ALONE ? 1 : cluster.num_blocks(), rank = ALONE ? 0 : cluster.block_rank();
  const uint32_t unit = ALONE ? blockIdx.x * kWarps + wid : blockIdx.x / nranks;
  if (ALONE && unit >= a.num_units) return;  // a warp of its own: no barrier of the CTA follows
  const uint32_t ht = unit % a.head_tiles;
  const uint32_t sg = unit / a.head_tiles;
  const uint32_t s = sg / a.num_kv_heads, g = sg - s * a.num_kv_heads;
  const int r = lane >> 2, p = lane & 3;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int h0 = ht * HEADS;  // first head of the tile within the group
  const int bs = 1 << a.log2_bs;

  int ctx = __ldg(a.context_lens + s);
  if (ctx < 0 || ctx > a.max_context_len) {
    if (g == 0 && ht == 0 && rank == 0 && (ALONE ? lane : tid) == 0) record_error(KVP_DEVERR_CTX, s);
    ctx = ctx < 0 ? 0 : a.max_context_len;
  }

  // queries: column r of head tile t is head h0 + 8 t + r
  uint32_t qf[NT][QW];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = h0 + t * 8 + r;
    const bool live = h < G;
    const T* q = static_cast<const T*>(a.q) +
                 (int64_t(s) * a.num_q_heads + int64_t(g) * G + (live ? h : 0)) * D;
#pragma unroll
    for (int i = 0; i < QW / 4; ++i) {
      // the channels of the lane's 16-byte key reads, chunks 2p and 2p + 1 of a segment
      const int d = FP8 ? (2 * p + (i >> 1)) * 16 + (i & 1) * 8 : (i >> 1) * 64 + (2 * p + (i & 1)) * 8;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (live) x = __ldg(reinterpret_cast<const uint4*>(q + d));
      qf[t][4 * i] = x.x, qf[t][4 * i + 1] = x.y, qf[t][4 * i + 2] = x.z, qf[t][4 * i + 3] = x.w;
    }
  }
  float scale[NT][2];  // of the logits of columns 2p, 2p + 1
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    scale[t][0] = scale[t][1] = FP8 ? a.scale_log2 * __ldg(a.k_scale + g) : a.scale_log2;
    if constexpr (kScaleQ) {
      // each head's queries times 2^k with the largest in [2^14, 2^15): what is
      // lost below fp16's normal range is 2^-39 of the largest or less
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < QW; ++i) big = __vmaxu2(big, qf[t][i] & 0x7fff7fffu);
      big = max(big >> 16, big & 0xffffu);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const uint32_t e = min(268u - (big >> 7), 253u);  // biased exponent of 2^k
      const float up = __uint_as_float(e << 23), down = __uint_as_float((254u - e) << 23);
#pragma unroll
      for (int i = 0; i < QW; ++i) {
        const float2 f = Elem<T>::to_float2(qf[t][i]);
        qf[t][i] = Elem<M>::pack2(f.x * up, f.y * up);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) scale[t][c] *= __shfl_sync(0xffffffffu, down, (2 * p + c) * 4);
    }
  }

  float acc[NT][MT][4];
  // m: the reference of the exponentials, a recent maximum less kLift; l: this lane's sum
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][j][e] = 0.f;
  }

  const int32_t* list = a.selected + int64_t(sg) * a.num_selected;
  const int32_t* table = a.block_tables + int64_t(s) * a.max_blocks_per_seq;
  const int halves = a.num_selected << (a.log2_bs - 3);  // half tiles of 8 tokens
  const int tiles = (halves + 1) >> 1;
  // Tile j of this CTA is tile ((j / kWarps) * nranks + rank) * kWarps + j % kWarps of
  // the list; a lone warp takes them all. `rounds`: tiles per warp.
  const int rounds = ALONE ? tiles : (tiles + kWarps * int(nranks) - 1) / (kWarps * int(nranks));
  constexpr int kPass = kChunk / kWarps;  // of them, located at a time
  auto place = [&](int i) { return ALONE ? wid * kPass + i : i * kWarps + wid; };

  // cache row (block, head, slot) of half tile `half`, and its tokens below ctx
  auto locate = [&](int half, uint32_t& row, int& valid) {
    row = 0;
    valid = 0;
    if (half >= halves) return;
    const int32_t lb = __ldg(list + (half >> (a.log2_bs - 3)));
    if (lb < 0) return;
    const int off = (half << 3) & (bs - 1);
    if (lb >= (ctx + int64_t(bs) - 1) >> a.log2_bs) {
      if (off == 0 && ht == 0) record_error(KVP_DEVERR_SELECTED, (uint64_t(sg) << 32) | uint32_t(lb));
      return;
    }
    const int32_t b = __ldg(table + lb);
    if (b < 0 || b >= a.num_blocks) {
      if (off == 0 && ht == 0) record_error(KVP_DEVERR_BLOCK_ID, (uint64_t(s) << 32) | uint32_t(lb));
      return;
    }
    row = ((uint32_t(b) * a.num_kv_heads + g) << a.log2_bs) + off;
    valid = max(0, min(8, ctx - (lb << a.log2_bs) - off));
  };

  uint64_t* bar = bars + wid * 16;
  if (lane < STAGES) mbar_init(bar + lane, 1);
  fence_mbar_init();
  unsigned char* ring = smem + wid * RING;
  const uint32_t stage0 = smem_u32(ring);
  // bytes between a tile's halves and between the segments of a row
  const uint32_t half_bytes = bs >= 16 ? 1024 : TILE / 2, seg_bytes = bs >= 16 ? 2048 : 1024;
  if ((ALONE ? lane : tid) == 0) prefetch_tensormap(&maps.k), prefetch_tensormap(&maps.v);
  const uint64_t policy = l2_policy_evict_first();
  uint32_t phases = 0;  // parity of each stage's next completion
  bool alive = true;

  auto sync = [&] {
    if constexpr (ALONE)
      __syncwarp();
    else
      __syncthreads();
  };
  for (int i0 = 0; i0 < rounds; i0 += kPass) {
    const int mine = min(kPass, rounds - i0);
    for (int j = ALONE ? lane : tid; j < (ALONE ? mine : mine * kWarps); j += ALONE ? 32 : kThreads) {
      const int t = ALONE ? i0 + j
                          : ((i0 + j / kWarps) * int(nranks) + int(rank)) * kWarps + j % kWarps;
      uint2 row;
      int va, vb;
      locate(2 * t, row.x, va);
      locate(2 * t + 1, row.y, vb);
      const int at = ALONE ? wid * kPass + j : j;
      rows[at] = row;
      valid[at] = uint16_t(va | (vb << 8));
    }
    sync();
    // loads of the warp's tile i into stage st, whole boxes: slots past the context
    // come along and are masked
    auto issue = [&](int i, int st) {
      const int j = place(i);
      const uint32_t v = valid[j];
      if (v == 0) return;
      const bool a0 = v & 0xffu, a1 = v >> 8;
      if (lane == 0)
        mbar_arrive_expect_tx(bar + st, bs >= 16 ? 2 * TILE : (uint32_t(a0) + uint32_t(a1)) * TILE);
      __syncwarp();
      if (lane < (bs >= 16 ? 2 : 4)) {  // lane bit 0: keys or values, bit 1: half tile
        const uint2 row = rows[j];
        if (lane >> 1 ? a1 : (a0 || bs >= 16)) {
          unsigned char* dst = ring + st * 2 * TILE + (lane & 1) * TILE + (lane >> 1) * (TILE / 2);
          const CUtensorMap* map = lane & 1 ? &maps.v : &maps.k;
          const int y = int(lane >> 1 ? row.y : row.x);
          if constexpr (ROW == 256)
            tma_load_3d(dst, map, bar + st, 0, y, 0, policy);
          else
            tma_load_2d(dst, map, bar + st, 0, y, policy);
        }
      }
    };
    if (alive)
      for (int i = 0; i < min(mine, STAGES - 1); ++i) issue(i, i);
    int st = -1, fill = STAGES - 2;  // stages of tile i and of tile i + STAGES - 1
    for (int i = 0; i < mine && alive; ++i) {
      st = st + 1 == STAGES ? 0 : st + 1;
      fill = fill + 1 == STAGES ? 0 : fill + 1;
      __syncwarp();  // every lane has read the stage that is filled next
      if (i + STAGES - 1 < mine) issue(i + STAGES - 1, fill);
      const int v = valid[place(i)], va = v & 0xff, vb = v >> 8;
      if (v == 0) continue;
      const bool ok = mbar_wait(bar + st, (phases >> st) & 1u, 0x5000u + st);
      phases ^= 1u << st;
      if (!__all_sync(0xffffffffu, ok)) {
        // give up: wait (each with the limit) for the copies in flight, read nothing
        for (int k = i + 1; k < min(mine, i + STAGES); ++k)
          if (valid[place(k)])
            mbar_wait(bar + k % STAGES, (phases >> (k % STAGES)) & 1u, 0x5000u + st);
        alive = false;
        break;
      }

      uint4 kx[2][KL], vx[4][VL];
      // 16-byte chunk c of a segment's row x is stored as chunk c ^ (x mod 8): the
      // eight lanes of each quarter warp read eight different chunks
      const uint32_t ks = stage0 + st * 2 * TILE, vs = ks + TILE;
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int j = 0; j < KL; ++j)
          kx[y][j] = lds128(ks + y * half_bytes + (j >> 1) * seg_bytes + r * 128 +
                            (((2 * p + (j & 1)) ^ r) << 4));
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t tok = 2 * p + (y & 1);
#pragma unroll
        for (int j = 0; j < VL; ++j)
          vx[y][j] = lds128(vs + (y >> 1) * half_bytes + j * seg_bytes + tok * 128 + ((r ^ tok) << 4));
      }
      const bool partial = va + vb < 16;
      if (partial) {  // a stage's unfilled value rows hold anything
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (2 * p + (y & 1) >= (y >> 1 ? vb : va))
#pragma unroll
            for (int j = 0; j < VL; ++j) vx[y][j] = make_uint4(0, 0, 0, 0);
      }

      // ---- logits: [16 tokens][8 heads] per head tile, in two chains ----
      float z[NT][4], z1[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[t][e] = z1[t][e] = 0.f;
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        if constexpr (FP8) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // word c: 4 channels, one k step
            const uint32_t x = word(kx[0][j], c), y = word(kx[1][j], c);
            const uint32_t af[4] = {e4m3x2_to_x2<M>(x & 0xffffu), e4m3x2_to_x2<M>(y & 0xffffu),
                                    e4m3x2_to_x2<M>(x >> 16), e4m3x2_to_x2<M>(y >> 16)};
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma16816<M>(c & 1 ? z1[t] : z[t], af, qf[t][j * 8 + 2 * c], qf[t][j * 8 + 2 * c + 1]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t af[4] = {word(kx[0][j], 2 * c), word(kx[1][j], 2 * c),
                                    word(kx[0][j], 2 * c + 1), word(kx[1][j], 2 * c + 1)};
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma16816<M>(c ? z1[t] : z[t], af, qf[t][j * 4 + 2 * c], qf[t][j * 4 + 2 * c + 1]);
          }
        }
      }

      // ---- online softmax, per head (columns 2p, 2p + 1; rows r and r + 8) ----
      // The reference of the exponentials follows the maximum only when a logit
      // exceeds it by more than 8 (a factor 256, so weights up to 2^15): one
      // vote per tile instead of a reduction over the lanes and a rescaling. The
      // difference is compared, since m + 8 rounds up where m has few bits below 8.
      bool rise = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[t][e] = (z[t][e] + z1[t][e]) * scale[t][e & 1];
          if (partial && r >= (e >> 1 ? vb : va)) z[t][e] = -INFINITY;
          rise |= z[t][e] - m[t][e & 1] > 8.f + kLift;
        }
      }
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(z[t][c], z[t][2 + c]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[t][c], mx - kLift);
            const float alpha = mn == -INFINITY ? 1.f : ex2(m[t][c] - mn);
            m[t][c] = mn;
            l[t][c] *= alpha;
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[t][j][c] *= alpha, acc[t][j][2 + c] *= alpha;
          }
      }
      uint32_t pb[NT][2], pl[NT][2];  // probabilities as the B operand, and their low parts
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[t][e & 1];
          pr[e] = ex2(z[t][e] - (ref == -INFINITY ? 0.f : ref));
          l[t][e & 1] += pr[e];
        }
        // p rounded once to 16 bits would cost up to as much again as the output's own
        // rounding (an eighth of it where fp16 products make a bf16 output), so it goes
        // as a high and a low part
        const uint32_t hi0 = Elem<M>::pack2(pr[0], pr[1]), hi1 = Elem<M>::pack2(pr[2], pr[3]);
        pb[t][0] = transpose8x8(hi0);
        pb[t][1] = transpose8x8(hi1);
        const float2 f0 = Elem<M>::to_float2(hi0), f1 = Elem<M>::to_float2(hi1);
        pl[t][0] = transpose8x8(Elem<M>::pack2(pr[0] - f0.x, pr[1] - f0.y));
        pl[t][1] = transpose8x8(Elem<M>::pack2(pr[2] - f1.x, pr[3] - f1.y));
      }

      // ---- output: [channels][heads] += values^T * p ----
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        uint32_t af[4];
        if constexpr (FP8) {
          // row tile j: channels r*16 + 2j, +1; bytes 2(j&1), +1 of word j/2
          const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
          const uint32_t x = __byte_perm(word(vx[0][0], j / 2), word(vx[1][0], j / 2), sel);
          const uint32_t y = __byte_perm(word(vx[2][0], j / 2), word(vx[3][0], j / 2), sel);
          af[0] = e4m3x2_to_x2<M>(x & 0xffffu), af[1] = e4m3x2_to_x2<M>(x >> 16);
          af[2] = e4m3x2_to_x2<M>(y & 0xffffu), af[3] = e4m3x2_to_x2<M>(y >> 16);
        } else {
          // row tile j: channels (j/4)*64 + r*8 + 2(j%4), +1: word j%4 of load j/4
          const uint32_t x0 = word(vx[0][j / 4], j % 4), x1 = word(vx[1][j / 4], j % 4);
          const uint32_t y0 = word(vx[2][j / 4], j % 4), y1 = word(vx[3][j / 4], j % 4);
          af[0] = __byte_perm(x0, x1, 0x5410), af[1] = __byte_perm(x0, x1, 0x7632);
          af[2] = __byte_perm(y0, y1, 0x5410), af[3] = __byte_perm(y0, y1, 0x7632);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816<M>(acc[t][j], af, pb[t][0], pb[t][1]);
          mma16816<M>(acc[t][j], af, pl[t][0], pl[t][1]);
        }
      }
    }
    sync();  // the located rows, or the stages, are written next
  }

  const int heads = min(HEADS, G - h0);
  const float vs = FP8 ? __ldg(a.v_scale + g) : 1.f;
  uint16_t* out = static_cast<uint16_t*>(a.out) +
                  (int64_t(s) * a.num_q_heads + int64_t(g) * G + h0) * D;

  if constexpr (ALONE) {
    // the lanes of a column have its sum; each writes its own channels
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[t][c];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int h = t * 8 + 2 * p + c;
        if (h >= heads) continue;
        const bool none = x == 0.f;
        uint32_t w[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j)
          w[j] = Elem<T>::pack2(none ? 0.f : acc[t][j][c] * vs / x, none ? 0.f : acc[t][j][2 + c] * vs / x);
#pragma unroll
        for (int j = 0; j < MT; j += 4) {
          const int d = FP8 ? r * 16 + 2 * j : (j / 4) * 64 + r * 8;
          *reinterpret_cast<uint4*>(out + h * D + d) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
        }
      }
    return;
  }

  // ---- merge: lanes of a column, warps, CTAs ----
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x = l[t][c];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int h = t * 8 + 2 * p + c;
      if (r == 0) sm_m[wid * HEADS + h] = m[t][c], sm_l[wid * HEADS + h] = x;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int d = FP8 ? r * 16 + 2 * j : (j / 4) * 64 + r * 8 + 2 * (j % 4);
        *reinterpret_cast<float2*>(sm_acc + (wid * HEADS + h) * D + d) =
            make_float2(acc[t][j][c], acc[t][j][2 + c]);
      }
    }
  __syncthreads();
  for (int i = tid; i < heads * D; i += kThreads) {  // into warp 0's buffer, or out
    const int h = i / D;
    float mx = sm_m[h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w * HEADS + h]);
    const float ms = mx == -INFINITY ? 0.f : mx;
    float o = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(sm_m[w * HEADS + h] - ms);
      o += f * sm_acc[w * HEADS * D + i];
      sum += f * sm_l[w * HEADS + h];
    }
    if (nranks == 1) {
      out[i] = Elem<T>::from_float(sum == 0.f ? 0.f : o * vs / sum);
      continue;
    }
    sm_acc[i] = o;
    if (i % D == 0) part_m[h] = mx, part_l[h] = sum;
  }
  if (nranks == 1) return;
  cluster.sync();
  for (int i = rank * kThreads + tid; i < heads * D; i += nranks * kThreads) {
    const int h = i / D;
    float mx = -INFINITY;
    for (uint32_t c = 0; c < nranks; ++c) mx = fmaxf(mx, cluster.map_shared_rank(part_m, c)[h]);
    const float ms = mx == -INFINITY ? 0.f : mx;
    float o = 0.f, sum = 0.f;
    for (uint32_t c = 0; c < nranks; ++c) {
      const float f = ex2(cluster.map_shared_rank(part_m, c)[h] - ms);
      o += f * cluster.map_shared_rank(sm_acc, c)[i];
      sum += f * cluster.map_shared_rank(part_l, c)[h];
    }
    out[i] = Elem<T>::from_float(sum == 0.f ? 0.f : o * vs / sum);
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace sparse
}  // namespace dev
}  // namespace kvp
