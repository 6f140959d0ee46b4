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
// half tiles of 8, so blocks of 8, 16 and 32 tokens are alike) that it loads
// from global memory straight into mma.sync operand registers: 8 KiB in flight
// per warp with no shared-memory round trip and no barrier, so occupancy alone
// covers the latency of the scattered reads. Keys and values are the A operand
// (16 tokens, or 16 channels, by 16) and up to 8 query heads per column tile the
// B operand: at the 2 to 32 FLOP per byte of this operator the legacy
// tensor-core path is nowhere near its limit, and a tcgen05 tile would need
// 128 rows staged in shared memory first.
//
// Operand layout. In m16n8k16, lane l holds rows l/4 and l/4 + 8 of A and, of
// each row, the k positions 2p, 2p+1, 2p+8, 2p+9 (p = l % 4). A contraction may
// take its k positions in any order if both operands agree:
//  - logits (k = channels): lane l loads 16 contiguous bytes of its token rows,
//    so a 16-byte load feeds two (E4M3: four) k steps; queries are loaded alike.
//  - output (rows = channels, k = tokens): lane l loads 16 bytes of channels
//    of tokens 2p, 2p+1, 2p+8, 2p+9 and pairs neighbouring tokens' values with
//    byte permutes; row l/4 of the row tiles stands for the lane's channels.
// The probabilities come out of the first product as [token][head] and enter
// the second as [token][head] with rows and columns swapped over the lanes: one
// 8x8 transpose (movmatrix) each.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace kvp {
namespace dev {
namespace sparse {

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
  int32_t head_tiles;  // CTAs (clusters) per (sequence, KV head): ceil(G / (8 NT))
  float scale_log2;
};

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                 uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

__device__ __forceinline__ uint32_t word(const uint4& x, int i) {
  return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
}

// T: queries, output and products; FP8: E4M3 cache (D = 128); NT: tiles of 8 heads.
template <typename T, bool FP8, int D, int NT>
__global__ void __launch_bounds__(kThreads) decode_sparse_kernel(const SparseArgs a) {
  namespace cg = cooperative_groups;
  constexpr int ROW = D * (FP8 ? 1 : 2);  // bytes of a cached row
  constexpr int KL = ROW / 64;            // 16-byte key loads per token row and lane
  constexpr int VL = ROW / 128;           // 16-byte value loads per token and lane
  constexpr int MT = D / 16;              // 16-channel row tiles of the output
  constexpr int QW = D / 8;               // query words per lane and head tile
  constexpr int HEADS = NT * 8;
  static_assert(!FP8 || D == 128, "E4M3 caches have head_dim 128");

  extern __shared__ float sm[];
  float* sm_acc = sm;                                 // [kWarps][HEADS][D]
  float* sm_m = sm + kWarps * HEADS * D;              // [kWarps][HEADS]
  float* sm_l = sm_m + kWarps * HEADS;
  float* part_m = sm_l + kWarps * HEADS;              // [HEADS], this CTA's merged partial
  float* part_l = part_m + HEADS;

  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t nranks = cluster.num_blocks(), rank = cluster.block_rank();
  const uint32_t unit = blockIdx.x / nranks;
  const uint32_t ht = unit % a.head_tiles;
  const uint32_t sg = unit / a.head_tiles;
  const uint32_t s = sg / a.num_kv_heads, g = sg - s * a.num_kv_heads;
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, p = lane & 3;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int h0 = ht * HEADS;  // first head of the tile within the group
  const int bs = 1 << a.log2_bs;

  int ctx = __ldg(a.context_lens + s);
  if (ctx < 0 || ctx > a.max_context_len) {
    if (g == 0 && ht == 0 && rank == 0 && tid == 0) record_error(KVP_DEVERR_CTX, s);
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
      // 16-bit rows: 8 channels at i*32 + p*8; E4M3 rows: 16 channels at (i/2)*64 + p*16
      const int d = FP8 ? (i / 2) * 64 + p * 16 + (i & 1) * 8 : i * 32 + p * 8;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (live) x = __ldg(reinterpret_cast<const uint4*>(q + d));
      qf[t][4 * i] = x.x, qf[t][4 * i + 1] = x.y, qf[t][4 * i + 2] = x.z, qf[t][4 * i + 3] = x.w;
    }
  }
  const float scale = FP8 ? a.scale_log2 * __ldg(a.k_scale + g) : a.scale_log2;

  float acc[NT][MT][4];
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
  const int stride = int(nranks) * kWarps, w0 = int(rank) * kWarps + wid;

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

  for (int base = w0; base < tiles; base += 32 * stride) {
    // lane i locates the warp's i-th tile of the next 32
    uint32_t row0 = 0, row1 = 0;
    int v0 = 0, v1 = 0;
    {
      const int t = base + lane * stride;
      if (t < tiles) {
        locate(2 * t, row0, v0);
        locate(2 * t + 1, row1, v1);
      }
    }
    const int batch = min(32, (tiles - base + stride - 1) / stride);
    for (int i = 0; i < batch; ++i) {
      const uint32_t ra = __shfl_sync(0xffffffffu, row0, i), rb = __shfl_sync(0xffffffffu, row1, i);
      const int va = __shfl_sync(0xffffffffu, v0, i), vb = __shfl_sync(0xffffffffu, v1, i);
      if (va + vb == 0) continue;

      // ---- loads; rows past the context are zeros, never read ----
      uint4 kx[2][KL], vx[4][VL];
      const char* kc = static_cast<const char*>(a.k_cache);
      const char* vc = static_cast<const char*>(a.v_cache);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const bool ok = r < (y ? vb : va);
        const char* src = kc + int64_t((y ? rb : ra) + r) * ROW + p * 16;
#pragma unroll
        for (int j = 0; j < KL; ++j) {
          kx[y][j] = make_uint4(0, 0, 0, 0);
          if (ok) kx[y][j] = ld_stream(src + j * 64);
        }
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int tok = 2 * p + (y & 1);
        const bool ok = tok < (y >> 1 ? vb : va);
        const char* src = vc + int64_t((y >> 1 ? rb : ra) + tok) * ROW + r * 16;
#pragma unroll
        for (int j = 0; j < VL; ++j) {
          vx[y][j] = make_uint4(0, 0, 0, 0);
          if (ok) vx[y][j] = ld_stream(src + j * 128);
        }
      }

      // ---- logits: [16 tokens][8 heads] per head tile ----
      float z[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) z[t][0] = z[t][1] = z[t][2] = z[t][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        if constexpr (FP8) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // word c: 4 channels, one k step
            const uint32_t x = word(kx[0][j], c), y = word(kx[1][j], c);
            const uint32_t af[4] = {e4m3x2_to_x2<T>(x & 0xffffu), e4m3x2_to_x2<T>(y & 0xffffu),
                                    e4m3x2_to_x2<T>(x >> 16), e4m3x2_to_x2<T>(y >> 16)};
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma16816<T>(z[t], af, qf[t][j * 8 + 2 * c], qf[t][j * 8 + 2 * c + 1]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t af[4] = {word(kx[0][j], 2 * c), word(kx[1][j], 2 * c),
                                    word(kx[0][j], 2 * c + 1), word(kx[1][j], 2 * c + 1)};
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma16816<T>(z[t], af, qf[t][j * 4 + 2 * c], qf[t][j * 4 + 2 * c + 1]);
          }
        }
      }

      // ---- online softmax over the tile's tokens, per head (columns 2p, 2p + 1) ----
      uint32_t pb[NT][2], pl[NT][2];  // probabilities as the B operand, and their low parts
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float pr[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float x = r < va ? z[t][c] * scale : -INFINITY;
          const float y = r < vb ? z[t][2 + c] * scale : -INFINITY;
          float mx = fmaxf(x, y);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[t][c], mx);
          const float ms = mn == -INFINITY ? 0.f : mn;
          const float alpha = exp2f(m[t][c] - ms);
          pr[c] = r < va ? exp2f(x - ms) : 0.f;
          pr[2 + c] = r < vb ? exp2f(y - ms) : 0.f;
          m[t][c] = mn;
          l[t][c] = l[t][c] * alpha + pr[c] + pr[2 + c];
#pragma unroll
          for (int j = 0; j < MT; ++j) acc[t][j][c] *= alpha, acc[t][j][2 + c] *= alpha;
        }
        // one rounding of p to 11 bits for fp16; bf16's 8 bits would cost more
        // than the output's own rounding, so p goes as a high and a low part
        const uint32_t hi0 = Elem<T>::pack2(pr[0], pr[1]), hi1 = Elem<T>::pack2(pr[2], pr[3]);
        pb[t][0] = transpose8x8(hi0);
        pb[t][1] = transpose8x8(hi1);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          const float2 f0 = Elem<T>::to_float2(hi0), f1 = Elem<T>::to_float2(hi1);
          pl[t][0] = transpose8x8(Elem<T>::pack2(pr[0] - f0.x, pr[1] - f0.y));
          pl[t][1] = transpose8x8(Elem<T>::pack2(pr[2] - f1.x, pr[3] - f1.y));
        }
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
          af[0] = e4m3x2_to_x2<T>(x & 0xffffu), af[1] = e4m3x2_to_x2<T>(x >> 16);
          af[2] = e4m3x2_to_x2<T>(y & 0xffffu), af[3] = e4m3x2_to_x2<T>(y >> 16);
        } else {
          // row tile j: channels (j/4)*64 + r*8 + 2(j%4), +1: word j%4 of load j/4
          const uint32_t x0 = word(vx[0][j / 4], j % 4), x1 = word(vx[1][j / 4], j % 4);
          const uint32_t y0 = word(vx[2][j / 4], j % 4), y1 = word(vx[3][j / 4], j % 4);
          af[0] = __byte_perm(x0, x1, 0x5410), af[1] = __byte_perm(x0, x1, 0x7632);
          af[2] = __byte_perm(y0, y1, 0x5410), af[3] = __byte_perm(y0, y1, 0x7632);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816<T>(acc[t][j], af, pb[t][0], pb[t][1]);
          if constexpr (std::is_same<T, __nv_bfloat16>::value)
            mma16816<T>(acc[t][j], af, pl[t][0], pl[t][1]);
        }
      }
    }
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
  const int heads = min(HEADS, G - h0);
  for (int i = tid; i < heads * D; i += kThreads) {  // into warp 0's buffer
    const int h = i / D;
    float mx = sm_m[h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w * HEADS + h]);
    const float ms = mx == -INFINITY ? 0.f : mx;
    float o = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(sm_m[w * HEADS + h] - ms);
      o += f * sm_acc[w * HEADS * D + i];
      sum += f * sm_l[w * HEADS + h];
    }
    sm_acc[i] = o;
    if (i % D == 0) part_m[h] = mx, part_l[h] = sum;
  }
  cluster.sync();
  const float vs = FP8 ? __ldg(a.v_scale + g) : 1.f;
  uint16_t* out = static_cast<uint16_t*>(a.out) +
                  (int64_t(s) * a.num_q_heads + int64_t(g) * G + h0) * D;
  for (int i = rank * kThreads + tid; i < heads * D; i += nranks * kThreads) {
    const int h = i / D;
    float mx = -INFINITY;
    for (uint32_t c = 0; c < nranks; ++c) mx = fmaxf(mx, cluster.map_shared_rank(part_m, c)[h]);
    const float ms = mx == -INFINITY ? 0.f : mx;
    float o = 0.f, sum = 0.f;
    for (uint32_t c = 0; c < nranks; ++c) {
      const float f = exp2f(cluster.map_shared_rank(part_m, c)[h] - ms);
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
