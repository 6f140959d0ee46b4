// rope_reshape_and_cache: the position rotation of new queries and keys, the
// queries to q_out, the keys and values to their slots of the paged pool.
//
// For channel pair i of a row at position p, with c = cos_sin[p][i] and
// s = cos_sin[p][r/2 + i] (r = rot_dim):
//   y_a = x_a * c - x_b * s,   y_b = x_b * c + x_a * s,
// (a, b) = (i, r/2 + i) or, interleaved, (2i, 2i + 1). Channels from r on pass
// through. Products and sums are fp32, each rounded to nearest on its own (no
// fused multiply-add), so the result is the same bits as the two formulas
// written in fp32 anywhere; one rounding to the stored type follows.
//
// Bound by HBM: each of q, k and v is read once and written once. A CTA serves
// one token (or several, of few rows); a thread owns 16 channels (both ends of 8 pairs) of every row it
// visits, so its 8 cosines and 8 sines are loaded once and stay in registers
// while it walks the token's heads. 4 x 4,095 tokens of 32 + 8 heads into E4M3
// (373 MB) take 64 us, 5.8 TB/s; what is left is the latency of slot, table row
// and rows in turn, which many resident warps cover best: 12 CTAs per SM (40
// registers) 64 us, 10 67, 16 66. Four rows per thread in flight (80 registers) took
// 74 us, one pass per CTA 77, CTAs that stay for many tokens 71, and E4M3 codes by a
// bracketed reciprocal instead of 16 divisions per item (56 registers) 69.
#pragma once

#include "common.cuh"

namespace kvp {
namespace dev {

// Kind of the error word (beside DevErr's): position outside the table.
constexpr uint32_t KVP_DEVERR_POSITION = 6;

struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
  const float* cos_sin;                                // [max_positions][rot_dim]
  const int64_t* positions;
  int64_t max_positions;
  void* k_cache;
  void* v_cache;
  const int64_t* slots;
  const float* k_scale;
  const float* v_scale;
  int64_t num_slots;
  int32_t num_q_heads, num_kv_heads;
  int32_t rot_dim;
  int32_t log2_ipr;  // items (16 channels) per row
  int32_t log2_bs;
  int32_t rows_per_cta;  // rows (heads of q, k, v) per CTA, grid.y slices
  int32_t num_tokens;
  int32_t log2_tpt;  // threads per token; fewer than a CTA's where a token has few rows
};

constexpr int kRopeLog2Threads = 7, kRopeThreads = 1 << kRopeLog2Threads;

// T: 16-bit element; FP8: the cache holds E4M3 codes; PAIRED: interleaved pairs;
// PACKED: several tokens per CTA (14,124 tokens of 3 rows of 64 channels: 15.7 -> 4.2
// us; the general form costs the large case above 10 us in registers).
template <typename T, bool FP8, bool PAIRED, bool PACKED>
__global__ void __launch_bounds__(kRopeThreads, FP8 && !PACKED ? 12 : 10) rope_cache_kernel(const RopeArgs a) {
  const int log2_tpt = PACKED ? a.log2_tpt : kRopeLog2Threads;
  const int in_token = threadIdx.x & ((1 << log2_tpt) - 1);
  const int64_t t = int64_t(blockIdx.x) * (kRopeThreads >> log2_tpt) + (threadIdx.x >> log2_tpt);
  if (PACKED && t >= a.num_tokens) return;
  const int64_t slot = __ldg(a.slots + t);
  const int64_t pos = __ldg(a.positions + t);
  if (pos < 0 || pos >= a.max_positions) {
    // a padding token may carry any negative position; all else is a mistake
    if (!(slot < 0 && pos < 0) && blockIdx.y == 0 && in_token == 0)
      record_error(KVP_DEVERR_POSITION, uint64_t(t));
    return;
  }
  const bool store_kv = slot >= 0 && slot < a.num_slots;
  if (slot >= a.num_slots && blockIdx.y == 0 && in_token == 0)
    record_error(KVP_DEVERR_SLOT, uint64_t(t));

  const int j = in_token & ((1 << a.log2_ipr) - 1);
  const int rows_per_pass = (1 << log2_tpt) >> a.log2_ipr;
  const int D = 16 << a.log2_ipr;
  const bool rotated = j * 16 < a.rot_dim;
  // the item's two runs of 8 channels
  const int d0 = (PAIRED || !rotated) ? j * 16 : j * 8;
  const int d1 = (PAIRED || !rotated) ? j * 16 + 8 : a.rot_dim / 2 + j * 8;

  float c[8], s[8];
  if (rotated) {
    const float4* row = reinterpret_cast<const float4*>(a.cos_sin + pos * a.rot_dim + j * 8);
    const float4* row_s =
        reinterpret_cast<const float4*>(a.cos_sin + pos * a.rot_dim + a.rot_dim / 2 + j * 8);
    const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row_s), s1 = __ldg(row_s + 1);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w;
    c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w;
    s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }

  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  const int row_end = min(rows, int(blockIdx.y + 1) * a.rows_per_cta);
  for (int row = blockIdx.y * a.rows_per_cta + (in_token >> a.log2_ipr); row < row_end;
       row += rows_per_pass) {
    const bool is_q = row < a.num_q_heads;
    const bool is_v = row >= a.num_q_heads + a.num_kv_heads;
    const int h = is_q ? row : row - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
    if (!is_q && !store_kv) continue;
    const T* src = is_q ? static_cast<const T*>(a.q) + t * a.q_stride
                        : is_v ? static_cast<const T*>(a.v) + t * a.v_stride
                               : static_cast<const T*>(a.k) + t * a.k_stride;
    src += int64_t(h) * D;
    // plain loads: q_out may be q itself
    uint4 x0 = *reinterpret_cast<const uint4*>(src + d0);
    uint4 x1 = *reinterpret_cast<const uint4*>(src + d1);
    const bool turn = rotated && !is_v;
    if (!FP8 || is_q) {
      if (turn) {
        uint32_t* w0 = reinterpret_cast<uint32_t*>(&x0);
        uint32_t* w1 = reinterpret_cast<uint32_t*>(&x1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = Elem<T>::to_float2(w0[i]), w = Elem<T>::to_float2(w1[i]);
          if constexpr (PAIRED) {  // u is pair i, w is pair 4 + i
            w0[i] = Elem<T>::pack2(
                __fsub_rn(__fmul_rn(u.x, c[i]), __fmul_rn(u.y, s[i])),
                __fadd_rn(__fmul_rn(u.y, c[i]), __fmul_rn(u.x, s[i])));
            w1[i] = Elem<T>::pack2(
                __fsub_rn(__fmul_rn(w.x, c[4 + i]), __fmul_rn(w.y, s[4 + i])),
                __fadd_rn(__fmul_rn(w.y, c[4 + i]), __fmul_rn(w.x, s[4 + i])));
          } else {  // u.x with w.x is pair 2i, u.y with w.y pair 2i + 1
            w0[i] = Elem<T>::pack2(
                __fsub_rn(__fmul_rn(u.x, c[2 * i]), __fmul_rn(w.x, s[2 * i])),
                __fsub_rn(__fmul_rn(u.y, c[2 * i + 1]), __fmul_rn(w.y, s[2 * i + 1])));
            w1[i] = Elem<T>::pack2(
                __fadd_rn(__fmul_rn(w.x, c[2 * i]), __fmul_rn(u.x, s[2 * i])),
                __fadd_rn(__fmul_rn(w.y, c[2 * i + 1]), __fmul_rn(u.y, s[2 * i + 1])));
          }
        }
      }
      T* dst;
      if (is_q) {
        dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + int64_t(h) * D;
      } else {
        const int64_t blk = slot >> a.log2_bs, off = slot & ((int64_t(1) << a.log2_bs) - 1);
        dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) +
              (((blk * a.num_kv_heads + h) << a.log2_bs) + off) * D;
      }
      *reinterpret_cast<uint4*>(dst + d0) = x0;
      *reinterpret_cast<uint4*>(dst + d1) = x1;
    } else {
      // E4M3 codes of the rotated value over the head's scale (one rounding)
      const float scale = __ldg((is_v ? a.v_scale : a.k_scale) + h);
      const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
      uint32_t o0[4], o1[4];  // two codes each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 u = Elem<T>::to_float2(w0[i]), w = Elem<T>::to_float2(w1[i]);
        if (turn) {
          float2 y, z;
          if constexpr (PAIRED) {
            y.x = __fsub_rn(__fmul_rn(u.x, c[i]), __fmul_rn(u.y, s[i]));
            y.y = __fadd_rn(__fmul_rn(u.y, c[i]), __fmul_rn(u.x, s[i]));
            z.x = __fsub_rn(__fmul_rn(w.x, c[4 + i]), __fmul_rn(w.y, s[4 + i]));
            z.y = __fadd_rn(__fmul_rn(w.y, c[4 + i]), __fmul_rn(w.x, s[4 + i]));
          } else {
            y.x = __fsub_rn(__fmul_rn(u.x, c[2 * i]), __fmul_rn(w.x, s[2 * i]));
            y.y = __fsub_rn(__fmul_rn(u.y, c[2 * i + 1]), __fmul_rn(w.y, s[2 * i + 1]));
            z.x = __fadd_rn(__fmul_rn(w.x, c[2 * i]), __fmul_rn(u.x, s[2 * i]));
            z.y = __fadd_rn(__fmul_rn(w.y, c[2 * i + 1]), __fmul_rn(u.y, s[2 * i + 1]));
          }
          u = y, w = z;
        }
        o0[i] = float2_to_e4m3x2(__fdiv_rn(u.x, scale), __fdiv_rn(u.y, scale));
        o1[i] = float2_to_e4m3x2(__fdiv_rn(w.x, scale), __fdiv_rn(w.y, scale));
      }
      const int64_t blk = slot >> a.log2_bs, off = slot & ((int64_t(1) << a.log2_bs) - 1);
      uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                     (((blk * a.num_kv_heads + h) << a.log2_bs) + off) * D;
      *reinterpret_cast<uint2*>(dst + d0) = make_uint2(o0[0] | (o0[1] << 16), o0[2] | (o0[3] << 16));
      *reinterpret_cast<uint2*>(dst + d1) = make_uint2(o1[0] | (o1[1] << 16), o1[2] | (o1[3] << 16));
    }
  }
}

}  // namespace dev
}  // namespace kvp
