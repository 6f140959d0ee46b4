// Entry points of block-sparse decoding (C ABI): the rotary append, the
// per-block key bounds, the block selection and the decode over the selected
// blocks. Argument checks, kernel selection by geometry, launches on the
// caller's stream. Included at the end of kvp_device.cu, whose helpers and device
// error word it shares.
#pragma once

#include <array>
#include <type_traits>

#include "kernels/decode_sparse.cuh"
#include "kernels/key_bounds.cuh"
#include "kernels/rope_cache.cuh"
#include "kernels/select_blocks.cuh"

namespace {

// Launch of `units` clusters of `ranks` CTAs along x; max_smem: the most dynamic
// shared memory that any launch of this kernel takes.
template <typename... Args>
int launch_clusters(const char* fn, void (*kernel)(Args...), int64_t units, int ranks, int threads,
                    int smem, int max_smem, cudaStream_t st,
                    const std::remove_const_t<Args>&... args) {
  if (units * ranks >= (int64_t(1) << 31)) return fail(KVP_ERR_INVALID, "%s: batch too large", fn);
  if (smem > 32 * 1024) {  // beside up to 16 KiB of static shared memory
    cudaError_t e = ensure_smem(kernel, max_smem);
    if (e != cudaSuccess) return cuda_fail(e, fn);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(units * ranks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {unsigned(ranks), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? KVP_OK : cuda_fail(e, fn);
}

// Clusters of `ranks` (1 to 8) CTAs that are on the current device at once, asked
// once per kernel, device and size. The kernel's shared-memory limit has been raised.
template <typename... Args>
int resident_clusters(void (*kernel)(Args...), int ranks, int threads, int smem) {
  static std::mutex mu;
  static std::unordered_map<const void*, std::array<int, kMaxDevices * 8>> known;
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return sm_count() / (2 * ranks);
  std::lock_guard<std::mutex> guard(mu);
  int& n = known[reinterpret_cast<const void*>(kernel)][d * 8 + ranks - 1];  // 0: not asked
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(ranks));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {unsigned(ranks), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 1;
    }
  }
  return n;
}

// Checks that select_blocks and paged_attention_decode_sparse share.
int check_rows(const char* fn, int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
               int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t max_blocks_per_seq,
               int32_t max_context_len, int32_t num_selected, int32_t dtype, int32_t cache_dtype) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || max_context_len < 0)
    return fail(KVP_ERR_INVALID, "%s: bad sizes", fn);
  if (num_q_heads % num_kv_heads) return fail(KVP_ERR_INVALID, "%s: num_q_heads %% num_kv_heads != 0", fn);
  if (block_size != 8 && block_size != 16 && block_size != 32)
    return fail(KVP_ERR_INVALID, "%s: block_size must be 8, 16 or 32", fn);
  if (dtype != KVP_F16 && dtype != KVP_BF16) return fail(KVP_ERR_INVALID, "%s: bad dtype", fn);
  if (cache_dtype != dtype && cache_dtype != KVP_FP8_E4M3)
    return fail(KVP_ERR_INVALID, "%s: the cache is of the queries' type or E4M3", fn);
  if (head_dim != 128 && (head_dim != 64 || cache_dtype == KVP_FP8_E4M3))
    return fail(KVP_ERR_INVALID, "%s: head_dim must be 64 or 128 (E4M3: 128)", fn);
  if (int64_t(max_context_len) > int64_t(max_blocks_per_seq) * block_size)
    return fail(KVP_ERR_INVALID, "%s: max_context_len > max_blocks_per_seq * block_size", fn);
  if (num_selected <= 0 || num_selected > (1 << 24))
    return fail(KVP_ERR_INVALID, "%s: num_selected must be in [1, 2^24]", fn);
  return KVP_OK;
}

// Whether two sets of num_tokens 16-bit rows (strides in elements) may share an
// element. Exact for rows of one stride, as views of one projection's output
// have; rows of different strides count as overlapping where their extents do.
bool rows_overlap(const void* a, int64_t a_stride, int64_t a_row, const void* b, int64_t b_stride,
                  int64_t b_row, int32_t num_tokens) {
  const int64_t x = int64_t(reinterpret_cast<uintptr_t>(a) / 2);
  const int64_t y = int64_t(reinterpret_cast<uintptr_t>(b) / 2);
  const int64_t n = num_tokens - 1;
  if (x + n * a_stride + a_row <= y || y + n * b_stride + b_row <= x) return false;
  if (n == 0 || a_stride != b_stride || a_stride <= 0) return true;
  const int64_t delta = ((y - x) % a_stride + a_stride) % a_stride;  // from a row of a to b's next
  return delta < a_row || a_stride - delta < b_row;
}

// Channel counts per row that the 16-channel items of the append cover.
int log2_items(int32_t head_dim) { return head_dim % 16 ? -1 : ilog2(head_dim / 16); }

template <typename T, bool FP8>
int launch_rope(const kvp::dev::RopeArgs& a, dim3 grid, bool interleaved, cudaStream_t st) {
  const bool packed = a.log2_tpt < kvp::dev::kRopeLog2Threads;
  auto k = packed ? (interleaved ? kvp::dev::rope_cache_kernel<T, FP8, true, true>
                                 : kvp::dev::rope_cache_kernel<T, FP8, false, true>)
                  : (interleaved ? kvp::dev::rope_cache_kernel<T, FP8, true, false>
                                 : kvp::dev::rope_cache_kernel<T, FP8, false, false>);
  k<<<grid, kvp::dev::kRopeThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? KVP_OK : cuda_fail(e, "rope_reshape_and_cache: launch");
}

template <typename T, bool FP8, int D>
int launch_bounds(const kvp::dev::BoundsArgs& a, int64_t warps, cudaStream_t st) {
  const int64_t ctas = (warps + kvp::dev::kBoundsWarps - 1) / kvp::dev::kBoundsWarps;
  kvp::dev::key_bounds_kernel<T, FP8, D><<<unsigned(ctas), kvp::dev::kBoundsWarps * 32, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? KVP_OK : cuda_fail(e, "update_key_bounds: launch");
}

template <typename TQ, typename TB>
int launch_select(const kvp::dev::SelectArgs& a, int head_dim, cudaStream_t st) {
  using kvp::dev::kSelMaxKeys;
  const int64_t units = int64_t(a.num_seqs) * a.num_kv_heads;
  const int bs = 1 << a.log2_bs;
  const int blocks = int((int64_t(a.max_context_len) + bs - 1) / bs);
  if (blocks > 8 * kSelMaxKeys)
    return fail(KVP_ERR_INVALID, "select_blocks: more than %d blocks per sequence", 8 * kSelMaxKeys);
  // one CTA holds every key, or each of eight its share
  const bool gather = blocks <= kSelMaxKeys;
  const int smem = gather ? (blocks > 0 ? blocks : 1) * 8 : kSelMaxKeys * 8;
  // more CTAs per row while the rows alone leave SMs idle and each still has 128
  // blocks (32 x 8 rows of 1,500 blocks: one CTA each 46 us, two 53, four 64)
  int ranks = gather ? 1 : 8;
  while (ranks < 8 && units * ranks < sm_count() && blocks >= 256 * ranks) ranks *= 2;
  if (head_dim == 64)
    return launch_clusters("select_blocks", kvp::dev::select_blocks_kernel<TQ, TB, 64, 8>, units,
                           ranks, 256, smem, kSelMaxKeys * 8, st, a);
  // one CTA per SM or fewer: twice the warps (8 rows of 8,192 blocks: 24.4 -> 20.9
  // us; 16 CTAs per row do not all fit the GPCs at once: 24.0); else two CTAs per SM, so that one may load while one selects
  return units * ranks <= sm_count() && blocks >= 256 * ranks
             ? launch_clusters("select_blocks", kvp::dev::select_blocks_kernel<TQ, TB, 128, 16>,
                               units, ranks, 512, smem, kSelMaxKeys * 8, st, a)
             : launch_clusters("select_blocks", kvp::dev::select_blocks_kernel<TQ, TB, 128, 8>,
                               units, ranks, 256, smem, kSelMaxKeys * 8, st, a);
}

template <typename T, bool FP8, int D, int NT>
int launch_sparse_nt(kvp::dev::sparse::SparseArgs a, cudaStream_t st) {
  using namespace kvp::dev::sparse;
  const int G = a.num_q_heads / a.num_kv_heads;
  a.head_tiles = (G + 8 * NT - 1) / (8 * NT);
  const int64_t units = int64_t(a.num_seqs) * a.num_kv_heads * a.head_tiles;
  if (units >= (int64_t(1) << 28))
    return fail(KVP_ERR_INVALID, "paged_attention_decode_sparse: batch too large");
  const int64_t tiles = ((int64_t(a.num_selected) << a.log2_bs) + 15) / 16;
  SparseMaps maps;
  const uint64_t rows = (uint64_t(a.num_blocks) * a.num_kv_heads) << a.log2_bs;
  const uint32_t box = a.log2_bs == 3 ? 8 : 16;
  const int32_t dtype = std::is_same<T, __half>::value ? KVP_F16 : KVP_BF16;
  for (int i = 0; i < 2; ++i) {
    CUtensorMap* map = i ? &maps.v : &maps.k;
    const void* base = i ? a.v_cache : a.k_cache;
    const int rc = FP8 ? make_map_u8(map, base, rows, box)
                       : D == 128 ? make_map_halves(map, base, dtype, rows, box)
                                  : make_map(map, base, dtype, rows, D, box);
    if (rc) return rc;
  }
  constexpr int warps = kSparseWarps<FP8, D, NT, false>;
  auto narrow = decode_sparse_kernel<T, FP8, D, NT, CTA>;
  auto wide = decode_sparse_kernel<T, FP8, D, NT, WIDE_CTA>;
  auto solo = decode_sparse_kernel<T, FP8, D, NT, SOLO>;
  constexpr int smem = kSmemBytes<false>, wide_smem = kSmemBytes<true>;
  a.num_units = uint32_t(units);
  // A warp per row where lists are short (128 KiB of keys and values) and rows many:
  // by the time of a start and a merge (about 4 us, of a lone warp 3) and of a tile
  // (1 us per warp), in rounds of what is on the GPU at once. 154 x 40 rows of 5 tiles
  // of 8 KiB 65 -> 38 us, 256 x 40 of up to 16 134 -> 104, 58 x 40 of up to 20 of 4 KiB
  // 42 -> 24; 64 x 40 rows of up to 32 of 8 KiB lose, 87 -> 93.
  const int64_t at_once = int64_t(sm_count()) * (NT == 1 && warps == 4 ? 3 : 2);
  const int64_t cta_us = (units + at_once - 1) / at_once * (4 * warps + tiles) / warps;
  const int64_t solo_us = (units + at_once * warps - 1) / (at_once * warps) * (3 + tiles);
  if (tiles * 32 * D * (FP8 ? 1 : 2) <= 128 * 1024 && solo_us < cta_us)
    return launch_clusters("paged_attention_decode_sparse", solo, (units + warps - 1) / warps, 1,
                           warps * 32, smem, smem, st, maps, a);
  // more CTAs per row while the rows alone leave SMs idle and each warp still has 2
  // tiles (256 rows of 4,096 tokens: one CTA each 93 us, two 99, four 105)
  int ranks = 1;
  while (ranks < 8 && units * ranks < sm_count() && tiles >= 4 * warps * ranks) ranks *= 2;
  if (units <= sm_count()) {
    // few rows: CTAs of twice the warps, as many per row as are on the GPU at once
    cudaError_t e = ensure_smem(wide, wide_smem);
    if (e != cudaSuccess) return cuda_fail(e, "paged_attention_decode_sparse");
    int r = 8;
    while (r > 1 && (tiles < 4 * warps * r || units > resident_clusters(wide, r, warps * 64, wide_smem)))
      --r;
    if (2 * r > ranks && tiles >= 4 * warps * r)
      return launch_clusters("paged_attention_decode_sparse", wide, units, r, warps * 64, wide_smem,
                             wide_smem, st, maps, a);
  }
  return launch_clusters("paged_attention_decode_sparse", narrow, units, ranks, warps * 32, smem,
                         smem, st, maps, a);
}

template <typename T, bool FP8, int D>
int launch_sparse(const kvp::dev::sparse::SparseArgs& a, cudaStream_t st) {
  // groups of more than 8 query heads take two column tiles per pass over the blocks
  return a.num_q_heads / a.num_kv_heads <= 8 ? launch_sparse_nt<T, FP8, D, 1>(a, st)
                                             : launch_sparse_nt<T, FP8, D, 2>(a, st);
}

}  // namespace

extern "C" {

int rope_reshape_and_cache(const void* q, const void* k_new, const void* v_new, void* q_out,
                           int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           int64_t q_out_stride, const float* cos_sin, const int64_t* positions,
                           int64_t max_positions, int32_t rot_dim, int32_t interleaved,
                           void* k_cache, void* v_cache, const int64_t* slot_mapping,
                           const float* k_scale, const float* v_scale, int32_t num_tokens,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t block_size, int32_t num_blocks, int32_t dtype,
                           int32_t cache_dtype, kvp_stream_t stream) {
  const char* fn = "rope_reshape_and_cache";
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      block_size <= 0 || max_positions <= 0)
    return fail(KVP_ERR_INVALID, "%s: bad sizes", fn);
  if (num_q_heads > (1 << 20) || num_kv_heads > (1 << 20))
    return fail(KVP_ERR_INVALID, "%s: too many heads", fn);
  if (dtype != KVP_F16 && dtype != KVP_BF16) return fail(KVP_ERR_INVALID, "%s: bad dtype", fn);
  if (cache_dtype != dtype && cache_dtype != KVP_FP8_E4M3)
    return fail(KVP_ERR_INVALID, "%s: the cache is of the queries' type or E4M3", fn);
  const int items = log2_items(head_dim), lbs = ilog2(block_size);
  if (items < 0 || head_dim > 1024 || lbs < 0)
    return fail(KVP_ERR_INVALID, "%s: head_dim / 16 (up to 64) and block_size must be powers of two", fn);
  if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 16)
    return fail(KVP_ERR_INVALID, "%s: rot_dim must be a multiple of 16 in [16, head_dim]", fn);
  if (num_tokens == 0) return KVP_OK;
  const bool fp8 = cache_dtype == KVP_FP8_E4M3;
  if (!q || !k_new || !v_new || !q_out || !cos_sin || !positions || !k_cache || !v_cache ||
      !slot_mapping || (fp8 && (!k_scale || !v_scale)))
    return fail(KVP_ERR_INVALID, "%s: NULL pointer", fn);
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16) ||
      !aligned(cos_sin, 16) || !aligned(positions, 8) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 8) ||
      (fp8 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return fail(KVP_ERR_INVALID, "%s: misaligned pointer", fn);
  const int64_t strides[] = {q_stride, k_stride, v_stride, q_out_stride};
  for (int64_t x : strides)
    if (x < 0 || x % 8 || x > (int64_t(1) << 31))
      return fail(KVP_ERR_INVALID, "%s: token strides must be multiples of 8 elements", fn);
  const int64_t q_row = int64_t(num_q_heads) * head_dim, kv_row = int64_t(num_kv_heads) * head_dim;
  if (num_tokens > 1 && q_out_stride < q_row)
    return fail(KVP_ERR_INVALID, "%s: the rows of q_out overlap", fn);
  const bool in_place = q_out == q && (q_out_stride == q_stride || num_tokens == 1);
  if ((!in_place && rows_overlap(q_out, q_out_stride, q_row, q, q_stride, q_row, num_tokens)) ||
      rows_overlap(q_out, q_out_stride, q_row, k_new, k_stride, kv_row, num_tokens) ||
      rows_overlap(q_out, q_out_stride, q_row, v_new, v_stride, kv_row, num_tokens))
    return fail(KVP_ERR_INVALID, "%s: q_out overlaps an input and is not q itself", fn);
  kvp::dev::RopeArgs a{};
  a.q = q;
  a.k = k_new;
  a.v = v_new;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.max_positions = max_positions;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.slots = slot_mapping;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.num_slots = int64_t(num_blocks) * block_size;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.rot_dim = rot_dim;
  a.log2_ipr = items;
  a.log2_bs = lbs;
  // threads per token: a CTA's, or as many as its few rows need
  const int rows = num_q_heads + 2 * num_kv_heads;
  a.num_tokens = num_tokens;
  a.log2_tpt = items;
  while (a.log2_tpt < kvp::dev::kRopeLog2Threads && (1 << (a.log2_tpt - items)) < rows) ++a.log2_tpt;
  // many tokens, 16-bit pools: fewer threads per token where that leaves fewer of them
  // without a row in the last pass (25,000 tokens of 8 + 1 heads of 128: 35 -> 27 us). Into
  // E4M3 the packed kernel has 10 CTAs per SM instead of 12, which costs more than it gains
  // where many rows are codes (21,780 tokens of 8 + 8 heads 51 -> 55; of 8 + 1 it would
  // gain, 38 -> 32)
  auto idle = [&](int log2_threads) {
    const int per = 1 << (log2_threads - items);
    return double((rows + per - 1) / per * per) / rows;
  };
  if (!fp8 && int64_t(num_tokens) >= int64_t(32) * sm_count())
    for (int l = a.log2_tpt - 1; l >= items && l >= 5; --l)
      if (idle(l) < idle(a.log2_tpt) - 0.1) a.log2_tpt = l;
  // few tokens: a token's rows over several CTAs, one pass of each; many: one pass after another
  const int pass = (1 << a.log2_tpt) >> items, tokens = kvp::dev::kRopeThreads >> a.log2_tpt;
  const int64_t ctas = (int64_t(num_tokens) + tokens - 1) / tokens;
  int64_t slices = (rows + pass - 1) / pass;
  const int64_t wanted = (int64_t(8) * sm_count() + ctas - 1) / ctas;
  if (slices > wanted) slices = wanted;
  if (slices > 65535) slices = 65535;
  a.rows_per_cta = int(((rows + slices - 1) / slices + pass - 1) / pass * pass);
  const dim3 grid(unsigned(ctas), unsigned((rows + a.rows_per_cta - 1) / a.rows_per_cta));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fp8)
    return dtype == KVP_F16 ? launch_rope<__half, true>(a, grid, interleaved != 0, st)
                            : launch_rope<__nv_bfloat16, true>(a, grid, interleaved != 0, st);
  return dtype == KVP_F16 ? launch_rope<__half, false>(a, grid, interleaved != 0, st)
                          : launch_rope<__nv_bfloat16, false>(a, grid, interleaved != 0, st);
}

int update_key_bounds(const void* k_cache, void* key_bounds, const int32_t* block_tables,
                      const int32_t* context_lens, const int32_t* new_tokens, int32_t num_seqs,
                      int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                      int32_t num_blocks, int32_t max_blocks_per_seq, int32_t max_context_len,
                      int32_t max_new_tokens, int32_t cache_dtype, kvp_stream_t stream) {
  const char* fn = "update_key_bounds";
  if (num_seqs < 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 ||
      max_context_len < 0 || max_new_tokens < 0)
    return fail(KVP_ERR_INVALID, "%s: bad sizes", fn);
  if (block_size != 8 && block_size != 16 && block_size != 32)
    return fail(KVP_ERR_INVALID, "%s: block_size must be 8, 16 or 32", fn);
  if (cache_dtype != KVP_F16 && cache_dtype != KVP_BF16 && cache_dtype != KVP_FP8_E4M3)
    return fail(KVP_ERR_INVALID, "%s: bad dtype", fn);
  if (head_dim != 128 && (head_dim != 64 || cache_dtype == KVP_FP8_E4M3))
    return fail(KVP_ERR_INVALID, "%s: head_dim must be 64 or 128 (E4M3: 128)", fn);
  if (int64_t(max_context_len) > int64_t(max_blocks_per_seq) * block_size)
    return fail(KVP_ERR_INVALID, "%s: max_context_len > max_blocks_per_seq * block_size", fn);
  if (num_seqs == 0 || max_context_len == 0 || (new_tokens && max_new_tokens == 0)) return KVP_OK;
  if (!k_cache || !key_bounds || !block_tables || !context_lens)
    return fail(KVP_ERR_INVALID, "%s: NULL pointer", fn);
  if (!aligned(k_cache, 16) || !aligned(key_bounds, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(new_tokens, 4))
    return fail(KVP_ERR_INVALID, "%s: misaligned pointer", fn);
  kvp::dev::BoundsArgs a{};
  a.k_cache = k_cache;
  a.bounds = key_bounds;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.new_tokens = new_tokens;
  a.num_seqs = num_seqs;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_context_len = max_context_len;
  a.max_new_tokens = new_tokens ? max_new_tokens : max_context_len;
  a.log2_bs = ilog2(block_size);
  const int64_t all = (int64_t(max_context_len) + block_size - 1) / block_size;
  // n neighbouring tokens lie in (n + 2 bs - 2) / bs blocks at most
  const int64_t touched = (int64_t(a.max_new_tokens) + 2 * block_size - 2) / block_size;
  a.blocks_per_seq = int32_t(touched < all ? touched : all);
  // several heads per warp once there are more tiles than 64 per SM
  const int64_t tiles = int64_t(num_seqs) * a.blocks_per_seq * num_kv_heads;
  const int64_t hpw = tiles / (int64_t(sm_count()) * 64);
  a.heads_per_warp = int32_t(hpw < 1 ? 1 : hpw < num_kv_heads ? hpw : num_kv_heads);
  a.head_groups = (num_kv_heads + a.heads_per_warp - 1) / a.heads_per_warp;
  const int64_t warps = int64_t(num_seqs) * a.blocks_per_seq * a.head_groups;
  if (warps >= (int64_t(1) << 31) || int64_t(a.blocks_per_seq) * num_kv_heads >= (int64_t(1) << 31))
    return fail(KVP_ERR_INVALID, "%s: too many blocks in one call", fn);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache_dtype == KVP_FP8_E4M3) return launch_bounds<__half, true, 128>(a, warps, st);
  if (head_dim == 128)
    return cache_dtype == KVP_F16 ? launch_bounds<__half, false, 128>(a, warps, st)
                                  : launch_bounds<__nv_bfloat16, false, 128>(a, warps, st);
  return cache_dtype == KVP_F16 ? launch_bounds<__half, false, 64>(a, warps, st)
                                : launch_bounds<__nv_bfloat16, false, 64>(a, warps, st);
}

int select_blocks(const void* q, const void* key_bounds, const int32_t* block_tables,
                  const int32_t* context_lens, int32_t* selected, int32_t num_seqs,
                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                  int32_t num_blocks, int32_t max_blocks_per_seq, int32_t max_context_len,
                  int32_t num_selected, int32_t num_sink, int32_t num_recent, int32_t dtype,
                  int32_t cache_dtype, kvp_stream_t stream) try {
  const char* fn = "select_blocks";
  int rc = check_rows(fn, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                      max_blocks_per_seq, max_context_len, num_selected, dtype, cache_dtype);
  if (rc) return rc;
  if (num_sink < 0 || num_recent < 0 || int64_t(num_sink) + num_recent > num_selected)
    return fail(KVP_ERR_INVALID, "%s: num_sink + num_recent must be in [0, num_selected]", fn);
  if (num_seqs == 0) return KVP_OK;
  if (!q || !key_bounds || !block_tables || !context_lens || !selected)
    return fail(KVP_ERR_INVALID, "%s: NULL pointer", fn);
  if (!aligned(q, 16) || !aligned(key_bounds, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(selected, 4))
    return fail(KVP_ERR_INVALID, "%s: misaligned pointer", fn);
  kvp::dev::SelectArgs a{};
  a.q = q;
  a.bounds = key_bounds;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.out = selected;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_context_len = max_context_len;
  a.log2_bs = ilog2(block_size);
  a.keep = num_selected;
  a.sink = num_sink;
  a.recent = num_recent;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == KVP_F16) return launch_select<__half, __half>(a, head_dim, st);
  return cache_dtype == KVP_BF16 ? launch_select<__nv_bfloat16, __nv_bfloat16>(a, head_dim, st)
                                 : launch_select<__nv_bfloat16, __half>(a, head_dim, st);
} catch (...) {  // the launch helpers' records take host memory
  return fail(KVP_ERR_OOM, "select_blocks: no host memory");
}

int paged_attention_decode_sparse(const void* q, const void* k_cache, const void* v_cache,
                                  const float* k_scale, const float* v_scale,
                                  const int32_t* block_tables, const int32_t* context_lens,
                                  const int32_t* selected, int32_t num_seqs, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                  int32_t num_blocks, int32_t max_blocks_per_seq,
                                  int32_t max_context_len, int32_t num_selected, float scale,
                                  void* out, int32_t dtype, int32_t cache_dtype,
                                  kvp_stream_t stream) try {
  const char* fn = "paged_attention_decode_sparse";
  int rc = check_rows(fn, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                      max_blocks_per_seq, max_context_len, num_selected, dtype, cache_dtype);
  if (rc) return rc;
  if (int64_t(num_blocks) * num_kv_heads * block_size >= (int64_t(1) << 31))
    return fail(KVP_ERR_INVALID, "%s: pool too large for 32-bit row coordinates", fn);
  if (!std::isfinite(scale)) return fail(KVP_ERR_INVALID, "%s: scale not finite", fn);
  if (num_seqs == 0) return KVP_OK;
  const bool fp8 = cache_dtype == KVP_FP8_E4M3;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !selected || !out ||
      (fp8 && (!k_scale || !v_scale)))
    return fail(KVP_ERR_INVALID, "%s: NULL pointer", fn);
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(selected, 4) ||
      (fp8 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return fail(KVP_ERR_INVALID, "%s: misaligned pointer", fn);
  kvp::dev::sparse::SparseArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.selected = selected;
  a.out = out;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_context_len = max_context_len;
  a.log2_bs = ilog2(block_size);
  a.num_selected = num_selected;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fp8)
    return dtype == KVP_F16 ? launch_sparse<__half, true, 128>(a, st)
                            : launch_sparse<__nv_bfloat16, true, 128>(a, st);
  if (head_dim == 128)
    return dtype == KVP_F16 ? launch_sparse<__half, false, 128>(a, st)
                            : launch_sparse<__nv_bfloat16, false, 128>(a, st);
  return dtype == KVP_F16 ? launch_sparse<__half, false, 64>(a, st)
                          : launch_sparse<__nv_bfloat16, false, 64>(a, st);
} catch (...) {  // the launch helpers' records take host memory
  return fail(KVP_ERR_OOM, "paged_attention_decode_sparse: no host memory");
}

}  // extern "C"
