// cache_api.cu -- the C entry points around the decode that write new tokens
// and choose what the sparse attention reads: rotary positions, appends to the
// paged caches, index queries, the index score and the selection
// (include/mla.h). Every argument check happens before anything is enqueued.
#include "checks.h"
#include "index_score.cuh"
#include "params.h"
#include "rows.cuh"
#include "select.cuh"

using namespace mla;

namespace {

// Rows of (token, head) from which a thread of the rotation takes four heads of
// a token, which share its table row (256 x 128 rows 2.5 us
// against 2.9 with one, 4095 x 128 22.9 against 29.9; 64 x 128, where one head a
// thread fills the card better, 2.4 against 1.8).
constexpr int64_t kManyRows = 32768;
// tokens of a row and columns written: room for the kernels' strides in 31 bits
constexpr int64_t kMaxColumns = kMaxRows - 65536;

}  // namespace

extern "C" {

mla_status mla_append_kv(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t r_stride, int dtype,
                         const int32_t* slots, const int32_t* positions, const float* rope_table,
                         int64_t max_positions, int rope_style, int64_t n, void* kvcache, int64_t num_blocks,
                         int page_block, int kv_format, uint32_t* status, void* stream) {
  if (n < 0 || n >= kMaxRows || max_positions <= 0 || !cache_ok(num_blocks, page_block)) return MLA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || kv_format < MLA_KV_16BIT || kv_format > MLA_KV_FP4_288) return MLA_ERR_INVALID_ARG;
  if (rope_style != MLA_ROPE_PAIRS && rope_style != MLA_ROPE_HALVES) return MLA_ERR_INVALID_ARG;
  const int latent = kv_format >= MLA_KV_FP8_528 ? kDV41 - rows::kRope : kDV;
  if (!stride_ok(c_stride, latent, n) || !stride_ok(r_stride, rows::kRope, n)) return MLA_ERR_INVALID_ARG;
  if (status && !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (kv_format && dtype != MLA_DTYPE_BF16) return MLA_ERR_UNSUPPORTED;  // quantised rows pair with bf16
  if (n == 0) return MLA_OK;
  if (!c_kv || !k_rope || !slots || !kvcache || !aligned(c_kv, 16) || !aligned(k_rope, 16) || !aligned(slots, 4) ||
      !aligned(kvcache, 16))
    return MLA_ERR_INVALID_ARG;
  rows::AppendParams p{c_kv, k_rope, c_stride, r_stride, slots,
                       {positions, rope_table, max_positions, rope_style == MLA_ROPE_HALVES, status},
                       n, static_cast<uint8_t*>(kvcache), num_blocks * kTile};
  if (const mla_status v = check_positions(p.pos)) return v;
  static constexpr int64_t row_bytes[4] = {kDK * 2, kRowBytesFp8, kRowBytesFp8_528, kRowBytesFp4_288};
  if (!apart({{kvcache, p.num_rows * row_bytes[kv_format]}, status_span(status)},
             {{c_kv, 2 * ((n - 1) * c_stride + latent)}, {k_rope, 2 * ((n - 1) * r_stride + rows::kRope)},
              int32_span(slots, n), int32_span(positions, n), table_span(p.pos)}))
    return MLA_ERR_INVALID_ARG;
  const dim3 grid((unsigned)((n + rows::kAppendWarps - 1) / rows::kAppendWarps));
  const int threads = 32 * rows::kAppendWarps;
  if (kv_format == MLA_KV_FP8_656)
    return launch(rows::mla_append_kv_kernel<false, MLA_KV_FP8_656>, grid, threads, 0, stream, p);
  if (kv_format == MLA_KV_FP8_528)
    return launch(rows::mla_append_kv_kernel<false, MLA_KV_FP8_528>, grid, threads, 0, stream, p);
  if (kv_format == MLA_KV_FP4_288)
    return launch(rows::mla_append_kv_kernel<false, MLA_KV_FP4_288>, grid, threads, 0, stream, p);
  if (dtype == MLA_DTYPE_FP16)
    return launch(rows::mla_append_kv_kernel<true, MLA_KV_16BIT>, grid, threads, 0, stream, p);
  return launch(rows::mla_append_kv_kernel<false, MLA_KV_16BIT>, grid, threads, 0, stream, p);
}

mla_status mla_rotate_q(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
                        int64_t out_token_stride, int64_t out_head_stride, int dtype, const int32_t* positions,
                        const float* rope_table, int64_t max_positions, int rope_style, int64_t tokens, int heads,
                        uint32_t* status, void* stream) {
  if (tokens < 0 || heads < 1 || tokens >= kMaxRows / heads || max_positions <= 0) return MLA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (rope_style != MLA_ROPE_PAIRS && rope_style != MLA_ROPE_HALVES)) return MLA_ERR_INVALID_ARG;
  const int64_t xt = x_token_stride, xh = x_head_stride, ot = out_token_stride, oh = out_head_stride, w = rows::kRope;
  if (!stride_ok(xt, 0, tokens) || !stride_ok(xh, 0, heads) || !stride_ok(ot, w, tokens) || !stride_ok(oh, w, heads))
    return MLA_ERR_INVALID_ARG;
  if (status && !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (tokens == 0) return MLA_OK;
  if (!x || !out || !aligned(x, 16) || !aligned(out, 16)) return MLA_ERR_INVALID_ARG;
  // rows of the output must not overlap one another
  if (tokens > 1 && heads > 1 && ot < (heads - 1) * oh + w && oh < (tokens - 1) * ot + w) return MLA_ERR_INVALID_ARG;
  // in place (the same rows), between the rows of x, or apart
  const intptr_t xb = reinterpret_cast<intptr_t>(x), ob = reinterpret_cast<intptr_t>(out);
  const int64_t xspan = 2 * ((tokens - 1) * xt + (heads - 1) * xh + w), ospan = 2 * ((tokens - 1) * ot + (heads - 1) * oh + w);
  if (xb < ob + ospan && ob < xb + xspan) {
    const bool same = (xt == ot || tokens == 1) && (xh == oh || heads == 1);
    const bool heads_inside = heads > 1 && (oh < ot || tokens == 1);
    if (!same || (xb != ob && (heads_inside ? rows_meet((ob - xb) / 2, ot, tokens, oh, heads, w)
                                            : rows_meet((ob - xb) / 2, oh, heads, ot, tokens, w))))
      return MLA_ERR_INVALID_ARG;
  }
  rows::RotateParams p{static_cast<const uint16_t*>(x), static_cast<uint16_t*>(out), xt, xh, ot, oh,
                       {positions, rope_table, max_positions, rope_style == MLA_ROPE_HALVES, status},
                       tokens, heads, 0};
  if (const mla_status v = check_positions(p.pos)) return v;
  if (!apart({{out, ospan}, status_span(status)}, {int32_span(positions, tokens), table_span(p.pos)}) ||
      status_span(status).meets({x, xspan}))
    return MLA_ERR_INVALID_ARG;
  constexpr int kU = 4;
  const bool many = tokens * heads >= kManyRows;
  p.heads_per_slot = (uint32_t)(many ? (heads + kU - 1) / kU : heads);
  const int64_t items = tokens * p.heads_per_slot * 4;
  const dim3 grid((unsigned)((items + rows::kRotateThreads - 1) / rows::kRotateThreads));
  if (dtype == MLA_DTYPE_FP16)
    return many ? launch(rows::mla_rotate_kernel<true, kU>, grid, rows::kRotateThreads, 0, stream, p)
                : launch(rows::mla_rotate_kernel<true, 1>, grid, rows::kRotateThreads, 0, stream, p);
  return many ? launch(rows::mla_rotate_kernel<false, kU>, grid, rows::kRotateThreads, 0, stream, p)
              : launch(rows::mla_rotate_kernel<false, 1>, grid, rows::kRotateThreads, 0, stream, p);
}

mla_status mla_append_index_k(const void* k, int64_t k_stride, int dtype, const int32_t* slots,
                              const int32_t* positions, const float* rope_table, int64_t max_positions,
                              int rope_style, int64_t n, void* index_cache, int64_t num_blocks, int page_block,
                              int index_format, uint32_t* status, void* stream) {
  if (n < 0 || n >= kMaxRows || max_positions <= 0 || !cache_ok(num_blocks, page_block)) return MLA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (index_format != MLA_INDEX_16BIT && index_format != MLA_INDEX_FP8)) return MLA_ERR_INVALID_ARG;
  if (rope_style != MLA_ROPE_PAIRS && rope_style != MLA_ROPE_HALVES) return MLA_ERR_INVALID_ARG;
  if (!stride_ok(k_stride, rows::kIndexDim, n) || (status && !aligned(status, 4))) return MLA_ERR_INVALID_ARG;
  if (n == 0) return MLA_OK;
  if (!k || !slots || !index_cache || !aligned(k, 16) || !aligned(slots, 4) || !aligned(index_cache, 16))
    return MLA_ERR_INVALID_ARG;
  rows::IndexRowParams p{static_cast<const uint16_t*>(k), k_stride, 0, slots, nullptr,
                         {positions, rope_table, max_positions, rope_style == MLA_ROPE_HALVES, status},
                         n, 1, 1, 1, static_cast<uint8_t*>(index_cache), nullptr, num_blocks * kTile};
  if (const mla_status v = check_positions(p.pos)) return v;
  const int64_t page = index_format == MLA_INDEX_FP8 ? rows::kIndexPageFp8 : kTile * 2 * rows::kIndexDim;
  if (!apart({{index_cache, num_blocks * page}, status_span(status)},
             {{k, 2 * ((n - 1) * k_stride + rows::kIndexDim)}, int32_span(slots, n), int32_span(positions, n), table_span(p.pos)}))
    return MLA_ERR_INVALID_ARG;
  const int per = rows::kIndexGroups;
  const dim3 grid((unsigned)((n + per - 1) / per));
  const bool fp16 = dtype == MLA_DTYPE_FP16;
  if (index_format == MLA_INDEX_FP8)
    return fp16 ? launch(rows::mla_index_rows_kernel<true, true, true>, grid, rows::kIndexThreads, 0, stream, p)
                : launch(rows::mla_index_rows_kernel<false, true, true>, grid, rows::kIndexThreads, 0, stream, p);
  return fp16 ? launch(rows::mla_index_rows_kernel<true, false, true>, grid, rows::kIndexThreads, 0, stream, p)
              : launch(rows::mla_index_rows_kernel<false, false, true>, grid, rows::kIndexThreads, 0, stream, p);
}

mla_status mla_quantize_index_q(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
                                const float* weights, const int32_t* positions, const float* rope_table,
                                int64_t max_positions, int rope_style, int64_t tokens, int heads, uint8_t* q_out,
                                float* weights_out, uint32_t* status, void* stream) {
  if (tokens < 0 || heads < 1 || tokens >= kMaxRows / heads || max_positions <= 0) return MLA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (rope_style != MLA_ROPE_PAIRS && rope_style != MLA_ROPE_HALVES)) return MLA_ERR_INVALID_ARG;
  if (!stride_ok(q_token_stride, 0, tokens) || !stride_ok(q_head_stride, 0, heads) || (status && !aligned(status, 4)))
    return MLA_ERR_INVALID_ARG;
  if (tokens == 0) return MLA_OK;
  if (!q || !weights || !q_out || !weights_out || !aligned(q, 16) || !aligned(weights, 4) || !aligned(q_out, 16) ||
      !aligned(weights_out, 4))
    return MLA_ERR_INVALID_ARG;
  rows::IndexRowParams p{static_cast<const uint16_t*>(q), q_token_stride, q_head_stride, nullptr, weights,
                         {positions, rope_table, max_positions, rope_style == MLA_ROPE_HALVES, status},
                         tokens, heads, heads, 1, q_out, weights_out, 0};
  if (const mla_status v = check_positions(p.pos)) return v;
  const Span in{q, 2 * ((tokens - 1) * q_token_stride + (heads - 1) * q_head_stride + rows::kIndexDim)},
      w_in{weights, 4 * tokens * heads}, w_to{weights_out, 4 * tokens * heads}, codes{q_out, rows::kIndexDim * tokens * heads},
      flags = status_span(status);
  // the weights may be scaled in place
  if (!apart({codes, w_to, flags}, {in, int32_span(positions, tokens), table_span(p.pos)}) || codes.meets(w_in) || flags.meets(w_in) ||
      (weights != weights_out && w_in.meets(w_to)))
    return MLA_ERR_INVALID_ARG;
  // up to eight heads to a lane group, as long as that leaves kFewGroups of them: half the card's lanes. Measured with
  // 64 heads (GB300): 512 tokens 4.0 us (two heads a group), 5.5 with eight; 4096 tokens 20.6 with eight, 24.5 with two
  constexpr int64_t kFewGroups = 16384;
  const int64_t steps = tokens * heads / kFewGroups;
  p.steps = (int)(steps < 1 ? 1 : steps > 8 ? 8 : steps);
  p.slots_per_token = (heads + p.steps - 1) / p.steps;
  const int64_t groups = tokens * p.slots_per_token;
  const int per = rows::kIndexGroups;
  const dim3 grid((unsigned)((groups + per - 1) / per));
  return dtype == MLA_DTYPE_FP16
             ? launch(rows::mla_index_rows_kernel<true, true, false>, grid, rows::kIndexThreads, 0, stream, p)
             : launch(rows::mla_index_rows_kernel<false, true, false>, grid, rows::kIndexThreads, 0, stream, p);
}

}  // extern "C"

namespace {

// rows of 128-byte chunks {x, y, z} with a 128-byte-swizzled box {128 B, by, bz}
bool make_map_rows(CUtensorMap* m, const void* base, bool fp8, CUtensorMapDataType dt, uint64_t y, uint64_t z,
                   uint64_t y_bytes, uint64_t z_bytes, uint32_t by, uint32_t bz) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)score::kDim, y, z};
  cuuint64_t strides[2] = {y_bytes, z_bytes};
  cuuint32_t box[3] = {fp8 ? 128u : 64u, by, bz};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kType, int kHp, bool kPages>
mla_status launch_score(int dev, int grid, uint32_t smem, void* stream, const CUtensorMap& tq, const CUtensorMap& tk,
                        const score::ScoreParams& p) {
  static std::atomic<bool> set[kMaxDevices];
  auto kernel = score::mla_index_score_kernel<kType, kHp, kPages>;
  if (!set[dev].load(std::memory_order_relaxed)) {
    MLA_CUDA(set_smem(kernel, 232448));
    set[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(score::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  MLA_CUDA(cudaLaunchKernelEx(&cfg, kernel, tq, tk, p));
  return MLA_OK;
}
// `most`: columns of the longest possible row
template <bool kPages>
mla_status launch_select(select::SelectParams p, int64_t most, int sms, void* stream) {
  const int64_t rows = (int64_t)p.batch * p.s_q;
  constexpr int kWide = 32 * select::kMaxWarps;
  auto blocks = [&](int keys) {  // of a row, at `keys` scores per thread
    int c = 1;
    while (c < select::kMaxCluster && (int64_t)c * kWide * keys < most) c *= 2;
    return c;
  };
  // One block a row where it holds the row, with the fewest scores per thread
  // (32 rows of 12288: 5.5 us in one block, 7.2 in clusters of 2 with 16 scores a
  // thread; 64 rows of 8192: 4.8 with 16, 5.7 with 32). Longer rows go to
  // clusters, of 16 scores per thread while all of them run at once (8 rows of
  // 32768: 8.0 us, 8.8 with 32), else of 32.
  int keys = 0, cluster = select::kMaxCluster;
  for (const int k : {4, 16, 32}) {
    const int c = blocks(k);
    const bool holds = (int64_t)c * kWide * k >= most, at_once = rows * c <= 2 * sms;
    if (!holds || (c > 1 && (k == 4 || most <= select::kBlockKeys || (k == 16 && !at_once)))) continue;
    keys = k;
    cluster = c;
    break;
  }
  while (1 << p.cluster_log2 < cluster) ++p.cluster_log2;
  // More rows than SMs: narrow blocks with more scores per thread, since a warp's
  // scans, barriers and start cost as much as its sweeps (4096 rows of up to 2048
  // scores, topk an eighth: 25 us, 65 in wide blocks; of 8192: 54, 88; 256 rows of
  // 2048 4.6, 5.2, but 128 rows 4.3, 4.2). Rows beyond 8192 stay wide: 64 scores a
  // thread halve the warps in flight (16384: 121 us, 113).
  int threads = kWide;
  const bool many = rows > sms && most <= select::kBlockKeys / 2;
  auto kernel = keys == 4    ? select::mla_select_topk_kernel<kPages, 4, 16>
                : keys == 16 ? select::mla_select_topk_kernel<kPages, 16, 16>
                : keys       ? select::mla_select_topk_kernel<kPages, 32, 16>
                             : select::mla_select_topk_kernel<kPages, 0, 16>;
  if (many) {
    threads = most <= 4096 ? 128 : 256;
    kernel = most <= 2048   ? select::mla_select_topk_kernel<kPages, 16, 4>
             : most <= 4096 ? select::mla_select_topk_kernel<kPages, 32, 4>
                            : select::mla_select_topk_kernel<kPages, 32, 8>;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cluster), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  MLA_CUDA(cudaLaunchKernelEx(&cfg, kernel, p));
  return MLA_OK;
}

template <int kType, int kHp, typename... A>
mla_status launch_score_block(bool pages, A&&... a) {
  return pages ? launch_score<kType, kHp, true>(a...) : launch_score<kType, kHp, false>(a...);
}
template <int kType, typename... A>
mla_status launch_score_heads(int hp, A&&... a) {
  if (hp == 16) return launch_score_block<kType, 16>(a...);
  if (hp == 32) return launch_score_block<kType, 32>(a...);
  return launch_score_block<kType, 64>(a...);
}

}  // namespace

extern "C" {

mla_status mla_index_score(const void* q, int q_dtype, const float* weights, const void* index_cache,
                           int index_format, int64_t num_blocks, int page_block, const int32_t* block_table,
                           int max_blocks, const int32_t* cache_seqlens, int batch, int s_q, int heads, int causal,
                           int block, float* scores, int64_t score_stride, int width, uint32_t* status,
                           void* stream) {
  if (index_format != MLA_INDEX_16BIT && index_format != MLA_INDEX_FP8) return MLA_ERR_INVALID_ARG;
  const bool fp8 = index_format == MLA_INDEX_FP8, pages = block == kTile;
  if (!fp8 && !dtype_ok(q_dtype)) return MLA_ERR_INVALID_ARG;
  if (!cache_ok(num_blocks, page_block) || max_blocks <= 0 || batch <= 0 || s_q <= 0 || width <= 0 ||
      score_stride < width || (block != 1 && !pages))
    return MLA_ERR_INVALID_ARG;
  if (heads < 1) return MLA_ERR_INVALID_ARG;
  if (heads > 64) return MLA_ERR_UNSUPPORTED;
  if ((int64_t)batch * s_q >= kMaxRows / heads || !in_memory(score_stride, (int64_t)batch * s_q) || !in_memory(max_blocks, batch))
    return MLA_ERR_INVALID_ARG;
  if (!q || !weights || !index_cache || !block_table || !cache_seqlens || !scores || !aligned(q, 16) ||
      !aligned(weights, 4) || !aligned(index_cache, 16) || !aligned(block_table, 4) || !aligned(cache_seqlens, 4) ||
      !aligned(scores, 4) || (status && !aligned(status, 4)))
    return MLA_ERR_INVALID_ARG;
  const int64_t columns = (int64_t)width * (pages ? kTile : 1), reach = (int64_t)max_blocks * kTile;
  const int64_t cover = columns < reach ? columns : reach;
  if (cover > kMaxColumns || width > kMaxColumns) return MLA_ERR_INVALID_ARG;

  score::ScoreParams p{};
  const int hp = heads <= 16 ? 16 : heads <= 32 ? 32 : 64;
  const int most = score::kMaxN / hp, all = (s_q + most - 1) / most;  // groups of a request
  p.nq = (s_q + all - 1) / all;
  p.groups = all > 1 ? 2 : 1;
  p.units = (s_q + p.nq * p.groups - 1) / (p.nq * p.groups);
  const int64_t pairs = (int64_t)batch * p.units * ((cover + score::kTokens - 1) / score::kTokens);
  if (pairs >= kMaxRows) return MLA_ERR_UNSUPPORTED;
  const int64_t queries = (int64_t)batch * s_q, row_bytes = fp8 ? 128 : 256;
  if (!apart({{scores, 4 * ((queries - 1) * score_stride + width)}, status_span(status)},
             {{q, queries * heads * row_bytes}, {weights, 4 * queries * heads}, {block_table, 4 * (int64_t)batch * max_blocks},
              {cache_seqlens, 4 * (int64_t)batch}, {index_cache, num_blocks * (fp8 ? rows::kIndexPageFp8 : kTile * 256)}}))
    return MLA_ERR_INVALID_ARG;
  const uint32_t q_bytes = (uint32_t)(p.groups * p.nq * hp) * (fp8 ? 128u : 256u);
  uint32_t ring = (232448u - score::smem_bytes(q_bytes, 0)) / score::kUnit;
  ring = ring > score::kMaxRing ? score::kMaxRing : ring;
  p.ring = (int)ring;
  p.weights = weights;
  p.cache = static_cast<const uint8_t*>(index_cache);
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.scores = scores;
  p.stride = score_stride;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks;
  p.batch = batch;
  p.s_q = s_q;
  p.heads = heads;
  p.causal = causal ? 1 : 0;
  p.cover = (int)cover;
  p.width = width;
  p.status = status;
  p.stall_cycles = g_test_stall.load(std::memory_order_relaxed);

  int dev = 0, sms = 0;
  if (const mla_status v = sm_count(&dev, &sms)) return v;
  const int grid = (int)(pairs < sms ? pairs : sms);
  const CUtensorMapDataType dt = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : q_dtype == MLA_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t row = fp8 ? 128 : 256, page = fp8 ? rows::kIndexPageFp8 : kTile * 256;
  CUtensorMap tq, tk;
  if (!make_map_rows(&tq, q, fp8, dt, heads, (uint64_t)batch * s_q, row, row * heads, hp, p.nq) ||
      !make_map_rows(&tk, index_cache, fp8, dt, kTile, num_blocks, row, page, kTile, 1))
    return MLA_ERR_CUDA;
  const uint32_t smem = score::smem_bytes(q_bytes, ring);
  if (fp8) return launch_score_heads<score::K_FP8>(hp, pages, dev, grid, smem, stream, tq, tk, p);
  if (q_dtype == MLA_DTYPE_FP16)
    return launch_score_heads<score::K_FP16>(hp, pages, dev, grid, smem, stream, tq, tk, p);
  return launch_score_heads<score::K_BF16>(hp, pages, dev, grid, smem, stream, tq, tk, p);
}

mla_status mla_select_topk(const float* scores, int64_t score_stride, int width, const int32_t* cache_seqlens,
                           int batch, int s_q, int causal, int block, int topk, const int32_t* block_table,
                           int max_blocks, int64_t num_blocks, int page_block, int32_t* indices, int32_t* lens,
                           uint32_t* status, void* stream) {
  const bool pages = block == kTile;
  if (!cache_ok(num_blocks, page_block) || max_blocks <= 0 || batch <= 0 || s_q <= 0 || width <= 0 || topk <= 0 ||
      score_stride < width || (block != 1 && !pages))
    return MLA_ERR_INVALID_ARG;
  if ((int64_t)batch * s_q >= kMaxRows || !in_memory(score_stride, (int64_t)batch * s_q) || !in_memory(max_blocks, batch))
    return MLA_ERR_INVALID_ARG;
  const int64_t columns = (int64_t)width * (pages ? kTile : 1), reach = (int64_t)max_blocks * kTile;
  if ((columns < reach ? columns : reach) > kMaxColumns || topk > kMaxColumns) return MLA_ERR_INVALID_ARG;
  if ((int64_t)batch * s_q >= kMaxRows / select::kMaxCluster) return MLA_ERR_UNSUPPORTED;
  if (!scores || !cache_seqlens || !block_table || !indices || (pages && !lens) || !aligned(scores, 4) ||
      !aligned(cache_seqlens, 4) || !aligned(block_table, 4) || !aligned(indices, 4) || (lens && !aligned(lens, 4)) ||
      (status && !aligned(status, 4)))
    return MLA_ERR_INVALID_ARG;
  const int64_t queries = (int64_t)batch * s_q;
  if (!apart({int32_span(indices, queries * topk), int32_span(lens, queries), status_span(status)},
             {{scores, 4 * ((queries - 1) * score_stride + width)}, int32_span(block_table, (int64_t)batch * max_blocks),
              int32_span(cache_seqlens, batch)}))
    return MLA_ERR_INVALID_ARG;
  select::SelectParams p{scores, score_stride, width, cache_seqlens, block_table, num_blocks, max_blocks,
                         batch, s_q, causal ? 1 : 0, topk, 0, indices, lens, status};
  int dev = 0, sms = 0;
  if (const mla_status v = sm_count(&dev, &sms)) return v;
  const int64_t most = pages ? ((columns < reach ? columns : reach) + kTile - 1) / kTile : columns < reach ? columns : reach;
  return pages ? launch_select<true>(p, most, sms, stream) : launch_select<false>(p, most, sms, stream);
}

}  // extern "C"
