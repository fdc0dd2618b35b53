// prompt_api.cu -- the C entry points of prompts over the paged latent cache:
// norms with the rotary positions, the normalised append, rows read back, and
// the attention of many new tokens (include/mla.h). Every argument check
// happens before anything is enqueued.
#include <cmath>

#include "checks.h"
#include "norms.cuh"
#include "prefill_few.cuh"
#include "prefill_pair.cuh"
#include "read.cuh"

using namespace mla;

namespace {

// rows of `inner` heads and `outer` tokens do not overlap one another
bool rows_apart(int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride, int64_t w) {
  return tokens <= 1 || heads <= 1 || token_stride >= (heads - 1) * head_stride + w || head_stride >= (tokens - 1) * token_stride + w;
}
bool style_ok(int s) { return s == MLA_ROPE_PAIRS || s == MLA_ROPE_HALVES; }
bool eps_ok(float e) { return e >= 0.f && std::isfinite(e); }

template <bool kFp16, int kLanes, int kChunks, int kU>
mla_status launch_norm(norms::NormRotateParams p, void* stream) {
  p.groups_per_token = (uint32_t)((p.heads + kU - 1) / kU);
  constexpr int per = norms::kNormThreads / kLanes;
  const int64_t groups = p.tokens * p.groups_per_token;
  return launch(norms::mla_norm_rotate_kernel<kFp16, kLanes, kChunks, kU>, dim3((unsigned)((groups + per - 1) / per)),
                norms::kNormThreads, 0, stream, p);
}
// Rows of (token, head) from which a lane group takes two heads of a token, which share the table row and the weights
// (4095 x 128 rows of 192: 66.6 us against 74.1 with one and 86.5 with four; 64 x 128, where one fills the card better,
// 2.1 against 2.5 and 4.4).
constexpr int64_t kTwoHeads = 32768;
template <bool kFp16>
mla_status launch_norm_dim(const norms::NormRotateParams& p, void* stream) {
  const int rest = (p.dim - rows::kRope) / 8;
  const bool two = p.heads > 1 && p.tokens * p.heads >= kTwoHeads;
  if (rest <= 8) return two ? launch_norm<kFp16, 8, 1, 2>(p, stream) : launch_norm<kFp16, 8, 1, 1>(p, stream);
  if (rest <= 16) return two ? launch_norm<kFp16, 8, 2, 2>(p, stream) : launch_norm<kFp16, 8, 2, 1>(p, stream);
  if (rest <= 24) return launch_norm<kFp16, 8, 3, 1>(p, stream);
  return launch_norm<kFp16, 32, 2, 1>(p, stream);
}

template <int kFormat, bool kFp16>
mla_status launch_read(const read::ReadParams& p, void* stream) {
  constexpr int64_t per = read::kReadWarps * read::kReadRows;
  return launch(read::mla_read_kv_kernel<kFormat, kFp16>, dim3((unsigned)((p.total + per - 1) / per)),
                32 * read::kReadWarps, 0, stream, p);
}

constexpr int kCardSms = 152;
constexpr int kMostPieces = 16;
static_assert(kMostPieces <= 32 && 4 * kMostPieces <= 2 * prefill::kV);   // the join: a lane, and a word of a row of out, to a piece
// How the attention is launched, from sizes that the host knows.
struct PrefillPlan {
  bool pair;         // two CTAs to a unit of 512 queries, or one to a unit of 128
  int64_t units;     // most units there can be
  int pieces;        // most pieces of a unit
  int piece_tiles;   // key tiles of a piece
};
// A unit's key tiles are cut where the units would fill the card's places less than twice: into as many pieces as fill
// them twice if the documents are alike, and of one length, so that long documents get more of them (up to twice as
// many). Measured (GB300, us): 16 units of 512 tiles 102 in 16 pieces each, 138 in 10, which leave a second round of 8
// pieces; 128 units of 43 to 128 tiles 131 to 140 in 2 to 4 pieces, 154 uncut; but 256 units of 64 tiles 172 uncut, 187
// in 2 pieces. A piece costs some 4 tiles more than its own (the pipeline's start, its share of the output to memory and
// back), so that 8 units of 256 tiles take 36 in 16 pieces and 43 in 32.
//
// Documents of up to 256 queries on average go to one CTA a unit: 16 of 256 over 4096 keys, 16 heads 162 us, 210 in
// pairs; of 300 228 either way; of 400 269 and 231; 64 of 256 by themselves 92 and 94, of 512 241 and 140.
constexpr int kFewRows = 256;
PrefillPlan plan_prefill(int64_t tq, int64_t tk, int64_t batch, int64_t heads) {
  PrefillPlan plan{};
  plan.pieces = plan.piece_tiles = 1;
  if (batch <= 0 || tq <= 0) return plan;
  plan.pair = tq / batch > kFewRows;
  const int64_t block = plan.pair ? prefill::pair::UnitP::kBlock : prefill::few::UnitF::kBlock, places = plan.pair ? kCardSms / 2 : kCardSms;
  const int64_t some = batch < tq ? batch : tq;     // documents with a query, at most
  plan.units = (tq + (block - 1) * some) / block * heads;
  const int64_t alike = some * ((tq / some + block - 1) / block) * heads;   // units of documents of one length
  const int64_t tiles = (tk / batch + prefill::kKeys - 1) / prefill::kKeys;
  int64_t want = 2 * places / alike, most = tiles / prefill::kPieceTiles;
  if (want < 1 || most < 1) return plan;
  want = want < most ? want : most;
  want = want < kMostPieces ? want : kMostPieces;
  plan.piece_tiles = (int)((tiles + want - 1) / want);
  plan.pieces = (int)(2 * want < kMostPieces ? 2 * want : kMostPieces);
  return plan;
}
size_t piece_bytes(int64_t tq, int64_t heads) { return (size_t)tq * (size_t)heads * (prefill::kV + 1) * 4; }

// rows of `dim` elements of [rows, heads]: box of 64 elements by `box_rows` rows of a head
bool make_map_heads(CUtensorMap* m, const void* base, bool fp16, int dim, int64_t heads, int64_t rows, int64_t head_stride,
                    int64_t row_stride, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)row_stride * 2};
  cuuint32_t box[3] = {64, 1, box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
            strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `maps`: of the queries, keys, rotated keys, values, and for a pair of the outputs
template <bool kFp16, bool kPair, typename... M>
mla_status launch_prefill(int dev, int64_t units, void* stream, const prefill::PrefillParams& p, const M&... maps) {
  namespace pf = prefill;
  static std::atomic<bool> set[kMaxDevices];
  auto kernel = [] {
    if constexpr (kPair) return pf::pair::mla_prefill_pair_kernel<kFp16>;
    else return pf::few::mla_prefill_few_kernel<kFp16>;
  }();
  constexpr uint32_t smem = kPair ? pf::pair::kSmem : pf::few::kSmem;
  constexpr int block = kPair ? pf::pair::UnitP::kBlock : pf::few::UnitF::kBlock;
  if (!set[dev].load(std::memory_order_relaxed)) {
    // the softmax warps wait for the registers that the launch gave the others: without them they would wait for good
    cudaFuncAttributes at;
    MLA_CUDA(cudaFuncGetAttributes(&at, kernel));
    if (at.numRegs < pf::kRegsLaunch) return MLA_ERR_UNSUPPORTED;
    MLA_CUDA(set_smem(kernel, smem));
    set[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * p.splits * (kPair ? 2 : 1)), 1, 1);
  cfg.blockDim = dim3(pf::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = kPair ? 2 : 1;
  MLA_CUDA(cudaLaunchKernelEx(&cfg, kernel, maps..., p));
  if (p.splits == 1) return MLA_OK;
  const int64_t warps = pf::kCombineThreads / 32, items = p.tq * p.heads;
  return launch(pf::mla_prefill_combine_kernel<kFp16, block>,
                dim3((unsigned)((items + warps - 1) / warps)), pf::kCombineThreads, 0, stream, p);
}

}  // namespace

extern "C" {

mla_status mla_norm_rotate(const void* x, int64_t x_token_stride, int64_t x_head_stride, const void* weight, float eps,
                           int dim, int rope_at, void* out, int64_t out_token_stride, int64_t out_head_stride,
                           void* rope_out, int64_t rope_token_stride, int64_t rope_head_stride, int dtype,
                           const int32_t* positions, const float* rope_table, int64_t max_positions, int rope_style,
                           int64_t tokens, int heads, uint32_t* status, void* stream) {
  if (tokens < 0 || heads < 1 || tokens >= kMaxRows / heads || max_positions <= 0) return MLA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || !style_ok(rope_style) || !eps_ok(eps)) return MLA_ERR_INVALID_ARG;
  if (dim < rows::kRope || dim % 8 || rope_at < 0 || rope_at % 8 || rope_at > dim - rows::kRope) return MLA_ERR_INVALID_ARG;
  if (dim > norms::kMaxDim) return MLA_ERR_UNSUPPORTED;
  const int64_t w = rope_out ? dim - rows::kRope : dim;   // values of a row of out
  const int64_t xt = x_token_stride, xh = x_head_stride, ot = out_token_stride, oh = out_head_stride;
  if (!stride_ok(xt, 0, tokens) || !stride_ok(xh, 0, heads)) return MLA_ERR_INVALID_ARG;
  if (w && (!stride_ok(ot, w, tokens) || !stride_ok(oh, w, heads))) return MLA_ERR_INVALID_ARG;
  if (rope_out && (!stride_ok(rope_token_stride, rows::kRope, tokens) || !stride_ok(rope_head_stride, rows::kRope, heads)))
    return MLA_ERR_INVALID_ARG;
  if (status && !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (tokens == 0) return MLA_OK;
  if (!x || (w && !out) || !aligned(x, 16) || !aligned(out, 16) || !aligned(rope_out, 16) || !aligned(weight, 16))
    return MLA_ERR_INVALID_ARG;
  if (w && !rows_apart(tokens, ot, heads, oh, w)) return MLA_ERR_INVALID_ARG;
  if (rope_out && !rows_apart(tokens, rope_token_stride, heads, rope_head_stride, rows::kRope)) return MLA_ERR_INVALID_ARG;
  norms::NormRotateParams p{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(out),
                            static_cast<uint16_t*>(rope_out), xt, xh, ot, oh, rope_token_stride, rope_head_stride,
                            {positions, rope_table, max_positions, rope_style == MLA_ROPE_HALVES, status},
                            tokens, heads, dim, rope_at, eps, 0};
  if (const mla_status v = check_positions(p.pos)) return v;
  auto span = [&](const void* at, int64_t ts, int64_t hs, int64_t width) {
    return Span{at, 2 * ((tokens - 1) * ts + (heads - 1) * hs + width)};
  };
  const Span sx = span(x, xt, xh, dim), so = w ? span(out, ot, oh, w) : Span{nullptr, 0},
             sr = rope_out ? span(rope_out, rope_token_stride, rope_head_stride, rows::kRope) : Span{nullptr, 0};
  // in place: the same rows, each read as a whole before it is written
  const bool in_place = !rope_out && out == x && (xt == ot || tokens == 1) && (xh == oh || heads == 1);
  if (!apart({so, sr, status_span(status)}, {{weight, 2 * (int64_t)dim}, int32_span(positions, tokens), table_span(p.pos)}) ||
      (!in_place && so.meets(sx)) || sr.meets(sx) || status_span(status).meets(sx))
    return MLA_ERR_INVALID_ARG;
  return dtype == MLA_DTYPE_FP16 ? launch_norm_dim<true>(p, stream) : launch_norm_dim<false>(p, stream);
}

mla_status mla_norm_append_kv(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t r_stride, const void* weight,
                              float eps, int dtype, const int32_t* slots, const int32_t* positions,
                              const float* rope_table, int64_t max_positions, int rope_style, int64_t n, void* kvcache,
                              int64_t num_blocks, int page_block, int kv_format, void* rows_out, int64_t rows_stride,
                              uint32_t* status, void* stream) {
  if (n < 0 || n >= kMaxRows || max_positions <= 0 || !cache_ok(num_blocks, page_block)) return MLA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || kv_format < MLA_KV_16BIT || kv_format > MLA_KV_FP4_288) return MLA_ERR_INVALID_ARG;
  if (!style_ok(rope_style) || !eps_ok(eps)) return MLA_ERR_INVALID_ARG;
  const int latent = kv_format >= MLA_KV_FP8_528 ? kDV41 - rows::kRope : kDV, width = latent + rows::kRope;
  if (!stride_ok(c_stride, latent, n) || !stride_ok(r_stride, rows::kRope, n)) return MLA_ERR_INVALID_ARG;
  if (rows_out && !stride_ok(rows_stride, width, n)) return MLA_ERR_INVALID_ARG;
  if (status && !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (kv_format && dtype != MLA_DTYPE_BF16) return MLA_ERR_UNSUPPORTED;  // quantised rows pair with bf16
  if (n == 0) return MLA_OK;
  if (!c_kv || !k_rope || !slots || !kvcache || !aligned(c_kv, 16) || !aligned(k_rope, 16) || !aligned(slots, 4) ||
      !aligned(kvcache, 16) || !aligned(weight, 16) || !aligned(rows_out, 16))
    return MLA_ERR_INVALID_ARG;
  norms::NormAppendParams p{{c_kv, k_rope, c_stride, r_stride, slots,
                             {positions, rope_table, max_positions, rope_style == MLA_ROPE_HALVES, status},
                             n, static_cast<uint8_t*>(kvcache), num_blocks * kTile},
                            static_cast<const uint16_t*>(weight), eps, static_cast<uint16_t*>(rows_out), rows_stride,
                            aligned(rows_out, 32) && rows_stride % 16 == 0};
  if (const mla_status v = check_positions(p.a.pos)) return v;
  static constexpr int64_t row_bytes[4] = {kDK * 2, kRowBytesFp8, kRowBytesFp8_528, kRowBytesFp4_288};
  if (!apart({{kvcache, p.a.num_rows * row_bytes[kv_format]}, {rows_out, 2 * ((n - 1) * rows_stride + width)}, status_span(status)},
             {{c_kv, 2 * ((n - 1) * c_stride + latent)}, {k_rope, 2 * ((n - 1) * r_stride + rows::kRope)},
              {weight, 2 * (int64_t)latent}, int32_span(slots, n), int32_span(positions, n), table_span(p.a.pos)}))
    return MLA_ERR_INVALID_ARG;
  const dim3 grid((unsigned)((n + rows::kAppendWarps - 1) / rows::kAppendWarps));
  const int threads = 32 * rows::kAppendWarps;
  if (kv_format == MLA_KV_FP8_656) return launch(norms::mla_norm_append_kv_kernel<false, MLA_KV_FP8_656>, grid, threads, 0, stream, p);
  if (kv_format == MLA_KV_FP8_528) return launch(norms::mla_norm_append_kv_kernel<false, MLA_KV_FP8_528>, grid, threads, 0, stream, p);
  if (kv_format == MLA_KV_FP4_288) return launch(norms::mla_norm_append_kv_kernel<false, MLA_KV_FP4_288>, grid, threads, 0, stream, p);
  if (dtype == MLA_DTYPE_FP16) return launch(norms::mla_norm_append_kv_kernel<true, MLA_KV_16BIT>, grid, threads, 0, stream, p);
  return launch(norms::mla_norm_append_kv_kernel<false, MLA_KV_16BIT>, grid, threads, 0, stream, p);
}

mla_status mla_read_kv(const void* kvcache, int64_t num_blocks, int page_block, int kv_format, const int32_t* block_table,
                       int max_blocks, const int32_t* offsets, const int32_t* starts, int batch, int64_t total, void* out,
                       int64_t out_stride, int dtype, uint32_t* status, void* stream) {
  if (!cache_ok(num_blocks, page_block) || kv_format < MLA_KV_16BIT || kv_format > MLA_KV_FP4_288 || !dtype_ok(dtype))
    return MLA_ERR_INVALID_ARG;
  if (batch < 0 || max_blocks <= 0 || !in_memory(max_blocks, batch) || total < 0 || total >= kMaxRows) return MLA_ERR_INVALID_ARG;
  const int width = kv_format >= MLA_KV_FP8_528 ? kDV41 : kDK;
  if (!stride_ok(out_stride, width, total) || (status && !aligned(status, 4))) return MLA_ERR_INVALID_ARG;
  if (total == 0 || batch == 0) return MLA_OK;
  if (!kvcache || !block_table || !offsets || !out || !aligned(kvcache, 16) || !aligned(block_table, 4) || !aligned(offsets, 4) ||
      !aligned(starts, 4) || !aligned(out, 16))
    return MLA_ERR_INVALID_ARG;
  static constexpr int64_t row_bytes[4] = {kDK * 2, kRowBytesFp8, kRowBytesFp8_528, kRowBytesFp4_288};
  if (!apart({{out, 2 * ((total - 1) * out_stride + width)}, status_span(status)},
             {{kvcache, num_blocks * kTile * row_bytes[kv_format]}, int32_span(block_table, (int64_t)batch * max_blocks),
              int32_span(offsets, (int64_t)batch + 1), int32_span(starts, batch)}))
    return MLA_ERR_INVALID_ARG;
  const read::ReadParams p{static_cast<const uint8_t*>(kvcache), block_table, offsets, starts, num_blocks, batch, max_blocks,
                           total, static_cast<uint16_t*>(out), out_stride, aligned(out, 32) && out_stride % 16 == 0, status};
  const bool fp16 = dtype == MLA_DTYPE_FP16;
  if (kv_format == MLA_KV_16BIT) return launch_read<MLA_KV_16BIT, false>(p, stream);   // copied, whatever the type
  if (kv_format == MLA_KV_FP8_656) return fp16 ? launch_read<MLA_KV_FP8_656, true>(p, stream) : launch_read<MLA_KV_FP8_656, false>(p, stream);
  if (kv_format == MLA_KV_FP8_528) return fp16 ? launch_read<MLA_KV_FP8_528, true>(p, stream) : launch_read<MLA_KV_FP8_528, false>(p, stream);
  return fp16 ? launch_read<MLA_KV_FP4_288, true>(p, stream) : launch_read<MLA_KV_FP4_288, false>(p, stream);
}

size_t mla_prefill_workspace_size(int64_t tokens_q, int64_t tokens_k, int batch, int heads) {
  if (tokens_q <= 0 || tokens_k < 0 || batch <= 0 || heads <= 0 || tokens_q >= kMaxRows || tokens_k >= kMaxRows) return 0;
  const int n = plan_prefill(tokens_q, tokens_k, batch, heads).pieces;
  return n > 1 ? n * piece_bytes(tokens_q, heads) : 0;
}

mla_status mla_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_nope,
                       int64_t k_token_stride, int64_t k_head_stride, const void* k_rope, int64_t rope_stride,
                       const void* v, int64_t v_token_stride, int64_t v_head_stride, int dtype, const int32_t* cu_seqlens_q,
                       const int32_t* cu_seqlens_k, const int32_t* prefix_lens, int batch, int64_t tokens_q,
                       int64_t tokens_k, int heads, float softmax_scale, int causal, void* out, int64_t out_token_stride,
                       int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes, uint32_t* status,
                       void* stream) {
  namespace pf = prefill;
  const int64_t tq = tokens_q, tk = tokens_k;
  if (tq < 0 || tk < 0 || batch < 0 || heads < 1 || tq >= kMaxRows - 512 || tk >= kMaxRows - 512 || !dtype_ok(dtype))
    return MLA_ERR_INVALID_ARG;
  // so that 8 / (scale log2 e), the reference's step in raw scores, and the factor itself stay normal numbers
  if (!(softmax_scale >= 0x1p-100f) || !(softmax_scale <= 0x1p100f)) return MLA_ERR_INVALID_ARG;
  if (tq >= (int64_t(1) << 44) / heads || tk >= (int64_t(1) << 44) / heads) return MLA_ERR_INVALID_ARG;
  // TMA strides lie below 2^40 bytes
  constexpr int64_t kStride = int64_t(1) << 39;
  auto strides_ok = [&](int64_t token, int64_t head, int64_t rows, int64_t w) {
    return stride_ok(token, w, rows) && stride_ok(head, w, heads) && token < kStride && head < kStride;
  };
  if (out_token_stride >= kStride || out_head_stride >= kStride || !strides_ok(q_token_stride, q_head_stride, tq, pf::kQk) || !strides_ok(k_token_stride, k_head_stride, tk, pf::kNope) ||
      !strides_ok(v_token_stride, v_head_stride, tk, pf::kV) || !stride_ok(rope_stride, pf::kRopeDim, tk) || rope_stride >= kStride ||
      !stride_ok(out_token_stride, pf::kV, tq) || !stride_ok(out_head_stride, pf::kV, heads))
    return MLA_ERR_INVALID_ARG;
  if (status && !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (tq == 0 || batch == 0) return MLA_OK;
  if (!q || !out || !lse || !cu_seqlens_q || !cu_seqlens_k || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) || !aligned(prefix_lens, 4))
    return MLA_ERR_INVALID_ARG;
  if (tk > 0 && (!k_nope || !k_rope || !v || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16))) return MLA_ERR_INVALID_ARG;
  if (!rows_apart(tq, out_token_stride, heads, out_head_stride, pf::kV)) return MLA_ERR_INVALID_ARG;
  const PrefillPlan plan = plan_prefill(tq, tk, batch, heads);
  const int splits = plan.pieces;
  if (plan.units * splits >= kMaxRows / 2 || tq * heads >= (kMaxRows - 1) * (pf::kCombineThreads / 32)) return MLA_ERR_UNSUPPORTED;
  const size_t need = splits > 1 ? splits * piece_bytes(tq, heads) : 0;
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return MLA_ERR_INVALID_ARG;
  auto span = [&](const void* at, int64_t ts, int64_t hs, int64_t rows, int64_t width) {
    return rows ? Span{at, 2 * ((rows - 1) * ts + (heads - 1) * hs + width)} : Span{nullptr, 0};
  };
  if (!apart({span(out, out_token_stride, out_head_stride, tq, pf::kV), {lse, 4 * tq * heads},
              {need ? workspace : nullptr, (int64_t)need}, status_span(status)},
             {span(q, q_token_stride, q_head_stride, tq, pf::kQk), span(k_nope, k_token_stride, k_head_stride, tk, pf::kNope),
              span(v, v_token_stride, v_head_stride, tk, pf::kV), {tk ? k_rope : nullptr, 2 * ((tk - 1) * rope_stride + pf::kRopeDim)},
              int32_span(cu_seqlens_q, (int64_t)batch + 1), int32_span(cu_seqlens_k, (int64_t)batch + 1), int32_span(prefix_lens, batch)}))
    return MLA_ERR_INVALID_ARG;

  pf::PrefillParams p{};
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.prefix = causal ? prefix_lens : nullptr;
  p.tq = tq;
  p.tk = tk;
  p.batch = batch;
  p.heads = heads;
  p.causal = causal ? 1 : 0;
  p.splits = splits;
  p.piece_tiles = plan.piece_tiles;
  p.scale = softmax_scale;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = out;
  p.out_token = out_token_stride;
  p.out_head = out_head_stride;
  p.lse = lse;
  p.o_part = static_cast<float*>(workspace);
  p.ref_part = need ? p.o_part + (int64_t)splits * tq * heads * pf::kV : nullptr;
  p.wide = (aligned(out, 32) && out_token_stride % 16 == 0 && out_head_stride % 16 == 0 ? 1 : 0) | (aligned(workspace, 32) ? 2 : 0);
  p.status = status;
  p.stall_cycles = g_test_stall.load(std::memory_order_relaxed);
  int dev = 0, sms = 0;
  if (const mla_status v = sm_count(&dev, &sms)) return v;
  const bool fp16 = dtype == MLA_DTYPE_FP16;
  CUtensorMap mq, mk, mr, mv;
  // without keys nothing is copied through the last three
  const bool some = tk > 0;
  const uint32_t key_rows = plan.pair ? pf::kKeys / 2 : pf::kKeys;   // a CTA of a pair copies half of the keys
  if (!make_map_heads(&mq, q, fp16, pf::kQk, heads, tq, q_head_stride, q_token_stride, pf::kRows) ||
      !make_map_heads(&mk, some ? k_nope : q, fp16, pf::kNope, some ? heads : 1, some ? tk : 1, some ? k_head_stride : pf::kNope,
                      some ? k_token_stride : pf::kNope, key_rows) ||
      !make_map_heads(&mr, some ? k_rope : q, fp16, pf::kRopeDim, 1, some ? tk : 1, pf::kRopeDim, some ? rope_stride : pf::kRopeDim,
                      key_rows) ||
      !make_map_heads(&mv, some ? v : q, fp16, pf::kV, some ? heads : 1, some ? tk : 1, some ? v_head_stride : pf::kV,
                      some ? v_token_stride : pf::kV, pf::kKeys))
    return MLA_ERR_CUDA;
  if (plan.pair) {
    CUtensorMap mo;
    if (!make_map_heads(&mo, out, fp16, pf::kV, heads, tq, out_head_stride, out_token_stride, 32)) return MLA_ERR_CUDA;
    return fp16 ? launch_prefill<true, true>(dev, plan.units, stream, p, mq, mk, mr, mv, mo)
                : launch_prefill<false, true>(dev, plan.units, stream, p, mq, mk, mr, mv, mo);
  }
  return fp16 ? launch_prefill<true, false>(dev, plan.units, stream, p, mq, mk, mr, mv)
              : launch_prefill<false, false>(dev, plan.units, stream, p, mq, mk, mr, mv);
}

}  // extern "C"
