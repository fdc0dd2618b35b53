/*
 * mla.h -- C ABI of libmla: Multi-head Latent Attention (MLA) decode over a
 * paged, compressed latent KV cache, for NVIDIA GB300 (sm_103a).
 *
 * What is computed. After weight absorption every query head scores one shared
 * 576-wide cache row per token (512 latent dims c^KV + 64 decoupled-RoPE dims
 * k^R): score = q~ . c + q^R . k^R, and the value is the 512-wide latent c
 * itself; decode is therefore MQA with h_kv = 1, d_k = 576, d_v = 512
 * ("矩阵、注意力与 GPU：拆解 DeepGEMM 与 FlashMLA", §六 '吸收' and '结果：decode
 * 变成 MQA'). For every request b, query position i and head h:
 *     out[b,i,h,:] = sum_t softmax_t(scale * q[b,i,h,:] . K_t) * K_t[0:512]
 *     lse[b,i,h]   = ln sum_t exp(scale * q[b,i,h,:] . K_t)
 * over the visible tokens t (§五 '注意力：两个 GEMM 加一个 softmax' of the same
 * page; the kernels use the online softmax and the split-KV combine of §五/§七,
 * which reorder but do not approximate it).
 *
 * Conventions for every call below:
 *  - Pointers marked (device) are CUDA device pointers owned by the caller; the
 *    library never allocates, frees or retains them past the call (except that
 *    the kernels it enqueues read/write them until they complete on `stream`).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    All work is enqueued asynchronously; no call synchronises the host except
 *    mla_read_status().
 *  - Argument errors are detected on the host before anything is enqueued and
 *    return MLA_ERR_INVALID_ARG / MLA_ERR_UNSUPPORTED; nothing is written then.
 *  - Problems only visible on the device (an out-of-range page or index, a
 *    stale metadata buffer, a pipeline wait that timed out) never trap: the
 *    kernel sets a bit in the status word kept in the workspace, and
 *    mla_read_status() reports it.
 *  - All entry points are thread-safe; calls on one stream execute in order.
 */
#ifndef MLA_GB300_H_
#define MLA_GB300_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MLA_API __attribute__((visibility("default")))
#else
#define MLA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,      /* bad shape, pointer, alignment or flag combination */
  MLA_ERR_UNSUPPORTED = 2,      /* valid request the library does not implement   */
  MLA_ERR_STALE_METADATA = 3,   /* metadata computed for a different shape/lengths */
  MLA_ERR_INDEX = 4,            /* an out-of-range page or sparse index was skipped */
  MLA_ERR_TIMEOUT = 5,          /* a device pipeline wait gave up (kernel returned early) */
  MLA_ERR_CUDA = 6,             /* a CUDA runtime/driver call failed */
  MLA_ERR_RANGE = 7             /* quantised cache: a value or a score beyond the certified range (see below) */
} mla_status;

typedef enum { MLA_DTYPE_BF16 = 0, MLA_DTYPE_FP16 = 1 } mla_dtype;

/* Cache row formats (the `kv_format` argument; 0 and 1 are the reference's
 * is_fp8_kvcache = false / true):
 *  MLA_KV_16BIT    576 values of q_dtype (512 latent + 64 RoPE), 1152 B;
 *  MLA_KV_FP8_656  512 e4m3 latent values, 4 fp32 scales (one per 128), the 64
 *                  RoPE dims as bf16: 656 B ("FlashMLA 实战：MLA 注意力加速指南",
 *                  §FP8 缓存怎么把 KV 压掉四成);
 *  MLA_KV_FP8_528  the V4.1 row of 512 values (latent and RoPE together): 512
 *                  e4m3 codes, then 16 UE8M0 scales, byte j = k + 127 for the
 *                  scale 2^k of values [32j, 32j+32): 528 B;
 *  MLA_KV_FP4_288  the FP4 row of 512 values: 256 bytes of e2m1 codes (value 2i
 *                  in the low nibble of byte i), then 32 e4m3 scales, byte j for
 *                  values [16j, 16j+16): 288 B
 * ("矩阵、注意力与 GPU：拆解 DeepGEMM 与 FlashMLA", §八 '版本漂移' and the §十
 * format table). With the V4.1 rows a key is 512 wide and the value is the
 * whole row: q is [batch, s_q, h_q, 512] and head_dim_v is 512. */
typedef enum { MLA_KV_16BIT = 0, MLA_KV_FP8_656 = 1, MLA_KV_FP8_528 = 2, MLA_KV_FP4_288 = 3 } mla_kv_format;

#define MLA_HEAD_DIM_K 576
#define MLA_HEAD_DIM_V 512
#define MLA_FP8_ROW_BYTES 656
#define MLA_V41_DIM 512
#define MLA_FP8_528_ROW_BYTES 528
#define MLA_FP4_288_ROW_BYTES 288

/* Human-readable name of a status code (static string). */
MLA_API const char* mla_status_string(int status);

/* Number of work partitions ("SM parts") the 128-head decode kernels use on
 * `device`: the number of co-resident 2-CTA clusters of the dense/FP8 decode
 * kernel. Returns a value <= 0 on failure (no device). */
MLA_API int mla_num_sm_parts(int device);

/* The same for a given number of query heads: h_q = 128 as above; h_q = 16
 * (the transposed few-heads kernel, one CTA per part, after the FlashMLA-ETAP
 * page, §3.1) the number of its co-resident CTAs. Returns a value <= 0 on
 * failure or for an unsupported h_q. */
MLA_API int mla_num_sm_parts_for(int device, int h_q);

/* Bytes of the metadata buffer for a decode shape. */
MLA_API size_t mla_metadata_size(int batch, int s_q, int num_sm_parts);

/*
 * Split-KV work schedule ("矩阵、注意力与 GPU：拆解 DeepGEMM 与 FlashMLA",
 * §七 'split-KV：把长序列切开': the schedule decides which SM part handles which
 * requests and KV blocks and how many pieces each request is cut into; it is
 * computed once and reused by every layer and step of the same shape).
 *
 * The (request, query position) pairs v = i*batch + b ("virtual requests")
 * are cut into 64-token tiles (visible length per query position: dense
 * L_b, or L_b - s_q + 1 + i when causal; sparse: topk) and the tile list is
 * cut into `num_sm_parts` contiguous ranges of nearly equal cost.
 *
 * cache_seqlens (device) int32 [batch]; may be NULL when topk > 0 (sparse).
 * metadata      (device) mla_metadata_size() bytes, written.
 * num_splits    (device) int32 [batch*s_q + 1], written: exclusive prefix sum
 *               of the number of pieces of each virtual request.
 * kv_format: an mla_kv_format, the one the decode calls will pass.
 * h_q must be 128, or 16 for dense 16-bit caches (the few-heads kernel);
 * h_kv must be 1, page_block 64.
 * Computed entirely on the device (no host synchronisation). The decode call
 * checks on the device that the metadata matches its own arguments and the
 * current cache_seqlens, and reports MLA_ERR_STALE_METADATA otherwise.
 */
MLA_API mla_status mla_get_metadata(const int32_t* cache_seqlens, int batch, int s_q, int h_q, int h_kv,
                            int topk, int kv_format, int causal, int page_block, int num_sm_parts,
                            void* metadata, int32_t* num_splits, void* stream);

/* Bytes of decode workspace (status word, fp32 split partials, and one bit per
 * (query position, head) row for the exact recompute). */
MLA_API size_t mla_workspace_size(int batch, int s_q, int h_q, int num_sm_parts);

/*
 * Decode attention over the latent cache ("FlashMLA 实战：MLA 注意力加速指南",
 * §最小调用: out, lse = flash_mla_with_kvcache(q, kvcache, block_table,
 * cache_seqlens, head_dim_v=512, metadata, num_splits, softmax_scale, causal,
 * is_fp8_kvcache, indices)).
 *
 * q            (device) [batch, s_q, h_q, 576] (V4.1 rows: 512), `q_dtype`,
 *              contiguous, 16-B aligned; bf16 with every quantised format.
 * kvcache      (device) [num_blocks, page_block, 1, row] contiguous, 16-B
 *              aligned: 576 values of q_dtype (kv_format = MLA_KV_16BIT), or
 *              uint8 rows of 656, 528 or 288 bytes (MLA_KV_FP8_656,
 *              MLA_KV_FP8_528, MLA_KV_FP4_288; see the quantisers below).
 *              Token-sparse decode (indices) reads the quantised formats.
 * block_table  (device) int32 [batch, max_blocks], logical page -> physical page;
 *              may be NULL when indices != NULL.
 * cache_seqlens(device) int32 [batch] tokens per request (ignored when indices != NULL).
 * head_dim_v   must be 512.
 * metadata, num_splits: from mla_get_metadata() with the same shape/flags.
 * softmax_scale: multiplies q.K (e.g. 576^-0.5).
 * causal       bottom-right aligned mask for s_q > 1; must be 0 with indices.
 * indices      (device) int32 [batch, s_q, topk] absolute cache rows
 *              (page * page_block + slot), -1 = unused slot; NULL for dense.
 *              Rows must lie in [0, num_blocks*page_block); others are skipped
 *              and flagged as MLA_ERR_INDEX ("拆解" page, §八 sparse indices).
 * out          (device) [batch, s_q, h_q, 512] of q_dtype, written.
 * lse          (device) fp32 [batch, s_q, h_q], natural log, written.
 * workspace    (device) mla_workspace_size() bytes, 256-B aligned, zeroed once
 *              before first use: it holds the status word (mla_read_status
 *              clears it), the fp32 partials of cut requests and one bit per
 *              (query position, head) row that the combine recomputes exactly
 *              (the library leaves those bits zero after every call).
 * A request with no visible token gets out = 0 and lse = -inf.
 * 656-byte FP8 rows run the latent product in fp16: the bf16 query is
 * rounded to fp16 and each cache value is formed as fp16(code) x fp16(block
 * scale), rounded to fp16. Within range the dequantised value has relative
 * error <= 2^-10; a block whose amax is below 448 * 2^-14 (~0.027) has an
 * fp16-subnormal scale, and its values carry an absolute error <= 2^-15
 * instead. Out of range -- a query entry beyond 65504 in magnitude (saturated
 * to +-65504) or a block scale above 146 (block amax above 65408) -- the
 * status word records MLA_ERR_RANGE.
 * The V4.1 rows run in fp16 as well (query rounded to fp16, with the same
 * 65504 limit): e2m1 x e4m3 is always exact in fp16; e4m3 x 2^k is exact for
 * k in [-15, 7]; a block with a smaller scale (amax below 448 * 2^-16) carries
 * an absolute error of at most 2^-25, and a larger one (amax above 57344,
 * UE8M0 byte above 134) is reported as MLA_ERR_RANGE.
 * Every cache type splits the dims of a score between the two CTAs of a
 * pair, which exchange fp16 factors 2^(partial score - partial max). The
 * result is certified exact (to fp16 precision) for a row of a 64-token tile
 * unless the two partial scores of its tokens disagree by more than about 22
 * binades; such a row is recomputed exactly from q and the cache rows for
 * 16-bit caches (by the combine step, so mla_decode_splitkv alone leaves it
 * uncorrected until mla_combine_splits runs), and reported as MLA_ERR_RANGE
 * for quantised caches.
 * h_q = 128 with any cache; h_q = 16 with a dense 16-bit cache only: the few
 * heads fill the MMA's N dimension and the 64 tokens of a tile its M
 * dimension, the transposed formulation S^T = K Q^T, O^T = V^T P^T of the
 * FlashMLA-ETAP page (§2.2, §3.2); same results and layouts.
 */
MLA_API mla_status mla_decode_with_kvcache(const void* q, int q_dtype, const void* kvcache, int64_t num_blocks,
                                   int page_block, const int32_t* block_table, int max_blocks,
                                   const int32_t* cache_seqlens, int batch, int s_q, int h_q,
                                   int head_dim_v, const void* metadata, const int32_t* num_splits,
                                   int num_sm_parts, float softmax_scale, int causal, int kv_format,
                                   const int32_t* indices, int topk, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * The two launches mla_decode_with_kvcache() is made of, for callers that
 * schedule them separately (same arguments, same checks):
 *  - mla_decode_splitkv: the split-KV kernel ("矩阵、注意力与 GPU：拆解 DeepGEMM 与
 *    FlashMLA", §七 'split-KV'); requests that are one piece get their final
 *    out/lse, the pieces of cut requests get fp32 partials (o, lse) in the
 *    workspace;
 *  - mla_combine_splits: merges those partials into out/lse (m = max lse_i,
 *    o = sum o_i e^{lse_i - m} / sum e^{lse_i - m}, same section) and writes
 *    out = 0, lse = -inf for requests with no visible token. It must follow
 *    mla_decode_splitkv of the same arguments on the same stream.
 */
MLA_API mla_status mla_decode_splitkv(const void* q, int q_dtype, const void* kvcache, int64_t num_blocks,
                                      int page_block, const int32_t* block_table, int max_blocks,
                                      const int32_t* cache_seqlens, int batch, int s_q, int h_q,
                                      int head_dim_v, const void* metadata, const int32_t* num_splits,
                                      int num_sm_parts, float softmax_scale, int causal, int kv_format,
                                      const int32_t* indices, int topk, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream);
MLA_API mla_status mla_combine_splits(const void* q, int q_dtype, const void* kvcache, int64_t num_blocks,
                                      int page_block, const int32_t* block_table, int max_blocks,
                                      const int32_t* cache_seqlens, int batch, int s_q, int h_q,
                                      int head_dim_v, const void* metadata, const int32_t* num_splits,
                                      int num_sm_parts, float softmax_scale, int causal, int kv_format,
                                      const int32_t* indices, int topk, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * mla_decode_with_kvcache without a caller-supplied workspace, for callers that
 * cannot allocate device memory on demand (cudaMalloc may synchronise the
 * device and can fail once memory is committed -- unacceptable inside a
 * fixed-latency serving loop, or for a plug-in whose host application owns
 * every device allocation). The pages describe no such entry point; it is an
 * engineering addition of this library.
 *
 * Same arguments and results as mla_decode_with_kvcache, except:
 *  - the split-KV scratch is a fixed 32 MiB array inside the library, one per
 *    device, held until the process exits; a shape whose mla_workspace_size()
 *    exceeds 32 MiB is rejected with MLA_ERR_INVALID_ARG (use
 *    mla_decode_with_kvcache for it);
 *  - nothing is allocated or freed;
 *  - all calls on a device share the array: calls that may overlap on the GPU
 *    (e.g. on different streams) race and must be serialised by the caller;
 *  - the first call on a device looks up the array's device address (once,
 *    with that device current); make that first call before any stream
 *    capture;
 *  - status (device, optional, 4-B aligned): receives the device-side status
 *    bits of this call (1 = index/page skipped, 2 = wait timeout, 4 = stale
 *    metadata, 8 = range of a quantised cache), or NULL to discard them.
 */
MLA_API mla_status mla_decode_with_kvcache_noalloc(const void* q, int q_dtype, const void* kvcache,
                                                   int64_t num_blocks, int page_block,
                                                   const int32_t* block_table, int max_blocks,
                                                   const int32_t* cache_seqlens, int batch, int s_q, int h_q,
                                                   int head_dim_v, const void* metadata,
                                                   const int32_t* num_splits, int num_sm_parts,
                                                   float softmax_scale, int causal, int kv_format,
                                                   const int32_t* indices, int topk, void* out, float* lse,
                                                   uint32_t* status, void* stream);

/*
 * Write the 656-byte FP8 cache rows ("FlashMLA 实战：MLA 注意力加速指南",
 * §FP8 缓存怎么把 KV 压掉四成): bytes [0,512) e4m3 codes of the 512 latent dims,
 * quantised per 128 values with scale = fp32(amax/448) (1.0 for an all-zero
 * block) and code = round-to-nearest-even(fp32(x/scale)) saturated to +-448;
 * bytes [512,528) the 4 scales as fp32; bytes [528,656) the 64 RoPE dims copied
 * as bf16.
 * kv (device) bf16 [n, 576] (row stride 576 elements); out (device) uint8 [n, 656].
 */
MLA_API mla_status mla_quantize_kv_fp8(const void* kv, uint8_t* out, int64_t n, void* stream);

/*
 * Write the V4.1 rows of 512 values ("矩阵、注意力与 GPU：拆解 DeepGEMM 与
 * FlashMLA", §八 '版本漂移', §十 format table; §三 'UE8M0': a power-of-two
 * scale, rounded up). The page prints no quantiser; these follow the plainest
 * reading of it, and the oracle defines the same decisions independently:
 *  - mla_quantize_kv_fp8_528: per 32 values the scale is the smallest 2^k
 *    (k >= -127) with 448 * 2^k >= amax; byte 512 + j = k + 127; byte d =
 *    e4m3 round-to-nearest-even of x_d / 2^k (exact division);
 *  - mla_quantize_kv_fp4_288: per 16 values the scale is the smallest
 *    non-negative e4m3 value v with 6 v >= amax (448 when none is, values then
 *    saturate to +-6); byte 256 + j = its code; each value becomes the e2m1
 *    code nearest to x / v (ties to the even code, the sign of x kept), value
 *    2i in the low nibble of byte i.
 * kv (device) bf16 [n, 512] (row stride 512 elements, finite values); out
 * (device) uint8 [n, 528] or [n, 288]; both 16-B aligned.
 */
MLA_API mla_status mla_quantize_kv_fp8_528(const void* kv, uint8_t* out, int64_t n, void* stream);
MLA_API mla_status mla_quantize_kv_fp4_288(const void* kv, uint8_t* out, int64_t n, void* stream);

/*
 * The per-head GEMMs around the kernel ("矩阵、注意力与 GPU：拆解 DeepGEMM 与
 * FlashMLA", §六 '吸收'): with the key up-projection W^UK_i (d_h x d_c) absorbed
 * into the query, q~_{t,i} = W^UK_i^T q^C_{t,i}, every head scores the shared
 * latent row; the value up-projection is applied once to the attention-weighted
 * latent, o_{t,i} = W^UV_i o~_{t,i}. Here d_h = 128 and d_c = 512; tokens is the
 * number of query tokens (batch * s_q), h_q the number of heads; dtype is
 * MLA_DTYPE_BF16 or MLA_DTYPE_FP16 for every operand. Products accumulate in
 * fp32 and are rounded once to dtype. All pointers are (device), 16-B aligned.
 *
 * mla_absorb_q: q_nope [tokens, h_q, 128], w_uk [h_q, 128, 512] (W^UK_i row d
 * holds the 512 latent weights of output dim d); writes dims [0, 512) of every
 * row of q_out [tokens, h_q, 576], the layout mla_decode_with_kvcache reads,
 * and leaves the 64 RoPE dims [512, 576) to the caller.
 *
 * mla_up_project: o_lat [tokens, h_q, 512] (the decode output), w_uv
 * [h_q, 128, 512]; writes o_out [tokens, h_q, 128].
 *
 * status (device, optional, 4-B aligned): a status word the kernels OR bit 2
 * (wait timeout) into when a bounded wait gave up (nothing is stored then);
 * read and clear it with mla_read_status(). NULL discards it.
 *
 * tokens = 0 enqueues nothing. Returns MLA_ERR_INVALID_ARG for a negative size,
 * a null or misaligned pointer, or an unknown dtype.
 */
MLA_API mla_status mla_absorb_q(const void* q_nope, const void* w_uk, void* q_out, int tokens, int h_q, int dtype,
                                uint32_t* status, void* stream);
MLA_API mla_status mla_up_project(const void* o_lat, const void* w_uv, void* o_out, int tokens, int h_q, int dtype,
                                  uint32_t* status, void* stream);

/*
 * ---------------------------------------------------------------------------
 * From new tokens to the rows that the sparse attention reads. The pages stop
 * at the decode itself; these calls are this library's own: they write the
 * caches that the decode reads, rotate its queries, and produce the `indices`
 * of its token-sparse mode, or a block table that names only the pages worth
 * attending, for the paged mode of any cache format.
 *
 * Rotary positions. A row of 64 dims at position p has its 32 pairs turned by
 * the angles of row p of `rope_table` (device) fp32 [max_positions, 64], 32
 * cosines then 32 sines, 16-B aligned: y0 = x0 cos - x1 sin, y1 = x0 sin +
 * x1 cos, with every product and sum rounded to fp32 and the result rounded
 * once to the type it is stored in. Pair i is dims (2i, 2i + 1) with
 * MLA_ROPE_PAIRS, dims (i, i + 32) with MLA_ROPE_HALVES.
 * `positions` (device) int32, one per token.
 *
 * Common to the writers: a token with slot < 0 (for the calls without slots:
 * position < 0) is padding and leaves its destination as it was; a slot or
 * position out of range is skipped and recorded as an index error (bit 1) in
 * `status` (device, optional, 4-B aligned; read it with mla_read_status).
 * Values must be finite. Strides are in elements and multiples of 8, row
 * starts are 16-B aligned.
 *
 * Common to all six: an output (`status` is one) that shares memory with another
 * argument is refused, but for the cases named below. An array's memory is all
 * from its first to its last byte, gaps between its rows included.
 */
typedef enum { MLA_ROPE_PAIRS = 0, MLA_ROPE_HALVES = 1 } mla_rope_style;

/*
 * Append n tokens to the paged latent cache, rotating the RoPE dims on the way.
 * c_kv   (device) [n, 512] latent dims (V4.1 rows: 448), `dtype`, rows c_stride apart.
 * k_rope (device) [n, 64] RoPE dims before rotation, rows r_stride apart; both
 *        may be column ranges of one projection output.
 * slots  (device) int32 [n] cache row page * 64 + offset of each token. The
 *        slots of one call are distinct (of two equal ones, either token's
 *        bytes may end up in the row).
 * kvcache (device) written: rows of `kv_format` as mla_decode_with_kvcache
 *        reads them. 16-bit rows: [latent, rotated RoPE] in `dtype`. 656-byte
 *        rows: the latent dims quantised as in mla_quantize_kv_fp8, the rotated
 *        RoPE dims rounded to bf16. V4.1 rows: 448 latent and 64 rotated RoPE
 *        dims as one row of 512 values, quantised (the RoPE dims from their
 *        fp32 values) as in mla_quantize_kv_fp8_528 / mla_quantize_kv_fp4_288.
 *        Quantised formats take bf16 input (else MLA_ERR_UNSUPPORTED).
 */
MLA_API mla_status mla_append_kv(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t r_stride, int dtype,
                                 const int32_t* slots, const int32_t* positions, const float* rope_table,
                                 int64_t max_positions, int rope_style, int64_t n, void* kvcache,
                                 int64_t num_blocks, int page_block, int kv_format, uint32_t* status, void* stream);

/*
 * Rotate the RoPE dims of queries: out[t, h, :] = R(x[t, h, :]) over rows of 64.
 * x, out (device) [tokens, heads, 64] with token and head strides; a typical
 * call reads a slice of the query projection and writes dims [512, 576) of the
 * decode's query (the ones mla_absorb_q leaves). out may be x (in place) or, with
 * x's strides, lie between its rows (other columns, other heads of the same
 * tokens); any other overlap, gaps between rows included, is refused.
 */
MLA_API mla_status mla_rotate_q(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
                                int64_t out_token_stride, int64_t out_head_stride, int dtype,
                                const int32_t* positions, const float* rope_table, int64_t max_positions,
                                int rope_style, int64_t tokens, int heads, uint32_t* status, void* stream);

/*
 * The index cache: one 128-wide key per cached token, in pages of 64 like the
 * latent cache and addressed by the same block table.
 *  MLA_INDEX_16BIT  [num_blocks, 64, 128] of bf16 or fp16;
 *  MLA_INDEX_FP8    pages of 8448 bytes: 64 rows of 128 e4m3 codes, then 64
 *                   fp32 scales (amax / 448 of the row, 1 for a zero row).
 *
 * mla_append_index_k: k (device) [n, 128] of `dtype`, rows k_stride apart; dims
 * [0, 64) are rotated, [64, 128) are kept; a 16-bit cache has type `dtype`.
 *
 * mla_quantize_index_q: the queries of an FP8 index. q (device) [tokens, heads,
 * 128] with strides, dims [0, 64) rotated, every row quantised like a key; its
 * scale is folded into the head's weight: q_out (device) uint8 [tokens, heads,
 * 128] e4m3, weights_out[t, h] = weights[t, h] * scale (device fp32, contiguous;
 * may be the same array). Index queries for a 16-bit cache are rotated by
 * mla_rotate_q.
 */
typedef enum { MLA_INDEX_16BIT = 0, MLA_INDEX_FP8 = 1 } mla_index_format;

#define MLA_INDEX_DIM 128
#define MLA_INDEX_FP8_PAGE_BYTES 8448

MLA_API mla_status mla_append_index_k(const void* k, int64_t k_stride, int dtype, const int32_t* slots,
                                      const int32_t* positions, const float* rope_table, int64_t max_positions,
                                      int rope_style, int64_t n, void* index_cache, int64_t num_blocks,
                                      int page_block, int index_format, uint32_t* status, void* stream);
MLA_API mla_status mla_quantize_index_q(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
                                        const float* weights, const int32_t* positions, const float* rope_table,
                                        int64_t max_positions, int rope_style, int64_t tokens, int heads,
                                        uint8_t* q_out, float* weights_out, uint32_t* status, void* stream);

/*
 * The cheap score:
 *     s[b, i, t] = ks_t * sum_h weights[b, i, h] * max(0, q[b, i, h, :] . k_t)
 * over the visible tokens t of request b (L_b, or L_b - s_q + 1 + i when
 * causal), accumulated in fp32; ks_t is the scale of an e4m3 key, else 1. A NaN
 * dot counts as 0 (what stands behind the visible tokens does not matter).
 * q       (device) [batch, s_q, heads, 128] contiguous, 16-B aligned: `q_dtype`
 *         and a 16-bit index cache of the same type, or e4m3 (q_dtype is not
 *         read) with MLA_INDEX_FP8. heads is 1 to 64.
 * weights (device) fp32 [batch, s_q, heads] (softmax scale and head gate).
 * block   1: scores (device) fp32, column t of row b * s_q + i is token t;
 *         64: column j is the maximum over the visible tokens of page j.
 *         Rows are score_stride floats apart; columns [0, width) are written,
 *         -inf where no token is visible.
 * A request longer than `width` or its block-table row is scored as far as they
 * reach, a token on an out-of-range page scores -inf; both are recorded as an
 * index error in `status`.
 */
MLA_API mla_status mla_index_score(const void* q, int q_dtype, const float* weights, const void* index_cache,
                                   int index_format, int64_t num_blocks, int page_block,
                                   const int32_t* block_table, int max_blocks, const int32_t* cache_seqlens,
                                   int batch, int s_q, int heads, int causal, int block, float* scores,
                                   int64_t score_stride, int width, uint32_t* status, void* stream);

/*
 * The topk best columns of each row of `scores` (any fp32 matrix laid out like
 * mla_index_score's; only the visible columns are read). Equal scores go to the
 * lower position, NaN counts as -inf; the selected ones are written in
 * ascending position.
 * block = 1:  indices (device) int32 [batch, s_q, topk]: absolute cache rows
 *             page * 64 + offset, -1 behind the last one: the `indices` of
 *             mla_decode_with_kvcache. lens (device, optional) int32
 *             [batch, s_q]: how many are selected.
 * block = 64: indices: physical pages, -1 behind the last one; lens (required)
 *             the tokens they hold. The last visible page always takes part and
 *             comes last, so (indices, lens) are a block table [batch * s_q,
 *             topk] and the cache_seqlens of a paged decode with one query per
 *             request (batch * s_q requests, s_q = 1; a decode takes up to 8192
 *             requests).
 * A row with no visible token gets -1 everywhere and lens 0. An out-of-range
 * page yields -1 in its place and an index error in `status`.
 */
MLA_API mla_status mla_select_topk(const float* scores, int64_t score_stride, int width,
                                   const int32_t* cache_seqlens, int batch, int s_q, int causal, int block, int topk,
                                   const int32_t* block_table, int max_blocks, int64_t num_blocks, int page_block,
                                   int32_t* indices, int32_t* lens, uint32_t* status, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Prompts over the paged latent cache: the norms of the projections with the
 * rotary positions in the same pass, the normalised append, cached rows read
 * back in 16 bits, and the attention of many new tokens. The pages stop at the
 * decode; these calls are this library's own. The conventions of the calls
 * above hold (positions and table, slots, status, strides, no shared memory
 * between an output and another argument but where it is named).
 *
 * RMS norm of a row of d values: y = x * (1 / sqrt(mean(x^2) + eps)) * weight, in
 * fp32 (the sum of squares too), with weight (device, 16-B aligned) of the row's
 * type or NULL for ones. y stays in fp32 through the rotation or quantisation
 * that follows and is rounded once, to the type it is stored in. eps >= 0. The sum of
 * squares has to lie within fp32 (rows of bf16 beyond some 2^59 are outside, and, with
 * eps = 0, those below some 2^-60 and rows of zeros); the product with the weight may lie
 * anywhere that y does.
 */

/*
 * Norm and rotation of queries or keys for each head: x (device) [tokens, heads,
 * dim] with token and head strides, dim a multiple of 8 from 64 to 576 (above:
 * MLA_ERR_UNSUPPORTED); the norm is over all dim values, then dims [rope_at,
 * rope_at + 64) are turned (rope_at a multiple of 8).
 * out (device) [tokens, heads, dim], or, with rope_out, the dim - 64 other values
 * of each row side by side, rope_out [tokens, heads, 64] taking the turned ones:
 * a decode's query wants the others dense for mla_absorb_q and the turned ones
 * in dims [512, 576) of its own rows. out may be x itself (in place, without
 * rope_out); with dim 64 and rope_out, out is not read and may be NULL.
 */
MLA_API mla_status mla_norm_rotate(const void* x, int64_t x_token_stride, int64_t x_head_stride, const void* weight,
                                   float eps, int dim, int rope_at, void* out, int64_t out_token_stride,
                                   int64_t out_head_stride, void* rope_out, int64_t rope_token_stride,
                                   int64_t rope_head_stride, int dtype, const int32_t* positions,
                                   const float* rope_table, int64_t max_positions, int rope_style, int64_t tokens,
                                   int heads, uint32_t* status, void* stream);

/*
 * mla_append_kv with the latent dims normalised on the way (the norm is over the
 * 512 latent dims of a token, 448 for V4.1 rows; the RoPE dims take no part).
 * Quantised rows are formed from the norm's fp32 values.
 * rows_out (device, optional) [n, 576] (V4.1 rows: 512) of `dtype`, rows
 *          rows_stride apart: the same rows as a 16-bit cache would hold them,
 *          for the prompt's own attention; skipped tokens leave theirs as it was.
 */
MLA_API mla_status mla_norm_append_kv(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t r_stride,
                                      const void* weight, float eps, int dtype, const int32_t* slots,
                                      const int32_t* positions, const float* rope_table, int64_t max_positions,
                                      int rope_style, int64_t n, void* kvcache, int64_t num_blocks, int page_block,
                                      int kv_format, void* rows_out, int64_t rows_stride, uint32_t* status,
                                      void* stream);

/*
 * Rows of the cache read back in 16 bits, packed: row o of out, offsets[b] <= o <
 * offsets[b + 1], is token starts[b] + o - offsets[b] of request b (starts NULL:
 * 0). Values are code x scale, formed in fp32 and rounded once to `dtype`; 16-bit
 * rows are copied (`dtype` is the cache's type then).
 * offsets (device) int32 [batch + 1], ascending; starts (device) int32 [batch].
 * out     (device) [total, 576] (V4.1 rows: 512, the last 64 of them RoPE dims),
 *         rows out_stride apart. Rows before offsets[0] and behind offsets[batch]
 *         are left as they were; offsets behind `total` are not written.
 * A token whose page is out of range, or lies behind its block-table row, reads
 * as zeros and is recorded as an index error in `status`.
 */
MLA_API mla_status mla_read_kv(const void* kvcache, int64_t num_blocks, int page_block, int kv_format,
                               const int32_t* block_table, int max_blocks, const int32_t* offsets,
                               const int32_t* starts, int batch, int64_t total, void* out, int64_t out_stride,
                               int dtype, uint32_t* status, void* stream);

/*
 * Attention of many new tokens in the expanded form: documents b of packed rows
 * cu_seqlens_q[b] .. cu_seqlens_q[b + 1] (n_q queries) and cu_seqlens_k[b] ..
 * cu_seqlens_k[b + 1] (n_k keys). For query i of document b and head h:
 *     s_j = softmax_scale (q[i, h, 0:128] . k_nope[j, h] + q[i, h, 128:192] . k_rope[j])
 *     out[i, h] = sum_j softmax(s)_j v[j, h],   lse[i, h] = ln sum_j exp s_j
 * over its visible keys j: all n_k, or with `causal` those below n_k - n_q + i + 1
 * (the last query sees all keys), but at least the first prefix_lens[b] (a prefix
 * that all queries see). A query that sees no key gets out = 0, lse = -inf.
 * softmax_scale lies between 2^-100 and 2^100. The dots q . k are summed in fp32; scaled
 * scores may lie beyond its range (out is right then, lse infinite). A query with a dot above
 * that range, or none of whose dots lies within it, gets NaN.
 * Softmax and sums are fp32; the weights are rounded to `dtype` for the product with v, where
 * fp16 loses those below 2^-32 of the query's largest.
 * Per (query, key) pair 640 FLOP a head, where the decode's absorbed form takes
 * 2176: the form for prompts and their chunks; keys and values come from the
 * latent rows by the model's up-projections.
 * q      (device) [tokens_q, heads, 192], `dtype`, any token and head strides of at
 *        least a row (a head stride of 0, shared heads, is refused).
 * k_nope, v (device) [tokens_k, heads, 128] likewise (column ranges of one
 *        projection are fine); k_rope (device) [tokens_k, 64], rotated, shared by
 *        the heads. What stands behind a document's keys does not matter, and a key
 *        that is not finite reaches only the queries that see it. A value that is not
 *        finite reaches them too, and, as 0 times it is NaN, may reach queries that
 *        miss its key by less than 383 keys.
 * cu_seqlens_q, cu_seqlens_k (device) int32 [batch + 1], ascending; prefix_lens
 *        (device, optional) int32 [batch], kept within [0, n_k]; not read unless
 *        causal. A document whose offsets descend or leave the tensors is skipped
 *        and recorded as an index error in `status` (with tokens_q = 0 nothing is
 *        looked at). Where offsets of queries descend, documents behind may share
 *        rows with others: what their rows hold then is not defined.
 * out    (device) [tokens_q, heads, 128] with strides; lse (device) fp32 [tokens_q,
 *        heads]. Rows of no document are left as they were.
 * workspace (device, 16-B aligned) of mla_prefill_workspace_size() bytes (0: none
 *        needed), for the call alone until it has run; its contents do not matter.
 */
MLA_API size_t mla_prefill_workspace_size(int64_t tokens_q, int64_t tokens_k, int batch, int heads);
MLA_API mla_status mla_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_nope,
                               int64_t k_token_stride, int64_t k_head_stride, const void* k_rope, int64_t rope_stride,
                               const void* v, int64_t v_token_stride, int64_t v_head_stride, int dtype,
                               const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, const int32_t* prefix_lens,
                               int batch, int64_t tokens_q, int64_t tokens_k, int heads, float softmax_scale,
                               int causal, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                               void* workspace, size_t workspace_bytes, uint32_t* status, void* stream);

/*
 * Synchronise `stream`, read and clear the status word of `workspace` (or of
 * any 4-B status word, e.g. the one given to mla_absorb_q), and return the
 * first error it records, in the order timeout, stale metadata, index, range
 * (MLA_OK if none). *bits (optional) receives the raw bits: 1 = index/page
 * skipped, 2 = wait timeout, 4 = stale metadata, 8 = range of a quantised cache.
 */
MLA_API mla_status mla_read_status(void* workspace, void* stream, uint32_t* bits);

/*
 * Test hook for the time-out path (0, the default, turns it off). While it is
 * non-zero, every decode kernel (mla_decode_with_kvcache and its variants),
 * absorption kernel (mla_absorb_q, mla_up_project), index score and prompt attention
 * (mla_prefill) launched by this library first has one thread per CTA wait `cycles` SM cycles on a barrier
 * that nothing arrives at, before any copy or MMA is issued; the wait gives up, the kernel records the wait
 * time-out (status bit 2, MLA_ERR_TIMEOUT) and the CTA skips its work, so the
 * outputs of those launches are undefined. Process-wide; not for production
 * use. The pages describe no such hook: it exists so that a test can check that
 * a device wait which runs out is reported and leaves the context usable.
 */
MLA_API void mla_set_test_stall(uint32_t cycles);

#ifdef __cplusplus
}
#endif
#endif /* MLA_GB300_H_ */
