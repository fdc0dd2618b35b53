// select.cuh -- the topk best of each query's scores, as the index list of the
// token-sparse decode or as the page list (block table and length) of the
// paged decode.
//
// Scores are compared as 32-bit keys in the order of their values (NaN below
// everything, -0 equal to +0); the threshold key is found digit by digit from
// histograms (a radix select), and ties at the threshold go to the lowest
// positions. The output is in ascending position: the attention's gathers run
// forward through memory, and with pages the last visible page (the only one
// that may be partly filled; it always takes part) comes last.
#pragma once
#include "params.h"
#include "ptx.cuh"

namespace mla {
namespace select {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;  // 11 bits a pass: 11 + 11 + 10

struct SelectParams {
  const float* scores;         // rows `stride` floats apart
  int64_t stride;
  int width;                   // columns of a row
  const int32_t* seqlens;      // [batch]
  const int32_t* block_table;  // [batch, max_blocks]
  int64_t num_blocks;
  int max_blocks, batch, s_q, causal, topk;
  int32_t* indices;            // [batch * s_q, topk]
  int32_t* lens;               // [batch * s_q], or null (tokens only)
  uint32_t* status;            // or null
};

// order-preserving key: unsigned comparison of keys is the order of values
MLA_DEV uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;  // NaN
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// exclusive prefix of `v` over the block's threads, and the block's total.
// `scratch`: kWarps words.
MLA_DEV int block_scan(int v, int* scratch, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  const int w = scratch[lane];  // kWarps == 32
  int wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += x;
  }
  total = __shfl_sync(0xffffffffu, wi, 31);
  return __shfl_sync(0xffffffffu, wi - w, warp) + incl - v;
}

template <bool kPages>
__global__ void __launch_bounds__(kThreads) mla_select_topk_kernel(const SelectParams p) {
  __shared__ int hist[kBins];
  __shared__ int scratch[kWarps];
  __shared__ int found[2];
  pdl_wait();
  const int64_t r = blockIdx.x;
  const int b = (int)(r / p.s_q), i = (int)(r - (int64_t)b * p.s_q);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = __ldg(p.seqlens + b);
  int seen = p.causal ? len - (p.s_q - 1 - i) : len;
  seen = seen < 0 ? 0 : seen;
  // columns that the row and the block table reach
  const int64_t cover = min((int64_t)p.width * (kPages ? kTile : 1), (int64_t)p.max_blocks * kTile);
  if (seen > cover) {
    seen = (int)cover;
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, STATUS_INDEX);
  }
  const int n = kPages ? (seen + kTile - 1) / kTile : seen;
  const float* row = p.scores + r * p.stride;
  const int count = n < p.topk ? n : p.topk;
  // the last visible page takes part whatever its score
  auto key_at = [&](int c) { return kPages && c == n - 1 ? 0xFFFFFFFFu : score_key(__ldg(row + c)); };

  // ---- the threshold: the smallest selected key, and how many equal to it are selected ----
  uint32_t threshold = 0;
  int ties = 0;  // selected among the keys equal to the threshold
  if (count < n) {
    int need = count;
    int shift = 21;
    uint32_t mask = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int bins = pass < 2 ? kBins : kBins / 2;
      for (int c = threadIdx.x; c < bins; c += kThreads) hist[c] = 0;
      __syncthreads();
      for (int c = threadIdx.x; c < n; c += kThreads) {
        const uint32_t key = key_at(c);
        if ((key & mask) == threshold) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // thread t holds bins from the top: the one where the count from above reaches `need`
      const int per = bins / kThreads;  // 2, or 1
      int mine = 0;
      for (int k = 0; k < per; ++k) mine += hist[bins - 1 - ((int)threadIdx.x * per + k)];
      int total;
      int above = block_scan(mine, scratch, total);
      for (int k = 0; k < per; ++k) {
        const int bin = bins - 1 - ((int)threadIdx.x * per + k), h = hist[bin];
        if (above < need && need <= above + h) {
          found[0] = bin;
          found[1] = need - above;
        }
        above += h;
      }
      __syncthreads();
      threshold |= (uint32_t)found[0] << shift;
      need = found[1];
      mask |= (uint32_t)(bins - 1) << shift;
      shift = pass == 0 ? 10 : 0;
      __syncthreads();
    }
    ties = need;
  }

  // ---- compaction in ascending position: each warp owns a contiguous range ----
  const int32_t* table = p.block_table + (int64_t)b * p.max_blocks;
  int32_t* out = p.indices + r * p.topk;
  const int span = ((n + kThreads - 1) / kThreads) * 32;  // columns of a warp
  const int c0 = min(warp * span, n), c1 = min(c0 + span, n);
  int above = 0, equal = 0;
  if (count < n) {
    for (int c = c0 + lane; c < c1; c += 32) {
      const uint32_t key = key_at(c);
      above += key > threshold;
      equal += key == threshold;
    }
  }
  const bool all = count == n;
  int total;
  int eq_before = block_scan(equal, scratch, total), gt_before = block_scan(above, scratch, total);
  // the warp's exclusive prefixes
  eq_before = __shfl_sync(0xffffffffu, eq_before, 0);
  gt_before = __shfl_sync(0xffffffffu, gt_before, 0);
  for (int base = c0; base < c1; base += 32) {
    const int c = base + lane;
    const uint32_t key = !all && c < c1 ? key_at(c) : 0u;
    const bool gt = c < c1 && (all || key > threshold), eq = !all && c < c1 && key == threshold;
    const uint32_t m_eq = __ballot_sync(0xffffffffu, eq), m_gt = __ballot_sync(0xffffffffu, gt);
    const uint32_t below = (1u << lane) - 1u;
    const int eq_rank = eq_before + __popc(m_eq & below);
    const int at = (all ? c : gt_before + __popc(m_gt & below) + min(eq_rank, ties));
    if (gt || (eq && eq_rank < ties)) {
      const int pg = __ldg(table + (kPages ? c : c / kTile));
      const bool good = pg >= 0 && pg < p.num_blocks;
      if (!good && p.status) atomicOr(p.status, STATUS_INDEX);
      out[at] = !good ? -1 : kPages ? pg : pg * kTile + c % kTile;
    }
    eq_before += __popc(m_eq);
    gt_before += __popc(m_gt);
  }
  for (int c = count + threadIdx.x; c < p.topk; c += kThreads) out[c] = -1;
  if (threadIdx.x == 0 && p.lens) p.lens[r] = !kPages ? count : count > 0 ? (count - 1) * kTile + seen - (n - 1) * kTile : 0;
}

}  // namespace select
}  // namespace mla
