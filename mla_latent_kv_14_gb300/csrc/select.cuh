// select.cuh -- the topk best of each query's scores, as the index list of the
// token-sparse decode or as the page list (block table and length) of the
// paged decode.
//
// NaN counts as -inf, -0 equals +0, ties at the threshold go to the lowest
// positions. The output is in ascending position: the attention's gathers run
// forward through memory, and with pages the last visible page (the only one
// that may be partly filled) comes last. That page always takes part: it is
// set apart, and topk - 1 are selected from the others.
//
// Measured (GB300): 4 x 1024 rows of up to 16384 scores, topk an eighth, 106 us
// (the read alone 43 us; 64 % of the issue slots busy), of up to 8192 51, 2048 25,
// 4096 rows of 512 21; 32 rows of 131072, topk 2048, 13.2 us, 64 rows of up to 512
// pages 4.9 us: there, and in the short rows, the steps'
// latencies, of 1 to 2 us for a cluster's barriers and remote reads.
//
// The floor is one read of the visible scores. A row is therefore loaded once
// and stays in registers (up to 32 scores per thread); a row longer than one
// block holds is shared by a cluster of up to 8 blocks through distributed
// shared memory. Only rows beyond 8 x 16384 scores are read again (from L2).
// Beyond the read, the sweeps over the held scores bound the kernel (the ALU
// pipe), so they are few and short, without branches or range tests (the
// padding behind a row is NaN, which fails every comparison):
//  1. a sample of two scores a thread brackets the threshold between two values;
//  2. sweep: the scores from the lower value on are counted in bins, equal steps
//     of value (two a thread); one fma gives a score's bin. Bins of equal steps
//     spread the shared memory atomics, where the digits of a radix select do
//     not (its first histogram has all scores in a few bins, and its atomics
//     queue). Scores below count in bins that are not read: a condition on
//     the atomic is a branch and a reconvergence in every step (106 us for the
//     first case above, 113 with it; a loop over marked scores alone: 137);
//  3. sweep: each lane marks its scores above the bin with the threshold and in
//     it; the latter, a handful, are listed and compared with one another;
//  4. the marks, transposed within a warp, are the selected columns in their
//     order; they are written through shared memory as whole lines.
// A sample that misled, or a bin of too many equal scores, falls back on a
// radix select by digits of 11, 11 and 10 bits of the scores' ordered keys.
#pragma once
#include <type_traits>

#include "params.h"
#include "ptx.cuh"

namespace mla {
namespace select {

constexpr int kMaxWarps = 16;                    // of a block
constexpr int kBins = 2048;                      // of a digit
constexpr int kStage = 3 * kBins;                // columns written through shared memory
constexpr int kMaxKeys = 32;                     // scores per thread
constexpr int kBlockKeys = 32 * kMaxWarps * kMaxKeys;  // scores that one block holds
constexpr int kMaxCluster = 8;

struct SelectParams {
  const float* scores;         // rows `stride` floats apart
  int64_t stride;
  int width;                   // columns of a row
  const int32_t* seqlens;      // [batch]
  const int32_t* block_table;  // [batch, max_blocks]
  int64_t num_blocks;
  int max_blocks, batch, s_q, causal, topk;
  int cluster_log2;            // blocks of a row
  int32_t* indices;            // [batch * s_q, topk]
  int32_t* lens;               // [batch * s_q], or null (tokens only)
  uint32_t* status;            // or null
};

// order-preserving key: unsigned comparison of keys is the order of values.
// -inf is 0x007FFFFF; keys below it stand for no score.
MLA_DEV uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(fmaxf(x, -INFINITY) + 0.0f);  // NaN -> -inf; -0 + 0 = +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
MLA_DEV float key_score(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

MLA_DEV uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
MLA_DEV int2 ld_cluster_int2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// adds 1 at a shared memory address
MLA_DEV void red_shared(uint32_t addr) {
  asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(addr) : "memory");
}
// bit k of lane l -> bit l of lane k
MLA_DEV uint32_t warp_transpose(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 16; j; j >>= 1) {
    const uint32_t low = 0xFFFFFFFFu / ((1u << j) + 1u);  // the lower j bits of every 2 j
    const bool up = lane & j;
    const uint32_t keep = up ? ~low : low, y = __shfl_xor_sync(0xffffffffu, x, j);
    x = (x & keep) | (__funnelshift_l(y, y, up ? 32 - j : j) & ~keep);
  }
  return x;
}

template <int kLanes = 32>
MLA_DEV int warp_inclusive(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// kKeys: scores per thread held in registers; 0: read again in each sweep
// kWarps: of a block; clusters have 16
template <bool kPages, int kKeys, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps) mla_select_topk_kernel(const SelectParams p) {
  constexpr int kThreads = 32 * kWarps, kWarpsLog2 = kWarps == 16 ? 4 : kWarps == 8 ? 3 : 2;
  static_assert(kWarps == 1 << kWarpsLog2, "");
  constexpr int kFine = 2 * kThreads;  // bins of the bracketed range
  constexpr int kBelow = 32;           // counters before the first bin
  constexpr int kList = 2 * kThreads;  // scores of one bin that are compared pairwise
  constexpr bool kClusters = kWarps == kMaxWarps && (kKeys == 0 || kKeys >= 16);
  __shared__ __align__(16) int hist[3][kBins];   // digits; then the staged columns
  __shared__ __align__(16) int fine_all[kBelow + kFine];  // counts of scores below the bracket, then the bins
  int* fine = fine_all + kBelow;
  __shared__ __align__(16) uint32_t list[kList];
  __shared__ uint32_t own_list[kClusters ? kList : 1];  // this block's share of it (of a cluster)
  __shared__ int warp_sum[kWarps];
  __shared__ int found[3];                       // bin, how many of it are selected, its size
  __shared__ int list_count;
  __shared__ int bracket[2];                     // digits: the lower end's, the upper end's
  __shared__ __align__(8) int2 warp_count[kWarps];
  __shared__ __align__(8) int2 block_count;      // scores above the threshold, scores equal to it
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cluster_log2 = kClusters ? p.cluster_log2 : 0, cluster = 1 << cluster_log2;
  const int rank = cluster > 1 ? (int)cluster_ctarank() : 0;
  const uint32_t r = blockIdx.x >> cluster_log2;  // below 2^28 (checked on the host)
  for (int c = threadIdx.x; c < kFine / 4; c += kThreads) reinterpret_cast<int4*>(fine)[c] = make_int4(0, 0, 0, 0);
  for (int c = threadIdx.x; c < kList / 4; c += kThreads) reinterpret_cast<int4*>(list)[c] = make_int4(0, 0, 0, 0);
  for (int c = threadIdx.x; c < kBins / 4; c += kThreads) reinterpret_cast<int4*>(hist)[c] = make_int4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    list_count = 0;
    found[0] = -1;
    bracket[0] = bracket[1] = -1;
  }
  pdl_wait();
  const int b = (int)(r / (uint32_t)p.s_q), i = (int)(r - (uint32_t)b * (uint32_t)p.s_q);
  const int len = __ldg(p.seqlens + b);
  int seen = p.causal ? len - (p.s_q - 1 - i) : len;
  seen = seen < 0 ? 0 : seen;
  // columns that the row and the block table reach
  const int64_t cover = min((int64_t)p.width * (kPages ? kTile : 1), (int64_t)p.max_blocks * kTile);
  if (seen > cover) {
    seen = (int)cover;
    if (rank == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, STATUS_INDEX);
  }
  const int visible = kPages ? (seen + kTile - 1) / kTile : seen;
  const int chosen_all = min(visible, p.topk);
  const int apart = kPages && visible > 0 ? 1 : 0;  // the last page, set apart
  const int n = visible - apart, count = chosen_all - apart;
  const bool all = count == n, none = count == 0;
  // each warp owns a contiguous range of whole 32-column steps
  const int ranges_log2 = cluster_log2 + kWarpsLog2;
  const int per_warp = (((n - 1) >> ranges_log2) + 32) & ~31;  // ceil(n / ranges), in whole steps; 0 for none
  const int c0 = min((rank * kWarps + warp) * per_warp, n), c1 = min(c0 + per_warp, n);
  const int steps = (c1 - c0 + 31) >> 5;
  // the block-table entries of what this lane or block may select, on their way
  // before they are needed: the page of the lane's 32 columns, or all pages
  const int32_t* table = p.block_table + (int64_t)b * p.max_blocks;
  constexpr bool kPagesHere = kPages && kKeys > 0 && kThreads * kKeys <= 2048;  // one block of up to 2048 pages
  __shared__ int page_ids[kPagesHere ? kThreads * kKeys : 1];
  int lane_page = 0;
  if (kPagesHere) {
    for (int c = threadIdx.x; c < n; c += kThreads) page_ids[c] = __ldg(table + c);
  } else if (!kPages && kKeys > 0 && c0 + 32 * lane < c1) {
    lane_page = __ldg(table + (c0 + 32 * lane) / kTile);
  }
  const float* first_score = p.scores + (int64_t)r * p.stride;
  const float* row = first_score + c0 + lane;
  const float kNan = __uint_as_float(0x7FFFFFFFu);
  const int mine = c1 - c0 - lane;  // step s is inside for this lane if 32 s < mine
  float held[kKeys > 0 ? kKeys : 1];
  if (kKeys > 0 && !all && !none) {
#pragma unroll
    for (int s = 0; s < kKeys; ++s) held[s] = 32 * s < mine ? __ldg(row + 32 * s) : kNan;
  }
  auto score_at = [&](int s) { return 32 * s < mine ? __ldg(row + 32 * s) : kNan; };
  // f(score, step) over the warp's steps and the padding behind them
  auto sweep = [&](auto&& f) {
    if (kKeys > 0) {
#pragma unroll
      for (int s = 0; s < kKeys; ++s) f(held[s], s);
    } else {
#pragma unroll 4
      for (int s = 0; s < steps; ++s) f(score_at(s), s);
    }
  };
  // The sample: 32 scores from the start and 32 from the middle of each warp's
  // range where the block has the whole row, else scores spread over the row,
  // the same for every block.
  uint32_t probe[2] = {0u, 0u};
  int samples = 2 * kThreads;
  if (!all && !none) {
    if (kKeys > 0 && cluster == 1) {
      const int middle = per_warp >> 6 << 5;  // 0: a range of one step
      if (middle > 0 && middle < mine) probe[1] = score_key(__ldg(row + middle));
      if (0 < mine) probe[0] = score_key(held[0]);
      const int full = (int)((uint32_t)n / (uint32_t)per_warp), rest = n - full * per_warp;
      samples = full * (middle > 0 ? 64 : 32) + min(rest, 32) + (middle > 0 ? min(max(rest - middle, 0), 32) : 0);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        probe[k] = score_key(__ldg(first_score + (int)((int64_t)n * (2 * (int)threadIdx.x + k) / (2 * kThreads))));
    }
  }
  __syncthreads();

  auto sync_row = [&]() {  // all blocks of the row
    __syncwarp();
    if (cluster > 1) cluster_sync();
    else __syncthreads();
  };
  // exclusive prefix of v over the block's threads
  auto before_in_block = [&](int v) {
    const int incl = warp_inclusive(v);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    const int w = lane < kWarps ? warp_sum[lane] : 0;
    return __shfl_sync(0xffffffffu, warp_inclusive<kWarps>(w) - w, warp) + incl - v;
  };
  // `h`: this block's histogram of kPer x kThreads bins. Finds, from the top
  // bin of the row's sum down, the one that reaches `need`.
  auto find_bin = [&](auto per, const int* h, int need) {
    constexpr int kPer = decltype(per)::value;
    const int top = kPer * (kThreads - 1 - (int)threadIdx.x);  // this thread's bins, the highest ones first
    int v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = 0;
    if (kClusters && cluster > 1) {
      const uint32_t addr = smem_u32(h + top);
      int2 part[kMaxCluster][kPer / 2];
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q)
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k)
          part[q][k] = q < cluster ? ld_cluster_int2(mapa(addr + 8 * k, q)) : make_int2(0, 0);
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q)
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
          v[2 * k] += part[q][k].x;
          v[2 * k + 1] += part[q][k].y;
        }
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = h[top + k];
    }
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum += v[k];
    int above = before_in_block(sum);
    if (above < need && need <= above + sum) {
#pragma unroll
      for (int k = kPer - 1; k >= 0; --k) {
        if (above < need && need <= above + v[k]) {
          found[0] = top + k;
          found[1] = need - above;
          found[2] = v[k];
        }
        above += v[k];
      }
    }
    __syncthreads();
  };

  // ---- the threshold: scores above it are selected, and `ties` of those equal to it ----
  uint32_t threshold = 0;  // a key
  int ties = 0;
  bool by_value = false;   // found by value: no NaN and no padding is selected or tied
  uint32_t above_marks = 0, in_marks = 0, lane_key = 0;  // held scores above the threshold's bin, in it; the last of those
  if (!all && !none) {
    // 1. the sample's histogram by the top digit of the keys
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (probe[k]) atomicAdd(&hist[0][probe[k] >> 21], 1);
    __syncthreads();
    {
      // Around the threshold's share of the sample: a quarter more and a few at
      // the lower end, about four standard deviations of that share at any
      // topk; half of it and a few fewer at the upper end.
      const int share = (int)(__fdividef((float)count, (float)n) * (float)samples);
      const int most = min(share + share / 4 + 8, samples), least = max(share / 2 - 8, 1);
      constexpr int kPer = kBins / kThreads;
      const int top = kPer * (kThreads - 1 - (int)threadIdx.x);
      int v[kPer], sum = 0;
#pragma unroll
      for (int k = 0; k < kPer; k += 4) {
        const int4 h4 = *reinterpret_cast<const int4*>(hist[0] + top + k);
        v[k] = h4.x;
        v[k + 1] = h4.y;
        v[k + 2] = h4.z;
        v[k + 3] = h4.w;
        sum += h4.x + h4.y + h4.z + h4.w;
      }
      int above = before_in_block(sum);
      if (sum > 0) {
#pragma unroll
        for (int k = kPer - 1; k >= 0; --k) {
          if (above < most && most <= above + v[k]) bracket[0] = top + k;
          if (above < least && least <= above + v[k]) bracket[1] = top + k;
          above += v[k];
        }
      }
      __syncthreads();
    }
    // Bin of a score: its distance from the lower end in steps, added to 2^23,
    // where an fp32 sum rounds to an integer: a monotone function of the score
    // (one fma). What is above the upper end joins the last bin.
    constexpr float kBase = 8388608.0f;
    const float low = key_score((uint32_t)bracket[0] << 21), high = key_score((uint32_t)(bracket[1] + 1) << 21);
    const float scale = (float)(kFine - 2) / (high - low), bias = kBase - low * scale;
    // false for the digits around zero, inf and NaN (and for no digit at all)
    const bool usable = scale > 1e-30f && scale < 1e30f && fabsf(bias) < 2.0f * kBase;
    if (usable) {
      constexpr float kLast = kBase + (kFine - 1);
      // 2. the bins
      const uint32_t fine_at = smem_u32(fine) - 4u * __float_as_uint(kBase);
      // below 2^23 fp32 steps by halves: lane l's scores there count from bin l - 32 on, in -1 at most
      static_assert(__builtin_bit_cast(uint32_t, kBase) - __builtin_bit_cast(uint32_t, kBase - 0.5f * kBelow) == kBelow, "");
      const float least = kBase - 0.5f * (float)(kBelow - lane);
      sweep([&](float x, int s) {
        (void)s;
        const float f = fminf(fmaxf(fmaf(x, scale, bias), least), kLast);  // NaN: least
        red_shared(fine_at + 4u * __float_as_uint(f));
      });
    }
    sync_row();
    if (usable) find_bin(std::integral_constant<int, kFine / kThreads>(), fine, count);
    const int bin = found[0], need = found[1], size = found[2];
    if (usable && bin >= 0 && bin < kFine - 1 && size <= kList) {
      // 3. the bin's scores, compared pairwise
      const float in_bin = kBase + (float)bin;
      uint32_t* to = kClusters && cluster > 1 ? own_list : list;
      if (kKeys > 0) {
        // bit s: the lane's score of step s lies above the bin, or in it
        uint32_t from = 0;
        sweep([&](float x, int s) {
          const float f = fmaf(x, scale, bias);
          from |= f >= in_bin ? 1u << s : 0u;
          in_marks |= f == in_bin ? 1u << s : 0u;
        });
        above_marks = from & ~in_marks;
        // few lanes have one in the bin: taken from the registers where that is no loop, else read again
        if (kKeys == 4) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (in_marks >> s & 1u) to[atomicAdd(&list_count, 1)] = score_key(held[s % (kKeys > 0 ? kKeys : 1)]);
        } else {
          for (uint32_t marks = in_marks; marks; marks &= marks - 1u) {
            lane_key = score_key(__ldg(row + 32 * (__ffs(marks) - 1)));
            to[atomicAdd(&list_count, 1)] = lane_key;
          }
        }
      } else {
        for (int s0 = 0; s0 < steps; s0 += 32) {
          uint32_t marks = 0;
#pragma unroll 4
          for (int s = s0; s < min(s0 + 32, steps); ++s)
            marks |= fmaf(score_at(s), scale, bias) == in_bin ? 1u << (s - s0) : 0u;
          for (; marks; marks &= marks - 1u)
            to[atomicAdd(&list_count, 1)] = score_key(__ldg(row + 32 * (s0 + __ffs(marks) - 1)));
        }
      }
      sync_row();
      if (cluster > 1) {
        // warp q copies block q's share behind those of the blocks before it
        const int m = lane < cluster ? (int)ld_cluster_u32(mapa(smem_u32(&list_count), lane)) : 0;
        const int upto = warp_inclusive(m), own = __shfl_sync(0xffffffffu, m, warp & 7);
        const int before = __shfl_sync(0xffffffffu, upto, warp & 7) - own;
        if (warp < cluster)
          for (int k = lane; k < own; k += 32) list[before + k] = ld_cluster_u32(mapa(smem_u32(own_list + k), warp));
        __syncthreads();
      }
      for (int k = threadIdx.x; k < size; k += kThreads) {
        const uint32_t key = list[k];
        int more = 0, same = 0;
        for (int o = 0; o < size; o += 4) {  // the list's end is zero: below every key
          const uint4 other = *reinterpret_cast<const uint4*>(list + o);
          more += (other.x > key) + (other.y > key) + (other.z > key) + (other.w > key);
          same += (other.x == key) + (other.y == key) + (other.z == key) + (other.w == key);
        }
        if (more < need && need <= more + same) {  // every thread with this key writes the same
          found[0] = (int)key;
          found[1] = need - more;
          found[2] = same;
        }
      }
      __syncthreads();
      threshold = (uint32_t)found[0];
      ties = found[1] == found[2] ? -1 : found[1];  // -1: every one of them
      by_value = true;
    } else {
      // the radix select, of keys formed again in each pass
      int left = count;
      uint32_t prefix = 0, mask = 0;
      for (int c = threadIdx.x; c < 3 * kBins / 4; c += kThreads)
        reinterpret_cast<int4*>(hist)[c] = make_int4(0, 0, 0, 0);
      __syncthreads();
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int digit = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        int* h = hist[pass];
#pragma unroll 4
        for (int s = 0; s < steps; ++s) {
          const uint32_t key = 32 * s < mine ? score_key(__ldg(row + 32 * s)) : 0u;
          if (key && (key & mask) == prefix) atomicAdd(&h[(key >> digit) & (kBins - 1)], 1);
        }
        sync_row();
        find_bin(std::integral_constant<int, kBins / kThreads>(), h, left);
        prefix |= (uint32_t)found[0] << digit;
        mask |= (uint32_t)(kBins - 1) << digit;
        left = found[1];
        threshold = prefix;
        ties = left;
        if (left == found[2]) {  // the whole bin: every key from its lowest on
          threshold = prefix - 1u;
          ties = 0;
          break;
        }
      }
    }
  }

  // ---- compaction in ascending position ----
  // A step's ballots are the bits of 32 consecutive columns; lane l keeps those
  // of step l (and, where the scores are read again, l + 32, ... in later rounds).
  int32_t* out = p.indices + (int64_t)r * p.topk;
  int* stage = &hist[0][0];
  // the columns first + (set bits), to dst[at ...]
  auto emit = [&](uint32_t bits, int first, int32_t* dst, int at) {
    int page = lane_page;
    bool good = true;
    if (!kPages && bits) {  // 32 columns from a multiple of 32 lie on one page
      if (kKeys == 0 || all) page = __ldg(table + first / kTile);
      good = page >= 0 && page < p.num_blocks;
      if (!good && p.status) atomicOr(p.status, STATUS_INDEX);
      page = page * kTile + first % kTile;
    }
    while (bits) {
      const int k = __ffs(bits) - 1;
      bits &= bits - 1u;
      int value = page + k;
      if (kPages) {
        value = kPagesHere ? page_ids[first + k] : __ldg(table + first + k);
        good = value >= 0 && value < p.num_blocks;
        if (!good && p.status) atomicOr(p.status, STATUS_INDEX);
      }
      dst[at++] = good ? value : -1;
    }
  };
  if (all) {
    for (int c = c0 + 32 * lane; c < c1; c += 1024)
      emit(c1 - c >= 32 ? 0xFFFFFFFFu : (1u << (c1 - c)) - 1u, c, out, c);
  } else if (!none) {
    uint32_t m_gt = 0, m_eq = 0;
    const float level = key_score(threshold);
    auto vote_value = [&](float x, int s) {  // from the threshold on
      const uint32_t g = __ballot_sync(0xffffffffu, x >= level);
      m_gt = lane == (s & 31) ? g : m_gt;
    };
    auto vote_equal = [&](float x, int s) {
      const uint32_t q = __ballot_sync(0xffffffffu, x == level);
      m_eq = lane == (s & 31) ? q : m_eq;
    };
    auto vote_key = [&](float x, int s) {
      const uint32_t key = 32 * s < mine ? score_key(x) : 0u;
      const uint32_t g = __ballot_sync(0xffffffffu, key > threshold), q = __ballot_sync(0xffffffffu, key == threshold);
      m_gt = lane == (s & 31) ? g : m_gt;
      m_eq = lane == (s & 31) ? q : m_eq;
    };
    auto vote = [&](auto&& over) {
      if (by_value) {
        over(vote_value);
        if (ties >= 0) {
          over(vote_equal);
          m_gt &= ~m_eq;
        }
      } else {
        over(vote_key);
      }
    };
    int gt = 0, eq = 0;  // selected and tied columns of this lane's
    if (kKeys > 0) {
      if (by_value) {
        // the bin's own scores against the threshold
        uint32_t equal_marks = 0;
        const bool single = (in_marks & (in_marks - 1u)) == 0;
        auto place = [&](uint32_t key, uint32_t bit) {
          if (key > threshold || (key == threshold && ties < 0)) above_marks |= bit;
          else if (key == threshold) equal_marks |= bit;
        };
        if (kKeys == 4) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (in_marks >> s & 1u) place(score_key(held[s % (kKeys > 0 ? kKeys : 1)]), 1u << s);
        } else {
          for (uint32_t marks = in_marks; marks; marks &= marks - 1u)
            place(single ? lane_key : score_key(__ldg(row + 32 * (__ffs(marks) - 1))), marks & (0u - marks));
        }
        if (kKeys == 4) {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t g = __ballot_sync(0xffffffffu, above_marks >> s & 1u), q = __ballot_sync(0xffffffffu, equal_marks >> s & 1u);
            m_gt = lane == s ? g : m_gt;
            m_eq = lane == s ? q : m_eq;
          }
        } else {
          m_gt = warp_transpose(above_marks);
          if (ties >= 0) m_eq = warp_transpose(equal_marks);
        }
      } else {
        vote(sweep);
      }
      gt = __popc(m_gt);
      eq = __popc(m_eq);
    } else {
#pragma unroll 4
      for (int s = 0; s < steps; ++s) {
        const uint32_t key = 32 * s < mine ? score_key(__ldg(row + 32 * s)) : 0u;
        gt += ties < 0 ? key >= threshold : key > threshold;
        eq += ties > 0 && key == threshold;
      }
    }
    const int equal = ties > 0 ? ties : 0;
    int gt_before = warp_inclusive(gt), eq_before = equal ? warp_inclusive(eq) : 0;
    if (lane == 31) warp_count[warp] = make_int2(gt_before, eq_before);
    gt_before -= gt;
    eq_before -= equal ? eq : 0;
    __syncthreads();
    const int2 per = lane < kWarps ? warp_count[lane] : make_int2(0, 0);
    const int upto_gt = warp_inclusive<kWarps>(per.x), upto_eq = equal ? warp_inclusive<kWarps>(per.y) : 0;
    const int2 block = make_int2(__shfl_sync(0xffffffffu, upto_gt, kWarps - 1), __shfl_sync(0xffffffffu, upto_eq, kWarps - 1));
    gt_before += __shfl_sync(0xffffffffu, upto_gt - per.x, warp);
    if (equal) eq_before += __shfl_sync(0xffffffffu, upto_eq - per.y, warp);
    int2 ahead = make_int2(0, 0);  // in the blocks before this one
    if (cluster > 1) {
      if (threadIdx.x == 0) block_count = block;
      sync_row();
      const int2 c = lane < rank ? ld_cluster_int2(mapa(smem_u32(&block_count), lane)) : make_int2(0, 0);
      ahead.x = (int)__reduce_add_sync(0xffffffffu, (unsigned)c.x);
      ahead.y = (int)__reduce_add_sync(0xffffffffu, (unsigned)c.y);
    }
    auto selected_before = [&](int g, int q) { return g + min(q, equal); };
    const int start = selected_before(ahead.x, ahead.y);
    const int chosen = selected_before(ahead.x + block.x, ahead.y + block.y) - start;  // by this block
    const bool staged = chosen <= kStage;
    gt_before += ahead.x;
    eq_before += ahead.y;
    // of the scores equal to the threshold, the first `equal` of the row
    auto write = [&](int first, int g, int q) {
      if (m_eq) {
        const int take = min(max(equal - q, 0), __popc(m_eq));
        while (__popc(m_eq) > take) m_eq &= ~(0x80000000u >> __clz(m_eq));
      }
      const int at = selected_before(g, q);
      emit(m_gt | m_eq, first, staged ? stage : out, staged ? at - start : at);
    };
    if (kKeys > 0) {
      write(c0 + 32 * lane, gt_before, eq_before);
    } else {
      // the warp's columns 1024 at a time
      int g0 = __shfl_sync(0xffffffffu, gt_before, 0), q0 = __shfl_sync(0xffffffffu, eq_before, 0);
      for (int s0 = 0; s0 < steps; s0 += 32) {
        m_gt = m_eq = 0;
        vote([&](auto&& f) {
          for (int s = s0; s < min(s0 + 32, steps); ++s) f(score_at(s), s);
        });
        const int n_gt = __popc(m_gt), n_eq = __popc(m_eq);
        const int p_gt = warp_inclusive(n_gt), p_eq = warp_inclusive(n_eq);
        write(c0 + 32 * (s0 + lane), g0 + p_gt - n_gt, q0 + p_eq - n_eq);
        g0 += __shfl_sync(0xffffffffu, p_gt, 31);
        q0 += __shfl_sync(0xffffffffu, p_eq, 31);
      }
    }
    if (staged) {
      __syncthreads();
      for (int c = threadIdx.x; c < chosen; c += kThreads) out[start + c] = stage[c];
    }
  }
  if (rank == 0) {
    if (apart && threadIdx.x == 0) {
      const int page = __ldg(table + n);
      const bool good = page >= 0 && page < p.num_blocks;
      if (!good && p.status) atomicOr(p.status, STATUS_INDEX);
      out[count] = good ? page : -1;
    }
    for (int c = chosen_all + threadIdx.x; c < p.topk; c += kThreads) out[c] = -1;
    if (threadIdx.x == 0 && p.lens)
      p.lens[r] = !kPages ? chosen_all : chosen_all > 0 ? (chosen_all - 1) * kTile + seen - (visible - 1) * kTile : 0;
  }
  __syncwarp();
  if (cluster > 1) cluster_sync();  // no block leaves while another reads its shared memory
}

}  // namespace select
}  // namespace mla
