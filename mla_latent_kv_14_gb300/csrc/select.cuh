// select.cuh -- the topk best of each query's scores, as the index list of the
// token-sparse decode or as the page list (block table and length) of the
// paged decode.
//
// Scores are compared as 32-bit keys in the order of their values (NaN as
// -inf, -0 equal to +0). Ties at the threshold go to the lowest positions. The
// output is in ascending position: the attention's gathers run forward through
// memory, and with pages the last visible page (the only one that may be
// partly filled; it always takes part) comes last.
//
// The floor is one read of the visible scores. A row is therefore loaded once
// and its keys stay in registers (up to 32 per thread); a row longer than one
// block holds is shared by a cluster of up to 8 blocks through distributed
// shared memory. Only rows beyond 8 x 16384 scores are read again (from L2).
// What is left is the latency of the steps on those keys, most of it shared
// memory atomics:
//  1. a sample of 1024 scores gives a key that a few more than topk reach;
//  2. the keys from there on are counted in 1024 bins of equal key range (they
//     spread over the bins, where the digits of a key do not: a radix select's
//     first histogram has all scores in a few bins, and its atomics queue);
//  3. the keys of the bin with the threshold, a handful, are compared with one
//     another;
//  4. each warp's ballots of the selected keys are counted, and the columns
//     written through shared memory as whole lines.
// A sample that misled (or a bin of too many equal keys) falls back on a radix
// select by digits of 11, 11 and 10 bits.
#pragma once
#include <type_traits>

#include "params.h"
#include "ptx.cuh"

namespace mla {
namespace select {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxKeys = 32;                     // per thread
constexpr int kBlockKeys = kThreads * kMaxKeys;  // scores that one block holds
constexpr int kMaxCluster = 8;
constexpr int kFine = 1024;                      // bins of the sampled range
constexpr int kList = 1024;                      // keys of one bin that are compared pairwise
constexpr int kStage = 3 * kBins;                // columns written through shared memory

struct SelectParams {
  const float* scores;         // rows `stride` floats apart
  int64_t stride;
  int width;                   // columns of a row
  const int32_t* seqlens;      // [batch]
  const int32_t* block_table;  // [batch, max_blocks]
  int64_t num_blocks;
  int max_blocks, batch, s_q, causal, topk;
  int cluster;                 // blocks of a row
  int32_t* indices;            // [batch * s_q, topk]
  int32_t* lens;               // [batch * s_q], or null (tokens only)
  uint32_t* status;            // or null
};

// order-preserving key: unsigned comparison of keys is the order of values
MLA_DEV uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(fmaxf(x, -INFINITY) + 0.0f);  // NaN -> -inf; -0 + 0 = +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
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

MLA_DEV int warp_inclusive(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// kKeys: scores per thread held in registers; 0: read again in each pass
template <bool kPages, int kKeys>
__global__ void __launch_bounds__(kThreads, 2) mla_select_topk_kernel(const SelectParams p) {
  __shared__ __align__(16) int hist[3][kBins];   // of the radix select; then the staged columns
  __shared__ __align__(16) int fine[kFine];
  __shared__ __align__(16) uint32_t list[kList];
  __shared__ uint32_t own_list[kList];           // this block's share of it (of a cluster)
  __shared__ int warp_sum[kWarps];
  __shared__ int found[3];                       // bin, how many of it are selected, its size
  __shared__ int list_count;
  __shared__ uint32_t range[2];                  // lowest key of the fine bins, their width as a shift
  __shared__ __align__(8) int2 warp_count[kWarps];
  __shared__ __align__(8) int2 block_count;      // keys above the threshold, keys equal to it
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = p.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int64_t r = p.cluster > 1 ? blockIdx.x / p.cluster : blockIdx.x;
  for (int c = threadIdx.x; c < kFine / 4; c += kThreads) reinterpret_cast<int4*>(fine)[c] = make_int4(0, 0, 0, 0);
  for (int c = threadIdx.x; c < kBins / 4; c += kThreads) reinterpret_cast<int4*>(hist)[c] = make_int4(0, 0, 0, 0);
  if (threadIdx.x == 0) {
    list_count = 0;
    found[0] = -1;
  }
  pdl_wait();
  const int b = (int)(r / p.s_q), i = (int)(r - (int64_t)b * p.s_q);
  const int len = __ldg(p.seqlens + b);
  int seen = p.causal ? len - (p.s_q - 1 - i) : len;
  seen = seen < 0 ? 0 : seen;
  // columns that the row and the block table reach
  const int64_t cover = min((int64_t)p.width * (kPages ? kTile : 1), (int64_t)p.max_blocks * kTile);
  if (seen > cover) {
    seen = (int)cover;
    if (rank == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, STATUS_INDEX);
  }
  const int n = kPages ? (seen + kTile - 1) / kTile : seen;
  const int count = n < p.topk ? n : p.topk;
  const bool all = count == n;
  // each warp owns a contiguous range of whole 32-column steps
  const int per_warp = ((n + p.cluster * kWarps - 1) / (p.cluster * kWarps) + 31) & ~31;
  const int c0 = min((rank * kWarps + warp) * per_warp, n), c1 = min(c0 + per_warp, n);
  const int steps = (c1 - c0 + 31) >> 5;
  const float* row = p.scores + r * p.stride + c0 + lane;
  // the last visible page takes part whatever its score; columns behind the
  // row have key 0, below every score's (that of -inf is 0x007FFFFF), so they
  // need no test: they are never above a threshold, equal to one, nor counted
  // in a bin that is looked at
  auto key_of = [&](int s) -> uint32_t {
    const int c = c0 + 32 * s + lane;
    if (c >= c1) return 0u;
    return kPages && c == n - 1 ? 0xFFFFFFFFu : score_key(__ldg(row + 32 * s));
  };
  // The sample: two of the warp's own scores per lane where the block has the
  // whole row, else scores spread over the row, the same for every block.
  uint32_t probe[2] = {0u, 0u};
  if (!all && (p.cluster > 1 || kKeys == 0)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = (int)((int64_t)n * (2 * (int)threadIdx.x + k) / (2 * kThreads));
      probe[k] = score_key(__ldg(p.scores + r * p.stride + c));
    }
  }
  uint32_t held[kKeys > 0 ? kKeys : 1];
  if (kKeys > 0 && !all) {
    float x[kKeys > 0 ? kKeys : 1];
#pragma unroll
    for (int s = 0; s < kKeys; ++s) x[s] = c0 + 32 * s + lane < c1 ? __ldg(row + 32 * s) : 0.f;
#pragma unroll
    for (int s = 0; s < kKeys; ++s) {
      const int c = c0 + 32 * s + lane;
      held[s] = c >= c1 ? 0u : kPages && c == n - 1 ? 0xFFFFFFFFu : score_key(x[s]);
    }
    if (p.cluster == 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k) probe[k] = held[k % (kKeys > 0 ? kKeys : 1)] == 0xFFFFFFFFu ? 0u : held[k % (kKeys > 0 ? kKeys : 1)];
    }
  }
  // f(key, step) over the warp's steps (and the padding behind them: no branches)
  auto for_keys = [&](auto&& f) {
    if (kKeys > 0) {
#pragma unroll
      for (int s = 0; s < kKeys; ++s) f(held[s], s);
    } else {
#pragma unroll 4
      for (int s = 0; s < steps; ++s) f(key_of(s), s);
    }
  };
  __syncthreads();

  auto sync_row = [&]() {  // all blocks of the row
    __syncwarp();
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
  };
  // `h`: this block's histogram of 4 x kThreads (kPer = 4) or 2 x kThreads bins.
  // Finds, from the top bin of the row's sum down, the one that reaches `need`.
  auto find_bin = [&](auto per, const int* h, int need) {
    constexpr int kPer = decltype(per)::value;
    const int top = kPer * (kThreads - 1 - (int)threadIdx.x);  // this thread's bins, the highest ones first
    int v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = 0;
    if (p.cluster > 1) {
      const uint32_t addr = smem_u32(h + top);
      int2 part[kMaxCluster][kPer / 2];
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q)
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k)
          part[q][k] = q < p.cluster ? ld_cluster_int2(mapa(addr + 8 * k, q)) : make_int2(0, 0);
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
    const int incl = warp_inclusive(sum);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int above = incl - sum;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w) above += w < warp ? warp_sum[w] : 0;
#pragma unroll
    for (int k = kPer - 1; k >= 0; --k) {
      if (above < need && need <= above + v[k]) {
        found[0] = top + k;
        found[1] = need - above;
        found[2] = v[k];
      }
      above += v[k];
    }
    __syncthreads();
  };

  // ---- the threshold: keys above it are selected, and `ties` of those equal to it ----
  uint32_t threshold = 0;
  int ties = 0;
  if (!all) {
    bool exact = false;
    // 1. the sample's histogram by the top digit; samples of the padding (key 0) fall into bin 0
#pragma unroll
    for (int k = 0; k < 2; ++k) atomicAdd(&hist[0][probe[k] >> 21], 1);
    __syncthreads();
    {
      // a quarter more of the sample than its share, and a few: about four
      // standard deviations of the share at any topk
      int samples = 2 * kThreads;
      if (kKeys > 0 && p.cluster == 1) {  // of each warp's range the first 64
        const int each = min(per_warp, 64);
        samples = n / per_warp * each + min(n % per_warp, each);
      }
      const int want = (int)(((int64_t)count * samples * 5) / ((int64_t)n * 4)) + 8;
      const int top = 4 * (kThreads - 1 - (int)threadIdx.x);
      const int4 h4 = *reinterpret_cast<const int4*>(hist[0] + top);
      const int v[4] = {h4.x, h4.y, h4.z, h4.w};
      const int sum = v[0] + v[1] + v[2] + v[3], incl = warp_inclusive(sum);
      if (lane == 31) warp_sum[warp] = incl;
      if (threadIdx.x == 0) range[0] = 0u;
      __syncthreads();
      int above = incl - sum;
#pragma unroll
      for (int w = 0; w < kWarps - 1; ++w) above += w < warp ? warp_sum[w] : 0;
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        if (above == 0 && v[k] > 0) range[1] = (uint32_t)(top + k);                              // highest digit
        if (above < want && want <= above + v[k]) range[0] = (uint32_t)(top + k) << 21;
        above += v[k];
      }
      __syncthreads();
    }
    const uint32_t low = range[0];
    // digits [low, highest] in kFine bins: a power of two wide
    const uint32_t digits = range[1] - (low >> 21) + 1u;
    const int shift = 11 + (32 - __clz((int)(digits - 1u | 1u)));  // 2^shift * kFine >= digits * 2^21
    // 2. the fine histogram; what is above the sample's highest digit joins the last bin
    for_keys([&](uint32_t key, int s) {
      (void)s;
      if (key >= low) atomicAdd(&fine[min((key - low) >> shift, (uint32_t)kFine - 1u)], 1);
    });
    sync_row();
    find_bin(std::integral_constant<int, kFine / kThreads>(), fine, count);
    const int bin = found[0], need1 = found[1], size = found[2];
    if (bin >= 0) {
      const uint32_t first = low + ((uint32_t)bin << shift);
      const uint32_t last = bin == kFine - 1 ? 0xFFFFFFFFu : first + (1u << shift) - 1u;
      if (need1 == size) {  // the whole bin
        threshold = first - 1u;
        exact = true;
      } else if (size <= kList) {
        // 3. the bin's keys, compared pairwise
        uint32_t* mine = p.cluster > 1 ? own_list : list;
        const uint32_t span = last - first;
        if (kKeys > 0) {
          // few lanes have one: marked without a branch per step, then read again
          uint32_t marks = 0;
          for_keys([&](uint32_t key, int s) { marks |= key - first <= span ? 1u << s : 0u; });
          while (marks) {
            const int s = __ffs(marks) - 1;
            marks &= marks - 1u;
            mine[atomicAdd(&list_count, 1)] = key_of(s);
          }
        } else {
          for_keys([&](uint32_t key, int s) {
            (void)s;
            if (key - first <= span) mine[atomicAdd(&list_count, 1)] = key;
          });
        }
        sync_row();
        if (p.cluster > 1) {
          // warp q copies block q's share behind those of the blocks before it
          const int m = lane < p.cluster ? (int)ld_cluster_u32(mapa(smem_u32(&list_count), lane)) : 0;
          const int upto = warp_inclusive(m), own = __shfl_sync(0xffffffffu, m, warp & 7);
          const int before = __shfl_sync(0xffffffffu, upto, warp & 7) - own;
          if (warp < p.cluster)
            for (int k = lane; k < own; k += 32) list[before + k] = ld_cluster_u32(mapa(smem_u32(own_list + k), warp));
          __syncthreads();
        }
        for (int k = threadIdx.x; k < size; k += kThreads) {
          const uint32_t key = list[k];
          int more = 0, same = 0;
          for (int o = 0; o < size; ++o) {
            more += list[o] > key;
            same += list[o] == key;
          }
          if (more < need1 && need1 <= more + same) {  // every thread with this key writes the same
            const bool whole = need1 == more + same;
            found[0] = (int)(whole ? key - 1u : key);
            found[1] = whole ? 0 : need1 - more;
          }
        }
        __syncthreads();
        threshold = (uint32_t)found[0];
        ties = found[1];
        exact = true;
      }
    }
    if (!exact) {
      int need = count;
      uint32_t prefix = 0, mask = 0;
      for (int c = threadIdx.x; c < 3 * kBins / 4; c += kThreads)
        reinterpret_cast<int4*>(hist)[c] = make_int4(0, 0, 0, 0);
      __syncthreads();
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int digit = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        int* h = hist[pass];
        for_keys([&](uint32_t key, int s) {
          (void)s;
          if ((key & mask) == prefix) atomicAdd(&h[(key >> digit) & (kBins - 1)], 1);
        });
        sync_row();
        find_bin(std::integral_constant<int, kBins / kThreads>(), h, need);
        prefix |= (uint32_t)found[0] << digit;
        mask |= (uint32_t)(kBins - 1) << digit;
        need = found[1];
        if (need == found[2]) {  // the whole bin: every key from its lowest on
          threshold = prefix - 1u;  // prefix > 0: not every key is selected
          ties = 0;
          break;
        }
        threshold = prefix;
        ties = need;
      }
    }
  }

  // ---- compaction in ascending position ----
  // A step's ballots are the bits of 32 consecutive columns; lane l keeps those
  // of step l (and, where the keys are read again, l + 32, ... in later rounds).
  const int32_t* table = p.block_table + (int64_t)b * p.max_blocks;
  int32_t* out = p.indices + r * p.topk;
  int* stage = &hist[0][0];
  // the columns first + (set bits), to dst[at ...]
  auto emit = [&](uint32_t bits, int first, int32_t* dst, int at) {
    int page = 0;
    bool good = true;
    if (!kPages && bits) {  // 32 columns from a multiple of 32 lie on one page
      page = __ldg(table + first / kTile);
      good = page >= 0 && page < p.num_blocks;
      if (!good && p.status) atomicOr(p.status, STATUS_INDEX);
      page = page * kTile + first % kTile;
    }
    while (bits) {
      const int k = __ffs(bits) - 1;
      bits &= bits - 1u;
      int value = page + k;
      if (kPages) {
        value = __ldg(table + first + k);
        good = value >= 0 && value < p.num_blocks;
        if (!good && p.status) atomicOr(p.status, STATUS_INDEX);
      }
      dst[at++] = good ? value : -1;
    }
  };
  if (all) {
    for (int c = c0 + 32 * lane; c < c1; c += 1024)
      emit(c1 - c >= 32 ? 0xFFFFFFFFu : (1u << (c1 - c)) - 1u, c, out, c);
  } else {
    uint32_t m_gt = 0, m_eq = 0;
    auto vote = [&](uint32_t key, int s) {
      const uint32_t g = __ballot_sync(0xffffffffu, key > threshold);
      m_gt = lane == (s & 31) ? g : m_gt;
    };
    auto vote_equal = [&](uint32_t key, int s) {
      const uint32_t q = __ballot_sync(0xffffffffu, key == threshold);
      m_eq = lane == (s & 31) ? q : m_eq;
    };
    int gt = 0, eq = 0;  // selected and tied columns of this lane's
    if (kKeys > 0) {
      for_keys(vote);
      if (ties > 0) for_keys(vote_equal);
      gt = __popc(m_gt);
      eq = __popc(m_eq);
    } else {
      for_keys([&](uint32_t key, int s) {
        (void)s;
        gt += key > threshold;
        eq += key == threshold;
      });
    }
    int gt_before = warp_inclusive(gt), eq_before = ties > 0 ? warp_inclusive(eq) : 0;
    if (lane == 31) warp_count[warp] = make_int2(gt_before, eq_before);
    gt_before -= gt;
    eq_before -= ties > 0 ? eq : 0;
    __syncthreads();
    int2 block = make_int2(0, 0), lower = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int2 c = warp_count[w];
      lower.x += w < warp ? c.x : 0;
      lower.y += w < warp ? c.y : 0;
      block.x += c.x;
      block.y += c.y;
    }
    int2 ahead = make_int2(0, 0);  // in the blocks before this one
    if (p.cluster > 1) {
      if (threadIdx.x == 0) block_count = block;
      sync_row();
      const int2 c = lane < rank ? ld_cluster_int2(mapa(smem_u32(&block_count), lane)) : make_int2(0, 0);
      ahead.x = (int)__reduce_add_sync(0xffffffffu, (unsigned)c.x);
      ahead.y = (int)__reduce_add_sync(0xffffffffu, (unsigned)c.y);
    }
    auto selected_before = [&](int g, int q) { return g + (q < ties ? q : ties); };
    const int start = selected_before(ahead.x, ahead.y);
    const int chosen = selected_before(ahead.x + block.x, ahead.y + block.y) - start;  // by this block
    const bool staged = chosen <= kStage;
    gt_before += ahead.x + lower.x;
    eq_before += ahead.y + lower.y;
    // of the keys equal to the threshold, the first `ties` of the row
    auto write = [&](int first, int g, int q) {
      int take = ties - q;
      const int n_eq = __popc(m_eq);
      take = take < 0 ? 0 : take < n_eq ? take : n_eq;
      while (__popc(m_eq) > take) m_eq &= ~(0x80000000u >> __clz(m_eq));
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
        for (int s = s0; s < min(s0 + 32, steps); ++s) {
          const uint32_t key = key_of(s);
          vote(key, s);
          vote_equal(key, s);
        }
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
    for (int c = count + threadIdx.x; c < p.topk; c += kThreads) out[c] = -1;
    if (threadIdx.x == 0 && p.lens)
      p.lens[r] = !kPages ? count : count > 0 ? (count - 1) * kTile + seen - (n - 1) * kTile : 0;
  }
  __syncwarp();
  if (p.cluster > 1) cluster_sync();  // no block leaves while another reads its shared memory
}

}  // namespace select
}  // namespace mla
