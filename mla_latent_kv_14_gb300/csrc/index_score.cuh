// index_score.cuh -- the cheap score that picks tokens or pages for the sparse
// attention, sm_103a.
//
//     score[q, t] = ks_t * sum_h w[q, h] * max(0, q_h . k_t)
//
// over the visible tokens t of the query's request (ks_t the scale of an e4m3
// key, 1 otherwise), -inf elsewhere; or the maximum over each 64-token page.
//
// Tokens are the M dimension of the UMMA and (query, head) pairs its N
// dimension, so that the sum over heads runs inside one thread: a 128-token
// tile times a group of `nq` queries x `hp` heads (N = nq * hp <= 256, the
// heads padded to 16, 32 or 64) gives one accumulator, and epilogue thread t
// holds all N products of token t. The products of a group need 128 x N x 128
// multiplies, 1024 tensor cycles in 16-bit at N = 256; the epilogue spends one
// addition and half a packed fma on each product. A unit is one request's two
// groups (`G` = 2), which share each key tile: the tensor pipe multiplies one
// group while the warps sum the other. With few queries per request (decode)
// N is small and the keys' bytes bound the kernel.
//
// The (unit, tile) pairs of all requests form one list, cut into equal
// contiguous ranges, one per CTA (one CTA per SM): ragged lengths balance, and
// a unit's queries are loaded once per range.
//
// Warp roles (384 threads): warp 0 lane 0 issues TMA; warp 1 owns TMEM and
// lane 0 issues the MMAs; warp 2 writes the -inf columns behind the visible
// tiles; warp 3 brings the head weights; warps 4-7 and 8-11 are the two
// epilogue groups, serving accumulator 0 and 1. Every wait is bounded; a wait
// that gives up sets the status word and the CTA unwinds.
#pragma once
#include <cuda.h>

#include "params.h"
#include "ptx.cuh"

namespace mla {
namespace score {

constexpr int kThreads = 384;
constexpr int kTokens = 128;                    // tokens of a tile (two pages)
constexpr int kDim = 128;
constexpr int kMaxN = 256;
constexpr uint32_t kUnit = 16384;               // ring unit: 128 tokens x 128 B
constexpr int kMaxRing = 12;

struct ScoreParams {
  const float* weights;        // [batch, s_q, heads]
  const uint8_t* cache;
  const int32_t* block_table;  // [batch, max_blocks]
  const int32_t* seqlens;      // [batch]
  float* scores;               // [batch * s_q] rows, `stride` floats apart
  int64_t stride;
  int64_t num_blocks;
  int max_blocks, batch, s_q, heads, causal;
  int nq;                      // queries per group
  int groups;                  // groups per unit (1 or 2)
  int units;                   // units per request
  int cover;                   // tokens that the columns and the block table reach
  int width;                   // columns written (tokens or pages)
  int ring;                    // ring units
  uint32_t* status;            // or null
  uint32_t stall_cycles;       // test hook, 0 in normal use
};

// shared memory: the query groups, the key ring, weights, barriers
constexpr uint32_t kWeightBytes = 2 * 2 * kMaxN * 4;  // [unit parity][group][256]
constexpr uint32_t kRedBytes = 2 * 2 * 4 * 16 * 4;    // page maxima: [group][parity][4 warps][16 queries]
enum : uint32_t {
  B_KFULL = 0, B_KEMPTY = B_KFULL + kMaxRing, B_QFULL = B_KEMPTY + kMaxRing, B_QEMPTY = B_QFULL + 2,
  B_AFULL = B_QEMPTY + 2, B_AEMPTY = B_AFULL + 2, B_WFULL = B_AEMPTY + 2, B_WEMPTY = B_WFULL + 2,
  B_RED = B_WEMPTY + 2, B_DRAIN = B_RED + 2, B_STALL = B_DRAIN + 1, B_COUNT = B_STALL + 1
};
constexpr uint32_t kTailBytes = kWeightBytes + kRedBytes + 8 * B_COUNT + 64 + 64;
constexpr uint32_t smem_bytes(uint32_t q_bytes, uint32_t ring) { return q_bytes + ring * kUnit + kTailBytes + 1024; }

// visible tokens of query i of a request with `len` tokens
MLA_DEV int visible(const ScoreParams& p, int len, int i) {
  const int v = p.causal ? len - (p.s_q - 1 - i) : len;
  return v < 0 ? 0 : (v > p.cover ? p.cover : v);
}
// key tiles of a unit: those that its last query sees
MLA_DEV int unit_tiles(const ScoreParams& p, int u) {
  const int b = u / p.units, k = u - b * p.units;
  const int per = p.nq * p.groups;
  int last = (k + 1) * per - 1;
  last = last < p.s_q - 1 ? last : p.s_q - 1;
  return (visible(p, __ldg(p.seqlens + b), last) + kTokens - 1) / kTokens;
}

// The CTA's range of the list of (unit, tile) pairs, walked in order.
struct Walk {
  int u, t, n, left;  // unit, tile, tiles of the unit, pairs left
  MLA_DEV Walk(const ScoreParams& p, int u0, int t0, int count) : u(u0), t(t0), n(0), left(count) {
    if (left > 0) n = unit_tiles(p, u);
  }
  MLA_DEV bool done() const { return left <= 0; }
  MLA_DEV bool last_of_unit() const { return t == n - 1 || left == 1; }
  MLA_DEV void next(const ScoreParams& p) {
    --left;
    if (++t < n || left <= 0) return;
    t = 0;
    do n = unit_tiles(p, ++u); while (n == 0);  // left > 0: a later unit has tiles
  }
};

// D[tmem] (+)= A[smem] * B[smem], e4m3 operands, fp32 accumulation
MLA_DEV void umma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
MLA_DEV void tma_load_3d_plain(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

enum : int { K_BF16 = 0, K_FP16 = 1, K_FP8 = 2 };

// tm_q: dims {128, heads, batch * s_q}, box {128 B, hp, nq};
// tm_k: dims {128, 64, num_blocks}, box {128 B, 64, 1}; both 128-B swizzled.
template <int kType, int kHp, bool kPages>
__global__ void __launch_bounds__(kThreads, 1)
    mla_index_score_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const ScoreParams p) {
  constexpr int kChunks = kType == K_FP8 ? 1 : 2;        // 128-byte chunks of a row
  constexpr int kChunkElems = kType == K_FP8 ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = p.nq * kHp;
  const uint32_t q_chunk = (uint32_t)N * 128u, q_group = kChunks * q_chunk;
  const uint32_t off_ring = p.groups * q_group;          // a multiple of 1024 (N is one of 16)
  const uint32_t off_w = off_ring + (uint32_t)p.ring * kUnit;
  const uint32_t off_red = off_w + kWeightBytes;
  const uint32_t off_bar = off_red + kRedBytes;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + off_bar + 8 * B_COUNT);
  volatile uint32_t* tmem_slot = misc;
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* ok_flag = misc + 2;
  volatile int* range = reinterpret_cast<volatile int*>(misc + 4);  // first unit, first tile, pairs
  int* scan = reinterpret_cast<int*>(smem + off_w);                 // [12 warps], before the weights arrive
  auto bar = [&](uint32_t i) { return sb + off_bar + 8u * i; };
  uint32_t* status = p.status ? p.status : misc + 3;
  const Guard guard{abort_flag, status, kWaitLimitCycles};

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(bar(B_KFULL + s), 1);
      mbar_init(bar(B_KEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_QFULL + s), 1);
      mbar_init(bar(B_QEMPTY + s), 1);
      mbar_init(bar(B_AFULL + s), 1);
      mbar_init(bar(B_AEMPTY + s), 4);
      mbar_init(bar(B_WFULL + s), 1);
      mbar_init(bar(B_WEMPTY + s), 8);
      mbar_init(bar(B_RED + s), 4);
    }
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_STALL), 1);
    *abort_flag = 0u;
    misc[3] = 0u;
    range[0] = range[1] = range[2] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  pdl_wait();  // nothing above reads global memory

  // ---- this CTA's range: scan of the units' tiles ----
  const int total_units = p.batch * p.units;
  const int seg = (total_units + kThreads - 1) / kThreads;
  const int u_lo = min((int)threadIdx.x * seg, total_units), u_hi = min(u_lo + seg, total_units);
  int mine = 0;
  for (int u = u_lo; u < u_hi; ++u) mine += unit_tiles(p, u);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  if (threadIdx.x == 0) {
    *ok_flag = 1u;
    if (p.stall_cycles) {
      // test hook: a bounded wait on a barrier nothing arrives at gives up
      // and reports STATUS_TIMEOUT before anything is issued
      const Guard g_stall{abort_flag, status, p.stall_cycles};
      if (!wait(bar(B_STALL), 0, g_stall)) *ok_flag = 0u;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  {
    int before = incl - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int s = scan[w];
      if (w < warp) before += s;
      total += s;
    }
    const int64_t lo = (int64_t)total * blockIdx.x / gridDim.x, hi = (int64_t)total * (blockIdx.x + 1) / gridDim.x;
    if (lo >= before && lo < before + mine) {  // one thread holds the first pair
      int at = before, u = u_lo;
      for (; u < u_hi; ++u) {
        const int n = unit_tiles(p, u);
        if (lo < at + n) break;
        at += n;
      }
      range[0] = u;
      range[1] = (int)(lo - at);
      range[2] = (int)(hi - lo);
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const bool ok = *ok_flag != 0u;
  Walk it(p, range[0], range[1], ok ? range[2] : 0);

  if (warp == 0 && lane == 0 && !it.done()) {
    // ---------------- producer: a unit's query groups, then key tiles ----------------
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    int n = 0, units = 0, unit = -1, last_q[2] = {-1, -1};
    bool stop = false;
    for (; !stop && !it.done(); it.next(p)) {
      const int b = it.u / p.units;
      if (it.u != unit) {
        unit = it.u;
        const int q0 = (it.u - b * p.units) * p.nq * p.groups;
        for (int g = 0; g < p.groups && !stop; ++g) {
          // a last group behind the request's queries reads others (or the
          // zero fill); its products are never stored
          if (!wait(bar(B_QEMPTY + g), (units & 1) ^ 1, guard)) { stop = true; break; }
          mbar_arrive_expect_tx(bar(B_QFULL + g), q_group);
          for (int c = 0; c < kChunks; ++c)
            tma_load_3d_plain(sb + g * q_group + c * q_chunk, &tm_q, bar(B_QFULL + g), c * kChunkElems, 0,
                              b * p.s_q + q0 + g * p.nq);
          last_q[g] = units;
        }
        ++units;
        if (stop) break;
      }
      int page[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = 2 * it.t + k;
        const int pg = at < p.max_blocks ? __ldg(p.block_table + (int64_t)b * p.max_blocks + at) : 0;
        page[k] = pg < 0 || pg >= p.num_blocks ? 0 : pg;  // a bad page is masked by the epilogue
      }
      for (int c = 0; c < kChunks; ++c, ++n) {
        const int s = n % p.ring;
        if (!wait(bar(B_KEMPTY + s), ((n / p.ring) & 1) ^ 1, guard)) { stop = true; break; }
        mbar_arrive_expect_tx(bar(B_KFULL + s), kUnit);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          tma_load_3d_plain(sb + off_ring + s * kUnit + k * (kUnit / 2), &tm_k, bar(B_KFULL + s), c * kChunkElems, 0,
                            page[k]);
      }
    }
    // never leave with a copy in flight into this CTA's shared memory
    const uint64_t t_0 = cycles();
    for (int k = n < p.ring ? 0 : n - p.ring; k < n; ++k)
      while (!mbar_try_wait(bar(B_KFULL + k % p.ring), (k / p.ring) & 1) && cycles() - t_0 < kDrainLimitCycles) {}
    for (int g = 0; g < 2; ++g)
      if (last_q[g] >= 0)
        while (!mbar_try_wait(bar(B_QFULL + g), last_q[g] & 1) && cycles() - t_0 < kDrainLimitCycles) {}
  } else if (warp == 1 && lane == 0 && !it.done()) {
    // ---------------- UMMA issue ----------------
    const uint32_t idesc = kType == K_FP8 ? ((1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24))
                                          : idesc_f16(128, N, kType == K_BF16, false, false);
    int n = 0, seq = 0, units = 0, unit = -1;
    bool failed = false;
    for (; !failed && !it.done(); it.next(p)) {
      const bool first = it.u != unit, last = it.last_of_unit();
      unit = it.u;
      for (int g = 0; g < p.groups && !failed; ++g, ++seq) {
        const int acc = seq & 1;
        if ((first && !wait(bar(B_QFULL + g), units & 1, guard)) ||
            !wait(bar(B_AEMPTY + acc), ((seq >> 1) & 1) ^ 1, guard)) {
          failed = true;
          break;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int s = (n + c) % p.ring;
          if (g == 0 && !wait(bar(B_KFULL + s), ((n + c) / p.ring) & 1, guard)) { failed = true; break; }
          tc_fence_after();
          const uint64_t da = sdesc_sw128(sb + off_ring + s * kUnit, 16, 1024);
          const uint64_t db = sdesc_sw128(sb + g * q_group + c * q_chunk, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of the contraction each
            if (kType == K_FP8)
              umma_ss_f8(tmem + (uint32_t)kMaxN * acc, da + 2u * kk, db + 2u * kk, idesc, (c | kk) ? 1u : 0u);
            else
              umma_ss(tmem + (uint32_t)kMaxN * acc, da + 2u * kk, db + 2u * kk, idesc, (c | kk) ? 1u : 0u);
          }
          if (g == p.groups - 1) umma_commit(bar(B_KEMPTY + s));
        }
        if (failed) break;
        umma_commit(bar(B_AFULL + acc));
        if (last) umma_commit(bar(B_QEMPTY + g));
      }
      n += kChunks;
      if (first) ++units;
    }
    // every UMMA this thread issued has completed before TMEM is released
    umma_commit(bar(B_DRAIN));
    const uint64_t t_0 = cycles();
    while (!mbar_try_wait(bar(B_DRAIN), 0) && cycles() - t_0 < kDrainLimitCycles) {}
  } else if (warp == 2 && ok) {
    // ---------------- -inf behind the last tile of each row's unit ----------------
    constexpr int kPerTile = kPages ? kTokens / kTile : kTokens;
    const int64_t rows = (int64_t)p.batch * p.s_q;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
      const int b = (int)(r / p.s_q), i = (int)(r - (int64_t)b * p.s_q);
      const int tiles = unit_tiles(p, b * p.units + i / (p.nq * p.groups));
      float* row = p.scores + r * p.stride;
      for (int c = tiles * kPerTile + lane; c < p.width; c += 32) row[c] = -INFINITY;
      if (lane == 0 && __ldg(p.seqlens + b) > p.cover) atomicOr(status, STATUS_INDEX);
    }
  } else if (warp == 3 && !it.done()) {
    // ---------------- head weights of each unit, padded heads zero ----------------
    int units = 0, unit = -1;
    for (; !it.done(); it.next(p)) {
      if (it.u == unit) continue;
      unit = it.u;
      const int par = units & 1;
      const bool free = wait(bar(B_WEMPTY + par), ((units >> 1) & 1) ^ 1, guard);
      if (!__all_sync(0xffffffffu, free)) break;
      const int b = unit / p.units, q0 = (unit - b * p.units) * p.nq * p.groups;
      float* dst = reinterpret_cast<float*>(smem + off_w) + par * 2 * kMaxN;
      for (int g = 0; g < p.groups; ++g)
        for (int e = lane; e < N; e += 32) {
          const int q = q0 + g * p.nq + e / kHp, h = e % kHp;
          dst[g * kMaxN + e] =
              q < p.s_q && h < p.heads ? __ldg(p.weights + ((int64_t)b * p.s_q + q) * p.heads + h) : 0.f;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_WFULL + par));
      ++units;
    }
  } else if (warp >= 4 && !it.done()) {
    // ---------------- epilogue: sum over heads ----------------
    const int e = (warp - 4) >> 2, q4 = warp & 3;  // accumulator, TMEM lane quarter
    const uint32_t tl = tmem + (uint32_t)kMaxN * e + ((uint32_t)(32 * q4) << 16);
    const float* weights = reinterpret_cast<const float*>(smem + off_w);
    float* red = reinterpret_cast<float*>(smem + off_red) + e * 2 * 4 * 16;
    int seq = 0, units = -1, unit = -1, done = 0;
    bool failed = false;
    for (; !failed && !it.done(); it.next(p)) {
      if (it.u != unit) {
        // the weights of the unit before are free once this warp has left it
        __syncwarp();
        if (unit >= 0 && lane == 0) mbar_arrive(bar(B_WEMPTY + (units & 1)));
        unit = it.u;
        ++units;
        if (!__all_sync(0xffffffffu, wait(bar(B_WFULL + (units & 1)), (units >> 1) & 1, guard))) break;
      }
      const int b = unit / p.units, q0 = (unit - b * p.units) * p.nq * p.groups;
      const int tok = it.t * kTokens + 32 * q4 + lane;
      // the page of this warp's 32 tokens
      const int at = 2 * it.t + (q4 >> 1);
      const int pg = at < p.max_blocks ? __ldg(p.block_table + (int64_t)b * p.max_blocks + at) : -1;
      const bool good = pg >= 0 && pg < p.num_blocks;
      const int len = __ldg(p.seqlens + b);
      if (!good && lane == 0 && 64 * at < min(len, p.cover)) atomicOr(status, STATUS_INDEX);
      float ks = 1.f;
      if (kType == K_FP8 && good)
        ks = __ldg(reinterpret_cast<const float*>(p.cache + (int64_t)pg * (kTile * (kDim + 4)) + kTile * kDim) +
                   (tok & (kTile - 1)));
      for (int g = 0; g < p.groups; ++g, ++seq) {
        if ((seq & 1) != e) continue;
        if (!__all_sync(0xffffffffu, wait(bar(B_AFULL + e), (seq >> 1) & 1, guard))) {
          failed = true;
          break;
        }
        tc_fence_after();
        const float* w = weights + (units & 1) * 2 * kMaxN + g * kMaxN;
#pragma unroll 1
        for (int j = 0; j < p.nq; ++j) {
          const int q = q0 + g * p.nq + j;
          if (q >= p.s_q) break;
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < kHp; c += 16) {
            uint32_t r[16];
            tmem_ld16(tl + (uint32_t)(j * kHp + c), r);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) sum = fmaf(w[j * kHp + c + k], fmaxf(__uint_as_float(r[k]), 0.f), sum);
          }
          const float s = good && tok < visible(p, len, q) ? sum * ks : -INFINITY;
          if (!kPages) {
            if (tok < p.width) p.scores[((int64_t)b * p.s_q + q) * p.stride + tok] = s;
          } else {
            float m = s;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) red[(done & 1) * 64 + q4 * 16 + j] = m;
          }
        }
        tc_fence_before();
        if (lane == 0) mbar_arrive(bar(B_AEMPTY + e));
        if (kPages) {
          // the page's other warp; bounded like every wait, so that a warp that
          // gave up leaves no one behind
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_RED + e));
          if (!__all_sync(0xffffffffu, wait(bar(B_RED + e), done & 1, guard))) {
            failed = true;
            break;
          }
          const int x = 32 * q4 + lane, j = x >> 1, k = x & 1;
          const int q = q0 + g * p.nq + j, page = 2 * it.t + k;
          if (j < p.nq && q < p.s_q && page < p.width) {
            const float* v = red + (done & 1) * 64 + 2 * k * 16 + j;
            p.scores[((int64_t)b * p.s_q + q) * p.stride + page] = fmaxf(v[0], v[16]);
          }
        }
        ++done;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace score
}  // namespace mla
