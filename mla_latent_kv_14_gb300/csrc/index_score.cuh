// index_score.cuh -- the cheap score that picks tokens or pages for the sparse
// attention, sm_103a.
//
//     score[q, t] = ks_t * sum_h w[q, h] * max(0, q_h . k_t)
//
// over the visible tokens t of the query's request (ks_t the scale of an e4m3
// key, 1 otherwise), -inf elsewhere; or the maximum over each 64-token page.
//
// Tokens are the M dimension of the UMMA and (query, head) pairs its N
// dimension, so that the sum over heads stays inside a warp: a 128-token tile
// times a group of `nq` queries x `hp` heads (N = nq * hp <= 256, the heads
// padded to 16, 32 or 64) gives one accumulator. A unit is one request's one or
// two groups, which share each key tile: the tensor pipe multiplies one group
// while the epilogue warps sum the other. With few queries per request (decode)
// N is small and the keys' bytes bound the kernel; with many the tensor pipe
// (1029 cycles an accumulator in 16-bit at N = 256) and the sums do.
//
// The sums: an accumulator is read as matrix fragments (16x256b), four lanes to
// a row, so that a lane needs the weights of a quarter of the columns, from two
// 64-column batches' worth of shared-memory loads, instead of all of them (one
// row per lane wants every weight in every lane, and its 256 broadcast loads an
// accumulator competed with the MMAs' operand reads for shared memory). The
// positive part and a packed fma take 1.5 operations a product; two exchanges
// among the four lanes finish a row.
//
// Measured (GB300): 32 requests of 131072 e4m3 keys, 64 heads, 99.9 us (5.7
// TB/s of keys and scores, 0.84 of the copy bandwidth); in bf16 174 us (0.92).
// 4 x 1024 causal queries over 16384 bf16 keys 675 us at full clocks (1.60
// PFLOP/s, 0.83 of the cuBLAS burst) and 728 us in long runs, where power lowers
// the clock; e4m3 687 us: there the epilogue bounds (without its sums the
// kernel took 389 us, in bf16 558) by the latency of its steps, with the issue
// slots (0.46) and the ALU pipe (46 %) half used. Page scores of the same
// queries 884 us: a maximum over 32 lanes for every query of a tile. A single
// tile takes 4.2 us, start to end.
//
// The (unit, tile) pairs of all requests form one list, cut into equal
// contiguous ranges, one per CTA (one CTA per SM): ragged lengths balance, and
// a unit's queries are loaded once per range.
//
// Warp roles (384 threads): warp 0 reads the block table 32 pages ahead and its
// lane 0 issues the copies (queries, key tiles, the scales and page flags of a
// tile); warp 1 owns TMEM and lane 0 issues the MMAs; warp 2 writes the -inf
// columns behind the visible tiles; warp 3 brings the head weights; warps 4-7
// and 8-11 are two epilogue groups. Accumulators of more than 128 columns (two
// of them) are summed by both, half of the queries each, so that one is free
// again soonest; of smaller ones (four of them) each group takes every other.
// Every wait is bounded; a wait that gives up sets the status word and the CTA
// unwinds.
#pragma once
#include <climits>
#include <cuda.h>

#include "params.h"
#include "pipe.cuh"
#include "ptx.cuh"

namespace mla {
namespace score {

constexpr int kThreads = 384;
constexpr int kGroups = 2;                      // epilogue groups of four warps
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
constexpr uint32_t kRedBytes = kGroups * 2 * 4 * 16 * 4;  // page maxima: [epilogue group][parity][4 warps][16 queries]
enum : uint32_t {
  B_KFULL = 0, B_KEMPTY = B_KFULL + kMaxRing, B_QFULL = B_KEMPTY + kMaxRing, B_QEMPTY = B_QFULL + 2,
  B_AFULL = B_QEMPTY + 2, B_AEMPTY = B_AFULL + 4, B_WFULL = B_AEMPTY + 4, B_WEMPTY = B_WFULL + 2,
  B_RED = B_WEMPTY + 2, B_DRAIN = B_RED + kGroups, B_STALL = B_DRAIN + 1, B_COUNT = B_STALL + 1
};
constexpr uint32_t kTailBytes = kWeightBytes + kRedBytes + 8 * B_COUNT + 128;
constexpr uint32_t smem_bytes(uint32_t q_bytes, uint32_t ring) { return q_bytes + ring * kUnit + kTailBytes + 1024; }

// visible tokens of query i of a request with `len` tokens
MLA_DEV int visible(const ScoreParams& p, int len, int i) {
  const int v = p.causal ? len - (p.s_q - 1 - i) : len;
  return v < 0 ? 0 : (v > p.cover ? p.cover : v);
}
// tokens that the last query of a unit sees (the most of its queries)
MLA_DEV int unit_visible(const ScoreParams& p, int u) {
  const int b = u / p.units, k = u - b * p.units;
  const int per = p.nq * p.groups;
  int last = (k + 1) * per - 1;
  last = last < p.s_q - 1 ? last : p.s_q - 1;
  return visible(p, __ldg(p.seqlens + b), last);
}
MLA_DEV int unit_tiles(const ScoreParams& p, int u) { return (unit_visible(p, u) + kTokens - 1) / kTokens; }

// The CTA's range of the list of (unit, tile) pairs, walked unit by unit, so
// that the loops over a unit's tiles hold nothing but their own work.
struct Walk {
  int u, t, m, left;  // unit, its first tile here, its tiles here, pairs left
  MLA_DEV Walk(const ScoreParams& p, int u0, int t0, int count) : u(u0), t(t0), m(0), left(count) {
    if (left > 0) m = min(unit_tiles(p, u) - t, left);
  }
  MLA_DEV bool done() const { return left <= 0; }
  MLA_DEV void next(const ScoreParams& p) {
    left -= m;
    if (left <= 0) return;
    t = 0;
    do m = unit_tiles(p, ++u); while (m == 0);  // left > 0: a later unit has tiles
    m = min(m, left);
  }
};

// Block-table entries of a request, 16 tiles (32 pages) to a warp's register
// and the next 16 on their way.
struct Pages {
  const int32_t* row;
  int base, entry, ahead;
  uint32_t bad;  // of `entry`: out of range
  MLA_DEV void mark(const ScoreParams& p) {
    bad = __ballot_sync(0xffffffffu, entry < 0 || entry >= p.num_blocks);
  }
  MLA_DEV int load(const ScoreParams& p, int t) const {
    const int at = 2 * t + (int)(threadIdx.x & 31);
    return at < p.max_blocks ? __ldg(row + at) : -1;
  }
  MLA_DEV void start(const ScoreParams& p, int b, int t) {
    row = p.block_table + (int64_t)b * p.max_blocks;
    base = t;
    entry = load(p, t);
    ahead = load(p, t + 16);
    mark(p);
  }
  MLA_DEV bool is_bad(int t, int k) const { return (bad >> (2 * (t - base) + k)) & 1u; }  // t below base + 16
  // page k (0 or 1) of tile t, at most 31 tiles behind base
  MLA_DEV int page(int t, int k) const {
    const int i = t - base;
    return __shfl_sync(0xffffffffu, i < 16 ? entry : ahead, (2 * i + k) & 31);
  }
  MLA_DEV void advance(const ScoreParams& p, int t) {
    if (t - base < 16) return;
    base += 16;
    entry = ahead;
    ahead = load(p, base + 16);
    mark(p);
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
// acc += w * max(0, (x0, x1)) on packed pairs. One asm block, so that the maxima
// are written as the pair that the packed fma reads: 785 us where separate
// expressions took 868 (4 x 1024 causal queries over 16384 bf16 keys, with one
// row of an accumulator per lane).
MLA_DEV void fma_positive(uint64_t& acc, uint32_t x0, uint32_t x1, uint64_t w) {
  asm("{\n\t.reg .f32 lo, hi;\n\t.reg .b64 x;\n\tmax.f32 lo, %1, 0f00000000;\n\tmax.f32 hi, %2, 0f00000000;\n\t"
      "mov.b64 x, {lo, hi};\n\tfma.rn.f32x2 %0, x, %3, %0;\n\t}"
      : "+l"(acc) : "f"(__uint_as_float(x0)), "f"(__uint_as_float(x1)), "l"(w));
}
MLA_DEV uint64_t ld_shared_64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
// 16 rows x 64 columns of an accumulator as matrix fragments: register 4k + 2i
// + x of lane l is row 8i + l / 4, column 8k + 2 (l % 4) + x
MLA_DEV void tmem_ld_16x64(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
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
  // the warp's number as a value that the compiler knows to be the same in all
  // its lanes: the roles' loops then run on the uniform registers that the
  // copy and MMA instructions take their operands from
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
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
  int* scan = reinterpret_cast<int*>(smem + off_w);                 // [warps], before the weights arrive
  const int acc_shift = N > 128 ? 1 : 2, accs = 1 << acc_shift;     // accumulators of 512 / accs columns
  const uint32_t acc_cols = 512u >> acc_shift;
  auto bar = [&](uint32_t i) { return sb + off_bar + 8u * i; };
  uint32_t* status = p.status ? p.status : misc + 3;
  const Guard guard{abort_flag, status, kWaitLimitCycles};

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(bar(B_KFULL + s), 1);
      mbar_init(bar(B_KEMPTY + s), 1);
    }
    for (int s = 0; s < accs; ++s) {
      mbar_init(bar(B_AFULL + s), 1);
      mbar_init(bar(B_AEMPTY + s), accs == 2 ? 4 * kGroups : 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_QFULL + s), 1);
      mbar_init(bar(B_QEMPTY + s), 1);
      mbar_init(bar(B_WFULL + s), 1);
      mbar_init(bar(B_WEMPTY + s), 4 * kGroups);
    }
    for (int s = 0; s < kGroups; ++s) mbar_init(bar(B_RED + s), 4);
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
  pdl_launch_dependents();
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

  if (warp == 0 && !it.done()) {
    // ---------------- producer: a unit's query groups, then key tiles ----------------
    const bool leader = elect_one();
    if (leader) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
    }
    int n = 0, units = 0, last_q[2] = {-1, -1};
    bool stop = false;
    Ring kr;
    Pages pages;
    for (; !stop && !it.done(); it.next(p), ++units) {
      const int b = it.u / p.units;
      pages.start(p, b, it.t);
      const int q0 = (it.u - b * p.units) * p.nq * p.groups;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        // a last group behind the request's queries reads others (or the
        // zero fill); its products are never stored
        if (g >= p.groups || stop) break;
        if (!__all_sync(0xffffffffu, wait_for(bar(B_QEMPTY + g), (units & 1) ^ 1, guard))) { stop = true; break; }
        if (leader) {
          mbar_arrive_expect_tx(bar(B_QFULL + g), q_group);
          for (int c = 0; c < kChunks; ++c)
            tma_load_3d_plain(sb + g * q_group + c * q_chunk, &tm_q, bar(B_QFULL + g), c * kChunkElems, 0,
                              b * p.s_q + q0 + g * p.nq);
        }
        last_q[g] = units;
      }
      const int t1 = it.t + it.m;
      for (int t = it.t; t < t1 && !stop; ++t) {
        pages.advance(p, t);
        int page[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          page[k] = pages.page(t, k);
          if (page[k] < 0 || page[k] >= p.num_blocks) page[k] = 0;  // a bad page's products are not stored
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (!__all_sync(0xffffffffu, wait_for(bar(B_KEMPTY + kr.slot), kr.phase ^ 1u, guard))) { stop = true; break; }
          if (leader) {
            mbar_arrive_expect_tx(bar(B_KFULL + kr.slot), kUnit);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              tma_load_3d_plain(sb + off_ring + kr.slot * kUnit + k * (kUnit / 2), &tm_k, bar(B_KFULL + kr.slot),
                                c * kChunkElems, 0, page[k]);
          }
          kr.step(p.ring);
          ++n;
        }
      }
    }
    // never leave with a copy in flight into this CTA's shared memory
    if (lane == 0) {
      const uint64_t t_0 = cycles();
      for (int k = n < p.ring ? 0 : n - p.ring; k < n; ++k)
        while (!mbar_try_wait(bar(B_KFULL + k % p.ring), (k / p.ring) & 1) && cycles() - t_0 < kDrainLimitCycles) {}
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (last_q[g] >= 0)
          while (!mbar_try_wait(bar(B_QFULL + g), last_q[g] & 1) && cycles() - t_0 < kDrainLimitCycles) {}
    }
  } else if (warp == 1 && !it.done()) {
    // ---------------- UMMA issue ----------------
    const uint32_t idesc = kType == K_FP8 ? ((1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24))
                                          : idesc_f16(128, N, kType == K_BF16, false, false);
    const uint64_t d_ring = sdesc_sw128(sb + off_ring, 16, 1024), d_q = sdesc_sw128(sb, 16, 1024);
    const bool leader = elect_one();  // issues every MMA and commit
    auto ready = [&](uint32_t i, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(bar(i), parity, guard)) != 0; };
    int seq = 0, units = 0;
    bool failed = false;
    Ring kr;
    for (; !failed && !it.done(); it.next(p), ++units) {
      if (!ready(B_QFULL, units & 1) || (p.groups == 2 && !ready(B_QFULL + 1, units & 1))) break;
      for (int i = 0; i < it.m && !failed; ++i) {
        Ring at = kr;
        for (int g = 0; g < p.groups; ++g, ++seq) {
          at = kr;  // every group reads the tile's units
          const int acc = seq & (accs - 1);
          const uint32_t d = tmem + acc_cols * acc;
          if (!ready(B_AEMPTY + acc, ((seq >> acc_shift) & 1) ^ 1)) { failed = true; break; }
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (g == 0 && !ready(B_KFULL + at.slot, at.phase)) { failed = true; break; }
            tc_fence_after();
            const uint64_t da = d_ring + (uint32_t)at.slot * (kUnit >> 4);
            const uint64_t db = d_q + ((g * q_group + c * q_chunk) >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of the contraction each
                if (kType == K_FP8)
                  umma_ss_f8(d, da + 2u * kk, db + 2u * kk, idesc, (c | kk) ? 1u : 0u);
                else
                  umma_ss(d, da + 2u * kk, db + 2u * kk, idesc, (c | kk) ? 1u : 0u);
              }
              if (g == p.groups - 1) umma_commit(bar(B_KEMPTY + at.slot));
              if (c == kChunks - 1) umma_commit(bar(B_AFULL + acc));
            }
            at.step(p.ring);
          }
          if (failed) break;
        }
        kr = at;
      }
      if (leader) {
        umma_commit(bar(B_QEMPTY));
        if (p.groups == 2) umma_commit(bar(B_QEMPTY + 1));
      }
    }
    // every UMMA this thread issued has completed before TMEM is released
    if (leader) umma_commit(bar(B_DRAIN));
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
    for (int units = 0; !it.done(); it.next(p), ++units) {
      const int par = units & 1;
      const bool free = wait_for(bar(B_WEMPTY + par), ((units >> 1) & 1) ^ 1, guard);
      if (!__all_sync(0xffffffffu, free)) break;
      const int b = it.u / p.units, q0 = (it.u - b * p.units) * p.nq * p.groups;
      float* dst = reinterpret_cast<float*>(smem + off_w) + par * 2 * kMaxN;
      for (int g = 0; g < p.groups; ++g)
        for (int e = lane; e < N; e += 32) {
          const int q = q0 + g * p.nq + e / kHp, h = e % kHp;
          dst[g * kMaxN + e] =
              q < p.s_q && h < p.heads ? __ldg(p.weights + ((int64_t)b * p.s_q + q) * p.heads + h) : 0.f;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_WFULL + par));
    }
  } else if (warp >= 4 && !it.done()) {
    // ---------------- epilogue: sum over heads ----------------
    const int e = (warp - 4) >> 2, q4 = warp & 3;  // epilogue group, TMEM lane quarter
    float* red = reinterpret_cast<float*>(smem + off_red) + e * 2 * 4 * 16;
    // two accumulators: both groups sum a share of each one's queries; four:
    // each group takes every other tile
    const bool shared = accs == 2;
    const int ways = shared ? 1 : kGroups;
    // queries [first, first + most) of a query group; a multiple of 32 columns lies before them
    constexpr int kAlign = kHp == 16 ? 2 : 1;
    const int share = shared ? (p.nq + kGroups * kAlign - 1) / (kGroups * kAlign) * kAlign : p.nq;
    const int first = shared ? e * share : 0, most = min(share, p.nq - first);
    const int row = 32 * q4 + 8 * (lane & 3) + (lane >> 2);  // this thread's token of a tile (see `reduce`)
    const uint32_t tl0 = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(first * kHp);
    const uint32_t w0 = sb + off_w + (uint32_t)(first * kHp) * 4u + 8u * (lane & 3);
    const int64_t group_step = p.nq * p.stride;
    constexpr int kQ = 64 / kHp;                   // queries of a batch of 64 columns
    // Four lanes hold parts of the same four rows (8i + l / 4): they exchange
    // halves, then quarters, and lane l ends with row 8 (l % 4) + l / 4.
    const bool up = lane & 2, odd = lane & 1;
    auto reduce = [&](const float (&v)[4]) {
      const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 2);
      const float c = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 2);
      return (odd ? c : a) + __shfl_xor_sync(0xffffffffu, odd ? a : c, 1);
    };
    int tiles = 0, done = 0;
    bool failed = false;
    Pages pages;
    for (int units = 0; !failed && !it.done(); it.next(p), ++units) {
      const int b = it.u / p.units, k0 = (it.u - b * p.units) * p.groups * p.nq + first;
      const int unit_seen = unit_visible(p, it.u);
      // tokens that query k0 sees, and each query behind it (a causal one more)
      const int len = __ldg(p.seqlens + b), seen0 = p.causal ? len - (p.s_q - 1 - k0) : len, later = p.causal ? 1 : 0;
      // tiles t of this unit with (number of the tile in the CTA's range) % ways == e
      int t = it.t + (shared ? 0 : (e - tiles) & (kGroups - 1));
      const int t1 = it.t + it.m;
      tiles += it.m;
      pages.start(p, b, it.t);
      // scale of this thread's token in tile `at` (its page's scales follow the page's rows)
      auto scale_at = [&](int at) {
        const int pg = pages.page(at, q4 >> 1);
        if (pg < 0 || pg >= p.num_blocks) return 1.f;
        return __ldg(reinterpret_cast<const float*>(p.cache + (int64_t)pg * (kTile * (kDim + 4)) + kTile * kDim) +
                     (row & (kTile - 1)));
      };
      float ks = 1.f, ks_next = 1.f;
      if (kType == K_FP8 && t < t1) ks_next = scale_at(t);
      float* out_unit = p.scores + ((int64_t)b * p.s_q + k0) * p.stride + (kPages ? 0 : t * kTokens + row);
      uint32_t w = w0 + (uint32_t)(units & 1) * (2 * kMaxN * 4);
      if (!__all_sync(0xffffffffu, wait_for(bar(B_WFULL + (units & 1)), (units >> 1) & 1, guard))) break;
#pragma unroll 1
      for (; t < t1; t += ways, out_unit += kPages ? 0 : kTokens * ways) {
        pages.advance(p, t);
        const bool bad = pages.is_bad(t, q4 >> 1);
        if (kType == K_FP8) {
          ks = ks_next;
          if (t + ways < t1) ks_next = scale_at(t + ways);
        }
        const int tok = t * kTokens + row;
        if (bad && lane == 0 && (tok & ~(kTile - 1)) < unit_seen) atomicOr(status, STATUS_INDEX);
        const int seen_unit = bad ? INT_MIN / 2 : seen0;
        // stores (or keeps for the page maximum) the score of query j of a group's share
        auto finish = [&](int g, int j, float total) {
          const float s = tok < min(seen_unit + later * (g * p.nq + j), p.cover) ? total * ks : -INFINITY;
          if (!kPages) {
            if (tok < p.width) out_unit[g * group_step + j * p.stride] = s;
          } else {
            float m = s;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) red[(done & 1) * 64 + q4 * 16 + j] = m;
          }
        };
        float v0[2][kQ][4], v1[2][kQ][4];  // sums over the lane's columns: [group][query of the batch][row]
        // sums of a group's share: over the four lanes of a row, for all of its queries together
        auto totals = [&](int g, int queries) {
          float total[2 * kQ];
#pragma unroll
          for (int j = 0; j < kQ; ++j) {
            total[j] = reduce(v0[g][j]);
            if (queries > kQ) total[kQ + j] = reduce(v1[g][j]);
          }
#pragma unroll
          for (int j = 0; j < 2 * kQ; ++j)
            if (j < queries) finish(g, j, total[j]);
        };
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (g >= p.groups) break;
          const int queries = min(most, p.s_q - k0 - g * p.nq);  // may be none in a request's last unit
          const bool two = queries > kQ;                        // batches of 64 columns
          const int seq = shared ? done : kGroups * done + e, acc = seq & (accs - 1);
          const uint32_t tl = tl0 + acc_cols * (uint32_t)acc;
          uint64_t wv[8];  // the lane's weights of a batch: columns 8k + 2 (lane % 4) + {0, 1}
          auto load_weights = [&](int c) {
#pragma unroll
            for (int k = 0; k < 8; ++k) wv[k] = ld_shared_64(w + g * (kMaxN * 4) + 256u * c + 32u * k);
          };
          // 16 rows of a batch: the lane's columns of rows l / 4 and 8 + l / 4, summed per query
          auto half = [&](const uint32_t* r, float (*v)[4], int i) {
#pragma unroll
            for (int j = 0; j < kQ; ++j) {
              uint64_t lo = 0, hi = 0;
#pragma unroll
              for (int k = j * (8 / kQ); k < (j + 1) * (8 / kQ); ++k) {
                fma_positive(lo, r[4 * k], r[4 * k + 1], wv[k]);
                fma_positive(hi, r[4 * k + 2], r[4 * k + 3], wv[k]);
              }
              const float2 x = f2_unpack(lo), y = f2_unpack(hi);
              v[j][i] = x.x + x.y;
              v[j][i + 1] = y.x + y.y;
            }
          };
          auto release = [&]() {  // the accumulator is free for the next products
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_AEMPTY + acc));
          };
          // two register buffers of 16 rows: one is loaded while the other is summed
          uint32_t ra[32], rb[32];
          load_weights(0);
          if (!__all_sync(0xffffffffu, wait_for(bar(B_AFULL + acc), (seq >> acc_shift) & 1, guard))) {
            failed = true;
            break;
          }
          tc_fence_after();
          tmem_ld_16x64(tl, ra);
          tmem_ld_16x64(tl + (16u << 16), rb);
          tmem_wait_ld();
          pin_regs32(ra);
          pin_regs32(rb);
          if (two) {
            half(ra, v0[g], 0);
            tmem_ld_16x64(tl + 64, ra);
            half(rb, v0[g], 2);
            load_weights(1);
            tmem_ld_16x64(tl + (16u << 16) + 64, rb);
            tmem_wait_ld();
            pin_regs32(ra);
            pin_regs32(rb);
            release();
            half(ra, v1[g], 0);
            half(rb, v1[g], 2);
          } else {
            release();
            half(ra, v0[g], 0);
            half(rb, v0[g], 2);
          }
          if (kPages || kHp < 64) totals(g, queries);
          if (kPages) {
            // the page's other warp; bounded like every wait, so that a warp that
            // gave up leaves no one behind
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_RED + e));
            if (!__all_sync(0xffffffffu, wait_for(bar(B_RED + e), done & 1, guard))) {
              failed = true;
              break;
            }
            const int x = 32 * q4 + lane, j = x >> 1, k = x & 1, page = 2 * t + k;
            if (j < queries && page < p.width) {
              const float* v = red + (done & 1) * 64 + 2 * k * 16 + j;
              out_unit[g * group_step + j * p.stride + page] = fmaxf(v[0], v[16]);
            }
          }
          ++done;
        }
        if (!kPages && kHp == 64 && !failed) {
          // the scores of both groups at once: the shuffles' latencies overlap
          totals(0, min(most, p.s_q - k0));
          if (p.groups == 2) totals(1, min(most, p.s_q - k0 - p.nq));
        }
        if (failed) break;
      }
      // the unit's weights are free once every warp has left it
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_WEMPTY + (units & 1)));
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
