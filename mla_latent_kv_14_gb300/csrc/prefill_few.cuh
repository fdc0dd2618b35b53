// prefill_few.cuh -- the attention of prefill.cuh for documents of few new
// tokens, one CTA to a unit of 128 queries.
//
// Few rows over long keys are bound by the keys' and values' bytes, so what
// counts is how much of them is on its way: the queries take 48 KB, the rest of
// shared memory is a ring of chunks of 128 rows x 128 bytes (three of keys, two
// of values a tile), 2.2 tiles. The two chains take every other key tile of the
// same queries, each with an accumulator and a reference of its own; the warps of
// the one that had the first tile join them at the unit's end. It is the other one
// that begins the next unit, so that units of a single tile overlap too. Warps none
// of whose 32 rows is a query only pass the tiles on.
//
// Measured (GB300, bf16): 8 x 4 queries over 5461 to 16384 keys, 16 heads 123 us
// (0.83 of the copy bandwidth; one query tile beside an empty one, a ring of 1.6
// tiles: 168), 16 x 4 over 8192 175 us (0.92), 16 x 256 over 4096 160 us, 64
// documents of 128 by themselves 38. The rest is the units' starts and ends (some
// 6000 cycles where they have one tile: queries wait for the scores before them)
// and the last ones' wait for each other. Tried without gain: the first keys ahead
// of the queries.
//
// Warp roles (384 threads): warp 0 issues the copies, warps 1 and 3 the MMAs of
// the first and the second chain (warp 1 owns TMEM), warp 2 finds the units,
// warps 4-7 and 8-11 are the softmax of the two chains, one row a thread. Every
// wait is bounded; a wait that gives up sets the status word and the CTA unwinds.
#pragma once
#include "prefill.cuh"

namespace mla {
namespace prefill {
namespace few {

using UnitF = Unit<kRows, 1>;
constexpr int kRing = 11;                  // chunks
constexpr int kUnits = 4;                  // units looked up ahead of the slowest reader
constexpr uint32_t kOffRing = kQTile;
constexpr uint32_t kOffBar = kOffRing + kRing * kChunk;
enum : uint32_t {
  B_FULL = 0, B_EMPTY = B_FULL + kRing, B_QFULL = B_EMPTY + kRing, B_QEMPTY = B_QFULL + 1, B_SFULL = B_QEMPTY + 1,
  B_PFULL = B_SFULL + 2, B_OFULL = B_PFULL + 4, B_OEMPTY = B_OFULL + 2, B_LFULL = B_OEMPTY + 2,
  B_UFULL = B_LFULL + 2, B_UEMPTY = B_UFULL + kUnits, B_WANT = B_UEMPTY + kUnits, B_NEXT = B_WANT + 1, B_DRAIN = B_NEXT + 1, B_STALL = B_DRAIN + 2,
  B_COUNT = B_STALL + 1
};
constexpr uint32_t kOffMisc = (kOffBar + 8 * B_COUNT + 15) / 16 * 16;
constexpr uint32_t kOffState = kOffMisc + 64 + 64 * kUnits;   // a chain's reference and sum of each row, for the other
constexpr uint32_t kSmem = kOffState + 8 * kRows + 1024;
static_assert(kSmem <= 232448);
constexpr int kUnitReaders = 11;           // producer, two issuing threads and eight softmax warps

// Ring positions: tile number `tile` of the CTA takes five consecutive chunks, three of keys and two of values; the two
// of values stand side by side (one descriptor covers both).
struct Slots {
  uint32_t first;    // chunks before this tile
  bool late;         // the values would wrap around: they come before the last chunk of keys
  MLA_DEV explicit Slots(uint32_t tile) : first(5u * tile), late((first + 3u) % kRing == kRing - 1u) {}
  MLA_DEV uint32_t key(int c) const { return first + (c < 2 ? c : late ? 4 : 2); }
  MLA_DEV uint32_t value(int c) const { return first + (late ? 2 : 3) + c; }
};
MLA_DEV uint32_t slot_of(uint32_t chunk) { return chunk % kRing; }
MLA_DEV uint32_t phase_of(uint32_t chunk) { return chunk / kRing & 1u; }

// tm_q: dims {192, heads, tq}; tm_k: {128, heads, tk}; tm_r: {64, 1, tk}; tm_v: {128, heads, tk}; boxes {64, 1, 128},
// 128-byte swizzled.
template <bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
                       const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + kOffMisc);  // 16-B aligned
  // misc: [0, 4) the answer of ask_next, 4 TMEM base, 5 abort, 6 ok, 7 status where none is given, 8 chunks asked
  // for, from 16 on the units
  volatile uint32_t* tmem_slot = misc + 4;
  volatile uint32_t* abort_flag = misc + 5;
  volatile uint32_t* ok_flag = misc + 6;
  int* units = reinterpret_cast<int*>(misc + 16);
  auto bar = [&](uint32_t i) { return sb + kOffBar + 8u * i; };
  uint32_t* status = p.status ? p.status : misc + 7;
  const Guard guard{abort_flag, status, kWaitLimitCycles};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    mbar_init(bar(B_QFULL), 1);
    mbar_init(bar(B_QEMPTY), 2);   // both chains
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(B_LFULL + w), 4);
      mbar_init(bar(B_SFULL + w), 1);
      mbar_init(bar(B_PFULL + w), 4);
      mbar_init(bar(B_PFULL + 2 + w), 4);
      mbar_init(bar(B_OFULL + w), 1);
      mbar_init(bar(B_OEMPTY + w), 4);
    }
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(bar(B_UFULL + s), 1);
      mbar_init(bar(B_UEMPTY + s), kUnitReaders);
    }
    mbar_init(bar(B_WANT), 1);
    mbar_init(bar(B_NEXT), 1);
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN + 1), 1);
    mbar_init(bar(B_STALL), 1);
    *abort_flag = 0u;
    *ok_flag = 1u;
    misc[7] = misc[8] = 0u;
    fence_mbar_init();
    if (p.stall_cycles) {
      // test hook: a bounded wait on a barrier nothing arrives at gives up and reports STATUS_TIMEOUT before
      // anything is issued
      const Guard g_stall{abort_flag, status, p.stall_cycles};
      pdl_wait();
      if (!wait(bar(B_STALL), 0, g_stall)) *ok_flag = 0u;
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc + 4), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();  // nothing above reads global memory
  const uint32_t tmem = *tmem_slot;
  const bool ok = *ok_flag != 0u;

  const uint32_t issued = smem_u32(misc + 8);
  auto ready = [&](uint32_t i, uint32_t parity) { return wait_inline<false>(bar(i), parity & 1u, guard); };
  auto ready_all = [&](uint32_t i, uint32_t parity) { return __all_sync(0xffffffffu, ready(i, parity)) != 0; };
  // a chain waits for its own tiles' chunks only
  auto landed = [&](uint32_t chunk) { return wait_issued(issued, chunk, guard) && ready(B_FULL + slot_of(chunk), phase_of(chunk)); };
  // the readers' side of the units: the n-th one, into registers; one lane reads for a role of a single thread
  auto take_one = [&](int n, UnitF& u) {
    if (!ready(B_UFULL + n % kUnits, n / kUnits)) return false;
    u.read(units + 16 * (n % kUnits));
    return true;
  };
  auto take = [&](int n, UnitF& u) {
    const bool got = __all_sync(0xffffffffu, take_one(n, u));
    if (got && lane == 0) mbar_arrive(bar(B_UEMPTY + n % kUnits));
    return got && u.head >= 0;
  };

  if (warp < 4) {
    set_registers_down<kRegsFew>();
    if (warp == 2 && ok) {
      // ---------------- the units ----------------
      Finder<UnitF> finder;
      finder.start();
      int64_t id = blockIdx.x;
      // A unit is taken only when the copies of the one before it come to their end: one taken early could not go to a
      // block that is free sooner.
      bool asking = false;
      int n = 0, asked = 0;
      while (true) {
        UnitF u{};
        u.head = -1;
        const bool found = id >= 0 && finder.find(p, id, u);
        if (found || id < 0) {
          const int s = n % kUnits;
          if (!ready_all(B_UEMPTY + s, (n / kUnits) ^ 1)) break;
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < UnitF::kWords; ++i) units[16 * s + i] = u.word(i);
            mbar_arrive(bar(B_UFULL + s));
          }
          __syncwarp();
        }
        if (id < 0) break;
        record_bad(p, id, gridDim.x);
        if (found && !ready_all(B_WANT, n++)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_NEXT), 16);
          ask_next(smem_u32(misc), bar(B_NEXT));
        }
        asking = true;
        if (!ready_all(B_NEXT, asked)) break;
        asking = false;
        ++asked;
        id = answer_next(smem_u32(misc));
        // read before the next answer is written over it
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (asking && lane == 0) {   // a wait gave up: the answer is still to be written
        const uint64_t t_0 = cycles();
        while (!mbar_try_wait(bar(B_NEXT), asked & 1) && cycles() - t_0 < kDrainLimitCycles) {}
      }
    } else if (warp == 0 && ok) {
      // ---------------- copies: a unit's queries, then its keys and values ----------------
      const bool leader = elect_one();
      if (leader) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_r);
        prefetch_tmap(&tm_v);
      }
      uint32_t loads = 0, tile = 0, q_loads = 0;
      bool stop = false;
      UnitF u;
      auto chunk = [&](const CUtensorMap* m, int x, int y, int z) {
        const uint32_t slot = slot_of(loads);
        if (stop || !ready_all(B_EMPTY + slot, phase_of(loads) ^ 1u)) {
          stop = true;
          return;
        }
        if (leader) {
          mbar_arrive_expect_tx(bar(B_FULL + slot), kChunk);
          tma_load_3d_plain(sb + kOffRing + slot * kChunk, m, bar(B_FULL + slot), x, y, z);
          set_issued(issued, loads + 1u);
        }
        ++loads;
      };
      auto want_next = [&]() {
        if (leader) mbar_arrive(bar(B_WANT));
      };
      for (int n = 0; !stop && take(n, u); ++n) {
        const int e = u.end(0, p.causal);
        if (e - u.t0 < 4) want_next();
        if (e <= u.t0) continue;
        if (!ready_all(B_QEMPTY, q_loads ^ 1u)) break;
        if (leader) {
          mbar_arrive_expect_tx(bar(B_QFULL), kQTile);
          for (int c = 0; c < 3; ++c) tma_load_3d_plain(sb + c * kChunk, &tm_q, bar(B_QFULL), 64 * c, u.head, u.row);
        }
        ++q_loads;
        for (int t = u.t0; t < e && !stop; ++t, ++tile) {
          if (t == e - 4) want_next();
          const int at = u.k0 + t * kKeys;
          const bool late = Slots(tile).late;
          chunk(&tm_k, 0, u.head, at);
          chunk(&tm_k, 64, u.head, at);
          if (!late) chunk(&tm_r, 0, 0, at);
          chunk(&tm_v, 0, u.head, at);
          chunk(&tm_v, 64, u.head, at);
          if (late) chunk(&tm_r, 0, 0, at);
        }
      }
      // never leave with a copy in flight into this CTA's shared memory
      if (lane == 0) {
        const uint64_t t_0 = cycles();
        for (uint32_t k = loads < kRing ? 0u : loads - kRing; k < loads; ++k)
          while (!mbar_try_wait(bar(B_FULL + slot_of(k)), phase_of(k)) && cycles() - t_0 < kDrainLimitCycles) {}
        if (q_loads)
          while (!mbar_try_wait(bar(B_QFULL), (q_loads - 1u) & 1u) && cycles() - t_0 < kDrainLimitCycles) {}
      }
    } else if ((warp & 1) && ok) {
      // ---------------- UMMA issue for chain w: one thread ----------------
      const int w = warp >> 1;
      if (elect_one()) {
        constexpr uint32_t idesc_qk = idesc_f16(128, kKeys, !kFp16, false, false);
        constexpr uint32_t idesc_pv = idesc_f16(128, kV, !kFp16, false, true);
        const uint64_t d_q = sdesc_sw128(sb, 16, 1024), d_ring = sdesc_sw128(sb + kOffRing, 16, 1024),
                       d_v = sdesc_sw128(sb + kOffRing, kChunk, 1024);
        const uint32_t t_s = tmem + 128u * w, t_o = tmem + kColO + 128u * w;
        uint32_t tile = 0, q_used = 0, p_used = 0, o_used = 0;
        auto scores = [&](const Slots& s, bool last) {   // S = Q K^T
          if (!landed(s.key(0)) || !landed(s.key(1)) || !landed(s.key(2))) return false;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const uint64_t a = d_q + c * (kChunk >> 4), b = d_ring + slot_of(s.key(c)) * (kChunk >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ss(t_s, a + 2u * k, b + 2u * k, idesc_qk, (c | k) ? 1u : 0u);
          }
          umma_commit(bar(B_SFULL + w));
#pragma unroll
          for (int c = 0; c < 3; ++c) umma_commit(bar(B_EMPTY + slot_of(s.key(c))));
          if (last) umma_commit(bar(B_QEMPTY));
          return true;
        };
        UnitF u;
        bool failed = false;
        for (int n = 0; !failed && take_one(n, u); ++n) {
          mbar_arrive(bar(B_UEMPTY + n % kUnits));
          if (u.head < 0) break;
          const int e = u.end(0, p.causal), first = u.t0 + (w ^ (n & 1));   // the chains begin a unit in turn
          if (e <= u.t0) continue;
          if (!ready(B_QFULL, q_used++)) break;
          if (first >= e) mbar_arrive(bar(B_QEMPTY));   // no tile for this chain
          else if (!scores(Slots(tile + (uint32_t)(first - u.t0)), first + 2 >= e)) break;
          for (int t = first; t < e; t += 2) {
            const Slots s(tile + (uint32_t)(t - u.t0));
            const uint32_t v0 = s.value(0), v1 = s.value(1);
            if (!landed(v0) || !landed(v1) || (t == first && !ready(B_OEMPTY + w, o_used++ ^ 1u)) || !ready(B_PFULL + w, p_used)) {
              failed = true;
              break;
            }
            tc_fence_after();
            // O (+)= P V, 16 keys at a time; the first half while the second is still formed
            const uint64_t b = d_v + slot_of(v0) * (kChunk >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ts(t_o, t_s + 8u * k, b + 128u * k, idesc_pv, (t == first && k == 0) ? 0u : 1u);
            if (!ready(B_PFULL + 2 + w, p_used++)) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int k = 4; k < 8; ++k) umma_ts(t_o, t_s + 8u * k, b + 128u * k, idesc_pv, 1u);
            umma_commit(bar(B_EMPTY + slot_of(v0)));
            umma_commit(bar(B_EMPTY + slot_of(v1)));
            // the next keys may wait for these values' place in the ring
            if (t + 2 >= e) umma_commit(bar(B_OFULL + w));
            else if (!scores(Slots(tile + (uint32_t)(t - u.t0) + 2), t + 4 >= e)) {
              failed = true;
              break;
            }
          }
          tile += e - u.t0;
        }
        // every UMMA this thread issued has completed before TMEM is released
        umma_commit(bar(B_DRAIN + w));
        const uint64_t t_0 = cycles();
        while (!mbar_try_wait(bar(B_DRAIN + w), 0) && cycles() - t_0 < kDrainLimitCycles) {}
      }
      __syncwarp();
    }
  } else {
    set_registers_up<kRegsMany>();
    // ---------------- softmax of chain w: row `r` ----------------
    const int w = (warp - 4) >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + tl + 128u * w, t_o = tmem + tl + kColO;
    float2* states = reinterpret_cast<float2*>(smem + kOffState);
    auto arrive = [&](uint32_t i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    uint32_t s_used = 0, o_used = 0, o_other = 0, l_used = 0, tile = 0;
    bool failed = !ok;
    UnitF u;
    for (int n = 0; !failed && take(n, u); ++n) {
      const int e = u.end(0, p.causal);
      const bool idle = r - lane >= u.rows;          // none of the warp's rows is a query
      const int seen = r < u.rows ? u.visible(r, p.causal) : u.nk, least = u.visible(0, p.causal);   // of the row; of all rows
      const bool leads = w == (n & 1);
      const int begin = u.t0 + (leads ? 0 : 1);
      Row state{-INFINITY, 0.f};
      for (int t = begin; t < e; t += 2) {
        if (!ready_all(B_SFULL + w, s_used++)) { failed = true; break; }
        tc_fence_after();
        const int rest = u.nk - t * kKeys;
        if (rest < kKeys) {
          // The value rows behind the document's keys may hold anything, and zero times NaN is NaN: they are cleared
          // before this tile's P is handed over.
          const Slots at(tile + (uint32_t)(t - u.t0));
          const uint32_t v0 = at.value(0), v1 = at.value(1);
          if (!__all_sync(0xffffffffu, landed(v0) && landed(v1))) {
            failed = true;
            break;
          }
          const uint32_t to = sb + kOffRing + slot_of(v0) * kChunk;   // v1 stands behind v0
          for (int i = rest * 8 + r; i < kKeys * 8; i += kRows) {
            st_shared_v4(to + 16u * i, 0u, 0u, 0u, 0u);
            st_shared_v4(to + kChunk + 16u * i, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (idle) {        // the rows' products are of no query: any P will do
          arrive(B_PFULL + w);
          arrive(B_PFULL + 2 + w);
          continue;
        }
        softmax_tile<kFp16>(state, t_s, t_o + 128u * w, p.scale_log2, (t + 1) * kKeys > least, seen - t * kKeys, t == begin,
                            [&](int h) { arrive(B_PFULL + 2 * h + w); });
      }
      if (failed) break;
      tile += max(e - u.t0, 0);
      const bool some = e > u.t0, both = e > u.t0 + 1;   // tiles of the chain that began, of the other
      const uint32_t o_round = o_used, other_round = o_other;
      o_used += leads ? some : both;
      o_other += leads ? both : some;
      if (!leads) {
        // this thread has read what stood here: it wrote the unit before
        states[r] = make_float2(state.m, state.l);
        arrive(B_LFULL + (w ^ 1));
        continue;
      }
      // The warps of the chain that began write the unit: both chains' shares, at the larger of their references. The
      // other chain's warps have by now seen the accumulators of the unit before, so that no older phase passes for these.
      if (!ready_all(B_LFULL + w, l_used++)) break;
      const float2 other = states[r];
      if ((some && !ready_all(B_OFULL + w, o_round)) || (both && !ready_all(B_OFULL + (w ^ 1), other_round))) break;
      tc_fence_after();
      const float m = fmaxf(state.m, other.x), ref = m == -INFINITY ? 0.f : m;
      const float f0 = exp2_approx((state.m - ref) * p.scale_log2), f1 = exp2_approx((other.x - ref) * p.scale_log2);
      const float l = f0 * state.l + f1 * other.y;
      const bool whole = u.pieces == 1, live = r < u.rows;
      const float inv = whole ? inverse(l, seen > 0) : 1.f;
      const int64_t at = (int64_t)u.row + r;
      if (live && whole) {
        p.lse[at * p.heads + u.head] = lse_of<kFp16>(p, m, l, seen > 0);
      } else if (live) {
        p.ref_part[((int64_t)u.piece * p.tq + at) * p.heads + u.head] = m;
        *sum_at(p, at, u.head, u.piece) = l;
      }
      // 32 dims of the row: f0 a + f1 b, over l if it is whole
      auto share = [&](int c, float* v) {
        uint32_t a[32], b[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) a[k] = b[k] = 0u;
        if (some) tmem_ld32(t_o + 128u * w + 32u * c, a);
        if (both) tmem_ld32(t_o + 128u * (w ^ 1) + 32u * c, b);
        tmem_wait_ld();
        pin_regs32(a);
        pin_regs32(b);
        if (c == 3) {      // both are read: the next unit may write them
          if (some) arrive(B_OEMPTY + w);
          if (both) arrive(B_OEMPTY + (w ^ 1));
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = (f0 * __uint_as_float(a[k]) + f1 * __uint_as_float(b[k])) * inv;
      };
      // Loops, not straight code: what runs once a unit is not in the instruction cache (64 documents of 256 queries 92
      // us; 109 with all of the row read and packed before the stores, 94 with one loop for both kinds).
      if (whole) {
        uint16_t* dst = static_cast<uint16_t*>(p.out) + at * p.out_token + u.head * p.out_head;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float v[32];
          share(c, v);
          if (live) store_share<kFp16>(dst + 32 * c, nullptr, v, p.wide);
        }
      } else {
        float* part = p.o_part + (((int64_t)u.piece * p.tq + at) * p.heads + u.head) * kV;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float v[32];
          share(c, v);
          if (live) store_share<kFp16>(nullptr, part + 32 * c, v, p.wide);
        }
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

}  // namespace few
}  // namespace prefill
}  // namespace mla
