// prefill_few.cuh -- the attention of prefill.cuh for documents of few new
// tokens, one CTA to a unit of 256 queries.
//
// Both query tiles read each chunk of 128 rows x 128 bytes of keys (three a
// tile) and values (two) from one ring.
//
// Warp roles (384 threads): warp 0 issues the copies, warps 1 and 3 the MMAs of
// the first and the second query tile (warp 1 owns TMEM), warp 2 finds the
// units, warps 4-7 and 8-11 are the softmax of the two query tiles, one row a
// thread. Every wait is bounded; a wait that gives up sets the status word and
// the CTA unwinds.
#pragma once
#include "prefill.cuh"

namespace mla {
namespace prefill {
namespace few {

constexpr int kRing = 8;                   // chunks: three of K, two of V a tile
constexpr uint32_t kOffRing = 2 * kQTile;
constexpr uint32_t kOffBar = kOffRing + kRing * kChunk;
enum : uint32_t {
  B_FULL = 0, B_EMPTY = B_FULL + kRing, B_QFULL = B_EMPTY + kRing, B_QEMPTY = B_QFULL + 2, B_SFULL = B_QEMPTY + 2,
  B_PFULL = B_SFULL + 2, B_OFULL = B_PFULL + 4, B_OEMPTY = B_OFULL + 2, B_UFULL = B_OEMPTY + 2, B_UEMPTY = B_UFULL + 2,
  B_NEXT = B_UEMPTY + 2, B_DRAIN = B_NEXT + 1, B_STALL = B_DRAIN + 2, B_COUNT = B_STALL + 1
};
constexpr uint32_t kOffMisc = (kOffBar + 8 * B_COUNT + 15) / 16 * 16;
constexpr uint32_t kSmem = kOffMisc + 256 + 1024;
constexpr int kUnitReaders = 11;           // producer, two MMA and eight softmax warps

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
  // misc: [0, 4) the answer of ask_next, 4 TMEM base, 5 abort, 6 ok, 7 status where none is given, [16, 48) two units
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
      mbar_init(bar(B_EMPTY + s), 2);   // both query tiles' products
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(B_QFULL + w), 1);
      mbar_init(bar(B_QEMPTY + w), 1);
      mbar_init(bar(B_SFULL + w), 1);
      mbar_init(bar(B_PFULL + w), 4);
      mbar_init(bar(B_PFULL + 2 + w), 4);
      mbar_init(bar(B_OFULL + w), 1);
      mbar_init(bar(B_OEMPTY + w), 4);
      mbar_init(bar(B_UFULL + w), 1);
      mbar_init(bar(B_UEMPTY + w), kUnitReaders);
    }
    mbar_init(bar(B_NEXT), 1);
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN + 1), 1);
    mbar_init(bar(B_STALL), 1);
    *abort_flag = 0u;
    *ok_flag = 1u;
    misc[7] = 0u;
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

  // the readers' side of the units: the n-th one, into registers; one lane reads for a role of a single thread
  auto take_one = [&](int n, Unit<kRows>& u) {
    const int s = n & 1;
    if (!wait_inline<false>(bar(B_UFULL + s), (n >> 1) & 1, guard)) return false;
    u.read(units + 16 * s);
    return true;
  };
  auto take = [&](int n, Unit<kRows>& u) {
    const bool got = __all_sync(0xffffffffu, take_one(n, u));
    if (got && lane == 0) mbar_arrive(bar(B_UEMPTY + (n & 1)));
    return got && u.head >= 0;
  };

  if (warp < 4) {
    set_registers_down<kRegsFew>();
    if (warp == 2 && ok) {
      // ---------------- the units ----------------
      Finder<kRows> finder;
      finder.start(p);
      int64_t id = blockIdx.x;
      bool more = true, asking = false;
      int n = 0, asked = 0;
      while (true) {
        // the next block's number travels while this one is looked up
        if (more) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_NEXT), 16);
            ask_next(smem_u32(misc), bar(B_NEXT));
          }
          asking = true;
        }
        Unit<kRows> u{};
        u.head = -1;
        bool past = false;
        const bool found = more && finder.find(p, id, u, past);
        if (found || !more) {
          if (!__all_sync(0xffffffffu, wait_inline<false>(bar(B_UEMPTY + (n & 1)), ((n >> 1) & 1) ^ 1, guard))) break;
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < Unit<kRows>::kWords; ++i) units[16 * (n & 1) + i] = u.word(i);
            mbar_arrive(bar(B_UFULL + (n & 1)));
          }
          __syncwarp();
          ++n;
        }
        if (!more) break;
        if (!__all_sync(0xffffffffu, wait_inline<false>(bar(B_NEXT), asked & 1, guard))) break;
        asking = false;
        ++asked;
        id = answer_next(smem_u32(misc));
        more = id >= 0;
        // read before the next answer is written over it
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (asking && lane == 0) {   // a wait gave up: the answer is still to be written
        const uint64_t t_0 = cycles();
        while (!mbar_try_wait(bar(B_NEXT), asked & 1) && cycles() - t_0 < kDrainLimitCycles) {}
      }
    } else if (warp == 0 && ok) {
      // ---------------- copies: a unit's query tiles, then its keys and values ----------------
      const bool leader = elect_one();
      if (leader) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_r);
        prefetch_tmap(&tm_v);
      }
      int n = 0, q_loads[2] = {0, 0};
      uint32_t loads = 0, tile = 0;
      bool stop = false;
      Unit<kRows> u;
      auto chunk = [&](const CUtensorMap* m, int x, int y, int z) {
        const uint32_t slot = slot_of(loads);
        if (stop || !__all_sync(0xffffffffu, wait_inline<false>(bar(B_EMPTY + slot), phase_of(loads) ^ 1u, guard))) {
          stop = true;
          return;
        }
        if (leader) {
          mbar_arrive_expect_tx(bar(B_FULL + slot), kChunk);
          tma_load_3d_plain(sb + kOffRing + slot * kChunk, m, bar(B_FULL + slot), x, y, z);
        }
        ++loads;
      };
      auto queries = [&](int w) {
        if (stop || !__all_sync(0xffffffffu, wait_inline<false>(bar(B_QEMPTY + w), (q_loads[w] & 1) ^ 1, guard))) {
          stop = true;
          return;
        }
        if (leader) {
          mbar_arrive_expect_tx(bar(B_QFULL + w), kQTile);
          for (int c = 0; c < 3; ++c)
            tma_load_3d_plain(sb + w * kQTile + c * kChunk, &tm_q, bar(B_QFULL + w), 64 * c, u.head, u.row + kRows * w);
        }
        ++q_loads[w];
      };
      for (; !stop && take(n, u); ++n) {
        const int e0 = u.end(0, p.causal), e1 = u.end(1, p.causal), e = max(e0, e1);
        if (e0 > u.t0) queries(0);
        for (int t = u.t0; t < e && !stop; ++t, ++tile) {
          const int at = u.k0 + t * kKeys;
          const bool late = Slots(tile).late;
          chunk(&tm_k, 0, u.head, at);
          chunk(&tm_k, 64, u.head, at);
          if (!late) chunk(&tm_r, 0, 0, at);
          // the second query tile is wanted after the first one's scores
          if (t == u.t0 && e1 > u.t0) queries(1);
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
        for (int w = 0; w < 2; ++w)
          if (q_loads[w])
            while (!mbar_try_wait(bar(B_QFULL + w), (q_loads[w] - 1) & 1) && cycles() - t_0 < kDrainLimitCycles) {}
      }
    } else if ((warp & 1) && ok) {
      // ---------------- UMMA issue for query tile w: one thread ----------------
      // The pipe takes an instruction about when it starts it, so a wait between two of them idles it, but for the
      // other tile's: all that can be waited for while the softmax runs (the next keys, the values) is, and the
      // products of a tile and the scores of the next follow in one go.
      const int w = warp >> 1;
      if (elect_one()) {
        constexpr uint32_t idesc_qk = idesc_f16(128, kKeys, !kFp16, false, false);
        constexpr uint32_t idesc_pv = idesc_f16(128, kV, !kFp16, false, true);
        const uint64_t d_q = sdesc_sw128(sb + w * kQTile, 16, 1024), d_ring = sdesc_sw128(sb + kOffRing, 16, 1024),
                       d_v = sdesc_sw128(sb + kOffRing, kChunk, 1024);
        const uint32_t t_s = tmem + 128u * w, t_o = tmem + kColO + 128u * w;
        uint32_t tile = 0, q_used = 0, p_used = 0, o_used = 0;
        auto ready = [&](uint32_t i, uint32_t parity) { return wait_inline<false>(bar(i), parity & 1u, guard); };
        auto keys_ready = [&](const Slots& s) {
          return ready(B_FULL + slot_of(s.key(0)), phase_of(s.key(0))) && ready(B_FULL + slot_of(s.key(1)), phase_of(s.key(1))) &&
                 ready(B_FULL + slot_of(s.key(2)), phase_of(s.key(2)));
        };
        // a chunk is free once both tiles' products that read it are done; `alone`: the other tile has none here
        auto release = [&](uint32_t chunk, bool alone) {
          umma_commit(bar(B_EMPTY + slot_of(chunk)));
          if (alone) umma_commit(bar(B_EMPTY + slot_of(chunk)));
        };
        auto scores = [&](const Slots& s, bool alone, bool last) {   // S = Q K^T
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const uint64_t a = d_q + c * (kChunk >> 4), b = d_ring + slot_of(s.key(c)) * (kChunk >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ss(t_s, a + 2u * k, b + 2u * k, idesc_qk, (c | k) ? 1u : 0u);
          }
          umma_commit(bar(B_SFULL + w));
#pragma unroll
          for (int c = 0; c < 3; ++c) release(s.key(c), alone);
          if (last) umma_commit(bar(B_QEMPTY + w));
        };
        Unit<kRows> u;
        bool failed = false;
        for (int n = 0; !failed && take_one(n, u); ++n) {
          mbar_arrive(bar(B_UEMPTY + (n & 1)));
          if (u.head < 0) break;
          const int end = u.end(w, p.causal), other = u.end(w ^ 1, p.causal);
          if (end > u.t0) {
            const Slots s(tile);
            if (!ready(B_QFULL + w, q_used++) || !keys_ready(s)) break;
            tc_fence_after();
            scores(s, u.t0 >= other, u.t0 + 1 == end);
          }
          for (int t = u.t0; t < end; ++t) {
            const Slots s(tile + (t - u.t0)), next(tile + (t - u.t0) + 1);
            const uint32_t v0 = s.value(0), v1 = s.value(1);
            if (!ready(B_FULL + slot_of(v0), phase_of(v0)) || !ready(B_FULL + slot_of(v1), phase_of(v1)) ||
                (t + 1 < end && !keys_ready(next)) || (t == u.t0 && !ready(B_OEMPTY + w, o_used++ ^ 1u)) ||
                !ready(B_PFULL + w, p_used)) {
              failed = true;
              break;
            }
            tc_fence_after();
            // O (+)= P V, 16 keys at a time; the first half while the second is still formed
            const uint64_t b = d_v + slot_of(v0) * (kChunk >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ts(t_o, t_s + 8u * k, b + 128u * k, idesc_pv, (t == u.t0 && k == 0) ? 0u : 1u);
            if (!ready(B_PFULL + 2 + w, p_used++)) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int k = 4; k < 8; ++k) umma_ts(t_o, t_s + 8u * k, b + 128u * k, idesc_pv, 1u);
            release(v0, t >= other);
            release(v1, t >= other);
            if (t + 1 < end) scores(next, t + 1 >= other, t + 2 == end);
            else umma_commit(bar(B_OFULL + w));
          }
          tile += max(end, other) - u.t0;
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
    // ---------------- softmax: row `r` of query tile w ----------------
    const int w = (warp - 4) >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + tl + 128u * w, t_o = tmem + tl + kColO + 128u * w;
    uint32_t s_used = 0, o_used = 0, tile = 0;
    bool failed = !ok;
    Unit<kRows> u;
    for (int n = 0; !failed && take(n, u); ++n) {
      const int end = u.end(w, p.causal), other = u.end(w ^ 1, p.causal), row = kRows * w + r;
      const int seen = row < u.rows ? u.visible(row, p.causal) : u.nk;
      const int least = kRows * w < u.rows ? u.visible(kRows * w, p.causal) : 0;  // keys that all rows see
      Row state{-INFINITY, 0.f};
      for (int t = u.t0; t < end; ++t) {
        if (!__all_sync(0xffffffffu, wait_inline<false>(bar(B_SFULL + w), s_used++ & 1, guard))) { failed = true; break; }
        tc_fence_after();
        const int rest = u.nk - t * kKeys;
        if (rest < kKeys) {
          // The value rows behind the document's keys may hold anything, and zero times NaN is NaN: they are cleared
          // before this tile's P is handed over (by both query tiles, with the same zeros).
          const Slots at(tile + (t - u.t0));
          const uint32_t v0 = at.value(0), v1 = at.value(1);
          if (!__all_sync(0xffffffffu, wait_inline<false>(bar(B_FULL + slot_of(v0)), phase_of(v0), guard) &&
                                           wait_inline<false>(bar(B_FULL + slot_of(v1)), phase_of(v1), guard))) {
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
        softmax_tile<kFp16>(state, t_s, t_o, p.scale_log2, (t + 1) * kKeys > least, seen - t * kKeys, t == u.t0, [&](int h) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PFULL + 2 * h + w));
        });
      }
      if (failed) break;
      tile += max(end, other) - u.t0;
      if (end > u.t0) {
        if (!__all_sync(0xffffffffu, wait_inline<false>(bar(B_OFULL + w), o_used++ & 1, guard))) break;
        tc_fence_after();
      }
      store_row<kFp16>(p, u, state, t_o, end > u.t0, row < u.rows, (int64_t)u.row + row, [&]() {
        tc_fence_before();   // O is read: the next unit may write it
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_OEMPTY + w));
      });
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
