// prefill_pair.cuh -- the attention of prefill.cuh, two CTAs on neighbouring SMs
// to a unit of 512 queries.
//
// Each product runs on both SMs' tensor cores (cta_group::2, M = 256): CTA r of
// the pair holds rows [128 r, 128 r + 128) of either query tile of 256, keys [64
// r, 64 r + 64) of a tile's K and dims [64 r, 64 r + 64) of its V, and the
// hardware brings the halves of K and V together. So an SM copies and keeps 40 KB
// of a tile of 128 keys where a CTA alone needs 80: two tiles fit beside the
// queries and the outputs on their way, and the L2 gives half the bytes (a CTA to
// 256 queries asked it for 7.5 TB/s and its ring of 1.6 tiles ran dry under that
// load).
//
// Measured (GB300, bf16): 2048 queries behind 32768 keys, 128 heads 2.82 ms in
// short runs (1.89 PFLOP/s, 1.01 of the cuBLAS burst) and 3.15 in long ones, where
// power lowers the clock to 1.72 GHz; 4 x 4096 causal 1.74 and 1.89 ms (0.84 and
// 0.77). In the steady state a chain takes some 3200 cycles a tile: 1600 from P to
// the next S (1280 of products, commits and arrivals across the pair), 1400 of
// softmax, and waits for the other chain's products. A unit's start and end: some
// 1200 cycles from its last P to its results, 2500 to write them, 4000 from there
// to the next unit's first scores (queries and keys on their way); and a causal
// unit's second tile sees two key tiles more than the first. Tried without gain:
// two threads a row (3.37 ms with one CTA a unit where one thread took 3.22: the
// exchanges cost more than the halves save), outputs by warps of their own, the
// running maximum left out of the steady state (it hides behind the exponentials),
// queries by a warp of their own or brought into the L2 ahead, keys a tile ahead
// of values, every stream polled (3.18 ms), three stages, the two issuing threads
// taking turns (3.02), waits that order memory in the CTA alone.
//
// Warp roles (384 threads a CTA): warp 0 copies this CTA's halves; in CTA 0 warps
// 1 and 3 issue the products of the first and the second query tile for both
// CTAs and warp 2 finds the units; warps 4-7 and 8-11 are the softmax of this
// CTA's rows of the two query tiles, one row a thread. Warp 1 of each CTA owns
// its TMEM. What the issuing threads wait for (copies, weights, accumulators
// that were read) arrives at barriers of CTA 0, from either CTA; what they
// complete is committed to both CTAs' barriers. Every wait is bounded; a wait
// that gives up sets the status word and the CTA unwinds.
#pragma once
#include "prefill.cuh"

namespace mla {
namespace prefill {
namespace pair {

constexpr int kTileRows = 2 * kRows;       // queries of a tile, of both CTAs
constexpr int kStages = 2;                 // tiles of K and of V held
constexpr uint32_t kKStage = kQTile / 2;   // 64 keys x 192 dims
constexpr uint32_t kVStage = kChunk;       // 128 keys x 64 dims
constexpr uint32_t kOffK = 2 * kQTile, kOffV = kOffK + kStages * kKStage, kOffOut = kOffV + kStages * kVStage,
                   kOffBar = kOffOut + 8 * kStage;
constexpr int kUnits = 4;                  // units looked up ahead of the slowest reader
using UnitP = Unit<kTileRows, 2>;
// Barriers of CTA 0: K, V, Q (from both CTAs' copies), P, O read, units read. Of each CTA: the others.
enum : uint32_t {
  B_KFULL = 0, B_KEMPTY = B_KFULL + kStages, B_VFULL = B_KEMPTY + kStages, B_VEMPTY = B_VFULL + kStages,
  B_QFULL = B_VEMPTY + kStages, B_QEMPTY = B_QFULL + 2, B_SFULL = B_QEMPTY + 2, B_PFULL = B_SFULL + 2, B_OFULL = B_PFULL + 4,
  B_OEMPTY = B_OFULL + 2, B_UFULL = B_OEMPTY + 2, B_UEMPTY = B_UFULL + kUnits, B_WANT = B_UEMPTY + kUnits, B_NEXT = B_WANT + 1,
  B_VTAIL = B_NEXT + 1, B_DRAIN = B_VTAIL + 1, B_STALL = B_DRAIN + 2, B_COUNT = B_STALL + 1
};
constexpr uint32_t kOffMisc = (kOffBar + 8 * B_COUNT + 15) / 16 * 16;
constexpr uint32_t kSmem = kOffMisc + 64 + 64 * kUnits + 1024;
static_assert(kSmem <= 232448 && UnitP::kWords <= 16);
constexpr int kUnitReaders = 11 + 9;       // CTA 0: producer, two issuing threads, eight softmax warps; CTA 1 without the issuers

// ---- the pair's forms of the tcgen05 and copy instructions ----
MLA_DEV void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}
MLA_DEV void tmem_relinquish_pair() { asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory"); }
MLA_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
MLA_DEV void umma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
MLA_DEV void umma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on the barrier at this offset in both CTAs when every product issued so far is done
MLA_DEV void umma_commit_both(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"((uint16_t)3)
               : "memory");
}
MLA_DEV void umma_commit_own(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// a copy into this CTA's shared memory, counted on a barrier of the pair (shared::cluster address)
MLA_DEV void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, uint32_t cluster_bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Nothing the thread wrote has to be visible with these arrivals, so they are relaxed ones: one that orders memory across
// the pair takes some 1000 cycles. The keys' is one of those all the same (kLate): with the other copies as early as they
// can be, keys that follow the values at once let the first query tile run ahead of the second until the ring holds it
// back, out of step on the tensor pipe (4 x 4096 causal 1926 us; 1754 so, 1767 with a pause of 1100 to 1600 cycles instead,
// 1879 and 1790 with 700 and 2200, 1776 with the values delayed and the keys not).
template <bool kLate = false>
MLA_DEV void mbar_arrive_expect_tx_cluster(uint32_t cluster_bar, uint32_t bytes) {
  if (kLate) asm volatile("mbarrier.arrive.expect_tx.release.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes) : "memory");
  else asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes) : "memory");
}
MLA_DEV void st_cluster_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// tm_q: dims {192, heads, tq}, tm_v: {128, heads, tk}: boxes {64, 1, 128}; tm_k: {128, heads, tk}, tm_r: {64, 1, tk}:
// boxes {64, 1, 64}; tm_out: {128, heads, tq}, box {64, 1, 32}; 128-byte swizzled.
template <bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ CUtensorMap tm_out, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both CTAs: the operands' descriptors and the barriers' addresses serve both
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + kOffMisc);  // 16-B aligned
  // misc: [0, 4) the answer of ask_next, 4 TMEM base, 5 abort, 6 ok, 7 status where none is given, 8 and 9 tiles of keys
  // and of values asked for, from 16 on the units
  volatile uint32_t* tmem_slot = misc + 4;
  volatile uint32_t* abort_flag = misc + 5;
  volatile uint32_t* ok_flag = misc + 6;
  int* units = reinterpret_cast<int*>(misc + 16);
  auto bar = [&](uint32_t i) { return sb + kOffBar + 8u * i; };
  auto lead_bar = [&](uint32_t i) { return mapa(bar(i), 0); };   // CTA 0's
  uint32_t* status = p.status ? p.status : misc + 7;
  const Guard guard{abort_flag, status, kWaitLimitCycles};
  const uint32_t issued = smem_u32(misc + 8);
  auto ready = [&](uint32_t i, uint32_t parity) { return wait_inline<true>(bar(i), parity & 1u, guard); };
  auto ready_all = [&](uint32_t i, uint32_t parity) { return __all_sync(0xffffffffu, ready(i, parity)) != 0; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(B_KFULL + s), 2);    // both CTAs' copies
      mbar_init(bar(B_KEMPTY + s), 2);   // both query tiles' products
      mbar_init(bar(B_VFULL + s), 2);
      mbar_init(bar(B_VEMPTY + s), 2);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(B_QFULL + w), 2);
      mbar_init(bar(B_QEMPTY + w), 1);
      mbar_init(bar(B_SFULL + w), 1);
      mbar_init(bar(B_PFULL + w), 8);
      mbar_init(bar(B_PFULL + 2 + w), 8);
      mbar_init(bar(B_OFULL + w), 1);
      mbar_init(bar(B_OEMPTY + w), 8);
      mbar_init(bar(B_DRAIN + w), 1);
    }
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(bar(B_UFULL + s), 1);
      mbar_init(bar(B_UEMPTY + s), kUnitReaders);
    }
    mbar_init(bar(B_WANT), 1);
    mbar_init(bar(B_NEXT), 1);
    mbar_init(bar(B_VTAIL), 1);
    mbar_init(bar(B_STALL), 1);
    *abort_flag = 0u;
    *ok_flag = 1u;
    misc[7] = misc[8] = misc[9] = 0u;
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
    tmem_alloc_pair(smem_u32(misc + 4), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // barriers and TMEM of both CTAs stand
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();  // nothing above reads global memory
  const uint32_t tmem = *tmem_slot;
  const bool ok = *ok_flag != 0u;

  // the readers' side of the units: the n-th one, into registers; one lane reads for a role of a single thread
  auto take_one = [&](int n, UnitP& u) {
    if (!ready(B_UFULL + n % kUnits, n / kUnits)) return false;
    u.read(units + 16 * (n % kUnits));
    return true;
  };
  // orders memory across the pair, so it is called where that delays nothing
  auto taken = [&](int n) {
    if (lane == 0) mbar_arrive_remote(lead_bar(B_UEMPTY + n % kUnits));
  };
  auto look = [&](int n, UnitP& u) { return __all_sync(0xffffffffu, take_one(n, u)) && u.head >= 0; };

  if (warp < 4) {
    set_registers_down<kRegsFew>();
    if (warp == 2 && rank == 0 && ok) {
      // ---------------- the units, for both CTAs ----------------
      Finder<UnitP> finder;
      finder.start();
      int64_t id = blockIdx.x >> 1;
      // A unit is taken only when the copies of the one before it come to their end: one taken early could not go to a
      // block that is free sooner.
      bool asking = false;
      int n = 0, asked = 0;
      const uint32_t peer_units = mapa(smem_u32(units), 1);
      while (true) {
        UnitP u{};
        u.head = -1;
        const bool found = id >= 0 && finder.find(p, id, u);
        if (found || id < 0) {
          const int s = n % kUnits;
          if (!ready_all(B_UEMPTY + s, (n / kUnits) ^ 1)) break;
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < UnitP::kWords; ++i) {
              units[16 * s + i] = u.word(i);
              st_cluster_u32(peer_units + 4u * (16 * s + i), (uint32_t)u.word(i));
            }
            mbar_arrive(bar(B_UFULL + s));
            mbar_arrive_remote(mapa(bar(B_UFULL + s), 1));
          }
          __syncwarp();
        }
        if (id < 0) break;
        record_bad(p, id, gridDim.x >> 1);
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
        id = id < 0 ? id : id >> 1;
        // read before the next answer is written over it
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (asking && lane == 0) {   // a wait gave up: the answer is still to be written
        const uint64_t t_0 = cycles();
        while (!mbar_try_wait(bar(B_NEXT), asked & 1) && cycles() - t_0 < kDrainLimitCycles) {}
      }
    } else if (warp == 0 && ok) {
      // ---------------- copies: this CTA's rows of the queries, its halves of the keys and values ----------------
      const bool leader = elect_one();
      if (leader) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_r);
        prefetch_tmap(&tm_v);
      }
      int n = 0;
      uint32_t tile = 0, q_loads[2] = {0, 0}, tails = 0;
      bool stop = false;
      UnitP u;
      auto queries = [&](int w) {
        if (!ready_all(B_QEMPTY + w, q_loads[w]++ ^ 1u)) {
          stop = true;
          return;
        }
        if (leader) {
          const uint32_t b = lead_bar(B_QFULL + w);
          mbar_arrive_expect_tx_cluster(b, kQTile);
          for (int c = 0; c < 3; ++c)
            tma_load_3d_pair(sb + w * kQTile + c * kChunk, &tm_q, b, 64 * c, u.head, u.row + kTileRows * w + kRows * rank);
        }
      };
      auto want_next = [&]() {
        if (leader && rank == 0) mbar_arrive(bar(B_WANT));
      };
      for (; !stop && look(n, u); ++n) {
        const int e0 = u.end(0, p.causal), e1 = u.end(1, p.causal), e = max(e0, e1);
        if (e0 > u.t0) queries(0);
        if (e - u.t0 < 2) want_next();
        if (e <= u.t0) taken(n);
        for (int t = u.t0; t < e && !stop; ++t, ++tile) {
          if (t == e - 2) want_next();
          const uint32_t s = tile % kStages, round = tile / kStages;
          const int at = u.k0 + t * kKeys, rest = u.nk - t * kKeys;
          if (!ready_all(B_KEMPTY + s, round ^ 1u)) { stop = true; break; }
          if (leader) {
            const uint32_t b = lead_bar(B_KFULL + s), to = sb + kOffK + s * kKStage;
            mbar_arrive_expect_tx_cluster<true>(b, kKStage);
            tma_load_3d_pair(to, &tm_k, b, 0, u.head, at + 64 * rank);
            tma_load_3d_pair(to + kChunk / 2, &tm_k, b, 64, u.head, at + 64 * rank);
            tma_load_3d_pair(to + kChunk, &tm_r, b, 0, 0, at + 64 * rank);
            set_issued(issued, tile + 1u);
          }
          // the second query tile is wanted after the first one's scores
          if (t == u.t0 && e1 > u.t0) queries(1);
          if (stop || !ready_all(B_VEMPTY + s, round ^ 1u)) { stop = true; break; }
          if (leader) set_issued(issued + 4u, tile + 1u);
          const uint32_t b = lead_bar(B_VFULL + s), to = sb + kOffV + s * kVStage;
          if (rest >= kKeys) {
            if (leader) {
              mbar_arrive_expect_tx_cluster(b, kVStage);
              tma_load_3d_pair(to, &tm_v, b, 64 * rank, u.head, at);
            }
            if (t == u.t0) taken(n);
            continue;
          }
          // The value rows behind the document's keys may hold anything, and zero times NaN is NaN: they are cleared
          // before the tile is handed over.
          if (leader) {
            mbar_arrive_expect_tx(bar(B_VTAIL), kVStage);
            tma_load_3d_plain(to, &tm_v, bar(B_VTAIL), 64 * rank, u.head, at);
          }
          __syncwarp();
          if (!ready_all(B_VTAIL, tails++)) { stop = true; break; }
          for (int i = rest * 8 + lane; i < kKeys * 8; i += 32) st_shared_v4(to + 16u * i, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (leader) mbar_arrive_remote(b);
          if (t == u.t0) taken(n);
        }
      }
    } else if ((warp & 1) && rank == 0 && ok) {
      // ---------------- products of query tile w, for both CTAs: one thread ----------------
      // The pipe takes an instruction about when it starts it, so a wait between two of them idles it, but for the
      // other tile's: all that can be waited for while the softmax runs (the next keys, the values) is, and the
      // products of a tile and the scores of the next follow in one go.
      const int w = warp >> 1;
      if (elect_one()) {
        constexpr uint32_t idesc_qk = idesc_f16(kTileRows, kKeys, !kFp16, false, false);
        constexpr uint32_t idesc_pv = idesc_f16(kTileRows, kV, !kFp16, false, true);
        const uint64_t d_q = sdesc_sw128(sb + w * kQTile, 16, 1024), d_k = sdesc_sw128(sb + kOffK, 16, 1024),
                       d_v = sdesc_sw128(sb + kOffV, kChunk, 1024);
        const uint32_t t_s = tmem + 128u * w, t_o = tmem + kColO + 128u * w;
        uint32_t tile = 0, q_used = 0, p_used = 0, o_used = 0;
        // a stage is free once both tiles' products that read it are done; `alone`: the other tile has none here
        auto release = [&](uint32_t i, bool alone) {
          umma_commit_both(bar(i));
          if (alone) umma_commit_both(bar(i));
        };
        auto scores = [&](uint32_t k_tile, bool alone, bool last) {   // S = Q K^T
          const uint32_t s = k_tile % kStages;
          const uint64_t k0 = d_k + s * (kKStage >> 4);
#pragma unroll
          for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_ss_pair(t_s, d_q + (c * (kChunk >> 4) + 2u * k), k0 + (c * (kChunk >> 5) + 2u * k), idesc_qk, (c | k) ? 1u : 0u);
          umma_commit_both(bar(B_SFULL + w));
          release(B_KEMPTY + s, alone);
          if (last) umma_commit_both(bar(B_QEMPTY + w));
        };
        // tiles of the other query tile only are not waited for
        auto keys_ready = [&](uint32_t k_tile) {
          return wait_issued(issued, k_tile, guard) && ready(B_KFULL + k_tile % kStages, k_tile / kStages);
        };
        auto values_ready = [&](uint32_t v_tile) {
          return wait_issued(issued + 4u, v_tile, guard) && ready(B_VFULL + v_tile % kStages, v_tile / kStages);
        };
        UnitP u;
        bool failed = false;
        for (int n = 0; !failed && take_one(n, u); ++n) {
          mbar_arrive(bar(B_UEMPTY + n % kUnits));
          if (u.head < 0) break;
          const int end = u.end(w, p.causal), other = u.end(w ^ 1, p.causal);
          if (end > u.t0) {
            if (!ready(B_QFULL + w, q_used++) || !keys_ready(tile)) break;
            tc_fence_after();
            scores(tile, u.t0 >= other, u.t0 + 1 == end);
          }
          for (int t = u.t0; t < end; ++t) {
            const uint32_t at = tile + (uint32_t)(t - u.t0), s = at % kStages;
            if (!values_ready(at) || (t + 1 < end && !keys_ready(at + 1)) ||
                (t == u.t0 && !ready(B_OEMPTY + w, o_used++ ^ 1u)) || !ready(B_PFULL + w, p_used)) {
              failed = true;
              break;
            }
            tc_fence_after();
            // O (+)= P V, 16 keys at a time; the first half while the second is still formed
            const uint64_t v0 = d_v + s * (kVStage >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ts_pair(t_o, t_s + 8u * k, v0 + 128u * k, idesc_pv, (t == u.t0 && k == 0) ? 0u : 1u);
            if (!ready(B_PFULL + 2 + w, p_used++)) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int k = 4; k < 8; ++k) umma_ts_pair(t_o, t_s + 8u * k, v0 + 128u * k, idesc_pv, 1u);
            release(B_VEMPTY + s, t >= other);
            if (t + 1 < end) scores(at + 1, t + 1 >= other, t + 2 == end);
            else umma_commit_both(bar(B_OFULL + w));
          }
          tile += max(end, other) - u.t0;
        }
        // every product this thread issued has completed before TMEM and the pair's memory are released
        umma_commit_own(bar(B_DRAIN + w));
        const uint64_t t_0 = cycles();
        while (!mbar_try_wait(bar(B_DRAIN + w), 0) && cycles() - t_0 < kDrainLimitCycles) {}
      }
      __syncwarp();
    }
  } else {
    set_registers_up<kRegsMany>();
    // ---------------- softmax: row `r` of this CTA's half of query tile w ----------------
    const int w = (warp - 4) >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + tl + 128u * w, t_o = tmem + tl + kColO + 128u * w;
    const int first_row = kTileRows * w + kRows * rank, row = first_row + r;
    // What a warp hands to CTA 0 lies in TMEM, written before (tcgen05.wait::st): no memory of its own has to be
    // visible with it, so the arrival is a relaxed one, half as long on its way as a release.
    auto arrive = [&](uint32_t i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(bar(i));
        else mbar_arrive_remote_relaxed(lead_bar(i));
      }
    };
    uint32_t s_used = 0, o_used = 0;
    bool failed = !ok;
    UnitP u;
    for (int n = 0; !failed && look(n, u); ++n) {
      const int end = u.end(w, p.causal);
      const int seen = row < u.rows ? u.visible(row, p.causal) : u.nk;
      const bool idle = first_row >= u.rows;                                  // none of this CTA's rows is a query
      const int least = idle ? 0 : u.visible(first_row, p.causal);            // keys that all rows see
      Row state{-INFINITY, 0.f};
      for (int t = u.t0; t < end; ++t) {
        if (!ready_all(B_SFULL + w, s_used++)) { failed = true; break; }
        tc_fence_after();
        if (idle) {        // the rows' products are of no query: any P will do
          arrive(B_PFULL + w);
          arrive(B_PFULL + 2 + w);
          continue;
        }
        softmax_tile<kFp16>(state, t_s, t_o, p.scale_log2, (t + 1) * kKeys > least, seen - t * kKeys, t == u.t0,
                            [&](int h) { arrive(B_PFULL + 2 * h + w); });
      }
      if (failed) break;
      taken(n);      // ahead of the unit's results: it would wait for their stores, some 2000 cycles
      if (end > u.t0) {
        if (!ready_all(B_OFULL + w, o_used++)) break;
        tc_fence_after();
      }
      if (idle) {
        if (end > u.t0) arrive(B_OEMPTY + w);
        continue;
      }
      // O is read: the next unit may write it
      store_rows<kFp16>(p, &tm_out, sb + kOffOut + (warp - 4) * kStage, u, state, t_o, end > u.t0, first_row + 32 * (warp & 3),
                        [&]() { arrive(B_OEMPTY + w); });
    }
    if (lane == 0) bulk_wait();
  }
  // Never leave with a copy in flight into this CTA's shared memory. Without a fault every copy has been waited for, by
  // the issuing threads or where it was asked for. With one, the last copies may be counted on barriers of CTA 0 that
  // wait for the other CTA's in vain, so the pair stays for longer than any copy takes.
  __syncthreads();
  if (warp == 0 && ok && *abort_flag) {
    const uint64_t t_0 = cycles();
    while (cycles() - t_0 < kDrainLimitCycles) {}
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // CTA 0's products read CTA 1's memory, and arrivals cross until here
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace pair
}  // namespace prefill
}  // namespace mla
