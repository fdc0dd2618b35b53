// prefill.cuh -- attention of many new tokens in MLA's expanded form, sm_103a.
//
// For document b, head h and its query i of n_q, over the keys j < vis(i):
//     s_j = scale (q^C . k^C_j + q^R . k^R_j)          (128 + 64 dims; k^R is shared by the heads)
//     out = sum_j softmax(s)_j v_j (128 dims),   lse = ln sum_j exp s_j
// vis(i) = n_k, or causal (the last query sees all keys) n_k - n_q + i + 1, at
// least prefix_b (a prefix that every query sees). 640 FLOP a visible pair and
// head, where the decode's absorbed form takes 2176.
//
// A unit is 256 consecutive queries of one (document, head): two query tiles of
// 128 rows, which share every tile of 128 keys and values and take turns on the
// tensor pipe: while one tile's scores go through the softmax, the pipe
// multiplies for the other. S (fp32) and P (16 bits, over the S that it comes
// from) and both accumulators fill TMEM: 2 x 128 + 2 x 128 columns.
//
// The softmax is online with a lazy reference: the reference maximum of a row
// moves only when a score passes it by more than 2^8 (P and its sum stay far
// from the types' limits), so that the accumulator is rarely rescaled.
//
// Blocks are persistent: the next unit is a block of the grid that has not
// started yet, which the block cancels and takes over (clusterlaunchcontrol), so
// that units of unequal length even out without a counter in memory.
//
// Few rows over long keys: a unit's key tiles are cut into pieces (p.splits at
// most), whose partial outputs mla_prefill_combine_kernel joins.
//
// Warp roles (384 threads): warp 0 issues the copies, warps 1 and 3 the MMAs of
// the first and the second query tile (warp 1 owns TMEM), warp 2 finds the
// units, warps 4-7 and 8-11 are the softmax of the two query tiles, one row a
// thread. Every wait is bounded; a wait that
// gives up sets the status word and the CTA unwinds.
#pragma once
#include <cuda.h>

#include "params.h"
#include "pipe.cuh"
#include "ptx.cuh"

namespace mla {
namespace prefill {

constexpr int kThreads = 384;
constexpr int kRows = 128;                 // queries of a tile (UMMA M)
constexpr int kBlock = 2 * kRows;          // queries of a unit
constexpr int kKeys = 128;                 // keys of a tile
constexpr int kNope = 128, kRopeDim = 64, kQk = kNope + kRopeDim, kV = 128;
constexpr int kPieceTiles = 8;             // key tiles that a piece of a cut unit has at least
constexpr uint32_t kChunk = 128 * 128;     // 128 rows x 128 bytes (64 dims)
constexpr uint32_t kQTile = 3 * kChunk;
constexpr int kRing = 8;                   // chunks: three of K, two of V a tile
constexpr uint32_t kOffRing = 2 * kQTile;
constexpr uint32_t kOffBar = kOffRing + kRing * kChunk;
enum : uint32_t {
  B_FULL = 0, B_EMPTY = B_FULL + kRing, B_QFULL = B_EMPTY + kRing, B_QEMPTY = B_QFULL + 2, B_SFULL = B_QEMPTY + 2,
  B_PFULL = B_SFULL + 2, B_OFULL = B_PFULL + 2, B_OEMPTY = B_OFULL + 2, B_UFULL = B_OEMPTY + 2, B_UEMPTY = B_UFULL + 2,
  B_NEXT = B_UEMPTY + 2, B_DRAIN = B_NEXT + 1, B_STALL = B_DRAIN + 2, B_COUNT = B_STALL + 1
};
constexpr uint32_t kOffMisc = (kOffBar + 8 * B_COUNT + 15) / 16 * 16;
constexpr uint32_t kSmem = kOffMisc + 256 + 1024;
constexpr uint32_t kColO = 256;            // TMEM: S_w at 128 w (P_w over it), O_w at 256 + 128 w
constexpr int kUnitReaders = 11;           // producer, two MMA and eight softmax warps

struct PrefillParams {
  const int32_t* cu_q;         // [batch + 1]
  const int32_t* cu_k;
  const int32_t* prefix;       // [batch] or null
  int64_t tq, tk;              // rows of q and of k, v
  int batch, heads, causal;
  int splits;                  // most pieces of a unit
  float scale, scale_log2;
  void* out;                   // [tq, heads, 128]
  int64_t out_token, out_head; // strides in elements
  float* lse;                  // [tq, heads]
  float* o_part;               // [splits][tq][heads][128], splits > 1
  float* lse_part;             // [splits][tq][heads]
  uint32_t* status;            // or null
  uint32_t stall_cycles;       // test hook, 0 in normal use
};

// One document's rows, kept inside the tensors whatever the offsets hold.
struct Span {
  int q0, nq, k0, nk, prefix;
  bool bad;
};
MLA_DEV Span span_of(const PrefillParams& p, int b) {
  const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
  Span s;
  s.bad = q0 < 0 || q1 < q0 || q1 > p.tq || k0 < 0 || k1 < k0 || k1 > p.tk;
  s.q0 = q0;
  s.k0 = k0;
  s.nq = s.bad ? 0 : q1 - q0;
  s.nk = s.bad ? 0 : k1 - k0;
  s.prefix = p.prefix ? min(max(__ldg(p.prefix + b), 0), s.nk) : 0;
  return s;
}
// keys that query i of a document sees
MLA_DEV int visible(const PrefillParams& p, const Span& s, int i) {
  return p.causal ? min(max(s.nk - s.nq + i + 1, s.prefix), s.nk) : s.nk;
}
MLA_DEV int pieces_of(const PrefillParams& p, int tiles) {
  return max(1, min(p.splits, tiles / kPieceTiles));
}

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

// A unit as its readers see it (one piece of 256 queries of a head).
struct Unit {
  int head;       // < 0: no more units
  int row;        // first row of q and out
  int rows;       // queries of the unit
  int k0, nk;     // keys of the document
  int seen;       // keys that its query 0 sees, before the clamp to [prefix, nk]
  int prefix;
  int t0, t1;     // key tiles of this piece
  int piece, pieces;
  // keys that row r sees
  MLA_DEV int visible(int r, int causal) const { return causal ? min(max(seen + r, prefix), nk) : nk; }
  // end of the piece's key tiles for query tile w
  MLA_DEV int end(int w, int causal) const {
    const int last = min(rows, kRows * (w + 1)) - 1;
    return last < kRows * w ? t0 : max(t0, min(t1, (visible(last, causal) + kKeys - 1) / kKeys));
  }
};

// Units in the order of the grid: documents, heads, blocks of 256 queries (those that see most first), pieces. The
// warp holds 32 documents' counts and moves on only.
struct Finder {
  int base;            // first of the 32 documents
  int64_t before;      // blocks (of one head) times heads before them
  int blocks;          // of this lane's document
  int64_t upto;        // inclusive prefix over the lanes, times heads
  int lane;
  MLA_DEV void load(const PrefillParams& p) {
    const int b = base + lane;
    blocks = 0;
    if (b < p.batch) {
      const Span s = span_of(p, b);
      blocks = (s.nq + kBlock - 1) / kBlock;
      if (s.bad && p.status) atomicOr(p.status, STATUS_INDEX);
    }
    int incl = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    upto = (int64_t)incl * p.heads;
  }
  MLA_DEV void start(const PrefillParams& p) {
    lane = threadIdx.x & 31;
    base = 0;
    before = 0;
    load(p);
  }
  // the unit of block `id` of the grid; false if there is none (a piece that its unit does not have)
  MLA_DEV bool find(const PrefillParams& p, int64_t id, Unit& u, bool& past) {
    const int64_t block = id / p.splits;
    const int piece = (int)(id - block * p.splits);
    past = false;
    int64_t all = __shfl_sync(0xffffffffu, upto, 31);
    while (block >= before + all) {
      if (base + 32 >= p.batch) {
        past = true;
        return false;
      }
      before += all;
      base += 32;
      load(p);
      all = __shfl_sync(0xffffffffu, upto, 31);
    }
    const int64_t at = block - before;
    const int which = __ffs(__ballot_sync(0xffffffffu, at < upto)) - 1;
    const int n = __shfl_sync(0xffffffffu, blocks, which);
    const int64_t first = __shfl_sync(0xffffffffu, upto, which) - (int64_t)n * p.heads;
    const int in = (int)(at - first), head = in / n, qb = n - 1 - (in - head * n);
    const Span s = span_of(p, base + which);
    u.head = head;
    u.row = s.q0 + qb * kBlock;
    u.rows = min(kBlock, s.nq - qb * kBlock);
    u.k0 = s.k0;
    u.nk = s.nk;
    u.seen = s.nk - s.nq + qb * kBlock + 1;
    u.prefix = s.prefix;
    const int tiles = (u.visible(u.rows - 1, p.causal) + kKeys - 1) / kKeys;
    u.piece = piece;
    u.pieces = pieces_of(p, tiles);
    if (piece >= u.pieces) return false;
    u.t0 = (int)((int64_t)tiles * piece / u.pieces);
    u.t1 = (int)((int64_t)tiles * (piece + 1) / u.pieces);
    return true;
  }
};

// asks for a block of the grid that has not started: 16 bytes at `dst`, counted on `bar`
MLA_DEV void ask_next(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
               "r"(bar)
               : "memory");
}
// its number, or -1
MLA_DEV int64_t answer_next(uint32_t src) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x) : "r"(src) : "memory");
  return got ? (int64_t)x : -1;
}

// A bounded wait without a call (a kernel that moves registers between its warps makes none).
MLA_DEV bool wait_inline(uint32_t bar, uint32_t parity, const Guard& g) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = cycles();
  while (!*g.abort) {
    if (mbar_try_wait(bar, parity)) return true;
    if (cycles() - t0 > g.limit) {
      *g.abort = 1u;
      atomicOr(g.status, STATUS_TIMEOUT);
    }
  }
  return false;
}
template <int kN>
MLA_DEV void set_registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN)); }
template <int kN>
MLA_DEV void set_registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN)); }
// The launch gives each thread 168 registers, 64512 in all; the four warps of the first group hand theirs on to the
// eight softmax warps, which hold a row of 128 scores: 128 x 120 + 256 x 192 = 64512.
constexpr int kRegsLaunch = 168, kRegsFew = 120, kRegsMany = 192;
static_assert(128 * kRegsFew + 256 * kRegsMany <= kThreads * kRegsLaunch);

template <bool kFp16>
MLA_DEV uint32_t pack_p(float lo, float hi) {
  return kFp16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// tm_q: dims {192, heads, tq}; tm_k: {128, heads, tk}; tm_r: {64, 1, tk}; tm_v: {128, heads, tk}; boxes {64, 1, 128},
// 128-byte swizzled.
template <bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
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
  auto take_one = [&](int n, Unit& u) {
    const int s = n & 1;
    if (!wait_inline(bar(B_UFULL + s), (n >> 1) & 1, guard)) return false;
    const volatile int* at = units + 16 * s;
    u.head = at[0]; u.row = at[1]; u.rows = at[2]; u.k0 = at[3]; u.nk = at[4]; u.seen = at[5]; u.prefix = at[6];
    u.t0 = at[7]; u.t1 = at[8]; u.piece = at[9]; u.pieces = at[10];
    return true;
  };
  auto take = [&](int n, Unit& u) {
    const bool got = __all_sync(0xffffffffu, take_one(n, u));
    if (got && lane == 0) mbar_arrive(bar(B_UEMPTY + (n & 1)));
    return got && u.head >= 0;
  };

  if (warp < 4) {
    set_registers_down<kRegsFew>();
    if (warp == 2 && ok) {
      // ---------------- the units ----------------
      Finder finder;
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
        Unit u;
        u.head = -1;
        bool past = false;
        const bool found = more && finder.find(p, id, u, past);
        if (found || !more) {
          if (!__all_sync(0xffffffffu, wait_inline(bar(B_UEMPTY + (n & 1)), ((n >> 1) & 1) ^ 1, guard))) break;
          if (lane == 0) {
            int* at = units + 16 * (n & 1);
            at[0] = u.head;
            if (found) {
              at[1] = u.row; at[2] = u.rows; at[3] = u.k0; at[4] = u.nk; at[5] = u.seen; at[6] = u.prefix;
              at[7] = u.t0; at[8] = u.t1; at[9] = u.piece; at[10] = u.pieces;
            }
            mbar_arrive(bar(B_UFULL + (n & 1)));
          }
          __syncwarp();
          ++n;
        }
        if (!more) break;
        if (!__all_sync(0xffffffffu, wait_inline(bar(B_NEXT), asked & 1, guard))) break;
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
      Unit u;
      auto chunk = [&](const CUtensorMap* m, int x, int y, int z) {
        const uint32_t slot = slot_of(loads);
        if (stop || !__all_sync(0xffffffffu, wait_inline(bar(B_EMPTY + slot), phase_of(loads) ^ 1u, guard))) {
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
        if (stop || !__all_sync(0xffffffffu, wait_inline(bar(B_QEMPTY + w), (q_loads[w] & 1) ^ 1, guard))) {
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
        auto ready = [&](uint32_t i, uint32_t parity) { return wait_inline(bar(i), parity & 1u, guard); };
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
        Unit u;
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
                !ready(B_PFULL + w, p_used++)) {
              failed = true;
              break;
            }
            tc_fence_after();
            const uint64_t b = d_v + slot_of(v0) * (kChunk >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)   // O (+)= P V
              umma_ts(t_o, t_s + 8u * k, b + 128u * k, idesc_pv, (t == u.t0 && k == 0) ? 0u : 1u);
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
    const float sl2 = p.scale_log2;
    const float slack = 8.f / sl2;        // raw score units
    uint32_t s_used = 0, o_used = 0, tile = 0;
    bool failed = !ok;
    Unit u;
    for (int n = 0; !failed && take(n, u); ++n) {
      const int end = u.end(w, p.causal), other = u.end(w ^ 1, p.causal), row = kRows * w + r;
      const int seen = row < u.rows ? u.visible(row, p.causal) : u.nk;
      const int least = kRows * w < u.rows ? u.visible(kRows * w, p.causal) : 0;  // keys that all rows see
      float m = -INFINITY, l = 0.f;
      for (int t = u.t0; t < end; ++t) {
        if (!__all_sync(0xffffffffu, wait_inline(bar(B_SFULL + w), s_used & 1, guard))) { failed = true; break; }
        ++s_used;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32u * c, s + 32 * c);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) pin_regs32(s + 32 * c);
        if ((t + 1) * kKeys > least) {
          const int left = seen - t * kKeys;
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k >= left) s[k] = 0xFF800000u;  // -inf
          const int rest = u.nk - t * kKeys;
          if (rest < kKeys) {
            // The value rows behind the document's keys may hold anything, and zero times NaN is NaN: they are cleared
            // before this tile's P is handed over (by both query tiles, with the same zeros).
            const Slots at(tile + (t - u.t0));
            const uint32_t v0 = at.value(0), v1 = at.value(1);
            if (!__all_sync(0xffffffffu, wait_inline(bar(B_FULL + slot_of(v0)), phase_of(v0), guard) &&
                                             wait_inline(bar(B_FULL + slot_of(v1)), phase_of(v1), guard))) {
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
        }
        const float top = fmaxf(tree_max64([&](int k) { return __uint_as_float(s[k]); }),
                                tree_max64([&](int k) { return __uint_as_float(s[64 + k]); }));
        const bool move = top > m + slack;   // from -inf with the first key that it sees
        if (__any_sync(0xffffffffu, move)) {
          const float next = move ? top : m;
          // rows that have seen nothing keep l = 0 and O = 0
          const float f = move ? exp2_approx((m - next) * sl2) : 1.f;
          m = next;
          l *= f;
          if (t > u.t0) {
            // S of this tile is complete, and with it every product issued before: O holds still until this
            // tile's P is handed over
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld16(t_o + 16u * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                asm volatile("" : "+r"(o[k]));
                o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              }
              tmem_st16(t_o + 16u * c, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : -m * sl2;
        const uint64_t scale2 = f2_pack(sl2, sl2), ref2 = f2_pack(ref, ref);
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t q[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = f2_unpack(f2_fma(f2_pack(__uint_as_float(s[32 * c + 2 * k]), __uint_as_float(s[32 * c + 2 * k + 1])), scale2, ref2));
            const float a = exp2_approx(x.x), b = exp2_approx(x.y);
            sum[k & 3] = f2_add(sum[k & 3], f2_pack(a, b));
            q[k] = pack_p<kFp16>(a, b);
          }
          tmem_st16(t_s + 16u * c, q);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL + w));
        const float2 x = f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])));
        l += x.x + x.y;
      }
      if (failed) break;
      tile += max(end, other) - u.t0;
      const bool live = row < u.rows;
      const int64_t at = (int64_t)u.row + row;
      const float inv = l > 0.f ? 1.f / l : l;   // NaN stays
      const bool whole = u.pieces == 1;
      if (end > u.t0) {
        if (!__all_sync(0xffffffffu, wait_inline(bar(B_OFULL + w), o_used & 1, guard))) { failed = true; break; }
        ++o_used;
        tc_fence_after();
      }
      if (live) {
        const float lse = l == 0.f ? -INFINITY : m * p.scale + logf(l);
        if (whole) p.lse[at * p.heads + u.head] = lse;
        else p.lse_part[((int64_t)u.piece * p.tq + at) * p.heads + u.head] = lse;
      }
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * p.out_token + u.head * p.out_head);
      float4* part = reinterpret_cast<float4*>(p.o_part + (((int64_t)u.piece * p.tq + at) * p.heads + u.head) * kV);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (end > u.t0) {
          tmem_ld32(t_o + 32u * c, o);
          tmem_wait_ld();
          pin_regs32(o);
          if (c == 3) {   // O is read: the next unit may write it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_OEMPTY + w));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (live) {
          // a row that sees nothing has l = 0 and gets zeros
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]) * inv;
          if (whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[4 * c + k] = make_uint4(pack_p<kFp16>(v[8 * k], v[8 * k + 1]), pack_p<kFp16>(v[8 * k + 2], v[8 * k + 3]),
                                          pack_p<kFp16>(v[8 * k + 4], v[8 * k + 5]), pack_p<kFp16>(v[8 * k + 6], v[8 * k + 7]));
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) part[8 * c + k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
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

// Joins the pieces of cut units: out = sum_i e^(lse_i - m) o_i / sum_i e^(lse_i - m), lse = m + ln sum. A warp to a
// (row, head), four dims a lane; rows whose unit was not cut are left as they are.
constexpr int kCombineThreads = 256;

template <bool kFp16>
__global__ void __launch_bounds__(kCombineThreads) mla_prefill_combine_kernel(const PrefillParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5);
  if (item >= p.tq * p.heads) return;
  const int64_t row = item / p.heads;
  const int head = (int)(item - row * p.heads);
  // the last document that starts at or before the row (empty ones before it start there too)
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_q + mid) <= row) lo = mid;
    else hi = mid;
  }
  const Span s = span_of(p, lo);
  if (row < s.q0 || row >= (int64_t)s.q0 + s.nq) return;   // behind the last document
  const int i = (int)(row - s.q0), last = min((i / kBlock + 1) * kBlock, s.nq) - 1;
  const int pieces = pieces_of(p, (visible(p, s, last) + kKeys - 1) / kKeys);
  if (pieces == 1) return;
  float m = -INFINITY;
  for (int k = 0; k < pieces; ++k) m = fmaxf(m, p.lse_part[((int64_t)k * p.tq + row) * p.heads + head]);
  const float ref = m == -INFINITY ? 0.f : m;
  float total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < pieces; ++k) {
    const int64_t at = ((int64_t)k * p.tq + row) * p.heads + head;
    const float f = expf(p.lse_part[at] - ref);
    const float4 v = reinterpret_cast<const float4*>(p.o_part + at * kV)[lane];
    total += f;
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  }
  const float inv = total > 0.f ? 1.f / total : total;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * p.out_token + head * p.out_head);
  dst[lane] = make_uint2(pack_p<kFp16>(acc.x * inv, acc.y * inv), pack_p<kFp16>(acc.z * inv, acc.w * inv));
  if (lane == 0) p.lse[item] = total == 0.f ? -INFINITY : ref + logf(total);
}

}  // namespace prefill
}  // namespace mla
