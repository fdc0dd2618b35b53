// prefill.cuh -- attention of many new tokens in MLA's expanded form, sm_103a:
// what its two kernels (prefill_pair.cuh, prefill_few.cuh) share, and the join
// of cut units.
//
// For document b, head h and its query i of n_q, over the keys j < vis(i):
//     s_j = scale (q^C . k^C_j + q^R . k^R_j)          (128 + 64 dims; k^R is shared by the heads)
//     out = sum_j softmax(s)_j v_j (128 dims),   lse = ln sum_j exp s_j
// vis(i) = n_k, or causal (the last query sees all keys) n_k - n_q + i + 1, at
// least prefix_b (a prefix that every query sees). 640 FLOP a visible pair and
// head, where the decode's absorbed form takes 2176.
//
// A unit is a block of consecutive queries of one (document, head). Two chains
// of score tile -> softmax -> product take turns on the tensor pipe: while one
// goes through the softmax, the pipe multiplies for the other. They are two query
// tiles over the same keys (prefill_pair.cuh) or every other key tile of the same
// queries (prefill_few.cuh). A chain's S (fp32), P (16 bits, over the S that it
// comes from) and accumulator take 256 columns of TMEM: two fill it.
//
// The softmax is online with a lazy reference: the reference maximum of a row
// moves only when a score passes it by more than 2^8 (P and its sum stay far
// from the types' limits), so that the accumulator is rarely rescaled. A weight
// is 2^(c s - c m), c = scale log2 e, its exponent one fma of s with the rounded
// c m: that rounding, up to 2^-25 c |m|, is the same for all of a row's weights
// and cancels, but where c |m| is large it would take them out of their types'
// range, or to zero. Such rows (beyond kFar) subtract first.
//
// Blocks are persistent: the next unit is a block of the grid that has not
// started yet, which the block cancels and takes over (clusterlaunchcontrol), so
// that units of unequal length even out without a counter in memory.
//
// Few rows over long keys: a unit's key tiles are cut into pieces (p.splits at
// most), whose accumulators, references and sums mla_prefill_combine_kernel
// joins. References and sums stay apart: a piece's lse would round away the sum
// beside a large reference. The sums stand in the row of the output that the
// join writes.
#pragma once
#include <cuda.h>

#include "params.h"
#include "pipe.cuh"
#include "ptx.cuh"

namespace mla {
namespace prefill {

constexpr int kThreads = 384;
constexpr int kRows = 128;                 // rows of a CTA in a query tile (TMEM lanes)
constexpr int kKeys = 128;                 // keys of a tile
constexpr int kNope = 128, kRopeDim = 64, kQk = kNope + kRopeDim, kV = 128;
constexpr int kPieceTiles = 8;             // key tiles that a piece of an average unit has at least
constexpr uint32_t kChunk = 128 * 128;     // 128 rows x 128 bytes (64 dims)
constexpr uint32_t kQTile = 3 * kChunk;
constexpr uint32_t kColO = 256;            // TMEM: S of chain w at 128 w (P over it), its accumulator at 256 + 128 w

struct PrefillParams {
  const int32_t* cu_q;         // [batch + 1]
  const int32_t* cu_k;
  const int32_t* prefix;       // [batch] or null
  int64_t tq, tk;              // rows of q and of k, v
  int batch, heads, causal;
  int splits;                  // most pieces of a unit
  int piece_tiles;             // key tiles of a piece
  float scale, scale_log2;
  void* out;                   // [tq, heads, 128]
  int64_t out_token, out_head; // strides in elements
  float* lse;                  // [tq, heads]
  float* o_part;               // [splits][tq][heads][128], splits > 1
  float* ref_part;             // [splits][tq][heads]: raw references
  int wide;                    // 1: rows of out are 32-B aligned, 2: those of o_part
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
  return max(1, min(p.splits, (tiles + p.piece_tiles - 1) / p.piece_tiles));
}

// A unit as its readers see it: one piece of a block of queries of a head, in kTiles query tiles of kTileRows rows.
template <int kTileRows, int kTiles>
struct Unit {
  static constexpr int kBlock = kTileRows * kTiles;
  int head;       // < 0: no more units
  int row;        // first row of q and out
  int rows;       // queries of the unit
  int k0, nk;     // keys of the document
  int seen;       // keys that its query 0 sees, before the clamp to [prefix, nk]
  int prefix;
  int t0, t1;     // key tiles of this piece
  int piece, pieces;
  static constexpr int kWords = 11;
  // keys that row r sees
  MLA_DEV int visible(int r, int causal) const { return causal ? min(max(seen + r, prefix), nk) : nk; }
  // end of the piece's key tiles for query tile w
  MLA_DEV int end(int w, int causal) const {
    const int last = min(rows, kTileRows * (w + 1)) - 1;
    return last < kTileRows * w ? t0 : max(t0, min(t1, (visible(last, causal) + kKeys - 1) / kKeys));
  }
  MLA_DEV void read(const volatile int* at) {
    head = at[0]; row = at[1]; rows = at[2]; k0 = at[3]; nk = at[4]; seen = at[5]; prefix = at[6];
    t0 = at[7]; t1 = at[8]; piece = at[9]; pieces = at[10];
  }
  MLA_DEV int word(int k) const {
    return k == 0 ? head : k == 1 ? row : k == 2 ? rows : k == 3 ? k0 : k == 4 ? nk : k == 5 ? seen : k == 6 ? prefix
         : k == 7 ? t0 : k == 8 ? t1 : k == 9 ? piece : pieces;
  }
};

// Units in the order of the grid: documents, heads, blocks of queries (those that see most first), pieces. The warp
// holds 32 documents' counts; the blocks of the grid that it is given lie further on each time, or it starts over. Of
// the 32 those with most keys come first, so that short units are left for the end (8 x 4 queries over 5461 to 16384
// keys 121 us, 130 in the order given; 24 documents of 1 to 2048 tokens 300, 305).
template <class U>
struct Finder {
  static constexpr int kBlock = U::kBlock;
  int base;            // first of the 32 documents, -32: none looked at
  int64_t before;      // blocks (of one head) times heads before them
  int document;        // of this lane
  int blocks;          // of its queries
  int64_t upto;        // inclusive prefix over the lanes, times heads
  int lane;
  MLA_DEV void load(const PrefillParams& p) {
    const int b = base + lane;
    int keys = -1;
    blocks = 0;
    if (b < p.batch) {
      const Span s = span_of(p, b);
      blocks = (s.nq + kBlock - 1) / kBlock;
      keys = s.nk;
    }
    // lane r takes the document of rank r
    int rank = 0, from = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int k = __shfl_sync(0xffffffffu, keys, i);
      rank += k > keys || (k == keys && i < lane);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (__shfl_sync(0xffffffffu, rank, i) == lane) from = i;
    blocks = __shfl_sync(0xffffffffu, blocks, from);
    document = b - lane + from;
    int incl = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    upto = (int64_t)incl * p.heads;
  }
  MLA_DEV void start() {
    lane = threadIdx.x & 31;
    base = -32;
    before = upto = 0;
  }
  // the unit of block `id` of the grid; false if there is none (behind the last unit, or a piece that it does not have)
  MLA_DEV bool find(const PrefillParams& p, int64_t id, U& u) {
    const int64_t block = id / p.splits;
    const int piece = (int)(id - block * p.splits);
    if (block < before) start();
    int64_t all = __shfl_sync(0xffffffffu, upto, 31);
    while (block >= before + all) {
      if (base + 32 >= p.batch) return false;
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
    const Span s = span_of(p, __shfl_sync(0xffffffffu, document, which));
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

// Documents that are skipped are recorded by the block `id` of the `ids` in the grid, whether it starts or is taken over:
// groups of 32 id, id + ids, ... The search for units is no place for it: it ends with the last unit, and documents
// behind may have none. Called when the unit is on its way to its readers.
MLA_DEV void record_bad(const PrefillParams& p, int64_t id, int64_t ids) {
  if (!p.status) return;
  for (int64_t b = 32 * id + (threadIdx.x & 31); b < p.batch; b += 32 * ids)
    if (span_of(p, (int)b).bad) atomicOr(p.status, STATUS_INDEX);
  __syncwarp();
}

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
template <bool kCluster>
MLA_DEV bool wait_inline(uint32_t bar, uint32_t parity, const Guard& g) {
  auto done = [&]() { return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (done()) return true;
  const uint64_t t0 = cycles();
  while (!*g.abort) {
    if (done()) return true;
    if (cycles() - t0 > g.limit) {
      *g.abort = 1u;
      atomicOr(g.status, STATUS_TIMEOUT);
    }
  }
  return false;
}
// A barrier tells one phase from the next by parity alone. A thread that leaves some of a ring's rounds to others may be
// ahead of its barriers by a phase or more and would take an old phase for the one it wants: so it first waits until the
// copies have been asked for (`*issued` counts them), when the place's round before is over.
MLA_DEV void set_issued(uint32_t count, uint32_t n) { asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(count), "r"(n) : "memory"); }
MLA_DEV bool wait_issued(uint32_t count, uint32_t index, const Guard& g) {
  const uint64_t t0 = cycles();
  while (true) {
    uint32_t n;
    asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(n) : "r"(count) : "memory");
    if (n > index) return true;
    if (*g.abort) return false;
    if (cycles() - t0 > g.limit) {
      *g.abort = 1u;
      atomicOr(g.status, STATUS_TIMEOUT);
    }
  }
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

// |c m| from which a row subtracts its reference first: up to there the rounding of c m changes a row's weights by 2^-13 of
// themselves, no more than the scores' own rounding to fp32 does. The branch costs calls all of whose rows are such 38 to 43 %
// (2048 queries behind 32768 keys 3.92 ms, 4 x 4096 causal 2.50) and others nothing: it is the one that moves references.
constexpr float kFar = 0x1p12f;

// Weights of fp16 are formed 2^7 larger: with the reference's slack of 2^8 they reach 2^15, and what fp16 loses, weights below
// 2^-25 of its units, begins at 2^-32 of the reference's. At a scale of 1 the many small weights of a long row would be
// missing from O but not from l. The factor cancels in O / l; l carries it until its logarithm is taken.
template <bool kFp16>
constexpr float kRaise = kFp16 ? 7.f : 0.f;

// A thread's row in the softmax of one query tile.
struct Row {
  float m, l;                  // reference (raw score) and sum of the weights
};

// S of one key tile -> P over it, for the thread's row (its TMEM lane): keys from `left` on are masked where `masked`.
// hand_over(h) gives keys [64 h, 64 h + 64) of P to the products. `first`: the unit's first tile, whose accumulator
// holds nothing yet.
template <bool kFp16, class F>
MLA_DEV void softmax_tile(Row& row, uint32_t t_s, uint32_t t_o, float scale_log2, bool masked, int left, bool first, F hand_over) {
  uint32_t s[128];
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32u * c, s + 32 * c);
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < 4; ++c) pin_regs32(s + 32 * c);
  if (masked) {
#pragma unroll
    for (int k = 0; k < 128; ++k)
      if (k >= left) s[k] = 0xFF800000u;  // -inf
  }
  uint64_t sum[2];
  const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
  constexpr float raise = kRaise<kFp16>;
  auto reference = [&]() { return row.m == -INFINITY ? raise : fmaf(-row.m, scale_log2, raise); };
  float ref = reference();
  // 2^(s - m) of keys [32 c, 32 c + 32), packed
  auto weights = [&](int c, uint32_t* q) {
    const uint64_t ref2 = f2_pack(ref, ref);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 x = f2_unpack(f2_fma(f2_pack(__uint_as_float(s[32 * c + 2 * k]), __uint_as_float(s[32 * c + 2 * k + 1])), scale2, ref2));
      const float a = exp2_approx(x.x), b = exp2_approx(x.y);
      sum[k & 1] = f2_add(sum[k & 1], f2_pack(a, b));
      q[k] = pack_p<kFp16>(a, b);
    }
  };
  // The first weights are formed with the reference as it stands, beside the search for the row's maximum; only where
  // that passes the reference by too much (in a document's first tiles, hardly ever later), or the row's reference is far
  // off, are they formed again.
  uint32_t q[16];
  sum[0] = sum[1] = 0;
  weights(0, q);
  const float top = fmaxf(tree_max64([&](int k) { return __uint_as_float(s[k]); }),
                          tree_max64([&](int k) { return __uint_as_float(s[64 + k]); }));
  const bool move = top - row.m > 8.f / scale_log2;   // from -inf with the first key that it sees
  if (__any_sync(0xffffffffu, move || fabsf(ref) > kFar)) {
    if (__any_sync(0xffffffffu, move)) {
      const float next = move ? top : row.m;
      // rows that have seen nothing keep l = 0 and O = 0
      const float f = move ? exp2_approx((row.m - next) * scale_log2) : 1.f;
      row.m = next;
      row.l *= f;
      if (!first) {
        // S of this tile is complete, and with it every product issued before: O holds still until this tile's P is
        // handed over
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
      ref = reference();
    }
    const bool far = fabsf(ref) > kFar;
    if (__any_sync(0xffffffffu, far)) {
      const float minus = far ? -row.m : 0.f;
      const uint64_t minus2 = f2_pack(minus, minus);
#pragma unroll
      for (int k = 0; k < 128; k += 2) {
        const float2 x = f2_unpack(f2_add(f2_pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), minus2));
        s[k] = __float_as_uint(x.x);
        s[k + 1] = __float_as_uint(x.y);
      }
      if (far) ref = raise;
    }
    sum[0] = sum[1] = 0;
    weights(0, q);
  }
  tmem_st16(t_s, q);
  weights(1, q);
  tmem_st16(t_s + 16u, q);
  tmem_wait_st();
  hand_over(0);
  weights(2, q);
  tmem_st16(t_s + 32u, q);
  weights(3, q);
  tmem_st16(t_s + 48u, q);
  tmem_wait_st();
  hand_over(1);
  const float2 x = f2_unpack(f2_add(sum[0], sum[1]));
  row.l += x.x + x.y;
}

// What takes the place of 1 / l and of ln l where l is 0: a query that sees no key gets zeros and -inf, one whose scores all
// are -inf (dots beyond fp32's range) NaN, as 0 / 0.
MLA_DEV float inverse(float l, bool sees) { return l == 0.f ? (sees ? NAN : 0.f) : 1.f / l; }
template <bool kFp16>
MLA_DEV float lse_of(const PrefillParams& p, float m, float l, bool sees) {
  return l == 0.f ? (sees ? NAN : -INFINITY) : m * p.scale + logf(kFp16 ? l * 0x1p-7f : l);
}

// where the sum of a piece's weights waits for the join
MLA_DEV float* sum_at(const PrefillParams& p, int64_t row, int head, int piece) {
  return reinterpret_cast<float*>(static_cast<uint16_t*>(p.out) + row * p.out_token + head * p.out_head) + piece;
}

// 16 words of a row to 16-B aligned memory, in stores of 32 bytes where that is aligned for them: the stores of a warp's 32
// rows touch 32 lines each, whatever their width
MLA_DEV void store_words16(void* dst, const uint32_t* w, bool wide) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (wide) {
      st_global_v8(static_cast<uint32_t*>(dst) + 8 * k, w + 8 * k);
    } else {
      static_cast<uint4*>(dst)[2 * k] = make_uint4(w[8 * k], w[8 * k + 1], w[8 * k + 2], w[8 * k + 3]);
      static_cast<uint4*>(dst)[2 * k + 1] = make_uint4(w[8 * k + 4], w[8 * k + 5], w[8 * k + 6], w[8 * k + 7]);
    }
  }
}

// 32 dims of a row: of the output, or, without one, of a piece's share
template <bool kFp16>
MLA_DEV void store_share(uint16_t* out, float* part, const float* v, int wide) {
  uint32_t w[32];
  if (out) {
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = pack_p<kFp16>(v[2 * k], v[2 * k + 1]);
    store_words16(out, w, wide & 1);
  } else {
#pragma unroll
    for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(v[k]);
    store_words16(part, w, wide & 2);
    store_words16(part + 16, w + 16, wide & 2);
  }
}

// 32 rows of 64 dims of the output from shared memory (128-byte swizzled), rows and dims all inside the tensor
MLA_DEV void store_rows64(const CUtensorMap* m, uint32_t src, int x, int head, int row) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)), "r"(src), "r"(x), "r"(head), "r"(row)
               : "memory");
}
MLA_DEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
MLA_DEV void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
MLA_DEV void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
constexpr uint32_t kStage = 32 * 128;   // a warp's 32 rows x 64 dims on their way out

// The warp's 32 results: O / l and lse, or a piece's O, m and l. `some`: the accumulators hold something; read() is
// called when they have been read. Rows of a warp that all belong to the unit leave through shared memory (`stage`) and
// the copy engine: the plain stores of 32 rows touch 32 lines each and kept the SM's load/store path, and with it every
// wait on a barrier, busy for some 3400 cycles a unit.
template <bool kFp16, class U, class F>
MLA_DEV void store_rows(const PrefillParams& p, const CUtensorMap* tm_out, uint32_t stage, const U& u, const Row& row, uint32_t t_o,
                        bool some, int first, F read) {
  const int lane = threadIdx.x & 31;
  const bool whole = u.pieces == 1, live = first + lane < u.rows;
  const bool sees = live && u.visible(first + lane, p.causal) > 0;
  const float inv = whole ? inverse(row.l, sees) : 1.f;
  const int64_t at = (int64_t)u.row + first + lane;
  if (live && whole) {
    p.lse[at * p.heads + u.head] = lse_of<kFp16>(p, row.m, row.l, sees);
  } else if (live) {
    p.ref_part[((int64_t)u.piece * p.tq + at) * p.heads + u.head] = row.m;
    *sum_at(p, at, u.head, u.piece) = row.l;
  }
  // 32 dims of the row, normalised if it is whole
  auto share = [&](int c, float* v) {
    uint32_t o[32];
    if (some) {
      tmem_ld32(t_o + 32u * c, o);
      tmem_wait_ld();
      pin_regs32(o);
      if (c == 3) read();
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = 0u;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]) * inv;
  };
  // loops, not straight code: what runs once a unit is not in the instruction cache
  if (whole && first + 32 <= u.rows) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t y[32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[32];
        share(2 * h + c, v);
#pragma unroll
        for (int k = 0; k < 16; ++k) y[16 * c + k] = pack_p<kFp16>(v[2 * k], v[2 * k + 1]);
      }
      if (lane == 0) bulk_wait_read();   // the stage's last rows are out of it
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        st_shared_v4(stage + 128u * lane + 16u * (k ^ (lane & 7)), y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        store_rows64(tm_out, stage, 64 * h, u.head, (int)at);
        bulk_commit();
      }
    }
    return;
  }
  uint16_t* dst = static_cast<uint16_t*>(p.out) + at * p.out_token + u.head * p.out_head;
  float* part = p.o_part + (((int64_t)u.piece * p.tq + at) * p.heads + u.head) * kV;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float v[32];
    share(c, v);
    if (live) store_share<kFp16>(whole ? dst + 32 * c : nullptr, part + 32 * c, v, p.wide);
  }
}

// Joins the pieces of cut units: with f_i = 2^(c (m_i - m)), m the largest m_i, out = sum_i f_i O_i / sum_i f_i l_i and
// lse = scale m + ln sum_i f_i l_i. A warp to a (row, head), four dims a lane; rows whose unit was not cut are left as they
// are.
constexpr int kCombineThreads = 256;

template <bool kFp16, int kBlock>
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
  // lane k: piece k
  float m = -INFINITY, l = 0.f;
  if (lane < pieces) {
    m = p.ref_part[((int64_t)lane * p.tq + row) * p.heads + head];
    l = *sum_at(p, row, head, lane);
  }
  float top = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float mine = exp2_approx((m - (top == -INFINITY ? 0.f : top)) * p.scale_log2);
  float total = mine * l;   // all sums are read before any lane writes the row
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < pieces; ++k) {
    const float f = __shfl_sync(0xffffffffu, mine, k);
    const float4 v = reinterpret_cast<const float4*>(p.o_part + (((int64_t)k * p.tq + row) * p.heads + head) * kV)[lane];
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  }
  const bool sees = visible(p, s, i) > 0;
  const float inv = inverse(total, sees);
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * p.out_token + head * p.out_head);
  dst[lane] = make_uint2(pack_p<kFp16>(acc.x * inv, acc.y * inv), pack_p<kFp16>(acc.z * inv, acc.w * inv));
  if (lane == 0) p.lse[item] = lse_of<kFp16>(p, top, total, sees);
}

}  // namespace prefill
}  // namespace mla
