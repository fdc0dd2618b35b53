// rows.cuh -- writers of new tokens: rotary positions, the paged latent cache,
// the paged index cache and the index queries.
//
// The rotation R_p of 64 dims at position p turns pair i (0..31) by the angle
// whose cosine and sine stand in the caller's table row p ([cos 0..31 | sin
// 0..31], fp32):
//     y0 = x0 cos - x1 sin,   y1 = x0 sin + x1 cos
// Pair i is dims (2i, 2i + 1), or (i, i + 32) with MLA_ROPE_HALVES. Products
// and sums are each rounded to fp32 (no fused multiply-add), so that a row's
// quantisation does not depend on how a compiler contracts them; the result is
// rounded once, to the row's own type.
//
// All of these are bound by their bytes (under 1 FLOP per byte) and, for a few
// tokens, by the latency of slot/position -> table row -> store. So each kernel
// has every load that does not depend on another one in flight first; only the
// append of 528- and 288-byte rows loads its RoPE dims behind the slot's test, in
// the four lanes that turn them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "codes.cuh"

namespace mla {
namespace rows {

constexpr int kRope = 64;
constexpr int kPairs = kRope / 2;
constexpr int kIndexDim = 128;
constexpr int kIndexPageFp8 = kTile * (kIndexDim + 4);  // 64 rows of codes, then their 64 fp32 scales

struct Positions {
  const int32_t* positions;  // [tokens]
  const float* table;        // [max_positions, 64]
  int64_t max_positions;
  int halves;                // pairs (i, i + 32) instead of (2i, 2i + 1)
  uint32_t* status;          // or null
};

struct AppendParams {
  const void* c_kv;          // [n, 512 or 448], 16-bit
  const void* k_rope;        // [n, 64]
  int64_t c_stride, r_stride;  // elements
  const int32_t* slots;      // [n], negative: skip
  Positions pos;
  int64_t n;
  uint8_t* kv;
  int64_t num_rows;
};

struct RotateParams {
  const uint16_t* x;
  uint16_t* out;
  int64_t x_token, x_head, out_token, out_head;  // strides in elements
  Positions pos;
  int64_t tokens;
  int heads;
  uint32_t heads_per_slot;   // ceil(heads / kU): head slots of a token
};

struct IndexRowParams {
  const uint16_t* x;         // [tokens, heads, 128]
  int64_t x_token, x_head;   // strides in elements
  const int32_t* cache_slots;  // keys: [tokens]
  const float* weights;      // queries: [tokens, heads]
  Positions pos;
  int64_t tokens;
  int heads;
  int slots_per_token;       // queries: lane groups of a token, ceil(heads / steps)
  int steps;                 // queries: heads a lane group takes
  uint8_t* out;              // keys: the index cache; queries: [tokens, heads, 128] codes
  float* w_out;              // queries: [tokens, heads]
  int64_t num_rows;          // keys: rows of the index cache
};

MLA_DEV void flag(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

template <bool kFp16>
MLA_DEV float to_f32(uint16_t v) {
  return kFp16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}
template <bool kFp16>
MLA_DEV float2 unpack2(uint32_t v) {
  if (kFp16) return unpack_f16x2(v);
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <bool kFp16>
MLA_DEV uint32_t pack2(float lo, float hi) {
  return kFp16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
template <bool kFp16, int kN>
MLA_DEV void unpack(const uint4* raw, float* x) {  // kN values (a multiple of 8)
#pragma unroll
  for (int k = 0; k < kN / 8; ++k) {
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = unpack2<kFp16>(w[j]);
      x[8 * k + 2 * j] = v.x;
      x[8 * k + 2 * j + 1] = v.y;
    }
  }
}
template <bool kFp16>
MLA_DEV uint4 pack8(const float* x) {
  return make_uint4(pack2<kFp16>(x[0], x[1]), pack2<kFp16>(x[2], x[3]), pack2<kFp16>(x[4], x[5]),
                    pack2<kFp16>(x[6], x[7]));
}

// (a, b) turned by the angle of (c, s)
MLA_DEV float turn_lo(float a, float b, float c, float s) { return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)); }
MLA_DEV float turn_hi(float a, float b, float c, float s) { return __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c)); }

// kN consecutive floats (a multiple of 4, 16-B aligned) of a table row
template <int kN>
MLA_DEV void load_row(const float* src, float* v) {
#pragma unroll
  for (int k = 0; k < kN / 4; ++k) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(src) + k);
    v[4 * k] = f.x;
    v[4 * k + 1] = f.y;
    v[4 * k + 2] = f.z;
    v[4 * k + 3] = f.w;
  }
}

// ---------------------------------------------------------------------------
// The paged latent cache: one warp per token, 32 contiguous bytes of latent
// dims per lane (eight lanes to a block of 128, so that its scale is formed
// once a lane and agreed on in three shuffles).
// Measured (GB300): 64 tokens 1.4 us; 32768 tokens, 16-bit rows 14.3 us (0.87 of
// the copy bandwidth), 656-byte rows 14.4 us (0.69; 16.9 at the 52 registers a
// thread takes unlimited, which leave 40 warps an SM instead of 48), 528-byte
// rows 15.0 us (0.58): these wait for their loads between two stretches of
// arithmetic, at half of the issue slots. 288-byte rows 24.5 us (0.31) are bound
// by the ALU pipe (82 %): seven two-sided comparisons a value choose its code.
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 8;

template <bool kFp16, int kFormat>  // kFormat: mla_kv_format
__global__ void __launch_bounds__(32 * kAppendWarps, kFormat == 0 ? 8 : 6) mla_append_kv_kernel(const AppendParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= p.n) return;
  const uint16_t* c = static_cast<const uint16_t*>(p.c_kv) + t * p.c_stride;
  const uint16_t* r = static_cast<const uint16_t*>(p.k_rope) + t * p.r_stride;
  // all that does not depend on the slot is on its way before the slot is
  // looked at: one round trip to memory, then the table row
  const int32_t slot = __ldg(p.slots + t), at = __ldg(p.pos.positions + t);
  uint4 raw[2];  // 16-bit rows: two strips of 512 bytes, else values [16 lane, 16 lane + 16)
  if (kFormat == 0) {
    raw[0] = __ldg(reinterpret_cast<const uint4*>(c) + lane);
    raw[1] = __ldg(reinterpret_cast<const uint4*>(c) + 32 + lane);
  } else if (kFormat == 1 || lane < 28) {
    raw[0] = __ldg(reinterpret_cast<const uint4*>(c) + 2 * lane);
    raw[1] = __ldg(reinterpret_cast<const uint4*>(c) + 2 * lane + 1);
  }
  float a = 0.f, b = 0.f;  // pair `lane`
  if (kFormat <= 1) {
    if (p.pos.halves) {
      a = to_f32<kFp16>(__ldg(r + lane));
      b = to_f32<kFp16>(__ldg(r + lane + kPairs));
    } else {
      const float2 v = unpack2<kFp16>(__ldg(reinterpret_cast<const uint32_t*>(r) + lane));
      a = v.x;
      b = v.y;
    }
  }
  if (slot < 0) return;  // padding
  if (slot >= p.num_rows || at < 0 || at >= p.pos.max_positions) {
    if (lane == 0) flag(p.pos.status, STATUS_INDEX);
    return;
  }
  const float* row = p.pos.table + (int64_t)at * kRope;

  if (kFormat <= 1) {
    // lane l turns pair l
    constexpr int kRow = kFormat == 0 ? kDK * 2 : kRowBytesFp8;
    constexpr int kLatentBytes = kFormat == 0 ? 1024 : 528;
    uint8_t* dst = p.kv + (int64_t)slot * kRow;
    const float cs = __ldg(row + lane), sn = __ldg(row + kPairs + lane);
    if (kFormat == 0) {
      reinterpret_cast<uint4*>(dst)[lane] = raw[0];
      reinterpret_cast<uint4*>(dst)[32 + lane] = raw[1];
    } else {
      // lane l owns values [16l, 16l + 16): eight lanes to a block of 128
      float x[16];
      unpack<false, 16>(raw, x);
      float amax = amax16(x);
#pragma unroll
      for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = e4m3_scale(amax);
      uint32_t w[4];
      e4m3_codes16(x, scale, w);
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
      if ((lane & 7) == 0) reinterpret_cast<float*>(dst)[128 + (lane >> 3)] = scale;
    }
    const uint32_t y = pack2<kFp16>(turn_lo(a, b, cs, sn), turn_hi(a, b, cs, sn));
    uint8_t* rd = dst + kLatentBytes;
    if (p.pos.halves) {
      reinterpret_cast<uint16_t*>(rd)[lane] = (uint16_t)y;
      reinterpret_cast<uint16_t*>(rd)[lane + kPairs] = (uint16_t)(y >> 16);
    } else {
      reinterpret_cast<uint32_t*>(rd)[lane] = y;
    }
  } else {
    // rows of 512 values: lane l owns [16l, 16l + 16); 448 latent dims in lanes
    // 0..27, RoPE dims [16j, 16j + 16) in lane 28 + j
    float x[16];
    if (lane < 28) {
      unpack<false, 16>(raw, x);
    } else {
      const int j = lane - 28;
      if (p.pos.halves) {
        // the lane's 16 dims are one side of pairs [16 (j & 1), +16)
        const int i = j & 1;
        const uint4* r4 = reinterpret_cast<const uint4*>(r);
        const uint4 ra[2] = {r4[2 * i], r4[2 * i + 1]}, rb[2] = {r4[4 + 2 * i], r4[5 + 2 * i]};
        float a[16], b[16], cs[16], sn[16];
        unpack<false, 16>(ra, a);
        unpack<false, 16>(rb, b);
        load_row<16>(row + 16 * i, cs);
        load_row<16>(row + kPairs + 16 * i, sn);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = j < 2 ? turn_lo(a[k], b[k], cs[k], sn[k]) : turn_hi(a[k], b[k], cs[k], sn[k]);
      } else {
        const uint4 raw[2] = {reinterpret_cast<const uint4*>(r)[2 * j], reinterpret_cast<const uint4*>(r)[2 * j + 1]};
        float a[16], cs[8], sn[8];
        unpack<false, 16>(raw, a);
        load_row<8>(row + 8 * j, cs);
        load_row<8>(row + kPairs + 8 * j, sn);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[2 * k] = turn_lo(a[2 * k], a[2 * k + 1], cs[k], sn[k]);
          x[2 * k + 1] = turn_hi(a[2 * k], a[2 * k + 1], cs[k], sn[k]);
        }
      }
    }
    __syncwarp();
    if (kFormat == 2) {
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // two lanes per block of 32
      const int k = ue8m0_exponent(amax);
      const float inv = exp2_neg(k);
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = e4m3x4_rn_sat(x[4 * q] * inv, x[4 * q + 1] * inv, x[4 * q + 2] * inv, x[4 * q + 3] * inv);
      uint8_t* dst = p.kv + (int64_t)slot * kRowBytesFp8_528;
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
      const uint32_t ue = (uint32_t)(k + 127);
      uint32_t word = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) word |= __shfl_sync(0xffffffffu, ue, (8 * lane + 2 * b) & 31) << (8 * b);
      if (lane < 4) reinterpret_cast<uint32_t*>(dst + 512)[lane] = word;
    } else {
      uint32_t lo, hi;
      const uint32_t code = fp4_block(x, lo, hi);
      uint8_t* dst = p.kv + (int64_t)slot * kRowBytesFp4_288;
      reinterpret_cast<uint2*>(dst)[lane] = make_uint2(lo, hi);
      uint32_t word = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) word |= __shfl_sync(0xffffffffu, code, (4 * lane + b) & 31) << (8 * b);
      if (lane < 8) reinterpret_cast<uint32_t*>(dst + 256)[lane] = word;
    }
  }
}

// ---------------------------------------------------------------------------
// Rotation of query rows: a thread turns 8 pairs (32 bytes) of kU heads of one
// token, four threads per row of 64 dims. The table row stays in registers for
// the kU heads.
// Measured (GB300): 64 tokens x 128 heads 1.8 us; 4095 x 128 22.3 to 22.9 us (0.89
// to 0.87 of the copy bandwidth).
// ---------------------------------------------------------------------------
constexpr int kRotateThreads = 256;

template <bool kFp16, int kU>
__global__ void __launch_bounds__(kRotateThreads) mla_rotate_kernel(const RotateParams p) {
  pdl_wait();
  const int64_t item = (int64_t)blockIdx.x * kRotateThreads + threadIdx.x;
  const int j = (int)(item & 3);
  const uint32_t group = (uint32_t)(item >> 2);  // below 2^31 (checked on the host)
  const uint32_t t = group / p.heads_per_slot, h0 = group - t * p.heads_per_slot;
  if (t >= p.tokens) return;
  const int32_t at = __ldg(p.pos.positions + t);
  // pairs [8j, 8j + 8): dims [16j, 16j + 16), or [8j, 8j + 8) and 32 behind
  const int d0 = p.pos.halves ? 8 * j : 16 * j, d1 = p.pos.halves ? 8 * j + 32 : 16 * j + 8;
  const uint16_t* src = p.x + t * p.x_token;
  uint16_t* dst = p.out + t * p.out_token;
  uint4 raw[kU][2];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t h = h0 + u * p.heads_per_slot;
    if (h < (uint32_t)p.heads) {
      raw[u][0] = *reinterpret_cast<const uint4*>(src + h * p.x_head + d0);
      raw[u][1] = *reinterpret_cast<const uint4*>(src + h * p.x_head + d1);
    }
  }
  if (at < 0) return;  // padding
  if (at >= p.pos.max_positions) {
    if (j == 0 && h0 == 0) flag(p.pos.status, STATUS_INDEX);
    return;
  }
  const float* row = p.pos.table + (int64_t)at * kRope + 8 * j;
  float cs[8], sn[8];
  load_row<8>(row, cs);
  load_row<8>(row + kPairs, sn);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t h = h0 + u * p.heads_per_slot;
    if (h >= (uint32_t)p.heads) break;
    float x[16], y[16];
    unpack<kFp16, 16>(raw[u], x);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (p.pos.halves) {
        y[k] = turn_lo(x[k], x[8 + k], cs[k], sn[k]);
        y[8 + k] = turn_hi(x[k], x[8 + k], cs[k], sn[k]);
      } else {
        y[2 * k] = turn_lo(x[2 * k], x[2 * k + 1], cs[k], sn[k]);
        y[2 * k + 1] = turn_hi(x[2 * k], x[2 * k + 1], cs[k], sn[k]);
      }
    }
    *reinterpret_cast<uint4*>(dst + h * p.out_head + d0) = pack8<kFp16>(y);
    *reinterpret_cast<uint4*>(dst + h * p.out_head + d1) = pack8<kFp16>(y + 8);
  }
}

// ---------------------------------------------------------------------------
// Index rows of 128 values, dims [0, 64) rotated: keys into the paged index
// cache, queries as e4m3 with their scale folded into the head's weight.
// Eight lanes per row: lane l holds dims [8l, 8l + 8) of the rotated half and
// [64 + 8l, 64 + 8l + 8) of the other, so that every lane turns four pairs. A
// lane group takes `steps` query heads of one token, which share the position
// and the table row, and loads a head ahead.
// Measured (GB300): 4096 x 64 e4m3 queries 20.6 us (0.74 of the copy bandwidth;
// 27 with two heads a group, their weight loaded where it is used and the scale
// divided; 42 with 16 lanes a row and a division per value as well): some 200
// instructions for 16 values of a lane. 32768 keys 4.2 us (0.75).
// ---------------------------------------------------------------------------
constexpr int kIndexThreads = 256;
constexpr int kIndexLanes = 8;
constexpr int kIndexGroups = kIndexThreads / kIndexLanes;

template <bool kFp16, bool kFp8, bool kKeys>
__global__ void __launch_bounds__(kIndexThreads, 4) mla_index_rows_kernel(const IndexRowParams p) {
  pdl_wait();
  const int l = threadIdx.x & (kIndexLanes - 1);
  const uint32_t group = blockIdx.x * kIndexGroups + threadIdx.x / kIndexLanes;
  const uint32_t slots = kKeys ? 1u : (uint32_t)p.slots_per_token;
  const uint32_t t = kKeys ? group : group / slots, h0 = kKeys ? 0u : group - t * slots;
  const int steps = kKeys ? 1 : p.steps;
  // every lane takes part in the shuffles below; rows past the end or to be
  // skipped work on zeros and store nothing
  const bool inside = t < p.tokens;
  const int32_t slot = kKeys && inside ? __ldg(p.cache_slots + t) : 0, at = inside ? __ldg(p.pos.positions + t) : -1;
  uint4 raw[2];
  float weight;
  auto fetch = [&](uint32_t h) {
    raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
    weight = 0.f;
    if (inside && h < (uint32_t)p.heads) {
      const uint4* src = reinterpret_cast<const uint4*>(p.x + t * p.x_token + h * p.x_head);
      raw[0] = __ldg(src + l);
      raw[1] = __ldg(src + 8 + l);
      if (!kKeys && l == 0) weight = p.weights[(int64_t)t * p.heads + h];
    }
  };
  fetch(h0);
  // padding: a negative slot, or for queries a negative position
  bool live = inside && (kKeys ? slot >= 0 : at >= 0);
  if (live && (at < 0 || at >= p.pos.max_positions || (kKeys && slot >= p.num_rows))) {
    if (l == 0 && h0 == 0) flag(p.pos.status, STATUS_INDEX);
    live = false;
  }
  const float* row = p.pos.table + (int64_t)at * kRope;  // read where live
  // The lane's cosines and sines: of its four pairs, or, with halves, of its
  // eight dims, each half of a pair (lanes 0..3 the first halves, 4..7 the
  // second, whose partner's sine enters with the other sign).
  float cs[8] = {}, sn[8] = {};
  if (live) {
    if (p.pos.halves) {
      load_row<8>(row + 8 * (l & 3), cs);
      load_row<8>(row + kPairs + 8 * (l & 3), sn);
#pragma unroll
      for (int k = 0; k < 8; ++k) sn[k] = l < 4 ? -sn[k] : sn[k];
    } else {
      load_row<4>(row + 4 * l, cs);
      load_row<4>(row + kPairs + 4 * l, sn);
    }
  }
#pragma unroll 1
  for (int u = 0; u < steps; ++u) {
    const uint32_t h = h0 + u * slots;
    const bool store = live && h < (uint32_t)p.heads;
    float x[16];
    unpack<kFp16, 16>(raw, x);
    const uint4 second = raw[1];
    const float w_head = weight;
    if (u + 1 < steps) fetch(h + slots);
    if (p.pos.halves) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = turn_hi(__shfl_xor_sync(0xffffffffu, x[k], 4), x[k], cs[k], sn[k]);  // other * sin + own * cos
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = x[2 * k], b = x[2 * k + 1];
        x[2 * k] = turn_lo(a, b, cs[k], sn[k]);
        x[2 * k + 1] = turn_hi(a, b, cs[k], sn[k]);
      }
    }
    if (!kFp8) {
      if (store) {
        uint4* dst = reinterpret_cast<uint4*>(p.out) + (int64_t)slot * 16;
        dst[l] = pack8<kFp16>(x);
        dst[8 + l] = second;
      }
      continue;
    }
    float amax = amax16(x);
#pragma unroll
    for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!store) continue;
    const float scale = e4m3_scale(amax);
    uint32_t w[4];
    e4m3_codes16(x, scale, w);
    uint2* dst;
    if (kKeys) {
      uint8_t* page = p.out + (int64_t)(slot / kTile) * kIndexPageFp8;
      const int in = slot % kTile;
      dst = reinterpret_cast<uint2*>(page) + in * 16;
      if (l == 0) reinterpret_cast<float*>(page + kTile * kIndexDim)[in] = scale;
    } else {
      const int64_t at = (int64_t)t * p.heads + h;
      dst = reinterpret_cast<uint2*>(p.out) + at * 16;
      if (l == 0) p.w_out[at] = __fmul_rn(w_head, scale);
    }
    dst[l] = make_uint2(w[0], w[1]);
    dst[8 + l] = make_uint2(w[2], w[3]);
  }
}

}  // namespace rows
}  // namespace mla
