// norms.cuh -- RMS norms in one pass with the rotary positions: queries and
// keys for each head, and the latent on its way into the paged cache.
//
//     y = x * (1 / sqrt(mean(x^2) + eps)) * w
//
// The mean is over a row's d dims (the latent dims of a cache row), summed in
// fp32. x is brought to the row's own size first, so that a product leaves
// fp32's range only where y does; x w first would be exact for most values, one
// rounding less, but overflows or loses bits for bf16 rows and weights near the
// ends of theirs. y stays in fp32 through the rotation (whose products and sums
// are each rounded to fp32, as in rows.cuh) or the quantisation and is rounded
// once, to the type that it is stored in. So a row is read once and written
// once, and both kernels are bound by those bytes (some 2 FLOP a byte) or, for a
// few tokens, by the latency of position -> table row -> store.
#pragma once
#include "rows.cuh"

namespace mla {
namespace norms {

using rows::kRope;
using rows::kPairs;

constexpr int kMaxDim = 576;

struct NormRotateParams {
  const uint16_t* x;
  const uint16_t* weight;      // [dim] or null
  uint16_t* out;               // dim values a row, or dim - 64 where rope_out is given
  uint16_t* rope_out;          // 64 values a row, or null
  int64_t x_token, x_head, out_token, out_head, rope_token, rope_head;  // strides in elements
  rows::Positions pos;
  int64_t tokens;
  int heads, dim, at;          // rotated dims: [at, at + 64)
  float eps;
  uint32_t groups_per_token;   // ceil(heads / kU)
};

template <int kLanes>
MLA_DEV float group_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A row belongs to kLanes lanes: lane l of the first eight holds dims [8l, 8l +
// 8) of the rotated 64, every lane the chunks l, l + kLanes, ... (kChunks of
// them) of the other dims, eight to a chunk. A lane group takes kU heads of one
// token, which share the table row and the weights, all of their loads in flight
// together.
//
// Measured (GB300): 4095 tokens x 128 heads of 192 66.6 us (0.89 of the copy
// bandwidth; 68.0 at the 80 registers a thread takes unlimited, which leave 24
// warps an SM instead of 32, 104 and 119 with spills at 48 and 40; 74.1 with one
// head a lane group). 64 x 128 2.1 us, 32768 rows of 128 5.4: the latency of
// position -> table row -> store.
constexpr int kNormThreads = 256;

template <bool kFp16, int kLanes, int kChunks, int kU>
__global__ void __launch_bounds__(kNormThreads, 4) mla_norm_rotate_kernel(const NormRotateParams p) {
  pdl_wait();
  const int l = threadIdx.x & (kLanes - 1);
  const uint32_t group = (uint32_t)(blockIdx.x * (kNormThreads / kLanes) + threadIdx.x / kLanes);
  const uint32_t t = group / p.groups_per_token, h0 = group - t * p.groups_per_token;
  // every lane takes part in the sums; rows past the end work on zeros and store nothing
  const bool inside = t < p.tokens;
  const int32_t pos = inside ? __ldg(p.pos.positions + t) : -1;
  const int rest = (p.dim - kRope) >> 3, at8 = p.at >> 3;   // chunks beside the rotated ones, and before them
  const bool turns = l < 8;
  uint4 raw[kU][kChunks + 1];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t h = h0 + u * p.groups_per_token;
    const bool on = inside && h < (uint32_t)p.heads;
    const uint4* src = reinterpret_cast<const uint4*>(p.x + t * p.x_token + h * p.x_head);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int c = l + kLanes * k;
      raw[u][k] = on && c < rest ? src[c < at8 ? c : c + 8] : make_uint4(0, 0, 0, 0);
    }
    raw[u][kChunks] = on && turns ? src[at8 + l] : make_uint4(0, 0, 0, 0);
  }
  bool live = inside && pos >= 0;    // padding otherwise
  if (live && pos >= p.pos.max_positions) {
    if (l == 0 && h0 == 0) rows::flag(p.pos.status, STATUS_INDEX);
    live = false;
  }
  uint4 weight[kChunks + 1];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const int c = l + kLanes * k;
    if (p.weight && c < rest) weight[k] = __ldg(reinterpret_cast<const uint4*>(p.weight) + (c < at8 ? c : c + 8));
  }
  if (p.weight && turns) weight[kChunks] = __ldg(reinterpret_cast<const uint4*>(p.weight) + at8 + l);
  // cosines and sines: of the lane's four pairs, or, with halves, of its eight dims, each one side of a pair (lanes 0
  // to 3 the first sides, whose partner's sine enters with the other sign)
  float cs[8] = {}, sn[8] = {};
  if (live && turns) {
    const float* row = p.pos.table + (int64_t)pos * kRope;
    if (p.pos.halves) {
      rows::load_row<8>(row + 8 * (l & 3), cs);
      rows::load_row<8>(row + kPairs + 8 * (l & 3), sn);
#pragma unroll
      for (int k = 0; k < 8; ++k) sn[k] = l < 4 ? -sn[k] : sn[k];
    } else {
      rows::load_row<4>(row + 4 * l, cs);
      rows::load_row<4>(row + kPairs + 4 * l, sn);
    }
  }
  const float inv_dim = 1.f / (float)p.dim;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t h = h0 + u * p.groups_per_token;
    const bool store = live && h < (uint32_t)p.heads;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k <= kChunks; ++k) {
      float x[8];
      rows::unpack<kFp16, 8>(&raw[u][k], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    }
    const float r = 1.f / sqrtf(group_sum<kLanes>(ss) * inv_dim + p.eps);
    auto normed = [&](int k, float* y) {
      rows::unpack<kFp16, 8>(&raw[u][k], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= r;
      if (p.weight) {
        float w[8];
        rows::unpack<kFp16, 8>(&weight[k], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= w[j];
      }
    };
    float y[8];
    normed(kChunks, y);
    if (p.pos.halves) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = rows::turn_hi(__shfl_xor_sync(0xffffffffu, y[j], 4), y[j], cs[j], sn[j]);  // other * sin + own * cos
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = y[2 * j], b = y[2 * j + 1];
        y[2 * j] = rows::turn_lo(a, b, cs[j], sn[j]);
        y[2 * j + 1] = rows::turn_hi(a, b, cs[j], sn[j]);
      }
    }
    if (!store) continue;
    uint4* dst = reinterpret_cast<uint4*>(p.out + t * p.out_token + h * p.out_head);
    if (turns) {
      if (p.rope_out) reinterpret_cast<uint4*>(p.rope_out + t * p.rope_token + h * p.rope_head)[l] = rows::pack8<kFp16>(y);
      else dst[at8 + l] = rows::pack8<kFp16>(y);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int c = l + kLanes * k;
      if (c >= rest) break;
      float v[8];
      normed(k, v);
      dst[p.rope_out || c < at8 ? c : c + 8] = rows::pack8<kFp16>(v);
    }
  }
}

// ---------------------------------------------------------------------------
// The latent normalised and appended to the paged cache: one warp per token, as
// mla_append_kv_kernel lays it out (16 latent values a lane), with the sum of
// squares agreed on in five shuffles before the row is formed. `rows`
// optionally takes the same row in 16 bits.
//
// Measured (GB300): 64 tokens, bf16 rows 1.5 us; 32768 tokens into 656-byte rows
// and `rows` 19.8 us (0.78 of the copy bandwidth): like mla_append_kv_kernel it
// waits for its loads in turn (slot and row, then the table row) between two
// stretches of arithmetic, at half of the issue slots.
// ---------------------------------------------------------------------------
struct NormAppendParams {
  rows::AppendParams a;
  const uint16_t* weight;      // [latent] or null
  float eps;
  uint16_t* rows;              // [n, latent + 64] or null
  int64_t rows_stride;
  int wide;                    // rows are 32-B aligned
};

template <bool kFp16, int kFormat>  // kFormat: mla_kv_format
__global__ void __launch_bounds__(32 * rows::kAppendWarps) mla_norm_append_kv_kernel(const NormAppendParams q) {
  using namespace rows;
  constexpr bool kNarrow = kFormat >= 2;                    // rows of 512 values, 448 of them latent
  constexpr int kLatent = kNarrow ? kDV41 - kRope : kDV;
  const AppendParams& p = q.a;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= p.n) return;
  const uint16_t* c = static_cast<const uint16_t*>(p.c_kv) + t * p.c_stride;
  const uint16_t* r = static_cast<const uint16_t*>(p.k_rope) + t * p.r_stride;
  const int32_t slot = __ldg(p.slots + t), at = __ldg(p.pos.positions + t);
  // 16-bit rows: two strips of 512 bytes, else values [16 lane, 16 lane + 16)
  const int c0 = kFormat == 0 ? lane : 2 * lane, c1 = kFormat == 0 ? 32 + lane : 2 * lane + 1;
  const bool latent = !kNarrow || lane < kLatent / 16;
  uint4 raw[2] = {}, wraw[2];
  if (latent) {
    raw[0] = __ldg(reinterpret_cast<const uint4*>(c) + c0);
    raw[1] = __ldg(reinterpret_cast<const uint4*>(c) + c1);
    if (q.weight) {
      wraw[0] = __ldg(reinterpret_cast<const uint4*>(q.weight) + c0);
      wraw[1] = __ldg(reinterpret_cast<const uint4*>(q.weight) + c1);
    }
  }
  float a, b;  // pair `lane` of the rotated dims
  if (p.pos.halves) {
    a = to_f32<kFp16>(__ldg(r + lane));
    b = to_f32<kFp16>(__ldg(r + lane + kPairs));
  } else {
    const float2 v = unpack2<kFp16>(__ldg(reinterpret_cast<const uint32_t*>(r) + lane));
    a = v.x;
    b = v.y;
  }
  if (slot < 0) return;  // padding
  if (slot >= p.num_rows || at < 0 || at >= p.pos.max_positions) {
    if (lane == 0) flag(p.pos.status, STATUS_INDEX);
    return;
  }
  const float* row = p.pos.table + (int64_t)at * kRope;
  const float cs = __ldg(row + lane), sn = __ldg(row + kPairs + lane);
  float x[16];
  unpack<kFp16, 16>(raw, x);
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) ss = fmaf(x[k], x[k], ss);
  const float inv = 1.f / sqrtf(group_sum<32>(ss) * (1.f / kLatent) + q.eps);
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] *= inv;
  if (q.weight && latent) {
    float w[16];
    unpack<kFp16, 16>(wraw, w);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= w[k];
  }
  const float lo = turn_lo(a, b, cs, sn), hi = turn_hi(a, b, cs, sn);
  // pair `lane` of the rotated dims at dst, 16 bits each
  auto store_rope = [&](uint16_t* dst) {
    const uint32_t y = pack2<kFp16>(lo, hi);
    if (p.pos.halves) {
      dst[lane] = (uint16_t)y;
      dst[lane + kPairs] = (uint16_t)(y >> 16);
    } else {
      reinterpret_cast<uint32_t*>(dst)[lane] = y;
    }
  };
  const uint4 y0 = pack8<kFp16>(x), y1 = pack8<kFp16>(x + 8);
  if (q.rows) {
    uint16_t* dst = q.rows + t * q.rows_stride;
    if (kFormat == 0) {
      reinterpret_cast<uint4*>(dst)[c0] = y0;
      reinterpret_cast<uint4*>(dst)[c1] = y1;
    } else if (latent) {
      store16<kFp16>(dst + 16 * lane, x, q.wide);
    }
    store_rope(dst + kLatent);
  }
  if (kFormat == 0) {
    uint8_t* dst = p.kv + (int64_t)slot * (kDK * 2);
    reinterpret_cast<uint4*>(dst)[c0] = y0;
    reinterpret_cast<uint4*>(dst)[c1] = y1;
    store_rope(reinterpret_cast<uint16_t*>(dst + 2 * kLatent));
  } else if (kFormat == 1) {
    uint8_t* dst = p.kv + (int64_t)slot * kRowBytesFp8;
    float amax = amax16(x);
#pragma unroll
    for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = e4m3_scale(amax);
    uint32_t w[4];
    e4m3_codes16(x, scale, w);
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    if ((lane & 7) == 0) reinterpret_cast<float*>(dst)[128 + (lane >> 3)] = scale;
    store_rope(reinterpret_cast<uint16_t*>(dst + 528));
  } else {
    // rows of 512 values, lane l owns [16l, 16l + 16): lanes 28 to 31 fetch the rotated dims from the lanes that
    // turned them; dims [16j, 16j + 16) are pairs [8j, 8j + 8), or one side of pairs [16 (j & 1), +16)
    const int j = lane - 28;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int from = p.pos.halves ? 16 * (j & 1) + k : 8 * (j & 3) + (k >> 1);
      const float vl = __shfl_sync(0xffffffffu, lo, from), vh = __shfl_sync(0xffffffffu, hi, from);
      const bool high = p.pos.halves ? j >= 2 : (k & 1);
      if (!latent) x[k] = high ? vh : vl;
    }
    if (kFormat == 2) {
      float amax = amax16(x);
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // two lanes per block of 32
      const int k = ue8m0_exponent(amax);
      const float scale = exp2_neg(k);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = e4m3x4_rn_sat(x[4 * i] * scale, x[4 * i + 1] * scale, x[4 * i + 2] * scale, x[4 * i + 3] * scale);
      uint8_t* dst = p.kv + (int64_t)slot * kRowBytesFp8_528;
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
      const uint32_t ue = (uint32_t)(k + 127);
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, ue, (8 * lane + 2 * i) & 31) << (8 * i);
      if (lane < 4) reinterpret_cast<uint32_t*>(dst + 512)[lane] = word;
    } else {
      uint32_t low, high;
      const uint32_t code = fp4_block(x, low, high);
      uint8_t* dst = p.kv + (int64_t)slot * kRowBytesFp4_288;
      reinterpret_cast<uint2*>(dst)[lane] = make_uint2(low, high);
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, code, (4 * lane + i) & 31) << (8 * i);
      if (lane < 8) reinterpret_cast<uint32_t*>(dst + 256)[lane] = word;
    }
  }
}

}  // namespace norms
}  // namespace mla
