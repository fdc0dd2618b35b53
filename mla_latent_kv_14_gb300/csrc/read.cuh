// read.cuh -- rows of the paged latent cache read back in 16 bits: the cached
// prefix that a prompt's next chunk expands into keys and values.
//
// Row o of the output (offsets[b] <= o < offsets[b + 1]) is token starts[b] + o
// - offsets[b] of request b; a quantised value is code x scale, formed exactly
// in fp32 (4 significant bits times a scale's 24, 1 or 4; the 656-byte rows'
// product rounds to fp32) and rounded once more to the output's type.
//
// Bound by its bytes: a row in, 1152 (1024) bytes out. Measured (GB300): 262144
// rows of 656 bytes 74.3 us (0.94 of the copy bandwidth), 88000 of 288 bytes 19.1
// us (0.84; 25 with two 16-byte stores of a lane's 32 bytes).
#pragma once
#include "rows.cuh"

namespace mla {
namespace read {

struct ReadParams {
  const uint8_t* kv;
  const int32_t* block_table;  // [batch, max_blocks]
  const int32_t* offsets;      // [batch + 1]
  const int32_t* starts;       // [batch] or null
  int64_t num_blocks;
  int batch, max_blocks;
  int64_t total;
  uint16_t* out;
  int64_t out_stride;          // elements
  int wide;                    // rows of out are 32-B aligned
  uint32_t* status;            // or null
};

// one warp takes two consecutive rows, all of their loads in flight together (262144 rows of 656 bytes: 75.8 us, 84.0
// with one row, 78.5 with four; 88000 of 288 bytes 21.9, 24.3 and 25.1, before the 32-byte stores)
constexpr int kReadWarps = 8;
constexpr int kReadRows = 2;

MLA_DEV float2 e4m3x2_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return unpack_f16x2(h);
}
// the eight e2m1 values of a word, the low nibble of the low byte first
MLA_DEV void e2m1x8_f32(uint32_t w, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\tcvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = unpack_f16x2(h[k]);
    v[2 * k] = x.x;
    v[2 * k + 1] = x.y;
  }
}

template <int kFormat, bool kFp16>  // kFp16: the output's type (16-bit rows are copied)
__global__ void __launch_bounds__(32 * kReadWarps) mla_read_kv_kernel(const ReadParams p) {
  constexpr int kRows = kReadRows;
  constexpr int kRow = kFormat == 0 ? 2 * kDK : kFormat == 1 ? kRowBytesFp8 : kFormat == 2 ? kRowBytesFp8_528 : kRowBytesFp4_288;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t first = ((int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5)) * kRows;
  // lane k (below kRows) finds row first + k: its request, page and cache row
  const int64_t o = first + lane;
  int64_t row = -2;            // -2: nothing to write, -1: zeros
  if (lane < kRows && o < p.total && o < __ldg(p.offsets + p.batch)) {
    int lo = 0, hi = p.batch;  // the last request that starts at or before o (empty ones before it start there too)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.offsets + mid) <= o) lo = mid;
      else hi = mid;
    }
    const int64_t in = o - __ldg(p.offsets + lo), token = (p.starts ? __ldg(p.starts + lo) : 0) + in;
    const int64_t page = token / kTile;
    if (in >= 0) row = -1;     // below 0: before the first request
    if (in >= 0 && token >= 0 && page < p.max_blocks) {
      const int32_t at = __ldg(p.block_table + (int64_t)lo * p.max_blocks + page);
      if (at >= 0 && at < p.num_blocks) row = (int64_t)at * kTile + token % kTile;
    }
    if (row == -1) rows::flag(p.status, STATUS_INDEX);
  }
  const uint8_t* src[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t r = __shfl_sync(0xffffffffu, row, k);
    src[k] = r >= 0 ? p.kv + r * kRow : r == -1 ? p.kv : nullptr;
  }
  const uint32_t zero = __ballot_sync(0xffffffffu, row == -1);
  if (kFormat == 0) {
    uint4 a[kRows], b[kRows];
    uint32_t c[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (src[k]) {
        a[k] = __ldg(reinterpret_cast<const uint4*>(src[k]) + lane);
        b[k] = __ldg(reinterpret_cast<const uint4*>(src[k]) + 32 + lane);
        c[k] = __ldg(reinterpret_cast<const uint32_t*>(src[k] + 1024) + lane);
      }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (src[k]) {
        if ((zero >> k) & 1u) {
          a[k] = b[k] = make_uint4(0, 0, 0, 0);
          c[k] = 0;
        }
        uint16_t* dst = p.out + (first + k) * p.out_stride;
        reinterpret_cast<uint4*>(dst)[lane] = a[k];
        reinterpret_cast<uint4*>(dst)[32 + lane] = b[k];
        reinterpret_cast<uint32_t*>(dst + 512)[lane] = c[k];
      }
  } else {
    // lane l holds values [16l, 16l + 16)
    uint4 code[kRows];
    float scale[kRows];
    uint32_t rope[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (src[k]) {
        if (kFormat == 3) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(src[k]) + lane);
          code[k] = make_uint4(v.x, v.y, 0, 0);
          scale[k] = __uint_as_float(__ldg(src[k] + 256 + lane));
        } else {
          code[k] = __ldg(reinterpret_cast<const uint4*>(src[k]) + lane);
          if (kFormat == 1) {
            scale[k] = __ldg(reinterpret_cast<const float*>(src[k] + 512) + (lane >> 3));
            rope[k] = __ldg(reinterpret_cast<const uint32_t*>(src[k] + 528) + lane);
          } else {
            scale[k] = __uint_as_float(__ldg(src[k] + 512 + (lane >> 1)));
          }
        }
      }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (src[k]) {
        float f = scale[k];
        if (kFormat == 2) {   // 2^(byte - 127); byte 0 is 2^-127, a subnormal, byte 255 NaN
          const uint32_t e = __float_as_uint(f);
          f = __uint_as_float(e == 255u ? 0x7FFFFFFFu : e ? e << 23 : 0x00400000u);
        } else if (kFormat == 3) {
          f = e4m3x2_f32(__float_as_uint(f)).x;
        }
        if ((zero >> k) & 1u) code[k] = make_uint4(0, 0, 0, 0), rope[k] = 0, f = 0.f;
        float v[16];
        const uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
        if (kFormat == 3) {
          e2m1x8_f32(w[0], v);
          e2m1x8_f32(w[1], v + 8);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 x = e4m3x2_f32((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
            v[2 * j] = x.x;
            v[2 * j + 1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j], f);
        uint16_t* dst = p.out + (first + k) * p.out_stride;
        rows::store16<kFp16>(dst + 16 * lane, v, p.wide);
        if (kFormat == 1) {
          if (kFp16) {
            const float2 x = rows::unpack2<false>(rope[k]);
            rope[k] = rows::pack2<true>(x.x, x.y);
          }
          reinterpret_cast<uint32_t*>(dst + 512)[lane] = rope[k];
        }
      }
  }
}

}  // namespace read
}  // namespace mla
