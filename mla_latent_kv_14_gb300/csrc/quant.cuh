// quant.cuh -- writer of the 656-byte FP8 cache rows
// ("FlashMLA 实战：MLA 注意力加速指南", §FP8 缓存怎么把 KV 压掉四成; "矩阵、注意力与
// GPU：拆解 DeepGEMM 与 FlashMLA", §八 '格式'): per 128 latent values one fp32
// scale = amax/448 (1.0 for an all-zero block), e4m3 code = round-to-nearest-
// even of x/scale saturated to +-448, both divisions IEEE round-to-nearest;
// then the 4 scales; then the 64 RoPE dims as bf16.
#pragma once
#include "codes.cuh"

namespace mla {

// One warp per row; lane l owns values [4l, 4l+4) of each 128-value block.
__global__ void __launch_bounds__(256) mla_quant_fp8_kernel(const uint16_t* __restrict__ kv,
                                                            uint8_t* __restrict__ out, int64_t n) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); row < n; row += warps) {
    const uint16_t* src = kv + row * kDK;
    uint8_t* dst = out + row * kRowBytesFp8;
    float scales[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint2 raw = *reinterpret_cast<const uint2*>(src + j * 128 + lane * 4);
      float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                    __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)};
      float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = e4m3_scale(amax);
      scales[j] = scale;
      *reinterpret_cast<uint32_t*>(dst + j * 128 + lane * 4) = e4m3x4_rn_sat(
          __fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale), __fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale));
    }
    if (lane == 0)
      *reinterpret_cast<float4*>(dst + 512) = make_float4(scales[0], scales[1], scales[2], scales[3]);
    // RoPE: 64 bf16 = 128 bytes, 4 per lane
    *reinterpret_cast<uint32_t*>(dst + 528 + lane * 4) =
        *reinterpret_cast<const uint32_t*>(src + 512 + lane * 2);
  }
}

}  // namespace mla

// ---------------------------------------------------------------------------
// Writers of the V4.1 rows of 512 values ("矩阵、注意力与 GPU：拆解 DeepGEMM 与
// FlashMLA", §八 '版本漂移' and the §十 format table; §三 'UE8M0': a scale is a
// power of two, rounded up). Input: bf16 rows [n, 512].
// ---------------------------------------------------------------------------
namespace mla {

// sixteen bf16 values from 32 bytes at src
__device__ __forceinline__ void load_bf16x16(const uint16_t* src, float* x) {
  const uint4 a = *reinterpret_cast<const uint4*>(src);
  const uint4 b = *reinterpret_cast<const uint4*>(src + 8);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// 528-byte rows: 512 e4m3 codes, then 16 UE8M0 scales (byte k + 127 for the
// scale 2^k of values [32j, 32j + 32); ue8m0_exponent gives k).
// One warp per row; lane l owns values [16l, 16l + 16) (two lanes per block).
__global__ void __launch_bounds__(256) mla_quant_fp8_528_kernel(const uint16_t* __restrict__ kv,
                                                                uint8_t* __restrict__ out, int64_t n) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); row < n; row += warps) {
    float x[16];
    load_bf16x16(kv + row * kDV41 + 16 * lane, x);
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const int k = ue8m0_exponent(amax);
    const float inv = exp2_neg(k);  // x * 2^-k is exact
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = e4m3x4_rn_sat(x[4 * q] * inv, x[4 * q + 1] * inv, x[4 * q + 2] * inv, x[4 * q + 3] * inv);
    }
    uint8_t* dst = out + row * kRowBytesFp8_528;
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    // the 16 scale bytes, gathered into lanes 0..3 (one word each)
    const uint32_t ue = (uint32_t)(k + 127);
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) word |= __shfl_sync(0xffffffffu, ue, (8 * lane + 2 * b) & 31) << (8 * b);
    if (lane < 4) *reinterpret_cast<uint32_t*>(dst + 512 + 4 * lane) = word;
  }
}

// 288-byte rows: 512 e2m1 codes (value 2i in the low nibble of byte i), then 32
// e4m3 scales (values [16j, 16j + 16); fp4_block takes every decision).
// One warp per row; lane l owns block l.
__global__ void __launch_bounds__(256) mla_quant_fp4_288_kernel(const uint16_t* __restrict__ kv,
                                                                uint8_t* __restrict__ out, int64_t n) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); row < n; row += warps) {
    float x[16];
    load_bf16x16(kv + row * kDV41 + 16 * lane, x);
    uint32_t lo, hi;
    const uint32_t c = fp4_block(x, lo, hi);
    uint8_t* dst = out + row * kRowBytesFp4_288;
    *reinterpret_cast<uint2*>(dst + 8 * lane) = make_uint2(lo, hi);
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) word |= __shfl_sync(0xffffffffu, c, (4 * lane + b) & 31) << (8 * b);
    if (lane < 8) *reinterpret_cast<uint32_t*>(dst + 256 + 4 * lane) = word;
  }
}

}  // namespace mla
