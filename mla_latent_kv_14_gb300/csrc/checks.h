// checks.h -- argument checks and launches that the entry points around the
// decode share.
#pragma once
#include <initializer_list>

#include "host.h"
#include "params.h"
#include "rows.cuh"

namespace mla {

constexpr int64_t kMaxRows = int64_t(1) << 31;

inline bool dtype_ok(int dtype) { return dtype == MLA_DTYPE_BF16 || dtype == MLA_DTYPE_FP16; }
inline bool cache_ok(int64_t num_blocks, int page_block) {
  return num_blocks > 0 && page_block == kTile && num_blocks < kMaxRows / kTile;
}
// `count` strides in the range of addresses
inline bool in_memory(int64_t stride, int64_t count) { return stride <= (int64_t(1) << 46) / (count > 0 ? count : 1); }
// strides in elements that keep 16-byte rows aligned
inline bool stride_ok(int64_t s, int64_t least, int64_t count) { return s >= least && s % 8 == 0 && in_memory(s, count); }
// memory of a call: `bytes` from `at` on (gaps between rows included). An
// output, the status word among them, must not share any with another argument:
// blocks read what others have already written.
struct Span {
  const void* at;
  int64_t bytes;
  bool meets(const Span& o) const {
    const intptr_t a = reinterpret_cast<intptr_t>(at), b = reinterpret_cast<intptr_t>(o.at);
    return at && o.at && a < b + o.bytes && b < a + bytes;
  }
};
// every output apart from the inputs and from the other outputs
inline bool apart(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span* other = outputs.begin(); other != o; ++other)
      if (o->meets(*other)) return false;
    for (const Span& i : inputs)
      if (o->meets(i)) return false;
  }
  return true;
}
inline Span int32_span(const int32_t* at, int64_t n) { return {at, 4 * n}; }
inline Span status_span(const uint32_t* at) { return {at, 4}; }
// the table's rows that an int32 position reaches
inline Span table_span(const rows::Positions& p) {
  return {p.table, 4 * rows::kRope * (p.max_positions < kMaxRows ? p.max_positions : kMaxRows)};
}
inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }
// Rows of `w` elements in runs of `inner` rows `pitch` apart (at least w), the
// `runs` starting `outer` apart (a run's length at least). True if the same rows
// `d` elements further on meet any of them: if d is less than w off some
// a outer + b pitch. Only two values of a, and two of b for each, come that near.
inline bool rows_meet(int64_t d, int64_t outer, int64_t runs, int64_t pitch, int64_t inner, int64_t w) {
  const int64_t a0 = runs > 1 ? floor_div(d, outer) : 0;
  for (int64_t a = a0; a <= a0 + 1; ++a) {
    if (a <= -runs || a >= runs) continue;
    const int64_t rest = d - a * outer, b0 = floor_div(rest, pitch);
    for (int64_t b = b0; b <= b0 + 1; ++b)
      if (b > -inner && b < inner && rest - b * pitch < w && b * pitch - rest < w) return true;
  }
  return false;
}
// Launched as a programmatic dependent: every kernel here waits for the grid
// before it (griddepcontrol.wait) ahead of its first global access, so only
// its launch overlaps that grid.
template <typename P, typename... A>
mla_status launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, void* stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  MLA_CUDA(cudaLaunchKernelEx(&cfg, kernel, p));
  return MLA_OK;
}

// SMs of the current device, asked once per device
inline mla_status sm_count(int* dev, int* sms) {
  static std::atomic<int> known[kMaxDevices];
  MLA_CUDA(cudaGetDevice(dev));
  if (*dev >= kMaxDevices) return MLA_ERR_UNSUPPORTED;
  *sms = known[*dev].load(std::memory_order_relaxed);
  if (*sms > 0) return MLA_OK;
  MLA_CUDA(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev));
  known[*dev].store(*sms, std::memory_order_relaxed);
  return MLA_OK;
}

inline mla_status check_positions(const rows::Positions& p) {
  if (!p.positions || !p.table || !aligned(p.positions, 4) || !aligned(p.table, 16)) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

}  // namespace mla
