// pipe.cuh -- what the persistent copy/MMA pipelines outside the decode share:
// waits, ring positions, copies.
#pragma once
#include <cuda.h>

#include "ptx.cuh"

namespace mla {

// The wait's slow path stands apart from the loops of the issuing threads:
// what they run per tile has to stay in the instruction cache.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, Guard g) { return wait(bar, parity, g); }
MLA_DEV bool wait_for(uint32_t bar, uint32_t parity, const Guard& g) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, g);
}

// a box of a 3-D tensor map, without a cache policy
MLA_DEV void tma_load_3d_plain(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// position in a ring whose length only the host knows: slot and phase are
// stepped, since a division per tile (some 150 cycles) is what the issuing
// threads would spend most of their time on
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  MLA_DEV void step(int length) {
    if (++slot == length) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

}  // namespace mla
