// Host-side argument checks shared by the C-ABI layers.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace check {

inline bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

inline bool aligned_to(const void *p, size_t e) { return (uintptr_t)p % e == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void *p, size_t bytes) {
  return Range{(uintptr_t)p, (uintptr_t)p + bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// Device must be a Blackwell datacenter part (compute capability 10.x): the
// library is compiled for sm_100a only.
inline kda_status_t check_device() {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return KDA_ERR_CUDA;
  return major == 10 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

}  // namespace check
}  // namespace kda
