// tree_common.h -- what the kernels on drafted token trees share.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "device_checks.h"
#include "specverify_tree.h"

namespace svtree {

constexpr int kWave = 64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

inline int launch_status() { return hipGetLastError() == hipSuccess ? SV_OK : SV_EHIP; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool pow2(int64_t x) { return x >= 1 && (x & (x - 1)) == 0; }

// Strides in elements. No memory holds rows that lie further apart, and below it a
// stride in bytes cannot overflow.
inline bool stride_ok(int64_t x) { return x >= 0 && x < (int64_t(1) << 48); }

inline int log2_of(int64_t x) { return 63 - __builtin_clzll(uint64_t(x)); }

inline bool workspace_ok(const void* ws, size_t have, size_t need, int* status) {
  if (ws == nullptr || have < need) {
    *status = SV_EWORKSPACE;
    return false;
  }
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) {
    *status = SV_EALIGN;
    return false;
  }
  return true;
}

// Whether the runs of `width` elements of an output lie apart: taken by rising
// stride, each axis steps over all that the axes before it span.
inline bool apart(int axes, const int64_t* sizes, const int64_t* strides, int64_t width) {
  bool taken[4] = {};
  __int128 span = width;
  for (int round = 0; round < axes; ++round) {
    int least = -1;
    for (int i = 0; i < axes; ++i)
      if (!taken[i] && (least < 0 || strides[i] < strides[least])) least = i;
    taken[least] = true;
    if (sizes[least] <= 1) continue;
    if (strides[least] < span) return false;
    span += __int128(strides[least]) * (sizes[least] - 1);
  }
  return true;
}

inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

__device__ __forceinline__ void set_error(int32_t* err, int bits) {
  if (err) atomicOr(err, bits);
}

// The rows of request b; n < 0 when node_start is no tree's there.
struct Nodes {
  int64_t first;
  int32_t n;
};
__device__ __forceinline__ Nodes nodes_of(const int32_t* __restrict__ node_start, int64_t b,
                                          int64_t T, int max_nodes) {
  const int64_t lo = node_start[b], hi = node_start[b + 1];
  if (lo < 0 || hi < lo || hi > T || hi - lo > max_nodes) return Nodes{0, -1};
  return Nodes{lo, int32_t(hi - lo)};
}

}  // namespace svtree
