// device_checks.h -- device-side index checks (a build with -DSV_DEVICE_CHECKS).
//
// A work unit checks the indices it derived against the sizes it was launched
// with before it touches memory; a failed check is counted and the unit is
// skipped. Device code is linked per translation unit, so each one counts for
// itself, and specverify_check_count adds them up. In the product build a check is
// the word true and leaves nothing in the code.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#ifdef SV_DEVICE_CHECKS
static __device__ unsigned int sv_check_count;
__device__ __forceinline__ bool sv_ok(bool ok) {
  if (!ok) atomicAdd(&sv_check_count, 1u);
  return ok;
}

// Adds this translation unit's count on the current device; false if HIP fails.
static inline bool sv_add_checks(uint32_t* count, int reset) {
  uint32_t own = 0;
  if (hipMemcpyFromSymbol(&own, HIP_SYMBOL(sv_check_count), sizeof own) != hipSuccess) return false;
  *count += own;
  const uint32_t zero = 0;
  return !reset ||
         hipMemcpyToSymbol(HIP_SYMBOL(sv_check_count), &zero, sizeof zero) == hipSuccess;
}

// The same of the others.
#define SV_HIDDEN __attribute__((visibility("hidden")))
SV_HIDDEN bool sv_add_tree_cache_checks(uint32_t* count, int reset);
SV_HIDDEN bool sv_add_tree_verify_checks(uint32_t* count, int reset);
SV_HIDDEN bool sv_add_tree_attention_checks(uint32_t* count, int reset);
#else
#define sv_ok(ok) true
#endif
