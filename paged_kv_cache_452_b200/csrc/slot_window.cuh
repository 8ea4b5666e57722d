// Index arithmetic of the row operators: division by a launch's constants, and
// windows of a slot list that a d-major e4m3 V pool is read and written by:
// 16 tokens whose slots fill an aligned half or whole block make one 16-byte
// vector per element of head_dim, instead of 16 single bytes.
#pragma once

#include <stdint.h>

#include "pa_kernels.h"

namespace pa {
namespace dev {

__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.mul) + n) >> f.shift; }

constexpr int kWindow = 16;  // tokens; divides every block size

// Where window i of the list starts: at token 16 i, or up to 15 tokens before
// it where those lead up to slot 16 i from a multiple of 16 (a run that does
// not start on one then still falls into aligned windows).  The windows are
// a partition of the list for every list: start(i) <= 16 i < start(i + 1).
__device__ __forceinline__ int64_t window_start(const int64_t* slots, int64_t num_tokens, int64_t i) {
  const int64_t t = i * kWindow;
  if (i == 0) return 0;
  if (t >= num_tokens) return num_tokens;
  const int64_t s = __ldg(slots + t);
  const int64_t r = s & (kWindow - 1);
  return s >= 0 && r > 0 && __ldg(slots + t - r) == s - r ? t - r : t;
}

// Whole warp: whether tokens t .. t + 15 have consecutive slots from an
// aligned one on, all in the pool; *first receives it.
__device__ __forceinline__ bool window_aligned(const int64_t* slots, int64_t t, int64_t n, int64_t num_slots,
                                               int64_t* first) {
  const int lane = threadIdx.x & 31;
  const int64_t s = lane < kWindow && lane < n ? __ldg(slots + t + lane) : -1;
  const int64_t s0 = __shfl_sync(0xffffffffu, s, 0);
  *first = s0;
  const bool fits = lane >= kWindow || (s == s0 + lane);
  return __all_sync(0xffffffffu, fits) && s0 >= 0 && (s0 & (kWindow - 1)) == 0 && s0 + kWindow <= num_slots;
}

}  // namespace dev
}  // namespace pa
