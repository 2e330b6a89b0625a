// swa_common.cuh -- what the kernels of masked window attention share: the interval of keys a query sees.
#pragma once

#include "layers.cuh"

namespace la {

struct KeySpan {
  int lo, hi;  // keys lo <= j < hi; empty when lo >= hi
};

// Query row i of sequence b, which has len tokens: its interval, clamped to the keys that exist.  Rows
// behind the last query and padding see nothing.
__device__ __forceinline__ KeySpan key_span(const SwaPrefillLaunch& a, int64_t b, int64_t i, int64_t len) {
  const int64_t p = a.q_pos0 + i;
  KeySpan s{0, 0};
  if (i >= a.Nq || p >= len) return s;
  int64_t lo = a.key_lo ? max(a.key_lo[b * a.Nq + i], 0) : 0;
  int64_t hi = a.key_hi ? (int64_t)a.key_hi[b * a.Nq + i] : p + 1;
  if (a.window > 0) lo = max(lo, p - a.window + 1);
  hi = min(hi, len);
  if (lo >= hi) return s;
  s.lo = (int)lo;
  s.hi = (int)hi;
  return s;
}

__device__ __forceinline__ bool finite1(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ bool finite4(float4 x) { return finite1(x.x) && finite1(x.y) && finite1(x.z) && finite1(x.w); }

}  // namespace la
