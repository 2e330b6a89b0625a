// swa_common.cuh -- what the kernels of masked window attention share: the interval of keys a query sees.
#pragma once

#include "layers.cuh"

namespace la {

struct KeySpan {
  int lo, hi;  // keys lo <= j < hi; empty when lo >= hi
};

// Query row i of sequence b, which has len tokens: its interval, clamped to the keys that exist.  Rows
// behind the last query and padding see nothing.
__device__ __forceinline__ KeySpan key_span(const SwaPrefillLaunch& a, int b, int i, int len) {
  const int p = (int)a.q_pos0 + i;
  KeySpan s{0, 0};
  if (i >= (int)a.Nq || p >= len) return s;
  const int64_t at = (int64_t)b * a.Nq + i;
  const int w = (int)min(a.window, (int64_t)INT32_MAX);
  int lo = a.key_lo ? max(a.key_lo[at], 0) : 0;
  const int hi = min(a.key_hi ? a.key_hi[at] : p + 1, len);
  if (w > 0) lo = max(lo, p - w + 1);
  if (lo < hi) s = KeySpan{lo, hi};
  return s;
}

__device__ __forceinline__ bool finite1(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ bool finite4(float4 x) { return finite1(x.x) && finite1(x.y) && finite1(x.z) && finite1(x.w); }

}  // namespace la
