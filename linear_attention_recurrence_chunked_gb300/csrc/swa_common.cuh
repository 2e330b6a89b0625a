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

// Where a bias counts a row's distances from.  A softmax is the same for scores that all have moved by as much, so what
// the row's keys have in common of slope |p - j| is left out: the distance from the row to its interval, which in fp32
// would cost the scores their lower bits (a row 70000 tokens from its 300 keys at a slope of 0.7 was off by 2e-3).  For a
// key j of the interval |p - j| less that distance is |c - j| with c, the row moved to its interval's end.
__device__ __forceinline__ int bias_origin(KeySpan s, int p) { return s.lo < s.hi ? max(s.lo, min(p, s.hi - 1)) : p; }

// tanh(z) / z in z^2 on [0, 1/4] through four Chebyshev nodes, off by 6e-7 of the value at most.  A capped score is
// cap tanh(z) = x Q(z^2) with z = x / cap up to kStraight, and cap - 2 cap / (1 + e^2z) beyond, where the difference
// loses nothing that the value itself would hold: as the only form it would leave an error of 1e-7 cap in scores
// that are far below a large cap.
constexpr float kStraight = 0.5f;
__device__ constexpr float kTanh[4] = {0.9999994636f, -0.3332628310f, 0.1318994015f, -0.0443927385f};

__device__ __forceinline__ float capped(float x, float cap, float inv_cap) {
  const float z = x * inv_cap, u = z * z;
  const float near = x * fmaf(fmaf(fmaf(kTanh[3], u, kTanh[2]), u, kTanh[1]), u, kTanh[0]);
  const float far = fmaf(-2.f * cap, rcp(1.f + ex2(z * (2.f * kLog2e))), cap);
  return fabsf(z) <= kStraight ? near : far;
}

__device__ __forceinline__ bool finite1(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ bool finite4(float4 x) { return finite1(x.x) && finite1(x.y) && finite1(x.z) && finite1(x.w); }

}  // namespace la
