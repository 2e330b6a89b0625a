// paged_decode.cuh -- what the kernels of a step over a paged cache share: the tokens a block takes, the scores, and where a
// block's result goes.
#pragma once

#include "paged.cuh"
#include "swa_common.cuh"

namespace la {

constexpr int kTile = 16;          // tokens that lie in one page: a page holds a multiple
constexpr int kPartTokens = 256;   // a part of a split sequence takes no fewer, but for the last one

// The tokens of a sequence that its query sees, [lo, hi), and how many parts they make of at most `splits`.  hi < 0: the
// length is out of range, and nothing of the sequence is written.
struct SeenTokens {
  int lo, hi, parts, tiles;  // tiles a part takes, counted from lo's tile
};
__device__ __forceinline__ SeenTokens seen_tokens(const PagedDecodeLaunch& a, int64_t s) {
  const int64_t n = a.lens[s];
  SeenTokens t{0, -1, 0, 0};
  if (n < 0 || n > a.c.width * a.c.page) return t;
  t.hi = (int)n;
  t.lo = a.window > 0 && a.window < n ? (int)(n - a.window) : 0;
  const int tiles = t.hi > t.lo ? (t.hi - 1) / kTile - t.lo / kTile + 1 : 0;
  t.tiles = max((tiles + a.splits - 1) / a.splits, kPartTokens / kTile);
  t.parts = (tiles + t.tiles - 1) / t.tiles;
  return t;
}

// The weighted mean; zero where no token has a weight: an empty sequence, pages that are not there, scores of -infinity alone.
__device__ __forceinline__ float mean_of(float sum, float total) { return total == 0.f ? 0.f : sum / total; }

// A capped score as by `capped`, which is off by ten half steps of fp32, to fp32: a fifth Chebyshev node leaves 2.6e-8 of the
// polynomial's value, and the difference from the cap is that of the magnitude: at -cap a quotient near one would be taken from it.
__device__ constexpr float kTanhFine[5] = {0.999999986757f, -0.333330679444f, 0.133247505048f, -0.0529842388285f, 0.0171313444313f};
__device__ __forceinline__ float capped_fine(float x, float cap, float inv_cap) {
  const float z = x * inv_cap, u = z * z;
  float q = kTanhFine[4];
#pragma unroll
  for (int i = 3; i >= 0; --i) q = fmaf(q, u, kTanhFine[i]);
  const float far = fmaf(-2.f * cap, rcp(1.f + ex2(fabsf(z) * (2.f * kLog2e))), cap);
  return fabsf(z) <= kStraight ? x * q : copysignf(far, x);
}

// Places of a part's sums, greatest score and sum of weights in the workspace.
__device__ __forceinline__ float* part_values(const PagedDecodeLaunch& a, int64_t s, int64_t h, int part) {
  return a.parts + ((s * a.H + h) * a.splits + part) * a.c.d;
}
__device__ __forceinline__ float2* part_sums(const PagedDecodeLaunch& a, int64_t s, int64_t h, int part) {
  return reinterpret_cast<float2*>(a.parts + a.S * a.H * a.splits * a.c.d) + (s * a.H + h) * a.splits + part;
}

cudaError_t launch_paged_decode_mma(const PagedDecodeLaunch& a, cudaStream_t stream);  // bf16 and 4-bit pages, without the join

}  // namespace la
