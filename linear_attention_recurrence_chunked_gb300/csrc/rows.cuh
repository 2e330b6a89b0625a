// rows.cuh -- rows of queries and keys in registers, eight elements a lane: loads and stores, and the position rotation's
// partners and factors.  What heads.cu and paged.cu share.
#pragma once

#include "layers.cuh"

namespace la {

// Eight consecutive elements in memory form.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void unpack(float (&o)[8]) const { unpack_vec(w, o); }
  __device__ __forceinline__ Raw8 from_lane(int lane) const {
    Raw8 r;
    r.w.x = __shfl_sync(kFullMask, w.x, lane); r.w.y = __shfl_sync(kFullMask, w.y, lane);
    r.w.z = __shfl_sync(kFullMask, w.z, lane); r.w.w = __shfl_sync(kFullMask, w.w, lane);
    return r;
  }
};
template <>
struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
  __device__ __forceinline__ void unpack(float (&o)[8]) const {
    float lo[4], hi[4];
    unpack_vec(a, lo);
    unpack_vec(b, hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) { o[i] = lo[i]; o[4 + i] = hi[i]; }
  }
  __device__ __forceinline__ Raw8 from_lane(int lane) const {
    Raw8 r;
    r.a.x = __shfl_sync(kFullMask, a.x, lane); r.a.y = __shfl_sync(kFullMask, a.y, lane);
    r.a.z = __shfl_sync(kFullMask, a.z, lane); r.a.w = __shfl_sync(kFullMask, a.w, lane);
    r.b.x = __shfl_sync(kFullMask, b.x, lane); r.b.y = __shfl_sync(kFullMask, b.y, lane);
    r.b.z = __shfl_sync(kFullMask, b.z, lane); r.b.w = __shfl_sync(kFullMask, b.w, lane);
    return r;
  }
};

// A lane's part in the rotation of its row's first `rot` elements (a multiple of 16).  Lane c of a row holds elements 8 c to
// 8 c + 7, so that with pairs (i, i + rot / 2) the partners of all eight are those of lane c +- rot / 16, in order; with
// neighbours as pairs they are the lane's own.  x cos + y sin with y the partner, sin negative for a pair's first element.
struct Turn {
  bool on;        // the lane's elements are rotated
  int partner;    // warp lane of the partners (pairs rot / 2 apart)
  float c[8], s[8];
  // cos, sin: the row of the token's position
  __device__ __forceinline__ void init(const float* cos, const float* sin, int rot, bool interleaved, int lane, int col) {
    on = col * 8 < rot;
    partner = lane;
    if (!on) {
#pragma unroll
      for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
      return;
    }
    if (interleaved) {
      const float4 cc = *reinterpret_cast<const float4*>(cos + 4 * col), ss = *reinterpret_cast<const float4*>(sin + 4 * col);
      const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = cv[i / 2];
        s[i] = i & 1 ? sv[i / 2] : -sv[i / 2];
      }
      return;
    }
    const int half = rot / 16;  // lanes of the pairs' first elements
    const bool second = col >= half;
    partner = second ? lane - half : lane + half;
    const int at = 8 * (second ? col - half : col);
    Raw8<float> cr, sr;
    cr.load(cos + at);
    sr.load(sin + at);
    cr.unpack(c);
    sr.unpack(s);
    if (!second) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
  }
};

// Position of token n of sequence b, or -1 outside the tables.
__device__ __forceinline__ int64_t table_row(int64_t first, int64_t n, int64_t positions) {
  const uint64_t p = (uint64_t)first + (uint64_t)n;
  return p < (uint64_t)positions ? (int64_t)p : -1;
}

}  // namespace la
