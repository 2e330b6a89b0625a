// rows.cuh -- rows of queries and keys in registers, eight elements a lane as four pairs of fp32, and the position rotation
// of pairs.  What heads.cu and paged.cu share.
#pragma once

#include "layers.cuh"

namespace la {

// How a row's pairs lie: not rotated, or neighbours, its lanes hold eight elements in a row; elements rot / 2 apart, a lane
// of the rotated part holds two runs of four, each other's partners.  So a lane turns its own elements whatever the pairs.
enum TurnKind { kTurnNone, kTurnNeighbours, kTurnHalves };

// First elements of lane `col`'s two runs of four.
template <TurnKind kTurn>
__device__ __forceinline__ int2 runs_of(int col, int rot) {
  if (kTurn == kTurnHalves && col * 8 < rot) return make_int2(4 * col, rot / 2 + 4 * col);
  return make_int2(8 * col, 8 * col + 4);
}

// Eight elements in memory form: two runs of four, 8 or 16 bytes each.  `whole`: they are one run of eight.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void zero() { a = b = make_uint2(0u, 0u); }
  template <bool whole>
  __device__ __forceinline__ void load(const __nv_bfloat16* x, int2 at) {
    if constexpr (whole) {
      const uint4 w = *reinterpret_cast<const uint4*>(x + at.x);
      a = make_uint2(w.x, w.y); b = make_uint2(w.z, w.w);
    } else {
      a = *reinterpret_cast<const uint2*>(x + at.x);
      b = *reinterpret_cast<const uint2*>(x + at.y);
    }
  }
  template <bool whole>
  __device__ __forceinline__ void store(__nv_bfloat16* y, int2 at) const {
    if constexpr (whole) {
      *reinterpret_cast<uint4*>(y + at.x) = make_uint4(a.x, a.y, b.x, b.y);
    } else {
      *reinterpret_cast<uint2*>(y + at.x) = a;
      *reinterpret_cast<uint2*>(y + at.y) = b;
    }
  }
  static __device__ __forceinline__ f32x2 wide(uint32_t w) { return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
  __device__ __forceinline__ void unpack(f32x2 (&v)[4]) const { v[0] = wide(a.x); v[1] = wide(a.y); v[2] = wide(b.x); v[3] = wide(b.y); }
  static __device__ __forceinline__ uint32_t narrow(f32x2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ void pack(const f32x2 (&v)[4]) {
    a = make_uint2(narrow(v[0]), narrow(v[1]));
    b = make_uint2(narrow(v[2]), narrow(v[3]));
  }
};
template <>
struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  template <bool whole>
  __device__ __forceinline__ void load(const float* x, int2 at) {
    a = *reinterpret_cast<const uint4*>(x + at.x);
    b = *reinterpret_cast<const uint4*>(x + at.y);
  }
  template <bool whole>
  __device__ __forceinline__ void store(float* y, int2 at) const {
    *reinterpret_cast<uint4*>(y + at.x) = a;
    *reinterpret_cast<uint4*>(y + at.y) = b;
  }
  static __device__ __forceinline__ f32x2 two(uint32_t lo, uint32_t hi) { return pack2(__uint_as_float(lo), __uint_as_float(hi)); }
  __device__ __forceinline__ void unpack(f32x2 (&v)[4]) const { v[0] = two(a.x, a.y); v[1] = two(a.z, a.w); v[2] = two(b.x, b.y); v[3] = two(b.z, b.w); }
  __device__ __forceinline__ void pack(const f32x2 (&v)[4]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
    a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
};

// A lane's angles: x cos + y sin with y the partner, sin negative for a pair's first element.  Pairs of registers hold two
// elements of a run (halves: v[0], v[1] and their partners v[2], v[3], four angles) or a pair (neighbours).
template <TurnKind kTurn>
struct Turn {
  bool on;  // the lane's elements are rotated
  f32x2 c[kTurn == kTurnNeighbours ? 4 : 2], s[kTurn == kTurnNeighbours ? 4 : 2], n[2];  // cosines, sines, their negatives
  // cos, sin: the row of the token's position
  __device__ __forceinline__ void init(const float* cos, const float* sin, int rot, int col) {
    on = kTurn != kTurnNone && col * 8 < rot;
    if (!on) return;
    const float4 cc = *reinterpret_cast<const float4*>(cos + 4 * col), ss = *reinterpret_cast<const float4*>(sin + 4 * col);
    if constexpr (kTurn == kTurnNeighbours) {
      c[0] = pack2(cc.x, cc.x); c[1] = pack2(cc.y, cc.y); c[2] = pack2(cc.z, cc.z); c[3] = pack2(cc.w, cc.w);
      s[0] = pack2(-ss.x, ss.x); s[1] = pack2(-ss.y, ss.y); s[2] = pack2(-ss.z, ss.z); s[3] = pack2(-ss.w, ss.w);
    } else {
      c[0] = pack2(cc.x, cc.y); c[1] = pack2(cc.z, cc.w);
      s[0] = pack2(ss.x, ss.y); s[1] = pack2(ss.z, ss.w);
      n[0] = pack2(-ss.x, -ss.y); n[1] = pack2(-ss.z, -ss.w);
    }
  }
  // fn(x, c, y, s): x c + y s of two elements
  template <typename Fn>
  __device__ __forceinline__ void apply(f32x2 (&v)[4], Fn fn) const {
    if constexpr (kTurn == kTurnNeighbours) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(v[i], lo, hi);
        v[i] = fn(v[i], c[i], pack2(hi, lo), s[i]);
      }
    } else if constexpr (kTurn == kTurnHalves) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x2 a = v[i], b = v[2 + i];
        v[i] = fn(a, c[i], b, n[i]);
        v[2 + i] = fn(b, c[i], a, s[i]);
      }
    }
  }
};
__device__ __forceinline__ f32x2 turn_rounded(f32x2 x, f32x2 c, f32x2 y, f32x2 s) { return fma2(x, c, mul2(y, s)); }

// Row of the tables of a token's position, first + n, or -1 outside them.
__device__ __forceinline__ int64_t table_row(int64_t first, int64_t n, int64_t positions) {
  const uint64_t p = (uint64_t)first + (uint64_t)n;
  return p < (uint64_t)positions ? (int64_t)p : -1;
}

// Division by a number that the host knows: a product and two shifts (Granlund and Montgomery 1994), where the instruction
// sequence of a division takes thirty.
struct Divisor {
  uint32_t d, factor, shift;
  Divisor() = default;
  explicit Divisor(int64_t by) : d((uint32_t)by), factor(0), shift(0) {
    while (shift < 32 && (uint64_t(1) << shift) < d) ++shift;
    factor = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d)) / d + 1);
  }
  // n / d for every 32-bit n
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    const uint32_t t = __umulhi(n, factor);
    return shift == 0 ? n : (t + ((n - t) >> 1)) >> (shift - 1);
  }
};

}  // namespace la
