// layers.cuh -- device helpers shared by the convolution, the selective scan and the masked window
// attention: 16-byte vectors of either element type, and the scalar functions of their epilogues.
#pragma once

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace la {

// Lets `kernel` use `bytes` of dynamic shared memory on the current device; `done` (one per kernel) remembers the
// devices that know.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// elements of T in a 16-byte vector
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack_vec(uint4 u, float (&o)[8]) {  // 8 bf16
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(w[i] << 16);
    o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack_vec(uint4 u, float (&o)[4]) {  // 4 fp32
  o[0] = __uint_as_float(u.x); o[1] = __uint_as_float(u.y); o[2] = __uint_as_float(u.z); o[3] = __uint_as_float(u.w);
}

// Four elements in memory form, and whole or partial (zero beyond `valid`) access to them.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void unpack(float (&o)[4]) const { unpack_vec(w, o); }
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void load(const float* p, int valid) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = i < valid ? __float_as_uint(p[i]) : 0u;
    w = make_uint4(x[0], x[1], x[2], x[3]);
  }
  __device__ __forceinline__ void store(float* p, int valid) const {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < valid) p[i] = __uint_as_float(x[i]);
  }
};
template <>
struct Raw4<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void zero() { w = make_uint2(0u, 0u); }
  __device__ __forceinline__ void unpack(float (&o)[4]) const {
    o[0] = __uint_as_float(w.x << 16); o[1] = __uint_as_float(w.x & 0xffff0000u);
    o[2] = __uint_as_float(w.y << 16); o[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int valid) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = i < valid ? (uint32_t)__bfloat16_as_ushort(p[i]) : 0u;
    w = make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int valid) const {
    const uint32_t x[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < valid) p[i] = __ushort_as_bfloat16((unsigned short)x[i]);
  }
};

// Raw vector of the elements [0, valid) at p (zero beyond); `vec` says that a 16-byte access is allowed.
template <typename T>
__device__ __forceinline__ uint4 load_raw(const T* p, int valid, bool vec) {
  if (vec && valid >= kVec<T>) return *reinterpret_cast<const uint4*>(p);
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    if (i < valid) {
      if constexpr (sizeof(T) == 2) w[i / 2] |= (uint32_t)__bfloat16_as_ushort(p[i]) << (16 * (i & 1));
      else w[i] = __float_as_uint(p[i]);
    }
  }
  return u;
}
template <typename T>
__device__ __forceinline__ void store_raw(T* p, uint4 u, int valid, bool vec) {
  if (vec && valid >= kVec<T>) {
    *reinterpret_cast<uint4*>(p) = u;
    return;
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    if (i < valid) {
      if constexpr (sizeof(T) == 2) p[i] = __ushort_as_bfloat16((unsigned short)(w[i / 2] >> (16 * (i & 1))));
      else p[i] = __uint_as_float(w[i]);
    }
  }
}

// N consecutive floats as TOut (round to nearest even); `vec`: the address is aligned to the vector
// (16 bytes, or 8 for four bf16).
template <int N>
__device__ __forceinline__ void store_floats(float* p, const float (&x)[N], int valid, bool vec) {
  if (vec && valid >= N) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < valid) p[i] = x[i];
}
template <int N>
__device__ __forceinline__ void store_floats(__nv_bfloat16* p, const float (&x)[N], int valid, bool vec) {
  if (vec && valid >= N) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < valid) p[i] = __float2bfloat16_rn(x[i]);
}

// Paired fp32 operations: two independent lanes of a 64-bit register pair.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ f32x2 ex2_2(f32x2 x) {
  float lo, hi;
  unpack2(x, lo, hi);
  return pack2(ex2(lo), ex2(hi));
}

// x / (1 + exp(-x)).  exp(-x) overflows to infinity below x = -88, where the product with the reciprocal
// is the limit 0.
__device__ __forceinline__ float silu(float x) { return x * rcp(1.f + ex2(-kLog2e * x)); }

// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|).  The logarithm of 1 + e would lose the small
// values that a step size takes (e = 1e-3 keeps 13 bits of it), so log1p(e) = 2 atanh(r), r = e / (2 + e)
// in (0, 1/3].  atanh(r) / r = 1 + q/3 + q^2/5 + ..., q = r^2 <= 1/9, as 1 + q times the cubic that meets the
// series at the four Chebyshev nodes of [0, 1/9]: off by 1.6e-8 of the value at most, a quarter of an fp32
// rounding.  expf, not its fast form, whose error of 1.2 |x| ulp would reach every state.  A NaN passes
// through e.
__device__ __forceinline__ float softplus(float x) {
  const float e = expf(-fabsf(x));
  const float r = e * rcp(2.f + e), q = r * r;
  float p = fmaf(0.1342574954f, q, 0.1411830932f);
  p = fmaf(p, q, 0.2000378072f);
  p = fmaf(p, q, 0.3333331943f);
  p = fmaf(p, q, 1.f);
  return fmaf(2.f * r, p, fmaxf(x, 0.f));
}

// Tokens of sequence b, or -1 (and the status bit) where its length lies outside [0, N].
__device__ __forceinline__ int64_t sequence_length(const int64_t* lens, int64_t b, int64_t N, unsigned* status, bool report) {
  if (!lens) return N;
  const int64_t n = lens[b];
  if (n >= 0 && n <= N) return n;
  if (report) atomicOr(status, kStatusBadIndex);
  return -1;
}

}  // namespace la
