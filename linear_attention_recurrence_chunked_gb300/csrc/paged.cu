// paged.cu -- keys and values of new tokens into a paged cache, the keys rotated on the way, and a cache's tokens back into
// rows.  Both read and write every element once, so memory bounds them.  As in heads.cu a lane has eight elements of a row:
// one 32-bit word of 4-bit codes, whose group of 64 elements is eight neighbouring lanes.
#include "paged.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;  // rows of a lane on their way at once

int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : 16; }

// x c + y s, the exact value rounded to fp32 but for a 2^-20th of an ulp: the products' errors and the sum's are added last.
// (Next to a border of the 4-bit codes an fp32 rounding more could be a whole code.)
__device__ __forceinline__ float turn_exact(float x, float c, float y, float s) {
  const float p = __fmul_rn(x, c), ep = __fmaf_rn(x, c, -p);
  const float q = __fmul_rn(y, s), eq = __fmaf_rn(y, s, -q);
  const float sum = __fadd_rn(p, q), t = __fsub_rn(sum, p);
  const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, t)), __fsub_rn(q, t));
  const float r = __fadd_rn(sum, __fadd_rn(es, __fadd_rn(ep, eq)));
  return fabsf(sum) <= 3.402823466e38f ? r : sum;  // the parts of an infinity are NaN
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight bf16 elements of a lane, whose group is eight neighbouring lanes: their codes and the group's scale (lower half) and offset.
__device__ __forceinline__ void quantise(const float (&v)[8], uint32_t& codes, uint32_t& meta) {
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = min_nan(lo, v[e]);
    hi = max_nan(hi, v[e]);
  }
#pragma unroll
  for (int off = 4; off >= 1; off /= 2) {
    lo = min_nan(lo, __shfl_xor_sync(kFullMask, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(kFullMask, hi, off));
  }
  const float spread = __fsub_rn(hi, lo);
  codes = 0;
  if (!(spread <= 3.402823466e38f)) {
    meta = 0x7fc07fc0u;
    return;
  }
  const __nv_bfloat16 step = __float2bfloat16_rn(__fdiv_rn(spread, 15.f));
  const float scale = __bfloat162float(step);
  meta = (uint32_t)__bfloat16_as_ushort(step) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo)) << 16;
  if (!(scale > 0.f)) return;
  // A product with the reciprocal is within 3e-6 of the quotient, which decides where it could lie on the other side of a border.
  const float inv = __fdiv_rn(1.f, scale);
  const bool tiny = !(inv <= 3.402823466e38f);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __fsub_rn(v[e], lo);
    const float y = x * inv;
    float r = rintf(y);
    if (tiny || fabsf(y - r) > 0.4999f) r = rintf(__fdiv_rn(x, scale));
    codes |= (uint32_t)(int)fminf(r, 15.f) << (4 * e);
  }
}

// A warp stores a token's keys or its values, `per` heads of them.
template <typename T, bool kFour, int LPR>
__global__ void __launch_bounds__(kThreads)
paged_append_kernel(const PagedAppendLaunch a, const int per, const int64_t parts) {
  constexpr int R = 32 / LPR;
  const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
  grid_dependents_trigger();
  grid_dependency_wait();
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t token = unit / (2 * parts), b = token / a.N, n = token - b * a.N;
  if (b >= a.B) return;  // whole warps
  const int64_t part = unit - token * 2 * parts;
  const bool values = part >= parts;
  const bool report = lane == 0 && part == 0;
  if (n >= sequence_length(a.lens, b, a.N, a.c.status, report && n == 0)) return;
  const int64_t p = table_row(a.seen[b], n, a.c.width * a.c.page);
  const int page = p < 0 || (a.rot > 0 && p >= a.positions) ? -1 : table_page(a.c, b, p / a.c.page);
  if (page < 0) {
    if (report) atomicOr(a.c.status, kStatusBadIndex);
    return;
  }
  const int slot = (int)(p % a.c.page), d = a.c.d;
  const bool on = col * 8 < d, turned = a.rot > 0 && !values;
  const int64_t h0 = (values ? part - parts : part) * per, h1 = min(h0 + per, a.c.Hkv);
  const View4& view = values ? a.v : a.k;
  const T* x = static_cast<const T*>(view.ptr) + b * view.sb + n * view.st + col * 8;
  const int64_t size = page_bytes(a.c);
  uint8_t* y = static_cast<uint8_t*>(values ? a.c.v : a.c.k) + page * a.c.Hkv * size;  // this token's page, head 0
  Turn turn;
  turn.on = false;
  if (turned) turn.init(a.cos + p * (a.rot / 2), a.sin + p * (a.rot / 2), a.rot, a.interleaved, lane, col);

  for (int64_t h = h0; h < h1; h += kRows * R) {
    Raw8<T> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      raw[i].zero();
      const int64_t at = h + i * R + sub;
      if (on && at < h1) raw[i].load(x + at * view.sh);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (h + i * R >= h1) break;  // the same for the whole warp
      const int64_t at = h + i * R + sub;
      const bool store = on && at < h1;
      float v[8];
      raw[i].unpack(v);
      if (turned) {
        float u[8];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = v[e ^ 1];
        } else {
          raw[i].from_lane(turn.partner).unpack(u);
        }
        if (turn.on) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (kFour) v[e] = __bfloat162float(__float2bfloat16_rn(turn_exact(v[e], turn.c[e], u[e], turn.s[e])));
            else v[e] = fmaf(v[e], turn.c[e], u[e] * turn.s[e]);
          }
        }
      }
      if constexpr (kFour) {
        uint32_t codes, meta;
        quantise(v, codes, meta);
        const int groups = d / kGroup, g = col / 8, e = col % 8;
        uint8_t* head = y + at * size;
        if (store) {
          reinterpret_cast<uint32_t*>(head + (int64_t)slot * (d / 2))[code_word(g, e, groups)] = codes;
          if (e == 0) reinterpret_cast<uint32_t*>(head + (int64_t)a.c.page * (d / 2))[slot * groups + g] = meta;
        }
      } else if (store) {
        T* row = reinterpret_cast<T*>(y + at * size) + (int64_t)slot * d + col * 8;
        if (turned) store_floats(row, v, 8, true);
        else raw[i].store(row);  // as they are, whatever they hold
      }
    }
  }
}

// A warp reads 16 tokens of one head, keys or values.
template <typename T, typename TOut, bool kFour, int LPR>
__global__ void __launch_bounds__(kThreads)
paged_read_kernel(const PagedReadLaunch a, const int64_t tiles) {
  constexpr int R = 32 / LPR;
  const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
  grid_dependents_trigger();
  grid_dependency_wait();
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  int64_t rest = unit / tiles;
  const int64_t n0 = (unit - rest * tiles) * 16;
  const bool values = rest & 1;
  rest >>= 1;
  const int64_t b = rest / a.c.Hkv, h = rest - b * a.c.Hkv;
  if (b >= a.B) return;  // whole warps
  const int d = a.c.d;
  const bool on = col * 8 < d, report = lane == 0 && h == 0 && !values;
  const int64_t len = sequence_length(a.lens, b, a.N, a.c.status, report && n0 == 0);
  int64_t have = min(len, n0 + 16);  // tokens below are in the cache
  int page = -1;
  if (n0 < have) {
    page = n0 < a.c.width * a.c.page ? table_page(a.c, b, n0 / a.c.page) : -1;
    if (page < 0) {
      if (report) atomicOr(a.c.status, kStatusBadIndex);
      have = n0;
    }
  }
  const int64_t end = min(n0 + 16, a.N), size = page_bytes(a.c);
  const int slot0 = (int)(n0 % a.c.page);
  const uint8_t* x = static_cast<const uint8_t*>(values ? a.c.v : a.c.k) + (page * a.c.Hkv + h) * size;
  TOut* y = static_cast<TOut*>(values ? a.v : a.k) + b * (values ? a.v_sb : a.k_sb) + h * (values ? a.v_sh : a.k_sh) + col * 8;
  const int64_t yt = values ? a.v_st : a.k_st;

#pragma unroll
  for (int i0 = 0; i0 < 16 / R; i0 += kRows) {
    Raw8<T> raw[kRows];
    uint32_t codes[kRows], meta[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = (i0 + i) * R + sub;
      if (!on || n0 + r >= have) continue;
      if constexpr (kFour) {
        const int groups = d / kGroup, g = col / 8, e = col % 8;
        codes[i] = reinterpret_cast<const uint32_t*>(x + (int64_t)(slot0 + r) * (d / 2))[code_word(g, e, groups)];
        meta[i] = reinterpret_cast<const uint32_t*>(x + (int64_t)a.c.page * (d / 2))[(slot0 + r) * groups + g];
      } else {
        raw[i].load(reinterpret_cast<const T*>(x) + (int64_t)(slot0 + r) * d + col * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t n = n0 + (i0 + i) * R + sub;
      if (!on || n >= end) continue;
      float v[8];
      if (n >= have) {
        if (!a.fill) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      } else if constexpr (kFour) {
        const float scale = __uint_as_float(meta[i] << 16), offset = __uint_as_float(meta[i] & 0xffff0000u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf((float)(codes[i] >> (4 * e) & 15u), scale, offset);
      } else {
        raw[i].unpack(v);
      }
      store_floats(y + n * yt, v, 8, true);
    }
  }
}

template <typename T, bool kFour, int LPR>
cudaError_t append(const PagedAppendLaunch& a, cudaStream_t stream) {
  constexpr int R = 32 / LPR;
  int per = R;
  int64_t parts = 0;
  for (int m = kRows; m >= 1; m /= 2) {  // as many heads a warp as leave 32 warps to each of 152 SMs
    per = R * m;
    parts = (a.c.Hkv + per - 1) / per;
    if (2 * a.B * a.N * parts >= 152 * 32) break;
  }
  const int64_t blocks = (2 * a.B * a.N * parts + kWarps - 1) / kWarps;
  return launch_dependent(paged_append_kernel<T, kFour, LPR>, dim3((unsigned)blocks), kThreads, 0, stream, a, per, parts);
}

template <typename T, typename TOut, bool kFour, int LPR>
cudaError_t read(const PagedReadLaunch& a, cudaStream_t stream) {
  const int64_t tiles = (a.N + 15) / 16, blocks = (2 * a.B * a.c.Hkv * tiles + kWarps - 1) / kWarps;
  return launch_dependent(paged_read_kernel<T, TOut, kFour, LPR>, dim3((unsigned)blocks), kThreads, 0, stream, a, tiles);
}

template <typename T, typename TOut>
cudaError_t read_rows(const PagedReadLaunch& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.c.d);
  return lanes == 4 ? read<T, TOut, false, 4>(a, stream) : lanes == 8 ? read<T, TOut, false, 8>(a, stream) : read<T, TOut, false, 16>(a, stream);
}

template <typename T>
cudaError_t append_rows(const PagedAppendLaunch& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.c.d);
  return lanes == 4 ? append<T, false, 4>(a, stream) : lanes == 8 ? append<T, false, 8>(a, stream) : append<T, false, 16>(a, stream);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.c.four) return a.c.d == 64 ? append<bf, true, 8>(a, stream) : append<bf, true, 16>(a, stream);
  return a.c.bf16 ? append_rows<bf>(a, stream) : append_rows<float>(a, stream);
}

cudaError_t launch_paged_read(const PagedReadLaunch& a, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.c.four && a.c.d == 64) return a.out_bf16 ? read<bf, bf, true, 8>(a, stream) : read<bf, float, true, 8>(a, stream);
  if (a.c.four) return a.out_bf16 ? read<bf, bf, true, 16>(a, stream) : read<bf, float, true, 16>(a, stream);
  if (a.c.bf16) return a.out_bf16 ? read_rows<bf, bf>(a, stream) : read_rows<bf, float>(a, stream);
  return a.out_bf16 ? read_rows<float, bf>(a, stream) : read_rows<float, float>(a, stream);
}

}  // namespace la
