// heads.cu -- norms of queries and keys for each head with the position rotation in the same pass:
//   x <- w x / sqrt(mean x^2 + eps) (or the sum in the mean's place), then pairs of the first elements turned by their
//   token's angle.
// Every element is read and written once, so memory bounds it.  A warp takes a token's query heads or its key heads, a part
// of them where there are few tokens: eight elements a lane and d / 8 lanes a row, so that the weights and the angles of a
// lane's elements stay in registers from head to head.  Sums of squares meet by shuffles, and so do the pairs.
#include "la.h"
#include "rows.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;  // rows of a lane on their way at once

struct Plan {
  int per;                 // heads a warp takes
  int64_t q_parts, parts;  // warps for a token's queries, for its queries and keys
  int64_t blocks;
};

int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// As many heads a warp (up to eight times its rows of one load) as leave 32 warps to each of 152 SMs.
Plan plan_of(int64_t B, int64_t H, int64_t Hkv, int64_t N, int d) {
  const int rows = 32 / lanes_of(d);
  Plan p{};
  for (int m = 8; m >= 1; m /= 2) {
    p.per = rows * m;
    p.q_parts = (H + p.per - 1) / p.per;
    p.parts = p.q_parts + (Hkv + p.per - 1) / p.per;
    if (B * N * p.parts >= 152 * 32) break;
  }
  p.blocks = (B * N * p.parts + kWarps - 1) / kWarps;
  return p;
}

template <typename TIn, typename TOut, int LPR>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(const QkNormRopeLaunch a, const Plan p) {
  constexpr int R = 32 / LPR;
  const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
  grid_dependents_trigger();
  grid_dependency_wait();
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t token = unit / p.parts, b = token / a.N, n = token - b * a.N;
  if (b >= a.B) return;  // whole warps
  const int64_t part = unit - token * p.parts;
  const bool keys = part >= p.q_parts;
  const int64_t h0 = (keys ? part - p.q_parts : part) * p.per, heads = keys ? a.Hkv : a.H, h1 = min(h0 + p.per, heads);
  const bool on = col * 8 < a.d;

  const TIn* x = static_cast<const TIn*>(keys ? a.k.ptr : a.q.ptr) + b * (keys ? a.k.sb : a.q.sb) + n * (keys ? a.k.st : a.q.st) + col * 8;
  TOut* y = static_cast<TOut*>(keys ? a.k_out : a.q_out) + b * (keys ? a.k_sb : a.q_sb) + n * (keys ? a.k_st : a.q_st) + col * 8;
  const int64_t xh = keys ? a.k.sh : a.q.sh, yh = keys ? a.k_sh : a.q_sh;

  // ---- the token: padding and positions outside the tables are left alone or become zeros
  const int64_t len = sequence_length(a.lens, b, a.N, a.status, lane == 0 && part == 0 && n == 0);
  int64_t row = 0;
  bool alive = n < len;
  if (alive && a.rot > 0) {
    row = table_row(a.pos ? a.pos[a.pos_each ? token : b] : 0, a.pos && a.pos_each ? 0 : n, a.positions);
    alive = row >= 0;
    if (!alive && lane == 0 && part == 0) atomicOr(a.status, kStatusBadIndex);
  }
  if (!alive) {
    if (!a.fill) return;
    Raw8<TOut> zero;
    zero.zero();
    for (int64_t h = h0 + sub; h < h1; h += R)
      if (on) zero.store(y + h * yh);
    return;
  }

  float w[8];
  const void* weight = keys ? a.k_weight : a.q_weight;
  if (weight && on) {
    if (a.w_bf16) {
      Raw8<__nv_bfloat16> r;
      r.load(static_cast<const __nv_bfloat16*>(weight) + col * 8);
      r.unpack(w);
    } else {
      Raw8<float> r;
      r.load(static_cast<const float*>(weight) + col * 8);
      r.unpack(w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  }
  Turn turn;
  turn.on = false;
  if (a.rot > 0) turn.init(a.cos + row * (a.rot / 2), a.sin + row * (a.rot / 2), a.rot, a.interleaved, lane, col);
  const float share = a.norm == LA_NORM_RMS ? 1.f / (float)a.d : 1.f;

  for (int64_t h = h0; h < h1; h += kRows * R) {
    Raw8<TIn> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      raw[i].zero();
      const int64_t at = h + i * R + sub;
      if (on && at < h1) raw[i].load(x + at * xh);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (h + i * R >= h1) break;  // the same for the whole warp
      float v[8];
      raw[i].unpack(v);
      float scale = 1.f;
      if (a.norm != LA_NORM_NONE) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
#pragma unroll
        for (int off = LPR / 2; off >= 1; off /= 2) sum += __shfl_xor_sync(kFullMask, sum, off);
        scale = rsqrtf(fmaf(sum, share, a.eps));
        if (__any_sync(kFullMask, !(sum <= 3.402823466e38f))) {
          // Squares beyond fp32 (elements above 1e18): the same of the row's 2^-80th, whose squares stay below 2^96, so
          // that eps no longer counts.  NaN and infinities stay what they are.
          float small = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) small = fmaf(v[e] * 0x1p-80f, v[e] * 0x1p-80f, small);
#pragma unroll
          for (int off = LPR / 2; off >= 1; off /= 2) small += __shfl_xor_sync(kFullMask, small, off);
          if (!(sum <= 3.402823466e38f)) scale = rsqrtf(small * share) * 0x1p-80f;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * scale * w[e];
      if (a.rot > 0) {
        float u[8];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = v[e ^ 1];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = __shfl_sync(kFullMask, v[e], turn.partner);
        }
        if (turn.on) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], turn.c[e], u[e] * turn.s[e]);
        }
      }
      const int64_t at = h + i * R + sub;
      if (on && at < h1) store_floats(y + at * yh, v, 8, true);
    }
  }
}

template <typename TIn, typename TOut>
cudaError_t launch(const QkNormRopeLaunch& a, cudaStream_t stream) {
  const Plan p = plan_of(a.B, a.H, a.Hkv, a.N, a.d);
  const dim3 grid((unsigned)p.blocks);
  switch (lanes_of(a.d)) {
    case 4: return launch_dependent(qk_norm_rope_kernel<TIn, TOut, 4>, grid, kThreads, 0, stream, a, p);
    case 8: return launch_dependent(qk_norm_rope_kernel<TIn, TOut, 8>, grid, kThreads, 0, stream, a, p);
    case 16: return launch_dependent(qk_norm_rope_kernel<TIn, TOut, 16>, grid, kThreads, 0, stream, a, p);
    default: return launch_dependent(qk_norm_rope_kernel<TIn, TOut, 32>, grid, kThreads, 0, stream, a, p);
  }
}

}  // namespace

int64_t qk_norm_rope_blocks(int64_t B, int64_t H, int64_t Hkv, int64_t N, int d) { return plan_of(B, H, Hkv, N, d).blocks; }

cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& a, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.in_bf16) return a.out_bf16 ? launch<bf, bf>(a, stream) : launch<bf, float>(a, stream);
  return a.out_bf16 ? launch<float, bf>(a, stream) : launch<float, float>(a, stream);
}

}  // namespace la
