// heads.cu -- norms of queries and keys for each head with the position rotation in the same pass:
//   x <- w x / sqrt(mean x^2 + eps) (or the sum in the mean's place), then pairs of the first elements turned by their
//   token's angle.
// Every element is read and written once, so memory bounds it.  A warp takes a token's heads, a part of them where there are
// few tokens: eight elements a lane and d / 8 lanes a row, so that the angles of a lane's elements stay in registers from
// head to head.  Sums of squares meet by shuffles, those of four rows at a time.  4 x 16384 tokens of 32 heads x 128 to unit
// length in bf16 take 159 us, the measured copy rate; 3 x 8191 tokens of 36 heads with weights and rotation 78.6 us, 86 % of it.
#include <type_traits>

#include "la.h"
#include "rows.cuh"

namespace la {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Rows of a lane on their way at once, with 24 warps an SM beside them: with rotation 80 us; 2 rows and 32 warps 97, 6 rows and 16
// warps 92.  (Blocks of eight warps, as those were; of four 78.)
constexpr int kRows = 4;

struct Plan {
  int per;  // heads a warp takes, of the queries' and then the keys'
  int64_t blocks;
  Divisor parts, tokens;  // warps for a token; tokens of a sequence
};

int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// As many heads a warp (up to eight times its rows of one load) as leave 32 warps to each of 152 SMs.
Plan plan_of(int64_t B, int64_t H, int64_t Hkv, int64_t N, int d) {
  const int rows = 32 / lanes_of(d);
  Plan p{};
  int64_t parts = 0;
  for (int m = 8 * kRows; m >= 1; m /= 2) {
    p.per = rows * m;
    parts = (H + Hkv + p.per - 1) / p.per;
    if (B * N * parts >= 152 * 32) break;
  }
  p.blocks = (B * N * parts + kWarps - 1) / kWarps;
  p.parts = Divisor(parts);
  p.tokens = Divisor(N);
  return p;
}

template <typename TIn, typename TOut, int LPR, TurnKind kTurn, bool kNorm>
__global__ void __launch_bounds__(kThreads, 6)
qk_norm_rope_kernel(const QkNormRopeLaunch a, const Plan p) {
  constexpr int R = 32 / LPR;
  constexpr bool kWhole = kTurn != kTurnHalves;
  const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
  grid_dependents_trigger();
  grid_dependency_wait();
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), token = p.parts(unit), b = p.tokens(token), n = token - b * p.tokens.d;
  if (b >= a.B) return;  // whole warps
  const int part = (int)(unit - token * p.parts.d);
  const bool on = col * 8 < a.d;
  const int2 at = runs_of<kTurn>(on ? col : 0, a.rot);

  // ---- the token: padding and positions outside the tables are left alone or become zeros
  const int64_t len = sequence_length(a.lens, b, a.N, a.status, lane == 0 && part == 0 && n == 0);
  int64_t row = 0;
  bool alive = n < len;
  if (kTurn != kTurnNone && alive) {
    row = table_row(a.pos ? a.pos[a.pos_each ? token : b] : 0, a.pos && a.pos_each ? 0 : n, a.positions);
    alive = row >= 0;
    if (!alive && lane == 0 && part == 0) atomicOr(a.status, kStatusBadIndex);
  }
  if (!alive && !a.fill) return;
  Turn<kTurn> turn;
  turn.on = false;
  if (kTurn != kTurnNone && alive && on) turn.init(a.cos + row * (a.rot / 2), a.sin + row * (a.rot / 2), a.rot, col);
  const float share = a.norm == LA_NORM_RMS ? 1.f / (float)a.d : 1.f;

#pragma unroll 1
  for (int keys = 0; keys < 2; ++keys) {
    // this warp's heads of the queries, or of the keys
    const int before = keys ? (int)a.H : 0, heads = keys ? (int)a.Hkv : (int)a.H;
    const int h0 = max(part * p.per - before, 0), h1 = min((part + 1) * p.per - before, heads);
    if (h0 >= h1) continue;
    const TIn* x = keys ? a.k.at<const TIn>(b, h0 + sub, n) : a.q.at<const TIn>(b, h0 + sub, n);
    TOut* y = keys ? a.k_out.at<TOut>(b, h0 + sub, n) : a.q_out.at<TOut>(b, h0 + sub, n);
    const int64_t xr = R * (keys ? a.k.step<TIn>() : a.q.step<TIn>()), yr = R * (keys ? a.k_out.step<TOut>() : a.q_out.step<TOut>());
    if (!alive) {
      Raw8<TOut> zero;
      zero.zero();
      for (int h = h0 + sub; h < h1; h += R) {
        if (on) zero.template store<kWhole>(y, at);
        y += yr;
      }
      continue;
    }
    const void* weight = keys ? a.k_weight : a.q_weight;
    f32x2 w[4];
    if (kNorm && weight) {
      if (a.w_bf16) {
        Raw8<__nv_bfloat16> r;
        r.template load<kWhole>(static_cast<const __nv_bfloat16*>(weight), at);
        r.unpack(w);
      } else {
        Raw8<float> r;
        r.template load<kWhole>(static_cast<const float*>(weight), at);
        r.unpack(w);
      }
    }

    int left = on ? h1 - h0 - sub : 0;  // this lane's rows: every R-th while it is positive
#pragma unroll 1
    for (int more = h1 - h0; more > 0; more -= kRows * R, left -= kRows * R) {
      Raw8<TIn> raw[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        raw[i].zero();
        if (left > i * R) raw[i].template load<kWhole>(x, at);
        x += xr;
      }
      float scale[kRows];
      bool beyond = false;  // a row of the warp's
      if constexpr (kNorm) {
        float sum[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          f32x2 v[4];
          raw[i].unpack(v);
          f32x2 t = mul2(v[0], v[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) t = fma2(v[e], v[e], t);
          float lo, hi;
          unpack2(t, lo, hi);
          sum[i] = lo + hi;
        }
#pragma unroll
        for (int off = LPR / 2; off >= 1; off /= 2)
#pragma unroll
          for (int i = 0; i < kRows; ++i) sum[i] += __shfl_xor_sync(kFullMask, sum[i], off);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          sum[i] = fmaf(sum[i], share, a.eps);
          scale[i] = rsqrtf(sum[i]);
          beyond |= !(sum[i] <= 3.402823466e38f);
        }
        beyond = __any_sync(kFullMask, beyond);
        if (beyond) {
          // Beyond fp32 (elements above 1e18): the same of the row's 2^-80th, whose squares stay below 2^96, and of eps's
          // 2^-160th.  The factor keeps its bits: a 2^-80th of it would be a subnormal number for the largest rows, so it is
          // marked by its sign, and the elements take both.  NaN and infinities stay what they are.
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            f32x2 v[4], t = pack2(0.f, 0.f);
            raw[i].unpack(v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[e] = mul2(v[e], pack2(0x1p-80f, 0x1p-80f));
              t = fma2(v[e], v[e], t);
            }
            float lo, hi;
            unpack2(t, lo, hi);
            float small = lo + hi;
#pragma unroll
            for (int off = LPR / 2; off >= 1; off /= 2) small += __shfl_xor_sync(kFullMask, small, off);
            if (!(sum[i] <= 3.402823466e38f)) scale[i] = -rsqrtf(fmaf(small, share, a.eps * 0x1p-80f * 0x1p-80f));
          }
        }
      }
      auto finish = [&](auto marked) {  // marked: rows whose factor has a sign (without a loop of their own 1.6 % slower)
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          if (left <= i * R) break;
          f32x2 v[4];
          raw[i].unpack(v);
          if constexpr (kNorm) {
            const f32x2 both = pack2(scale[i], scale[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], both);
            if (decltype(marked)::value && __float_as_int(scale[i]) < 0) {
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], pack2(-0x1p-80f, -0x1p-80f));
            }
            if (weight) {
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], w[e]);
            }
          }
          if (turn.on) turn.apply(v, turn_rounded);
          Raw8<TOut> out;
          out.pack(v);
          out.template store<kWhole>(y, at);
          y += yr;
        }
      };
      if (beyond) finish(std::true_type{});
      else finish(std::false_type{});
    }
  }
}

template <typename TIn, typename TOut, int LPR, TurnKind kTurn>
cudaError_t launch_turn(const QkNormRopeLaunch& a, cudaStream_t stream) {
  const Plan p = plan_of(a.B, a.H, a.Hkv, a.N, a.d);
  const dim3 grid((unsigned)p.blocks);
  if (a.norm == LA_NORM_NONE) return launch_dependent(qk_norm_rope_kernel<TIn, TOut, LPR, kTurn, false>, grid, kThreads, 0, stream, a, p);
  return launch_dependent(qk_norm_rope_kernel<TIn, TOut, LPR, kTurn, true>, grid, kThreads, 0, stream, a, p);
}
template <typename TIn, typename TOut, int LPR>
cudaError_t launch_row(const QkNormRopeLaunch& a, cudaStream_t stream) {
  return a.rot == 0 ? launch_turn<TIn, TOut, LPR, kTurnNone>(a, stream) : a.interleaved ? launch_turn<TIn, TOut, LPR, kTurnNeighbours>(a, stream)
                                                                        : launch_turn<TIn, TOut, LPR, kTurnHalves>(a, stream);
}
template <typename TIn, typename TOut>
cudaError_t launch(const QkNormRopeLaunch& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.d);
  return lanes == 4 ? launch_row<TIn, TOut, 4>(a, stream) : lanes == 8 ? launch_row<TIn, TOut, 8>(a, stream)
       : lanes == 16 ? launch_row<TIn, TOut, 16>(a, stream) : launch_row<TIn, TOut, 32>(a, stream);
}

}  // namespace

int64_t qk_norm_rope_blocks(int64_t B, int64_t H, int64_t Hkv, int64_t N, int d) { return plan_of(B, H, Hkv, N, d).blocks; }

cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& a, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.in_bf16) return a.out_bf16 ? launch<bf, bf>(a, stream) : launch<bf, float>(a, stream);
  return a.out_bf16 ? launch<float, bf>(a, stream) : launch<float, float>(a, stream);
}

}  // namespace la
