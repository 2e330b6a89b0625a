// paged_decode.cu -- attention of one token of each sequence over a paged cache:
//   s_j = cap tanh(scale q.k_j / cap) - slope (n - 1 - j),   o = sum_j softmax_j(s_j) v_j,   max(0, n - window) <= j < n.
// This file: the join of a split sequence's parts, the choice of the split, and the kernel of fp32 pages, on the CUDA cores
// (64 sequences of up to 4096 tokens: 8 heads of their own at d = 64 120 us, 83 % of the copy rate; at d = 128 32 heads over 4
// 280 us, 35 %, and 64 over 4, whose pages are read twice, 527 us, 19 %).
//
// A warp takes tiles of 32 tokens of its block's part in turn.  It scores them for a few query heads of the group, four
// elements a lane and d / 4 lanes a row, takes their softmax a token a lane with the running maximum and sum of its
// tokens so far, and adds up its value rows, the next few rows always on their way; warps do not wait for one another before the end, where their sums meet in
// shared memory.
#include <algorithm>

#include "paged_decode.cuh"

namespace la {
namespace {

constexpr int kWarps = 4;
constexpr int kTokens = 32;  // of a warp's tile: two of 16
constexpr int kLoads = 4;    // row loads in flight
constexpr int kMaxD = 128;

// LPR lanes a row, HG query heads a pass
template <typename TOut, int LPR, int HG>
__global__ void __launch_bounds__(32 * kWarps)
paged_decode_f32_kernel(const PagedDecodeLaunch a, const int passes) {
  constexpr int R = 32 / LPR, kBatch = kLoads * R, kBatches = kTokens / kBatch, NV = kLoads * HG;
  __shared__ float s_p[kWarps][kTokens][HG];  // scores, then weights
  __shared__ float s_o[kWarps][HG][kMaxD];
  __shared__ float s_m[kWarps][HG], s_l[kWarps][HG];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependents_trigger();
  grid_dependency_wait();
  const int part = (int)(blockIdx.x % a.splits);
  int64_t rest = blockIdx.x / a.splits;
  const int pass = (int)(rest % passes);
  rest /= passes;
  const int64_t s = rest / a.c.Hkv, hk = rest - s * a.c.Hkv;
  const int d = a.c.d, group = (int)(a.H / a.c.Hkv), heads = min(HG, group - pass * HG);
  const int64_t h0 = hk * group + pass * HG;
  const SeenTokens t = seen_tokens(a, s);
  const bool report = part == 0 && pass == 0 && hk == 0 && threadIdx.x == 0;
  if (t.hi < 0) {
    if (report) atomicOr(a.c.status, kStatusBadIndex);
    return;
  }
  if (part >= max(t.parts, 1)) return;
  const int first = (t.lo / kTile + part * t.tiles) * kTile, last = min(t.hi, first + t.tiles * kTile);  // this part's tokens
  const int lane_col = lane % LPR * 4, sub = lane / LPR;
  const bool on = lane_col < d;
  const int col = on ? lane_col : 0;

  float q[HG][4], o[HG][4], m[HG], l[HG];
#pragma unroll
  for (int g = 0; g < HG; ++g) {
    Raw4<float> r;
    r.zero();
    if (on && g < heads) r.load(static_cast<const float*>(a.q.ptr) + s * a.q.sb + (h0 + g) * a.q.sh + col);
    r.unpack(q[g]);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[g][e] = 0.f;
    m[g] = -INFINITY;
    l[g] = 0.f;
  }

  // A tile's place: its tokens' two pages; tokens of a page that is not there are not seen.
  struct Tile { int t0, page[2], slot[2]; };
  auto lookup = [&](int t0) {
    Tile n{t0, {-1, -1}, {0, 0}};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = t0 + i * kTile;
      if (at >= last) continue;
      n.page[i] = table_page(a.c, s, at / a.c.page);
      n.slot[i] = at % a.c.page;
      if (n.page[i] < 0 && hk == 0 && pass == 0 && lane == 0) atomicOr(a.c.status, kStatusBadIndex);
    }
    return n;
  };
  auto seen = [&](const Tile& n, int r) { return n.t0 + r >= t.lo && n.t0 + r < last && (r < kTile ? n.page[0] : n.page[1]) >= 0; };
  // batch bt of a tile: its keys, then its values; zeros where nothing is seen
  auto fetch = [&](const Tile& n, int bt, Raw4<float> (&raw)[kLoads]) {
    const float* pool = static_cast<const float*>(bt < kBatches ? a.c.k : a.c.v) + col;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = bt % kBatches * kBatch + i * R + sub;
      raw[i].zero();
      if (on && seen(n, r)) {
        const int64_t at = ((r < kTile ? n.page[0] : n.page[1]) * a.c.Hkv + hk) * a.c.page + (r < kTile ? n.slot[0] + r : n.slot[1] + r - kTile);
        raw[i].load(pool + at * d);
      }
    }
  };
  constexpr int kStep = kWarps * kTokens;
  Tile now = lookup(first + warp * kTokens), next = lookup(first + warp * kTokens + kStep);
  Raw4<float> raw[kLoads], ahead[kLoads];
  fetch(now, 0, ahead);
#pragma unroll 1
  for (; now.t0 < last; now = next, next = lookup(now.t0 + kStep)) {
    // ---- scores
#pragma unroll
    for (int bt = 0; bt < kBatches; ++bt) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) raw[i] = ahead[i];
      fetch(now, bt + 1, ahead);  // the first values behind the last keys
      float sum[NV];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float k[4];
        raw[i].unpack(k);
#pragma unroll
        for (int g = 0; g < HG; ++g) sum[i * HG + g] = fmaf(q[g][3], k[3], fmaf(q[g][2], k[2], fmaf(q[g][1], k[1], q[g][0] * k[0])));
      }
      // sums over the row's lanes: halve the values while there are lanes to share them with
      int at = 0, left = NV;
#pragma unroll
      for (int off = LPR / 2; off >= 1; off /= 2) {
        if (left > 1) {
          const int half = left / 2;
          const bool up = (lane & off) != 0;
#pragma unroll
          for (int e = 0; e < NV / 2; ++e) {
            if (e < half) {
              const float send = up ? sum[e] : sum[e + half];
              sum[e] = (up ? sum[e + half] : sum[e]) + __shfl_xor_sync(kFullMask, send, off);
            }
          }
          at += up ? half : 0;
          left = half;
        } else {
          sum[0] += __shfl_xor_sync(kFullMask, sum[0], off);
        }
      }
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (e < left) s_p[warp][bt * kBatch + (at + e) / HG * R + sub][(at + e) % HG] = sum[e];
    }
    __syncwarp();
    // ---- softmax with what came before, a token a lane
    const bool mine = seen(now, lane);
    float f[HG];
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      float x = s_p[warp][lane][g] * a.scale;
      if (a.softcap != 0.f) x = a.softcap * tanhf(x / a.softcap);  // fp32 throughout: the polynomial of `capped` is off by 10 half steps
      x *= kLog2e;
      if (a.slopes && g < heads) x = fmaf(-a.slopes[h0 + g] * kLog2e, (float)(t.hi - 1 - now.t0 - lane), x);
      if (!mine) x = -INFINITY;
      float top = x;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
      top = fmaxf(top, m[g]);
      const float base = top == -INFINITY ? 0.f : top;
      f[g] = ex2(m[g] - base);
      x = ex2(x - base);
      l[g] = fmaf(l[g], f[g], warp_sum(x));
      m[g] = top;
      s_p[warp][lane][g] = x;
    }
    __syncwarp();
    // ---- values
#pragma unroll
    for (int g = 0; g < HG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[g][e] *= f[g];
#pragma unroll
    for (int bt = 0; bt < kBatches; ++bt) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) raw[i] = ahead[i];
      if (bt + 1 < kBatches) fetch(now, kBatches + bt + 1, ahead);
      else fetch(next, 0, ahead);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float v[4];
        raw[i].unpack(v);
#pragma unroll
        for (int g = 0; g < HG; ++g) {
          const float p = s_p[warp][bt * kBatch + i * R + sub][g];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[g][e] = fmaf(p, v[e], o[g][e]);
        }
      }
    }
    __syncwarp();  // the weights are used up
  }

  // ---- the warps' sums together
#pragma unroll
  for (int g = 0; g < HG; ++g) {
#pragma unroll
    for (int off = LPR; off < 32; off *= 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[g][e] += __shfl_xor_sync(kFullMask, o[g][e], off);
    if (sub == 0 && on) *reinterpret_cast<float4*>(&s_o[warp][g][col]) = make_float4(o[g][0], o[g][1], o[g][2], o[g][3]);
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < heads * d; e += blockDim.x) {
    const int g = e / d, c = e - g * d;
    float top = s_m[0][g];
#pragma unroll
    for (int u = 1; u < kWarps; ++u) top = fmaxf(top, s_m[u][g]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, total = 0.f;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) {
      const float w = ex2(s_m[u][g] - base);
      sum = fmaf(w, s_o[u][g][c], sum);
      total = fmaf(w, s_l[u][g], total);
    }
    if (a.splits > 1) {
      part_values(a, s, h0 + g, part)[c] = sum;
      if (c == 0) *part_sums(a, s, h0 + g, part) = make_float2(top, total);
    } else {
      store1(static_cast<TOut*>(a.out) + s * a.o_sb + (h0 + g) * a.o_sh + c, mean_of(sum, total));
    }
  }
}

constexpr int kJoinWarps = 8;
constexpr int kMostParts = 32 * kJoinWarps;

// The parts of a split sequence together: a block a query head, with a thread for every part.  A warp adds up every kJoinWarps-th
// part (every one, of few), four elements a lane; the first of them are on their way while the parts' weights are made.
template <typename TOut>
__global__ void __launch_bounds__(32 * kJoinWarps)
paged_join_kernel(const PagedDecodeLaunch a) {
  constexpr int kAhead = 8;
  __shared__ float s_o[kJoinWarps][kMaxD], s_w[kMostParts], s_top[kJoinWarps], s_l[kJoinWarps];
  grid_dependents_trigger();
  grid_dependency_wait();
  const int64_t s = blockIdx.x / a.H, h = blockIdx.x - s * a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, d = a.c.d;
  const SeenTokens t = seen_tokens(a, s);
  if (t.hi < 0) return;
  const float2 mine = (int)threadIdx.x < t.parts ? part_sums(a, s, h, 0)[threadIdx.x] : make_float2(-INFINITY, 0.f);
  const bool on = lane * 4 < d;
  const float* values = part_values(a, s, h, 0) + (on ? lane * 4 : 0);
  float4 ahead[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = warp + j * warps;
    ahead[j] = i < t.parts ? *reinterpret_cast<const float4*>(values + (int64_t)i * d) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float top = mine.x;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  for (int u = 0; u < warps; ++u) top = fmaxf(top, s_top[u]);
  const float weight = ex2(mine.x - (top == -INFINITY ? 0.f : top));
  s_w[threadIdx.x] = weight;
  const float l = warp_sum((int)threadIdx.x < t.parts ? weight * mine.y : 0.f);
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](int i, float4 v) {
    const float w = s_w[i];
    o[0] = fmaf(w, v.x, o[0]); o[1] = fmaf(w, v.y, o[1]); o[2] = fmaf(w, v.z, o[2]); o[3] = fmaf(w, v.w, o[3]);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (warp + j * warps < t.parts) add(warp + j * warps, ahead[j]);
#pragma unroll 8
  for (int i = warp + kAhead * warps; i < t.parts; i += warps) add(i, *reinterpret_cast<const float4*>(values + (int64_t)i * d));
  if (on) *reinterpret_cast<float4*>(&s_o[warp][lane * 4]) = make_float4(o[0], o[1], o[2], o[3]);
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float sum = 0.f, total = 0.f;
    for (int u = 0; u < warps; ++u) {
      sum += s_o[u][c];
      total += s_l[u];
    }
    store1(static_cast<TOut*>(a.out) + s * a.o_sb + h * a.o_sh + c, mean_of(sum, total));
  }
}

template <typename TOut, int LPR, int HG>
cudaError_t launch(const PagedDecodeLaunch& a, cudaStream_t stream) {
  const int group = (int)(a.H / a.c.Hkv), passes = (group + HG - 1) / HG;
  return launch_dependent(paged_decode_f32_kernel<TOut, LPR, HG>, dim3((unsigned)(a.S * a.c.Hkv * passes * a.splits)), 32 * kWarps, 0, stream, a, passes);
}
template <typename TOut, int LPR>
cudaError_t by_group(const PagedDecodeLaunch& a, cudaStream_t stream) {
  const int group = (int)(a.H / a.c.Hkv);
  return group == 1 ? launch<TOut, LPR, 1>(a, stream) : group == 2 ? launch<TOut, LPR, 2>(a, stream)
       : group <= 4 ? launch<TOut, LPR, 4>(a, stream) : launch<TOut, LPR, 8>(a, stream);
}
template <typename TOut>
cudaError_t by_width(const PagedDecodeLaunch& a, cudaStream_t stream) {
  return a.c.d <= 32 ? by_group<TOut, 8>(a, stream) : a.c.d <= 64 ? by_group<TOut, 16>(a, stream) : by_group<TOut, 32>(a, stream);
}

}  // namespace

// Blocks of one part each would leave SMs idle, or end one long sequence after the others.  As many parts as make 16 blocks an SM,
// so that sequences of unequal lengths even out (256 sequences of 4 key heads, bf16, 391 us; 396 with 8), and no more than the
// table has twice kPartTokens tokens (64 sequences of up to 300 tokens over 8 key heads: 15 us, 20 with kPartTokens); of few
// sequences 5 blocks an SM, since every part is written and read again (2 sequences of up to 262144 tokens: 129 us with 5, 140 with
// 16), of kPartTokens or more (1 sequence of 2000 tokens: 9.4 us, 11.2 with twice as many).  The lengths are not known here: where
// a table is much wider than its sequences are long, their parts are those of kPartTokens tokens that the device makes (the 64
// sequences behind a table for 8192 tokens: 25 us).
int paged_decode_splits(int64_t S, int64_t Hkv, int64_t tokens) {
  const int64_t blocks = S * Hkv, part = blocks < 152 ? kPartTokens : 2 * kPartTokens, most = (tokens + part - 1) / part;
  const int64_t want = (152 * (blocks < 152 ? 5 : 16) + blocks - 1) / blocks;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), kMostParts));
}

cudaError_t launch_paged_decode(const PagedDecodeLaunch& a, cudaStream_t stream) {
  const cudaError_t e = a.c.bf16 ? launch_paged_decode_mma(a, stream) : a.out_bf16 ? by_width<__nv_bfloat16>(a, stream) : by_width<float>(a, stream);
  if (e != cudaSuccess || a.splits == 1) return e;
  const dim3 grid((unsigned)(a.S * a.H)), block(a.splits <= 8 ? 32 : 32 * kJoinWarps);
  return a.out_bf16 ? launch_dependent(paged_join_kernel<__nv_bfloat16>, grid, block, 0, stream, a)
                    : launch_dependent(paged_join_kernel<float>, grid, block, 0, stream, a);
}

}  // namespace la
