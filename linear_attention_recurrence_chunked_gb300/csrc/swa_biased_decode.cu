// swa_biased_decode.cu -- one decode step of window attention with grouped heads, capped scores and a
// distance bias, over the rings of swa_decode.cu (token p in slot p % window):
//   s_j = cap tanh(scale q.k_j / cap) - slope (pos - j),   o = sum_j softmax_j(s_j) v_j.
// The step reads each ring once and little else, so memory bounds it.  One CTA per (sequence, key head), one
// warp per 32 slots of the ring: a warp scores its slots for up to four query heads of the group at a time
// (rows read as 16-byte vectors, a row over LPR lanes, four loads a lane in flight; the sums over a row's
// lanes are one reduce-scatter for four rows and four heads), takes the softmax of its own slots and adds up
// its own value rows, so that no warp waits for another before the end, where the warps' parts meet in
// shared memory.  The new token is used from the arguments; the warp of its slot writes it there.
#include "layers.cuh"

namespace la {
namespace {

constexpr int kMaxD = 128;
constexpr int kSlots = 32;     // per warp
constexpr int kMaxWarps = 8;   // window up to 256
constexpr int kHeads = 4;      // query heads per pass
constexpr int kLoads = 4;      // row loads in flight

template <typename T>
__device__ __forceinline__ uint4 load_row(const T* p) { return *reinterpret_cast<const uint4*>(p); }

template <typename TIn, typename TOut, int LPR>
__global__ void __launch_bounds__(32 * kMaxWarps, LPR >= 16 ? 2 : 1)
swa_biased_decode_kernel(const SwaBiasedDecodeLaunch a) {
  constexpr int V = kVec<TIn>, R = 32 / LPR;        // elements of a vector; rows per load of the warp
  constexpr int kBatch = kLoads * R, kBatches = kSlots / kBatch;
  constexpr int NV = kLoads * kHeads;               // partial scores a lane holds per batch
  __shared__ float4 s_p[kMaxWarps][kSlots];         // scores, then weights, of the four heads
  __shared__ float s_o[kMaxWarps][kHeads][kMaxD];
  __shared__ float s_m[kMaxWarps][kHeads], s_l[kMaxWarps][kHeads];
  const SwaDecodeLaunch& c = a.base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t sk = blockIdx.x, s = sk / a.Hkv, hk = sk - s * a.Hkv;
  grid_dependents_trigger();
  grid_dependency_wait();  // the rings, positions and inputs of this step are in memory
  const int d = c.d, w = c.window, group = (int)(c.H / a.Hkv);
  const int64_t pos = c.pos[s];
  if (pos < 0) {  // uniform over the CTA
    if (threadIdx.x == 0 && hk == 0) atomicOr(c.status, kStatusBadIndex);
    return;
  }
  const int slot_new = (int)(pos % w);
  const int n = pos + 1 < w ? (int)(pos + 1) : w;
  const int col = lane % LPR * V, sub = lane / LPR, first = warp * kSlots;
  const bool on = col < d;
  const TIn* kn = reinterpret_cast<const TIn*>(c.k) + sk * d + col;
  const TIn* vn = reinterpret_cast<const TIn*>(c.v) + sk * d + col;
  TIn* kc = reinterpret_cast<TIn*>(c.k_cache) + sk * (int64_t)w * d + col;
  TIn* vc = reinterpret_cast<TIn*>(c.v_cache) + sk * (int64_t)w * d + col;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto row = [&](const TIn* ring, const TIn* fresh, int slot) {
    return on && slot < n ? load_row(slot == slot_new ? fresh : ring + (int64_t)slot * d) : zero;
  };

  for (int g0 = 0; g0 < group; g0 += kHeads) {
    const int64_t h0 = hk * group + g0;
    const int heads = min(kHeads, group - g0);
    float q[kHeads][V];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      unpack_vec(on && g < heads ? load_row(reinterpret_cast<const TIn*>(c.q) + (s * c.H + h0 + g) * d + col) : zero, q[g]);
#pragma unroll
      for (int e = 0; e < V; ++e) q[g][e] *= c.scale;
    }
    // ---- scores of this warp's slots
    uint4 raw[kLoads], ahead[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw[i] = row(kc, kn, first + i * R + sub);
#pragma unroll
    for (int bt = 0; bt < kBatches; ++bt) {
      if (bt + 1 < kBatches) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) ahead[i] = row(kc, kn, first + (bt + 1) * kBatch + i * R + sub);
      } else {  // the first value rows, behind the last keys
#pragma unroll
        for (int i = 0; i < kLoads; ++i) ahead[i] = row(vc, vn, first + i * R + sub);
      }
      float part[NV];  // [load][head]
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float k[V];
        unpack_vec(raw[i], k);
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
          float x = q[g][0] * k[0];
#pragma unroll
          for (int e = 1; e < V; ++e) x = fmaf(q[g][e], k[e], x);
          part[i * kHeads + g] = x;
        }
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
              const float send = up ? part[e] : part[e + half];
              part[e] = (up ? part[e + half] : part[e]) + __shfl_xor_sync(kFullMask, send, off);
            }
          }
          at += up ? half : 0;
          left = half;
        } else {
          part[0] += __shfl_xor_sync(kFullMask, part[0], off);
        }
      }
      // this lane has the sums of values [at, at + left)
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (e < left) {
          const int i = (at + e) / kHeads, g = (at + e) % kHeads;
          reinterpret_cast<float*>(&s_p[warp][bt * kBatch + i * R + sub])[g] = part[e];
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) raw[i] = ahead[i];
    }
    __syncwarp();
    // ---- softmax of this warp's slots, a slot a lane
    {
      const int slot = first + lane;
      const float4 x4 = s_p[warp][lane];
      float x[kHeads] = {x4.x, x4.y, x4.z, x4.w};
      const float age = (float)(slot_new >= slot ? slot_new - slot : slot_new - slot + w);
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        if (a.softcap != 0.f) x[g] = fmaf(-2.f * a.softcap, rcp(1.f + ex2(x[g] * (2.f * kLog2e / a.softcap))), a.softcap);
        if (a.slopes && g < heads) x[g] = fmaf(-a.slopes[h0 + g], age, x[g]);
        if (slot >= n) x[g] = -INFINITY;
        float m = x[g];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, off));
        x[g] = ex2((x[g] - (m == -INFINITY ? 0.f : m)) * kLog2e);
        const float l = warp_sum(x[g]);
        if (lane == 0) {
          s_m[warp][g] = m;
          s_l[warp][g] = l;
        }
      }
      s_p[warp][lane] = make_float4(x[0], x[1], x[2], x[3]);
    }
    __syncwarp();
    // ---- this warp's value rows
    float o[kHeads][V];
#pragma unroll
    for (int g = 0; g < kHeads; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) o[g][e] = 0.f;
#pragma unroll
    for (int bt = 0; bt < kBatches; ++bt) {
      if (bt + 1 < kBatches) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) ahead[i] = row(vc, vn, first + (bt + 1) * kBatch + i * R + sub);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float v[V];
        unpack_vec(raw[i], v);
        const float4 p = s_p[warp][bt * kBatch + i * R + sub];
        const float pg[kHeads] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int g = 0; g < kHeads; ++g)
#pragma unroll
          for (int e = 0; e < V; ++e) o[g][e] = fmaf(pg[g], v[e], o[g][e]);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) raw[i] = ahead[i];
    }
#pragma unroll
    for (int g = 0; g < kHeads; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int off = LPR; off < 32; off *= 2) o[g][e] += __shfl_xor_sync(kFullMask, o[g][e], off);
      }
    if (sub == 0 && on) {
#pragma unroll
      for (int g = 0; g < kHeads; ++g)
#pragma unroll
        for (int e = 0; e < V; e += 4) *reinterpret_cast<float4*>(&s_o[warp][g][col + e]) = make_float4(o[g][e], o[g][e + 1], o[g][e + 2], o[g][e + 3]);
    }
    // the new token into its slot, once and by the warp that read this slot from the arguments
    if (g0 == 0 && slot_new / kSlots == warp && sub == 0 && on) {
      *reinterpret_cast<uint4*>(kc + (int64_t)slot_new * d) = load_row(kn);
      *reinterpret_cast<uint4*>(vc + (int64_t)slot_new * d) = load_row(vn);
    }
    __syncthreads();
    // ---- the warps' parts together
    for (int e = threadIdx.x; e < heads * d; e += blockDim.x) {
      const int g = e / d, x = e - g * d;
      float m = s_m[0][g];
      for (int u = 1; u < warps; ++u) m = fmaxf(m, s_m[u][g]);
      float sum = 0.f, l = 0.f;
      for (int u = 0; u < warps; ++u) {
        const float f = ex2((s_m[u][g] - m) * kLog2e);
        sum = fmaf(f, s_o[u][g][x], sum);
        l = fmaf(f, s_l[u][g], l);
      }
      store1(reinterpret_cast<TOut*>(c.out) + (s * c.H + h0 + g) * d + x, sum / l);
    }
    if (g0 + kHeads < group) __syncthreads();  // the parts are read before the next heads' are written
  }
}

template <typename TIn, typename TOut>
cudaError_t launch_typed(const SwaBiasedDecodeLaunch& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(a.base.S * a.Hkv)), block((unsigned)(32 * ((a.base.window + kSlots - 1) / kSlots)));
  const int vecs = a.base.d / kVec<TIn>;
  if (vecs > 16) {
    if constexpr (sizeof(TIn) == 4) return launch_dependent(swa_biased_decode_kernel<TIn, TOut, 32>, grid, block, 0, stream, a);
  }
  if (vecs > 8) return launch_dependent(swa_biased_decode_kernel<TIn, TOut, 16>, grid, block, 0, stream, a);
  if (vecs > 4) return launch_dependent(swa_biased_decode_kernel<TIn, TOut, 8>, grid, block, 0, stream, a);
  return launch_dependent(swa_biased_decode_kernel<TIn, TOut, 4>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_swa_biased_decode(const SwaBiasedDecodeLaunch& a, cudaStream_t stream) {
  const bool in = a.base.in_bf16, out = a.base.out_bf16;
  if (in && out) return launch_typed<__nv_bfloat16, __nv_bfloat16>(a, stream);
  if (in) return launch_typed<__nv_bfloat16, float>(a, stream);
  if (out) return launch_typed<float, __nv_bfloat16>(a, stream);
  return launch_typed<float, float>(a, stream);
}

}  // namespace la
