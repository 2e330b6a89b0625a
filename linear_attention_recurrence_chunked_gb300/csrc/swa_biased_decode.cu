// swa_biased_decode.cu -- one decode step of window attention with grouped heads, capped scores and a
// distance bias, over the rings of swa_decode.cu (token p in slot p % window):
//   s_j = cap tanh(scale q.k_j / cap) - slope (pos - j),   o = sum_j softmax_j(s_j) v_j.
// The step reads each ring once and little else, so memory bounds it.  One CTA per (sequence, key head),
// one warp per query head of the group; the group's warps share the ring's rows through L1.  The new
// token is used from the arguments, not from its slot, which warp 0 writes meanwhile.
#include "layers.cuh"

namespace la {
namespace {

constexpr int kMaxWindow = 256, kMaxD = 128, kSlots = kMaxWindow / 32;

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(512)
swa_biased_decode_kernel(const SwaBiasedDecodeLaunch a) {
  __shared__ float qs[16][kMaxD];
  __shared__ float ps[16][kMaxWindow];
  const SwaDecodeLaunch& c = a.base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = blockDim.x >> 5;
  const int64_t sk = blockIdx.x, s = sk / a.Hkv, hk = sk - s * a.Hkv, h = hk * group + warp;
  grid_dependents_trigger();
  grid_dependency_wait();  // the rings, positions and inputs of this step are in memory
  const int d = c.d, w = c.window;
  const int64_t pos = c.pos[s];
  if (pos < 0) {
    if (threadIdx.x == 0 && hk == 0) atomicOr(c.status, kStatusBadIndex);
    return;
  }
  const int slot_new = (int)(pos % w);
  const int n = pos + 1 < w ? (int)(pos + 1) : w;
  const TIn* q = reinterpret_cast<const TIn*>(c.q) + (s * c.H + h) * d;
  const TIn* k = reinterpret_cast<const TIn*>(c.k) + sk * d;
  const TIn* v = reinterpret_cast<const TIn*>(c.v) + sk * d;
  TIn* kc = reinterpret_cast<TIn*>(c.k_cache) + sk * (int64_t)w * d;
  TIn* vc = reinterpret_cast<TIn*>(c.v_cache) + sk * (int64_t)w * d;
  for (int e = lane; e < d; e += 32) {
    qs[warp][e] = to_f(q[e]) * c.scale;
    if (warp == 0) {
      kc[(int64_t)slot_new * d + e] = k[e];
      vc[(int64_t)slot_new * d + e] = v[e];
    }
  }
  __syncwarp();
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  float sc[kSlots], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int j = lane + 32 * i;
    float x = -INFINITY;
    if (j < n) {
      const TIn* kr = j == slot_new ? k : kc + (int64_t)j * d;
      x = 0.f;
      for (int e = 0; e < d; e += 4) x += dot4(*reinterpret_cast<const float4*>(&qs[warp][e]), load4(kr + e));
      if (a.softcap != 0.f) x = a.softcap * tanhf(x / a.softcap);
      const int age = slot_new >= j ? slot_new - j : slot_new - j + w;
      x -= slope * (float)age;
    }
    sc[i] = x;
    m = fmaxf(m, x);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, off));
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int j = lane + 32 * i;
    if (j < n) {
      const float e = __expf(sc[i] - m);
      ps[warp][j] = e;
      l += e;
    }
  }
  l = warp_sum(l);
  __syncwarp();
  const float inv = 1.f / l;
  TOut* out = reinterpret_cast<TOut*>(c.out) + (s * c.H + h) * d;
  for (int e = lane * 4; e < d; e += 128) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < n; ++j) {
      const float4 x = load4((j == slot_new ? v : vc + (int64_t)j * d) + e);
      const float p = ps[warp][j];
      acc.x = fmaf(p, x.x, acc.x);
      acc.y = fmaf(p, x.y, acc.y);
      acc.z = fmaf(p, x.z, acc.z);
      acc.w = fmaf(p, x.w, acc.w);
    }
    const float o[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    store_floats(out + e, o, 4, true);
  }
}

template <typename TIn, typename TOut>
cudaError_t launch_typed(const SwaBiasedDecodeLaunch& a, cudaStream_t stream) {
  const int group = (int)(a.base.H / a.Hkv);
  return launch_dependent(swa_biased_decode_kernel<TIn, TOut>, dim3((unsigned)(a.base.S * a.Hkv)), dim3(32 * group), 0,
                          stream, a);
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
