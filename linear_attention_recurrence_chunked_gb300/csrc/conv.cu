// conv.cu -- short causal depthwise convolution with optional SiLU, the layer in front of a gated-delta-
// rule or selective-scan recurrence (NoteBank App. C.6, Eq. (20) counts its 4-tap cache; the short
// convolutions of BASED):
//   y_t[c] = act(bias[c] + sum_{i<W} w[c,i] x_{t-W+1+i}[c]),   state = the last W - 1 inputs.
// Each input is read once and each output written once; 2 W operations per 4 bytes of bf16 leave the
// kernel to memory bandwidth.  A thread owns one 16-byte vector of channels over a run of tokens and
// keeps the last W - 1 of them in registers, so a run re-reads W - 1 rows (from L2) and nothing else.
#include <algorithm>

#include "layers.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 8;  // token rows a thread has in flight

template <typename TW, int V, int W>
__device__ __forceinline__ void load_taps(const void* w, const void* bias, int64_t c0, int valid, float (&wt)[W][V],
                                          float (&bs)[V]) {
  // the V channels' taps are V * W consecutive elements; whole vectors of them but for three bf16 taps
  // of four fp32 channels
  const TW* p = reinterpret_cast<const TW*>(w) + c0 * W;
  float flat[V * W];
  if (V * W % kVec<TW> == 0 && valid == V) {
#pragma unroll
    for (int i = 0; i + kVec<TW> <= V * W; i += kVec<TW>) {
      float x[kVec<TW>];
      unpack_vec(*reinterpret_cast<const uint4*>(p + i), x);
#pragma unroll
      for (int j = 0; j < kVec<TW>; ++j) flat[i + j] = x[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V * W; ++i) flat[i] = i < valid * W ? to_f(p[i]) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) wt[i][j] = flat[j * W + i];
  const TW* bp = reinterpret_cast<const TW*>(bias) + c0;
#pragma unroll
  for (int j = 0; j < V; ++j) bs[j] = bias != nullptr && j < valid ? to_f(bp[j]) : 0.f;
}

template <typename TIn, typename TOut, typename TW, int W, bool FULL>
__global__ void __launch_bounds__(kThreads, 2)
conv_prefill_kernel(const ConvLaunch a, int64_t vecs, int64_t runs, int run_len) {
  constexpr int V = kVec<TIn>;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t vec = id % vecs, r = id / vecs, b = r / runs, run = r - b * runs;
  if (b >= a.B) return;
  const int64_t n = sequence_length(a.lens, b, a.N, a.status, vec == 0 && run == 0);
  const int64_t t0 = run * run_len;
  if (n < 0 || (t0 >= n && run > 0)) return;
  const int64_t c0 = vec * V, t1 = min(t0 + run_len, n);
  const int valid = FULL ? V : (int)min((int64_t)V, a.C - c0);  // FULL: C is a multiple of V
  const bool state_vec = FULL;
  const TIn* x = reinterpret_cast<const TIn*>(a.x) + b * a.x_sb + c0;
  const TIn* s_in = a.state_in ? reinterpret_cast<const TIn*>(a.state_in) + b * (W - 1) * a.C + c0 : nullptr;

  float wt[W][V], bs[V], hist[W - 1][V];
  load_taps<TW, V, W>(a.w, a.bias, c0, valid, wt, bs);
  // row t of the sequence with the state in front of it (t >= 1 - W)
  auto row = [&](int64_t t) -> uint4 {
    if (t >= 0) return load_raw(x + t * a.x_st, valid, true);
    return s_in ? load_raw(s_in + (W - 1 + t) * a.C, valid, state_vec) : make_uint4(0u, 0u, 0u, 0u);
  };
#pragma unroll
  for (int i = 0; i < W - 1; ++i) unpack_vec(row(t0 + i - (W - 1)), hist[i]);

  TOut* y = reinterpret_cast<TOut*>(a.y) + b * a.y_sb + c0;
  for (int64_t t = t0; t < t1; t += kInFlight) {
    uint4 raw[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (t + u < t1) raw[u] = load_raw(x + (t + u) * a.x_st, valid, true);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      if (t + u < t1) {
        float cur[V], o[V];
        unpack_vec(raw[u], cur);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float acc = bs[j];
#pragma unroll
          for (int i = 0; i < W - 1; ++i) acc = fmaf(wt[i][j], hist[i][j], acc);
          acc = fmaf(wt[W - 1][j], cur[j], acc);
          o[j] = a.silu ? silu(acc) : acc;
#pragma unroll
          for (int i = 0; i + 1 < W - 1; ++i) hist[i][j] = hist[i + 1][j];
          hist[W - 2][j] = cur[j];
        }
        store_floats(y + (t + u) * a.y_st, o, valid, true);
      }
    }
  }
  if (run == 0) {
    // Only this thread reads and writes these channels' state, and its history came from it above.  With
    // fewer than W - 1 tokens row i takes row n + i of the old state: never one that is already replaced.
    TIn* s_out = reinterpret_cast<TIn*>(a.state_out) + b * (W - 1) * a.C + c0;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) store_raw(s_out + i * a.C, row(n - (W - 1) + i), valid, state_vec);
  }
}

template <typename TIn, typename TOut, typename TW, int W>
__global__ void __launch_bounds__(kThreads)
conv_decode_kernel(const ConvLaunch a, int64_t vecs) {
  constexpr int V = kVec<TIn>;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t vec = id % vecs, s = id / vecs;
  grid_dependents_trigger();
  if (s >= a.B) return;
  grid_dependency_wait();  // the state and this step's input are in memory
  const int64_t c0 = vec * V;
  const int valid = (int)min((int64_t)V, a.C - c0);
  const bool state_vec = a.C % V == 0;
  const TIn* s_in = reinterpret_cast<const TIn*>(a.state_in) + s * (W - 1) * a.C + c0;
  TIn* s_out = reinterpret_cast<TIn*>(a.state_out) + s * (W - 1) * a.C + c0;
  uint4 raw[W];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) raw[i] = load_raw(s_in + i * a.C, valid, state_vec);
  raw[W - 1] = load_raw(reinterpret_cast<const TIn*>(a.x) + s * a.x_sb + c0, valid, true);
  float wt[W][V], o[V];
  load_taps<TW, V, W>(a.w, a.bias, c0, valid, wt, o);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    float cur[V];
    unpack_vec(raw[i], cur);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = fmaf(wt[i][j], cur[j], o[j]);
  }
  if (a.silu) {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = silu(o[j]);
  }
  store_floats(reinterpret_cast<TOut*>(a.y) + s * a.y_sb + c0, o, valid, true);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) store_raw(s_out + i * a.C, raw[i + 1], valid, state_vec);
}

template <typename TIn, typename TOut, typename TW, int W>
cudaError_t launch_typed(const ConvLaunch& a, bool decode, cudaStream_t stream) {
  const int64_t vecs = (a.C + kVec<TIn> - 1) / kVec<TIn>;
  if (decode) {
    const int64_t grid = (a.B * vecs + kThreads - 1) / kThreads;
    return launch_dependent(conv_decode_kernel<TIn, TOut, TW, W>, dim3((unsigned)grid), dim3(kThreads), 0, stream, a, vecs);
  }
  // a run of 32 tokens re-reads 3 rows of 35; shorter runs where the problem would leave SMs idle
  int run_len = 32;
  while (run_len > 4 && a.B * vecs * ((a.N + run_len - 1) / run_len) < 152 * 1024) run_len /= 2;
  const int64_t runs = std::max<int64_t>(1, (a.N + run_len - 1) / run_len);
  const int64_t grid = (a.B * vecs * runs + kThreads - 1) / kThreads;
  if (a.C % kVec<TIn> == 0)
    conv_prefill_kernel<TIn, TOut, TW, W, true><<<(unsigned)grid, kThreads, 0, stream>>>(a, vecs, runs, run_len);
  else
    conv_prefill_kernel<TIn, TOut, TW, W, false><<<(unsigned)grid, kThreads, 0, stream>>>(a, vecs, runs, run_len);
  return cudaGetLastError();
}

template <typename TIn, typename TOut, typename TW>
cudaError_t launch_taps(const ConvLaunch& a, bool decode, cudaStream_t stream) {
  switch (a.W) {
    case 2: return launch_typed<TIn, TOut, TW, 2>(a, decode, stream);
    case 3: return launch_typed<TIn, TOut, TW, 3>(a, decode, stream);
    default: return launch_typed<TIn, TOut, TW, 4>(a, decode, stream);
  }
}

template <typename TIn, typename TOut>
cudaError_t launch_weights(const ConvLaunch& a, bool decode, cudaStream_t stream) {
  return a.w_bf16 ? launch_taps<TIn, TOut, __nv_bfloat16>(a, decode, stream) : launch_taps<TIn, TOut, float>(a, decode, stream);
}

cudaError_t launch_any(const ConvLaunch& a, bool decode, cudaStream_t stream) {
  if (a.in_bf16 && a.out_bf16) return launch_weights<__nv_bfloat16, __nv_bfloat16>(a, decode, stream);
  if (a.in_bf16) return launch_weights<__nv_bfloat16, float>(a, decode, stream);
  if (a.out_bf16) return launch_weights<float, __nv_bfloat16>(a, decode, stream);
  return launch_weights<float, float>(a, decode, stream);
}

}  // namespace

cudaError_t launch_conv_prefill(const ConvLaunch& a, cudaStream_t stream) { return launch_any(a, false, stream); }
cudaError_t launch_conv_decode(const ConvLaunch& a, cudaStream_t stream) { return launch_any(a, true, stream); }

}  // namespace la
