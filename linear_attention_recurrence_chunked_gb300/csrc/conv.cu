// conv.cu -- short causal depthwise convolution with optional SiLU, the layer in front of a gated-delta-
// rule or selective-scan recurrence (NoteBank App. C.6, Eq. (20) counts its 4-tap cache; the short
// convolutions of BASED):
//   y_t[c] = act(bias[c] + sum_{i<W} w[c,i] x_{t-W+1+i}[c]),   state = the last W - 1 inputs.
// Each input is read once and each output written once; 2 W operations per 4 bytes of bf16 leave the
// kernel to memory bandwidth.  A thread owns four channels over a run of tokens and keeps the last W - 1 of
// them in registers, so a run re-reads W - 1 rows (from L2) and nothing else.  4 x 16384 x 2048 bf16, 4 taps with SiLU:
// 100 us, 5.3 TB/s, 80 % of the measured copy rate (211 us a row at a time).
#include <algorithm>

#include "layers.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kV = 4;         // channels per thread
constexpr int kInFlight = 8;  // token rows a thread has in flight

template <typename TW, int W>
__device__ __forceinline__ void load_taps(const void* w, const void* bias, int64_t c0, int valid, float (&wt)[W][kV],
                                          float (&bs)[kV]) {
  // the four channels' taps are 4 W consecutive elements
  const TW* p = reinterpret_cast<const TW*>(w) + c0 * W;
  float flat[kV * W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    float x[4];
    Raw4<TW> r;
    if (valid == kV) r.load(p + 4 * i);
    else r.load(p + 4 * i, valid * W - 4 * i);
    r.unpack(x);
#pragma unroll
    for (int j = 0; j < 4; ++j) flat[4 * i + j] = x[j];
  }
#pragma unroll
  for (int j = 0; j < kV; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) wt[i][j] = flat[j * W + i];
  const TW* bp = reinterpret_cast<const TW*>(bias) + c0;
#pragma unroll
  for (int j = 0; j < kV; ++j) bs[j] = bias != nullptr && j < valid ? to_f(bp[j]) : 0.f;
}

// FULL: C is a multiple of four, so every thread's channels are whole vectors
template <bool FULL, typename T>
__device__ __forceinline__ Raw4<T> load_row(const T* p, int valid) {
  Raw4<T> r;
  if (FULL) r.load(p);
  else r.load(p, valid);
  return r;
}

template <typename TIn, typename TOut, typename TW, int W, bool FULL>
__global__ void __launch_bounds__(kThreads, FULL ? 3 : 1)
conv_prefill_kernel(const ConvLaunch a, int64_t vecs, int64_t runs, int run_len) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t vec = id % vecs, r = id / vecs, b = r / runs, run = r - b * runs;
  if (b >= a.B) return;
  const int64_t n = sequence_length(a.lens, b, a.N, a.status, vec == 0 && run == 0);
  const int64_t t0 = run * run_len;
  if (n < 0 || (t0 >= n && run > 0)) return;
  const int64_t c0 = vec * kV;
  const int count = (int)(min(t0 + run_len, n) - t0);
  const int valid = FULL ? kV : (int)min((int64_t)kV, a.C - c0);
  const TIn* x = reinterpret_cast<const TIn*>(a.x) + b * a.x_sb + c0;
  const TIn* s_in = a.state_in ? reinterpret_cast<const TIn*>(a.state_in) + b * (W - 1) * a.C + c0 : nullptr;

  float wt[W][kV], bs[kV], hist[W - 1][kV];
  load_taps<TW, W>(a.w, a.bias, c0, valid, wt, bs);
  // row t of the sequence with the state in front of it (t >= 1 - W)
  auto row = [&](int64_t t) {
    Raw4<TIn> z;
    z.zero();
    if (t >= 0) return load_row<FULL>(x + t * a.x_st, valid);
    return s_in ? load_row<FULL>(s_in + (W - 1 + t) * a.C, valid) : z;
  };
#pragma unroll
  for (int i = 0; i < W - 1; ++i) row(t0 + i - (W - 1)).unpack(hist[i]);

  // pairs of channels from here on
  f32x2 w2[W][2], b2[2], h2[W - 1][2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    b2[p] = pack2(bs[2 * p], bs[2 * p + 1]);
#pragma unroll
    for (int i = 0; i < W; ++i) w2[i][p] = pack2(wt[i][2 * p], wt[i][2 * p + 1]);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) h2[i][p] = pack2(hist[i][2 * p], hist[i][2 * p + 1]);
  }
  auto token = [&](const Raw4<TIn>& raw, TOut* yp) {
    float cur[kV], o[kV];
    raw.unpack(cur);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      f32x2 acc = b2[p];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) acc = fma2(w2[i][p], h2[i][p], acc);
      const f32x2 now = pack2(cur[2 * p], cur[2 * p + 1]);
      acc = fma2(w2[W - 1][p], now, acc);
      unpack2(acc, o[2 * p], o[2 * p + 1]);
      if (a.silu) {
        float e0, e1;
        unpack2(add2(ex2_2(mul2(acc, pack2(-kLog2e, -kLog2e))), pack2(1.f, 1.f)), e0, e1);
        unpack2(mul2(acc, pack2(rcp(e0), rcp(e1))), o[2 * p], o[2 * p + 1]);
      }
#pragma unroll
      for (int i = 0; i + 1 < W - 1; ++i) h2[i][p] = h2[i + 1][p];
      h2[W - 2][p] = now;
    }
    store_floats(yp, o, valid, FULL);
  };
  const TIn* xp = x + t0 * a.x_st;
  TOut* yp = reinterpret_cast<TOut*>(a.y) + b * a.y_sb + c0 + t0 * a.y_st;
  int t = 0;
  for (; t + kInFlight <= count; t += kInFlight) {
    Raw4<TIn> raw[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u, xp += a.x_st) raw[u] = load_row<FULL>(xp, valid);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u, yp += a.y_st) token(raw[u], yp);
  }
  for (; t < count; ++t, xp += a.x_st, yp += a.y_st) token(load_row<FULL>(xp, valid), yp);
  if (run == 0) {
    // Only this thread reads and writes these channels' state, and its history came from it above.  With
    // fewer than W - 1 tokens row i takes row n + i of the old state: never one that is already replaced.
    TIn* s_out = reinterpret_cast<TIn*>(a.state_out) + b * (W - 1) * a.C + c0;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const Raw4<TIn> last = row(n - (W - 1) + i);
      if (FULL) last.store(s_out + i * a.C);
      else last.store(s_out + i * a.C, valid);
    }
  }
}

template <typename TIn, typename TOut, typename TW, int W, bool FULL>
__global__ void __launch_bounds__(kThreads)
conv_decode_kernel(const ConvLaunch a, int64_t vecs) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t vec = id % vecs, s = id / vecs;
  grid_dependents_trigger();
  if (s >= a.B) return;
  grid_dependency_wait();  // the state and this step's input are in memory
  const int64_t c0 = vec * kV;
  const int valid = FULL ? kV : (int)min((int64_t)kV, a.C - c0);
  const TIn* s_in = reinterpret_cast<const TIn*>(a.state_in) + s * (W - 1) * a.C + c0;
  TIn* s_out = reinterpret_cast<TIn*>(a.state_out) + s * (W - 1) * a.C + c0;
  Raw4<TIn> raw[W];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) raw[i] = load_row<FULL>(s_in + i * a.C, valid);
  raw[W - 1] = load_row<FULL>(reinterpret_cast<const TIn*>(a.x) + s * a.x_sb + c0, valid);
  float wt[W][kV], o[kV];
  load_taps<TW, W>(a.w, a.bias, c0, valid, wt, o);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    float cur[kV];
    raw[i].unpack(cur);
#pragma unroll
    for (int j = 0; j < kV; ++j) o[j] = fmaf(wt[i][j], cur[j], o[j]);
  }
  if (a.silu) {
#pragma unroll
    for (int j = 0; j < kV; ++j) o[j] = silu(o[j]);
  }
  store_floats(reinterpret_cast<TOut*>(a.y) + s * a.y_sb + c0, o, valid, FULL);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    if (FULL) raw[i + 1].store(s_out + i * a.C);
    else raw[i + 1].store(s_out + i * a.C, valid);
  }
}

template <typename TIn, typename TOut, typename TW, int W>
cudaError_t launch_typed(const ConvLaunch& a, bool decode, cudaStream_t stream) {
  const int64_t vecs = (a.C + kV - 1) / kV;
  const bool full = a.C % kV == 0;
  if (decode) {
    const dim3 grid((unsigned)((a.B * vecs + kThreads - 1) / kThreads));
    return full ? launch_dependent(conv_decode_kernel<TIn, TOut, TW, W, true>, grid, dim3(kThreads), 0, stream, a, vecs)
                : launch_dependent(conv_decode_kernel<TIn, TOut, TW, W, false>, grid, dim3(kThreads), 0, stream, a, vecs);
  }
  // a run of 32 tokens re-reads 3 rows of 35; shorter runs where the problem would leave SMs idle
  int run_len = 32;
  while (run_len > 4 && a.B * vecs * ((a.N + run_len - 1) / run_len) < 152 * 1024) run_len /= 2;
  const int64_t runs = std::max<int64_t>(1, (a.N + run_len - 1) / run_len);
  const unsigned grid = (unsigned)((a.B * vecs * runs + kThreads - 1) / kThreads);
  if (full) conv_prefill_kernel<TIn, TOut, TW, W, true><<<grid, kThreads, 0, stream>>>(a, vecs, runs, run_len);
  else conv_prefill_kernel<TIn, TOut, TW, W, false><<<grid, kThreads, 0, stream>>>(a, vecs, runs, run_len);
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
