// ssm.cu -- selective state space scan and its one-token step:
//   dt = f(delta + delta_bias),  h[c,s] <- exp(dt A[c,s]) h[c,s] + dt u B[g,s],
//   y = (sum_s C[g,s] h[c,s] + D u) silu(z)
// per token, channel c of group g and state s (NoteBank Sec. 2 Eq. (1) with a diagonal A_t).
//
// Per (token, channel, state) the scan needs one exponential and about four fp32 operations, per (token,
// channel) four 2-byte elements of memory: with 16 states the special-function unit (16 results per SM and
// clock) bounds it at three times the memory time.  The decay differs per (channel, state), so no chunk
// form on the tensor cores exists: the tokens are walked in order, with the channels and states in
// parallel.  L lanes share a channel, four states in each lane's registers; B_t, C_t and (dt, dt u) of a
// tile of tokens are staged in shared memory, where each (token, channel)'s softplus is computed once.
// The readout's sum over a channel's lanes is a reduce-scatter over four tokens at a time.
#include <algorithm>

#include "layers.cuh"

namespace la {
namespace {

constexpr int kThreads = 128;
constexpr int kK = 4;  // states per lane

// tokens of a tile: enough to make its loads and barriers rare, few enough for shared memory
constexpr int tile_tokens(int L) { return L >= 8 ? 64 : 32; }

// A log2(e), kept finite so that a step of dt = 0 changes nothing even for the lowest A
__device__ __forceinline__ float log2_rate(float A) {
  const float x = A * kLog2e;
  return x < -3.402823466e38f ? -3.402823466e38f : x;
}

// Time segments: segment g of a sequence takes tokens [g * len, (g + 1) * len).
struct Segments {
  int count;
  int64_t len;
};

// kFull walks a whole sequence; kLocal leaves a segment's state from zero and its
// sum of dt in the workspace; kFinal walks a segment from the state in the workspace.
enum Mode { kFull, kLocal, kFinal };

__host__ __device__ constexpr int lanes_of(int n) { return n <= 4 ? 1 : n <= 8 ? 2 : n <= 16 ? 4 : n <= 32 ? 8 : 16; }

template <int L, typename TIn, typename TOut, int MODE>
__global__ void __launch_bounds__(kThreads)
ssm_scan_kernel(const SsmLaunch a, Segments seg, float* ws_h, float* ws_dt) {
  constexpr int CT = kThreads / L, TT = tile_tokens(L), NP = L * kK;
  constexpr int V = kVec<TIn>, VPR = CT / V > 0 ? CT / V : 1;  // vectors per row of the tile
  constexpr int NVEC = TT * VPR, NVI = (NVEC + kThreads - 1) / kThreads;
  constexpr int NB = TT * NP / kThreads;
  __shared__ __align__(16) float2 s_dt[TT][CT];  // (dt, dt u); the readout replaces dt
  __shared__ __align__(16) float s_B[TT][NP], s_C[MODE == kLocal ? 1 : TT][NP];

  const int tid = threadIdx.x, l = tid % L, ch = tid / L;
  const int64_t Cg = a.C / a.G, tiles = (Cg + CT - 1) / CT;
  const int64_t g = blockIdx.x / tiles, b = blockIdx.y;
  const int64_t c_base = g * Cg + (blockIdx.x % tiles) * CT, c_end = (g + 1) * Cg;
  const int64_t sid = blockIdx.z;
  const int64_t len = sequence_length(a.lens, b, a.N, a.status, blockIdx.x == 0 && sid == 0 && tid == 0);
  if (len < 0) return;  // uniform over the block
  const int64_t t0 = sid * seg.len, t1 = min(t0 + seg.len, len);

  const int64_t c = c_base + ch;
  const bool live = c < c_end;
  float A2[kK], h[kK];
  const int64_t hrow = (b * a.C + c) * a.n;
  const int64_t wrow = ((b * seg.count + sid) * a.C + c) * a.n;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int s = l * kK + k;
    const bool on = live && s < a.n;
    A2[k] = on ? log2_rate(a.A[c * a.n + s]) : 0.f;
    h[k] = 0.f;
    if (MODE == kFull && on && a.h_in) h[k] = a.h_in[hrow + s];
    if (MODE == kFinal && on) h[k] = ws_h[wrow + s];
  }
  float dt_sum = 0.f;

  const TIn* u_p = reinterpret_cast<const TIn*>(a.u) + b * a.u_sb;
  const TIn* d_p = reinterpret_cast<const TIn*>(a.delta) + b * a.d_sb;
  const TIn* z_p = MODE != kLocal && a.z ? reinterpret_cast<const TIn*>(a.z) + b * a.z_sb : nullptr;
  const TIn* B_p = reinterpret_cast<const TIn*>(a.Bm.ptr) + b * a.Bm.sb + g * a.Bm.sh;
  const TIn* C_p = reinterpret_cast<const TIn*>(a.Cm.ptr) + b * a.Cm.sb + g * a.Cm.sh;
  TOut* y_p = reinterpret_cast<TOut*>(a.y) + b * a.y_sb;
  const bool vec = (c_base * sizeof(TIn)) % 16 == 0;             // rows are 16-byte aligned, c_base may not be
  const bool yvec = (c_base * sizeof(TOut)) % (V * sizeof(TOut)) == 0;

  // this thread's vectors of the tile: row i / VPR, channels c_base + V (i % VPR)
  uint4 ru[NVI], rd[NVI], rz[NVI];
  TIn rB[NB], rC[NB];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < NVI; ++i) {
      const int e = tid + i * kThreads, r = e / VPR, v = e % VPR;
      const int64_t cc = c_base + v * V;
      const int valid = (NVEC % kThreads == 0 || e < NVEC) && t + r < t1 ? (int)max((int64_t)0, min((int64_t)min(V, CT), c_end - cc)) : 0;
      if (valid > 0) {
        ru[i] = load_raw(u_p + (t + r) * a.u_st + cc, valid, vec);
        rd[i] = load_raw(d_p + (t + r) * a.d_st + cc, valid, vec);
        if (z_p) rz[i] = load_raw(z_p + (t + r) * a.z_st + cc, valid, vec);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int e = tid + i * kThreads, r = e / NP, s = e % NP;
      const bool on = t + r < t1 && s < a.n;
      rB[i] = on ? B_p[(t + r) * a.Bm.st + s] : TIn(0.f);
      if (MODE != kLocal) rC[i] = on ? C_p[(t + r) * a.Cm.st + s] : TIn(0.f);
    }
  };
  if (t0 < t1) fetch(t0);

  for (int64_t t = t0; t < t1; t += TT) {
    // ---- the tile's step sizes and B, C into shared memory; a token behind the end changes nothing (dt = 0)
    uint4 cu[NVI], cz[NVI];
#pragma unroll
    for (int i = 0; i < NVI; ++i) {
      cu[i] = ru[i];
      cz[i] = rz[i];
      const int e = tid + i * kThreads, r = e / VPR, v = e % VPR;
      if (NVEC % kThreads != 0 && e >= NVEC) continue;
      float fu[V], fd[V];
      unpack_vec(ru[i], fu);
      unpack_vec(rd[i], fd);
#pragma unroll
      for (int j = 0; j < V && j < CT; ++j) {
        const int64_t cc = c_base + v * V + j;
        float dt = 0.f, dtu = 0.f;
        if (t + r < t1 && cc < c_end) {
          const float x = a.delta_bias ? fd[j] + a.delta_bias[cc] : fd[j];
          dt = a.softplus ? softplus(x) : x;
          dtu = dt * fu[j];
        }
        s_dt[r][v * V + j] = make_float2(dt, dtu);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int e = tid + i * kThreads;
      s_B[e / NP][e % NP] = to_f(rB[i]);
      if (MODE != kLocal) s_C[e / NP][e % NP] = to_f(rC[i]);
    }
    __syncthreads();
    if (t + TT < t1) fetch(t + TT);
    // ---- the recurrence, four tokens at a time
#pragma unroll 2
    for (int r = 0; r < TT; r += 4) {
      float acc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 d = s_dt[r + q][ch];
        const float4 Bv = *reinterpret_cast<const float4*>(&s_B[r + q][l * kK]);
        const float Bk[4] = {Bv.x, Bv.y, Bv.z, Bv.w};
#pragma unroll
        for (int k = 0; k < kK; ++k) h[k] = fmaf(ex2(d.x * A2[k]), h[k], d.y * Bk[k]);
        if constexpr (MODE == kLocal) {
          dt_sum += d.x;
        } else {
          const float4 Cv = *reinterpret_cast<const float4*>(&s_C[r + q][l * kK]);
          acc[q] = fmaf(Cv.x, h[0], Cv.y * h[1]) + fmaf(Cv.z, h[2], Cv.w * h[3]);
        }
      }
      if constexpr (MODE != kLocal) {
        // sum over the channel's lanes; the halving steps leave token `q` with its share of the lanes
        if constexpr (L == 1) {
#pragma unroll
          for (int q = 0; q < 4; ++q) s_dt[r + q][ch].x = acc[q];
        } else {
          const bool up1 = (l & (L / 2)) != 0;
          float p0 = up1 ? acc[2] : acc[0], p1 = up1 ? acc[3] : acc[1];
          p0 += __shfl_xor_sync(kFullMask, up1 ? acc[0] : acc[2], L / 2);
          p1 += __shfl_xor_sync(kFullMask, up1 ? acc[1] : acc[3], L / 2);
          if constexpr (L == 2) {
            s_dt[r + 2 * up1][ch].x = p0;
            s_dt[r + 2 * up1 + 1][ch].x = p1;
          } else {
            const bool up2 = (l & (L / 4)) != 0;
            float p = up2 ? p1 : p0;
            p += __shfl_xor_sync(kFullMask, up2 ? p0 : p1, L / 4);
#pragma unroll
            for (int off = L / 8; off >= 1; off >>= 1) p += __shfl_xor_sync(kFullMask, p, off);
            if (l % (L / 4) == 0) s_dt[r + 2 * up1 + up2][ch].x = p;
          }
        }
      }
    }
    __syncthreads();
    // ---- skip term, gate and store; each thread reads the entries it writes for the next tile
    if constexpr (MODE != kLocal) {
#pragma unroll
      for (int i = 0; i < NVI; ++i) {
        const int e = tid + i * kThreads, r = e / VPR, v = e % VPR;
        const int64_t cc = c_base + v * V;
        const int valid = (NVEC % kThreads == 0 || e < NVEC) && t + r < t1 ? (int)max((int64_t)0, min((int64_t)min(V, CT), c_end - cc)) : 0;
        if (valid > 0) {
          float fu[V], fz[V], o[V];
          unpack_vec(cu[i], fu);
          unpack_vec(cz[i], fz);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            o[j] = 0.f;
            if (j < valid) {
              o[j] = s_dt[r][v * V + j].x;
              if (a.D) o[j] = fmaf(a.D[cc + j], fu[j], o[j]);
              if (z_p) o[j] *= silu(fz[j]);
            }
          }
          store_floats(y_p + (t + r) * a.y_st + cc, o, valid, yvec);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int s = l * kK + k;
    if (live && s < a.n) {
      if (MODE == kLocal) ws_h[wrow + s] = h[k];
      else if (MODE == kFull || sid == seg.count - 1) a.h_out[hrow + s] = h[k];
    }
  }
  if (MODE == kLocal && live && l == 0) ws_dt[(b * seg.count + sid) * a.C + c] = dt_sum;
}

// The state that enters each segment, in place of the segment's local state: over a segment a state
// decays by exp(A * sum of dt).
__global__ void __launch_bounds__(256)
ssm_combine_kernel(const SsmLaunch a, Segments seg, float* ws_h, const float* ws_dt) {
  const int64_t per = a.C * a.n;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= a.B * per) return;
  const int64_t b = id / per, e = id - b * per, c = e / a.n;
  if (sequence_length(a.lens, b, a.N, a.status, false) < 0) return;
  const float A2 = log2_rate(a.A[e]);
  float h = a.h_in ? a.h_in[id] : 0.f;
  float* p = ws_h + b * seg.count * per + e;
  const float* d = ws_dt + b * seg.count * a.C + c;
  for (int g = 0; g + 1 < seg.count; ++g) {
    const float local = p[g * per];
    p[g * per] = h;
    h = fmaf(ex2(A2 * d[(int64_t)g * a.C]), h, local);
  }
  p[(seg.count - 1) * per] = h;
}

// ---------------------------------------------------------------------------------------------- one token
constexpr int kStepThreads = 256;
constexpr int kStepSeqs = 4;  // sequences per thread: its A, D and bias loads serve all of them

template <int L, typename TIn, typename TOut>
__global__ void __launch_bounds__(kStepThreads)
ssm_decode_kernel(const SsmLaunch a) {
  const int tid = threadIdx.x, l = tid % L;
  const int64_t c = (int64_t)blockIdx.x * (kStepThreads / L) + tid / L;
  const int64_t s0 = (int64_t)blockIdx.y * kStepSeqs;
  const bool live = c < a.C;
  const int64_t cc = live ? c : 0, g = cc / (a.C / a.G);
  const bool vec = a.n % 4 == 0;
  grid_dependents_trigger();
  grid_dependency_wait();  // the states and this step's inputs are in memory
  float4 h[kStepSeqs];
  float u[kStepSeqs], dt[kStepSeqs], z[kStepSeqs];
  const int s_lo = l * kK;
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    h[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t s = s0 + q;
    if (live && s < a.B) {
      const float* p = a.h_in + (s * a.C + cc) * a.n + s_lo;
      if (vec && s_lo < a.n) {
        h[q] = __ldcs(reinterpret_cast<const float4*>(p));
      } else {
        if (s_lo + 0 < a.n) h[q].x = p[0];
        if (s_lo + 1 < a.n) h[q].y = p[1];
        if (s_lo + 2 < a.n) h[q].z = p[2];
        if (s_lo + 3 < a.n) h[q].w = p[3];
      }
    }
  }
  float A2[kK];
#pragma unroll
  for (int k = 0; k < kK; ++k) A2[k] = s_lo + k < a.n ? log2_rate(a.A[cc * a.n + s_lo + k]) : 0.f;
  const float Dc = a.D ? a.D[cc] : 0.f, bias = a.delta_bias ? a.delta_bias[cc] : 0.f;
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int64_t s = min(s0 + q, a.B - 1);
    u[q] = to_f(reinterpret_cast<const TIn*>(a.u)[s * a.u_sb + cc]);
    const float x = to_f(reinterpret_cast<const TIn*>(a.delta)[s * a.d_sb + cc]) + bias;
    dt[q] = a.softplus ? softplus(x) : x;
    z[q] = a.z ? silu(to_f(reinterpret_cast<const TIn*>(a.z)[s * a.z_sb + cc])) : 1.f;
  }
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int64_t s = s0 + q;
    if (s >= a.B) break;  // uniform over the block
    const TIn* Bp = reinterpret_cast<const TIn*>(a.Bm.ptr) + s * a.Bm.sb + g * a.Bm.sh + s_lo;
    const TIn* Cp = reinterpret_cast<const TIn*>(a.Cm.ptr) + s * a.Cm.sb + g * a.Cm.sh + s_lo;
    float hk[kK] = {h[q].x, h[q].y, h[q].z, h[q].w};
    float acc = 0.f;
    const float dtu = dt[q] * u[q];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      if (s_lo + k < a.n) {
        hk[k] = fmaf(ex2(dt[q] * A2[k]), hk[k], dtu * to_f(Bp[k]));
        acc = fmaf(to_f(Cp[k]), hk[k], acc);
      }
    }
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) acc += __shfl_xor_sync(kFullMask, acc, off);
    if (live) {
      float* p = a.h_out + (s * a.C + c) * a.n + s_lo;
      if (vec && s_lo < a.n) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(hk[0], hk[1], hk[2], hk[3]));
      } else {
#pragma unroll
        for (int k = 0; k < kK; ++k)
          if (s_lo + k < a.n) p[k] = hk[k];
      }
      if (l == 0) store1(reinterpret_cast<TOut*>(a.y) + s * a.y_sb + c, fmaf(Dc, u[q], acc) * z[q]);
    }
  }
}

Segments plan(int64_t B, int64_t N, int64_t C, int n, int64_t G) {
  const int L = lanes_of(n), CT = kThreads / L, TT = tile_tokens(L);
  const int64_t blocks = B * G * ((C / G + CT - 1) / CT);
  // A segmented scan does the exponentials twice, so it pays from about three segments' worth of idle SMs
  // on, and segments of a few tiles at least.
  const int64_t want = std::min<int64_t>(304 / std::max<int64_t>(blocks, 1), N / (4 * TT));
  if (want < 3) return Segments{1, N};
  const int64_t len = ((N + want - 1) / want + TT - 1) / TT * TT;
  return Segments{(int)((N + len - 1) / len), len};
}

template <int L, typename TIn, typename TOut>
cudaError_t launch_scan(const SsmLaunch& a, void* ws, const Segments& seg, cudaStream_t stream) {
  constexpr int CT = kThreads / L;
  const dim3 grid((unsigned)(a.G * ((a.C / a.G + CT - 1) / CT)), (unsigned)a.B, (unsigned)seg.count);
  if (seg.count == 1) {
    ssm_scan_kernel<L, TIn, TOut, kFull><<<grid, kThreads, 0, stream>>>(a, seg, nullptr, nullptr);
    return cudaGetLastError();
  }
  float* ws_h = static_cast<float*>(ws);
  float* ws_dt = ws_h + a.B * seg.count * a.C * a.n;
  const dim3 grid_local(grid.x, grid.y, grid.z - 1);  // nothing enters from the last segment
  ssm_scan_kernel<L, TIn, TOut, kLocal><<<grid_local, kThreads, 0, stream>>>(a, seg, ws_h, ws_dt);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t states = a.B * a.C * a.n;
  ssm_combine_kernel<<<(unsigned)((states + 255) / 256), 256, 0, stream>>>(a, seg, ws_h, ws_dt);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ssm_scan_kernel<L, TIn, TOut, kFinal><<<grid, kThreads, 0, stream>>>(a, seg, ws_h, ws_dt);
  return cudaGetLastError();
}

template <typename TIn, typename TOut>
cudaError_t launch_lanes(const SsmLaunch& a, void* ws, const Segments* seg, cudaStream_t stream) {
  auto step = [&](auto kernel, int L) {
    const int64_t per = kStepThreads / L;
    const dim3 grid((unsigned)((a.C + per - 1) / per), (unsigned)((a.B + kStepSeqs - 1) / kStepSeqs));
    return launch_dependent(kernel, grid, dim3(kStepThreads), 0, stream, a);
  };
  switch (lanes_of(a.n)) {
    case 1: return seg ? launch_scan<1, TIn, TOut>(a, ws, *seg, stream) : step(ssm_decode_kernel<1, TIn, TOut>, 1);
    case 2: return seg ? launch_scan<2, TIn, TOut>(a, ws, *seg, stream) : step(ssm_decode_kernel<2, TIn, TOut>, 2);
    case 4: return seg ? launch_scan<4, TIn, TOut>(a, ws, *seg, stream) : step(ssm_decode_kernel<4, TIn, TOut>, 4);
    case 8: return seg ? launch_scan<8, TIn, TOut>(a, ws, *seg, stream) : step(ssm_decode_kernel<8, TIn, TOut>, 8);
    default: return seg ? launch_scan<16, TIn, TOut>(a, ws, *seg, stream) : step(ssm_decode_kernel<16, TIn, TOut>, 16);
  }
}

cudaError_t launch_any(const SsmLaunch& a, void* ws, const Segments* seg, cudaStream_t stream) {
  if (a.in_bf16 && a.out_bf16) return launch_lanes<__nv_bfloat16, __nv_bfloat16>(a, ws, seg, stream);
  if (a.in_bf16) return launch_lanes<__nv_bfloat16, float>(a, ws, seg, stream);
  if (a.out_bf16) return launch_lanes<float, __nv_bfloat16>(a, ws, seg, stream);
  return launch_lanes<float, float>(a, ws, seg, stream);
}

}  // namespace

size_t ssm_workspace_bytes(int64_t B, int64_t N, int64_t C, int n, int64_t G) {
  const Segments s = plan(B, N, C, n, G);
  return s.count == 1 ? 0 : (size_t)(B * s.count * C * (n + 1)) * sizeof(float);
}

cudaError_t launch_ssm_prefill(const SsmLaunch& a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const Segments seg = plan(a.B, a.N, a.C, a.n, a.G);
  if (seg.count > 1 && ws_bytes < ssm_workspace_bytes(a.B, a.N, a.C, a.n, a.G)) return cudaErrorInvalidValue;
  return launch_any(a, ws, &seg, stream);
}

cudaError_t launch_ssm_decode(const SsmLaunch& a, cudaStream_t stream) { return launch_any(a, nullptr, nullptr, stream); }

}  // namespace la
