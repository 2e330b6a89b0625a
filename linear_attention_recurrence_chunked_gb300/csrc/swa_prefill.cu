// swa_prefill.cu -- masked window attention over a prompt, fp32 inputs, and the rings that the decode
// steps read.  For query i at key position p_i and head h:
//   s_ij = cap tanh(scale q_i.k_j / cap) - slope_h |p_i - j|,  o_i = sum_j softmax_j(s_ij) v_j
// over the keys lo_i <= j < hi_i (one interval per query; empty: o_i = 0).  One pass over the keys with
// the running maximum and sum of the softmax (fp32).
//
// A CTA takes 64 queries of one head and walks the key tiles between its lowest lo and highest hi; each
// of its 256 threads holds a 4 x 4 piece of the scores and 4 rows x d/16 columns of the output.  fp32
// products run on the CUDA cores (bf16 operands would not keep fp32's accuracy), which bound it.
// Where the query tiles leave SMs idle, the CTAs of a cluster share a tile's keys; their maxima, sums and outputs
// meet in distributed shared memory, so that no workspace is needed (6 heads of 133 queries over 333 keys at d = 40:
// 47 -> 25 us).  16 heads of 512 queries over 16384 keys at d = 64: 1260 us, 27 TFLOP/s of 80: each float4 read from
// shared memory feeds eight multiply-adds, half of what the cores could take.
#include <cooperative_groups.h>

#include <algorithm>

#include "layers.cuh"
#include "swa_common.cuh"

namespace la {
namespace {

constexpr int kBM = 64, kBN = 64, kThreads = 256, kSMs = 152;

template <typename TOut, int DP>
__global__ void __launch_bounds__(kThreads)
swa_simt_kernel(const SwaPrefillLaunch a, int q_tiles, int parts) {
  constexpr int LD = DP + 4;       // row pitch of Q, K, V in floats: rows start 4 banks apart
  constexpr int LP = kBN + 4;
  constexpr int NC = DP / 16;      // output columns per thread: tx + 16 j
  extern __shared__ __align__(16) float smem[];
  float* Qs = smem;                // [64][LD]
  float* Ks = Qs + kBM * LD;
  float* Vs = Ks + kBN * LD;
  float* Ps = Vs + kBN * LD;       // [64][LP]
  __shared__ int s_lo[kBM], s_hi[kBM];
  __shared__ int s_range[2];
  __shared__ float s_m[kBM], s_l[kBM];  // of this CTA's share of the keys

  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int part = (int)(blockIdx.x % parts);  // the cluster's rank
  const int64_t tile = blockIdx.x / parts, bh = tile / q_tiles;
  const int qt = (int)(tile % q_tiles);
  const int64_t b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hkv);
  const int64_t len = sequence_length(a.lens, b, a.Nk, a.status, h == 0 && qt == 0 && part == 0 && tid == 0);
  if (len < 0) return;  // the whole cluster
  const int64_t i0 = (int64_t)qt * kBM;
  if (tid == 0) {
    s_range[0] = INT32_MAX;
    s_range[1] = 0;
  }
  __syncthreads();
  if (tid < kBM) {
    const KeySpan sp = key_span(a, (int)b, (int)i0 + tid, (int)len);
    s_lo[tid] = sp.lo;
    s_hi[tid] = sp.hi;
    if (sp.lo < sp.hi) {
      atomicMin(&s_range[0], sp.lo);
      atomicMax(&s_range[1], sp.hi);
    }
  }
  const float* q = reinterpret_cast<const float*>(a.q.ptr) + b * a.q.sb + h * a.q.sh;
  const float* k = reinterpret_cast<const float*>(a.k.ptr) + b * a.k.sb + hk * a.k.sh;
  const float* v = reinterpret_cast<const float*>(a.v.ptr) + b * a.v.sb + hk * a.v.sh;
  for (int e = tid; e < kBM * (DP / 4); e += kThreads) {
    const int r = e / (DP / 4), c = e % (DP / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i0 + r < a.Nq && c < a.d) x = load4(q + (i0 + r) * a.q.st + c);
    *reinterpret_cast<float4*>(Qs + r * LD + c) = make_float4(x.x * a.scale, x.y * a.scale, x.z * a.scale, x.w * a.scale);
  }
  __syncthreads();
  const int first = s_range[0], last = s_range[1];

  float o[4][NC], m[4], l[4];
  int lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    lo[i] = s_lo[ty * 4 + i];
    hi[i] = s_hi[ty * 4 + i];
#pragma unroll
    for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
  }
  const float slope = a.slopes ? a.slopes[h] : 0.f;

  for (int j0 = last > 0 ? first + part * kBN : 0; j0 < last; j0 += parts * kBN) {  // none seen: last = 0
    __syncthreads();  // the previous tile is used up
    bool bad = false;
    for (int e = tid; e < kBN * (DP / 4); e += kThreads) {
      const int r = e / (DP / 4), c = e % (DP / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (j0 + r < last && c < a.d) {
        x = load4(k + (int64_t)(j0 + r) * a.k.st + c);
        y = load4(v + (int64_t)(j0 + r) * a.v.st + c);
      }
      *reinterpret_cast<float4*>(Ks + r * LD + c) = x;
      *reinterpret_cast<float4*>(Vs + r * LD + c) = y;
      bad = bad || !finite4(y);
    }
    const bool guard = __syncthreads_or(bad);  // a masked value must not reach a row as 0 * NaN
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < DP; c += 4) {
      float4 kv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * LD + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(Qs + (ty * 4 + i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] += dot4(qv, kv[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = bias_origin(KeySpan{lo[i], hi[i]}, (int)(a.q_pos0 + i0) + ty * 4 + i);
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        float x = s[i][j];
        if (a.softcap != 0.f) x = a.softcap * tanhf(x / a.softcap);
        if (slope != 0.f) x -= slope * fabsf((float)(pos - key));
        s[i][j] = key >= lo[i] && key < hi[i] ? x : -INFINITY;
        mt = fmaxf(mt, s[i][j]);
      }
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(kFullMask, mt, off));
      const float mn = fmaxf(m[i], mt);
      const float base = mn == -INFINITY ? 0.f : mn;  // nothing seen so far: every weight below is 0
      const float f = __expf(m[i] - base);
      float lt = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = __expf(s[i][j] - base);
        Ps[(ty * 4 + i) * LP + tx + 16 * j] = p;
        lt += p;
      }
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) lt += __shfl_xor_sync(kFullMask, lt, off);
      l[i] = l[i] * f + lt;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c] *= f;
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
    if (!guard) {
#pragma unroll 2
      for (int j = 0; j < kBN; j += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(Ps + (ty * 4 + i) * LP + j);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float* vp = Vs + j * LD + tx + 16 * c;
          const float v0 = vp[0], v1 = vp[LD], v2 = vp[2 * LD], v3 = vp[3 * LD];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i][c] = fmaf(p[i].w, v3, fmaf(p[i].z, v2, fmaf(p[i].y, v1, fmaf(p[i].x, v0, o[i][c]))));
        }
      }
    } else {
      for (int j = 0; j < kBN; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + j >= lo[i] && j0 + j < hi[i]) {
            const float p = Ps[(ty * 4 + i) * LP + j];
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] = fmaf(p, Vs[j * LD + tx + 16 * c], o[i][c]);
          }
    }
  }
  TOut* out = reinterpret_cast<TOut*>(a.o) + b * a.o_sb + h * a.o_sh;
  if (parts > 1) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __syncthreads();  // the last tile is used up: its place takes the output
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
#pragma unroll
      for (int c = 0; c < NC; ++c) Ks[r * LD + tx + 16 * c] = o[i][c];
      if (tx == 0) {
        s_m[r] = m[i];
        s_l[r] = l[i];
      }
    }
    cluster.sync();
    // rows part, part + parts, ...: a half warp a row
    for (int r = part + (tid >> 4) * parts; r < kBM; r += (kThreads / 16) * parts) {
      const int64_t row = i0 + r;
      if (row < a.Nq && a.q_pos0 + row < len) {
        float top = -INFINITY, total = 0.f, sum[NC];
        for (int u = 0; u < parts; ++u) top = fmaxf(top, *cluster.map_shared_rank(&s_m[r], u));
#pragma unroll
        for (int c = 0; c < NC; ++c) sum[c] = 0.f;
        for (int u = 0; u < parts; ++u) {
          const float mu = *cluster.map_shared_rank(&s_m[r], u), lu = *cluster.map_shared_rank(&s_l[r], u);
          if (lu == 0.f) continue;  // this share holds none of the row's keys
          const float f = __expf(mu - (top == -INFINITY ? 0.f : top));
          const float* x = cluster.map_shared_rank(Ks + r * LD, u);
          total = fmaf(f, lu, total);
#pragma unroll
          for (int c = 0; c < NC; ++c) sum[c] = fmaf(f, x[tx + 16 * c], sum[c]);
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;  // a row that sees nothing gives zeros
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (tx + 16 * c < a.d) store1(out + row * a.o_st + tx + 16 * c, sum[c] * inv);
      }
    }
    cluster.sync();  // the parts are read before a CTA ends
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = i0 + ty * 4 + i;
    if (row < a.Nq && a.q_pos0 + row < len) {
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // a row that sees nothing gives zeros
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (tx + 16 * c < a.d) store1(out + row * a.o_st + tx + 16 * c, o[i][c] * inv);
    }
  }
}

// One warp per (sequence, key head, slot): the newest token of the slot, as the decode steps expect it.
template <typename T>
__global__ void __launch_bounds__(256)
swa_fill_rings_kernel(const SwaPrefillLaunch a) {
  const int64_t id = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = a.window, slot = id % w, bh = id / w, b = bh / a.Hkv, h = bh - b * a.Hkv;
  if (b >= a.B) return;
  const int64_t len = sequence_length(a.lens, b, a.Nk, a.status, false);
  if (slot >= len) return;  // also a sequence that is skipped (len = -1)
  const int64_t t = len - 1 - (len - 1 - slot) % w;
  const T* k = reinterpret_cast<const T*>(a.k.ptr) + b * a.k.sb + h * a.k.sh + t * a.k.st;
  const T* v = reinterpret_cast<const T*>(a.v.ptr) + b * a.v.sb + h * a.v.sh + t * a.v.st;
  T* kc = reinterpret_cast<T*>(a.k_cache) + id * a.d;
  T* vc = reinterpret_cast<T*>(a.v_cache) + id * a.d;
  const int vecs = a.d / kVec<T>;  // rows are whole 16-byte vectors: d is a multiple of 8
  for (int i = lane; i < 2 * vecs; i += 32) {
    const bool second = i >= vecs;
    const int e = second ? i - vecs : i;
    reinterpret_cast<uint4*>(second ? vc : kc)[e] = reinterpret_cast<const uint4*>(second ? v : k)[e];
  }
}

template <typename TOut, int DP>
cudaError_t launch_simt(const SwaPrefillLaunch& a, cudaStream_t stream) {
  constexpr int kSmem = (3 * 64 * (DP + 4) + kBM * (kBN + 4)) * (int)sizeof(float);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(swa_simt_kernel<TOut, DP>, kSmem, done);
  if (e != cudaSuccess) return e;
  const int q_tiles = (int)((a.Nq + kBM - 1) / kBM);
  const int64_t tiles = a.B * a.H * q_tiles;
  // key tiles of a query tile at most
  const int64_t keys = std::min<int64_t>((a.Nk + kBN - 1) / kBN, a.window > 0 ? (a.window + kBM + 2 * kBN - 2) / kBN : INT32_MAX);
  int parts = 1;
  while (parts < 8 && tiles * parts < kSMs && parts < keys) parts *= 2;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)parts;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, swa_simt_kernel<TOut, DP>, a, q_tiles, parts);
}

template <typename TOut>
cudaError_t launch_width(const SwaPrefillLaunch& a, cudaStream_t stream) {
  if (a.d <= 32) return launch_simt<TOut, 32>(a, stream);
  if (a.d <= 64) return launch_simt<TOut, 64>(a, stream);
  return launch_simt<TOut, 128>(a, stream);
}

}  // namespace

cudaError_t launch_swa_prefill_simt(const SwaPrefillLaunch& a, cudaStream_t stream) {
  return a.out_bf16 ? launch_width<__nv_bfloat16>(a, stream) : launch_width<float>(a, stream);
}

cudaError_t launch_swa_fill_rings(const SwaPrefillLaunch& a, cudaStream_t stream) {
  const int64_t rows = a.B * a.Hkv * a.window;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  if (a.in_bf16) swa_fill_rings_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
  else swa_fill_rings_kernel<float><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace la
