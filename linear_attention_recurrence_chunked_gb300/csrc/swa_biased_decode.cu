// swa_biased_decode.cu -- one decode step of window attention with grouped heads, capped scores and a
// distance bias, over the rings of swa_decode.cu (token p in slot p % window):
//   s_j = cap tanh(scale q.k_j / cap) - slope (pos - j),   o = sum_j softmax_j(s_j) v_j.
// The step reads each ring once and little else, so memory bounds it: 256 x 16 heads over 4 key heads and 256 slots
// at d = 128, capped and biased, takes 28 us, 4.9 TB/s, 73 % of the measured copy rate.  One CTA per (sequence, key head), one
// warp per 32 slots of the ring: a warp scores its slots for all query heads of the group, takes the softmax
// of its own slots and adds up its own value rows, so that no warp waits for another before the end, where
// the warps' parts meet in shared memory.  The new token is used from the arguments; the warp of its slot
// writes it there.
//
// bf16: a key row meets up to 16 query heads, too many operations for the CUDA cores beside the loads (58 us for
// 256 x 16 heads over 4 key heads and 256 slots at d = 128, three times the time of its bytes) and too few rows
// for tcgen05, so the products are mma.m16n8k16 with the heads as the 16 rows.  Keys go from memory to the
// operand registers directly: a lane's 16 bytes are elements of one slot, and which elements of the sum they are
// is the same for the queries.  Values come by asynchronous copies, all 32 rows of a warp at once, and are
// transposed on the way from shared memory.  The weights meet them in two bf16 parts.
// fp32: CUDA cores, four query heads at a time.
#include "layers.cuh"
#include "swa_common.cuh"
#include "tc.cuh"

namespace la {
namespace {

constexpr int kMaxD = 128;
constexpr int kSlots = 32;     // per warp
constexpr int kMaxWarps = 8;   // window up to 256
constexpr int kHeads = 4;      // query heads per pass
constexpr int kLoads = 4;      // row loads in flight

template <typename T>
__device__ __forceinline__ uint4 load_row(const T* p) { return *reinterpret_cast<const uint4*>(p); }

// ---------------------------------------------------------------------------------------------- bf16
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// DP: width padded to 64 or 128
template <typename TOut, int DP>
__global__ void __launch_bounds__(32 * kMaxWarps, 2)
swa_biased_decode_mma_kernel(const SwaBiasedDecodeLaunch a) {
  using T = __nv_bfloat16;
  constexpr int kGroups = DP / 32;               // of 32 columns: a load of eight slots each
  constexpr int kPairs = DP / 16;                // of 8-column output tiles
  constexpr int kRegion = kSlots * DP * 2;       // a warp's shared memory: its value rows, then its output
  static_assert(kRegion >= 16 * DP * 4, "");
  extern __shared__ __align__(128) uint8_t sw_smem[];
  __shared__ float s_m[kMaxWarps][16], s_l[kMaxWarps][16];
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
  const int n = pos < w ? (int)pos + 1 : w;
  const int first = warp * kSlots, h0 = (int)hk * group;
  const T* kn = reinterpret_cast<const T*>(c.k) + sk * d;
  const T* vn = reinterpret_cast<const T*>(c.v) + sk * d;
  T* kc = reinterpret_cast<T*>(c.k_cache) + sk * (int64_t)w * d;
  T* vc = reinterpret_cast<T*>(c.v_cache) + sk * (int64_t)w * d;
  uint8_t* region = sw_smem + warp * kRegion;
  const uint32_t rbase = tc::smem_u32(region);
  const int chunks = d / 8;
  // place of 16-byte chunk `ch` of value row r: eight neighbouring rows meet eight different banks
  auto at = [](int r, int ch) { return (uint32_t)(r * (DP * 2) + ((ch ^ (r & 7)) << 4)); };

  // ---- value rows on their way; slots that hold nothing become zeros
#pragma unroll
  for (int i = 0; i < kSlots * (DP / 8) / 32; ++i) {
    const int e = lane + 32 * i, r = e / (DP / 8), ch = e % (DP / 8), slot = first + r;
    const T* src = slot == slot_new ? vn : vc + (int64_t)slot * d;
    const bool on = slot < n && ch < chunks;
    tc::cp_async16(rbase + at(r, ch), on ? src + ch * 8 : vn, on ? 16u : 0u);
  }
  tc::cp_async_commit();

  // ---- scores: rows = heads (lane / 4 and that + 8), columns = slots
  const int hr = lane >> 2, q4 = lane & 3;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const T* q = reinterpret_cast<const T*>(c.q) + (s * c.H + h0) * d;
  uint4 ql[kGroups], qh[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int col = g * 32 + q4 * 8;
    ql[g] = hr < group && col < d ? *reinterpret_cast<const uint4*>(q + hr * d + col) : zero;
    qh[g] = hr + 8 < group && col < d ? *reinterpret_cast<const uint4*>(q + (hr + 8) * d + col) : zero;
  }
  float x[4][4];
  uint4 kr[2][2][kGroups];  // two tiles of eight slots now, two on their way
  auto fetch = [&](int half) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int slot = first + (half * 2 + t) * 8 + hr;
      const T* src = slot == slot_new ? kn : kc + (int64_t)slot * d;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int col = g * 32 + q4 * 8;
        kr[half][t][g] = slot < n && col < d ? *reinterpret_cast<const uint4*>(src + col) : zero;
      }
    }
  };
  fetch(0);
  fetch(1);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint4 k = kr[t / 2][t % 2][g];
      mma16816(x[t], ql[g].x, qh[g].x, ql[g].y, qh[g].y, k.x, k.y);
      mma16816(x[t], ql[g].z, qh[g].z, ql[g].w, qh[g].w, k.z, k.w);
    }
  }
  // ---- softmax of this warp's slots
  const bool spare = group <= 8;  // rows 8 to 15 have no head
  const float inv_cap = 1.f / a.softcap;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= 2 && spare) continue;
      const int slot = first + t * 8 + q4 * 2 + (e & 1), h = hr + (e >> 1) * 8;
      float y = x[t][e] * c.scale;
      if (a.softcap != 0.f) y = capped(y, a.softcap, inv_cap);
      const float age = (float)(slot_new >= slot ? slot_new - slot : slot_new - slot + w);
      if (a.slopes && h < group) y = fmaf(-a.slopes[h0 + h], age, y);
      x[t][e] = slot < n ? y : -INFINITY;
      m[e >> 1] = fmaxf(m[e >> 1], x[t][e]);
    }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (r == 1 && spare) continue;
    m[r] = fmaxf(m[r], __shfl_xor_sync(kFullMask, m[r], 1));
    m[r] = fmaxf(m[r], __shfl_xor_sync(kFullMask, m[r], 2));
    const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 2 * r; e < 2 * r + 2; ++e) {
        x[t][e] = ex2((x[t][e] - base) * kLog2e);
        l[r] += x[t][e];
      }
    l[r] += __shfl_xor_sync(kFullMask, l[r], 1);
    l[r] += __shfl_xor_sync(kFullMask, l[r], 2);
    if (q4 == 0) {
      s_m[warp][hr + 8 * r] = m[r];
      s_l[warp][hr + 8 * r] = l[r];
    }
  }
  // ---- this warp's value rows
  float o[2 * kPairs][4];
#pragma unroll
  for (int t = 0; t < 2 * kPairs; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
  tc::cp_async_wait_all();
  __syncwarp();
  // Weights in two bf16 parts, the second one what the first leaves: a weight is off by 2^-17 of itself, where one part
  // would leave 2^-8, more than an fp32 output can hide.  Up to eight heads the second parts take the rows that have no
  // head and no product is added; beyond, they are products of their own (256 x 64 heads over 4: 44 us, 41.3 with one
  // part).  What second parts make of a value that is not finite is left out: the first ones' result stands.
  auto products = [&](auto a) {  // a(kt): the weights of sixteen slots as an operand
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      const int r = kt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
      const uint4 w = a(kt);
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        uint32_t b[4];
        ldmatrix_trans(b, rbase + at(r, 2 * p + (lane >> 4)));
        mma16816(o[2 * p], w.x, w.y, w.z, w.w, b[0], b[1]);
        mma16816(o[2 * p + 1], w.x, w.y, w.z, w.w, b[2], b[3]);
      }
    }
  };
  // rows of half h (0: lane / 4, 1: that + 8) of tile t: two slots' first parts, and what they leave
  auto major = [&](int t, int h) { return tc::pack2_bf16(x[t][2 * h], x[t][2 * h + 1]); };
  auto minor = [&](int t, int h) {
    const uint32_t w = major(t, h);
    return tc::pack2_bf16(x[t][2 * h] - __uint_as_float(w << 16), x[t][2 * h + 1] - __uint_as_float(w & 0xffff0000u));
  };
  if (spare) {
    products([&](int kt) { return make_uint4(major(2 * kt, 0), minor(2 * kt, 0), major(2 * kt + 1, 0), minor(2 * kt + 1, 0)); });
#pragma unroll
    for (int t = 0; t < 2 * kPairs; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) o[t][e] += finite1(o[t][2 + e]) ? o[t][2 + e] : 0.f;
  } else {
    products([&](int kt) { return make_uint4(major(2 * kt, 0), major(2 * kt, 1), major(2 * kt + 1, 0), major(2 * kt + 1, 1)); });
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < 2 * kPairs; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fmaf(0.f, o[t][e], sum);
    if (__all_sync(kFullMask, sum == 0.f))
      products([&](int kt) { return make_uint4(minor(2 * kt, 0), minor(2 * kt, 1), minor(2 * kt + 1, 0), minor(2 * kt + 1, 1)); });
  }
  // the new token into its slot, by the warp that used it from the arguments
  if (slot_new / kSlots == warp && lane < chunks) {
    reinterpret_cast<uint4*>(kc + (int64_t)slot_new * d)[lane] = reinterpret_cast<const uint4*>(kn)[lane];
    reinterpret_cast<uint4*>(vc + (int64_t)slot_new * d)[lane] = reinterpret_cast<const uint4*>(vn)[lane];
  }
  __syncwarp();  // the value rows are used up: their place takes the output
  float* part = reinterpret_cast<float*>(region);
#pragma unroll
  for (int t = 0; t < 2 * kPairs; ++t) {
    if (t * 8 < d) {
      const int col = t * 8 + q4 * 2;
      if (hr < group) *reinterpret_cast<float2*>(part + hr * d + col) = make_float2(o[t][0], o[t][1]);
      if (hr + 8 < group) *reinterpret_cast<float2*>(part + (hr + 8) * d + col) = make_float2(o[t][2], o[t][3]);
    }
  }
  __syncthreads();
  // ---- the warps' parts together
  for (int e = threadIdx.x * 2; e < group * d; e += blockDim.x * 2) {
    const int g = e / d;
    float hi = s_m[0][g];
    for (int u = 1; u < warps; ++u) hi = fmaxf(hi, s_m[u][g]);
    float2 sum = make_float2(0.f, 0.f);
    float total = 0.f;
    for (int u = 0; u < warps; ++u) {
      const float f = ex2((s_m[u][g] - hi) * kLog2e);
      const float2 y = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(sw_smem + u * kRegion) + e);
      sum.x = fmaf(f, y.x, sum.x);
      sum.y = fmaf(f, y.y, sum.y);
      total = fmaf(f, s_l[u][g], total);
    }
    TOut* out = reinterpret_cast<TOut*>(c.out) + (s * c.H + h0) * d + e;
    store1(out, sum.x / total);
    store1(out + 1, sum.y / total);
  }
}

// ---------------------------------------------------------------------------------------------- fp32
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
  const int n = pos < w ? (int)pos + 1 : w;
  const int col = lane % LPR * V, sub = lane / LPR, first = warp * kSlots;
  const bool on = col < d;
  const TIn* kn = reinterpret_cast<const TIn*>(c.k) + sk * d + col;
  const TIn* vn = reinterpret_cast<const TIn*>(c.v) + sk * d + col;
  TIn* kc = reinterpret_cast<TIn*>(c.k_cache) + sk * (int64_t)w * d + col;
  TIn* vc = reinterpret_cast<TIn*>(c.v_cache) + sk * (int64_t)w * d + col;
  const float inv_cap = 1.f / a.softcap;
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
        if (a.softcap != 0.f) x[g] = capped(x[g], a.softcap, inv_cap);
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

template <typename TOut, int DP>
cudaError_t launch_mma(const SwaBiasedDecodeLaunch& a, cudaStream_t stream) {
  constexpr int kRegion = kSlots * DP * 2;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(swa_biased_decode_mma_kernel<TOut, DP>, kMaxWarps * kRegion, done);
  if (e != cudaSuccess) return e;
  const int warps = (a.base.window + kSlots - 1) / kSlots;
  return launch_dependent(swa_biased_decode_mma_kernel<TOut, DP>, dim3((unsigned)(a.base.S * a.Hkv)), dim3((unsigned)(32 * warps)),
                          (size_t)(warps * kRegion), stream, a);
}

template <typename TOut>
cudaError_t launch_fp32(const SwaBiasedDecodeLaunch& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(a.base.S * a.Hkv)), block((unsigned)(32 * ((a.base.window + kSlots - 1) / kSlots)));
  const int vecs = a.base.d / kVec<float>;
  if (vecs > 16) return launch_dependent(swa_biased_decode_kernel<float, TOut, 32>, grid, block, 0, stream, a);
  if (vecs > 8) return launch_dependent(swa_biased_decode_kernel<float, TOut, 16>, grid, block, 0, stream, a);
  return launch_dependent(swa_biased_decode_kernel<float, TOut, 8>, grid, block, 0, stream, a);
}

template <typename TOut>
cudaError_t launch_out(const SwaBiasedDecodeLaunch& a, cudaStream_t stream) {
  if (!a.base.in_bf16) return launch_fp32<TOut>(a, stream);
  return a.base.d <= 64 ? launch_mma<TOut, 64>(a, stream) : launch_mma<TOut, 128>(a, stream);
}

}  // namespace

cudaError_t launch_swa_biased_decode(const SwaBiasedDecodeLaunch& a, cudaStream_t stream) {
  return a.base.out_bf16 ? launch_out<__nv_bfloat16>(a, stream) : launch_out<float>(a, stream);
}

}  // namespace la
