// ssm.cu -- selective state space scan and its one-token step:
//   dt = f(delta + delta_bias),  h[c,s] <- exp(dt A[c,s]) h[c,s] + dt u B[g,s],
//   y = (sum_s C[g,s] h[c,s] + D u) silu(z)
// per token, channel c of group g and state s (NoteBank Sec. 2 Eq. (1) with a diagonal A_t).
//
// Per (token, channel, state) the scan needs one exponential and four fp32 operations, per (token, channel)
// four 2-byte elements of memory: with 16 states the special-function unit (32 results an SM and clock) needs
// 1.4 times what memory does.  The decay differs per (channel, state), so no chunk form on
// the tensor cores exists: the tokens are walked in order, with the channels and states in parallel.
// 4 x 16384 x 2048 channels with 16 states, bf16: 818 us.  The bytes alone take 161 us and the exponentials 220 us, at the
// 2.0 GHz it ran at, on all SMs; 128 blocks leave 24 of 152 without one.  A (token, channel) costs 126 instructions, about
// 70 of them the recurrence's own with its loads and stores; nothing is near its limit (the special-function pipe at 31 %,
// fp32 at 25 %, shared memory at 24 % of elapsed), and the warps wait most for the barrier of a tile, on one another.
//
// A block has four scan warps, four layout warps for each channel of a lane, and four output warps, which work on
// tiles of tokens in turn through shared memory, one barrier a tile.  While the scan warps walk tile i, the layout warps prepare tile
// i + 1 (the step sizes with their softplus, once per (token, channel), and B_t, C_t in fp32), with the raw
// inputs of the tiles behind it on their way, and the output warps add up the readout of tile i - 1, apply
// the skip term and the gate and store it.  In the scan L lanes share kCh channels; a lane holds four states
// of each, as pairs for the paired fp32 operations.  The inputs of the next tokens are read before the parts
// of the readout are written: the compiler keeps that order (it cannot tell the two apart), and the other one
// would put a shared-memory round trip, an exponential and four operations in a row for every token.
#include <algorithm>

#include "layers.cuh"
#include "tc.cuh"

namespace la {
namespace {

constexpr int kScan = 128;    // threads of the four scan warps
constexpr int kOutput = 128;  // and of the output warps
// Channels per scan lane.  Two halve a state's share of the reads of B and C (a lane's bytes count there, 128
// a clock and SM, also where lanes read the same), which bound the scan with one, but leave half the blocks.
// 4 x 16384 x 2048 channels, 16 states: 818 us with two, 928 us with one; with at most one block of one channel
// per lane on each SM, one channel is faster.
constexpr int layout_threads(int ch) { return ch * kScan; }
constexpr int block_threads(int ch) { return kScan + layout_threads(ch) + kOutput; }
// tokens whose inputs a scan lane reads ahead: one block with two channels per lane has an SM's registers for
// itself
constexpr int read_ahead(int ch) { return ch == 2 ? 4 : 2; }
constexpr int kK = 4;              // states per lane

// A log2(e), kept finite so that a step of dt = 0 changes nothing even for the lowest A
__device__ __forceinline__ float log2_rate(float A) {
  const float x = A * kLog2e;
  return x < -3.402823466e38f ? -3.402823466e38f : x;
}

// Added to the exponent x, which costs nothing in its multiplication: the unit's 2^x comes out low on average, and a state
// takes one such factor per token, so that the errors add up along its memory.  Against fp64 over 2^20 arguments per
// factor of two, the mean is -1.6e-8 to -2.7e-8 of the value for 2^-8 < |x| < 1 and -5e-9 to -1e-8 for 2^-19 < |x| < 2^-8,
// where results are so close to 1 that they are nearly rounded to nearest.  Each range has a centre of its own; below 9e-9
// is left for 2^-8 < |x| < 1/2, and below 4e-9 from there down to 2^-19, where memories are long.  (3.6e-8 for all left
// 2e-8 there: a memory of 6000 tokens was off by 5e-5 in one pass, now by less than 2e-5, and 2000 tokens of 4096
// channels by 5.2e-7, now 1.9e-7.)  Both are below half a rounding at 1: dt = 0 stays the identity.
__device__ __forceinline__ float centre_of(float x) { return fabsf(x) > 0.00390625f ? 3.6e-8f : 9e-9f; }

// Time segments: segment g of a sequence takes tokens [g * len, (g + 1) * len).
struct Segments {
  int count;
  int64_t len;
};

// kFull walks a whole sequence; kLocal leaves a segment's state from zero and its
// sum of dt in the workspace; kFinal walks a segment from the state in the workspace.
enum Mode { kFull, kLocal, kFinal };

__host__ __device__ constexpr int lanes_of(int n) { return n <= 4 ? 1 : n <= 8 ? 2 : n <= 16 ? 4 : n <= 32 ? 8 : 16; }

// Four states' B and C for one lane.
struct LaneBC {
  ulonglong2 b, c;
};

template <int L, int kCh, typename TIn>
struct Tile {
  static constexpr int TT = L >= 4 ? 32 : 8 * L;  // tokens
  static constexpr int CT = kCh * kScan / L;      // channels of a block
  static constexpr int kRaw = sizeof(TIn) == 2 ? 5 : 4;  // tiles of raw inputs: from the one being stored to the last on its way
  struct Raw {
    TIn u[TT * CT], delta[TT * CT], z[TT * CT], bc[2][TT * L * kK];
  };
  struct Work {
    float2 dt[TT][CT];                            // (dt, dt u)
    LaneBC bc[TT][L];
    float y[kCh][TT][kScan];                      // the lanes' parts of the readout
  };
  Work work[2];
  Raw raw[kRaw];
  // Place of channel c in row r of dt, and of its lanes' parts in y (in units of L).  Eight neighbouring
  // layout or output threads, which hold vectors of channels, and the scan's lanes, which hold neighbouring
  // channels, both meet different banks.  The places repeat every kPeriod rows.
  static constexpr int kPeriod = L >= 4 * kCh ? L / 2 / kCh : 1;
  __device__ static __forceinline__ int dt_at(int r, int c) {
    return kCh == 1 ? c ^ ((((r * CT + c) >> 4) & 3) << 1) : c ^ ((((r * (CT / 2) + (c >> 1)) >> 3) & 3) << 1);
  }
  __device__ static __forceinline__ int y_at(int r, int c) {
    return kCh == 1 ? c ^ (((r * CT + c) >> 3) & 7) : (c >> 1) ^ (((r * (CT / 2) + (c >> 1)) >> 3) & 3);
  }
};

template <int L, int kCh, typename TIn, typename TOut, int MODE>
__global__ void __launch_bounds__(block_threads(kCh), kCh == 2 ? 1 : 2)
ssm_scan_kernel(const SsmLaunch a, Segments seg, float* ws_h, float* ws_dt) {
  using T = Tile<L, kCh, TIn>;
  constexpr int CT = T::CT, TT = T::TT, kLayout = layout_threads(kCh), kAhead = read_ahead(kCh);
  extern __shared__ __align__(16) uint8_t ssm_smem[];
  T& sm = *reinterpret_cast<T*>(ssm_smem);

  const int tid = threadIdx.x;
  const int64_t Cg = a.C / a.G, tiles = (Cg + CT - 1) / CT;
  const int64_t g = blockIdx.x / tiles, b = blockIdx.y;
  const int64_t c_base = g * Cg + (blockIdx.x % tiles) * CT, c_end = (g + 1) * Cg;
  const int64_t sid = blockIdx.z;
  const int64_t len = sequence_length(a.lens, b, a.N, a.status, blockIdx.x == 0 && sid == 0 && tid == 0);
  if (len < 0) return;  // uniform over the block
  const int64_t t0 = sid * seg.len;
  const int tokens = t0 < len ? (int)(min(t0 + seg.len, len) - t0) : 0;
  const int count = (tokens + TT - 1) / TT;  // tiles

  if (tid < kScan) {
    // ================================================================ scan warps
    const int l = tid % L, p = tid / L;
    const int64_t c = c_base + p * kCh;
    f32x2 A01[kCh], A23[kCh], h01[kCh], h23[kCh];
    float dt_sum[kCh], slowest = INFINITY;  // of the lane's states
#pragma unroll
    for (int e = 0; e < kCh; ++e) {
      float A2[kK], h[kK];
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int s = l * kK + k;
        const bool on = c + e < c_end && s < a.n;
        A2[k] = on ? log2_rate(a.A[(c + e) * a.n + s]) : 0.f;
        if (on) slowest = fminf(slowest, fabsf(A2[k]));
        h[k] = 0.f;
        if (MODE == kFull && on && a.h_in) h[k] = a.h_in[(b * a.C + c + e) * a.n + s];
        if (MODE == kFinal && on) h[k] = ws_h[((b * seg.count + sid) * a.C + c + e) * a.n + s];
      }
      A01[e] = pack2(A2[0], A2[1]);
      A23[e] = pack2(A2[2], A2[3]);
      h01[e] = pack2(h[0], h[1]);
      h23[e] = pack2(h[2], h[3]);
      dt_sum[e] = 0.f;
    }
    int dt_at[T::kPeriod], y_at[T::kPeriod];
#pragma unroll
    for (int r = 0; r < T::kPeriod; ++r) {
      dt_at[r] = T::dt_at(r, p * kCh);
      y_at[r] = T::y_at(r, p * kCh) * L + l;
    }
    struct In {
      float dt[kCh], dtu[kCh];
      LaneBC bc;
    };
    // A lane's states share a centre, that of the slowest: a pair of registers for each state took 848 us for the prompt
    // above, one centre for all states and tokens 809, this 818.  A tile's goes by the last step of the tile before, the
    // first tile's by its own first step.
    f32x2 centre;
    auto centre_by = [&](const float (&dt)[kCh]) {
      const float m = centre_of(slowest * fminf(fabsf(dt[0]), fabsf(dt[kCh - 1])));
      centre = pack2(m, m);
    };
    __syncthreads();  // tile 0 is laid out
    {
      float dt[kCh];
#pragma unroll
      for (int e = 0; e < kCh; ++e) dt[e] = sm.work[0].dt[0][dt_at[0] + e].x;
      centre_by(dt);
    }
    for (int i = 0; i < count; ++i) {
      typename T::Work& q = sm.work[i & 1];
      auto read = [&](int r) {
        In x;
        if constexpr (kCh == 1) {
          const float2 d = q.dt[r][dt_at[r % T::kPeriod]];
          x.dt[0] = d.x;
          x.dtu[0] = d.y;
        } else {
          const float4 d = *reinterpret_cast<const float4*>(&q.dt[r][dt_at[r % T::kPeriod]]);
          x.dt[0] = d.x;
          x.dtu[0] = d.y;
          x.dt[kCh - 1] = d.z;
          x.dtu[kCh - 1] = d.w;
        }
        x.bc = q.bc[r][l];
        return x;
      };
      In cur[kAhead], next[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) cur[k] = read(k);
#pragma unroll
      for (int r = 0; r < TT; r += kAhead) {
        if (r + kAhead < TT) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k) next[k] = read(r + kAhead + k);
        }
        float y[kAhead][kCh];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int e = 0; e < kCh; ++e) {
            const In& x = cur[k];
            const f32x2 dt2 = pack2(x.dt[e], x.dt[e]), dtu2 = pack2(x.dtu[e], x.dtu[e]);
            h01[e] = fma2(ex2_2(fma2(dt2, A01[e], centre)), h01[e], mul2(dtu2, x.bc.b.x));
            h23[e] = fma2(ex2_2(fma2(dt2, A23[e], centre)), h23[e], mul2(dtu2, x.bc.b.y));
            if constexpr (MODE == kLocal) {
              dt_sum[e] += x.dt[e];
            } else {
              float lo, hi;
              unpack2(fma2(x.bc.c.y, h23[e], mul2(x.bc.c.x, h01[e])), lo, hi);
              y[k][e] = lo + hi;
            }
          }
        if constexpr (MODE != kLocal) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int e = 0; e < kCh; ++e) q.y[e][r + k][y_at[(r + k) % T::kPeriod]] = y[k][e];
        }
        if (r + kAhead < TT) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k) cur[k] = next[k];
        }
      }
      centre_by(cur[kAhead - 1].dt);
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < kCh; ++e) {
      float h[kK];
      unpack2(h01[e], h[0], h[1]);
      unpack2(h23[e], h[2], h[3]);
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int s = l * kK + k;
        if (c + e < c_end && s < a.n) {
          if (MODE == kLocal) ws_h[((b * seg.count + sid) * a.C + c + e) * a.n + s] = h[k];
          else if (MODE == kFull || sid == seg.count - 1) a.h_out[(b * a.C + c + e) * a.n + s] = h[k];
        }
      }
      if (MODE == kLocal && l == 0 && c + e < c_end) ws_dt[(b * seg.count + sid) * a.C + c + e] = dt_sum[e];
    }
    return;
  }

  // A layout or output thread's vectors of a tile: rows r0 + i RS, V channels from v0 on.
  constexpr int V = kVec<TIn>, VPR = CT / V;
  const int ht = tid < kScan + kLayout ? tid - kScan : tid - kScan - kLayout;
  const int r0 = ht / VPR, v0 = ht % VPR * V;
  const int64_t cv = c_base + v0;
  const int valid = (int)max((int64_t)0, min((int64_t)V, c_end - cv));
  const bool gate = MODE != kLocal && a.z != nullptr;

  if (tid < kScan + kLayout) {
    // ================================================================ layout warps
    constexpr int RS = kLayout / VPR, NVI = (TT + RS - 1) / RS;
    auto slot = [&](int i) { return ((r0 + i * RS) * VPR + ht % VPR) * V; };  // of vector i in a raw tile
    auto in_tile = [&](int i) { return TT % RS == 0 || r0 + i * RS < TT; };
    constexpr int NP = L * kK, BS = kLayout / NP, NB = (TT + BS - 1) / BS;  // a thread's elements of B and C: BS rows apart
    // rows are 16-byte aligned, but a group's first channel may not be, nor rows of B and C
    const bool vec = (c_base * sizeof(TIn)) % 16 == 0 && valid == V;
    const int rb = ht / NP, sb = ht % NP;
    const TIn* u_p = reinterpret_cast<const TIn*>(a.u) + b * a.u_sb + (t0 + r0) * a.u_st + cv;
    const TIn* d_p = reinterpret_cast<const TIn*>(a.delta) + b * a.d_sb + (t0 + r0) * a.d_st + cv;
    const TIn* z_p = reinterpret_cast<const TIn*>(a.z) + b * a.z_sb + (t0 + r0) * a.z_st + cv;
    const TIn* B_p = reinterpret_cast<const TIn*>(a.Bm.ptr) + b * a.Bm.sb + g * a.Bm.sh + t0 * a.Bm.st;
    const TIn* C_p = reinterpret_cast<const TIn*>(a.Cm.ptr) + b * a.Cm.sb + g * a.Cm.sh + t0 * a.Cm.st;
    const bool bc_vec = a.n == NP && ((reinterpret_cast<uintptr_t>(B_p) | reinterpret_cast<uintptr_t>(C_p) |
                                       (uintptr_t)((a.Bm.st | a.Cm.st) * (int64_t)sizeof(TIn))) & 15u) == 0 && NP % V == 0;
    float bias[V];
    int dt_at[NVI][V / 2];  // where the channels of a vector lie in a tile
#pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = a.delta_bias && j < valid ? a.delta_bias[cv + j] : 0.f;
#pragma unroll
    for (int i = 0; i < NVI; ++i)
#pragma unroll
      for (int j = 0; j < V; j += 2) dt_at[i][j / 2] = (r0 + i * RS) * CT + T::dt_at(r0 + i * RS, v0 + j);

    // one vector of a raw tile: asynchronously, or by elements where it is partial or not aligned
    auto copy = [&](TIn* dst, const TIn* src, int n, bool whole) {
      if (whole) tc::cp_async16(tc::smem_u32(dst), src, 16u);
      else *reinterpret_cast<uint4*>(dst) = load_raw(src, n, false);
    };
    auto fetch = [&](int k) {  // raw inputs of tile k; what lies behind the end is not read
      if (k < count) {
        typename T::Raw& w = sm.raw[k % T::kRaw];
        const int left = tokens - k * TT;
#pragma unroll
        for (int i = 0; i < NVI; ++i) {
          const int r = k * TT + i * RS;
          if (in_tile(i) && r0 + i * RS < left && valid > 0) {
            copy(w.u + slot(i), u_p + r * a.u_st, valid, vec);
            copy(w.delta + slot(i), d_p + r * a.d_st, valid, vec);
            if (gate) copy(w.z + slot(i), z_p + r * a.z_st, valid, vec);
          }
        }
        if (bc_vec) {
          constexpr int per = NP / V > 0 ? NP / V : 1;  // vectors per row
          for (int e = ht; e < 2 * TT * per; e += kLayout) {
            const int m = e / (TT * per), r = e / per % TT, v = e % per * V;
            if (r < left && (MODE != kLocal || m == 0))
              copy(w.bc[m] + r * NP + v, (m ? C_p + (int64_t)(k * TT + r) * a.Cm.st : B_p + (int64_t)(k * TT + r) * a.Bm.st) + v, V, true);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const int r = rb + i * BS;
            if (r < TT && r < left && sb < a.n) {
              w.bc[0][r * NP + sb] = B_p[(int64_t)(k * TT + r) * a.Bm.st + sb];
              if (MODE != kLocal) w.bc[1][r * NP + sb] = C_p[(int64_t)(k * TT + r) * a.Cm.st + sb];
            }
          }
        }
      }
      tc::cp_async_commit();  // a group per tile, also for none
    };
    auto lay_out = [&](int k) {  // a token behind the end changes nothing (dt = 0, B = C = 0)
      const typename T::Raw& w = sm.raw[k % T::kRaw];
      typename T::Work& q = sm.work[k & 1];
      const int left = tokens - k * TT;
#pragma unroll
      for (int i = 0; i < NVI; ++i) {
        if (!in_tile(i)) continue;
        float fu[V], fd[V], dt[V];
        const bool on = r0 + i * RS < left && valid > 0;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        unpack_vec(on ? *reinterpret_cast<const uint4*>(w.u + slot(i)) : zero, fu);
        unpack_vec(on ? *reinterpret_cast<const uint4*>(w.delta + slot(i)) : zero, fd);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float x = fd[j] + bias[j];
          dt[j] = a.softplus ? softplus(x) : x;
          if (!on) dt[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < V; j += 2)
          *reinterpret_cast<float4*>(&q.dt[0][0] + dt_at[i][j / 2]) = make_float4(dt[j], dt[j] * fu[j], dt[j + 1], dt[j + 1] * fu[j + 1]);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int r = rb + i * BS;
        if (TT % BS != 0 && r >= TT) continue;
        const bool on = r < left && sb < a.n;
        float* x = reinterpret_cast<float*>(&q.bc[r][sb / kK]) + sb % kK;
        x[0] = on ? to_f(w.bc[0][r * NP + sb]) : 0.f;
        if (MODE != kLocal) x[kK] = on ? to_f(w.bc[1][r * NP + sb]) : 0.f;
      }
    };
    // Tile k is on its way from iteration k - kAheadTiles on; its raw inputs stay until its outputs are
    // stored in iteration k + 1.  The four layout warps exchange B and C among themselves: barrier 1.
    constexpr int kAheadTiles = T::kRaw - 2;
    for (int k = 0; k < kAheadTiles; ++k) fetch(k);
    auto arrived = [&]() {  // the oldest of kAheadTiles groups has landed, for all layout warps
      asm volatile("cp.async.wait_group %0;" ::"n"(kAheadTiles - 1) : "memory");
      tc::named_bar_sync(1, kLayout);
    };
    arrived();
    if (count > 0) lay_out(0);
    __syncthreads();  // tile 0 is laid out
    for (int i = 0; i < count; ++i) {
      fetch(i + kAheadTiles);
      arrived();
      if (i + 1 < count) lay_out(i + 1);
      __syncthreads();
    }
    tc::cp_async_wait_all();
  } else {
    // ================================================================ output warps
    constexpr int RS = kOutput / VPR, NVI = (TT + RS - 1) / RS;
    auto slot = [&](int i) { return ((r0 + i * RS) * VPR + ht % VPR) * V; };
    auto in_tile = [&](int i) { return TT % RS == 0 || r0 + i * RS < TT; };
    TOut* y_p = reinterpret_cast<TOut*>(a.y) + b * a.y_sb + (t0 + r0) * a.y_st + cv;
    const bool yvec = c_base % V == 0;
    float skip[V];
    int y_at[NVI][V];
#pragma unroll
    for (int j = 0; j < V; ++j) skip[j] = MODE != kLocal && a.D && j < valid ? a.D[cv + j] : 0.f;
#pragma unroll
    for (int i = 0; i < NVI; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int r = r0 + i * RS;
        y_at[i][j] = ((v0 + j) % kCh) * (TT * kScan) + r * kScan + T::y_at(r, v0 + j) * L;
      }
    auto store = [&](int k) {  // readout, skip term and gate of tile k
      const typename T::Raw& w = sm.raw[k % T::kRaw];
      const typename T::Work& q = sm.work[k & 1];
#pragma unroll
      for (int i = 0; i < NVI; ++i) {
        if (!in_tile(i) || r0 + i * RS >= tokens - k * TT || valid == 0) continue;
        float fu[V], fz[V], o[V];
        unpack_vec(*reinterpret_cast<const uint4*>(w.u + slot(i)), fu);
        if (gate) unpack_vec(*reinterpret_cast<const uint4*>(w.z + slot(i)), fz);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float* part = &q.y[0][0][0] + y_at[i][j];
          float y;
          if constexpr (L >= 4) {
            y = 0.f;
#pragma unroll
            for (int e = 0; e < L; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(part + e);
              y += (x.x + x.y) + (x.z + x.w);
            }
          } else if constexpr (L == 2) {
            y = part[0] + part[1];
          } else {
            y = part[0];
          }
          y = fmaf(skip[j], fu[j], y);
          o[j] = gate ? y * silu(fz[j]) : y;
        }
        store_floats(y_p + (int64_t)(k * TT + i * RS) * a.y_st, o, valid, yvec);
      }
    };
    __syncthreads();  // tile 0 is laid out
    for (int i = 0; i < count; ++i) {
      if (MODE != kLocal && i > 0) store(i - 1);
      __syncthreads();
    }
    if (MODE != kLocal && count > 0) store(count - 1);
  }
}

// The state that enters each segment, in place of the segment's local state: over a segment a state
// decays by exp(A * sum of dt).  A state may grow too, and over a segment by more than fp32 holds: the factor comes in two
// halves, and a state of zero, which a token's finite factors leave at zero, takes none.
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
    const float half = ex2(0.5f * (A2 * d[(int64_t)g * a.C]));
    h = h == 0.f ? local : fmaf(half * h, half, local);
  }
  p[(seg.count - 1) * per] = h;
}

// ---------------------------------------------------------------------------------------------- one token
// The step reads and writes each state once, which bounds it: 256 x 4096 x 16 takes 25 us, 5.7 TB/s, 85 % of the
// measured copy rate (33 us with the loads behind the arithmetic that uses them).  L lanes share a channel, four states a lane, for
// four sequences at a time: A, D and the bias are loaded once for them, the four states' loads are in flight
// together, and of the channel's lanes each computes the step size and the gate of a sequence of its own.
constexpr int kStepThreads = 256;
constexpr int kStepSeqs = 4;

template <int L, typename TIn, typename TOut>
__global__ void __launch_bounds__(kStepThreads)
ssm_decode_kernel(const SsmLaunch a, bool a_vec, bool bc_vec) {
  constexpr int NQ = L >= kStepSeqs ? 1 : kStepSeqs / L;  // sequences whose gates this lane computes
  const int tid = threadIdx.x, l = tid % L;
  const int64_t c = (int64_t)blockIdx.x * (kStepThreads / L) + tid / L;
  const int64_t s0 = (int64_t)blockIdx.y * kStepSeqs;
  const bool live = c < a.C;
  const int64_t cc = live ? c : 0;
  const int g = a.G == 1 ? 0 : (int)cc / ((int)a.C / (int)a.G);  // channels are 32-bit here
  const int s_lo = l * kK, count = max(0, min(kK, a.n - s_lo));
  const bool on = live && count > 0, vec = a_vec;
  const int q_own = L >= kStepSeqs ? l / (L >= kStepSeqs ? L / kStepSeqs : 1) : l * NQ;
  grid_dependents_trigger();
  grid_dependency_wait();  // the states and this step's inputs are in memory
  float h[kStepSeqs][kK];
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
#pragma unroll
    for (int k = 0; k < kK; ++k) h[q][k] = 0.f;
    if (on && s0 + q < a.B) {
      const float* p = a.h_in + ((s0 + q) * a.C + cc) * a.n + s_lo;
      if (vec) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
        h[q][0] = x.x; h[q][1] = x.y; h[q][2] = x.z; h[q][3] = x.w;
      } else {
#pragma unroll
        for (int k = 0; k < kK; ++k) h[q][k] = k < count ? p[k] : 0.f;
      }
    }
  }
  // everything else that the step reads, behind the states and before any of it is used
  Raw4<TIn> Br[kStepSeqs], Cr[kStepSeqs];
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int64_t s = min(s0 + q, a.B - 1);
    const TIn* Bp = reinterpret_cast<const TIn*>(a.Bm.ptr) + s * a.Bm.sb + g * a.Bm.sh + s_lo;
    const TIn* Cp = reinterpret_cast<const TIn*>(a.Cm.ptr) + s * a.Cm.sb + g * a.Cm.sh + s_lo;
    if (bc_vec && count > 0) {
      Br[q].load(Bp);
      Cr[q].load(Cp);
    } else {
      Br[q].load(Bp, count);
      Cr[q].load(Cp, count);
    }
  }
  float u_own[NQ], dt_own[NQ], z_own[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int64_t s = min(s0 + q_own + i, a.B - 1);
    u_own[i] = to_f(reinterpret_cast<const TIn*>(a.u)[s * a.u_sb + cc]);
    dt_own[i] = to_f(reinterpret_cast<const TIn*>(a.delta)[s * a.d_sb + cc]);
    z_own[i] = a.z ? to_f(reinterpret_cast<const TIn*>(a.z)[s * a.z_sb + cc]) : 0.f;
  }
  const float bias = a.delta_bias ? a.delta_bias[cc] : 0.f, skip = a.D ? a.D[cc] : 0.f;
  float A2[kK];
  if (vec && count > 0) {
    const float4 x = *reinterpret_cast<const float4*>(a.A + cc * a.n + s_lo);
    A2[0] = log2_rate(x.x); A2[1] = log2_rate(x.y); A2[2] = log2_rate(x.z); A2[3] = log2_rate(x.w);
  } else {
#pragma unroll
    for (int k = 0; k < kK; ++k) A2[k] = k < count ? log2_rate(a.A[cc * a.n + s_lo + k]) : 0.f;
  }
  float slowest = INFINITY;  // of the lane's states, which share a centre
#pragma unroll
  for (int k = 0; k < kK; ++k) slowest = k < count ? fminf(slowest, fabsf(A2[k])) : slowest;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const float x = dt_own[i] + bias;
    dt_own[i] = a.softplus ? softplus(x) : x;
  }
  float acc[kStepSeqs];
  const int group_lane = (tid & 31) - l;
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int src = group_lane + (L >= kStepSeqs ? q * (L / kStepSeqs) : q / NQ);
    const float dt = L == 1 ? dt_own[q % NQ] : __shfl_sync(kFullMask, dt_own[q % NQ], src);
    const float u = L == 1 ? u_own[q % NQ] : __shfl_sync(kFullMask, u_own[q % NQ], src);
    float Bk[kK], Ck[kK];
    Br[q].unpack(Bk);
    Cr[q].unpack(Ck);
    const float dtu = dt * u, centre = centre_of(dt * slowest);
    acc[q] = 0.f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      h[q][k] = fmaf(ex2(fmaf(dt, A2[k], centre)), h[q][k], dtu * Bk[k]);
      acc[q] = fmaf(Ck[k], h[q][k], acc[q]);
    }
    if (on && s0 + q < a.B) {
      float* p = a.h_out + ((s0 + q) * a.C + cc) * a.n + s_lo;
      if (vec) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(h[q][0], h[q][1], h[q][2], h[q][3]));
      } else {
#pragma unroll
        for (int k = 0; k < kK; ++k)
          if (k < count) p[k] = h[q][k];
      }
    }
  }
  // sums over the channel's lanes, each ending with its own sequences'
  float y[NQ];
  if constexpr (L == 1) {
#pragma unroll
    for (int q = 0; q < kStepSeqs; ++q) y[q % NQ] = acc[q];
  } else {
    const bool up = (l & (L / 2)) != 0;
    float p0 = up ? acc[2] : acc[0], p1 = up ? acc[3] : acc[1];
    p0 += __shfl_xor_sync(kFullMask, up ? acc[0] : acc[2], L / 2);
    p1 += __shfl_xor_sync(kFullMask, up ? acc[1] : acc[3], L / 2);
    if constexpr (L == 2) {
      y[0] = p0;
      y[NQ - 1] = p1;
    } else {
      const bool up2 = (l & (L / 4)) != 0;
      y[0] = (up2 ? p1 : p0) + __shfl_xor_sync(kFullMask, up2 ? p0 : p1, L / 4);
#pragma unroll
      for (int off = L / 8; off >= 1; off >>= 1) y[0] += __shfl_xor_sync(kFullMask, y[0], off);
    }
  }
  if (live && (L < kStepSeqs || l % (L >= kStepSeqs ? L / kStepSeqs : 1) == 0)) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int64_t s = s0 + q_own + i;
      if (s < a.B) {
        float o = fmaf(skip, u_own[i], y[i]);
        if (a.z) o *= silu(z_own[i]);
        store1(reinterpret_cast<TOut*>(a.y) + s * a.y_sb + c, o);
      }
    }
  }
}

// Blocks of one sequence batch with `ch` channels per lane.
int64_t scan_blocks(int64_t B, int64_t C, int n, int64_t G, int ch) {
  const int CT = ch * kScan / lanes_of(n);
  return B * G * ((C / G + CT - 1) / CT);
}

Segments plan(int64_t B, int64_t N, int64_t C, int n, int64_t G) {
  // A segmented scan does the exponentials twice, so it pays from about three segments' worth of idle SMs
  // on, and segments of a few tiles at least.
  constexpr int kTile = 32;
  const int64_t want = std::min<int64_t>(304 / std::max<int64_t>(scan_blocks(B, C, n, G, 1), 1), N / (4 * kTile));
  if (want < 3) return Segments{1, N};
  const int64_t len = ((N + want - 1) / want + kTile - 1) / kTile * kTile;
  return Segments{(int)((N + len - 1) / len), len};
}

template <int L, int kCh, typename TIn, typename TOut, int MODE>
cudaError_t launch_mode(const SsmLaunch& a, const Segments& seg, int segments, float* ws_h, float* ws_dt, cudaStream_t stream) {
  using T = Tile<L, kCh, TIn>;
  const auto kernel = ssm_scan_kernel<L, kCh, TIn, TOut, MODE>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, (int)sizeof(T), done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.G * ((a.C / a.G + T::CT - 1) / T::CT)), (unsigned)a.B, (unsigned)segments);
  kernel<<<grid, block_threads(kCh), sizeof(T), stream>>>(a, seg, ws_h, ws_dt);
  return cudaGetLastError();
}

template <int L, typename TIn, typename TOut>
cudaError_t launch_scan(const SsmLaunch& a, void* ws, const Segments& seg, cudaStream_t stream) {
  if (seg.count == 1) {
    return scan_blocks(a.B, a.C, a.n, a.G, 1) > 152 ? launch_mode<L, 2, TIn, TOut, kFull>(a, seg, 1, nullptr, nullptr, stream)
                                                    : launch_mode<L, 1, TIn, TOut, kFull>(a, seg, 1, nullptr, nullptr, stream);
  }
  float* ws_h = static_cast<float*>(ws);
  float* ws_dt = ws_h + a.B * seg.count * a.C * a.n;
  cudaError_t e = launch_mode<L, 1, TIn, float, kLocal>(a, seg, seg.count - 1, ws_h, ws_dt, stream);  // nothing enters from the last
  if (e != cudaSuccess) return e;
  const int64_t states = a.B * a.C * a.n;
  ssm_combine_kernel<<<(unsigned)((states + 255) / 256), 256, 0, stream>>>(a, seg, ws_h, ws_dt);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_mode<L, 1, TIn, TOut, kFinal>(a, seg, seg.count, ws_h, ws_dt, stream);
}

template <typename TIn, typename TOut>
cudaError_t launch_lanes(const SsmLaunch& a, void* ws, const Segments* seg, cudaStream_t stream) {
  // four states of B and C in one load: rows of whole quadruples on their boundary
  constexpr int64_t quad = 4 * (int64_t)sizeof(TIn);
  const bool a_vec = a.n % kK == 0 && (reinterpret_cast<uintptr_t>(a.A) & 15u) == 0;
  const bool bc_vec = a.n % kK == 0 && ((reinterpret_cast<uintptr_t>(a.Bm.ptr) | reinterpret_cast<uintptr_t>(a.Cm.ptr) |
                                         (uintptr_t)((a.Bm.sb | a.Bm.sh | a.Cm.sb | a.Cm.sh) * (int64_t)sizeof(TIn))) % quad) == 0;
  auto step = [&](auto kernel, int L) {
    const int64_t per = kStepThreads / L;
    const dim3 grid((unsigned)((a.C + per - 1) / per), (unsigned)((a.B + kStepSeqs - 1) / kStepSeqs));
    return launch_dependent(kernel, grid, dim3(kStepThreads), 0, stream, a, a_vec, bc_vec);
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
