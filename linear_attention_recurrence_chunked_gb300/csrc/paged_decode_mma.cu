// paged_decode_mma.cu -- a step over bf16 pages and over 4-bit pages.
//
// A key row meets up to 16 query heads, too many operations for the CUDA cores beside the loads and too few rows for
// tcgen05, so the products are mma.m16n8k16 with the heads as the 16 rows, as in swa_biased_decode.cu.  Each warp takes
// tiles of its block's part in turn, through a ring of its own in shared memory that asynchronous copies fill, with the
// running maximum and sum of its tokens; no warp waits for another before the end, where their sums meet.  A tile's pages
// are looked up one tile (4 bits: sixteen tiles) ahead of its copies.  256 sequences of up to 8192 tokens, 32 heads over 4 and
// d = 128 in bf16 take 391 us, the measured copy rate; of up to 16384 tokens in 4 bits 398 us, 56 % of it: 920 warp
// instructions for 32 tokens, of which 290 turn codes into bf16, at 2.2 a clock.  With 64 heads over 4, 128 sequences take
// 231 us in bf16 (86 %) and 322 in 4 bits (35 %, 144 bytes a thread spilled).
//
// The running maximum moves only where a score is more than 2^kSlack times beyond it: until then weights are up to 2^kSlack,
// which costs fp32 sums nothing, and the sums of values need not be scaled.
//
// Weights (in 4 bits times their value's scale) are split into bf16 parts for their product with the values.  Two leave them
// off by 2^-17, a 500th of a bf16 output's own half step.  An fp32 output would show it (1.5e-6 of an output's norm over
// 8192 tokens, where PyTorch in fp32 is off by 6e-7), so it takes three, off by less than fp32's own rounding (5.5e-7): 395 us
// instead of 391 for the bf16 batch above, 446 instead of 398 for the one in 4 bits; bf16 steps with 16 heads a key head 5 %,
// with one of d = 64 11 %.  Its capped scores take a term more for the same reason (4e-6 of the norm with a cap of 30, 7e-7 so).
//
// 4 bits: scales and offsets meet whole sums of codes in fp32 (keys), and weights once per group (values):
//   q.k = sum over groups of scale (q.code) + offset sum q
//   sum_j p_j v_j = sum_j (16 scale_j p_j) (code_j - 8) / 16 + sum_j p_j (offset_j + 8 scale_j)
// A key's code is the last bits of a bf16 number, a whole number of 2^-133, which takes a mask, and a head's query is scaled up by
// a power of two to match (398 us; 415 with keys made like values).  A value's code is put into the mantissa of a one,
// 1 + code / 16, and less 3/2: sums over thousands of tokens of centred codes come out near zero, while sums of ones would not
// (off by 5e-4 of an output's norm over 131071 tokens, where tensor cores cut sums off; 2 to 4e-6 centred, fp32 outputs).  Values as whole numbers
// too, weights scaled by the largest scale so far, took 1 % off for a rescaling and more spilled registers.
#include <algorithm>

#include "paged_decode.cuh"
#include "tc.cuh"

namespace la {
namespace {

constexpr int kMostWarps = 4;  // of a block: this many, or one
constexpr float kSlack = 8.f;
constexpr uint32_t kTiny = 0x00010001u;  // two bf16 2^-133
template <typename TOut>
constexpr bool kFine = sizeof(TOut) == 4;  // weights in three parts, not two; caps to fp32

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two values as bf16, and what that leaves of them as bf16: together off by 2^-17 of a value.
__device__ __forceinline__ void two_parts(float lo, float hi, uint32_t& major, uint32_t& minor) {
  major = tc::pack2_bf16(lo, hi);
  minor = tc::pack2_bf16(lo - __uint_as_float(major << 16), hi - __uint_as_float(major & 0xffff0000u));
}

// ... and what both leave, as bf16: together off by 2^-26 of a value.  `three` false: last stays as it is.
template <bool three>
__device__ __forceinline__ void in_parts(float lo, float hi, uint32_t& major, uint32_t& minor, uint32_t& last) {
  two_parts(lo, hi, major, minor);
  if constexpr (three)
    last = tc::pack2_bf16(lo - __uint_as_float(major << 16) - __uint_as_float(minor << 16),
                          hi - __uint_as_float(major & 0xffff0000u) - __uint_as_float(minor & 0xffff0000u));
}

// Two bf16 values, zero in the place of what is not finite.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// What every warp of a block knows.
struct Part {
  int64_t s, hk, h0;
  int group, part, first, last;  // tokens [first, last), first a multiple of kTile
  SeenTokens seen;
};
// False: nothing to do.
__device__ __forceinline__ bool part_of(const PagedDecodeLaunch& a, Part& p) {
  p.part = (int)(blockIdx.x % a.splits);
  const int64_t rest = blockIdx.x / a.splits;
  p.s = rest / a.c.Hkv;
  p.hk = rest - p.s * a.c.Hkv;
  p.group = (int)(a.H / a.c.Hkv);
  p.h0 = p.hk * p.group;
  p.seen = seen_tokens(a, p.s);
  if (p.seen.hi < 0 && p.part == 0 && p.hk == 0 && threadIdx.x == 0) atomicOr(a.c.status, kStatusBadIndex);
  if (p.seen.hi < 0 || p.part >= max(p.seen.parts, 1)) return false;
  p.first = (p.seen.lo / kTile + p.part * p.seen.tiles) * kTile;
  p.last = min(p.seen.hi, p.first + p.seen.tiles * kTile);
  return true;
}

// The running softmax of a warp: rows lane / 4 (0) and that + 8 (1), a quad's lanes with the same maximum and sums of their own.
// No score is below the first maximum but -infinity, whose weight is zero beside any.
struct Running {
  float m[2] = {-3.402823466e38f, -3.402823466e38f}, l[2] = {0.f, 0.f};
};

// Scores of T tiles of eight tokens into weights; f: the factors of the sums so far, and whether they are not one.
template <int T, int kRowsUsed>
__device__ __forceinline__ bool weigh(Running& r, float (&x)[T][4], float (&f)[2]) {
  bool moves = false;
  float top[2];
#pragma unroll
  for (int i = 0; i < kRowsUsed; ++i) {
    float y = x[0][2 * i];
#pragma unroll
    for (int t = 0; t < T; ++t) y = fmaxf(y, fmaxf(x[t][2 * i], x[t][2 * i + 1]));
    y = fmaxf(y, __shfl_xor_sync(kFullMask, y, 1));
    top[i] = fmaxf(y, __shfl_xor_sync(kFullMask, y, 2));
    moves |= top[i] > r.m[i] + kSlack;
  }
  moves = __any_sync(kFullMask, moves);
  if (moves) {
#pragma unroll
    for (int i = 0; i < kRowsUsed; ++i) {
      const float m = fmaxf(r.m[i], top[i]);
      f[i] = ex2(r.m[i] - m);
      r.m[i] = m;
      r.l[i] *= f[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsUsed; ++i) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int e = 2 * i; e < 2 * i + 2; ++e) {
        x[t][e] = ex2(x[t][e] - r.m[i]);
        r.l[i] += x[t][e];
      }
  }
  return moves;
}

// The warps' sums together and out: s_m, s_l [warp][16], `values` warp w's sums of row g at w * stride + g * d.
template <typename TOut, int kWarps>
__device__ __forceinline__ void finish(const PagedDecodeLaunch& a, const Part& p, const float (*s_m)[16], const float (*s_l)[16],
                                       const float* values, int stride) {
  const int d = a.c.d;
  for (int e = threadIdx.x * 2; e < p.group * d; e += 32 * kWarps * 2) {
    const int g = e / d, c = e - g * d;
    float top = s_m[0][g];
#pragma unroll
    for (int u = 1; u < kWarps; ++u) top = fmaxf(top, s_m[u][g]);
    float2 sum = make_float2(0.f, 0.f);
    float total = 0.f;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) {
      const float w = ex2(s_m[u][g] - top);
      const float2 y = *reinterpret_cast<const float2*>(values + u * stride + e);
      sum.x = fmaf(w, y.x, sum.x);
      sum.y = fmaf(w, y.y, sum.y);
      total = fmaf(w, s_l[u][g], total);
    }
    const int64_t h = p.h0 + g;
    if (a.splits > 1) {
      *reinterpret_cast<float2*>(part_values(a, p.s, h, p.part) + c) = sum;
      if (c == 0) *part_sums(a, p.s, h, p.part) = make_float2(top, total);
      continue;
    }
    sum = make_float2(mean_of(sum.x, total), mean_of(sum.y, total));
    TOut* to = static_cast<TOut*>(a.out) + p.s * a.o_sb + h * a.o_sh + c;
    if constexpr (sizeof(TOut) == 2) *reinterpret_cast<uint32_t*>(to) = tc::pack2_bf16(sum.x, sum.y);
    else *reinterpret_cast<float2*>(to) = sum;
  }
}

// What a product is multiplied by: scores are in units of log2, but in front of a cap.
__device__ __forceinline__ float score_scale(const PagedDecodeLaunch& a) { return a.softcap != 0.f ? a.scale : a.scale * kLog2e; }

// A warp's rows of scores: caps, biases and what is not seen.  tokens(t, e): of tile t, entry e's token's distance from the
// warp tile's first one.
template <bool fine, int T, int kRowsUsed, typename Tokens>
__device__ __forceinline__ void bias_and_mask(const PagedDecodeLaunch& a, float (&x)[T][4], const float (&slope)[2], float inv_cap, int age0,
                                              uint32_t seen, uint32_t whole, Tokens tokens) {
  auto each = [&](auto fn) {
#pragma unroll
    for (int i = 0; i < kRowsUsed; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int e = 2 * i; e < 2 * i + 2; ++e) x[t][e] = fn(x[t][e], i, t, e & 1);
  };
  if (a.softcap != 0.f) each([&](float y, int, int, int) { return (fine ? capped_fine(y, a.softcap, inv_cap) : capped(y, a.softcap, inv_cap)) * kLog2e; });
  if (a.slopes) each([&](float y, int i, int t, int e) { return fmaf(-slope[i], (float)(age0 - tokens(t, e)), y); });
  if (seen != whole) each([&](float y, int, int t, int e) { return seen >> tokens(t, e) & 1u ? y : -INFINITY; });
}

// Where a warp's tiles lie in the table: the tiles are `step` tokens apart, and a division at every one would cost as much as
// a product.
struct Place {
  int column, slot, step_columns, step_slots, page;
  __device__ __forceinline__ Place(int token, int step, int page_) : page(page_) {
    column = token / page;
    slot = token - column * page;
    step_columns = step / page;
    step_slots = step - step_columns * page;
  }
  __device__ __forceinline__ void advance() {
    column += step_columns;
    slot += step_slots;
    if (slot >= page) {
      slot -= page;
      ++column;
    }
  }
};

// Bits of the tokens [t0, t0 + n) that lie in [lo, hi).
__device__ __forceinline__ uint32_t token_bits(int t0, int n, int lo, int hi) {
  const int from = min(max(lo - t0, 0), n), to = min(max(hi - t0, 0), n);
  if (from >= to) return 0u;
  return (to == 32 ? 0xffffffffu : (1u << to) - 1u) & ~((1u << from) - 1u);
}

// ---------------------------------------------------------------------------------------------- bf16
// DP: width padded to 64 or 128.  kSpare: at most eight heads a group; the weights' second parts take rows 8 to 15.
template <int DP>
constexpr int kStages = DP == 128 ? 3 : 5;
template <int DP>
constexpr int kTileBytes = 2 * kTile * DP * 2;  // keys, then values
template <int DP>
constexpr int kSmem = kStages<DP> * kTileBytes<DP>;  // of a warp

template <typename TOut, int DP, bool kSpare, int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
paged_decode_bf16_kernel(const PagedDecodeLaunch a) {
  using T = __nv_bfloat16;
  constexpr int kRows = kSpare ? 1 : 2, kSteps = DP / 16, kChunks = DP / 8, kS = kStages<DP>;
  extern __shared__ __align__(128) uint8_t pd_smem[];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  __shared__ uint32_t s_seen[kWarps][kS];
  const int warp = kWarps > 1 ? threadIdx.x >> 5 : 0, lane = threadIdx.x & 31, row = lane >> 2, q4 = lane & 3;
  grid_dependents_trigger();
  grid_dependency_wait();
  Part p;
  if (!part_of(a, p)) return;
  const int d = a.c.d, page = a.c.page;
  uint8_t* region = pd_smem + warp * kS * kTileBytes<DP>;
  const uint32_t base = tc::smem_u32(region);
  // place of 16-byte chunk `ch` of row r: eight neighbouring rows meet eight different banks
  auto at = [](int r, int ch) { return (uint32_t)(r * (DP * 2) + ((ch ^ (r & 7)) << 4)); };

  const int tiles = p.last > p.first ? (p.last - p.first + kTile - 1) / kTile : 0;
  struct Next { int page, slot; };
  auto lookup = [&](Place& at, int i) {  // where this warp's i-th tile lies: page -1 behind the last one or where there is none
    Next n{-1, at.slot};
    if (warp + i * kWarps < tiles) {
      n.page = table_page(a.c, p.s, at.column);
      if (n.page < 0 && p.hk == 0 && lane == 0) atomicOr(a.c.status, kStatusBadIndex);
    }
    at.advance();
    return n;
  };
  auto fetch = [&](int i, int stage, Next n) {  // this warp's i-th tile into its stage
    const int t0 = p.first + (warp + i * kWarps) * kTile;
    const uint32_t seen = n.page < 0 ? 0u : token_bits(t0, kTile, p.seen.lo, p.last);
    if (lane == 0) s_seen[warp][stage] = seen;
    if (n.page < 0) return;
    const int64_t from = ((n.page * a.c.Hkv + p.hk) * page + n.slot) * d;
    const uint32_t to = base + stage * kTileBytes<DP>;
#pragma unroll
    for (int j = 0; j < kTile * kChunks / 32; ++j) {
      const int e = lane + 32 * j, r = e / kChunks, ch = e % kChunks;
      const bool on = (seen >> r & 1u) && ch * 8 < d;  // what is not seen becomes zeros: a weight of zero times NaN is NaN
      const int64_t off = from + r * d + (ch * 8 < d ? ch * 8 : 0);
      tc::cp_async16(to + at(r, ch), static_cast<const T*>(a.c.k) + off, on ? 16u : 0u);
      tc::cp_async16(to + kTileBytes<DP> / 2 + at(r, ch), static_cast<const T*>(a.c.v) + off, on ? 16u : 0u);
    }
  };

  // ---- queries as operands
  uint32_t qa[kSteps][2 * kRows];
  float slope[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int g = row + 8 * i;
    const T* q = static_cast<const T*>(a.q.ptr) + p.s * a.q.sb + (p.h0 + (g < p.group ? g : 0)) * a.q.sh;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int col = 16 * k + 8 * u + 2 * q4;
        qa[k][i * 2 + u] = g < p.group && col < d ? *reinterpret_cast<const uint32_t*>(q + col) : 0u;
      }
    if (a.slopes && g < p.group) slope[i] = a.slopes[p.h0 + g] * kLog2e;
  }
  const float scale = score_scale(a), inv_cap = 1.f / a.softcap;

  float o[2 * kSteps][4];
  Running run;
  const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
  for (bool guarded = false;; guarded = true) {
#pragma unroll
    for (int t = 0; t < 2 * kSteps; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    Place place(p.first + warp * kTile, kWarps * kTile, page);
    Next next = lookup(place, 0);
#pragma unroll
    for (int i = 0; i < kS - 1; ++i) {
      if (i < mine) fetch(i, i, next);
      tc::cp_async_commit();
      next = lookup(place, i + 1);
    }
    for (int i = 0, stage = 0, into = kS - 1; i < mine; ++i, stage = stage + 1 == kS ? 0 : stage + 1, into = into + 1 == kS ? 0 : into + 1) {
      cp_async_wait<kS - 2>();
      __syncwarp();  // every lane's copies of this tile are in, and its reads of the stage that is filled next are done
      if (i + kS - 1 < mine) fetch(i + kS - 1, into, next);
      tc::cp_async_commit();
      next = lookup(place, i + kS);
      const uint32_t keys = base + stage * kTileBytes<DP>, vals = keys + kTileBytes<DP> / 2;
      const uint32_t seen = s_seen[warp][stage];
      if (seen == 0u) continue;
      float x[2][4];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t b[4];
        ldmatrix(b, keys + at((lane >> 4) * 8 + (lane & 7), 2 * k + ((lane >> 3) & 1)));
        const uint32_t a0 = qa[k][0], a1 = kSpare ? 0u : qa[k][2 * kRows - 2], a2 = qa[k][1], a3 = kSpare ? 0u : qa[k][2 * kRows - 1];
        if (k == 0) {
          mma16816_first(x[0], a0, a1, a2, a3, b[0], b[1]);
          mma16816_first(x[1], a0, a1, a2, a3, b[2], b[3]);
        } else {
          mma16816(x[0], a0, a1, a2, a3, b[0], b[1]);
          mma16816(x[1], a0, a1, a2, a3, b[2], b[3]);
        }
      }
      const int t0 = p.first + (warp + i * kWarps) * kTile;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2 * kRows; ++e) x[t][e] *= scale;
      bias_and_mask<kFine<TOut>, 2, kRows>(a, x, slope, inv_cap, p.seen.hi - 1 - t0, seen, 0xffffu, [&](int t, int e) { return t * 8 + q4 * 2 + e; });
      float f[2];
      if (weigh<2, kRows>(run, x, f)) {
#pragma unroll
        for (int t = 0; t < 2 * kSteps; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] *= f[kSpare ? 0 : e >> 1];
      }
      uint32_t w[4], z[4], y[4];  // first, second and third parts: rows row and row + 8 of tile 0, then of tile 1
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < kRows; ++u) in_parts<kFine<TOut>>(x[t][2 * u], x[t][2 * u + 1], w[2 * t + u], z[2 * t + u], y[2 * t + u]);
      if constexpr (kSpare) {
        w[1] = z[0];
        w[3] = z[2];
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t b[4];
        ldmatrix_trans(b, vals + at(((lane >> 3) & 1) * 8 + (lane & 7), 2 * k + (lane >> 4)));
        mma16816(o[2 * k], w[0], w[1], w[2], w[3], b[0], b[1]);
        mma16816(o[2 * k + 1], w[0], w[1], w[2], w[3], b[2], b[3]);
        if constexpr (kSpare && kFine<TOut>) {
          // Third parts in the second ones' rows; what the other rows get is nothing beside a weight, and keeps infinities.
          mma16816(o[2 * k], kTiny, y[0], kTiny, y[2], b[0], b[1]);
          mma16816(o[2 * k + 1], kTiny, y[0], kTiny, y[2], b[2], b[3]);
        }
        if constexpr (!kSpare) {
          if (guarded) {
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = finite_or_zero(b[e]);
          }
          mma16816(o[2 * k], z[0], z[1], z[2], z[3], b[0], b[1]);
          mma16816(o[2 * k + 1], z[0], z[1], z[2], z[3], b[2], b[3]);
          if constexpr (kFine<TOut>) {
            mma16816(o[2 * k], y[0], y[1], y[2], y[3], b[0], b[1]);
            mma16816(o[2 * k + 1], y[0], y[1], y[2], y[3], b[2], b[3]);
          }
        }
      }
    }
    tc::cp_async_wait_all();
    __syncwarp();
    // What second parts make of a value that is not finite is left out: the first ones' result stands.  With rows of their
    // own they are added here; otherwise the warp's tiles are gone through again with zeros for such values in their product.
    if constexpr (kSpare) {
#pragma unroll
      for (int t = 0; t < 2 * kSteps; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[t][e] += finite1(o[t][2 + e]) ? o[t][2 + e] : 0.f;
      break;
    } else {
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 2 * kSteps; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = fmaf(0.f, o[t][e], sum);
      if (guarded || __all_sync(kFullMask, sum == 0.f)) break;
      run = Running();
    }
  }
  // ---- this warp's sums into its place
  float* part = reinterpret_cast<float*>(region);
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    float l = run.l[u];
    l += __shfl_xor_sync(kFullMask, l, 1);
    l += __shfl_xor_sync(kFullMask, l, 2);
    if (q4 == 0) {
      s_m[warp][row + 8 * u] = run.m[u];
      s_l[warp][row + 8 * u] = l;
    }
    if (row + 8 * u < p.group) {
#pragma unroll
      for (int t = 0; t < 2 * kSteps; ++t)
        if (t * 8 < d) *reinterpret_cast<float2*>(part + (row + 8 * u) * d + t * 8 + q4 * 2) = make_float2(o[t][2 * u], o[t][2 * u + 1]);
    }
  }
  __syncthreads();
  finish<TOut, kWarps>(a, p, s_m, s_l, reinterpret_cast<const float*>(pd_smem), kS * kTileBytes<DP> / 4);
}

// ---------------------------------------------------------------------------------------------- 4 bits
constexpr int kPair = 2 * kTile;  // tokens of a warp's tile: two of a page's sixteenths
constexpr int kStages4 = 3;
template <int D>
constexpr int kCodes = kPair * D / 2;
template <int D>
constexpr int kMeta = kPair * (D / kGroup) * 4;
template <int D>
constexpr int kTileBytes4 = 2 * (kCodes<D> + kMeta<D>);  // codes of keys and values, then their scales and offsets
template <int D>
constexpr int kRing4 = kStages4 * kTileBytes4<D>;
// Where sixteen tokens lie in the pools, and which of them the query sees.
struct __align__(16) Spot {
  int64_t codes;  // byte of the first one's codes, or -1: no page
  int meta;       // from there to its scales and offsets
  uint32_t seen;
};
constexpr int kBatch = 16;  // tiles that a warp looks up at once; the spots of two batches are kept
// ... and each token's factors, of its keys' groups and of its values', and the spots
template <int D>
constexpr int kFactors = 2 * kPair * (D / kGroup) * 8;
template <int D>
constexpr int kSmem4 = kRing4<D> + kFactors<D> + 4 * kBatch * (int)sizeof(Spot);  // of a warp

// (1 + code / 16) of nibbles m and m + 4 of a word, as bf16.  `one`: two bf16 ones, in a register so that mask and or are
// one instruction (from C the compiler made two, 1.3 times the whole kernel's).
template <int m>
__device__ __forceinline__ uint32_t ones(uint32_t w, uint32_t one) {
  const uint32_t x = m == 0 ? w << 3 : w >> (4 * m - 3);
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00780078, %2, 0xea;" : "=r"(r) : "r"(x), "r"(one));  // (x & mask) | one
  return r;
}

// The same less 3/2, exact: (code - 8) / 16.
template <int m>
__device__ __forceinline__ uint32_t centred(uint32_t w, uint32_t one) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(ones<m>(w, one)), "r"(0x3fc03fc0u));
  return r;
}

// Nibbles m and m + 4 of a word as two bf16 numbers, code 2^-133 or (m odd) 16 times that: the last eight bits of a bf16 number,
// the others zero, are a whole number of 2^-133 (subnormals and the first binade have the same step).
template <int m>
__device__ __forceinline__ uint32_t whole(uint32_t w, uint32_t w8) {  // w8: w >> 8
  return (m < 2 ? w : w8) & (m & 1 ? 0x00f000f0u : 0x000f000fu);
}

// Place of a row's 16-byte chunk: the rows that a product's lanes read together lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t place4(int r, int ch) {
  if constexpr (D == 128) return (uint32_t)((r >> 1) * 128 + ((r ^ (r >> 2)) & 1) * 64 + (ch ^ (r & 2)) * 16);
  else return (uint32_t)((r >> 2) * 128 + ((r & 3) ^ ((r >> 1) & 2)) * 32 + ch * 16);
}

template <typename TOut, int D, bool kSpare, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 12 / kWarps)
paged_decode_four_kernel(const PagedDecodeLaunch a) {
  using T = __nv_bfloat16;
  constexpr int kRows = kSpare ? 1 : 2, kGroups = D / kGroup, kS = kStages4;
  constexpr int kHalf = kTile * D / 2 / 16;            // chunks of codes of 16 tokens
  constexpr int kHalfMeta = kTile * kGroups * 4 / 16;  // and of their scales and offsets
  extern __shared__ __align__(128) uint8_t pd_smem[];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  const int warp = kWarps > 1 ? threadIdx.x >> 5 : 0, lane = threadIdx.x & 31, row = lane >> 2, q4 = lane & 3;
  grid_dependents_trigger();
  grid_dependency_wait();
  Part p;
  if (!part_of(a, p)) return;
  const int page = a.c.page;
  uint8_t* region = pd_smem + warp * kRing4<D>;
  const uint32_t base = tc::smem_u32(region);
  float* factors = reinterpret_cast<float*>(pd_smem + kWarps * kRing4<D> + warp * kFactors<D>);
  Spot* spots = reinterpret_cast<Spot*>(pd_smem + kWarps * (kRing4<D> + kFactors<D>)) + warp * 4 * kBatch;
  const int64_t size = page_bytes(a.c);

  const int tiles = p.last > p.first ? (p.last - p.first + kPair - 1) / kPair : 0;
  const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
  // ---- where the tiles lie: sixteen tiles at a time, a sixteenth of a page a lane, their pages looked up sixteen tiles ahead
  auto first_token = [&](int batch) { return p.first + (warp + (batch * kBatch + (lane >> 1)) * kWarps) * kPair + (lane & 1) * kTile; };
  auto lookup = [&](int batch) {  // -1 behind the last token or where there is no page
    const int t0 = first_token(batch);
    if (t0 >= p.last) return -1;
    const int pg = table_page(a.c, p.s, t0 / page);
    if (pg < 0 && p.hk == 0) atomicOr(a.c.status, kStatusBadIndex);
    return pg;
  };
  auto place = [&](int batch, int pg) {
    const int t0 = first_token(batch), slot = t0 % page;
    Spot n{-1, 0, 0u};
    if (pg >= 0) {
      n.codes = (pg * a.c.Hkv + p.hk) * size + slot * (D / 2);
      n.meta = page * (D / 2) + slot * (kGroups * 4 - D / 2);
      n.seen = token_bits(t0, kTile, p.seen.lo, p.last);
    }
    spots[batch % 2 * 32 + lane] = n;
  };
  // a lane's places in a tile: of the codes' chunk `lane` (later ones lie 32 chunks on), and of the scales'
  const uint8_t* kp = static_cast<const uint8_t*>(a.c.k) + lane * 16;
  const uint8_t* vp = static_cast<const uint8_t*>(a.c.v) + lane * 16;
  const int meta_half = lane / kHalfMeta & 1;
  const uint8_t* meta_pool = static_cast<const uint8_t*>(lane < 2 * kHalfMeta ? a.c.k : a.c.v) + lane % kHalfMeta * 16;
  const int meta_to = 2 * kCodes<D> + lane / (2 * kHalfMeta) * kMeta<D> + meta_half * (kMeta<D> / 2) + lane % kHalfMeta * 16;
  auto fetch = [&](int i, int stage) {
    const Spot* spot = spots + i % (2 * kBatch) * 2;
    const uint32_t to = base + stage * kTileBytes4<D>;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t from = spot[h].codes;
      if (from < 0) continue;  // codes of anything, whose tokens get no scale and no weight
#pragma unroll
      for (int j = 0; j < kHalf / 32; ++j) {
        const uint32_t at = place4<D>(h * kTile + (lane + 32 * j) / (D / 32), (lane + 32 * j) % (D / 32));
        tc::cp_async16(to + at, kp + from + j * 512, 16u);
        tc::cp_async16(to + kCodes<D> + at, vp + from + j * 512, 16u);
      }
    }
    const Spot m = spot[meta_half];
    if (lane < 4 * kHalfMeta && m.codes >= 0) tc::cp_async16(to + meta_to, meta_pool + m.codes + m.meta, 16u);
  };

  // ---- queries as operands: word e = 2 q4 + u of group g holds elements 64 g + 8 e + (0..7), whose pairs (m, m + 4) are a
  // product's neighbours; and the groups' sums of them
  // Each head's largest element becomes 2^120 to 2^121 (larger from 2^121 on, and at most times 2^127), so that its products with
  // whole numbers of 2^-133 are in the middle of fp32's range; scores are multiplied by 2^126 over that, the scales by 2^7.
  float q_down[kRows];
  uint32_t qa[kGroups][2][4 * kRows];  // [group][word][m, row]
  float qs[kGroups][2] = {}, slope[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int h = row + 8 * i;
    const T* q = static_cast<const T*>(a.q.ptr) + p.s * a.q.sb + (p.h0 + (h < p.group ? h : 0)) * a.q.sh;
    uint4 words[kGroups][2];
    int top = 0;  // the largest biased exponent
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4& w = words[g][u];
        w = make_uint4(0u, 0u, 0u, 0u);
        if (h < p.group) w = *reinterpret_cast<const uint4*>(q + kGroup * g + 8 * (2 * q4 + u));
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max((int)(x[e] >> 7 & 0xffu), (int)(x[e] >> 23 & 0xffu)));
      }
    top = max(top, __shfl_xor_sync(kFullMask, top, 1));
    top = max(top, __shfl_xor_sync(kFullMask, top, 2));
    const int up = min(max(374 - top, 126), 254);  // biased exponents
    const float q_up = __uint_as_float((uint32_t)up << 23);
    q_down[i] = __uint_as_float((uint32_t)(380 - up) << 23) * score_scale(a);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float v[8];
        unpack_vec(words[g][u], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= q_up;
        // a sixteenth where the code is the upper one of its byte; powers of two, exact
        uint32_t x[4];  // pairs (0, 1) (2, 3) (4, 5) (6, 7)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = tc::pack2_bf16(v[2 * e], v[2 * e + 1] * 0.0625f);
#pragma unroll
        for (int m = 0; m < 4; ++m) qa[g][u][m * kRows + i] = __byte_perm(x[m / 2], x[2 + m / 2], m & 1 ? 0x7632 : 0x5410);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[e], 0x1p-126f, sum);
      }
      sum += __shfl_xor_sync(kFullMask, sum, 1);
      qs[g][i] = sum + __shfl_xor_sync(kFullMask, sum, 2);
    }
    if (a.slopes && h < p.group) slope[i] = a.slopes[p.h0 + h] * kLog2e;
  }
  uint32_t one = 0x3f803f80u;
  asm volatile("" : "+r"(one));
  const float inv_cap = 1.f / a.softcap;
  // tile t's column c is this token of the warp's 32, so that a lane's four weights of a 16-token product are tokens
  // q4, q4 + 4, q4 + 8, q4 + 12 of it
  auto token = [](int t, int c) { return (t >> 1) * kTile + (c >> 1) + 4 * (2 * (t & 1) + (c & 1)); };

  // Sums of products, elements as rows and heads as columns: [heads 0-7, 8-15][group, m], elements 8 row + m (and that + 4) of
  // the group, heads 2 q4 and 2 q4 + 1.  The scores' layout is that of such a product's second operand.
  float o[kRows][4 * kGroups][4], bias[kGroups][2] = {};  // bias: sums of offsets, of head `row` and a lane's tokens
#pragma unroll
  for (int u = 0; u < kRows; ++u)
#pragma unroll
    for (int t = 0; t < 4 * kGroups; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[u][t][e] = 0.f;
  Running run;
  // where a lane's words lie: of keys, of values of tokens q4 and q4 + 4; eight tokens on are 8 rows on, whatever the place
  const int key_at = place4<D>(token(0, row), D == 128 ? q4 : q4 >> 1) + (D == 128 ? 0 : (q4 & 1) * 8);
  int val_at[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    val_at[j] = kCodes<D> + (D == 128 ? place4<D>(q4 + 4 * j, row >> 1) + (row & 1) * 8 : place4<D>(q4 + 4 * j, row >> 2) + (row & 3) * 4);
  int next = lookup(0);
  place(0, next);
  next = lookup(1);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kS - 1; ++i) {
    if (i < mine) fetch(i, i);
    tc::cp_async_commit();
  }
  for (int i = 0, stage = 0, into = kS - 1; i < mine; ++i, stage = stage + 1 == kS ? 0 : stage + 1, into = into + 1 == kS ? 0 : into + 1) {
    cp_async_wait<kS - 2>();
    const int ahead = i + kS - 1;
    if (ahead % kBatch == 0) {
      place(ahead / kBatch, next);
      next = lookup(ahead / kBatch + 1);
    }
    __syncwarp();  // every lane's copies of this tile are in, and its reads of the stage that is filled next are done
    if (ahead < mine) fetch(ahead, into);
    tc::cp_async_commit();
    const uint8_t* tile = region + stage * kTileBytes4<D>;
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(tile + 2 * kCodes<D>);
    const uint32_t seen = spots[i % (2 * kBatch) * 2].seen | spots[i % (2 * kBatch) * 2 + 1].seen << 16;
    // ---- a token a lane: 2^7 scale and offset of keys, 16 scale and offset + 8 scale of values
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint32_t w[kGroups];
      float f[2 * kGroups];
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(meta + (v * kPair + lane) * kGroups);
        w[0] = x.x; w[1] = x.y;
      } else {
        w[0] = meta[v * kPair + lane];
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float step = __uint_as_float(w[g] << 16), offset = __uint_as_float(w[g] & 0xffff0000u);
        f[2 * g] = v == 0 ? 128.f * step : 16.f * step;
        f[2 * g + 1] = v == 0 ? offset : fmaf(8.f, step, offset);
      }
      if (!(seen >> lane & 1u)) {
#pragma unroll
        for (int e = 0; e < 2 * kGroups; ++e) f[e] = 0.f;
      }
      float* to = factors + (v * kPair + lane) * 2 * kGroups;
      if constexpr (D == 128) *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
      else *reinterpret_cast<float2*>(to) = make_float2(f[0], f[1]);
    }
    __syncwarp();
    auto factors_of = [&](int v, int token, float (&f)[2 * kGroups]) {
      const float* from = factors + (v * kPair + token) * 2 * kGroups;
      if constexpr (D == 128) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(from);
        f[0] = x.x; f[1] = x.y;
      }
    };
    // ---- scores
    float x[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint8_t* at = tile + key_at + t * 8 * (D / 2);
      uint32_t w[kGroups][2];  // [group][word]
      if constexpr (D == 128) {
        const uint4 c = *reinterpret_cast<const uint4*>(at);
        w[0][0] = c.x; w[1][0] = c.y; w[0][1] = c.z; w[1][1] = c.w;
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(at);
        w[0][0] = c.x; w[0][1] = c.y;
      }
      float y[kGroups][4], z[kGroups][4];
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t(&q)[4 * kRows] = qa[g][u];
          const uint32_t w8 = w[g][u] >> 8, b0 = whole<0>(w[g][u], w8), b1 = whole<1>(w[g][u], w8), b2 = whole<2>(w[g][u], w8), b3 = whole<3>(w[g][u], w8);
          if constexpr (kSpare) {
            // Four registers of one head's elements as one operand, m = 0 and 2 in its rows 0 to 7, 1 and 3 in the others: the
            // rows that do not match a product's second operand are not used (zeros for them would take registers, or moves).
            if (u == 0) {
              mma16816_first(y[g], q[0], q[1], q[2], q[3], b0, b2);
              mma16816_first(z[g], q[0], q[1], q[2], q[3], b1, b3);
            } else {
              mma16816(y[g], q[0], q[1], q[2], q[3], b0, b2);
              mma16816(z[g], q[0], q[1], q[2], q[3], b1, b3);
            }
          } else {
            if (u == 0) mma16816_first(y[g], q[0], q[1], q[2], q[3], b0, b1);
            else mma16816(y[g], q[0], q[1], q[2], q[3], b0, b1);
            mma16816(y[g], q[4 * kRows - 4], q[4 * kRows - 3], q[4 * kRows - 2], q[4 * kRows - 1], b2, b3);
          }
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float f[2 * kGroups];
        factors_of(0, token(t, 2 * q4 + c), f);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          float sum = 0.f;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const float product = kSpare ? y[g][c] + z[g][2 + c] : y[g][2 * u + c];
            sum = g == 0 ? f[1] * qs[0][u] : fmaf(f[2 * g + 1], qs[g][u], sum);
            sum = fmaf(f[2 * g], product, sum);
          }
          x[t][2 * u + c] = sum * q_down[u];
        }
      }
    }
    const int t0 = p.first + (warp + i * kWarps) * kPair;
    bias_and_mask<kFine<TOut>, 4, kRows>(a, x, slope, inv_cap, p.seen.hi - 1 - t0, seen, 0xffffffffu, [&](int t, int e) { return token(t, 2 * q4 + e); });
    float f[2];
    if (weigh<4, kRows>(run, x, f)) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const float f0 = __shfl_sync(kFullMask, f[u], 8 * q4), f1 = __shfl_sync(kFullMask, f[u], 8 * q4 + 4);  // of heads 2 q4, 2 q4 + 1
#pragma unroll
        for (int t = 0; t < 4 * kGroups; ++t) {
          o[u][t][0] *= f0; o[u][t][1] *= f1; o[u][t][2] *= f0; o[u][t][3] *= f1;
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) bias[g][u] *= f[u];
      }
    }
    // ---- values, 16 tokens a product
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint32_t w[4][kGroups];  // the word e = row of each group, of tokens q4 + 4 j
      float f[4][2 * kGroups];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* at = tile + val_at[j & 1] + (2 * ks + (j >> 1)) * 8 * (D / 2);
        if constexpr (D == 128) {
          const uint2 c = *reinterpret_cast<const uint2*>(at);
          w[j][0] = c.x; w[j][1] = c.y;
        } else {
          w[j][0] = *reinterpret_cast<const uint32_t*>(at);
        }
        factors_of(1, ks * kTile + q4 + 4 * j, f[j]);
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        uint32_t major[kRows][2], minor[kRows][2], last[kRows][2];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float pa = x[2 * ks + t][2 * u], pb = x[2 * ks + t][2 * u + 1];
            bias[g][u] = fmaf(pa, f[2 * t][2 * g + 1], fmaf(pb, f[2 * t + 1][2 * g + 1], bias[g][u]));
            in_parts<kFine<TOut>>(pa * f[2 * t][2 * g], pb * f[2 * t + 1][2 * g], major[u][t], minor[u][t], last[u][t]);
          }
        // words of two tokens side by side: elements 0 to 3 in `lo`, 4 to 7 in `hi`
        const uint32_t lo0 = __byte_perm(w[0][g], w[1][g], 0x5410), hi0 = __byte_perm(w[0][g], w[1][g], 0x7632);
        const uint32_t lo1 = __byte_perm(w[2][g], w[3][g], 0x5410), hi1 = __byte_perm(w[2][g], w[3][g], 0x7632);
        auto product = [&](int m, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int u = 0; u < kRows; ++u) {
            mma16816(o[u][4 * g + m], a0, a1, a2, a3, major[u][0], major[u][1]);
            mma16816(o[u][4 * g + m], a0, a1, a2, a3, minor[u][0], minor[u][1]);
            if constexpr (kFine<TOut>) mma16816(o[u][4 * g + m], a0, a1, a2, a3, last[u][0], last[u][1]);
          }
        };
        product(0, centred<0>(lo0, one), centred<0>(hi0, one), centred<0>(lo1, one), centred<0>(hi1, one));
        product(1, centred<1>(lo0, one), centred<1>(hi0, one), centred<1>(lo1, one), centred<1>(hi1, one));
        product(2, centred<2>(lo0, one), centred<2>(hi0, one), centred<2>(lo1, one), centred<2>(hi1, one));
        product(3, centred<3>(lo0, one), centred<3>(hi0, one), centred<3>(lo1, one), centred<3>(hi1, one));
      }
    }
    __syncwarp();  // the factors are used up
  }
  tc::cp_async_wait_all();
  __syncwarp();
  // ---- this warp's sums into its place
  float* part = reinterpret_cast<float*>(region);
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    float l = run.l[u];
    l += __shfl_xor_sync(kFullMask, l, 1);
    l += __shfl_xor_sync(kFullMask, l, 2);
    if (q4 == 0) {
      s_m[warp][row + 8 * u] = run.m[u];
      s_l[warp][row + 8 * u] = l;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float off = bias[g][u];
      off += __shfl_xor_sync(kFullMask, off, 1);
      off += __shfl_xor_sync(kFullMask, off, 2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 2 * q4 + c + 8 * u;
        const float y = __shfl_sync(kFullMask, off, 4 * (2 * q4 + c));
        if (h >= p.group) continue;
        float4* to = reinterpret_cast<float4*>(part + h * D + kGroup * g + 8 * row);
        to[0] = make_float4(o[u][4 * g][c] + y, o[u][4 * g + 1][c] + y, o[u][4 * g + 2][c] + y, o[u][4 * g + 3][c] + y);
        to[1] = make_float4(o[u][4 * g][2 + c] + y, o[u][4 * g + 1][2 + c] + y, o[u][4 * g + 2][2 + c] + y, o[u][4 * g + 3][2 + c] + y);
      }
    }
  }
  __syncthreads();
  finish<TOut, kWarps>(a, p, s_m, s_l, reinterpret_cast<const float*>(pd_smem), kRing4<D> / 4);
}

template <typename K>
cudaError_t launch(K kernel, int warps, int smem, std::atomic<uint64_t>& done, const PagedDecodeLaunch& a, cudaStream_t stream) {
  const cudaError_t e = allow_smem(kernel, warps * smem, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)(a.S * a.c.Hkv * a.splits)), 32 * warps, warps * smem, stream, a);
}

// Many blocks of few tokens: blocks of one warp, so that more sequences are in their chain of length, page and rows at once (512
// sequences of up to 20 tokens over 8 key heads, bf16: 28 us, 56 with four warps a block).  Few by the table, as lengths are not
// known here: behind a table for 4096 tokens the same sequences take the 56 us.
bool one_warp(const PagedDecodeLaunch& a) { return a.S * a.c.Hkv * a.splits >= 152 * 16 && a.c.width * a.c.page / a.splits <= 512; }

template <typename TOut, int DP, bool kSpare>
cudaError_t launch_bf16(const PagedDecodeLaunch& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  static_assert(kStages<DP> * kTileBytes<DP> >= 16 * DP * 4, "a warp's sums take the place of its ring");
  return one_warp(a) ? launch(paged_decode_bf16_kernel<TOut, DP, kSpare, 1>, 1, kSmem<DP>, done[0], a, stream)
                     : launch(paged_decode_bf16_kernel<TOut, DP, kSpare, kMostWarps>, kMostWarps, kSmem<DP>, done[1], a, stream);
}
template <typename TOut, int D, bool kSpare>
cudaError_t launch_four(const PagedDecodeLaunch& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  static_assert(kRing4<D> >= 16 * D * 4, "a warp's sums take the place of its ring");
  return one_warp(a) ? launch(paged_decode_four_kernel<TOut, D, kSpare, 1>, 1, kSmem4<D>, done[0], a, stream)
                     : launch(paged_decode_four_kernel<TOut, D, kSpare, kMostWarps>, kMostWarps, kSmem4<D>, done[1], a, stream);
}
template <typename TOut, bool kSpare>
cudaError_t by_width(const PagedDecodeLaunch& a, cudaStream_t stream) {
  if (a.c.four) return a.c.d == 64 ? launch_four<TOut, 64, kSpare>(a, stream) : launch_four<TOut, 128, kSpare>(a, stream);
  return a.c.d <= 64 ? launch_bf16<TOut, 64, kSpare>(a, stream) : launch_bf16<TOut, 128, kSpare>(a, stream);
}
template <typename TOut>
cudaError_t by_group(const PagedDecodeLaunch& a, cudaStream_t stream) {
  return a.H / a.c.Hkv <= 8 ? by_width<TOut, true>(a, stream) : by_width<TOut, false>(a, stream);
}

}  // namespace

cudaError_t launch_paged_decode_mma(const PagedDecodeLaunch& a, cudaStream_t stream) {
  return a.out_bf16 ? by_group<__nv_bfloat16>(a, stream) : by_group<float>(a, stream);
}

}  // namespace la
