// swa_prefill_tc.cu -- masked window attention over a prompt for bf16 inputs, on tcgen05.
//
//   s_ij = cap tanh(scale q_i.k_j / cap) - slope_h |p_i - j|,  o_i = sum_j softmax_j(s_ij) v_j
// over the keys lo_i <= j < hi_i (empty: o_i = 0), in one pass over the keys: with the running maximum m
// and sum l, a block of keys adds P = exp(s - m) to l and P V to the output, which is scaled when m grows.
// All exponentials are base 2 (scores carry a factor log2 e).  The scale-up is put off while m grows by
// less than 2^8: P then stays below 256, which fp32 sums and bf16 weights hold as exactly as values below 1.
//
// Work is cut into items of 256 queries of one head: two tiles of 128 rows that share the key and value
// blocks.  Per block and tile: S = Q K^T into tensor memory (tcgen05, both operands from shared memory), one
// thread per row turns S into P (bf16, into shared memory), O += P V (tcgen05).  P does not take S's place in
// tensor memory: as soon as the threads hold S in registers the product for the next block may run, so that
// neither the products nor the hand-offs lie on the threads' way.  (With P over S the threads waited 1600 of
// 3100 clocks a block of 128 keys.  Blocks of 64 keys with two buffers of S were slower too: a product with
// N = 64 reads as much of Q from shared memory as one with N = 128 and takes as long.)  At d = 128 the products
// of a block of 128 keys take 1024 clocks a tile, the 16,384 exponentials 512.  Key and value blocks come by
// TMA through one ring, in the order in which the products take them: K0, K1, V0, K2, V1, ...  CTAs are
// persistent: the copies and the first products of the next item run while the rows of the last one are
// finished.  Widths up to 64 with narrow windows take blocks of 64 keys and two CTAs an SM: their blocks are
// few, and a chain of product, softmax and product is mostly latency.
//
// 2 x 16 heads of 8192 tokens over 4 key heads at d = 128, causal: 387 us, 1420 TFLOP/s, 74 % of the measured bf16 rate;
// with a cap of 30 535-575 us from box to box.  There neither the tensor pipe (35 %) nor the exponential unit (17 %) nor
// the issue slots (38 %) are near their limit: two row warps a scheduler wait for tensor-memory reads and for
// instructions.  8 x 16 x 4096 at d = 64 with a window of 64: 94 us with the rings, of which its bytes take 40; a block's
// chain of product, softmax and product bounds it.  Documents of 700 tokens with prefixes, a window of 1024 and a bias
// at d = 96 (2 x 8 x 4099): 69 us, 48 us without the bias, on 272 items for 152 SMs; where a prefix reaches ahead of its
// rows the bias takes the distance column by column (a form of that in registers too made it 70 us).
//
// Where items leave SMs idle and see several blocks, the CTAs of a cluster share an item's blocks; each leaves its
// rows' outputs, divided by their sums, and m + log2 l in its shared memory, where the cluster joins them.
//
// Warps 0-3 and 4-7: rows of tile 0 and 1; warps 8 and 11: their MMAs; warp 9: copies; warp 10: looks at each
// value block before it is used.  A value that a row does not see enters its product as 0 * v, which a NaN or an
// infinity would spoil: rows of padding are overwritten with zeros in shared memory, and where a block that
// is not seen as a whole holds other values that are not finite, the item's rows are computed again, key by
// key, on the CUDA cores (a rare path: only the keys in a row's interval are touched there).
//
// Every wait is bounded.  One that expires sets the status word and a flag in shared memory, after which no wait of the
// CTA lasts, no copy is issued and no row is stored, nor by the other CTAs of its cluster.  The loops still run to their
// end, with products of whatever shared memory holds, which only such rows would see.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "layers.cuh"
#include "swa_common.cuh"
#include "tc.cuh"

namespace la {
namespace {
using namespace tc;

constexpr int kRows = 128;                    // queries per tile
constexpr int kThreads = 384;                 // three warpgroups: rows of tile 0, of tile 1, and the rest
constexpr float kGrowth = 8.f;                // log2 of how far P may exceed 1 before the output is scaled
constexpr int kSMs = 152;
// What a wait's limit grows by for each key.  One tile may be at work on all keys, or its rows may be computed again over
// them, while warps wait for what comes behind; the latter took 2.9 us a key (32 rows a warp, d = 8, 1.2 million keys) and
// takes a few times that at d = 128.
constexpr uint64_t kWaitPerKeyNs = 50000;
// Capped scores may take a bound on their size, up to this in log2 units, for their maximum.  A row's running maximum is
// never lowered, and its true one lies 2 kBound below it at most; the exponential drops what lies 126 below the running
// one.  What is lost then lies 46 or more below the row's largest score: 2^24 such keys add 2^-22 to its sum.  (With a
// limit of 60 a key six binades below the largest was lost.)  The polynomial's part ends at half the cap, 0.72 cap in
// these units: caps up to 55 never meet the limit.
constexpr float kBound = 40.f;
// Windows up to this are narrow: blocks of 64 keys, two CTAs an SM.  8 x 16 x 4096 at d = 64: 88 us against 118
// with blocks of 128 for a window of 64, 124 against 132 for 256, 168 against 170 for 512.
constexpr int64_t kNarrow = 512;
// Blocks of keys that a CTA of a cluster gets at least (128 keys each).  8 heads of 16 queries over 65536 keys: 118 us
// with clusters of 8 against 853 without; 64 over 1024 (a share of 2): 16 against 21; 1024 over 1024 under the
// causal mask: 24 against 22; with shares of 3 or more the second and the third take 20 and 30 us.
constexpr int64_t kShare = 2;

// DP: width padded to whole 64-column blocks; KB: keys per block
template <int DP, int KB>
struct Shape {
  static constexpr int kCtas = KB == 64 ? 2 : 1;             // per SM
  static constexpr uint32_t kSlots = DP == 128 ? 3 : KB == 128 ? 6 : 5;  // of the ring of key and value blocks
  static constexpr uint32_t kBlk = DP / 64;                  // 64-column blocks per row
  static constexpr uint32_t kQTile = kRows * DP * 2;         // bytes
  static constexpr uint32_t kPTile = kRows * KB * 2;
  static constexpr uint32_t kKTile = KB * DP * 2;
  static constexpr uint32_t kOffP = 2 * kQTile, kOffR = kOffP + 2 * kPTile;
  static constexpr uint32_t kSmem = kOffR + kSlots * kKTile + 1024;  // + alignment of the base
  static_assert(kCtas * (kSmem + 2048) <= 228 * 1024, "");
  static constexpr uint32_t kColO = 2 * KB, kTmemCols = kCtas == 2 ? 256 : 512;
  static_assert(kColO + 2 * DP <= kTmemCols, "");
  // The row threads take more registers than the launch gives a thread; the third warpgroup gives them up first.
  static constexpr int kRegs = kCtas == 2 ? 80 : 168, kRegsRows = kCtas == 2 ? 96 : 208, kRegsRest = kCtas == 2 ? 48 : 88;
  static_assert(2 * kRegsRows + kRegsRest <= 3 * kRegs, "");
};

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Bounded wait without a sleep (the hand-offs lie on one chain); over at once when `dead` is set.
__device__ __forceinline__ void mbar_spin(uint64_t* bar, uint32_t parity, volatile uint32_t* dead, const SwaPrefillLaunch& a) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !mbar_try_wait(smem_u32(bar), parity & 1u); ++n) {
    if (n % 8 == 0) {  // a try that fails takes 1.4 us
      if (*dead) return;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      else if (t - t0 > a.wait_ns) {
        *dead = 1;
        atomicOr(a.status, kStatusTimeout);
        return;
      }
    }
  }
}

// Products and completions for a warp that runs as one, with the instruction itself left to one lane: inside a
// branch of one lane every operand would have to be moved to a uniform register first, about 100 clocks a
// product.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// Shared-memory descriptors in halves: the lower one holds the address (in units of 16 bytes) and the distance
// between 64-column blocks, the upper one is the same for all: 1024 bytes between 8-row groups, version 1,
// 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t blocks_apart) { return ((addr & 0x3FFFFu) >> 4) | (blocks_apart >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate, uint32_t mine) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(mine), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t mine) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(mine)
      : "memory");
}

// 0 * x summed over the eight bf16 of a vector: NaN exactly where one of them is not finite
__device__ __forceinline__ __nv_bfloat162 add_zero_times(uint4 u, __nv_bfloat162 acc) {
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), zero, acc);
  return acc;
}

// One row by one warp on the CUDA cores, reading only the keys of its interval.  Score in log2 units.
template <bool CAP, bool BIAS>
__device__ __noinline__ void slow_row(const SwaPrefillLaunch& a, int64_t b, int64_t h, int64_t hk, int64_t i, KeySpan sp, float slope2) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q.ptr) + b * a.q.sb + h * a.q.sh + i * a.q.st;
  const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(a.k.ptr) + b * a.k.sb + hk * a.k.sh;
  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v.ptr) + b * a.v.sb + hk * a.v.sh;
  const int pos = bias_origin(sp, (int)(a.q_pos0 + i));
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = sp.lo; j0 < sp.hi; j0 += 32) {
    const int j = j0 + lane;
    float x = -INFINITY;
    if (j < sp.hi) {
      x = 0.f;
      for (int c = 0; c < a.d; c += 4) x += dot4(load4(q + c), load4(k + (int64_t)j * a.k.st + c));
      if (CAP) x = a.softcap * kLog2e * tanhf(x * a.scale / a.softcap);
      else x *= a.scale * kLog2e;
      if (BIAS) x -= slope2 * fabsf((float)(pos - j));
    }
    float mn = x;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kFullMask, mn, off));
    mn = fmaxf(mn, m);
    const float base = mn == -INFINITY ? 0.f : mn, f = ex2(m - base);
    const float p = ex2(x - base);
    l = l * f + warp_sum(p);
    m = mn;
    o.x *= f; o.y *= f; o.z *= f; o.w *= f;
    const int n = min(32, sp.hi - j0);
    for (int t = 0; t < n; ++t) {
      const float w = __shfl_sync(kFullMask, p, t);
      if (lane * 4 < a.d) {
        const float4 y = load4(v + (int64_t)(j0 + t) * a.v.st + lane * 4);
        o.x = fmaf(w, y.x, o.x); o.y = fmaf(w, y.y, o.y); o.z = fmaf(w, y.z, o.z); o.w = fmaf(w, y.w, o.w);
      }
    }
  }
  if (lane * 4 < a.d) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float r[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    const int64_t at = b * a.o_sb + h * a.o_sh + i * a.o_st + lane * 4;
    if (a.out_bf16) store_floats(reinterpret_cast<__nv_bfloat16*>(a.o) + at, r, 4, true);
    else store_floats(reinterpret_cast<float*>(a.o) + at, r, 4, true);
  }
}

// The keys of 128 rows from i0 on, found by one warp (every lane gets them): [lo, hi) that some row sees, and
// [f_lo, f_hi) that every row sees that sees any.  (The loops here stay rolled: the kernel's four roles each
// have a copy, and code that every launch has to fetch costs small problems most.)
struct TileSpan {
  int lo, hi, f_lo, f_hi;
};
__device__ __forceinline__ TileSpan tile_span(const SwaPrefillLaunch& a, int b, int i0, int len) {
  TileSpan t{INT32_MAX, 0, 0, INT32_MAX};
  if (!a.key_lo && !a.key_hi) {  // intervals that move up with the rows: the first and the last row have them all
    const int last = min(i0 + kRows, min((int)a.Nq, len - (int)a.q_pos0)) - 1;
    if (last >= i0) {
      const KeySpan s0 = key_span(a, b, i0, len), s1 = key_span(a, b, last, len);
      t = TileSpan{s0.lo, s1.hi, s1.lo, s0.hi};
    }
    return t;
  }
#pragma unroll 1
  for (int i = i0 + (threadIdx.x & 31); i < i0 + kRows; i += 32) {
    const KeySpan s = key_span(a, b, i, len);
    if (s.lo < s.hi) t = TileSpan{min(t.lo, s.lo), max(t.hi, s.hi), max(t.f_lo, s.lo), min(t.f_hi, s.hi)};
  }
  t.lo = __reduce_min_sync(kFullMask, t.lo);
  t.hi = __reduce_max_sync(kFullMask, t.hi);
  t.f_lo = __reduce_max_sync(kFullMask, t.f_lo);
  t.f_hi = __reduce_min_sync(kFullMask, t.f_hi);
  return t;
}

// An item: 256 queries of one head.
struct Item {
  int b, h, i0, len;
  // The last queries see the most keys under the causal mask: items go from the last tiles to the first, and
  // every other round of CTAs takes its items in reverse.  False: there is none, or its sequence is skipped.
  // (Parts of an item are neighbouring CTAs, and then there is one round.)
  __device__ __forceinline__ bool place(const SwaPrefillLaunch& a, int round, int items, int q_tiles, int parts, bool report) {
    const int64_t at = parts > 1 ? blockIdx.x / parts
                                 : (int64_t)round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (at >= items) return false;
    const int heads = (int)(a.B * a.H), bh = (int)at % heads;
    i0 = (q_tiles - 1 - (int)at / heads) * (2 * kRows);
    b = bh / (int)a.H;
    h = bh - b * (int)a.H;
    len = (int)sequence_length(a.lens, b, a.Nk, a.status, report && h == 0 && i0 == 0);
    return len >= 0;
  }
};

// The blocks of keys that an item's two tiles see.
template <int KB>
struct Blocks {
  int jb[2], je[2];      // blocks [jb, je) of each tile
  int f_lo[2], f_hi[2];
  int j0, j1;            // and of both

  __device__ __forceinline__ Blocks(const SwaPrefillLaunch& a, const Item& it, int parts) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const TileSpan s = tile_span(a, it.b, it.i0 + t * kRows, it.len);
      jb[t] = s.lo < s.hi ? s.lo / KB : 0;
      je[t] = s.lo < s.hi ? (s.hi + KB - 1) / KB : 0;
      f_lo[t] = s.f_lo;
      f_hi[t] = s.f_hi;
    }
    bounds();
    if (parts > 1) {  // this CTA's share
      const int share = (j1 - j0 + parts - 1) / parts, from = j0 + (int)(blockIdx.x % parts) * share, to = from + share;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        jb[t] = max(jb[t], from);
        je[t] = min(je[t], to);
        if (jb[t] >= je[t]) jb[t] = je[t] = 0;
      }
      bounds();
    }
  }
  __device__ __forceinline__ void bounds() {
    const bool any0 = jb[0] < je[0], any1 = jb[1] < je[1];
    j0 = any0 && any1 ? min(jb[0], jb[1]) : any0 ? jb[0] : jb[1];
    j1 = max(je[0], je[1]);
  }
  __device__ __forceinline__ bool active(int t, int j) const { return j >= jb[t] && j < je[t]; }
  __device__ __forceinline__ bool active(int j) const { return active(0, j) || active(1, j); }
  __device__ __forceinline__ int next(int j) const {  // the next block that a tile is at work on, or j1
    do ++j; while (j < j1 && !active(j));
    return j;
  }
  // whether tile t is at work on block j and some of its rows do not see all of it
  __device__ __forceinline__ bool partial(int t, int j) const { return active(t, j) && (j * KB < f_lo[t] || j * KB + KB > f_hi[t]); }
};

// Where a part's output has four columns of a row of tile t: the lower half of the columns in the place of the
// queries, the upper one in that of the weights.
template <int DP, int KB>
__device__ __forceinline__ float4* part_at(uint8_t* sm, int t, int row, int c4) {
  using S = Shape<DP, KB>;
  constexpr int kHalf = DP / 8;  // float4 per half row
  const uint32_t base = c4 < kHalf ? t * S::kQTile : S::kOffP + t * S::kPTile;
  return reinterpret_cast<float4*>(sm + base) + row * kHalf + ((c4 % kHalf) ^ (row & 7));
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The item's rows out of the cluster's parts; every CTA takes rows of its own, a warp a row.
template <int DP, int KB, bool CAP, bool BIAS>
__device__ __noinline__ void join_parts(const SwaPrefillLaunch& a, const Item& it, uint8_t* sm, float* lse, uint32_t* redo, int parts,
                                        uint32_t* dead) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t again[2] = {0, 0}, given_up = 0;
  for (int u = 0; u < parts; ++u) {
    for (int t = 0; t < 2; ++t) again[t] |= *cluster.map_shared_rank(redo + t, u);
    given_up |= *cluster.map_shared_rank(dead, u);  // a part that is not whole spoils the rows of all
  }
  if (given_up) return;
#pragma unroll 1
  for (int r = (int)(blockIdx.x % parts) + warp * parts; r < 2 * kRows; r += 8 * parts) {
    const int row = it.i0 + r;
    if (row >= a.Nq || a.q_pos0 + row >= it.len) continue;
    if (r < kRows ? again[0] : again[1]) {
      slow_row<CAP, BIAS>(a, it.b, it.h, it.h / (a.H / a.Hkv), row, key_span(a, it.b, row, it.len),
                          BIAS && a.slopes ? a.slopes[it.h] * kLog2e : 0.f);
      continue;
    }
    float e[8], top = -INFINITY, total = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      e[u] = u < parts ? *cluster.map_shared_rank(lse + r, u) : -INFINITY;
      top = fmaxf(top, e[u]);
    }
    if (top == -INFINITY) top = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (e[u] == -INFINITY) continue;  // no keys of this row there, and no output
      const float f = ex2(e[u] - top);
      total += f;
      if (lane * 4 < a.d) {
        const float4 x = *cluster.map_shared_rank(part_at<DP, KB>(sm, r / kRows, r % kRows, lane), u);
        o.x = fmaf(f, x.x, o.x); o.y = fmaf(f, x.y, o.y); o.z = fmaf(f, x.z, o.z); o.w = fmaf(f, x.w, o.w);
      }
    }
    if (lane * 4 < a.d) {
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
      const int64_t at = (int64_t)it.b * a.o_sb + (int64_t)it.h * a.o_sh + (int64_t)row * a.o_st + lane * 4;
      if (a.out_bf16) store_floats(reinterpret_cast<__nv_bfloat16*>(a.o) + at, v, 4, true);
      else store_floats(reinterpret_cast<float*>(a.o) + at, v, 4, true);
    }
  }
}

// JOIN: an item belongs to a cluster of `clusters` CTAs
template <int DP, int KB, bool CAP, bool BIAS, bool JOIN>
__global__ void __launch_bounds__(kThreads, Shape<DP, KB>::kCtas)
swa_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const __grid_constant__ SwaPrefillLaunch a, int items, int q_tiles, int clusters) {
  const int parts = JOIN ? clusters : 1;
  using S = Shape<DP, KB>;
  constexpr uint32_t kSlots = S::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bar_q, bar_qfree;                           // queries of an item: here; used up
  __shared__ uint64_t bar_full[kSlots], bar_free[kSlots];         // of the ring
  __shared__ uint64_t bar_vok[kSlots];                            // warp 10: a value block holds what the products may read
  // per tile: S here, S read, P here, P V done, O read
  __shared__ uint64_t bar_s[2], bar_sfree[2], bar_p[2], bar_o[2], bar_ofree[2];
  __shared__ uint64_t bar_fin;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile uint32_t dead;
  // bad[t][n % 8] == n + 1: the n-th item at whose keys tile t is at work has values that are not finite in a block
  // that the tile's rows do not all see as a whole.  Warp 10 is at most kSlots + 1 < 8 such items ahead of the rows: a
  // product of the next one waits for the rows to have read this one's output, and the ring holds kSlots blocks.  (Items
  // that see nothing pass without a wait, any number of them, and do not count.)
  __shared__ volatile uint32_t bad[2][8];
  // with parts: a row's m + log2 l (no keys: -infinity), and whether a tile's rows have to be computed again
  __shared__ float lse[JOIN ? 2 * kRows : 1];
  __shared__ uint32_t redo[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(sm);
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar_q), 1);
    mbar_init(smem_u32(&bar_qfree), 2);  // what both tiles use up: an arrival of each one's products
    for (uint32_t s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_free[s]), 2);
      mbar_init(smem_u32(&bar_vok[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bar_s[t]), 1);
      mbar_init(smem_u32(&bar_sfree[t]), 4);  // one arrival per warp of the tile
      mbar_init(smem_u32(&bar_p[t]), 4);
      mbar_init(smem_u32(&bar_o[t]), 1);
      mbar_init(smem_u32(&bar_ofree[t]), 4);
    }
    mbar_init(smem_u32(&bar_fin), 2);
    dead = 0;
    redo[0] = redo[1] = 0;
    for (int n = 0; n < 16; ++n) bad[n / 8][n % 8] = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&tmem_base_sh), S::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  auto wait = [&](uint64_t* bar, uint32_t parity) { mbar_spin(bar, parity, &dead, a); };
  // slot and phase of the i-th block that passes through the ring
  auto slot = [](uint32_t i) { return i % kSlots; };
  auto phase = [](uint32_t i) { return i / kSlots; };
  const int group = (int)(a.H / a.Hkv);
  const int rounds = JOIN ? 1 : (items + (int)gridDim.x - 1) / (int)gridDim.x;
  Item it;

  if (warp >= 8) {
    regs_dec<S::kRegsRest>();
    if (warp == 9) {
      // ================================================================ copies: one thread
      uint32_t i = 0, n = 0;
      for (int r = 0; r < rounds; ++r) {
        if (!it.place(a, r, items, q_tiles, parts, false)) continue;
        const Blocks<KB> bl(a, it, parts);
        if (bl.j0 >= bl.j1) continue;
        if (lane == 0) {
          // an axis repeated with stride 0 has one entry in its map
          const int q_b = a.q.sb ? it.b : 0, q_h = a.q.sh ? it.h : 0;
          if (n > 0) wait(&bar_qfree, n - 1);
          if (!dead) {
            mbar_arrive_expect_tx(smem_u32(&bar_q), 2 * S::kQTile);
#pragma unroll 1
            for (int t = 0; t < 2; ++t)
#pragma unroll 1
              for (uint32_t c = 0; c < S::kBlk; ++c)
                tma_load_4d(sbase + t * S::kQTile + c * (kRows * 128), &map_q, c * 64, it.i0 + t * kRows, q_h, q_b, smem_u32(&bar_q));
            ++n;
          }
          auto load = [&](const CUtensorMap* map, const View4& x, int j) {
            const uint32_t s = slot(i);
            if (i >= kSlots) wait(&bar_free[s], phase(i - kSlots));
            if (dead) return;
            mbar_arrive_expect_tx(smem_u32(&bar_full[s]), S::kKTile);
#pragma unroll 1
            for (uint32_t c = 0; c < S::kBlk; ++c)
              tma_load_4d(sbase + S::kOffR + s * S::kKTile + c * (KB * 128), map, c * 64, j * KB, x.sh ? it.h / group : 0, x.sb ? it.b : 0, smem_u32(&bar_full[s]));
            ++i;
          };
          // keys a block ahead of values
          for (int jk = bl.j0, jv = bl.j0; jv < bl.j1;) {
            const bool keys = jk < bl.j1 && jk <= bl.next(jv);
            load(keys ? &map_k : &map_v, keys ? a.k : a.v, keys ? jk : jv);
            if (keys) jk = bl.next(jk);
            else jv = bl.next(jv);
          }
        }
        __syncwarp();
      }
      if (lane == 0) {  // the last copies land before the CTA ends, whatever became of those that use them
        for (uint32_t k = i > kSlots ? i - kSlots : 0; k < i; ++k) mbar_wait(smem_u32(&bar_full[slot(k)]), phase(k) & 1u, a.status);
        if (n > 0) mbar_wait(smem_u32(&bar_q), (n - 1) & 1u, a.status);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ================================================================ a look at each value block
      uint32_t i = 0, iv = 0, n0 = 0, n1 = 0;
      for (int r = 0; r < rounds; ++r) {
        if (!it.place(a, r, items, q_tiles, parts, lane == 0 && (parts == 1 || blockIdx.x % parts == 0))) continue;
        const Blocks<KB> bl(a, it, parts);
        const bool any0 = bl.jb[0] < bl.je[0], any1 = bl.jb[1] < bl.je[1];
        if (any0) ++n0;
        if (any1) ++n1;
        if (bl.j0 < bl.j1) ++i;  // the first block of keys
        for (int j = bl.j0, after; j < bl.j1; j = after) {
          after = bl.next(j);
          if (after < bl.j1) ++i;  // the next block of keys
          wait(&bar_full[slot(i)], phase(i));
          __syncwarp();
          uint8_t* v = sm + S::kOffR + slot(i) * S::kKTile;
          if ((j + 1) * KB > it.len) {  // rows of padding (TMA has zeroed those behind the last key only)
            for (int e = lane; e < (int)(S::kBlk * KB * 8); e += 32)
              if (j * KB + e / 8 % KB >= it.len) *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
          const bool part0 = bl.partial(0, j), part1 = bl.partial(1, j);
          if (part0 || part1) {
            __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 4
            for (int e = lane; e < (int)(S::kBlk * KB * 8); e += 32) acc = add_zero_times(*reinterpret_cast<const uint4*>(v + e * 16), acc);
            if (__any_sync(kFullMask, __hisnan(acc.x) || __hisnan(acc.y)) && lane == 0) {
              // (only of a tile that has yet to use the block: the other one's rows may or may not have looked by now)
              if (part0) bad[0][(n0 - 1) % 8] = n0;
              if (part1) bad[1][(n1 - 1) % 8] = n1;
            }
          }
          warp_arrive(smem_u32(&bar_vok[slot(iv)]));
          ++i;
          ++iv;
        }
      }
    } else {
      // ================================================================ products: warp 8 of tile 0, warp 11 of tile 1
      // S = Q K^T a block ahead of O += P V.  Both warps pass through every block, also where only one has work,
      // so that a block counts as used up once for each.
      const int t = warp == 8 ? 0 : 1;
      const uint32_t id_s = idesc_bf16(kRows, KB, 0, 0), id_o = idesc_bf16(kRows, DP, 0, 1);
      const uint32_t mine = elect_one();
      uint32_t i = 0, iv = 0, n = 0;         // blocks and value blocks used, items
      uint32_t ns = 0, np = 0, no = 0;       // S issued, P used, outputs begun
      const uint32_t q_lo = desc_lo(sbase + t * S::kQTile, 0), p_lo = desc_lo(sbase + S::kOffP + t * S::kPTile, 0);
      const uint32_t s_col = tmem + t * KB, o_col = tmem + S::kColO + t * DP;
      for (int r = 0; r < rounds; ++r) {
        if (!it.place(a, r, items, q_tiles, parts, false)) continue;
        const Blocks<KB> bl(a, it, parts);
        if (bl.j0 >= bl.j1) continue;
        const int jb = t ? bl.jb[1] : bl.jb[0], je = t ? bl.je[1] : bl.je[0];
        wait(&bar_q, n);
        auto step_s = [&](int j) {
          wait(&bar_full[slot(i)], phase(i));
          if (j >= jb && j < je) {
            if (ns > 0) wait(&bar_sfree[t], ns - 1);  // the rows hold the last S in registers
            tc_fence_after();
            const uint32_t k_lo = desc_lo(sbase + S::kOffR + slot(i) * S::kKTile, 0);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
              const uint32_t blk = ks >> 2, in = (ks & 3) * 32;
              mma_ss(s_col, q_lo + (blk * (kRows * 128) + in) / 16, k_lo + (blk * (KB * 128) + in) / 16, id_s, ks > 0, mine);
            }
            commit(&bar_s[t], mine);
            ++ns;
          }
          commit(&bar_free[slot(i)], mine);
          if (j == bl.j1 - 1) commit(&bar_qfree, mine);
          ++i;
        };
        bool ahead = false;
        for (int j = bl.j0, jq = bl.j0; j < bl.j1;) {
          if (jq < bl.j1) {
            step_s(jq);
            jq = bl.next(jq);
          }
          if (!ahead) {  // the first S alone
            ahead = true;
            continue;
          }
          wait(&bar_vok[slot(iv)], phase(iv));
          if (j >= jb && j < je) {
            const bool begin = j == jb;
            if (begin && no > 0) wait(&bar_ofree[t], no - 1);  // the rows have read the last item's output
            wait(&bar_p[t], np);
            tc_fence_after();
            const uint32_t v_lo = desc_lo(sbase + S::kOffR + slot(i) * S::kKTile, KB * 128);
#pragma unroll
            for (int ks = 0; ks < KB / 16; ++ks) {
              const uint32_t blk = ks >> 2, in = (ks & 3) * 32;
              mma_ss(o_col, p_lo + (blk * (kRows * 128) + in) / 16, v_lo + ks * 2048 / 16, id_o, (!begin || ks > 0) ? 1u : 0u, mine);
            }
            commit(&bar_o[t], mine);
            ++np;
            if (j == je - 1) ++no;
          }
          commit(&bar_free[slot(i)], mine);
          ++i;
          ++iv;
          j = bl.next(j);
        }
        ++n;
      }
      // every product has completed before tensor memory is given back
      commit(&bar_fin, mine);
      __syncwarp();
      mbar_wait(smem_u32(&bar_fin), 0, a.status);
      __syncwarp();
    }
    if constexpr (JOIN) {  // the rows join their parts
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ================================================================ one thread per row
    regs_inc<S::kRegsRows>();
    const int t = warp >> 2;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint8_t* p_tile = sm + S::kOffP + t * S::kPTile;
    const uint32_t p_row = threadIdx.x % kRows;
    const uint32_t cs = tl + t * KB, col_o = tl + S::kColO + t * DP;
    const float c1 = a.scale * kLog2e;
    // With a cap: z = zc x for a product x.  Where whole rows are straight the factors are drawn into the polynomial's
    // coefficients, cap tanh(z) = x Q(x^2) in log2 units (as long as they stay normal numbers).
    const float zc = CAP ? a.scale / a.softcap : 0.f, cz = zc * (2.f * kLog2e), capl = a.softcap * kLog2e;
    [[maybe_unused]] const bool drawn = zc > 2e-5f && zc < 1e3f;
    // the difference's error of 1e-7 cap stays below a hundredth of the weights' rounding: any row may take it
    [[maybe_unused]] const bool small_cap = capl <= 400.f;
    float kq[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (CAP) {
      const float z2 = zc * zc;
      kq[0] = kTanh[0] * capl * zc;
      kq[1] = kTanh[1] * capl * zc * z2;
      kq[2] = kTanh[2] * capl * zc * z2 * z2;
      kq[3] = kTanh[3] * capl * zc * z2 * z2 * z2;
    }
    [[maybe_unused]] auto straight_tanh = [&](float v) {
      const float u = v * v;
      return fmaf(fmaf(fmaf(kq[3], u, kq[2]), u, kq[1]), u, kq[0]);
    };
    [[maybe_unused]] auto straight_tanh2 = [&](f32x2 v) {
      const f32x2 u = mul2(v, v);
      return fma2(fma2(fma2(pack2(kq[3], kq[3]), u, pack2(kq[2], kq[2])), u, pack2(kq[1], kq[1])), u, pack2(kq[0], kq[0]));
    };
    const bool al32 = ((reinterpret_cast<uintptr_t>(a.o) | (uintptr_t)((a.o_sb | a.o_sh | a.o_st) * (a.out_bf16 ? 2 : 4))) & 31u) == 0;
    uint32_t ns = 0, n = 0;  // blocks, items at whose keys this tile is at work
    for (int round = 0; round < rounds; ++round) {
      if (!it.place(a, round, items, q_tiles, parts, false)) continue;
      const int i = it.i0 + (int)threadIdx.x;
      const KeySpan span = key_span(a, it.b, i, it.len);
      const TileSpan ts = tile_span(a, it.b, it.i0 + t * kRows, it.len);
      int jb = ts.lo < ts.hi ? ts.lo / KB : 0, je = ts.lo < ts.hi ? (ts.hi + KB - 1) / KB : 0;
      if (JOIN) {
        const Blocks<KB> bl(a, it, parts);
        jb = t ? bl.jb[1] : bl.jb[0];
        je = t ? bl.je[1] : bl.je[0];
      }
      const int pos = bias_origin(span, (int)a.q_pos0 + i);
      const float slope2 = BIAS && a.slopes ? a.slopes[it.h] * kLog2e : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int j = jb; j < je; ++j, ++ns) {
        wait(&bar_s[t], ns);
        __syncwarp();
        tc_fence_after();
        const int k0 = j * KB;
        const int va = span.lo - k0, vb = span.hi - k0;  // columns va <= c < vb are seen
        auto s_read = [&]() {  // the product for the next block may take S's place
          tc_fence_before();
          warp_arrive(smem_u32(&bar_sfree[t]));
        };
        // The products of the block before: P's place is free and the output at rest behind them.
        bool o_rests = j == jb;
        auto wait_o = [&]() {
          if (!o_rests) {
            wait(&bar_o[t], ns - 1);
            __syncwarp();
            tc_fence_after();
          }
          o_rests = true;
        };
        // The running maximum takes in this block's, mn (or a bound of it); returns what the exponentials subtract.
        auto update = [&](float mn) {
          if (m == -INFINITY) m = mn;  // nothing seen before: the output holds zeros, or nothing yet
          const bool grow = mn > m + kGrowth;
          if (__any_sync(kFullMask, grow)) {
            const float f = grow ? ex2(m - mn) : 1.f;
            if (grow) m = mn;
            l *= f;
            wait_o();
            if (j > jb) {
#pragma unroll 1
              for (int c = 0; c < DP; c += 16) {
                float o[16];
                tmem_ld16(col_o + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= f;
                tmem_st16(col_o + c, o);
              }
            }
          }
          return m == -INFINITY ? 0.f : m;
        };
        f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
        // Two columns' weights as bf16, which is what a product with bf16 values takes.  Their roundings, up to 2^-8 of a
        // weight each and without a common sign, left the outputs of the measured prompts off by 1.4e-3 of their norm, less than
        // the 1.7e-3 of a bf16 output's own rounding; l sums the weights before it.  A second bf16 part of each weight
        // would take half as much again of the tensor pipe and 32 KB that the ring of keys and values fills.
        auto weight = [&](f32x2 y, int e) {
          const f32x2 p2 = ex2_2(y);
          sum[e & 1] = add2(sum[e & 1], p2);
          float p0, p1;
          unpack2(p2, p0, p1);
          return pack2_bf16(p0, p1);
        };
        // The whole row in registers: with a cap for blocks that the whole warp sees, with a bias for blocks of which
        // its rows see what lies behind them, and with neither for any.  A cap comes from the polynomial as the scores are used
        // (straight; false, with nothing done, where products leave the part that it is good for or scores spread too
        // far for the bound below), or else from the difference, in place.  2 x 16 x 8192 at d = 128 takes 387 us without
        // a cap, 535 with the one and 826 with the other, against 1340 where a row is read in parts.
        auto row_at_once = [&](auto straight) {
          constexpr bool kPoly = CAP && decltype(straight)::value, kFar = CAP && !kPoly;
          constexpr int kAll = KB == 128 ? KB : 2;
          float x[kAll];
#pragma unroll
          for (int c = 0; c + 32 <= kAll; c += 32) tmem_ld32(cs + c, x + c);
          tmem_ld_wait();
          const float unit = kFar ? 1.f : c1;
          f32x2 c2 = pack2(unit, unit);
          if constexpr (kPoly) {
            float hi[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kAll; ++c) hi[c & 3] = fmaxf(hi[c & 3], fabsf(x[c]));
            const float h = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
            if (!__all_sync(kFullMask, h * zc <= kStraight && h * c1 <= kBound)) return false;
            s_read();
            // No score exceeds cap tanh(zc h): the bound serves as the maximum.
            if constexpr (!BIAS) {
              const float base = update(h * straight_tanh(h));
              c2 = pack2(-base, -base);
            }
          } else {
            s_read();
          }
          if constexpr (kFar) {
#pragma unroll
            for (int c = 0; c < kAll; ++c) x[c] = fmaf(-2.f * capl, rcp(1.f + ex2(x[c] * cz)), capl);
          }
          if constexpr (BIAS) {
#pragma unroll
            for (int c = 0; c < kAll; c += 32) {  // - slope (pos - k0 - c): two columns more add 2 slope
              const float far = slope2 * (float)(k0 + c - pos);
              f32x2 off = pack2(far, far + slope2);
              const f32x2 step = pack2(2.f * slope2, 2.f * slope2);
#pragma unroll
              for (int e = 0; e < 32 && c + e < kAll; e += 2) {
                const f32x2 v = pack2(x[c + e], x[c + e + 1]);
                unpack2(fma2(v, kPoly ? straight_tanh2(v) : c2, off), x[c + e], x[c + e + 1]);
                off = add2(off, step);
              }
            }
          }
          if constexpr (!kPoly) {
            if (!__all_sync(kFullMask, va <= 0 && vb >= KB)) {
#pragma unroll
              for (int c = 0; c < kAll; ++c) x[c] = c >= va && c < vb ? x[c] : -INFINITY;
            }
          }
          f32x2 base2 = c2;
          if constexpr (BIAS || !kPoly) {
            float mx[4] = {x[0], x[0], x[0], x[0]};
#pragma unroll
            for (int c = 0; c < kAll; ++c) mx[c & 3] = fmaxf(mx[c & 3], x[c]);
            float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (!BIAS && mn != -INFINITY) mn *= unit;  // the scale is positive here
            const float base = update(mn);
            base2 = pack2(-base, -base);
          }
          uint32_t w[kAll / 2];
#pragma unroll
          for (int e = 0; e < kAll / 2; ++e) {
            const f32x2 v = pack2(x[2 * e], x[2 * e + 1]);
            w[e] = weight(BIAS ? add2(v, base2) : fma2(v, kPoly ? straight_tanh2(v) : c2, base2), e);
          }
          wait_o();  // the products of the block before may have read P's place until here
#pragma unroll
          for (int e = 0; e < kAll / 8; ++e)
            *reinterpret_cast<uint4*>(p_tile + sw128_off(p_row, 8 * e, kRows)) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          return true;
        };
        // 32 columns at a time, read once for the maximum and once more for the weights.  Columns that no row of
        // the warp sees are passed over (their weights are zeros), ones that all see are not masked.
        auto row_by_parts = [&]() {
          constexpr bool raw = !CAP && !BIAS;  // products serve as scores until the exponential
          auto none = [&](int c0) { return __all_sync(kFullMask, vb <= c0 || va >= c0 + 32 || va >= vb); };
          auto read = [&](int c0, float (&v)[32]) {
            tmem_ld32(cs + c0, v);
            tmem_ld_wait();
            const float dist = (float)(pos - k0 - c0);
            if constexpr (CAP) {
              float hi[2] = {0.f, 0.f};
#pragma unroll
              for (int c = 0; c < 32; ++c) hi[c & 1] = fmaxf(hi[c & 1], fabsf(v[c]));
              // half a warp each way would cost both
              bool near = fmaxf(hi[0], hi[1]) * fabsf(zc) <= kStraight;
              if (small_cap) near = __all_sync(kFullMask, near);
              if (near) {
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  const f32x2 x = pack2(v[c], v[c + 1]), z = mul2(x, pack2(zc, zc)), u = mul2(z, z);
                  f32x2 q = pack2(kTanh[3], kTanh[3]);
#pragma unroll
                  for (int e = 2; e >= 0; --e) q = fma2(q, u, pack2(kTanh[e], kTanh[e]));
                  unpack2(mul2(mul2(x, pack2(c1, c1)), q), v[c], v[c + 1]);
                }
              } else {  // beside a score of half the cap an error of 1e-7 cap is one of the score's own rounding
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = fmaf(-2.f * capl, rcp(1.f + ex2(v[c] * cz)), capl);
              }
            } else if constexpr (BIAS) {
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] *= c1;
            }
            if constexpr (BIAS) {
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = fmaf(-slope2, fabsf(dist - (float)c), v[c]);
            }
            if (!__all_sync(kFullMask, va <= c0 && vb >= c0 + 32)) {
              const uint32_t from = va - c0 >= 32 ? 0u : ~0u << max(va - c0, 0), to = vb - c0 >= 32 ? ~0u : (1u << max(vb - c0, 0)) - 1u;
              const uint32_t seen = from & to;
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = seen & (1u << c) ? v[c] : -INFINITY;
            }
          };
          float mn = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < KB; c0 += 32) {
            if (none(c0)) continue;
            float v[32];
            read(c0, v);
            float mx[2] = {v[0], v[1]};
#pragma unroll
            for (int c = 2; c < 32; ++c) mx[c & 1] = fmaxf(mx[c & 1], v[c]);
            mn = fmaxf(mn, fmaxf(mx[0], mx[1]));
          }
          if (raw && mn != -INFINITY) mn *= c1;  // the scale is positive here
          const float base = update(mn);
          const f32x2 base2 = pack2(-base, -base), c2 = pack2(c1, c1);
          wait_o();
#pragma unroll 1
          for (int c0 = 0; c0 < KB; c0 += 32) {
            uint32_t w[16];
            if (none(c0)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = 0u;
            } else {
              float v[32];
              read(c0, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const f32x2 y = pack2(v[2 * e], v[2 * e + 1]);
                w[e] = weight(raw ? fma2(y, c2, base2) : add2(y, base2), e);
              }
            }
            if (c0 + 32 == KB) s_read();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(p_tile + sw128_off(p_row, c0 + 8 * e, kRows)) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        };
        if constexpr (KB == 64) {  // such blocks are few, and hardly ever seen as a whole
          row_by_parts();
        } else if constexpr (!CAP && !BIAS) {
          row_at_once(std::false_type{});
        } else {
          // what a row sees lies behind it: |pos - key| is linear there
          const bool behind = !BIAS || va >= vb || pos - k0 >= min(vb, KB) - 1;
          const bool whole = __all_sync(kFullMask, behind && (!CAP || (va <= 0 && vb >= KB)));
          bool done = false;
          if constexpr (CAP) {
            done = whole && ((drawn && row_at_once(std::true_type{})) || (small_cap && row_at_once(std::false_type{})));
          } else if (whole) {
            done = row_at_once(std::false_type{});
          }
          if (!done) row_by_parts();
        }
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        tmem_st_wait();  // of a scaled output
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(smem_u32(&bar_p[t]));
      }
      bool again = false;
      if (jb < je) {
        wait(&bar_o[t], ns - 1);
        __syncwarp();
        tc_fence_after();
        ++n;
        again = __all_sync(kFullMask, bad[t][(n - 1) % 8] == n && !dead);
      }
      if (JOIN) {
        // The tile's own queries and weights are used up: their places take its outputs.  (Queries may still be on
        // their way to a tile that is not at work, which leaves nothing.)
        const float inv = l != 0.f ? 1.f / l : 0.f;
        if (jb < je) {
#pragma unroll 1
          for (int c = 0; c < DP; c += 16) {
            float o[16];
            tmem_ld16(col_o + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *part_at<DP, KB>(sm, t, (int)p_row, (c + e) / 4) = make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
          }
        }
        lse[threadIdx.x] = l != 0.f ? m + __log2f(l) : -INFINITY;
        if (again && lane == 0) redo[t] = 1;
        break;
      }
      const bool live = i < a.Nq && a.q_pos0 + i < it.len && !dead;
      const bool seen = l != 0.f;  // also a row whose sum is NaN
      const float inv = seen ? 1.f / l : 0.f;
      const int64_t at = (int64_t)it.b * a.o_sb + (int64_t)it.h * a.o_sh + (int64_t)i * a.o_st;
#pragma unroll 1
      for (int c = 0; c < DP; c += 16) {
        float o[16];
        if (jb < je) {
          tmem_ld16(col_o + c, o);
          tmem_ld_wait();
          if (c + 16 == DP) {  // the output is in registers: the next item's may be begun
            tc_fence_before();
            warp_arrive(smem_u32(&bar_ofree[t]));
          }
        }
        if (live && !again && c < a.d) {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = seen ? o[e] * inv : 0.f;
          const bool two = c + 8 < a.d;  // d is a multiple of 8
          if (a.out_bf16) {
            __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(a.o) + at + c;
            const uint4 u = pack8_bf16(o), v = pack8_bf16(o + 8);
            if (two && al32) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u.x), "r"(u.y), "r"(u.z),
                           "r"(u.w), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(p) = u;
              if (two) *reinterpret_cast<uint4*>(p + 8) = v;
            }
          } else {
            float* p = reinterpret_cast<float*>(a.o) + at + c;
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              if (k < 8 || two) *reinterpret_cast<float4*>(p + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
      }
      if (again) {  // the rows of this warp once more, from their own keys only
#pragma unroll 1
        for (int r = 0; r < 32; ++r) {
          const int row = it.i0 + warp * 32 + r;
          const KeySpan sp{__shfl_sync(kFullMask, span.lo, r), __shfl_sync(kFullMask, span.hi, r)};
          if (row < a.Nq && a.q_pos0 + row < it.len) slow_row<CAP, BIAS>(a, it.b, it.h, it.h / group, row, sp, slope2);
        }
      }
    }
    if (JOIN) {
      cluster_sync();
      if (it.place(a, 0, items, q_tiles, parts, false)) join_parts<DP, KB, CAP, BIAS>(a, it, sm, lse, redo, parts, const_cast<uint32_t*>(&dead));
      cluster_sync();  // the parts are read before a CTA ends
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, S::kTmemCols);
}

// [B, H, N, d] bf16 view as boxes of `rows` x 64 columns, columns and rows behind the ends filled with zeros.  Sequences
// or heads repeated with stride 0 are an axis with one entry.
bool encode(CUtensorMap* map, const View4& x, int64_t B, int64_t H, int64_t N, int d, int rows) {
  const tc::EncodeTiledFn fn = tc::encode_tiled();
  if (!fn) return false;
  if (x.sh == 0) H = 1;
  if (x.sb == 0) B = 1;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)B};
  // the stride of an axis with one entry is never used, but has to be one that a map can hold
  const cuuint64_t row = (cuuint64_t)d * 2;
  const cuuint64_t strides[3] = {N > 1 ? (cuuint64_t)x.st * 2 : row, H > 1 ? (cuuint64_t)x.sh * 2 : row,
                                 B > 1 ? (cuuint64_t)x.sb * 2 : row};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// blocks of keys that an item may see
int64_t key_blocks(const SwaPrefillLaunch& a, int KB) { return (a.window > 0 ? std::min(a.Nk, a.window + 2 * kRows) : a.Nk) / KB; }

template <int DP, int KB, bool CAP, bool BIAS, bool JOIN>
cudaError_t launch_typed(const SwaPrefillLaunch& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  using S = Shape<DP, KB>;
  const auto kernel = swa_tc_kernel<DP, KB, CAP, BIAS, JOIN>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, (int)S::kSmem, done);
  if (e != cudaSuccess) return e;
  // the row threads' registers come out of the launch's own: with fewer they would be waited for without end
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes f{};
    e = cudaFuncGetAttributes(&f, kernel);
    if (e != cudaSuccess) return e;
    regs.store(f.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < S::kRegs) return cudaErrorInvalidConfiguration;
  const int q_tiles = (int)((a.Nq + 2 * kRows - 1) / (2 * kRows));
  const int64_t items = a.B * a.H * q_tiles;
  cudaLaunchAttribute cluster;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cfg.attrs = &cluster;
  int parts = 1;
  if constexpr (JOIN) {
    static std::atomic<int> room[4] = {};  // clusters of 2, 4 and 8 that the GPU holds at once (its SMs come in groups), + 1
    for (int log = 3; log >= 1 && parts == 1; --log) {
      if (key_blocks(a, KB) < (kShare << log) || items > (kSMs >> log)) continue;
      cluster.id = cudaLaunchAttributeClusterDimension;
      cluster.val.clusterDim.x = 1u << log;
      cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
      cfg.numAttrs = 1;
      cfg.gridDim = dim3((unsigned)(items << log));
      int n = room[log].load(std::memory_order_relaxed);
      if (n == 0) {
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        room[log].store(++n, std::memory_order_relaxed);
      }
      if (items < n) parts = 1 << log;
    }
    if (parts == 1) return cudaErrorNotReady;  // for the kernel without
  } else {
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, S::kCtas * kSMs));
  }
  return cudaLaunchKernelEx(&cfg, kernel, q, k, v, a, (int)items, q_tiles, parts);
}

template <int DP, int KB, bool CAP, bool BIAS>
cudaError_t launch_parts(const SwaPrefillLaunch& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  if constexpr (KB == 128) {
    if (a.B * a.H * ((a.Nq + 2 * kRows - 1) / (2 * kRows)) <= kSMs / 2 && key_blocks(a, KB) >= 2 * kShare) {
      const cudaError_t e = launch_typed<DP, KB, CAP, BIAS, true>(a, q, k, v, stream);
      if (e != cudaErrorNotReady) return e;
    }
  }
  return launch_typed<DP, KB, CAP, BIAS, false>(a, q, k, v, stream);
}

template <int DP, int KB>
cudaError_t launch_width(const SwaPrefillLaunch& a, cudaStream_t stream) {
  CUtensorMap q, k, v;
  if (!encode(&q, a.q, a.B, a.H, a.Nq, a.d, kRows) || !encode(&k, a.k, a.B, a.Hkv, a.Nk, a.d, KB) ||
      !encode(&v, a.v, a.B, a.Hkv, a.Nk, a.d, KB))
    return cudaErrorInvalidValue;
  // without a bias the maximum is taken of the raw products, which the scale must not turn round
  const bool cap = a.softcap != 0.f, bias = a.slopes != nullptr || !(a.scale > 0.f);
  if (cap && bias) return launch_parts<DP, KB, true, true>(a, q, k, v, stream);
  if (cap) return launch_parts<DP, KB, true, false>(a, q, k, v, stream);
  if (bias) return launch_parts<DP, KB, false, true>(a, q, k, v, stream);
  return launch_parts<DP, KB, false, false>(a, q, k, v, stream);
}

}  // namespace

cudaError_t launch_swa_prefill_tc(const SwaPrefillLaunch& args, cudaStream_t stream) {
  SwaPrefillLaunch a = args;
  a.wait_ns = kWaitLimitNs + kWaitPerKeyNs * (uint64_t)a.Nk;
  if (a.d > 64) return launch_width<128, 128>(a, stream);
  return a.window > 0 && a.window <= kNarrow ? launch_width<64, 64>(a, stream) : launch_width<64, 128>(a, stream);
}

}  // namespace la
