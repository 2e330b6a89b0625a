// swa_prefill_tc.cu -- masked window attention over a prompt for bf16 inputs, on tcgen05.
//
//   s_ij = cap tanh(scale q_i.k_j / cap) - slope_h |p_i - j|,  o_i = sum_j softmax_j(s_ij) v_j
// over the keys lo_i <= j < hi_i (empty: o_i = 0), in one pass over the keys: with the running maximum m
// and sum l, a block of keys adds P = exp(s - m) to l and P V to the output, which is scaled when m grows.
// All exponentials are base 2 (scores carry a factor log2 e).  The scale-up is put off while m grows by
// less than 2^8: P then stays below 256, which fp32 sums and bf16 weights hold as exactly as values below 1.
//
// One CTA takes 256 queries of one head as two tiles of 128 rows that share the key and value blocks.  Per
// block and tile: S = Q K^T into tensor memory (tcgen05, both operands from shared memory), one thread per
// row turns S into P (bf16, over the first half of S's columns), O += P V (tcgen05, P from tensor memory).
// While the threads of one tile work on its P, the tensor core works for the other tile: of a block of 128
// keys at d = 128 the products take 1024 clocks a tile and the 16,384 exponentials as many.  K and V come by
// TMA into two-stage rings.  Widths up to 64 use blocks of 64 keys, so that two CTAs fit an SM (256 columns
// of tensor memory and 96 KB each) and one's prologue and epilogue hide behind the other's work.
//
// Warps 0-3 and 4-7: rows of tile 0 and 1; warp 8: MMAs; warp 9: copies; warp 10: looks at each value block
// before it is used.  A value that a row does not see enters its product as 0 * v, which a NaN or an
// infinity would spoil: rows of padding are overwritten with zeros in shared memory, and where a block that
// is not seen as a whole holds other values that are not finite, the CTA computes its rows again, key by
// key, on the CUDA cores (a rare path: only the keys in a row's interval are touched there).
#include <mutex>

#include "layers.cuh"
#include "swa_common.cuh"
#include "tc.cuh"

namespace la {
namespace {
using namespace tc;

constexpr int kRows = 128;                    // queries per tile
constexpr int kThreads = 352;                 // 11 warps
constexpr uint32_t kStages = 2;
constexpr float kGrowth = 8.f;                // log2 of how far P may exceed 1 before the output is scaled

template <int DP>
struct Shape {
  static constexpr int KB = DP == 64 ? 64 : 128;             // keys per block
  static constexpr uint32_t kBlk = DP / 64;                  // 64-column blocks per row
  static constexpr uint32_t kQTile = kRows * DP * 2;         // bytes
  static constexpr uint32_t kKTile = KB * DP * 2;
  static constexpr uint32_t kOffK = 2 * kQTile, kOffV = kOffK + kStages * kKTile;
  static constexpr uint32_t kSmem = kOffV + kStages * kKTile + 1024;  // + alignment of the base
  static constexpr uint32_t kColO = 2 * KB, kTmemCols = 2 * KB + 2 * DP;
};

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
__device__ void slow_row(const SwaPrefillLaunch& a, int64_t b, int64_t h, int64_t hk, int64_t i, KeySpan sp, float slope2) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q.ptr) + b * a.q.sb + h * a.q.sh + i * a.q.st;
  const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(a.k.ptr) + b * a.k.sb + hk * a.k.sh;
  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v.ptr) + b * a.v.sb + hk * a.v.sh;
  const int pos = (int)(a.q_pos0 + i);
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

template <int DP, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 2 : 1)
swa_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const SwaPrefillLaunch a, int q_tiles) {
  using S = Shape<DP>;
  constexpr int KB = S::KB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bar_q, bar_k[kStages], bar_v[kStages], bar_kfree[kStages], bar_vfree[kStages];
  __shared__ uint64_t bar_vok[kStages];  // warp 10: the block holds what the products may read
  __shared__ uint64_t bar_s[2], bar_p[2], bar_o[2], bar_fin;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int r_lo[2], r_hi[2];       // keys that a tile's rows see: lowest lo, highest hi
  __shared__ int f_lo[2], f_hi[2];       // keys that every row sees that sees any: highest lo, lowest hi
  __shared__ int bad;                    // a block that is not seen as a whole holds a value that is not finite

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t heads = a.B * a.H;
  const int64_t bh = blockIdx.x % heads;
  // the last queries see the most keys under the causal mask: they start first
  const int64_t i0 = (int64_t)(q_tiles - 1 - blockIdx.x / heads) * (2 * kRows);
  const int64_t b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hkv);
  const int64_t len = sequence_length(a.lens, b, a.Nk, a.status, h == 0 && i0 == 0 && tid == 0);
  if (len < 0) return;  // uniform over the CTA
  const uint32_t sbase = smem_u32(sm);

  if (tid == 0) {
    mbar_init(smem_u32(&bar_q), 1);
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&bar_k[s]), 1);
      mbar_init(smem_u32(&bar_v[s]), 1);
      mbar_init(smem_u32(&bar_kfree[s]), 1);
      mbar_init(smem_u32(&bar_vfree[s]), 1);
      mbar_init(smem_u32(&bar_vok[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bar_s[t]), 1);
      mbar_init(smem_u32(&bar_p[t]), 4);  // one arrival per warp of the tile
      mbar_init(smem_u32(&bar_o[t]), 1);
      r_lo[t] = INT32_MAX;
      r_hi[t] = 0;
      f_lo[t] = 0;
      f_hi[t] = INT32_MAX;
    }
    mbar_init(smem_u32(&bar_fin), 1);
    fence_mbar_init();
    bad = 0;
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
  __syncthreads();
  // thread t < 256 owns row i0 + t
  KeySpan span{0, 0};
  if (warp < 8) {
    span = key_span(a, b, i0 + tid, len);
    const bool any = span.lo < span.hi;
    const int t = warp >> 2;
    const int lo = __reduce_min_sync(kFullMask, any ? span.lo : INT32_MAX), hi = __reduce_max_sync(kFullMask, any ? span.hi : 0);
    const int flo = __reduce_max_sync(kFullMask, any ? span.lo : 0), fhi = __reduce_min_sync(kFullMask, any ? span.hi : INT32_MAX);
    if (lane == 0 && lo < hi) {
      atomicMin(&r_lo[t], lo);
      atomicMax(&r_hi[t], hi);
      atomicMax(&f_lo[t], flo);
      atomicMin(&f_hi[t], fhi);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  // blocks [jb, je) of each tile, and of both
  int jb[2], je[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const bool any = r_lo[t] < r_hi[t];
    jb[t] = any ? r_lo[t] / KB : 0;
    je[t] = any ? (r_hi[t] + KB - 1) / KB : 0;
  }
  const bool any0 = jb[0] < je[0], any1 = jb[1] < je[1];
  const int J0 = any0 && any1 ? min(jb[0], jb[1]) : any0 ? jb[0] : jb[1];
  const int J1 = max(je[0], je[1]);
  auto active = [&](int t, int j) { return j >= jb[t] && j < je[t]; };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(smem_u32(bar), parity, a.status); };
  // waits of a whole warp whose lanes leave together
  auto wwait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFullMask, wait(bar, parity)); };
  // stage and parity of the i-th block that passes through a ring
  auto stage = [](uint32_t i) { return i % kStages; };
  auto phase = [](uint32_t i) { return (i / kStages) & 1u; };

  if (warp == 9) {
    // ================================================================ copies
    uint32_t i = 0;
    bool ok = true;
    if (J0 < J1 && lane == 0) {
      mbar_arrive_expect_tx(smem_u32(&bar_q), 2 * S::kQTile);
      for (int t = 0; t < 2; ++t)
        for (uint32_t c = 0; c < S::kBlk; ++c)
          tma_load_4d(sbase + t * S::kQTile + c * (kRows * 128), &map_q, c * 64, (int)i0 + t * kRows, (int)h, (int)b, smem_u32(&bar_q));
    }
    for (int j = J0; j < J1 && ok; ++j) {
      if (!active(0, j) && !active(1, j)) continue;
      const uint32_t s = stage(i);
      if (i >= kStages) ok = wwait(&bar_kfree[s], phase(i - kStages));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&bar_k[s]), S::kKTile);
        for (uint32_t c = 0; c < S::kBlk; ++c)
          tma_load_4d(sbase + S::kOffK + s * S::kKTile + c * (KB * 128), &map_k, c * 64, j * KB, (int)hk, (int)b, smem_u32(&bar_k[s]));
      }
      if (i >= kStages) ok = wwait(&bar_vfree[s], phase(i - kStages));
      if (!ok) {
        wwait(&bar_k[s], phase(i));  // the copy in flight lands before the CTA ends
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&bar_v[s]), S::kKTile);
        for (uint32_t c = 0; c < S::kBlk; ++c)
          tma_load_4d(sbase + S::kOffV + s * S::kKTile + c * (KB * 128), &map_v, c * 64, j * KB, (int)hk, (int)b, smem_u32(&bar_v[s]));
      }
      __syncwarp();
      ++i;
    }
    // nobody may be left to wait for the last blocks after an expired wait elsewhere: their copies land here
    for (uint32_t k = i > kStages ? i - kStages : 0; k < i; ++k) {
      wwait(&bar_k[stage(k)], phase(k));
      wwait(&bar_v[stage(k)], phase(k));
    }
    if (J0 < J1) wwait(&bar_q, 0);
  } else if (warp == 10) {
    // ================================================================ a look at each value block
    uint32_t i = 0;
    bool ok = true;
    for (int j = J0; j < J1 && ok; ++j) {
      const bool on0 = active(0, j), on1 = active(1, j);
      if (!on0 && !on1) continue;
      const uint32_t s = stage(i);
      ok = wwait(&bar_v[s], phase(i));
      if (!ok) break;
      uint8_t* v = sm + S::kOffV + s * S::kKTile;
      const int k0 = j * KB, k1 = k0 + KB;
      if (k1 > len) {  // rows of padding (TMA has zeroed those behind the last key only)
        for (int e = lane; e < (int)(S::kBlk * KB * 8); e += 32) {
          const int row = e / 8 % KB;
          if (k0 + row >= len) *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const bool whole = (!on0 || (k0 >= f_lo[0] && k1 <= f_hi[0])) && (!on1 || (k0 >= f_lo[1] && k1 <= f_hi[1]));
      if (!whole) {
        __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 8
        for (int e = lane; e < (int)(S::kBlk * KB * 8); e += 32) acc = add_zero_times(*reinterpret_cast<const uint4*>(v + e * 16), acc);
        if (__any_sync(kFullMask, __hisnan(acc.x) || __hisnan(acc.y)) && lane == 0) bad = 1;
      }
      warp_arrive(smem_u32(&bar_vok[s]));
      ++i;
    }
  } else if (warp == 8) {
    // ================================================================ products
    // Order: per block, tile 0 then tile 1: O += P V of the block before, then S = Q K^T of this one over
    // the same columns.  Products of one thread run in order, so S follows the reads of P, and the
    // completion that announces S covers the products before it.
    const uint32_t id_s = idesc_bf16(kRows, KB, 0, 0), id_o = idesc_bf16(kRows, DP, 0, 1);
    bool ok = J0 >= J1 || wwait(&bar_q, 0);
    bool issued = false;
    uint32_t i = 0, np[2] = {0u, 0u};
    bool have_prev = false;
    for (int j = J0; j <= J1 && ok; ++j) {
      const bool cur = j < J1 && (active(0, j) || active(1, j));
      if (!cur && !have_prev) continue;
      const uint32_t s = stage(i), sp = stage(i - 1);
      if (cur) {
        ok = wwait(&bar_k[s], phase(i));
        if (!ok) break;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (have_prev && active(t, j - 1)) {
          ok = ok && wwait(&bar_p[t], np[t] & 1u) && wwait(&bar_vok[sp], phase(i - 1));
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t v = sbase + S::kOffV + sp * S::kKTile;
#pragma unroll
            for (int ks = 0; ks < KB / 16; ++ks)
              mma_bf16_ts(tmem + S::kColO + t * DP, tmem + t * KB + 8 * ks, sw128_desc(v + ks * 2048, KB * 128, 1024), id_o,
                          (np[t] > 0 || ks > 0) ? 1u : 0u);
            if (j == je[t]) mma_commit(smem_u32(&bar_o[t]));
          }
          ++np[t];
          issued = true;
        }
        if (cur && active(t, j)) {
          tc_fence_after();
          if (lane == 0) {
            const uint32_t q = sbase + t * S::kQTile, k = sbase + S::kOffK + s * S::kKTile;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
              const uint32_t blk = ks >> 2, in = (ks & 3) * 32;
              mma_bf16(tmem + t * KB, sw128_desc(q + blk * (kRows * 128) + in, 0, 1024), sw128_desc(k + blk * (KB * 128) + in, 0, 1024),
                       id_s, ks > 0);
            }
            mma_commit(smem_u32(&bar_s[t]));
          }
          issued = true;
        }
      }
      if (!ok) break;
      if (lane == 0) {
        if (have_prev) mma_commit(smem_u32(&bar_vfree[sp]));
        if (cur) mma_commit(smem_u32(&bar_kfree[s]));
      }
      __syncwarp();
      if (cur) ++i;
      have_prev = cur;
    }
    if (issued) {  // every product has completed before tensor memory is given back
      if (lane == 0) mma_commit(smem_u32(&bar_fin));
      __syncwarp();
      wwait(&bar_fin, 0);
    }
  } else {
    // ================================================================ one thread per row
    const int t = warp >> 2;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t col_s = tl + t * KB, col_o = tl + S::kColO + t * DP;
    const int64_t i = i0 + tid;
    const int pos = (int)(a.q_pos0 + i);
    const float c1 = CAP ? a.scale / a.softcap * (2.f * kLog2e) : a.scale * kLog2e;
    const float capl = a.softcap * kLog2e;
    const float slope2 = BIAS ? a.slopes[h] * kLog2e : 0.f;
    float m = -INFINITY, l = 0.f;
    uint32_t n = 0;
    bool ok = true;
    for (int j = jb[t]; j < je[t]; ++j, ++n) {
      ok = ok && wait(&bar_s[t], n & 1u);
      __syncwarp();
      tc_fence_after();
      float x[KB];
#pragma unroll
      for (int c = 0; c < KB; c += 32) tmem_ld32(col_s + c, x + c);
      tmem_ld_wait();
      const int k0 = j * KB;
#pragma unroll
      for (int c = 0; c < KB; ++c) {
        if constexpr (CAP) x[c] = fmaf(-2.f * capl, rcp(1.f + ex2(x[c] * c1)), capl);  // cap tanh(y) = cap - 2 cap / (1 + e^2y)
        else x[c] *= c1;
      }
      if constexpr (BIAS) {
        const float dist = (float)(pos - k0);
#pragma unroll
        for (int c = 0; c < KB; ++c) x[c] = fmaf(-slope2, fabsf(dist - (float)c), x[c]);
      }
      const int va = span.lo - k0, vb = span.hi - k0;  // columns va <= c < vb are seen
      if (!__all_sync(kFullMask, va <= 0 && vb >= KB)) {
#pragma unroll
        for (int c = 0; c < KB; ++c) x[c] = c >= va && c < vb ? x[c] : -INFINITY;
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < KB; ++c) mx[c & 3] = fmaxf(mx[c & 3], x[c]);
      const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (m == -INFINITY) {
        m = mn;  // nothing seen before: the output holds zeros, or nothing yet
      }
      const bool grow = mn > m + kGrowth;
      if (__any_sync(kFullMask, grow)) {
        // S of this block was announced after P V of the block before: the output is at rest
        const float f = grow ? ex2(m - mn) : 1.f;
        if (grow) m = mn;
        l *= f;
        if (n > 0) {
#pragma unroll
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
      const float base = m == -INFINITY ? 0.f : m;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KB; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float p0 = ex2(x[c + e] - base), p1 = ex2(x[c + e + 1] - base);
          sum[e & 3] += p0;
          sum[(e & 3) + 1] += p1;
          w[e / 2] = pack2_bf16(p0, p1);
        }
        tmem_st16u(col_s + c / 2, w);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(smem_u32(&bar_p[t]));
    }
    if (n > 0) {
      ok = ok && wait(&bar_o[t], 0);
      __syncwarp();
      tc_fence_after();
    }
    const bool stored = ok && i < a.Nq && a.q_pos0 + i < len;
    const bool seen = l != 0.f;  // also a row whose sum is NaN
    const float inv = seen ? 1.f / l : 0.f;
    const int64_t at = b * a.o_sb + h * a.o_sh + i * a.o_st;
    const bool al32 = ((reinterpret_cast<uintptr_t>(a.o) | (uintptr_t)((a.o_sb | a.o_sh | a.o_st) * (a.out_bf16 ? 2 : 4))) & 31u) == 0;
#pragma unroll
    for (int c = 0; c < DP; c += 16) {
      float o[16];
      if (n > 0) {
        tmem_ld16(col_o + c, o);
        tmem_ld_wait();
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = seen ? o[e] * inv : 0.f;
      if (stored && c < a.d) {
        const bool two = c + 8 < a.d;  // d is a multiple of 8
        if (a.out_bf16) {
          __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(a.o) + at + c;
          const uint4 lo8 = pack8_bf16(o), hi8 = pack8_bf16(o + 8);
          if (two && al32) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(lo8.x), "r"(lo8.y), "r"(lo8.z),
                         "r"(lo8.w), "r"(hi8.x), "r"(hi8.y), "r"(hi8.z), "r"(hi8.w)
                         : "memory");
          } else {
            *reinterpret_cast<uint4*>(p) = lo8;
            if (two) *reinterpret_cast<uint4*>(p + 8) = hi8;
          }
        } else {
          float* p = reinterpret_cast<float*>(a.o) + at + c;
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            if (e < 8 || two) *reinterpret_cast<float4*>(p + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, S::kTmemCols);
  if (bad && warp < 8) {
    // the rows again, a warp at a time, from their own keys only
    const float slope2 = BIAS ? a.slopes[h] * kLog2e : 0.f;
    for (int r = 0; r < 32; ++r) {
      const int64_t i = i0 + warp * 32 + r;
      const KeySpan sp{__shfl_sync(kFullMask, span.lo, r), __shfl_sync(kFullMask, span.hi, r)};
      if (i < a.Nq && a.q_pos0 + i < len) slow_row<CAP, BIAS>(a, b, h, hk, i, sp, slope2);
    }
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// [B, H, N, d] bf16 view as boxes of `rows` x 64 columns, columns and rows behind the ends filled with zeros
bool encode(CUtensorMap* map, const View4& x, int64_t B, int64_t H, int64_t N, int d, int rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
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

template <int DP, bool CAP, bool BIAS>
cudaError_t launch_typed(const SwaPrefillLaunch& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(swa_tc_kernel<DP, CAP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<DP>::kSmem);
  });
  if (attr != cudaSuccess) return attr;
  const int q_tiles = (int)((a.Nq + 2 * kRows - 1) / (2 * kRows));
  swa_tc_kernel<DP, CAP, BIAS><<<(unsigned)(a.B * a.H * q_tiles), kThreads, Shape<DP>::kSmem, stream>>>(q, k, v, a, q_tiles);
  return cudaGetLastError();
}

template <int DP>
cudaError_t launch_width(const SwaPrefillLaunch& a, cudaStream_t stream) {
  CUtensorMap q, k, v;
  if (!encode(&q, a.q, a.B, a.H, a.Nq, a.d, kRows) || !encode(&k, a.k, a.B, a.Hkv, a.Nk, a.d, Shape<DP>::KB) ||
      !encode(&v, a.v, a.B, a.Hkv, a.Nk, a.d, Shape<DP>::KB))
    return cudaErrorNotSupported;  // strides that TMA cannot describe
  const bool cap = a.softcap != 0.f, bias = a.slopes != nullptr;
  if (cap && bias) return launch_typed<DP, true, true>(a, q, k, v, stream);
  if (cap) return launch_typed<DP, true, false>(a, q, k, v, stream);
  if (bias) return launch_typed<DP, false, true>(a, q, k, v, stream);
  return launch_typed<DP, false, false>(a, q, k, v, stream);
}

}  // namespace

cudaError_t launch_swa_prefill_tc(const SwaPrefillLaunch& a, cudaStream_t stream) {
  return a.d <= 64 ? launch_width<64>(a, stream) : launch_width<128>(a, stream);
}

}  // namespace la
