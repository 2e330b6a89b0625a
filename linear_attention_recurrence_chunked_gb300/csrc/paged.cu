// paged.cu -- keys and values of new tokens into a paged cache, the keys rotated on the way, and a cache's tokens back into
// rows.  Both read and write every element once, so memory bounds them.  As in heads.cu a lane has eight elements of a row,
// for 4 bits always consecutive ones: one 32-bit word of codes, whose group of 64 elements is eight neighbouring lanes.
// 8 ragged prompts of up to 4096 tokens, 4 heads x 128, bf16: 19 us for 102 MB, 5.3 TB/s (24 with a warp for the keys and one for
// the values, 22 with four rows of each at once); 4 x 2048 tokens of 8 heads into 4 bits 22 us (half of the instructions
// rotation and codes), 4 x up to 16048 tokens back 48 us, 6.7 TB/s.  4 x 16048 tokens of bf16 pages back 78 us, 99 % of the
// measured copy rate; 8 x 16048 of d = 32, two rows of a lane at once, 40.5 us, 96 %.
#include <type_traits>

#include "paged.cuh"

namespace la {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 2;   // rows of a lane on their way at once, of the keys and of the values, in an append
constexpr int kReads = 4;  // and in a read, where a lane has as many of a tile's tokens
constexpr int kTokens = 16;  // of a read's tile; a page holds a multiple

int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : 16; }

// x c + y s, the exact value rounded to fp32 but for a 2^-20th of an ulp: the products' errors and the sum's (Knuth's two-sum)
// are added last.  Next to a border of the 4-bit codes an fp32 rounding more could be a whole code.
__device__ __forceinline__ f32x2 turn_exact(f32x2 x, f32x2 c, f32x2 y, f32x2 s) {
  const f32x2 minus = pack2(-1.f, -1.f);
  auto sub = [&](f32x2 a, f32x2 b) { return fma2(b, minus, a); };
  const f32x2 p = mul2(x, c), ep = fma2(x, c, mul2(p, minus));
  const f32x2 q = mul2(y, s), eq = fma2(y, s, mul2(q, minus));
  const f32x2 sum = add2(p, q), t = sub(sum, p);
  const f32x2 es = add2(sub(p, sub(sum, t)), sub(q, t));
  return add2(sum, add2(es, add2(ep, eq)));  // of an infinity NaN, as the whole group then is
}

// A lane's angles for eight consecutive elements, whose partners at rot / 2 are those of lane +- rot / 16.
template <TurnKind kTurn>
struct TurnWide {
  bool on;
  int partner;
  f32x2 c[4], s[4];  // s negative for a pair's first element
  __device__ __forceinline__ void init(const float* cos, const float* sin, int rot, int lane, int col) {
    on = col * 8 < rot;
    partner = lane;
    if (!on) return;
    if constexpr (kTurn == kTurnNeighbours) {
      Turn<kTurnNeighbours> t;
      t.init(cos, sin, rot, col);
#pragma unroll
      for (int i = 0; i < 4; ++i) { c[i] = t.c[i]; s[i] = t.s[i]; }
    } else {
      const int half = rot / 16;  // lanes of the pairs' first elements
      const bool second = col >= half;
      partner = second ? lane - half : lane + half;
      const int at = 8 * (second ? col - half : col);
      Raw8<float> r;
      r.load<true>(cos, make_int2(at, at + 4));
      r.unpack(c);
      r.load<true>(sin, make_int2(at, at + 4));
      r.unpack(s);
      if (!second) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = mul2(s[i], pack2(-1.f, -1.f));
      }
    }
  }
  __device__ __forceinline__ void apply(Raw8<__nv_bfloat16>& raw) const {
    f32x2 v[4], u[4];
    raw.unpack(v);
    if constexpr (kTurn == kTurnNeighbours) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(v[i], lo, hi);
        u[i] = pack2(hi, lo);
      }
    } else {
      Raw8<__nv_bfloat16> other;
      other.a.x = __shfl_sync(kFullMask, raw.a.x, partner); other.a.y = __shfl_sync(kFullMask, raw.a.y, partner);
      other.b.x = __shfl_sync(kFullMask, raw.b.x, partner); other.b.y = __shfl_sync(kFullMask, raw.b.y, partner);
      other.unpack(u);
    }
    if (!on) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = turn_exact(v[i], c[i], u[i], s[i]);
    raw.pack(v);
  }
};

__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

constexpr float kLargestSpread = 0x1p119f;  // 16 scale times a weight of 2^8 stays within fp32

// Eight elements of a lane, whose group is eight neighbouring lanes: their codes and the group's scale (lower half) and offset.
__device__ __forceinline__ void quantise(const Raw8<__nv_bfloat16>& raw, uint32_t& codes, uint32_t& meta) {
  uint32_t lo2 = min_nan2(min_nan2(raw.a.x, raw.a.y), min_nan2(raw.b.x, raw.b.y));
  uint32_t hi2 = max_nan2(max_nan2(raw.a.x, raw.a.y), max_nan2(raw.b.x, raw.b.y));
  lo2 = min_nan2(lo2, __byte_perm(lo2, lo2, 0x1032));  // the least of the lane in both halves
  hi2 = max_nan2(hi2, __byte_perm(hi2, hi2, 0x1032));
  uint32_t ends = __byte_perm(lo2, hi2, 0x5410);  // least, greatest
#pragma unroll
  for (int off = 4; off >= 1; off /= 2) {
    const uint32_t other = __shfl_xor_sync(kFullMask, ends, off);
    ends = __byte_perm(min_nan2(ends, other), max_nan2(ends, other), 0x7610);
  }
  const float lo = __uint_as_float(ends << 16), spread = __uint_as_float(ends & 0xffff0000u) - lo;
  codes = 0;
  if (!(spread < kLargestSpread)) {  // NaN too
    meta = 0x7fc07fc0u;
    return;
  }
  // spread / 15 correctly rounded: a quotient with the rounded reciprocal, corrected by its remainder (Markstein 1990); all
  // 2^24 significands of two binades were compared with the division.
  constexpr float kFifteenth = 1.f / 15.f;
  const float q = spread * kFifteenth;
  const bool small = spread < 0x1p-100f;  // where remainders lose bits
  const __nv_bfloat16 step = __float2bfloat16_rn(small ? __fdiv_rn(spread, 15.f) : fmaf(fmaf(-15.f, q, spread), kFifteenth, q));
  float scale = __bfloat162float(step);
  meta = (uint32_t)__bfloat16_as_ushort(step) | ends << 16;
  f32x2 v[4];
  raw.unpack(v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = add2(v[i], pack2(-lo, -lo));
  if (small) {  // the same quotients of larger numbers
    scale *= 0x1p100f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], pack2(0x1p100f, 0x1p100f));
  }
  if (!(scale > 0.f)) return;
  // Bf16 elements often lie on a border, so the quotient has to be the rounded one (the remainder again): a border, which fp32
  // holds, then comes out as it is, and what is next to one does not.  The sum with 1.5 * 2^23 rounds it to even.
  const float inv = rcp(scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 y = mul2(v[i], pack2(inv, inv));
    f32x2 quotient = fma2(fma2(y, pack2(-scale, -scale), v[i]), pack2(inv, inv), y);
    float z[2];
    if (small) {  // where a scale has few bits, quotients can pass 15
      unpack2(quotient, z[0], z[1]);
      quotient = pack2(fminf(z[0], 15.f), fminf(z[1], 15.f));
    }
    unpack2(add2(quotient, pack2(12582912.f, 12582912.f)), z[0], z[1]);
    codes += __float_as_uint(z[0]) << (8 * i);
    codes += __float_as_uint(z[1]) << (8 * i + 4);
  }
  codes -= 0x4b400000u * 0x11111111u;  // the sums' bits are 0x4b400000 + code
}

// Where a token goes.
struct Place {
  int page, slot;
};

// A token's keys or values of some heads, kRows rows of each lane at a time: on their way from `load` on, stored by `store`.
template <typename T, bool kFour, int LPR, TurnKind kTurn>
struct HeadRows {
  static constexpr int R = 32 / LPR;
  static constexpr bool kWhole = kFour || kTurn != kTurnHalves;
  const T* x;
  int64_t step;
  int2 at;
  int left;  // this lane's rows: every R-th while it is positive
  Raw8<T> raw[kRows];

  __device__ __forceinline__ HeadRows(const PagedAppendLaunch& a, const Span4& view, uint32_t b, uint32_t n, int h0, int heads) {
    const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
    const bool on = col * 8 < (kFour ? 8 * LPR : a.c.d);
    at = runs_of<kFour ? kTurnNone : kTurn>(on ? col : 0, a.rot);
    x = view.at<const T>(b, h0 + sub, n);
    step = R * view.step<T>();
    left = on ? heads - sub : 0;
    load();
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      raw[i].zero();
      if (left > i * R) raw[i].template load<kWhole>(x, at);
      x += step;
    }
  }
  template <typename Angles>
  __device__ __forceinline__ void store(const PagedAppendLaunch& a, void* pool, const Place& place, int h0, int heads, const Angles& turn) {
    const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR, d = kFour ? 8 * LPR : a.c.d, size = page_bytes(a.c);
    uint8_t* y = static_cast<uint8_t*>(pool) + ((uint64_t)(uint32_t)place.page * (uint32_t)a.c.Hkv + (uint32_t)(h0 + sub)) * (uint32_t)size;
#pragma unroll 1
    for (int more = heads;;) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (more <= i * R) break;  // the same for the whole warp
        if constexpr (kFour) {
          if constexpr (kTurn != kTurnNone) turn.apply(raw[i]);
          uint32_t codes, meta;
          quantise(raw[i], codes, meta);
          constexpr int kGroups = LPR / 8;
          if (left > i * R) {
            reinterpret_cast<uint32_t*>(y + place.slot * (d / 2))[code_word(col / 8, col % 8, kGroups)] = codes;
            if (col % 8 == 0) reinterpret_cast<uint32_t*>(y + a.c.page * (d / 2))[place.slot * kGroups + col / 8] = meta;
          }
        } else if (left > i * R) {
          if (kTurn != kTurnNone && turn.on) {  // other rows and elements go as they are, whatever they hold
            f32x2 v[4];
            raw[i].unpack(v);
            turn.apply(v, turn_rounded);
            raw[i].pack(v);
          }
          raw[i].template store<kWhole>(reinterpret_cast<T*>(y) + place.slot * d, at);
        }
        y += (int64_t)R * size;
      }
      more -= kRows * R;
      if (more <= 0) return;
      left -= kRows * R;
      load();
    }
  }
};

// A warp stores a token's keys and values, `per` heads of them: one look at where it goes, while its first rows are on their way.
template <typename T, bool kFour, int LPR, TurnKind kTurn>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 6 : 8)
paged_append_kernel(const PagedAppendLaunch a, const int per, const Divisor parts, const Divisor tokens, const Divisor pages) {
  using Angles = std::conditional_t<kFour, TurnWide<kTurn>, Turn<kTurn>>;
  grid_dependents_trigger();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, col = lane % LPR;
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), token = parts(unit), b = tokens(token), n = token - b * tokens.d;
  if (b >= a.B) return;  // whole warps
  const int part = (int)(unit - token * parts.d), h0 = part * per, heads = min(per, (int)a.c.Hkv - h0);
  const bool report = part == 0 && lane == 0;
  HeadRows<T, kFour, LPR, kTurn> keys(a, a.k, b, n, h0, heads);
  HeadRows<T, kFour, LPR, kTurnNone> values(a, a.v, b, n, h0, heads);

  if (n >= sequence_length(a.lens, b, a.N, a.c.status, report && n == 0)) return;
  const int64_t position = table_row(a.seen[b], n, a.c.width * a.c.page);  // below 2^31
  const int column = (int)pages((uint32_t)position);
  Place place;
  place.page = position < 0 || (kTurn != kTurnNone && position >= a.positions) ? -1 : table_page(a.c, b, column);
  place.slot = (int)position - column * a.c.page;
  if (place.page < 0) {
    if (report) atomicOr(a.c.status, kStatusBadIndex);
    return;
  }
  Angles turn;
  turn.on = false;
  if constexpr (kTurn != kTurnNone) {
    const uint64_t row = (uint64_t)(uint32_t)position * (uint32_t)(a.rot / 2);
    if constexpr (kFour) turn.init(a.cos + row, a.sin + row, a.rot, lane, col);
    else if (col * 8 < a.c.d) turn.init(a.cos + row, a.sin + row, a.rot, col);
  }
  keys.store(a, a.c.k, place, h0, heads, turn);
  values.store(a, a.c.v, place, h0, heads, turn);
}

// A warp reads a tile of kTokens tokens, which lie in one page, of one head's keys or values.
template <typename T, typename TOut, bool kFour, int LPR>
__global__ void __launch_bounds__(kThreads)
paged_read_kernel(const PagedReadLaunch a, const Divisor tiles, const Divisor heads2, const Divisor pages) {
  constexpr int R = 32 / LPR, kLane = kTokens / R, kBatch = kReads < kLane ? kReads : kLane;  // a lane's rows of a tile, and at once
  static_assert(kLane % kBatch == 0, "a whole tile's batches check no row");
  const int lane = threadIdx.x & 31, col = lane % LPR, sub = lane / LPR;
  grid_dependents_trigger();
  grid_dependency_wait();
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), bhv = tiles(unit), b = heads2(bhv);
  if (b >= a.B) return;  // whole warps
  const int n0 = (int)(unit - bhv * tiles.d) * kTokens;
  const bool values = bhv & 1;
  const int h = (int)(bhv - b * heads2.d) >> 1, d = a.c.d;
  const bool on = col * 8 < d, report = lane == 0 && h == 0 && !values;
  const int len = (int)sequence_length(a.lens, b, a.N, a.c.status, report && n0 == 0), end = min(n0 + kTokens, (int)a.N);
  int have = max(n0, min(len, end));  // tokens below are in the cache
  int page = -1, slot = 0;
  if (n0 < have) {
    const int column = (int)pages((uint32_t)n0);
    slot = n0 - column * a.c.page;
    page = column < a.c.width ? table_page(a.c, b, column) : -1;
    if (page < 0) {
      if (report) atomicOr(a.c.status, kStatusBadIndex);
      have = n0;
    }
  }
  if (have == n0 && !a.fill) return;
  if (!on) return;  // no lane waits for another from here on
  const uint8_t* x = static_cast<const uint8_t*>(values ? a.c.v : a.c.k) + ((uint64_t)max(page, 0) * (uint32_t)a.c.Hkv + h) * (uint32_t)page_bytes(a.c);
  const Span4& out = values ? a.v : a.k;
  TOut* y = out.at<TOut>(b, h, n0 + sub);
  const int2 at = make_int2(8 * col, 8 * col + 4);
  const int there = have - n0 - sub, wanted = (a.fill ? end : have) - n0 - sub;  // this lane's rows: every R-th below
  constexpr int kGroups = LPR / 8, kWords = LPR;  // of a 4-bit row
  const uint32_t* words = reinterpret_cast<const uint32_t*>(x) + (slot + sub) * kWords + code_word(col / 8, col % 8, kGroups);
  const uint32_t* metas = reinterpret_cast<const uint32_t*>(x + a.c.page * (kWords * 4)) + (slot + sub) * kGroups + col / 8;
  const T* rows = reinterpret_cast<const T*>(x) + (int64_t)(slot + sub) * d;
  const int64_t yr = (int64_t)R * out.st * (16 / sizeof(TOut));
  uint32_t magic = 0x43004300u;  // two bf16 128
  asm volatile("" : "+r"(magic));

  auto batch = [&](auto all, int i0) {  // all: every row is there
    [[maybe_unused]] Raw8<T> raw[kBatch];
    [[maybe_unused]] uint32_t codes[kBatch], meta[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!decltype(all)::value && there <= (i0 + i) * R) continue;
      if constexpr (kFour) {
        codes[i] = words[i * R * kWords];
        meta[i] = metas[i * R * kGroups];
      } else {
        raw[i].template load<true>(rows + i * R * d, at);
      }
    }
    words += kBatch * R * kWords;
    metas += kBatch * R * kGroups;
    rows += kBatch * R * d;
#pragma unroll
    for (int i = 0; i < kBatch; ++i, y += yr) {
      if (!decltype(all)::value && wanted <= (i0 + i) * R) continue;
      f32x2 v[4];
      Raw8<TOut> packed;
      if (!decltype(all)::value && there <= (i0 + i) * R) {
        packed.zero();
      } else {
        if constexpr (kFour) {
          const f32x2 scale = Raw8<__nv_bfloat16>::wide(__byte_perm(meta[i], 0u, 0x1010)), offset = Raw8<__nv_bfloat16>::wide(__byte_perm(meta[i], 0u, 0x3232));
          float c[8];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            // codes m and m + 4 as bf16 128 + code, exact, and no conversion, of which an SM makes 16 a clock
            uint32_t w;
            asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(w) : "r"(codes[i] >> (4 * m)), "r"(magic));
            const f32x2 code = add2(Raw8<__nv_bfloat16>::wide(w), pack2(-128.f, -128.f));
            unpack2(fma2(code, scale, offset), c[m], c[4 + m]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = pack2(c[2 * e], c[2 * e + 1]);
        } else {
          raw[i].unpack(v);
        }
        packed.pack(v);
      }
      packed.template store<true>(y, at);
    }
  };
  if (have == n0 + kTokens) {
#pragma unroll
    for (int i0 = 0; i0 < kLane; i0 += kBatch) batch(std::true_type{}, i0);
  } else {
#pragma unroll 1
    for (int i0 = 0; i0 < kLane; i0 += kBatch) batch(std::false_type{}, i0);
  }
}

template <typename T, bool kFour, int LPR, TurnKind kTurn>
cudaError_t append_turn(const PagedAppendLaunch& a, cudaStream_t stream) {
  constexpr int R = 32 / LPR;
  int per = R;
  int64_t parts = 0;
  for (int m = 8; m >= 1; m /= 2) {  // as many heads a warp as leave 32 warps to each of 152 SMs
    per = R * m;
    parts = (a.c.Hkv + per - 1) / per;
    if (a.B * a.N * parts >= 152 * 32) break;
  }
  const int64_t blocks = (a.B * a.N * parts + kWarps - 1) / kWarps;
  return launch_dependent(paged_append_kernel<T, kFour, LPR, kTurn>, dim3((unsigned)blocks), kThreads, 0, stream, a, per, Divisor(parts), Divisor(a.N), Divisor(a.c.page));
}
template <typename T, bool kFour, int LPR>
cudaError_t append(const PagedAppendLaunch& a, cudaStream_t stream) {
  return a.rot == 0 ? append_turn<T, kFour, LPR, kTurnNone>(a, stream) : a.interleaved ? append_turn<T, kFour, LPR, kTurnNeighbours>(a, stream)
                                                                       : append_turn<T, kFour, LPR, kTurnHalves>(a, stream);
}

template <typename T, typename TOut, bool kFour, int LPR>
cudaError_t read(const PagedReadLaunch& a, cudaStream_t stream) {
  const int64_t tiles = (a.N + kTokens - 1) / kTokens, blocks = (2 * a.B * a.c.Hkv * tiles + kWarps - 1) / kWarps;
  return launch_dependent(paged_read_kernel<T, TOut, kFour, LPR>, dim3((unsigned)blocks), kThreads, 0, stream, a, Divisor(tiles), Divisor(2 * a.c.Hkv), Divisor(a.c.page));
}

template <typename T, typename TOut>
cudaError_t read_rows(const PagedReadLaunch& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.c.d);
  return lanes == 4 ? read<T, TOut, false, 4>(a, stream) : lanes == 8 ? read<T, TOut, false, 8>(a, stream) : read<T, TOut, false, 16>(a, stream);
}

template <typename T>
cudaError_t append_rows(const PagedAppendLaunch& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.c.d);
  return lanes == 4 ? append<T, false, 4>(a, stream) : lanes == 8 ? append<T, false, 8>(a, stream) : append<T, false, 16>(a, stream);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.c.four) return a.c.d == 64 ? append<bf, true, 8>(a, stream) : append<bf, true, 16>(a, stream);
  return a.c.bf16 ? append_rows<bf>(a, stream) : append_rows<float>(a, stream);
}

cudaError_t launch_paged_read(const PagedReadLaunch& a, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.c.four && a.c.d == 64) return a.out_bf16 ? read<bf, bf, true, 8>(a, stream) : read<bf, float, true, 8>(a, stream);
  if (a.c.four) return a.out_bf16 ? read<bf, bf, true, 16>(a, stream) : read<bf, float, true, 16>(a, stream);
  if (a.c.bf16) return a.out_bf16 ? read_rows<bf, bf>(a, stream) : read_rows<bf, float>(a, stream);
  return a.out_bf16 ? read_rows<float, bf>(a, stream) : read_rows<float, float>(a, stream);
}

}  // namespace la
