// Chunk attention on the 5th-generation tensor cores (sm_100a).
//
// For row i of a tile of 128 or 256 rows (a row is a token and one of the query
// heads that share the KV head), over the keys j that it sees,
//   out_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i),
//   s_ij = sm_scale log2(e) q_i . k_j,
// with a reference m_i that follows the running maximum.  At most 16 rows of 4-bit
// and 2-bit cells go to chunk_few.cuh, all else comes here.  Both products are
// 128 x N x 16 fp16 ones with fp32 sums in tensor memory.  fp16 and not bf16:
// with 8 bits the rounding of dequantised keys alone moved the weights by half a
// percent where channels stick out; powers of two a block keep it in range.
//
// One CTA: four warps for the softmax of each 128 rows (a row a thread), eight
// that turn a block of 16 stored tokens each into fp16 rows of a tile of 128
// (two stages of keys and of values), one that issues the products.  A step is
// 64 keys: its logits are read once, into registers, so that the next step's
// products run while its weights are worked out; the weights go back to tensor
// memory (two buffers) as the left operand of the second product.  Few CTAs
// split the context over a cluster and join through its shared memory.
//
// Measured on a B200 (device time), 16 heads of 128 over 4-bit cells: 2048
// tokens at 16384: 371 us, 695 TFLOP/s, 42 % of measured; 4 x up to 512 tokens
// beside 2048 stored: 67 us; bf16 cells, 6 x up to 301 tokens, 16 heads on 4 KV
// heads, context up to 1801: 58 us.  Bound by the softmax warps' latency (issue
// 60 % busy, tensor pipe 38 %, exp unit 31 %).  With 256 rows the compiler spills
// 16 to 28 bytes a thread.  The end of the kernel works its place out anew: what
// it needs, held over the steps, cost 395 us.
// Steps of 128 keys that reuse their logits' columns for the weights: 428-490 us
// (each product waits for the softmax); 16 dequantising warps of 56 registers:
// 510 us (spills); bf16x2-free softmax in scalar operations: 3 % slower.
#pragma once

#include <cuda_fp16.h>

#include "chunk_common.cuh"
#include "tcgen05.cuh"

namespace loopkv {

constexpr int kTileKeys = 128;                       // keys of one tile: eight blocks
constexpr int kStepKeys = 64;                        // keys of one step of products and softmax
constexpr int kBlockWarps = kTileKeys / kBlock;      // dequantising warps, a block each
constexpr int kExpRing = 4;
constexpr int kPolyPair = 3;                         // of four pairs of weights, the one worked out on the FMA units

// A block's keys (values) are stored as x 2^-e with e such that the largest is
// in [2^-7, 2^-6): then 2^24 times a 4-bit scale, at most 2^24 2 2^-6 / 15 <
// 35000 (2^22 times a 2-bit one: 2^22 2 2^-6 / 3 < 43700), is a finite fp16
// number (rounded to 16 bits as well), and the code itself, read as a subnormal
// fp16 number (code 2^-24; 2-bit codes stand two bits higher), needs no conversion.
constexpr int kTopExp = -6;

// The outputs of a row are held in units of 2^(m + v): m is the reference of its
// logits (of their sum too), v an exponent that with it follows the largest
// contribution so far, max over the blocks that the row sees of
// 2^(largest logit) 2^(value exponent).  A weight in fp16 is then 2^(logit - m)
// 2^(value exponent - v) <= 2^12 and precise relative to what the row adds up,
// whatever lies in blocks that it masks or gives no weight.
//
// A block's exponent below v counts down to 2^-60: what it adds is nothing beside
// the largest contribution, and the weights stay far above the 2^-126 that the
// exponentials end at.  (Above v it has no end: its logits are as far below m.)
constexpr float kLeastShift = -60.f;
constexpr float kNoValueRef = -1000.f;  // v before the first
constexpr float kLogitAbove = 8.f, kMostAbove = 12.f;  // what is not above m, v by more does not move them

// Whether a row's references move: its largest new logit, and the largest of its
// blocks' logits and value exponents together.
__device__ __forceinline__ bool refs_move(float m, float v, float top, float most) {
  return !(top <= m + kLogitAbove) || most > m + v + kMostAbove;
}
// m of a row after new logits of which `top` is the largest.  A NaN among them, or
// +inf, whose weight is inf - inf, is the row's reference from then on: the
// weights, the sum and with them all of the row are NaN.
__device__ __forceinline__ float logit_ref(float m, float top) {
  top = top < INFINITY ? top : NAN;
  return top > m + kLogitAbove || top != top ? top : m;
}
// v of a row whose reference moves from m to m_new and whose largest new
// contribution is 2^(m_new + most).  Rounded so that 2^(m + v) of what is there
// never grows by itself; and brought up to the new contribution, since O is
// rescaled anyway (left 2^12 behind, it would have to follow again soon).
__device__ __forceinline__ float value_ref(float v, float m, float m_new, float most) {
  if (m_new != m) v = m == -INFINITY ? kNoValueRef : fmaxf(v - ceilf(m_new - m), kNoValueRef);
  return fmaxf(v, ceilf(most));
}

// A partial result of a row: its outputs are in units of 2^(m + v), its sum of 2^m.
struct alignas(16) RowStats {
  float m, sum, v;
};

// The references of several partial results together: m is their largest, m + v the
// largest unit, and both NaN where one is.  `next` gives them one after another.
template <typename Next>
__device__ __forceinline__ RowStats join_refs(int count, Next&& next) {
  float m = -INFINITY, unit = -INFINITY;
  for (int i = 0; i < count; ++i) {
    const RowStats s = next(i);
    m = max_nan(m, s.m);
    unit = max_nan(unit, s.m == -INFINITY ? -INFINITY : s.m + s.v);
  }
  return RowStats{m, 0.f, unit - m};
}
// One of them into sum and outputs; skipped where it saw no key, or none with a
// weight.  An output is never given a weight of 0: it may be an infinity.
__device__ __forceinline__ void join_part(RowStats& all, const RowStats& s, float4& acc, const float4& x) {
  const float d = s.m - all.m, w = max_nan(fast_exp2(d + s.v - all.v), 0x1p-126f);
  all.sum = fmaf(fast_exp2(d), s.sum, all.sum);
  acc.x = fmaf(w, x.x, acc.x), acc.y = fmaf(w, x.y, acc.y), acc.z = fmaf(w, x.z, acc.z), acc.w = fmaf(w, x.w, acc.w);
}
// Outputs over sum, times their unit, in two steps: v may be beyond 127, and the
// average be finite where its sum is not.  0 / 0 where no logit is above -inf.
__device__ __forceinline__ uint2 join_result(const RowStats& all, const float4& acc) {
  const float inv = 1.f / all.sum, unit = fast_exp2(all.v * 0.5f);
  return make_uint2(pack_bf16(acc.x * inv * unit * unit, acc.y * inv * unit * unit),
                    pack_bf16(acc.z * inv * unit * unit, acc.w * inv * unit * unit));
}

template <int D, int MT>
struct ChunkSmem {
  static constexpr int kTile = kTileKeys * D * 2;    // one K or V stage, one Q tile
  static constexpr int kQ = 0;
  static constexpr int kK = MT * kTile;
  static constexpr int kV = kK + 2 * kTile;
  static constexpr int kMeta = kV + 2 * kTile;       // per key warp: its group's scales and minima, fp16
  static constexpr int kKExp = kMeta + kBlockWarps * D * 4;            // 16-byte aligned
  static constexpr int kVExp = kKExp + kExpRing * kBlockWarps * 4;
  static constexpr int kStats = kVExp + kExpRing * kBlockWarps * 4;     // RowStats
  static constexpr int kBars = kStats + MT * 128 * 16;
  static constexpr int kBarCount = 9 + 2 * 6;
  static constexpr int kTmem = kBars + kBarCount * 8;
  static constexpr int kOdd = kTmem + 8;             // OddRange
  static constexpr int kBytes = kOdd + 8;
  static constexpr int kPartial = kK;                // fp32 partial O over the stages: MT 128 D 4 = MT kTile 2 <= 4 kTile
};

// Warps: four for the softmax of each 128 rows, eight that dequantise (a block
// each), and four of which one issues the products: with MT = 2 registers move
// between the groups of four warps, and the idle three bring theirs.
template <int MT>
__host__ __device__ constexpr int chunk_threads() { return (MT * 4 + kBlockWarps + 4) * 32; }

// Registers a thread after the split.  They come out of what the block was
// launched with, 65536 / threads rounded down to a multiple of 8 a thread:
// MT = 2: 5 groups of 96 >= 2 x 128 + 2 x 88 + 48.  MT = 1: 4 of 128 each, as launched.
// (The build compares the 96 with what the compiler used.)
template <int MT>
struct ChunkRegs {
  static constexpr int kSoftmax = 128, kDequant = MT == 2 ? 88 : 128, kIssue = MT == 2 ? 48 : 128;
  static constexpr int kLaunch = 65536 / chunk_threads<MT>() / 8 * 8;
  static_assert(MT * kSoftmax + 2 * kDequant + kIssue <= (MT + 3) * kLaunch, "register split");
  static_assert(MT == 1 || kLaunch == 96, "LAUNCH_REGISTERS of build.py");
};

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// 2^e as a float, e in [-149, 127].
__device__ __forceinline__ float pow2f(int e) {
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}

// Exponent e of a block whose largest absolute value has the float bits u:
// the value times 2^-e is in [2^(TOP - 1), 2^TOP) (smaller where e is held at
// -100, or -127 for exact rows).  Exact rows have no codes to make room for: their keys, and a bf16
// cell's values, stand at 2^8, which leaves entries 2^-22 of the largest whole.
// Exact values beside quantised ones keep to the place of those, since one
// exponent serves the outputs of both.
constexpr int kExactTopExp = 8, kLeastExp = -127;
template <int TOP = kTopExp, int LEAST = -100>
__device__ __forceinline__ int block_exp(uint32_t abs_bits) {
  return max(static_cast<int>(abs_bits >> 23) - 127 - TOP + 1, LEAST);
}

// The upper two bits of each nibble from hi, the lower two from lo: one
// operation (mask ? hi : lo).
__device__ __forceinline__ uint32_t join_bits(uint32_t hi, uint32_t lo) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(0xCCCCCCCCu), "r"(hi), "r"(lo));
  return d;
}

// 2^(k - e) for the exponent e of a block, k in [20, 24]: a normal number.
template <int K>
__device__ __forceinline__ float block_unit(int e) {
  static_assert(K >= 20 && K <= 24, "e is in [-100, 134]");
  return __int_as_float((127 + K - e) << 23);
}

// Exponent of a query row whose largest absolute value has the bf16 bits u: the
// row times 2^-e has it in [2^13, 2^14) (bf16's 8 bits stay whole in fp16).
__device__ __forceinline__ int query_exp(uint32_t abs_bits) {
  return max(static_cast<int>(abs_bits >> 7) - 127 - 13, kLeastExp);
}
// What turns a product into a logit: the scale's mantissa times 2^e, e the sum of
// the scale's, the row's and the keys' exponents, each of which may be far out.
// At least 2^-126 (a scale of zero must not make a number of -inf), at most a
// finite number (nor one of a product of zero).
__device__ __forceinline__ float logit_scale(float mantissa, int e) {
  return __int_as_float(__float_as_int(mantissa) + (min(max(e, -126), 127) << 23));
}

// 16 channels' codes (hi << 2 | lo, two bits each plane; 2-bit cells: code << 2)
// as fp16 x = code s + m: eight half2 words of neighbouring channels.  s, m:
// scale and minimum of each channel pair; the scale of a pair is 2^24 or 2^20
// times its value by the place that its codes have in a word.
template <bool SPLIT, typename S, typename M>
__device__ __forceinline__ void codes_to_half(uint32_t hi, uint32_t lo, S&& s, M&& m, uint32_t (&out)[8]) {
  uint32_t even, odd;  // nibble n: channel 2 n, 2 n + 1
  if constexpr (SPLIT) {
    even = join_bits(hi << 2, lo);
    odd = join_bits(hi, lo >> 2);
  } else {
    even = (hi << 2) & 0xCCCCCCCCu;
    odd = hi & 0xCCCCCCCCu;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // channels 0-7, 8-15
    uint32_t x = __byte_perm(even, odd, j ? 0x7632 : 0x5410);
#pragma unroll
    for (int n = 0; n < 4; n += 2) {
      out[4 * j + n] = half2_bits(__hfma2(bits_half2(x & 0x000F000Fu), s(4 * j + n), m(4 * j + n)));
      out[4 * j + n + 1] = half2_bits(__hfma2(bits_half2(x & 0x00F000F0u), s(4 * j + n + 1), m(4 * j + n + 1)));
      x >>= 8;
    }
  }
}

// Byte offset of the 16-byte chunk of channels 8 c .. 8 c + 7 of row r in a
// swizzled tile of 128-byte rows (64 channels a row, 128 rows a sub-tile).
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (c >> 3) * (kTileKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

// bf16 pair without what is not finite.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  return w & ~__vcmpgtu2(w & 0x7FFF7FFFu, 0x7F7F7F7Fu);
}
__device__ __forceinline__ uint4 finite_bf16x8(const uint4& w) {
  return make_uint4(finite_bf16x2(w.x), finite_bf16x2(w.y), finite_bf16x2(w.z), finite_bf16x2(w.w));
}
__device__ __forceinline__ uint32_t abs_max_bf16x8(uint32_t m, const uint4& w) {
  return abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(m, w.x), w.y), w.z), w.w);
}
// (scale, min) that stands for values which are not all finite.
__device__ __forceinline__ bool odd_meta(uint32_t w) { return finite_bf16x2(w) != w; }

// bf16 pair times f (a power of two) as fp16 pair.
__device__ __forceinline__ uint32_t bf16x2_to_half(uint32_t w, float f) {
  return half2_bits(__floats2half2_rn(bf16_lo(w) * f, bf16_hi(w) * f));
}

// 2^x of two numbers x <= 100 on the FMA units: x = n + f with n the nearest
// integer (added to 1.5 2^23 and taken off again) and |f| <= 1/2, a cubic for
// 2^f (fitted at Chebyshev nodes to the least relative error, 7.5e-5, a third of
// what rounding a weight to fp16 may add), n into the exponent.  -inf and all
// below -126 give 2^-126, which is 0 as a weight, and so does a NaN: that shows
// in the row's other columns.
__device__ __forceinline__ void poly_exp2(uint64_t x2, float& a, float& b) {
  unpack2(x2, a, b);
  const uint64_t x = pack2(fmaxf(a, -126.f), fmaxf(b, -126.f));
  const uint64_t n = add2(x, pack2(12582912.f, 12582912.f));
  const uint64_t f = fma2(add2(n, pack2(-12582912.f, -12582912.f)), pack2(-1.f, -1.f), x);
  uint64_t y = fma2(f, pack2(5.517158285e-02f, 5.517158285e-02f), pack2(2.426111102e-01f, 2.426111102e-01f));
  y = fma2(y, f, pack2(6.932610273e-01f, 6.932610273e-01f));
  y = fma2(y, f, pack2(9.999280572e-01f, 9.999280572e-01f));
  float na, nb;
  unpack2(n, na, nb);
  unpack2(y, a, b);
  a = __int_as_float(__float_as_int(a) + (__float_as_int(na) << 23));
  b = __int_as_float(__float_as_int(b) + (__float_as_int(nb) << 23));
}

// Bounded wait of a whole warp; the same answer for all its threads.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  bool done = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, done)) {
    const unsigned long long t0 = global_timer_ns();
#pragma unroll 1
    do {
#pragma unroll 1
      for (int i = 0; i < 64 && !done; ++i) done = mbar_try_wait(bar, parity);
    } while (!done && global_timer_ns() - t0 <= kWaitTimeoutNs);
  }
  return __all_sync(0xffffffffu, done);
}

// Values that are not finite.  A weight of 0 times one would be NaN in rows that
// must not see it, so they enter the products as 0; where the blocks that hold
// them lie is noted here, and each row adds those that it sees at the end.  Keys
// count on: the stored tokens' tiles (groups), then the current rows'.
struct OddRange {
  int first, end;  // none: first >= end
};

// One thread's note of count keys from `first` on, to the range at a shared address.
__device__ __forceinline__ void note_odd_keys(uint32_t odd_at, int first, int count) {
  asm volatile("red.shared::cta.min.s32 [%0], %1;" ::"r"(odd_at), "r"(first) : "memory");
  asm volatile("red.shared::cta.max.s32 [%0], %1;" ::"r"(odd_at + 4), "r"(first + count) : "memory");
}

// The infinities that a row's channels get from the values that are not finite:
// of both signs, or a NaN, in one channel is NaN.
template <int D>
struct OddSum {
  uint32_t plus[D / 32], minus[D / 32];
};

// Those of odd's keys, for a whole warp, a row a lane: it sees `stored` stored
// tokens and `current` current rows.  Current rows count from key0 on; there are
// len of them.  Blocks without such values cost one look at their scales (their
// rows), the others two votes for each token and 32 channels, however many they are.
template <int KIND, int D>
__device__ __forceinline__ void odd_values(const ChunkAttnParams& p, int b, int hk, int stored, int current, int len, int key0,
                                           OddRange odd, OddSum<D>& sum) {
  using R = Rec<KIND, D>;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) sum.plus[w] = sum.minus[w] = 0u;
#pragma unroll 1
  for (int i = odd.first; i < odd.end; i += kBlock) {
    const bool exact = KIND == LOOPKV_CELL_BF16 || i >= key0;
    const uint8_t* rec = nullptr;
    if (i < key0) {
      const int phys = p.block_table[static_cast<size_t>(b) * p.max_blocks + min(i / kBlock, p.max_blocks - 1)];
      if (phys < 0 || phys >= p.num_blocks) continue;  // no block there: behind the last token
      rec = p.arena + (static_cast<size_t>(phys) * p.Hkv + hk) * R::kBytes;
    }
    auto row_of = [&](int t) {  // an exact row, or null
      if (i < key0) return reinterpret_cast<const __nv_bfloat16*>(rec + R::kBfV) + t * D;
      return i - key0 + t < len ? row_at(p.v_cur, b, i - key0 + t, hk) : nullptr;
    };
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(rec + R::kVMetaOff);  // [token][D / 32]
    bool some = false;
    if (exact) {
#pragma unroll 1
      for (int k = lane; k < kBlock * (D / 8); k += 32) {
        const __nv_bfloat16* row = row_of(k / (D / 8));
        if (!row) continue;
        const uint4 x = reinterpret_cast<const uint4*>(row)[k % (D / 8)], f = finite_bf16x8(x);
        some = some || x.x != f.x || x.y != f.y || x.z != f.z || x.w != f.w;
      }
    } else {
#pragma unroll 1
      for (int k = lane; k < kBlock * (D / kGroup); k += 32) some = some || odd_meta(meta[k]);
    }
    if (!__any_sync(0xffffffffu, some)) continue;
#pragma unroll 1
    for (int t = 0; t < kBlock; ++t) {
      const bool seen = i < key0 ? i + t < stored : i - key0 + t < current;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        float v = 0.f;
        if (exact) {
          const __nv_bfloat16* row = row_of(t);
          if (row) v = __bfloat162float(row[32 * w + lane]);
        } else {
          const uint32_t m = meta[t * (D / kGroup) + w];
          if (odd_meta(m)) {  // min + scale x code, as read_tokens gives it
            const int c = 32 * w + lane;
            uint32_t code = (rec[R::kVHi + c / 4 * kBlock + t] >> (2 * (c % 4))) & 3u;
            if constexpr (KIND == LOOPKV_CELL_Q4) code = code << 2 | ((rec[R::kQ4VLo + t * R::kRow + c / 4] >> (2 * (c % 4))) & 3u);
            v = fmaf(bf16_lo(m), static_cast<float>(code), bf16_hi(m));
          }
        }
        const uint32_t plus = __ballot_sync(0xffffffffu, !(v < INFINITY)), minus = __ballot_sync(0xffffffffu, !(v > -INFINITY));
        if (seen) sum.plus[w] |= plus, sum.minus[w] |= minus;
      }
    }
  }
}

// Each channel that gets any: add(channel, what).
template <int D, typename Add>
__device__ __forceinline__ void add_odd(const OddSum<D>& sum, Add&& add) {
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
#pragma unroll 1
    for (uint32_t left = sum.plus[w] | sum.minus[w]; left; left &= left - 1) {
      const uint32_t bit = left & -left;
      add(32 * w + __ffs(left) - 1, !(sum.minus[w] & bit) ? INFINITY : sum.plus[w] & bit ? NAN : -INFINITY);
    }
  }
}

// What the CTA works on.
struct ChunkJob {
  int b, hk, start, len;      // sequence, KV head, its chunk
  int stored;                 // tokens in the cell that its rows may see
  int stored_tiles;           // tiles over them; the chunk's own rows (exact) come after
  int tile0, tiles;           // this CTA's tiles
  bool current;
};

// Where the tile's row (token, query head) goes.
template <int D>
__device__ __forceinline__ __nv_bfloat16* chunk_out(const ChunkAttnParams& p, const ChunkJob& job, int row) {
  const int head = (job.hk << p.g_log2) + (row & ((1 << p.g_log2) - 1));
  return p.out + ((static_cast<size_t>(job.b) * p.chunk.T + (row >> p.g_log2)) * p.H + head) * D;
}

// The job of a CTA with rows row0 .. row0 + max_rows - 1 of sequence job.b and KV
// head job.hk: fills in the rest of it.  False where there is nothing left to
// do: no such rows, or rows that are zeros (written here if `writer`) because
// the sequence is skipped or at fault (flagged here if `report`).  The answer is
// the same for all CTAs of the sequence: every block id of it is looked at.
template <int D>
__device__ bool chunk_job(const ChunkAttnParams& p, ChunkJob& job, int row0, int max_rows, bool report, bool writer) {
  job.current = p.k_cur.p != nullptr;
  job.start = p.chunk.start_pos[job.b];
  job.len = p.chunk.new_lens ? p.chunk.new_lens[job.b] : p.chunk.T;
  if (job.len < 0 || job.len > p.chunk.T) {
    if (report && threadIdx.x == 0 && job.start >= 0) flag_error(p.chunk.err, LOOPKV_DEVERR_SEQ_LEN);
    return false;
  }
  const int rows = min((job.len << p.g_log2) - row0, max_rows);
  if (rows <= 0) return false;
  const int64_t stored = static_cast<int64_t>(job.start) + (job.current ? 0 : job.len);
  int fault = 0;
  if (job.start >= 0) {
    if (stored > p.max_stored) {
      fault = LOOPKV_DEVERR_SEQ_LEN;
    } else {
      const int blocks = (static_cast<int>(stored) + kBlock - 1) / kBlock;
      int bad = 0;
      for (int i = threadIdx.x; i < blocks; i += blockDim.x) {
        const int phys = p.block_table[static_cast<size_t>(job.b) * p.max_blocks + i];
        bad |= phys < 0 || phys >= p.num_blocks;
      }
      if (__syncthreads_or(bad)) fault = LOOPKV_DEVERR_BLOCK_ID;
    }
    if (!fault) {
      job.stored = static_cast<int>(stored);
      return true;
    }
    if (report && threadIdx.x == 0) flag_error(p.chunk.err, fault);
  }
  if (writer)
    for (int i = threadIdx.x; i < rows * (D / 8); i += blockDim.x)
      reinterpret_cast<uint4*>(chunk_out<D>(p, job, row0 + i / (D / 8)))[i % (D / 8)] = make_uint4(0, 0, 0, 0);
  return false;
}

// Four channels of a row out of its splits' partial results: RowStats at `stats`
// and channels at `part` in the shared memory of each CTA of the cluster.
template <int D>
__device__ __forceinline__ void join_splits(const ChunkAttnParams& p, const ChunkJob& job, int row, int quad, int splits,
                                            uint32_t stats, uint32_t part) {
  auto stats_of = [&](int s) {
    RowStats r;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(r.m), "=f"(r.sum) : "r"(peer_addr(stats, s)) : "memory");
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r.v) : "r"(peer_addr(stats + 8, s)) : "memory");
    return r;
  };
  RowStats all = join_refs(splits, stats_of);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < splits; ++s) {
    const RowStats st = stats_of(s);
    if (st.m == -INFINITY) continue;
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(peer_addr(part, s)) : "memory");
    join_part(all, st, acc, x);
  }
  reinterpret_cast<uint2*>(chunk_out<D>(p, job, row))[quad] = join_result(all, acc);
}

// ---------------------------------------------------------------- dequantising warps

// One block of 16 tokens: 16 channels a thread, KPL tokens a thread.
template <int KIND, int D>
struct BlockLoader {
  using R = Rec<KIND, D>;
  static constexpr int C16 = D / 16, SUBS = 32 / C16, KPL = kBlock / SUBS;
  static constexpr bool kQuant = KIND != LOOPKV_CELL_BF16;
  static constexpr bool kSplit = KIND == LOOPKV_CELL_Q4;

  struct RawKeys {  // of one block, as loaded
    uint32_t hi[KPL], lo[KPL], meta[D / 32];
  };
  struct RawValues {
    uint32_t hi[4], lo[KPL], meta[KPL];
  };

  const ChunkAttnParams& p;
  const ChunkJob& job;
  uint32_t odd_at;       // the CTA's OddRange
  int block, lane, c16, sub;
  int key0;              // first of the thread's tokens as a key: key0 + SUBS i
  int flip;              // its tokens as a value: sub KPL + (k ^ flip)
  uint32_t key_at, value_at[2];   // their rows' places in the tile, first 16 bytes; the second are at ^ 16

  // Where eight neighbouring threads would write rows of the same parity to
  // the same banks, half of them take the other row of a pair.
  __device__ BlockLoader(const ChunkAttnParams& p, const ChunkJob& job, uint32_t odd_at, int block, int lane)
      : p(p), job(job), odd_at(odd_at), block(block), lane(lane), c16(lane % C16), sub(lane / C16) {
    key0 = D == 128 ? sub ^ (c16 >> 2) : sub;
    flip = D == 128 ? c16 >> 2 : sub & 1;
    key_at = swz(block * kBlock + key0, 2 * c16);
    value_at[0] = swz(block * kBlock + sub * KPL + flip, 2 * c16);
    value_at[1] = swz(block * kBlock + sub * KPL + (1 ^ flip), 2 * c16);
  }

  __device__ int key_token(int it) const { return it * SUBS + key0; }
  __device__ int value_token(int k) const { return sub * KPL + (k ^ flip); }
  // a row SUBS (two) further on: as many rows of 128 bytes, and bit 2 (1) of the
  // row turns in the swizzle
  __device__ uint32_t key_place(int it) const {
    return SUBS == 8 ? key_at + it * 1024 : ((key_at + it * 512) ^ ((it & 1) << 6));
  }
  __device__ uint32_t value_place(int k) const { return k < 2 ? value_at[k] : ((value_at[k & 1] + 256) ^ 32); }

  __device__ int token0(int tile) const { return tile * kTileKeys + block * kBlock; }
  // the key group of the block is full, so its keys are quantised
  __device__ bool full(int t0) const { return (t0 & ~(kGroup - 1)) + kGroup <= job.stored; }

  // Physical ids of this warp's block and of its group's other one (all ids of
  // the sequence's stored blocks were checked); 0 where there is none.
  __device__ int2 ids(int tile) const {
    const int t0 = token0(tile);
    if (tile >= job.stored_tiles || t0 >= job.stored) return make_int2(0, 0);
    const int32_t* row = p.block_table + static_cast<size_t>(job.b) * p.max_blocks;
    return make_int2(row[t0 / kBlock], full(t0) ? row[(t0 ^ kBlock) / kBlock] : 0);
  }

  __device__ const uint8_t* record(int phys) const {
    return p.arena + (static_cast<size_t>(phys) * p.Hkv + job.hk) * R::kBytes;
  }

  __device__ void load(int tile, int2 id, RawKeys& r) const {
    const int t0 = token0(tile);
    if (!kQuant || tile >= job.stored_tiles || !full(t0)) return;
    const uint8_t* rec = record(id.x);
    const uint8_t* other = record(id.y);
    // this thread's D / 32 channels of the group's scales
    const int ch = lane * (D / 32);
    const uint8_t* mrec = ((ch >= D / 2) == ((t0 & kBlock) != 0) ? rec : other) + R::kKMetaOff + (ch % (D / 2)) * 4;
    if constexpr (D == 128) {
      const uint4 w = *reinterpret_cast<const uint4*>(mrec);
      r.meta[0] = w.x, r.meta[1] = w.y, r.meta[2] = w.z, r.meta[3] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(mrec);
      r.meta[0] = w.x, r.meta[1] = w.y;
    }
    const uint8_t* row = rec + key0 * R::kRow + 4 * c16;
#pragma unroll
    for (int it = 0; it < KPL; ++it) {
      r.hi[it] = *reinterpret_cast<const uint32_t*>(row + R::kKHi + it * SUBS * R::kRow);
      if constexpr (kSplit) r.lo[it] = *reinterpret_cast<const uint32_t*>(row + R::kQ4KLo + it * SUBS * R::kRow);
    }
  }

  __device__ void load(int tile, int2 id, RawValues& r) const {
    const int t0 = token0(tile);
    if (!kQuant || tile >= job.stored_tiles || t0 >= job.stored) return;
    const uint8_t* rec = record(id.x);
    const uint8_t* col = rec + R::kVHi + 4 * c16 * kBlock + sub * KPL;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      r.hi[q] = KPL == 4 ? *reinterpret_cast<const uint32_t*>(col + q * kBlock)
                         : *reinterpret_cast<const uint16_t*>(col + q * kBlock);
    constexpr int kMetaRow = (D / kGroup) * 4;
    const uint8_t* lo[2] = {rec + R::kQ4VLo + value_token(0) * R::kRow + 4 * c16,
                            rec + R::kQ4VLo + value_token(1) * R::kRow + 4 * c16};
    const uint8_t* meta[2] = {rec + R::kVMetaOff + value_token(0) * kMetaRow + (c16 / 2) * 4,
                              rec + R::kVMetaOff + value_token(1) * kMetaRow + (c16 / 2) * 4};
#pragma unroll
    for (int k = 0; k < KPL; ++k) {
      if constexpr (kSplit) r.lo[k] = *reinterpret_cast<const uint32_t*>(lo[k & 1] + (k & 2) * R::kRow);
      r.meta[k] = *reinterpret_cast<const uint32_t*>(meta[k & 1] + (k & 2) * kMetaRow);
    }
  }

  __device__ static void store_row(uint32_t at, const uint32_t (&x)[8]) {
    st_shared16(at, x[0], x[1], x[2], x[3]);
    st_shared16(at ^ 16, x[4], x[5], x[6], x[7]);
  }

  // Exact bf16 rows into the tile; row(token) is the token's row or null (zeros).
  // The exponent is that of the finite entries: others must not take theirs from
  // the rest of the block, which rows before them see.
  template <bool KEYS, typename Row>
  __device__ int store_exact(int tile, uint32_t tile_base, Row&& row) const {
    uint4 w[KPL][2];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < KPL; ++k) {
      const __nv_bfloat16* src = row(KEYS ? key_token(k) : value_token(k));
      w[k][0] = w[k][1] = make_uint4(0, 0, 0, 0);
      if (src) {
        w[k][0] = reinterpret_cast<const uint4*>(src + 16 * c16)[0];
        w[k][1] = reinterpret_cast<const uint4*>(src + 16 * c16)[1];
      }
    }
#pragma unroll
    for (int k = 0; k < KPL; ++k) top = abs_max_bf16x8(abs_max_bf16x8(top, w[k][0]), w[k][1]);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    if (top >= 0x7F80u) {
      asm volatile("");
      top = 0;
#pragma unroll
      for (int k = 0; k < KPL; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 x = finite_bf16x8(w[k][j]);
          top = abs_max_bf16x8(top, x);
          if constexpr (!KEYS) w[k][j] = x;
        }
      top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
      if (!KEYS && lane == 0) note_odd_keys(odd_at, token0(tile), kBlock);
    }
    const int e = block_exp<KEYS || !kQuant ? kExactTopExp : kTopExp, kLeastExp>(top << 16);
    const float f = pow2f(-e);
#pragma unroll
    for (int k = 0; k < KPL; ++k) {
      uint32_t x[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[4 * j] = bf16x2_to_half(w[k][j].x, f), x[4 * j + 1] = bf16x2_to_half(w[k][j].y, f);
        x[4 * j + 2] = bf16x2_to_half(w[k][j].z, f), x[4 * j + 3] = bf16x2_to_half(w[k][j].w, f);
      }
      store_row(tile_base + (KEYS ? key_place(k) : value_place(k)), x);
    }
    return e;
  }

  // Keys of the block into the tile; returns their exponent.
  __device__ int store(int tile, int2 id, const RawKeys& r, uint32_t tile_base, uint32_t meta) const {
    const int t0 = token0(tile);
    if (tile >= job.stored_tiles) {
      const int c0 = t0 - job.stored_tiles * kTileKeys;
      return store_exact<true>(tile, tile_base, [&](int t) {
        return c0 + t < job.len ? row_at(p.k_cur, job.b, c0 + t, job.hk) : nullptr;
      });
    }
    if constexpr (kQuant) {
      if (!full(t0)) {
        const __nv_bfloat16* res = p.residual + (static_cast<size_t>(job.b) * p.Hkv + job.hk) * kGroup * D;
        return store_exact<true>(tile, tile_base, [&](int t) {
          return t0 + t < job.stored ? res + ((t0 + t) % kGroup) * D : nullptr;
        });
      }
      // scales and minima of the group's channels, fp16, shared by the warp
      constexpr int CPT = D / 32;
      constexpr float kTop = kSplit ? 15.f : 3.f;
      float s[CPT], mn[CPT], top = 0.f;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        s[i] = bf16_lo(r.meta[i]), mn[i] = bf16_hi(r.meta[i]);
        top = fmaxf(top, fmaxf(fabsf(mn[i]), fabsf(fmaf(s[i], kTop, mn[i]))));
      }
      const int e = block_exp(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      const float fs = block_unit<kSplit ? 24 : 22>(e), f = fs * (kSplit ? 0x1p-24f : 0x1p-22f);
      // pair n of eight channels: 2^24 for even n, 2^20 for odd; parts of 16 bytes
      // [scale 0-7][scale 8-15][min 0-7][min 8-15] x C16 so that reads do not collide
#pragma unroll
      for (int i = 0; i < CPT; i += 2) {
        const int ch = lane * CPT + i, pair = (ch / 2) % 4;
        const float g = pair & 1 ? fs * 0.0625f : fs;
        const uint32_t at = meta + ((ch % 16) / 8 * C16 + ch / 16) * 16 + pair * 4;
        const uint32_t hs = half2_bits(__floats2half2_rn(s[i] * g, s[i + 1] * g));
        const uint32_t hm = half2_bits(__floats2half2_rn(mn[i] * f, mn[i + 1] * f));
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(hs) : "memory");
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 2 * C16 * 16), "r"(hm) : "memory");
      }
      __syncwarp();
      uint32_t sw[8], mw[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(sw[4 * j]), "=r"(sw[4 * j + 1]), "=r"(sw[4 * j + 2]), "=r"(sw[4 * j + 3])
                     : "r"(meta + (j * C16 + c16) * 16) : "memory");
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(mw[4 * j]), "=r"(mw[4 * j + 1]), "=r"(mw[4 * j + 2]), "=r"(mw[4 * j + 3])
                     : "r"(meta + ((2 + j) * C16 + c16) * 16) : "memory");
      }
      __syncwarp();
#pragma unroll
      for (int it = 0; it < KPL; ++it) {
        uint32_t x[8];
        codes_to_half<kSplit>(r.hi[it], kSplit ? r.lo[it] : 0u, [&](int n) { return bits_half2(sw[n]); },
                              [&](int n) { return bits_half2(mw[n]); }, x);
        store_row(tile_base + key_place(it), x);
      }
      return e;
    } else {
      const uint8_t* rec = record(id.x);
      return store_exact<true>(tile, tile_base, [&](int t) {
        return t0 + t < job.stored ? reinterpret_cast<const __nv_bfloat16*>(rec + R::kBfK) + t * D : nullptr;
      });
    }
  }

  // Values of the block into the tile; returns their exponent.
  __device__ int store(int tile, int2 id, RawValues& r, uint32_t tile_base) const {
    const int t0 = token0(tile);
    if (tile >= job.stored_tiles) {
      const int c0 = t0 - job.stored_tiles * kTileKeys;
      return store_exact<false>(tile, tile_base, [&](int t) {
        return c0 + t < job.len ? row_at(p.v_cur, job.b, c0 + t, job.hk) : nullptr;
      });
    }
    if constexpr (kQuant) {
      constexpr float kTop = kSplit ? 15.f : 3.f;
      float s[KPL], mn[KPL];
      uint32_t top_bits;
#pragma unroll 1
      for (bool again = false;; again = true) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KPL; ++k) {
          // what lies behind the last token is no value
          const uint32_t w = t0 + value_token(k) < job.stored ? r.meta[k] : 0u;
          s[k] = bf16_lo(w), mn[k] = bf16_hi(w);
          top = max3_nan(top, fabsf(mn[k]), fabsf(fmaf(s[k], kTop, mn[k])));
        }
        top_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if (top_bits < 0x7F800000u || again) break;
#pragma unroll
        for (int k = 0; k < KPL; ++k)
          if (odd_meta(r.meta[k])) r.meta[k] = 0u;
        if (lane == 0) note_odd_keys(odd_at, t0, kBlock);
      }
      const int e = block_exp(top_bits);
      const float fs = block_unit<kSplit ? 24 : 22>(e), f = fs * (kSplit ? 0x1p-24f : 0x1p-22f);
#pragma unroll
      for (int k = 0; k < KPL; ++k) {
        const uint32_t sel = ((k & 1) ^ flip) * 0x11 + 0x40 + (k & 2) * 0x11;  // the token's byte of the column words
        const uint32_t hi = __byte_perm(__byte_perm(r.hi[0], r.hi[1], sel), __byte_perm(r.hi[2], r.hi[3], sel), 0x5410);
        const __half2 sa = __float2half2_rn(s[k] * fs), sb = __float2half2_rn(s[k] * (fs * 0.0625f));
        const __half2 m = __float2half2_rn(mn[k] * f);
        uint32_t x[8];
        codes_to_half<kSplit>(hi, kSplit ? r.lo[k] : 0u, [&](int n) { return n & 1 ? sb : sa; }, [&](int) { return m; }, x);
        store_row(tile_base + value_place(k), x);
      }
      return e;
    } else {
      const uint8_t* rec = record(id.x);
      return store_exact<false>(tile, tile_base, [&](int t) {
        return t0 + t < job.stored ? reinterpret_cast<const __nv_bfloat16*>(rec + R::kBfV) + t * D : nullptr;
      });
    }
  }
};

// ---------------------------------------------------------------- the kernel

template <int KIND, int D, int MT>
__global__ void __launch_bounds__(chunk_threads<MT>(), 1) chunk_tensor_kernel(const __grid_constant__ ChunkAttnParams p, int row_tiles,
                                                                               int splits) {
  using L = ChunkSmem<D, MT>;
  constexpr int kRows = MT * 128;
  constexpr int kTmemCols = MT * (2 * kStepKeys + D) <= 256 ? 256 : 512;
  constexpr int kSoftmaxWarps = MT * 4, kIssueWarp = kSoftmaxWarps + kBlockWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % splits;
  const uint32_t unit = blockIdx.x / splits;
  const int tile = row_tiles - 1 - static_cast<int>(unit % row_tiles);  // the rows that see most come first

  ChunkJob job;
  job.hk = (unit / row_tiles) % p.Hkv;
  job.b = unit / row_tiles / p.Hkv;
  const int row0 = tile * kRows;
  if (!chunk_job<D>(p, job, row0, kRows, tile == 0 && job.hk == 0 && rank == 0, rank == 0)) return;
  const int row_end = min(job.len << p.g_log2, row0 + kRows), last_token = (row_end - 1) >> p.g_log2;
  const int my_row = min(row0 + static_cast<int>(threadIdx.x), row_end - 1);  // of the softmax warps' threads
  // keys that the tile's last row sees, 128 at a time; this CTA's share of them
  const int seen = job.current ? job.stored : min(job.stored, job.start + last_token + 1);
  job.stored_tiles = (seen + kTileKeys - 1) / kTileKeys;
  const int all_tiles = job.stored_tiles + (job.current ? last_token / kTileKeys + 1 : 0);
  job.tile0 = static_cast<int>(static_cast<int64_t>(all_tiles) * rank / splits);
  job.tiles = static_cast<int>(static_cast<int64_t>(all_tiles) * (rank + 1) / splits) - job.tile0;

  const uint32_t bars = sbase + L::kBars;
  auto k_full = [&](int s) { return bars + 8 * s; };
  auto k_empty = [&](int s) { return bars + 16 + 8 * s; };
  auto v_full = [&](int s) { return bars + 32 + 8 * s; };
  auto v_empty = [&](int s) { return bars + 48 + 8 * s; };
  const uint32_t q_full = bars + 64;
  auto s_full = [&](int m) { return bars + 72 + 8 * m; };                       // logits of a step are there
  auto s_free = [&](int m) { return bars + 88 + 8 * m; };                       // and have been read
  auto p_full = [&](int m, int buf) { return bars + 104 + 16 * m + 8 * buf; };  // its weights are there
  auto o_done = [&](int m, int buf) { return bars + 136 + 16 * m + 8 * buf; };  // and are in O
  int* k_exp = reinterpret_cast<int*>(smem + L::kKExp);
  float* v_exp = reinterpret_cast<float*>(smem + L::kVExp);
  OddRange* odd = reinterpret_cast<OddRange*>(smem + L::kOdd);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), kBlockWarps);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), kBlockWarps);
      mbar_init(v_empty(s), 1);
    }
    mbar_init(q_full, kSoftmaxWarps);
    for (int m = 0; m < 2; ++m) {
      mbar_init(s_full(m), 1);
      mbar_init(s_free(m), 4);
      for (int buf = 0; buf < 2; ++buf) {
        mbar_init(p_full(m, buf), 4);
        mbar_init(o_done(m, buf), 1);
      }
    }
    fence_mbar_init();
    *odd = OddRange{INT32_MAX, 0};
  }
  if (warp == kIssueWarp) tmem_alloc<kTmemCols>(sbase + L::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // tensor memory: the logits of a step, two buffers of weights, the outputs
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kTmem);
  const uint32_t tmem_p = tmem + MT * kStepKeys, tmem_o = tmem + MT * 2 * kStepKeys;
  bool ok = true;
  const int n = job.tiles, steps = 2 * n;
  // How the warps without rows end: what the join needs is then no burden on
  // their registers.
  auto leave = [&]() {
    if (!ok && lane == 0) flag_error(p.chunk.err, LOOPKV_DEVERR_TIMEOUT);
    __syncthreads();
    if (warp == kIssueWarp) tmem_free<kTmemCols>(tmem);
    if (splits > 1) {
      cluster_sync_all();
      cluster_sync_all();
    }
  };

  if (warp >= kSoftmaxWarps && warp < kIssueWarp) {
    // ------------------------------------------------------------ dequantise
    set_max_registers<ChunkRegs<MT>::kDequant, ChunkRegs<MT>::kLaunch>();
    const int block = warp - kSoftmaxWarps;
    const BlockLoader<KIND, D> loader(p, job, sbase + L::kOdd, block, lane);
    typename BlockLoader<KIND, D>::RawKeys keys = {};
    typename BlockLoader<KIND, D>::RawValues values = {};
    // The records' bytes come one tile ahead, each part into the registers that
    // the tile before has just left; the block ids two tiles ahead.
    int2 id = n > 0 ? loader.ids(job.tile0) : make_int2(0, 0), id_next = n > 1 ? loader.ids(job.tile0 + 1) : id;
    if (n > 0) {
      loader.load(job.tile0, id, keys);
      loader.load(job.tile0, id, values);
    }
    for (int j = 0; j < n; ++j) {
      const int s = j & 1, t = job.tile0 + j, ring = j % kExpRing * kBlockWarps + block;
      const int2 id_after = j + 2 < n ? loader.ids(t + 2) : id_next;
      if (j >= 2 && !(ok = warp_wait(k_empty(s), ((j >> 1) - 1) & 1))) break;
      int e = loader.store(t, id, keys, sbase + L::kK + s * L::kTile, sbase + L::kMeta + block * D * 4);
      if (lane == 0) k_exp[ring] = e;
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full(s));
      if (j + 1 < n) loader.load(t + 1, id_next, keys);
      if (j >= 2 && !(ok = warp_wait(v_empty(s), ((j >> 1) - 1) & 1))) break;
      e = loader.store(t, id, values, sbase + L::kV + s * L::kTile);
      if (lane == 0) v_exp[ring] = static_cast<float>(e);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(s));
      if (j + 1 < n) loader.load(t + 1, id_next, values);
      id = id_next;
      id_next = id_after;
    }
    leave();
    return;
  }
  if (warp >= kIssueWarp) {
    // ------------------------------------------------------------ multiply
    set_max_registers<ChunkRegs<MT>::kIssue, ChunkRegs<MT>::kLaunch>();
    if (warp == kIssueWarp && n > 0) {
      const uint32_t issue = elect_one();
      constexpr uint32_t kQKDesc = f16_idesc(kStepKeys, false), kPVDesc = f16_idesc(D, true);
      constexpr uint32_t kHalf = kStepKeys * 128;  // bytes between a tile's two steps
      const uint64_t q_desc = smem_desc(sbase + L::kQ, 16), k_desc = smem_desc(sbase + L::kK, 16);
      const uint64_t v_desc = smem_desc(sbase + L::kV, kTileKeys * 128);
      auto issue_qk = [&](int m, int h) {
        const uint64_t a = q_desc + ((m * L::kTile) >> 4);
        const uint64_t b = k_desc + ((((h >> 1) & 1) * L::kTile + (h & 1) * kHalf) >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          constexpr int kSub = kTileKeys * 128;  // 64 channels further on
          const uint32_t at = ((i / 4) * kSub + (i % 4) * 32) >> 4;
          mma_ss(issue, tmem + m * kStepKeys, a + at, b + at, kQKDesc, i > 0);
        }
        mma_commit(issue, s_full(m));
      };
      ok = warp_wait(q_full, 0) && warp_wait(k_full(0), 0);
      tc_fence_after();
      if (ok)
        for (int m = 0; m < MT; ++m) issue_qk(m, 0);
      for (int h = 0; h < steps && ok; ++h) {
        if (h + 1 < steps) {  // the next step's logits, as soon as this one's have been read
          if (h & 1) ok = warp_wait(k_full(((h + 1) >> 1) & 1), ((h + 1) >> 2) & 1);
          for (int m = 0; m < MT && ok; ++m) {
            ok = warp_wait(s_free(m), h & 1);
            if (!ok) break;
            tc_fence_after();
            issue_qk(m, h + 1);
          }
          if (!ok) break;
          if (!(h & 1)) mma_commit(issue, k_empty((h >> 1) & 1));
        }
        if (!(h & 1)) ok = warp_wait(v_full((h >> 1) & 1), (h >> 2) & 1);
        const uint64_t v = v_desc + ((((h >> 1) & 1) * L::kTile + (h & 1) * kHalf) >> 4);
        for (int m = 0; m < MT && ok; ++m) {
          ok = warp_wait(p_full(m, h & 1), (h >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t w = tmem_p + (2 * m + (h & 1)) * (kStepKeys / 2);
#pragma unroll
          for (int i = 0; i < kStepKeys / 16; ++i)
            mma_ts(issue, tmem_o + m * D, w + i * 8, v + i * (2048 >> 4), kPVDesc, h > 0 || i > 0);
          mma_commit(issue, o_done(m, h & 1));
        }
        if ((h & 1) && ok) mma_commit(issue, v_empty((h >> 1) & 1));
      }
    }
    leave();
    return;
  }
  {
    // ------------------------------------------------------------ softmax
    set_max_registers<ChunkRegs<MT>::kSoftmax, ChunkRegs<MT>::kLaunch>();
    const int m = warp / 4;
    const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;  // tensor-memory lanes 32 (warp % 4) on
    const uint32_t ts = tmem + m * kStepKeys + lanes, tp = tmem_p + m * kStepKeys + lanes, to = tmem_o + m * D + lanes;
    const bool idle = row0 + warp * 32 >= row_end;                 // no row of this warp is there
    const int token = my_row >> p.g_log2;
    // Queries: a row a thread, times a power of two, the scale's sign with it.
    int row_exp;
    {
      const uint4* src = reinterpret_cast<const uint4*>(row_at(p.q, job.b, token, (job.hk << p.g_log2) + (my_row & ((1 << p.g_log2) - 1))));
      uint32_t top = 0;
      uint4 w[D / 16];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) w[i] = src[half * (D / 16) + i];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          top = abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(top, w[i].x), w[i].y), w[i].z), w[i].w);
      }
      const int e = query_exp(max(top & 0xFFFFu, top >> 16));
      const float f = p.scale_negative ? -pow2f(-e) : pow2f(-e);
      row_exp = e + p.scale_exp;
      const uint32_t q = sbase + L::kQ + m * L::kTile;
#pragma unroll
      for (int half = 1; half >= 0; --half) {  // the second half is still here
        if (half == 0)
#pragma unroll
          for (int i = 0; i < D / 16; ++i) w[i] = src[i];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          st_shared16(q + swz(threadIdx.x % 128, half * (D / 16) + i), bf16x2_to_half(w[i].x, f), bf16x2_to_half(w[i].y, f),
                      bf16x2_to_half(w[i].z, f), bf16x2_to_half(w[i].w, f));
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    float m_ref = -INFINITY, sum = 0.f;
    float v_ref = kNoValueRef;
    for (int h = 0; h < steps && ok; ++h) {
      const int j = h >> 1, buf = h & 1, gt = job.tile0 + j;
      // The tile's exponents come with its values (its keys came before).  The
      // logits' arrival tells that all products issued before theirs are done,
      // those of two steps ago among them, which read the weights' buffer.
      ok = (buf || warp_wait(v_full(j & 1), (j >> 1) & 1)) && warp_wait(s_full(m), h & 1);
      if (!ok) break;
      if (idle) {
        if (lane == 0) {
          mbar_arrive(s_free(m));
          mbar_arrive(p_full(m, buf));
        }
        continue;
      }
      tc_fence_after();
      uint32_t r[kStepKeys];
      tmem_ld64(ts, r);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(m));
      // keys of this step that the row sees
      const int lim = (gt >= job.stored_tiles ? token + 1 - (gt - job.stored_tiles) * kTileKeys
                       : (job.current ? job.stored : job.start + token + 1) - gt * kTileKeys) - buf * kStepKeys;
      const bool masked = __any_sync(0xffffffffu, lim < kStepKeys);
      const int4 ke = *reinterpret_cast<const int4*>(k_exp + (j % kExpRing) * kBlockWarps + buf * 4);
      const float4 ve = *reinterpret_cast<const float4*>(v_exp + (j % kExpRing) * kBlockWarps + buf * 4);
      const float f[4] = {logit_scale(p.scale_mantissa, row_exp + ke.x), logit_scale(p.scale_mantissa, row_exp + ke.y),
                          logit_scale(p.scale_mantissa, row_exp + ke.z), logit_scale(p.scale_mantissa, row_exp + ke.w)};
      const float vexp[4] = {ve.x, ve.y, ve.z, ve.w};
      if (masked) {
        asm volatile("");  // a branch: most steps are not masked
#pragma unroll
        for (int i = 0; i < kStepKeys; ++i)
          if (i >= lim) r[i] = 0xFF800000u;
      }
      float block_top[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t* x = r + 16 * c;
        float a = max3_nan(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
        float b = max3_nan(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
        a = max3_nan(a, __uint_as_float(x[6]), __uint_as_float(x[7]));
        b = max3_nan(b, __uint_as_float(x[8]), __uint_as_float(x[9]));
        a = max3_nan(a, __uint_as_float(x[10]), __uint_as_float(x[11]));
        b = max3_nan(b, __uint_as_float(x[12]), __uint_as_float(x[13]));
        a = max_nan(max3_nan(a, __uint_as_float(x[14]), __uint_as_float(x[15])), b);
        block_top[c] = a * f[c];
      }
      const float top = max_nan(max3_nan(block_top[0], block_top[1], block_top[2]), block_top[3]);
      const float most = fmaxf(max3(block_top[0] + vexp[0], block_top[1] + vexp[1], block_top[2] + vexp[2]), block_top[3] + vexp[3]);
      // The references follow only what is far above them: O is rescaled rarely.
      if (__any_sync(0xffffffffu, refs_move(m_ref, v_ref, top, most))) {
        const float m_new = logit_ref(m_ref, top);
        float above = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) above = fmaxf(above, block_top[c] - m_new + vexp[c]);
        const float v_new = value_ref(v_ref, m_ref, m_new, above);
        const float shrink = m_new == m_ref ? 0.f : m_ref - m_new;
        sum *= fast_exp2(shrink);
        if (h > 0) {
          ok = warp_wait(o_done(m, buf ^ 1), ((h - 1) >> 1) & 1);
          tc_fence_after();
          const float f = fast_exp2(shrink + (v_ref - v_new));
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(to + c, o);
          }
        }
        m_ref = m_new;
        v_ref = v_new;
      }
      const float base = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float de = fmaxf(vexp[c] - v_ref, kLeastShift);
        const float off = de - base;
        const uint64_t f2 = pack2(f[c], f[c]), off2 = pack2(off, off);
        uint64_t part = 0;  // two sums of zero
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x, y;
          const uint64_t e = fma2(pack2(__uint_as_float(r[16 * c + 2 * i]), __uint_as_float(r[16 * c + 2 * i + 1])), f2, off2);
          if (i % 4 == kPolyPair) {
            poly_exp2(e, x, y);
          } else {
            unpack2(e, x, y);
            x = fast_exp2(x), y = fast_exp2(y);
          }
          part = add2(part, pack2(x, y));
          w[i] = half2_bits(__floats2half2_rn(x, y));
        }
        float pa, pb;
        unpack2(part, pa, pb);
        sum = fmaf(pa + pb, fast_exp2(-de), sum);
        tmem_st8(tp + buf * (kStepKeys / 2) + 8 * c, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(m, buf));
    }
    // ------------------------------------------------------------ results
    if (n > 0 && ok) ok = warp_wait(o_done(m, 1), (n - 1) & 1);
    tc_fence_after();
    // where the rows lie is worked out anew, so as not to hold it over the steps
    const uint32_t unit_again = cta_id_x() / splits;
    const int local = threadIdx.x, row = (row_tiles - 1 - static_cast<int>(unit_again % row_tiles)) * kRows + local;
    ChunkJob at;
    at.hk = (unit_again / row_tiles) % p.Hkv;
    at.b = unit_again / row_tiles / p.Hkv;
    const int rows = (p.chunk.new_lens ? p.chunk.new_lens[at.b] : p.chunk.T) << p.g_log2;
    if (row - lane < rows) {
      // Over the sum, times the unit, in two steps (v may be beyond 127); partial
      // results go as they are.  Every row sees a key: where no logit is above -inf
      // its weights are 0 / 0.
      const float near = fmaxf(fminf(v_ref, 100.f), -100.f);
      const float f1 = splits > 1 ? 1.f : m_ref == -INFINITY ? NAN : pow2f(static_cast<int>(near)) / sum;
      const float f2 = splits > 1 ? 1.f : pow2f(static_cast<int>(fmaxf(v_ref - near, -49.f)));
      const bool valid = row < rows;
      __nv_bfloat16* o = chunk_out<D>(p, at, min(row, rows - 1));
      if (splits > 1) reinterpret_cast<RowStats*>(smem + L::kStats)[local] = RowStats{m_ref, sum, v_ref};
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        if (n > 0) {
          tmem_ld32(to + c, r);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0;
        }
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = ok ? __uint_as_float(r[i]) * f1 * f2 : 0.f;
        if (splits == 1) {
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(o + c + i) =
                  make_uint4(pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3]), pack_bf16(x[i + 4], x[i + 5]),
                             pack_bf16(x[i + 6], x[i + 7]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(smem + L::kPartial + local * D * 4 + ((((c + i) / 4) ^ (local & (D / 4 - 1))) << 4)) =
                make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
      }
      // (all blocks' notes came before the last values' arrival)
      const OddRange found{*reinterpret_cast<volatile int*>(&odd->first), *reinterpret_cast<volatile int*>(&odd->end)};
      if (ok && found.first < found.end) {
        const int token = row >> p.g_log2, start = p.chunk.start_pos[at.b];
        OddSum<D> sum;
        odd_values<KIND, D>(p, at.b, at.hk, start + (p.k_cur.p ? 0 : token + 1), token + 1, rows >> p.g_log2,
                            job.stored_tiles * kTileKeys, found, sum);
        if (valid)
          add_odd<D>(sum, [&](int c, float v) {
            if (splits == 1)
              o[c] = __float2bfloat16_rn(__bfloat162float(o[c]) + v);
            else
              reinterpret_cast<float*>(smem + L::kPartial + local * D * 4 + (((c / 4) ^ (local & (D / 4 - 1))) << 4))[c % 4] += v;
          });
      }
    }
  }
  if (!ok && lane == 0) flag_error(p.chunk.err, LOOPKV_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (splits == 1) return;

  // ---------------------------------------------------------------- join the splits
  // Every CTA holds its partial rows and their RowStats; row i is put together by CTA i % splits from all of them.
  cluster_sync_all();
  {
    const uint32_t stats = sbase + L::kStats, partial = sbase + L::kPartial;
    constexpr int kQuads = D / 4, kRowsPerWarp = 32 / kQuads;
    const int quad = lane % kQuads;
    const uint32_t unit_again = cta_id_x() / splits;
    const int first = (row_tiles - 1 - static_cast<int>(unit_again % row_tiles)) * kRows;
    ChunkJob at;
    at.hk = (unit_again / row_tiles) % p.Hkv;
    at.b = unit_again / row_tiles / p.Hkv;
    const int rows = min(((p.chunk.new_lens ? p.chunk.new_lens[at.b] : p.chunk.T) << p.g_log2) - first, kRows);
    const int rank = cta_id_x() % splits;
    for (int i = warp * kRowsPerWarp + lane / kQuads;; i += kSoftmaxWarps * kRowsPerWarp) {
      const int row = i * splits + rank;
      if (row >= rows) break;
      join_splits<D>(p, at, first + row, quad, splits, stats + row * 16,
                     partial + row * D * 4 + ((quad ^ (row & (kQuads - 1))) << 4));
    }
  }
  cluster_sync_all();
}

}  // namespace loopkv
