// Norms of queries and keys for each head, the position rotation, and the
// append of a chunk's keys and values to a cell with both on the way (sm_100a).
//
// A row is a head's D channels at one position; eight channels a thread, so a
// row is 16 threads (D = 128) or 8 (D = 64) and every access is 16 bytes.
// The mathematics is in loopkv_chunk.h; every fp32 step is one rounded
// operation without contraction, and the mean of the squares is summed in 64
// bits, because the quantiser behind it decides codes by a border: the stored
// bytes are then a function of the inputs alone, whatever the order of a sum.
//
// The append: one CTA per (sequence, KV head, 32-token key group).  Keys meet
// in a shared tile (their scales run over the group's tokens), values are
// quantised in registers (their scales run over 32 channels = four threads),
// and the group's two records are put together in shared memory and leave as
// 16-byte stores where the call brings all 32 tokens.
//
// Measured on a B200 (device time, CUDA graph), with what bounds it:
//   norms and rotation of 3 x up to 2731 tokens, 32 + 8 heads of 64, rotation of
//   32: 20.5 us, 3.4 TB/s of 70 MB; instruction issue (27 a value)
//   64 sequences x 1 token, 16 + 16 heads of 128: 3.6 us; one pass' latency
//   append of 8191 tokens, 16 heads of 128, 4-bit, queries rotated: 60 us for
//   155 MB; instruction issue (the quantiser and the rotation); with 64
//   registers and eight CTAs an SM (72 and seven: 1 us more; rows unrolled four
//   times, 94 registers: 91 us, the code outgrows the instruction cache); heads
//   of 128 spill 8 to 12 bytes a thread
//   append of 64 x 1 token: 8.7 us, five dependent round trips
#include "append_ops.cuh"
#include "chunk_common.cuh"

namespace loopkv {
namespace {

constexpr int kThreads = 128;

// cos and signed sin of this thread's eight channels at one position (pairs of
// neighbours: of its four pairs, in the first four).
template <bool PAIRS>
struct Turn {
  float c[PAIRS ? 4 : 8], s[PAIRS ? 4 : 8];
};

// Channels 8 sub .. 8 sub + 7.  Halves: the partner of channel i is i +- rot / 2,
// the first half gives a cos - b sin, the second b cos + a sin (s carries the
// sign).  Neighbours: the same over (2 i, 2 i + 1).
template <bool PAIRS>
__device__ __forceinline__ void load_turn(const RotaryView& r, int pos, int sub, Turn<PAIRS>& t) {
  const int c0 = 8 * sub, half = r.rot / 2;
  if (c0 >= r.rot) return;  // also without a table
  const float* row = r.cos_sin + static_cast<size_t>(pos) * r.rot;
  const bool first = PAIRS || c0 < half;
  const float* at = row + (PAIRS ? c0 / 2 : first ? c0 : c0 - half);
#pragma unroll
  for (int i = 0; i < (PAIRS ? 4 : 8); i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(at + i);
    const float4 s = *reinterpret_cast<const float4*>(at + half + i);
    t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
    t.s[i] = first && !PAIRS ? -s.x : s.x, t.s[i + 1] = first && !PAIRS ? -s.y : s.y;
    t.s[i + 2] = first && !PAIRS ? -s.z : s.z, t.s[i + 3] = first && !PAIRS ? -s.w : s.w;
  }
}

// x^2 of a bf16 pair added to a 64-bit sum.  A bf16 number's exponent and
// mantissa are moved into a double's, which costs two integer operations where
// the conversion instruction runs at an eighth of their rate; 0 comes out as
// 2^-127, whose square is nothing beside eps (at least 1e-30), and infinities and
// NaN as 2^128 and more: a sum of 2^256, for which see kTinyNorm.
__device__ __forceinline__ double add_squares(uint32_t w, double sum) {
  const double a = __hiloint2double(static_cast<int>((w & 0x7FFFu) * 8192u + 0x38000000u), 0);
  const double b = __hiloint2double(static_cast<int>(((w & 0x7FFF0000u) >> 3) + 0x38000000u), 0);
  return fma(b, b, fma(a, a, sum));
}

__device__ __forceinline__ double squares(const uint4& raw) {
  return add_squares(raw.w, add_squares(raw.z, add_squares(raw.y, add_squares(raw.x, 0.0))));
}

// fp32(1 / sqrt(mean of a row's squares + eps)), sum the thread's part.
template <int D>
__device__ __forceinline__ float inverse_norm(double sum, double eps) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return static_cast<float>(rsqrt(sum * (1.0 / D) + eps));
}

// The same for four rows at once, that of row sub % 4: the first two rounds of
// the reduction pass on the rows that the partner keeps, and each thread takes
// one root instead of four.
template <int D>
__device__ __forceinline__ float inverse_norm4(const uint4 (&raw)[4], double eps, int sub) {
  const double q[4] = {squares(raw[0]), squares(raw[1]), squares(raw[2]), squares(raw[3])};
  const bool odd = sub & 1, high = sub & 2;
  const double a = (odd ? q[1] : q[0]) + __shfl_xor_sync(0xffffffffu, odd ? q[0] : q[1], 1);
  const double b = (odd ? q[3] : q[2]) + __shfl_xor_sync(0xffffffffu, odd ? q[2] : q[3], 1);
  double sum = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 2);
#pragma unroll
  for (int o = D / 16; o > 2; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return static_cast<float>(rsqrt(sum * (1.0 / D) + eps));
}

// A row with an infinity or a NaN (or finite squares of 2^255 and more together)
// has an inverse norm below this, and is taken of converted numbers: infinite or
// NaN where an entry is.
constexpr float kTinyNorm = 0x1p-120f;
template <int D>
__device__ __noinline__ float exact_norm(const __nv_bfloat16* row, double eps) {
  double sum = 0.0;
#pragma unroll 1
  for (int i = 0; i < D; ++i) {
    const double x = __bfloat162float(row[i]);
    sum = fma(x, x, sum);
  }
  return static_cast<float>(rsqrt(sum * (1.0 / D) + eps));
}

// Weights (if any; inv the row's inverse norm) and rotation of one row, raw its
// eight channels of this thread; whole warps call it, rows that are not there
// included.
template <int D, bool PAIRS>
__device__ __forceinline__ void weigh_rotate(const RotaryView& r, const __nv_bfloat16* weight, float inv,
                                             const Turn<PAIRS>& t, int sub, const uint4& raw, float (&x)[8]) {
  constexpr int LANES = D / 8;
  unpack8(raw, x);
  if (weight) {
    float ww[8];
    unpack8(*reinterpret_cast<const uint4*>(weight + 8 * sub), ww);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), ww[i]);
  }
  if (!r.rot) return;
  if constexpr (PAIRS) {
    if (8 * sub < r.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
        x[2 * i + 1] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
      }
    }
  } else {
    const int hl = r.rot / 16;  // threads of half the rotated channels
    const int peer = (sub < hl ? sub + hl : sub - hl) & (LANES - 1);
    float other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, x[i], peer, LANES);
    if (8 * sub < r.rot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], t.c[i]), __fmul_rn(other[i], t.s[i]));
    }
  }
}

// Four heads of one token of the chunk, for the threads of one row: the table's
// row is loaded once for the four (it is as many bytes as two rows of bf16).
// Whole warps call it; items past the last one do nothing.
constexpr int kHeadsPerItem = 4;

template <int D, bool PAIRS>
__device__ __forceinline__ void rotate_item(const RotateParams& p, uint32_t item, uint32_t items, int sub) {
  const int heads = p.H + p.Hk;
  const uint32_t per_token = (heads + kHeadsPerItem - 1) / kHeadsPerItem;
  bool active = item < items;
  if (!active) item = 0;
  const uint32_t bt = item / per_token;
  const int h0 = static_cast<int>(item - bt * per_token) * kHeadsPerItem;
  const int b = bt / p.chunk.T, t = bt - static_cast<uint32_t>(b) * p.chunk.T;
  const SeqChunk sc = seq_chunk(p.chunk, b, active && t == 0 && h0 == 0 && sub == 0);
  active = active && t < sc.len;
  uint4 raw[kHeadsPerItem];
#pragma unroll
  for (int i = 0; i < kHeadsPerItem; ++i) {
    const int h = h0 + i;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (active && h < heads)
      raw[i] = *reinterpret_cast<const uint4*>((h < p.H ? row_at(p.q, b, t, h) : row_at(p.k, b, t, h - p.H)) + 8 * sub);
  }
  Turn<PAIRS> turn;
  if (active) load_turn<PAIRS>(p.rot, sc.start + t, sub, turn);
  float norms = 1.f;
  if (p.rot.q_weight || p.rot.k_weight) {
    norms = inverse_norm4<D>(raw, p.rot.eps, sub);
    const int h = h0 + sub % 4;  // the row
    if (active && h < heads && norms < kTinyNorm)
      norms = exact_norm<D>(h < p.H ? row_at(p.q, b, t, h) : row_at(p.k, b, t, h - p.H), p.rot.eps);
    __syncwarp();  // rows are written, perhaps in place, after all of them have been read
  }
  const size_t token = static_cast<size_t>(b) * p.chunk.T + t;
#pragma unroll
  for (int i = 0; i < kHeadsPerItem; ++i) {
    const int h = h0 + i;
    const bool is_q = h < p.H;
    float x[8];
    const float inv = __shfl_sync(0xffffffffu, norms, i, D / 8);
    weigh_rotate<D, PAIRS>(p.rot, is_q ? p.rot.q_weight : p.rot.k_weight, inv, turn, sub, raw[i], x);
    if (active && h < heads) {
      __nv_bfloat16* o = is_q ? p.q_out + (token * p.H + h) * D : p.k_out + (token * p.Hk + (h - p.H)) * D;
      *reinterpret_cast<uint4*>(o + 8 * sub) = pack8(x);
    }
  }
}

uint32_t rotate_items(const RotateParams& p) {
  const uint32_t per_token = (p.H + p.Hk + kHeadsPerItem - 1) / kHeadsPerItem;
  return static_cast<uint32_t>(p.chunk.B) * p.chunk.T * per_token;
}

template <int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RotateParams p, uint32_t items) {
  constexpr int LANES = D / 8;
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  rotate_item<D, PAIRS>(p, item, items, threadIdx.x % LANES);
}

// The quantiser's divisions as they are defined, where a shortcut below cannot
// tell what they round to.
__device__ __noinline__ float exact_quotient(float a, float b) { return __fdiv_rn(a, b); }

// (scale, min) of a group, both bf16 numbers.
__device__ __forceinline__ uint32_t meta_of(float s, float mn) { return pack_bf16(s, mn); }

// group_params, its division by 15 (3) as a product: q is within 2^-22 of the
// rounded quotient, so unless q lies that near to a tie of bf16 (or is zero or
// very small) both round to the same bf16 number.  mn is a bf16 number.
template <int BITS>
__device__ __forceinline__ float quick_scale(float mn, float mx) {
  constexpr float kTop = static_cast<float>((1 << BITS) - 1);
  const float d = __fsub_rn(mx, mn);
  float q = __fmul_rn(d, 1.f / kTop);
  if (((__float_as_uint(q) & 0xFFFFu) - 0x7FF8u) <= 0x10u || !(q > 0x1p-100f)) q = exact_quotient(d, kTop);
  return __uint_as_float(pack_bf16(0.f, q));
}

// A scale whose inverse, and what it multiplies, are normal numbers.
__device__ __forceinline__ bool ordinary(float s) { return s > 0x1p-100f && s < 0x1p100f; }

// rint of four rounded quotients a / s, given their estimates t within 3e-6,
// where one of them lies within 1e-5 of a half h.  By the sign of the exact
// remainder a - h s; where that is neither zero nor 2^-18 s away from it, or
// the scale out of the ordinary, by the quotient itself.  0 for a NaN.
template <int BITS>
__device__ __noinline__ float4 settle_codes(float4 a, float4 s, float4 t) {
  constexpr float kTop = static_cast<float>((1 << BITS) - 1);
  const float aa[4] = {a.x, a.y, a.z, a.w}, ss[4] = {s.x, s.y, s.z, s.w}, tt[4] = {t.x, t.y, t.z, t.w};
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = rintf(tt[i]);
    if (!ordinary(ss[i])) {
      r[i] = ss[i] == 0.f ? 0.f : fminf(fmaxf(rintf(exact_quotient(aa[i], ss[i])), 0.f), kTop);
    } else if (aa[i] != aa[i]) {
      r[i] = 0.f;
    } else if (fabsf(tt[i] - r[i]) > 0.49999f) {
      const float h = r[i] > tt[i] ? r[i] - 0.5f : r[i] + 0.5f, rem = fmaf(-h, ss[i], aa[i]);
      r[i] = rem == 0.f ? rintf(h) : rem > 0.f ? h + 0.5f : h - 0.5f;
      if (rem != 0.f && fabsf(rem) < ss[i] * 0x1p-18f) r[i] = fminf(rintf(exact_quotient(aa[i], ss[i])), kTop);
    }
  }
  return make_float4(r[0], r[1], r[2], r[3]);
}

// Codes rint((x - mn) / s), at most the top one, of four values (as group_code;
// x >= mn), without the division, as one number: the first in the lowest BITS
// bits.  t = (x - mn) * (1 / s) is within 3e-6 of the rounded quotient, so where
// it is more than 1e-5 away from a half both round to the same integer (half to
// even by adding 1.5 2^23 and taking it off again).  bf16 numbers meet halves
// often enough (one in some thousand) for those to have a way of their own, and
// a NaN, which the minimum and the maximum here keep, takes that too.
// The four are put together as floats, exactly.
template <int BITS>
__device__ __forceinline__ uint32_t quick_codes(const float* x, const float (&s)[4], const float (&mn)[4],
                                                const float (&inv)[4], bool odd) {
  constexpr float kTop = static_cast<float>((1 << BITS) - 1), kBase = static_cast<float>(1 << BITS), kRound = 12582912.f;
  float r[4], t[4], off = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = min_nan(__fmul_rn(__fsub_rn(x[i], mn[i]), inv[i]), kTop);
    r[i] = __fsub_rn(__fadd_rn(t[i], kRound), kRound);
    off = max_nan(off, fabsf(__fsub_rn(t[i], r[i])));
  }
  if (!(off <= 0.49999f) || odd) {
    const float4 q = settle_codes<BITS>(
        make_float4(__fsub_rn(x[0], mn[0]), __fsub_rn(x[1], mn[1]), __fsub_rn(x[2], mn[2]), __fsub_rn(x[3], mn[3])),
        make_float4(s[0], s[1], s[2], s[3]), make_float4(t[0], t[1], t[2], t[3]));
    r[0] = q.x, r[1] = q.y, r[2] = q.z, r[3] = q.w;
  }
  return __float_as_uint(fmaf(fmaf(fmaf(r[3], kBase, r[2]), kBase, r[1]), kBase, r[0]) + 8388608.f);  // 2^23: low bits
}

// Nibbles to two-bit fields: the upper two bits of each of eight nibbles (of the
// two halves' four each) in the low 16 bits (the low 8 of each half).
__device__ __forceinline__ uint32_t two_bits(uint32_t n, bool halves) {
  n = (n | (n >> 2)) & 0x0F0F0F0Fu;
  n = (n | (n >> 4)) & 0x00FF00FFu;
  return halves ? n : (n | (n >> 8)) & 0xFFFFu;
}

template <int KIND, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 8) rope_append_kernel(const RopeAppendParams p, uint32_t kv_blocks,
                                                               uint32_t items) {
  constexpr int LANES = D / 8, ROWS = kThreads / LANES, ITERS = kGroup / ROWS;
  const int sub = threadIdx.x % LANES, row0 = threadIdx.x / LANES;
  if (blockIdx.x >= kv_blocks) {  // the queries
    const uint32_t item = (blockIdx.x - kv_blocks) * ROWS + row0;
    rotate_item<D, PAIRS>(p.rows, item, items, sub);
    return;
  }
  using R = Rec<KIND, D>;
  const int gi = blockIdx.x % p.key_blocks;
  const int h = (blockIdx.x / p.key_blocks) % p.Hkv;
  const int b = blockIdx.x / p.key_blocks / p.Hkv;
  const ChunkView& ch = p.rows.chunk;
  const SeqChunk sc = seq_chunk(ch, b, gi == 0 && h == 0 && threadIdx.x == 0);
  const int start = sc.start, end = start + sc.len;
  const int G = start / kGroup + gi, g0 = G * kGroup;
  if (sc.len == 0 || g0 >= end) return;
  const int tok0 = max(start, g0), tok1 = min(end, g0 + kGroup);  // the call's tokens of this group
  const bool complete = tok1 == g0 + kGroup;
  const CellRows cell{p.arena, p.block_table + static_cast<size_t>(b) * p.max_blocks, ch.err, p.Hkv, h,
                      p.max_blocks, p.num_blocks};
  const RotaryView& rot = p.rows.rot;
  const __nv_bfloat16* w = rot.k_weight;

  // Rows are taken ROWS at a time by a loop that is not unrolled: its code stays
  // in the instruction cache, and many CTAs on an SM keep the loads in flight.
  if constexpr (KIND == LOOPKV_CELL_BF16) {
#pragma unroll 1
    for (int it = 0; it < ITERS; ++it) {
      const int pos = g0 + it * ROWS + row0;
      const bool here = pos >= tok0 && pos < tok1;
      Turn<PAIRS> turn;
      uint4 k_raw = make_uint4(0, 0, 0, 0), v_raw = k_raw;
      if (here) {
        k_raw = *reinterpret_cast<const uint4*>(row_at(p.k, b, pos - start, h) + 8 * sub);
        v_raw = *reinterpret_cast<const uint4*>(row_at(p.v, b, pos - start, h) + 8 * sub);
        load_turn<PAIRS>(rot, pos, sub, turn);
      }
      float x[8];
      float inv_norm = w ? inverse_norm<D>(squares(k_raw), rot.eps) : 1.f;
      if (here && inv_norm < kTinyNorm) inv_norm = exact_norm<D>(row_at(p.k, b, pos - start, h), rot.eps);
      weigh_rotate<D, PAIRS>(rot, w, inv_norm, turn, sub, k_raw, x);
      uint8_t* rec = here ? record_at<KIND, D>(cell, pos) : nullptr;
      if (!rec) continue;
      const int row = pos % kBlock;
      *reinterpret_cast<uint4*>(rec + R::kBfK + row * D * 2 + 16 * sub) = pack8(x);
      *reinterpret_cast<uint4*>(rec + R::kBfV + row * D * 2 + 16 * sub) = v_raw;
    }
    return;
  } else {
    constexpr int BITS = KIND == LOOPKV_CELL_Q4 ? 4 : 2;
    constexpr bool kSplit = KIND == LOOPKV_CELL_Q4;
    constexpr int kVGroups = D / kGroup;
    // rows a little apart, so that threads of one column quad on different rows meet different banks
    constexpr int kStride = D * 2 + (D == 128 ? 32 : 16);
    __shared__ __align__(16) uint8_t tile[kGroup * kStride];
    __shared__ __align__(16) uint8_t rec[2 * R::kBytes];

    __nv_bfloat16* res = p.residual + (static_cast<size_t>(b) * p.Hkv + h) * kGroup * D;
    // The open group's exact keys belong to the call's last group, unless the
    // first group still has to read older ones from there: then its CTA, after
    // it has read them, writes the last group's keys too.
    const bool begun = start % kGroup != 0;

#pragma unroll 1
    for (int it = 0; it < ITERS; ++it) {
      const int r = it * ROWS + row0, pos = g0 + r;
      const bool here = pos >= tok0 && pos < tok1;
      if (g0 + it * ROWS >= tok1 || g0 + (it + 1) * ROWS <= tok0) {  // the whole CTA: none of the call's rows
        if (pos < tok0 && complete)
          *reinterpret_cast<uint4*>(tile + r * kStride + 16 * sub) = *reinterpret_cast<const uint4*>(res + r * D + 8 * sub);
        continue;
      }
      Turn<PAIRS> turn;
      uint4 k_raw = make_uint4(0, 0, 0, 0), v_raw = k_raw;
      if (here) {
        k_raw = *reinterpret_cast<const uint4*>(row_at(p.k, b, pos - start, h) + 8 * sub);
        v_raw = *reinterpret_cast<const uint4*>(row_at(p.v, b, pos - start, h) + 8 * sub);
        load_turn<PAIRS>(rot, pos, sub, turn);
      }
      float x[8];
      float inv_norm = w ? inverse_norm<D>(squares(k_raw), rot.eps) : 1.f;
      if (here && inv_norm < kTinyNorm) inv_norm = exact_norm<D>(row_at(p.k, b, pos - start, h), rot.eps);
      weigh_rotate<D, PAIRS>(rot, w, inv_norm, turn, sub, k_raw, x);
      // the value row: groups of 32 channels are four neighbouring threads
      float v[8];
      unpack8(v_raw, v);
      float mn = v[0], mx = v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mn = fminf(mn, v[i]), mx = fmaxf(mx, v[i]);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      }
      if (here) {
        uint4 packed = pack8(x);
        *reinterpret_cast<uint4*>(tile + r * kStride + 16 * sub) = packed;
        if (!complete && (gi == 0 || !begun)) *reinterpret_cast<uint4*>(res + r * D + 8 * sub) = packed;
        const float s_b = quick_scale<BITS>(mn, mx), inv = __frcp_rn(s_b);
        const float ss[4] = {s_b, s_b, s_b, s_b}, mm[4] = {mn, mn, mn, mn}, ii[4] = {inv, inv, inv, inv};
        const bool odd = !ordinary(s_b);
        const uint32_t c0 = quick_codes<BITS>(v, ss, mm, ii, odd), c1 = quick_codes<BITS>(v + 4, ss, mm, ii, odd);
        uint32_t hi, lo = 0;
        if constexpr (kSplit) {
          const uint32_t n = __byte_perm(c0, c1, 0x5410);
          hi = two_bits((n >> 2) & 0x33333333u, false);
          lo = two_bits(n & 0x33333333u, false);
        } else {
          hi = __byte_perm(c0, c1, 0x0040);
        }
        uint8_t* dst = rec + (r / kBlock) * R::kBytes;
        const int row = r % kBlock;
        dst[R::kVHi + (2 * sub) * kBlock + row] = static_cast<uint8_t>(hi);
        dst[R::kVHi + (2 * sub + 1) * kBlock + row] = static_cast<uint8_t>(hi >> 8);
        if constexpr (kSplit) *reinterpret_cast<uint16_t*>(dst + R::kQ4VLo + row * R::kRow + 2 * sub) = static_cast<uint16_t>(lo);
        if (sub % 4 == 0) *reinterpret_cast<uint32_t*>(dst + R::kVMetaOff + (row * kVGroups + sub / 4) * 4) = meta_of(s_b, mn);
      } else if (pos < tok0 && complete) {
        *reinterpret_cast<uint4*>(tile + r * kStride + 16 * sub) = *reinterpret_cast<const uint4*>(res + r * D + 8 * sub);
      }
    }
    __syncthreads();

    if (complete) {
      // keys per channel: four channels and every NS-th token a thread, the NS
      // threads of a channel quad side by side in a warp
      constexpr int NS = kThreads / (D / 4);
      const int ns = threadIdx.x % NS, quad = threadIdx.x / NS;
      float x[kGroup / NS][4];
      float mn[4], mx[4];
#pragma unroll
      for (int k = 0; k < kGroup / NS; ++k) {
        const uint2 u = *reinterpret_cast<const uint2*>(tile + (ns + NS * k) * kStride + 8 * quad);
        x[k][0] = bf16_lo(u.x), x[k][1] = bf16_hi(u.x), x[k][2] = bf16_lo(u.y), x[k][3] = bf16_hi(u.y);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mn[c] = k ? fminf(mn[c], x[k][c]) : x[k][c];
          mx[c] = k ? fmaxf(mx[c], x[k][c]) : x[k][c];
        }
      }
      float s_b[4], inv[4];
      bool odd = false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int o = 1; o < NS; o <<= 1) {
          mn[c] = fminf(mn[c], __shfl_xor_sync(0xffffffffu, mn[c], o));
          mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], o));
        }
        s_b[c] = quick_scale<BITS>(mn[c], mx[c]);
        inv[c] = __frcp_rn(s_b[c]);
        odd = odd || !ordinary(s_b[c]);
      }
#pragma unroll
      for (int k = 0; k < kGroup / NS; k += 2) {  // two tokens
        const uint32_t c0 = quick_codes<BITS>(x[k], s_b, mn, inv, odd), c1 = quick_codes<BITS>(x[k + 1], s_b, mn, inv, odd);
        uint32_t hi, lo = 0;
        if constexpr (kSplit) {
          const uint32_t n = __byte_perm(c0, c1, 0x5410);
          hi = two_bits((n >> 2) & 0x33333333u, true);
          lo = two_bits(n & 0x33333333u, true);
        } else {
          hi = __byte_perm(c0, c1, 0x5410);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = ns + NS * (k + j);
          uint8_t* dst = rec + (r / kBlock) * R::kBytes + (r % kBlock) * R::kRow + quad;
          dst[R::kKHi] = static_cast<uint8_t>(hi >> (16 * j));
          if constexpr (kSplit) dst[R::kQ4KLo] = static_cast<uint8_t>(lo >> (16 * j));
        }
      }
      if (ns == 0) {
        const int c0 = 4 * quad;
        uint8_t* dst = rec + (c0 < D / 2 ? 0 : R::kBytes) + R::kKMetaOff + (c0 % (D / 2)) * 4;
        *reinterpret_cast<uint4*>(dst) = make_uint4(meta_of(s_b[0], mn[0]), meta_of(s_b[1], mn[1]),
                                                    meta_of(s_b[2], mn[2]), meta_of(s_b[3], mn[3]));
      }
      __syncthreads();
    }

    // the records leave: whole, or what the call brought of them
    uint8_t* out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool needed = complete || (tok0 < g0 + kBlock * (j + 1) && tok1 > g0 + kBlock * j);
      out[j] = needed ? record_at<KIND, D>(cell, g0 + kBlock * j) : nullptr;
    }
    if (tok0 == g0 && complete) {
      constexpr int kVec = R::kBytes / 16;
      for (int i = threadIdx.x; i < 2 * kVec; i += kThreads) {
        uint8_t* o = i < kVec ? out[0] : out[1];
        if (o) reinterpret_cast<uint4*>(o)[i % kVec] = reinterpret_cast<const uint4*>(rec)[i];
      }
    } else {
      if (complete) {
        constexpr int kVec = (R::kKMetaOff + R::kKMeta) / 16;  // the key part of a record
        for (int i = threadIdx.x; i < 2 * kVec; i += kThreads) {
          const int j = i / kVec;
          if (uint8_t* o = out[j])
            reinterpret_cast<uint4*>(o)[i % kVec] = reinterpret_cast<const uint4*>(rec + j * R::kBytes)[i % kVec];
        }
      }
      const int rows = tok1 - tok0;
      for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {  // high plane, byte by byte
        const int r = tok0 - g0 + i % rows, at = R::kVHi + (i / rows) * kBlock + r % kBlock;
        if (uint8_t* o = out[r / kBlock]) o[at] = rec[(r / kBlock) * R::kBytes + at];
      }
      for (int i = threadIdx.x; i < rows * kVGroups; i += kThreads) {
        const int r = tok0 - g0 + i / kVGroups, at = R::kVMetaOff + ((r % kBlock) * kVGroups + i % kVGroups) * 4;
        if (uint8_t* o = out[r / kBlock])
          *reinterpret_cast<uint32_t*>(o + at) = *reinterpret_cast<const uint32_t*>(rec + (r / kBlock) * R::kBytes + at);
      }
      if constexpr (kSplit) {
        constexpr int kWords = R::kRow / 4;
        for (int i = threadIdx.x; i < rows * kWords; i += kThreads) {
          const int r = tok0 - g0 + i / kWords, at = R::kQ4VLo + (r % kBlock) * R::kRow + (i % kWords) * 4;
          if (uint8_t* o = out[r / kBlock])
            *reinterpret_cast<uint32_t*>(o + at) = *reinterpret_cast<const uint32_t*>(rec + (r / kBlock) * R::kBytes + at);
        }
      }
    }

    // a begun first group that is full: the later open group's exact keys
    if (gi == 0 && begun && complete && end % kGroup != 0) {
      const int tail0 = end / kGroup * kGroup;
#pragma unroll 1
      for (int it = 0; it < ITERS; ++it) {
        const int r = it * ROWS + row0, pos = tail0 + r;
        const bool here = pos < end;
        Turn<PAIRS> turn;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (here) {
          load_turn<PAIRS>(rot, pos, sub, turn);
          raw = *reinterpret_cast<const uint4*>(row_at(p.k, b, pos - start, h) + 8 * sub);
        }
        float x[8];
        float inv_norm = w ? inverse_norm<D>(squares(raw), rot.eps) : 1.f;
        if (here && inv_norm < kTinyNorm) inv_norm = exact_norm<D>(row_at(p.k, b, pos - start, h), rot.eps);
        weigh_rotate<D, PAIRS>(rot, w, inv_norm, turn, sub, raw, x);
        if (here) *reinterpret_cast<uint4*>(res + r * D + 8 * sub) = pack8(x);
      }
    }
  }
}

template <int KIND, int D>
cudaError_t launch_append_t(const RopeAppendParams& p, cudaStream_t stream) {
  constexpr uint32_t kRows = kThreads / (D / 8);
  const uint32_t kv_blocks = static_cast<uint32_t>(p.rows.chunk.B) * p.Hkv * p.key_blocks;
  const uint32_t items = p.rows.H ? rotate_items(p.rows) : 0;
  const uint32_t blocks = kv_blocks + (items + kRows - 1) / kRows;
  if (p.rows.rot.interleaved)
    rope_append_kernel<KIND, D, true><<<blocks, kThreads, 0, stream>>>(p, kv_blocks, items);
  else
    rope_append_kernel<KIND, D, false><<<blocks, kThreads, 0, stream>>>(p, kv_blocks, items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(int head_dim, const RotateParams& p, cudaStream_t stream) {
  const uint32_t items = rotate_items(p), rows = kThreads / (head_dim / 8);
  const uint32_t blocks = (items + rows - 1) / rows;
  auto kern = head_dim == 128 ? (p.rot.interleaved ? norm_rope_kernel<128, true> : norm_rope_kernel<128, false>)
                              : (p.rot.interleaved ? norm_rope_kernel<64, true> : norm_rope_kernel<64, false>);
  kern<<<blocks, kThreads, 0, stream>>>(p, items);
  return cudaGetLastError();
}

cudaError_t launch_rope_append(int kind, int head_dim, const RopeAppendParams& p, cudaStream_t stream) {
  switch (kind * 1000 + head_dim) {
    case LOOPKV_CELL_Q4 * 1000 + 128: return launch_append_t<LOOPKV_CELL_Q4, 128>(p, stream);
    case LOOPKV_CELL_Q4 * 1000 + 64: return launch_append_t<LOOPKV_CELL_Q4, 64>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 128: return launch_append_t<LOOPKV_CELL_Q2, 128>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 64: return launch_append_t<LOOPKV_CELL_Q2, 64>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 128: return launch_append_t<LOOPKV_CELL_BF16, 128>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 64: return launch_append_t<LOOPKV_CELL_BF16, 64>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace loopkv
