// Chunk attention for few rows (sm_100a): at most 16 (token, query head) rows
// of a KV head, over a 4-bit or 2-bit cell.
//
// The time is the cell's bytes, so a warp reads a 32-token group's two records
// once, by bulk copies into its own ring in shared memory, and dequantises them
// straight into the operand registers of 16 x 8 x 16 products: no tile is
// written back.  (The 128-row products of chunk_tensor.cuh would spend more on
// empty rows than the copy takes.)  Each warp of a CTA takes every so-many-th
// group, the CTAs of a cluster their share of the context; all join through
// shared memory at the end.
//
// Measured on a B200, four tokens of 32 sequences over 4096 4-bit tokens and 16
// heads of 128 (337 MB): 126 us, 2.7 TB/s, 41 % of measured; the 128-row kernel
// 311 us.  Bound by instruction issue and its latencies (1000 a group, half of
// the issue slots used with 12 warps an SM: the outputs and queries alone are 96
// registers, and 4 bytes a thread are spilled for heads of 128); 16 warps with the
// queries in shared memory spill more: 10 % slower.
//
// Operand layout.  A product's columns (keys, or channels) are the eight
// thread quads, its depth two pairs for each thread r of a quad.
//   logits : thread r holds channels D/4 r .. of its quad's key, so that a row
//            of the plane is read as whole words and queries need no shuffle;
//   outputs: the depth is a block's 16 tokens, thread r holds tokens 4 r ..
//            4 r + 3 (pairs (0, 2), (1, 3) of them: bytes of one word of the
//            column-major plane) of its quad's channels D/8 q ..; the logits'
//            columns are ordered to leave the weights in just these places.
#pragma once

#include "append_ops.cuh"
#include "chunk_tensor.cuh"

namespace loopkv {

constexpr int kFewRows = 16, kFewStages = 3, kFewWarpsPerSm = 12;

// WARPS of a CTA: 3, 6 or 12, with 168 registers a thread always twelve an SM.
template <int KIND, int D, int WARPS>
struct FewSmem {
  static constexpr int kGroupBytes = 2 * Rec<KIND, D>::kBytes;
  static constexpr int kRing = WARPS * kFewStages * kGroupBytes;
  static constexpr int kOut = WARPS * kFewRows * D * 4;          // the warps' partial outputs, over the ring
  static constexpr int kMeta = (kRing > kOut ? kRing : kOut);        // each warp: a group's key scales and minima
  static constexpr int kStats = kMeta + WARPS * D * 4;           // each warp: RowStats of 16 rows
  static constexpr int kOdd = kStats + WARPS * kFewRows * 16;    // each warp: OddRange
  static constexpr int kJoin = kOdd + WARPS * 16;
  static constexpr int kJoinStats = kJoin + kFewRows * D * 4;        // the CTA's own result, for its cluster
  static constexpr int kBars = kJoinStats + kFewRows * 16;
  static constexpr int kBytes = kBars + WARPS * kFewStages * 8;
};

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Block token of the quad's key in the first (second) eight columns of a block.
__device__ __forceinline__ int few_key(int quad, int second) { return 4 * (quad >> 1) + 2 * (quad & 1) + second; }

// One warp's work on a group.  PAIRS: channel pairs of a key that a thread
// holds; CH: channels of a value.
template <int KIND, int D>
struct FewWarp {
  using R = Rec<KIND, D>;
  static constexpr bool kSplit = KIND == LOOPKV_CELL_Q4;
  static constexpr int PAIRS = D / 8, STEPS = D / 16, CH = D / 8;
  static constexpr float kTop = kSplit ? 15.f : 3.f;
  static constexpr int kUnit = kSplit ? 24 : 22;               // codes stand 2 bits higher in 2-bit cells
  static constexpr float kPerUnit = kSplit ? 0x1p-24f : 0x1p-22f;

  const ChunkAttnParams& p;
  const ChunkJob& job;
  int lane, quad, r;
  uint32_t q[STEPS][4];
  int row_exp[2];              // rows quad, quad + 8: of the queries, and the scale's
  float m_ref[2], sum[2];
  float v_ref[2];
  float o[CH][4];

  __device__ FewWarp(const ChunkAttnParams& p, const ChunkJob& job, int lane)
      : p(p), job(job), lane(lane), quad(lane >> 2), r(lane & 3) {
    v_ref[0] = v_ref[1] = kNoValueRef;
    m_ref[0] = m_ref[1] = -INFINITY;
    sum[0] = sum[1] = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  // Rows quad and quad + 8, this thread's D / 4 channels.
  __device__ void load_queries(int rows) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = quad + 8 * i;
      uint4 w[D / 32];
#pragma unroll
      for (int k = 0; k < D / 32; ++k) w[k] = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(
            row_at(p.q, job.b, row >> p.g_log2, (job.hk << p.g_log2) + (row & ((1 << p.g_log2) - 1))) + r * (D / 4));
#pragma unroll
        for (int k = 0; k < D / 32; ++k) w[k] = src[k];
      }
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        top = abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(top, w[k].x), w[k].y), w[k].z), w[k].w);
      top = max(top & 0xFFFFu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = query_exp(top);
      const float f = p.scale_negative ? -pow2f(-e) : pow2f(-e);
      row_exp[i] = e + p.scale_exp;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {  // eight channels: two steps
        q[2 * k][i] = bf16x2_to_half(w[k].x, f), q[2 * k][2 + i] = bf16x2_to_half(w[k].y, f);
        q[2 * k + 1][i] = bf16x2_to_half(w[k].z, f), q[2 * k + 1][2 + i] = bf16x2_to_half(w[k].w, f);
      }
    }
  }

  // ---- logits of a group: s[n] is the n-th eight columns; returns the keys' exponent
  __device__ int quant_logits(const uint8_t* rec, uint32_t meta, float (&s)[4][4]) const {
    constexpr int CPT = D / 32;
    const int ch = lane * CPT;
    const uint8_t* mrec = rec + (ch >= D / 2 ? R::kBytes : 0) + R::kKMetaOff + (ch % (D / 2)) * 4;
    float sc[CPT], mn[CPT], top = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(mrec)[i];
      sc[i] = bf16_lo(w), mn[i] = bf16_hi(w);
      top = fmaxf(top, fmaxf(fabsf(mn[i]), fabsf(fmaf(sc[i], kTop, mn[i]))));
    }
    const int e = block_exp(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    const float fs = block_unit<kUnit>(e), f = fs * kPerUnit;
    // pairs of channels: [scale, min] words, a pair's scale 2^24 or 2^20 times its
    // value by its place; four pairs of scales, then of minima, for each thread r
#pragma unroll
    for (int i = 0; i < CPT; i += 2) {
      const int pair = (ch + i) / 2, n = pair % 4, part = pair % PAIRS / 4, who = pair / PAIRS;
      const float g = n & 1 ? fs * 0.0625f : fs;
      const uint32_t at = meta + ((part * 2 * 4 + who) * 4 + n) * 4;
      const uint32_t hs = half2_bits(__floats2half2_rn(sc[i] * g, sc[i + 1] * g));
      const uint32_t hm = half2_bits(__floats2half2_rn(mn[i] * f, mn[i + 1] * f));
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(hs) : "memory");
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 64), "r"(hm) : "memory");
    }
    __syncwarp();
    // this thread's words of its four keys: D / 4 channels of two bits
    constexpr int WORDS = D / 64;
    uint32_t hi[4][WORDS], lo[4][WORDS];
    const uint8_t* row0 = rec + few_key(quad, 0) * R::kRow + r * (D / 16);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const uint8_t* row = row0 + (n >> 1) * R::kBytes + (n & 1) * R::kRow;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        hi[n][w] = reinterpret_cast<const uint32_t*>(row + R::kKHi)[w];
        lo[n][w] = kSplit ? reinterpret_cast<const uint32_t*>(row + R::kQ4KLo)[w] : 0u;
      }
    }
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
      uint32_t sw[8], mw[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = meta + (((2 * w + j) * 2 * 4 + r) * 4) * 4;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(sw[4 * j]), "=r"(sw[4 * j + 1]), "=r"(sw[4 * j + 2]), "=r"(sw[4 * j + 3]) : "r"(at) : "memory");
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(mw[4 * j]), "=r"(mw[4 * j + 1]), "=r"(mw[4 * j + 2]), "=r"(mw[4 * j + 3]) : "r"(at + 64) : "memory");
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t x[8];
        codes_to_half<kSplit>(hi[n][w], lo[n][w], [&](int i) { return bits_half2(sw[i]); },
                              [&](int i) { return bits_half2(mw[i]); }, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_16816(s[n], q[4 * w + i], x[2 * i], x[2 * i + 1]);
      }
    }
    __syncwarp();
    return e;
  }

  // Exact rows: row(token of the group) is the key's row or null (zeros); the
  // exponent is that of the finite entries.
  template <typename Row>
  __device__ int exact_logits(Row&& row, float (&s)[4][4]) const {
    uint32_t top = 0;
#pragma unroll 1
    for (int n = 0; n < 4; ++n) {
      const __nv_bfloat16* src = row((n >> 1) * kBlock + few_key(quad, n & 1));
      if (src)
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          top = abs_max_bf16x8(top, finite_bf16x8(reinterpret_cast<const uint4*>(src + r * (D / 4))[k]));
        }
    }
    const int e = block_exp<kExactTopExp, kLeastExp>(__reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16)) << 16);
    const float f = pow2f(-e);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const __nv_bfloat16* src = row((n >> 1) * kBlock + few_key(quad, n & 1));
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (src) w = reinterpret_cast<const uint4*>(src + r * (D / 4))[k];
        mma_16816(s[n], q[2 * k], bf16x2_to_half(w.x, f), bf16x2_to_half(w.y, f));
        mma_16816(s[n], q[2 * k + 1], bf16x2_to_half(w.z, f), bf16x2_to_half(w.w, f));
      }
    }
    return e;
  }

  // Logits to weights, in place: 2^(logit - m_ref) 2^(ve - v_ref) as fp16 pairs a[block][4], the
  // products' left operand.  lim[i]: keys of the group that row quad + 8 i sees.
  __device__ void weights(float (&s)[4][4], int ke, int ve, const int (&lim)[2], uint32_t (&a)[2][4]) {
    bool masked = __any_sync(0xffffffffu, lim[0] < kGroup || lim[1] < kGroup);
    if (masked) {
      asm volatile("");
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((n >> 1) * kBlock + few_key(2 * r + (c & 1), n & 1) >= lim[c >> 1]) s[n][c] = -INFINITY;
    }
    const float value_exp = static_cast<float>(ve);
    float f[2], top[2];
    bool move = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[i] = logit_scale(p.scale_mantissa, row_exp[i] + ke);
      float t = max_nan(max3_nan(s[0][2 * i], s[0][2 * i + 1], s[1][2 * i]), max3_nan(s[1][2 * i + 1], s[2][2 * i], s[2][2 * i + 1]));
      t = max3_nan(t, s[3][2 * i], s[3][2 * i + 1]) * f[i];
      t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 1));
      top[i] = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 2));
      move = move || refs_move(m_ref[i], v_ref[i], top[i], top[i] + value_exp);
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float m_new = logit_ref(m_ref[i], top[i]);
        const float v_new = value_ref(v_ref[i], m_ref[i], m_new, top[i] - m_new + value_exp);
        const float shrink = m_new == m_ref[i] ? 0.f : m_ref[i] - m_new, g = fast_exp2(shrink + (v_ref[i] - v_new));
        sum[i] *= fast_exp2(shrink);
        m_ref[i] = m_new;
        v_ref[i] = v_new;
#pragma unroll
        for (int c = 0; c < CH; ++c) o[c][2 * i] *= g, o[c][2 * i + 1] *= g;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float de = fmaxf(value_exp - v_ref[i], kLeastShift);
      const float off = de - (m_ref[i] == -INFINITY ? 0.f : m_ref[i]);
      float part = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float x = fast_exp2(fmaf(s[n][2 * i], f[i], off)), y = fast_exp2(fmaf(s[n][2 * i + 1], f[i], off));
        part += x + y;
        a[n >> 1][2 * (n & 1) + i] = half2_bits(__floats2half2_rn(x, y));
      }
      sum[i] = fmaf(part, fast_exp2(-de), sum[i]);  // this thread's columns; the quad's are added at the end
    }
  }

  // (scale, min) words of the thread's tokens (4 r .. of each block) and channels;
  // tokens from n on are no values.  Returns the bits of the group's largest value,
  // those of infinity or above where one is not finite.
  __device__ uint32_t quant_value_meta(const uint8_t* rec, int n, uint32_t (&meta)[2][4]) const {
    const uint8_t* at = rec + R::kVMetaOff + (4 * r * (D / kGroup) + quad * CH / kGroup) * 4;
    float top = 0.f;
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        meta[blk][t] = *reinterpret_cast<const uint32_t*>(at + blk * R::kBytes + t * (D / kGroup) * 4);
    if (n < kGroup) {
      asm volatile("");  // a branch: most groups are full
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i >> 2) * kBlock + 4 * r + (i & 3) >= n) meta[i >> 2][i & 3] = 0u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = bf16_lo(meta[i >> 2][i & 3]), mn = bf16_hi(meta[i >> 2][i & 3]);
      top = max3_nan(top, fabsf(mn), fabsf(fmaf(s, kTop, mn)));
    }
    return __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  }

  // Zeros in the place of words that are not finite, which are left to odd_values.
  // Returns the bits of the largest of what remains.
  __device__ uint32_t finite_value_meta(uint32_t (&meta)[2][4]) const {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = meta[i >> 2][i & 3];
      if (odd_meta(w)) w = 0u;
      top = max3(top, fabsf(bf16_hi(w)), fabsf(fmaf(bf16_lo(w), kTop, bf16_hi(w))));
    }
    return __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  }

  __device__ void quant_output(const uint8_t* rec, const uint32_t (&meta)[2][4], int e, const uint32_t (&a)[2][4]) {
    const float fs = block_unit<kUnit>(e), f = fs * kPerUnit, fs4 = fs * 0.0625f;
    constexpr int COLS = D / 32;  // words of four channels that a thread has of a token quad
    const uint8_t* col = rec + R::kVHi + COLS * quad * kBlock + 4 * r;
    const uint8_t* row = rec + R::kQ4VLo + 4 * r * R::kRow + quad * (CH / 4);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      uint32_t hi[COLS], lo[4];
      float s[4], mn[4];
#pragma unroll
      for (int c = 0; c < COLS; ++c) hi[c] = *reinterpret_cast<const uint32_t*>(col + blk * R::kBytes + c * kBlock);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if constexpr (kSplit) {
          const uint8_t* at = row + blk * R::kBytes + t * R::kRow;
          lo[t] = D == 128 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
        }
        s[t] = bf16_lo(meta[blk][t]), mn[t] = bf16_hi(meta[blk][t]);
      }
      uint32_t b[CH][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // tokens (0, 2), (1, 3) of the four
        const __half2 sa = __floats2half2_rn(s[h] * fs, s[h + 2] * fs);
        const __half2 sb = __floats2half2_rn(s[h] * fs4, s[h + 2] * fs4);
        const __half2 m = __floats2half2_rn(mn[h] * f, mn[h + 2] * f);
#pragma unroll
        for (int c8 = 0; c8 < CH / 8; ++c8) {  // eight channels
          const uint32_t wh = __byte_perm(hi[2 * c8], hi[2 * c8 + 1], h ? 0x7351 : 0x6240);
          uint32_t even, odd;
          if constexpr (kSplit) {
            const uint32_t wl = __byte_perm(lo[h], lo[h + 2], c8 ? 0x7632 : 0x5410);
            even = join_bits(wh << 2, wl);
            odd = join_bits(wh, wl >> 2);
          } else {
            even = (wh << 2) & 0xCCCCCCCCu;
            odd = wh & 0xCCCCCCCCu;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // channels 2 i, 2 i + 1
            if (i == 2) even >>= 8, odd >>= 8;
            const uint32_t mask = i & 1 ? 0x00F000F0u : 0x000F000Fu;
            b[8 * c8 + 2 * i][h] = half2_bits(__hfma2(bits_half2(even & mask), i & 1 ? sb : sa, m));
            b[8 * c8 + 2 * i + 1][h] = half2_bits(__hfma2(bits_half2(odd & mask), i & 1 ? sb : sa, m));
          }
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) mma_16816(o[c], a[blk], b[c][0], b[c][1]);
    }
  }

  template <typename Row>
  __device__ int exact_value_exp(Row&& row, bool& odd) const {
    uint32_t top = 0;
    bool some = false;
#pragma unroll 1
    for (int t = 0; t < 8; ++t) {
      const __nv_bfloat16* src = row((t >> 2) * kBlock + 4 * r + (t & 3));
      if (src)
#pragma unroll
        for (int k = 0; k < CH / 8; ++k) {
          const uint4 w = reinterpret_cast<const uint4*>(src + quad * CH)[k], f = finite_bf16x8(w);
          some = some || w.x != f.x || w.y != f.y || w.z != f.z || w.w != f.w;
          top = abs_max_bf16x8(top, f);
        }
    }
    odd = __any_sync(0xffffffffu, some);
    return block_exp<kTopExp, kLeastExp>(__reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16)) << 16);
  }

  template <typename Row>
  __device__ void exact_output(Row&& row, int e, const uint32_t (&a)[2][4]) {
    const float f = pow2f(-e);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int k = 0; k < CH / 8; ++k) {  // eight channels
        uint32_t w[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const __nv_bfloat16* src = row(blk * kBlock + 4 * r + t);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (src) v = finite_bf16x8(reinterpret_cast<const uint4*>(src + quad * CH)[k]);
          w[t][0] = v.x, w[t][1] = v.y, w[t][2] = v.z, w[t][3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
          const uint32_t b0 = bf16x2_to_half(__byte_perm(w[0][i / 2], w[2][i / 2], sel), f);
          const uint32_t b1 = bf16x2_to_half(__byte_perm(w[1][i / 2], w[3][i / 2], sel), f);
          mma_16816(o[8 * k + i], a[blk], b0, b1);
        }
      }
  }
};

template <int KIND, int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, kFewWarpsPerSm / WARPS) chunk_few_kernel(const __grid_constant__ ChunkAttnParams p, int splits) {
  using L = FewSmem<KIND, D, WARPS>;
  using W = FewWarp<KIND, D>;
  using R = Rec<KIND, D>;
  constexpr int kThreads = WARPS * 32;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % splits;
  const uint32_t unit = blockIdx.x / splits;
  ChunkJob job;
  job.hk = unit % p.Hkv;
  job.b = unit / p.Hkv;
  if (!chunk_job<D>(p, job, 0, kFewRows, job.hk == 0 && rank == 0, rank == 0)) return;
  const int job_rows = job.len << p.g_log2;
  // groups over the stored tokens, then one over the chunk's own (at most 16) rows
  const int stored_groups = (job.stored + kGroup - 1) / kGroup, groups = stored_groups + (job.current ? 1 : 0);
  const int first = static_cast<int>(static_cast<int64_t>(groups) * rank / splits);
  const int last = static_cast<int>(static_cast<int64_t>(groups) * (rank + 1) / splits);
  const int mine = max(0, (last - first - warp + WARPS - 1) / WARPS);  // first + warp + WARPS i

  // this warp's ring: group i of its own in stage i % stages
  const uint32_t ring = sbase + warp * kFewStages * L::kGroupBytes, bar = sbase + L::kBars + warp * kFewStages * 8;
  const uint32_t odd_at = sbase + L::kOdd + warp * 16;
  if (lane == 0) {
    *reinterpret_cast<OddRange*>(smem + L::kOdd + warp * 16) = OddRange{INT32_MAX, 0};
    for (int s = 0; s < kFewStages; ++s) mbar_init(bar + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int32_t* table = p.block_table + static_cast<size_t>(job.b) * p.max_blocks;
  // block ids of 32 of its groups at a time, one group a thread
  int2 ids = make_int2(0, 0);
  auto load_ids = [&](int i0) {
    const int g = first + warp + (i0 + lane) * WARPS;
    if (i0 + lane < mine && g < stored_groups) {
      ids.x = table[2 * g];
      ids.y = 2 * g + 1 < (job.stored + kBlock - 1) / kBlock ? table[2 * g + 1] : -1;
    }
  };
  const uint64_t policy = l2_evict_first_policy();
  auto issue = [&](int i) {  // whole warp
    if (i % 32 == 0) load_ids(i);
    const int x = __shfl_sync(0xffffffffu, ids.x, i % 32), y = __shfl_sync(0xffffffffu, ids.y, i % 32);
    if (i < mine && first + warp + i * WARPS < stored_groups && lane == 0) {
      const uint32_t s = i % kFewStages, dst = ring + s * L::kGroupBytes;
      mbar_arrive_expect_tx(bar + 8 * s, (y >= 0 ? 2 : 1) * R::kBytes);
      bulk_load(dst, p.arena + (static_cast<size_t>(x) * p.Hkv + job.hk) * R::kBytes, R::kBytes, bar + 8 * s, policy);
      if (y >= 0)
        bulk_load(dst + R::kBytes, p.arena + (static_cast<size_t>(y) * p.Hkv + job.hk) * R::kBytes, R::kBytes, bar + 8 * s,
                  policy);
    }
  };
#pragma unroll 1
  for (int i = 0; i < kFewStages - 1; ++i) issue(i);

  W w(p, job, lane);
  w.load_queries(job_rows);
  const int token[2] = {min(w.quad, job_rows - 1) >> p.g_log2, min(w.quad + 8, job_rows - 1) >> p.g_log2};
  const uint32_t meta = sbase + L::kMeta + warp * D * 4;
  bool ok = true;
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    const int g = first + warp + i * WARPS, t0 = g * kGroup, s = i % kFewStages;
    __syncwarp();      // the stage that comes next has been read by all
    issue(i + kFewStages - 1);
    uint32_t a[2][4];
    if (g >= stored_groups) {
      float logit[4][4] = {};
      // the chunk's own rows, exactly
      auto key = [&](int t) { return t < job.len ? row_at(p.k_cur, job.b, t, job.hk) : nullptr; };
      auto value = [&](int t) { return t < job.len ? row_at(p.v_cur, job.b, t, job.hk) : nullptr; };
      const int lim[2] = {token[0] + 1, token[1] + 1};
      bool some;
      const int ke = w.exact_logits(key, logit), ve = w.exact_value_exp(value, some);
      if (some && lane == 0) note_odd_keys(odd_at, t0, kGroup);
      w.weights(logit, ke, ve, lim, a);
      w.exact_output(value, ve, a);
      continue;
    }
    ok = warp_wait(bar + 8 * s, (i / kFewStages) & 1);
    if (!ok) break;
    const uint8_t* rec = smem + (warp * kFewStages + s) * L::kGroupBytes;
    const int lim[2] = {(job.current ? job.stored : job.start + token[0] + 1) - t0,
                        (job.current ? job.stored : job.start + token[1] + 1) - t0};
    float logit[4][4] = {};
    int ke;
    if (t0 + kGroup <= job.stored) {
      ke = w.quant_logits(rec, meta, logit);
    } else {  // the open group's keys
      const __nv_bfloat16* res = p.residual + (static_cast<size_t>(job.b) * p.Hkv + job.hk) * kGroup * D;
      ke = w.exact_logits([&](int t) { return t0 + t < job.stored ? res + t * D : nullptr; }, logit);
    }
    uint32_t value_meta[2][4], top = w.quant_value_meta(rec, job.stored - t0, value_meta);
    if (top >= 0x7F800000u) {
      asm volatile("");
      if (lane == 0) note_odd_keys(odd_at, t0, kGroup);
      top = w.finite_value_meta(value_meta);
    }
    const int ve = block_exp(top);
    w.weights(logit, ke, ve, lim, a);
    w.quant_output(rec, value_meta, ve, a);
  }
  if (!ok) {  // later copies must not land in memory that has another use
    for (int s = 0; s < kFewStages; ++s) warp_wait(bar + 8 * s, 0), warp_wait(bar + 8 * s, 1);
    if (lane == 0) flag_error(p.chunk.err, LOOPKV_DEVERR_TIMEOUT);
  }

  // ---------------------------------------------------------------- join the warps
  __syncthreads();  // the rings are done with
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.sum[i] += __shfl_xor_sync(0xffffffffu, w.sum[i], 1);
    w.sum[i] += __shfl_xor_sync(0xffffffffu, w.sum[i], 2);
  }
  float* out = reinterpret_cast<float*>(smem) + warp * kFewRows * D;
  RowStats* stats = reinterpret_cast<RowStats*>(smem + L::kStats);      // [warp][16]
#pragma unroll
  for (int c = 0; c < W::CH; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k)  // column 2 r + (k & 1) of channel tile c: channel CH column + c
      out[(w.quad + 8 * (k >> 1)) * D + W::CH * (2 * w.r + (k & 1)) + c] = ok ? w.o[c][k] : 0.f;
  if (w.r == 0) {
    stats[warp * kFewRows + w.quad] = RowStats{w.m_ref[0], w.sum[0], w.v_ref[0]};
    stats[warp * kFewRows + w.quad + 8] = RowStats{w.m_ref[1], w.sum[1], w.v_ref[1]};
  }
  // what follows is worked out anew, so as not to hold it over the groups
  ChunkJob at;
  at.hk = (cta_id_x() / splits) % p.Hkv;
  at.b = (cta_id_x() / splits) / p.Hkv;
  const int tokens = p.chunk.new_lens ? p.chunk.new_lens[at.b] : p.chunk.T, rows = tokens << p.g_log2;
  __syncwarp();
  const OddRange odd = *reinterpret_cast<const OddRange*>(smem + L::kOdd + warp * 16);
  if (ok && odd.first < odd.end) {
    const int start = p.chunk.start_pos[at.b], stored = start + (p.k_cur.p ? 0 : tokens), t = lane >> p.g_log2;
    OddSum<D> sum;
    odd_values<KIND, D>(p, at.b, at.hk, start + (p.k_cur.p ? 0 : t + 1), t + 1, tokens,
                        (stored + kGroup - 1) / kGroup * kGroup, odd, sum);
    if (lane < rows) add_odd<D>(sum, [&](int c, float v) { out[lane * D + c] += v; });
  }
  __syncthreads();
  constexpr int kQuads = D / 4;
  float4* join = reinterpret_cast<float4*>(smem + L::kJoin);
  RowStats* join_stats = reinterpret_cast<RowStats*>(smem + L::kJoinStats);
  for (int i = threadIdx.x; i < rows * kQuads; i += kThreads) {
    const int row = i / kQuads, col = i % kQuads;
    auto stats_of = [&](int k) { return stats[k * kFewRows + row]; };
    RowStats all = join_refs(WARPS, stats_of);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < WARPS; ++k) {
      const RowStats st = stats_of(k);
      if (st.m == -INFINITY) continue;
      join_part(all, st, acc, reinterpret_cast<const float4*>(smem)[(k * kFewRows + row) * kQuads + col]);
    }
    if (splits == 1) {
      reinterpret_cast<uint2*>(chunk_out<D>(p, at, row))[col] = join_result(all, acc);
    } else {
      join[i] = acc;
      if (col == 0) join_stats[row] = all;
    }
  }
  if (splits == 1) return;
  const int rank_again = cta_id_x() % splits;
  cluster_sync_all();
  for (int i = threadIdx.x; i < rows * kQuads; i += kThreads) {
    if (i / 32 % splits != rank_again) continue;
    const int row = i / kQuads;
    join_splits<D>(p, at, row, i % kQuads, splits, sbase + L::kJoinStats + row * 16, sbase + L::kJoin + i * 16);
  }
  cluster_sync_all();
}

}  // namespace loopkv
