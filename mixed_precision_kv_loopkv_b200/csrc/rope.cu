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
#include "append_ops.cuh"
#include "chunk_common.cuh"

namespace loopkv {
namespace {

constexpr int kThreads = 128;

// Mask of the LANES threads of a row within its warp.
template <int LANES>
__device__ __forceinline__ uint32_t row_mask() {
  return (LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1)) << ((threadIdx.x & 31) & ~(LANES - 1));
}

// cos and signed sin of this thread's eight channels at one position.
struct Turn {
  float c[8], s[8];
};

// Channels 8 sub .. 8 sub + 7.  "Halves": the partner of channel i is i +- rot/2,
// first half y = a cos - b sin, second y = b cos + a sin; neighbours: the same
// over (2 i, 2 i + 1).  s carries the sign of the first half.
__device__ __forceinline__ void load_turn(const RotaryView& r, int pos, int sub, Turn& t) {
  const int c0 = 8 * sub, half = r.rot / 2;
  if (!r.cos_sin || c0 >= r.rot) return;
  const float* row = r.cos_sin + static_cast<size_t>(pos) * r.rot;
  if (r.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(row + c0 / 2);
    const float4 s = *reinterpret_cast<const float4*>(row + half + c0 / 2);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.c[2 * i] = t.c[2 * i + 1] = cc[i];
      t.s[2 * i] = -ss[i];
      t.s[2 * i + 1] = ss[i];
    }
  } else {
    const bool first = c0 < half;
    const float* at = row + (first ? c0 : c0 - half);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c = *reinterpret_cast<const float4*>(at + i);
      const float4 s = *reinterpret_cast<const float4*>(at + half + i);
      t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
      t.s[i] = first ? -s.x : s.x, t.s[i + 1] = first ? -s.y : s.y;
      t.s[i + 2] = first ? -s.z : s.z, t.s[i + 3] = first ? -s.w : s.w;
    }
  }
}

// Norm (w: this thread's eight weights, or null) and rotation of one row; the
// LANES threads of the row call it together.
template <int D>
__device__ __forceinline__ void norm_rotate(const RotaryView& r, const uint4* w, const Turn& t, int sub, float (&x)[8]) {
  constexpr int LANES = D / 8;
  const uint32_t mask = row_mask<LANES>();
  if (w) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sum);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
    const float inv = static_cast<float>(rsqrt(sum * (1.0 / D) + r.eps));
    float ww[8];
    unpack8(*w, ww);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), ww[i]);
  }
  if (!r.cos_sin) return;
  float other[8];
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = x[i ^ 1];
  } else {
    const int hl = r.rot / 16;  // threads of half the rotated channels
    const int peer = (sub < hl ? sub + hl : sub - hl) & (LANES - 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(mask, x[i], peer, LANES);
  }
  if (8 * sub < r.rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], t.c[i]), __fmul_rn(other[i], t.s[i]));
  }
}

// Four heads of one token of the chunk, for the threads of one row: the table's
// row is loaded once for the four (it is as many bytes as two rows of bf16).
constexpr int kHeadsPerItem = 4;

template <int D>
__device__ __forceinline__ void rotate_item(const RotateParams& p, uint32_t item, int sub) {
  const int heads = p.H + p.Hk;
  const uint32_t per_token = (heads + kHeadsPerItem - 1) / kHeadsPerItem;
  const uint32_t bt = item / per_token;
  const int h0 = static_cast<int>(item % per_token) * kHeadsPerItem;
  const int b = bt / p.chunk.T, t = bt % p.chunk.T;
  const SeqChunk sc = seq_chunk(p.chunk, b, t == 0 && h0 == 0 && sub == 0);
  if (t >= sc.len) return;
  uint4 raw[kHeadsPerItem];
#pragma unroll
  for (int i = 0; i < kHeadsPerItem; ++i) {
    const int h = h0 + i;
    if (h < heads)
      raw[i] = *reinterpret_cast<const uint4*>((h < p.H ? row_at(p.q, b, t, h) : row_at(p.k, b, t, h - p.H)) + 8 * sub);
  }
  Turn turn;
  load_turn(p.rot, sc.start + t, sub, turn);
#pragma unroll
  for (int i = 0; i < kHeadsPerItem; ++i) {
    const int h = h0 + i;
    if (h >= heads) break;
    const bool is_q = h < p.H;
    const __nv_bfloat16* weight = is_q ? p.rot.q_weight : p.rot.k_weight;
    uint4 w;
    if (weight) w = *reinterpret_cast<const uint4*>(weight + 8 * sub);
    float x[8];
    unpack8(raw[i], x);
    norm_rotate<D>(p.rot, weight ? &w : nullptr, turn, sub, x);
    const size_t token = static_cast<size_t>(b) * p.chunk.T + t;
    __nv_bfloat16* o = is_q ? p.q_out + (token * p.H + h) * D : p.k_out + (token * p.Hk + (h - p.H)) * D;
    *reinterpret_cast<uint4*>(o + 8 * sub) = pack8(x);
  }
}

uint32_t rotate_items(const RotateParams& p) {
  const uint32_t per_token = (p.H + p.Hk + kHeadsPerItem - 1) / kHeadsPerItem;
  return static_cast<uint32_t>(p.chunk.B) * p.chunk.T * per_token;
}

template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RotateParams p, uint32_t items) {
  constexpr int LANES = D / 8;
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  if (item < items) rotate_item<D>(p, item, threadIdx.x % LANES);
}

// The code of x in a group with scale s and minimum mn: rint((x - mn) / s),
// as group_code, without the division where it cannot matter.  t = a * (1/s) is
// within 2^-22 |t| < 1e-5 of the rounded quotient (|t| < 24), so where t is more
// than 1e-3 away from a half both round to the same integer; elsewhere (also
// where 1/s overflows and t is no number) the quotient itself is taken.
template <int BITS>
__device__ __forceinline__ uint32_t quick_code(float x, float s, float mn, float inv) {
  const float a = __fsub_rn(x, mn);
  const float t = __fmul_rn(a, inv);
  float r = rintf(t);
  if (!(fabsf(t - r) <= 0.499f)) r = s == 0.f ? 0.f : rintf(__fdiv_rn(a, s));
  return static_cast<uint32_t>(fminf(fmaxf(r, 0.f), static_cast<float>((1 << BITS) - 1)));
}

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeAppendParams p, uint32_t kv_blocks,
                                                               uint32_t items) {
  constexpr int LANES = D / 8, ROWS = kThreads / LANES, ITERS = kGroup / ROWS;
  const int sub = threadIdx.x % LANES, row0 = threadIdx.x / LANES;
  if (blockIdx.x >= kv_blocks) {  // the queries
    const uint32_t item = (blockIdx.x - kv_blocks) * ROWS + row0;
    if (item < items) rotate_item<D>(p.rows, item, sub);
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
  uint4 w_raw;
  if (rot.k_weight) w_raw = *reinterpret_cast<const uint4*>(rot.k_weight + 8 * sub);
  const uint4* w = rot.k_weight ? &w_raw : nullptr;

  uint4 k_raw[ITERS], v_raw[ITERS];
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int pos = g0 + it * ROWS + row0;
    if (pos >= tok0 && pos < tok1) {
      k_raw[it] = *reinterpret_cast<const uint4*>(row_at(p.k, b, pos - start, h) + 8 * sub);
      v_raw[it] = *reinterpret_cast<const uint4*>(row_at(p.v, b, pos - start, h) + 8 * sub);
    }
  }

  if constexpr (KIND == LOOPKV_CELL_BF16) {
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const int pos = g0 + it * ROWS + row0;
      if (pos < tok0 || pos >= tok1) continue;
      Turn turn;
      load_turn(rot, pos, sub, turn);
      float x[8];
      unpack8(k_raw[it], x);
      norm_rotate<D>(rot, w, turn, sub, x);
      uint8_t* rec = record_at<KIND, D>(cell, pos);
      if (!rec) continue;
      const int row = pos % kBlock;
      *reinterpret_cast<uint4*>(rec + R::kBfK + row * D * 2 + 16 * sub) = pack8(x);
      *reinterpret_cast<uint4*>(rec + R::kBfV + row * D * 2 + 16 * sub) = v_raw[it];
    }
    return;
  } else {
    constexpr int BITS = KIND == LOOPKV_CELL_Q4 ? 4 : 2;
    constexpr bool kSplit = KIND == LOOPKV_CELL_Q4;
    constexpr int kVGroups = D / kGroup;
    constexpr float kTop = static_cast<float>((1 << BITS) - 1);
    // rows a little apart, so that threads of one column quad on different rows meet different banks
    constexpr int kStride = D * 2 + (D == 128 ? 32 : 16);
    __shared__ __align__(16) uint8_t tile[kGroup * kStride];
    __shared__ __align__(16) uint8_t rec[2 * R::kBytes];

    __nv_bfloat16* res = p.residual + (static_cast<size_t>(b) * p.Hkv + h) * kGroup * D;
    // The open group's exact keys belong to the call's last group, unless the
    // first group still has to read older ones from there: then its CTA, after
    // it has read them, writes the last group's keys too.
    const bool begun = start % kGroup != 0;

#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const int r = it * ROWS + row0, pos = g0 + r;
      if (pos >= tok0 && pos < tok1) {
        Turn turn;
        load_turn(rot, pos, sub, turn);
        float x[8];
        unpack8(k_raw[it], x);
        norm_rotate<D>(rot, w, turn, sub, x);
        const uint4 packed = pack8(x);
        *reinterpret_cast<uint4*>(tile + r * kStride + 16 * sub) = packed;
        if (!complete && (gi == 0 || !begun)) *reinterpret_cast<uint4*>(res + r * D + 8 * sub) = packed;
        // the value row: groups of 32 channels are four neighbouring threads
        float v[8];
        unpack8(v_raw[it], v);
        float mn = v[0], mx = v[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mn = fminf(mn, v[i]), mx = fmaxf(mx, v[i]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          mn = fminf(mn, __shfl_xor_sync(row_mask<LANES>(), mn, o));
          mx = fmaxf(mx, __shfl_xor_sync(row_mask<LANES>(), mx, o));
        }
        float s_b, mn_b;
        group_params<BITS>(mn, mx, s_b, mn_b);
        const float inv = __frcp_rn(s_b);
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t code = quick_code<BITS>(v[i], s_b, mn_b, inv);
          hi |= (kSplit ? code >> 2 : code) << (2 * i);
          if constexpr (kSplit) lo |= (code & 3u) << (2 * i);
        }
        uint8_t* dst = rec + (r / kBlock) * R::kBytes;
        const int row = r % kBlock;
        dst[R::kVHi + (2 * sub) * kBlock + row] = static_cast<uint8_t>(hi);
        dst[R::kVHi + (2 * sub + 1) * kBlock + row] = static_cast<uint8_t>(hi >> 8);
        if constexpr (kSplit) *reinterpret_cast<uint16_t*>(dst + R::kQ4VLo + row * R::kRow + 2 * sub) = static_cast<uint16_t>(lo);
        if (sub % 4 == 0) *reinterpret_cast<uint32_t*>(dst + R::kVMetaOff + (row * kVGroups + sub / 4) * 4) = meta_word(s_b, mn_b);
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
      float s_b[4], mn_b[4], inv[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int o = 1; o < NS; o <<= 1) {
          mn[c] = fminf(mn[c], __shfl_xor_sync(0xffffffffu, mn[c], o));
          mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], o));
        }
        group_params<BITS>(mn[c], mx[c], s_b[c], mn_b[c]);
        inv[c] = __frcp_rn(s_b[c]);
      }
#pragma unroll
      for (int k = 0; k < kGroup / NS; ++k) {
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t code = quick_code<BITS>(x[k][c], s_b[c], mn_b[c], inv[c]);
          hi |= (kSplit ? code >> 2 : code) << (2 * c);
          if constexpr (kSplit) lo |= (code & 3u) << (2 * c);
        }
        const int r = ns + NS * k;
        uint8_t* dst = rec + (r / kBlock) * R::kBytes + (r % kBlock) * R::kRow + quad;
        dst[R::kKHi] = static_cast<uint8_t>(hi);
        if constexpr (kSplit) dst[R::kQ4KLo] = static_cast<uint8_t>(lo);
      }
      if (ns == 0) {
        const int c0 = 4 * quad;
        uint8_t* dst = rec + (c0 < D / 2 ? 0 : R::kBytes) + R::kKMetaOff + (c0 % (D / 2)) * 4;
        *reinterpret_cast<uint4*>(dst) = make_uint4(meta_word(s_b[0], mn_b[0]), meta_word(s_b[1], mn_b[1]),
                                                    meta_word(s_b[2], mn_b[2]), meta_word(s_b[3], mn_b[3]));
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
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        const int r = it * ROWS + row0, pos = tail0 + r;
        if (pos >= end) continue;
        Turn turn;
        load_turn(rot, pos, sub, turn);
        float x[8];
        unpack8(*reinterpret_cast<const uint4*>(row_at(p.k, b, pos - start, h) + 8 * sub), x);
        norm_rotate<D>(rot, w, turn, sub, x);
        *reinterpret_cast<uint4*>(res + r * D + 8 * sub) = pack8(x);
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
  rope_append_kernel<KIND, D><<<blocks, kThreads, 0, stream>>>(p, kv_blocks, items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(int head_dim, const RotateParams& p, cudaStream_t stream) {
  const uint32_t items = rotate_items(p), rows = kThreads / (head_dim / 8);
  const uint32_t blocks = (items + rows - 1) / rows;
  if (head_dim == 128)
    norm_rope_kernel<128><<<blocks, kThreads, 0, stream>>>(p, items);
  else
    norm_rope_kernel<64><<<blocks, kThreads, 0, stream>>>(p, items);
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
