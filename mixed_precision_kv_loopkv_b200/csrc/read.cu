// A range of a cell's tokens as the values that they stand for (sm_100a).
//
// One CTA per (sequence, KV head, 32-token group): the group's two records
// come in as 16-byte loads, every thread then turns eight channels of a token
// into bf16 (min + scale * code in fp32, rounded once).  4 x up to 8192 tokens of
// 16 4-bit heads of 128: 54 us on a B200, 4.8 TB/s of 258 MB, most of it stores.
#include "chunk_common.cuh"

namespace loopkv {
namespace {

constexpr int kThreads = 128;

// Eight channels' codes (two bits of each in hi and, of 4-bit cells, in lo) and
// their (scale, min) words -> values.  A code becomes a float as the low bits of
// 2^23 (the conversion instruction runs at a quarter of the rate).
template <bool SPLIT, typename Meta>
__device__ __forceinline__ uint4 stand_for(uint32_t hi, uint32_t lo, Meta&& meta) {
  constexpr uint32_t kMask = SPLIT ? 15u : 3u;
  // nibble n: channel 2 n, 2 n + 1
  const uint32_t even = SPLIT ? ((hi << 2) & 0xCCCCu) | (lo & 0x3333u) : hi;
  const uint32_t odd = SPLIT ? (hi & 0xCCCCu) | ((lo >> 2) & 0x3333u) : hi >> 2;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = meta(i), code = ((i & 1 ? odd : even) >> (4 * (i / 2))) & kMask;
    x[i] = fmaf(bf16_lo(m), __uint_as_float(code | 0x4B000000u) - 8388608.f, bf16_hi(m));
  }
  return pack8(x);
}

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  using R = Rec<KIND, D>;
  constexpr int LANES = D / 8, ROWS = kThreads / LANES, kVec = R::kBytes / 16;
  __shared__ __align__(16) uint8_t rec[KIND == LOOPKV_CELL_BF16 ? 16 : 2 * R::kBytes];
  const int gi = blockIdx.x % p.groups;
  const int h = (blockIdx.x / p.groups) % p.Hkv;
  const int b = blockIdx.x / p.groups / p.Hkv;
  const int start = p.start_pos[b], n = p.seq_lens[b];
  if (start < 0) return;
  if (n < 0 || n > static_cast<int64_t>(p.max_blocks) * kBlock) {
    if (gi == 0 && h == 0 && threadIdx.x == 0) flag_error(p.err, LOOPKV_DEVERR_SEQ_LEN);
    return;
  }
  const int end = static_cast<int>(min(static_cast<int64_t>(start) + p.T, static_cast<int64_t>(n)));
  const int64_t first = (static_cast<int64_t>(start) / kGroup + gi) * kGroup;
  if (first >= end) return;
  const int g0 = static_cast<int>(first);
  const int tok0 = max(start, g0), tok1 = min(end, g0 + kGroup);
  const bool complete = g0 + kGroup <= n;  // else its keys are still exact, in the residual

  const uint8_t* src[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    src[j] = nullptr;
    // a full group's key scales lie in both of its blocks, whatever is asked of it
    const bool asked = tok0 < g0 + kBlock * (j + 1) && tok1 > g0 + kBlock * j;
    if (!asked && !(complete && KIND != LOOPKV_CELL_BF16)) continue;
    const int phys = p.block_table[static_cast<size_t>(b) * p.max_blocks + g0 / kBlock + j];
    if (phys < 0 || phys >= p.num_blocks) {
      if (threadIdx.x == 0) flag_error(p.err, LOOPKV_DEVERR_BLOCK_ID);
      continue;
    }
    src[j] = p.arena + (static_cast<size_t>(phys) * p.Hkv + h) * R::kBytes;
  }
  const int sub = threadIdx.x % LANES, row0 = threadIdx.x / LANES;
  const size_t out0 = (static_cast<size_t>(b) * p.T * p.Hkv + h) * D + 8 * sub;
  const size_t out_stride = static_cast<size_t>(p.Hkv) * D;

  if constexpr (KIND == LOOPKV_CELL_BF16) {
#pragma unroll
    for (int it = 0; it < kGroup / ROWS; ++it) {
      const int r = it * ROWS + row0, pos = g0 + r;
      const uint8_t* s = src[r / kBlock];
      if (pos < tok0 || pos >= tok1 || !s) continue;
      const size_t o = out0 + (pos - start) * out_stride;
      const int at = (r % kBlock) * D * 2 + 16 * sub;
      if (p.k_out) *reinterpret_cast<uint4*>(p.k_out + o) = *reinterpret_cast<const uint4*>(s + R::kBfK + at);
      if (p.v_out) *reinterpret_cast<uint4*>(p.v_out + o) = *reinterpret_cast<const uint4*>(s + R::kBfV + at);
    }
  } else {
    constexpr bool kSplit = KIND == LOOPKV_CELL_Q4;
#pragma unroll
    for (int i = threadIdx.x; i < 2 * kVec; i += kThreads) {
      const uint8_t* s = i < kVec ? src[0] : src[1];
      if (s) reinterpret_cast<uint4*>(rec)[i] = reinterpret_cast<const uint4*>(s)[i % kVec];
    }
    __syncthreads();
    // a block that is missing takes its tokens with it; of a full group it also
    // takes the keys of the other block, whose scales it holds half of
    const bool keys_here = !complete || (src[0] && src[1]);
    const __nv_bfloat16* res = p.residual + (static_cast<size_t>(b) * p.Hkv + h) * kGroup * D;
#pragma unroll
    for (int it = 0; it < kGroup / ROWS; ++it) {
      const int r = it * ROWS + row0, pos = g0 + r, row = r % kBlock;
      if (pos < tok0 || pos >= tok1 || !src[r / kBlock]) continue;
      const uint8_t* rb = rec + (r / kBlock) * R::kBytes;
      const size_t o = out0 + (pos - start) * out_stride;
      if (p.k_out && keys_here) {
        if (!complete) {
          *reinterpret_cast<uint4*>(p.k_out + o) = *reinterpret_cast<const uint4*>(res + r * D + 8 * sub);
        } else {
          const uint32_t hi = *reinterpret_cast<const uint16_t*>(rb + R::kKHi + row * R::kRow + 2 * sub);
          const uint32_t lo = kSplit ? *reinterpret_cast<const uint16_t*>(rb + R::kQ4KLo + row * R::kRow + 2 * sub) : 0u;
          const uint4* mp = reinterpret_cast<const uint4*>(rec + (8 * sub < D / 2 ? 0 : R::kBytes) + R::kKMetaOff +
                                                           ((8 * sub) % (D / 2)) * 4);
          const uint4 m0 = mp[0], m1 = mp[1];
          const uint32_t m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
          *reinterpret_cast<uint4*>(p.k_out + o) = stand_for<kSplit>(hi, lo, [&](int i) { return m[i]; });
        }
      }
      if (p.v_out) {
        const uint32_t hi = rb[R::kVHi + (2 * sub) * kBlock + row] | (rb[R::kVHi + (2 * sub + 1) * kBlock + row] << 8);
        const uint32_t lo = kSplit ? *reinterpret_cast<const uint16_t*>(rb + R::kQ4VLo + row * R::kRow + 2 * sub) : 0u;
        const uint32_t m = *reinterpret_cast<const uint32_t*>(rb + R::kVMetaOff + (row * (D / kGroup) + sub / 4) * 4);
        *reinterpret_cast<uint4*>(p.v_out + o) = stand_for<kSplit>(hi, lo, [&](int) { return m; });
      }
    }
  }
}

template <int KIND, int D>
cudaError_t launch_read_t(const ReadParams& p, cudaStream_t stream) {
  read_kernel<KIND, D><<<static_cast<uint32_t>(p.B) * p.Hkv * p.groups, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_read(int kind, int head_dim, const ReadParams& p, cudaStream_t stream) {
  switch (kind * 1000 + head_dim) {
    case LOOPKV_CELL_Q4 * 1000 + 128: return launch_read_t<LOOPKV_CELL_Q4, 128>(p, stream);
    case LOOPKV_CELL_Q4 * 1000 + 64: return launch_read_t<LOOPKV_CELL_Q4, 64>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 128: return launch_read_t<LOOPKV_CELL_Q2, 128>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 64: return launch_read_t<LOOPKV_CELL_Q2, 64>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 128: return launch_read_t<LOOPKV_CELL_BF16, 128>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 64: return launch_read_t<LOOPKV_CELL_BF16, 64>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace loopkv
