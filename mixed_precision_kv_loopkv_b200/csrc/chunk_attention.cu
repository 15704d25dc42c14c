// Attention of a chunk of new tokens over a paged LoopKV cell (sm_100a).
//
// Plain form: one CTA per (sequence, KV head, 16 rows); a row is one (token,
// query head).  The CTA walks the keys 32 at a time, dequantises them in fp32
// into shared memory and updates the running maximum and sum of each row's
// softmax; a warp holds four rows, four output channels a thread.
#include "chunk_common.cuh"

namespace loopkv {
namespace {

constexpr int kThreads = 128, kRowsPerCta = 16, kRowsPerWarp = 4;

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) chunk_plain_kernel(const ChunkAttnParams p, int tiles) {
  using R = Rec<KIND, D>;
  constexpr int CPL = D / 32;
  __shared__ float ks[kGroup][D + 1];
  __shared__ float vs[kGroup][D];
  __shared__ float qs[kRowsPerCta][D];
  const int tile = blockIdx.x % tiles, hk = (blockIdx.x / tiles) % p.Hkv, b = blockIdx.x / tiles / p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = 1 << p.g_log2;
  bool bad;
  ChunkView view = p.chunk;
  const bool current = p.k_cur.p != nullptr;
  SeqChunk sc;
  sc.start = view.start_pos[b];
  sc.len = view.new_lens ? view.new_lens[b] : view.T;
  bad = sc.len < 0 || sc.len > view.T;
  const int64_t stored64 = static_cast<int64_t>(sc.start) + (current ? 0 : sc.len);
  bool zero = sc.start < 0;
  if (bad || (!zero && sc.len > 0 && stored64 > p.max_stored)) {
    if (threadIdx.x == 0) flag_error(view.err, LOOPKV_DEVERR_SEQ_LEN);
    zero = true;
    if (bad) sc.len = 0;
  }
  const int rows = sc.len << p.g_log2, row_first = tile * kRowsPerCta;
  if (row_first >= rows) return;
  const int row_last = min(rows, row_first + kRowsPerCta) - 1;
  const int stored = zero ? 0 : static_cast<int>(stored64);
  // keys this tile can see: stored ones, then the chunk's own rows
  const int seen_stored = current ? stored : min(stored, sc.start + (row_last >> p.g_log2) + 1);
  const int seen = zero ? 0 : seen_stored + (current ? (row_last >> p.g_log2) + 1 : 0);
  for (int i = threadIdx.x; i < kRowsPerCta * D; i += kThreads) {
    const int r = row_first + i / D;
    qs[i / D][i % D] = r <= row_last
        ? __bfloat162float(row_at(p.q, b, r >> p.g_log2, (hk << p.g_log2) + (r & (G - 1)))[i % D]) : 0.f;
  }
  float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][CPL] = {};
  for (int r = 0; r < kRowsPerWarp; ++r) m[r] = -INFINITY, l[r] = 0.f;
  int failed = 0;
  const int stored_groups = (seen_stored + 31) / 32;
  const int groups = stored_groups + (current && !zero ? ((row_last >> p.g_log2) + 32) / 32 : 0);
  for (int g = 0; g < groups; ++g) {
    __syncthreads();
    const bool own_rows = g >= stored_groups;
    const int t0 = own_rows ? (g - stored_groups) * 32 : g * 32;
    const int lim = own_rows ? (row_last >> p.g_log2) + 1 : seen_stored;
    const bool complete = !own_rows && t0 + 32 <= stored;
    const uint8_t* rec[2] = {nullptr, nullptr};
    if (!own_rows) {
      for (int j = 0; j < 2; ++j) {
        if (t0 + 16 * j >= stored) continue;
        const int phys = p.block_table[static_cast<size_t>(b) * p.max_blocks + t0 / kBlock + j];
        if (phys < 0 || phys >= p.num_blocks) failed = 1;
        else rec[j] = p.arena + (static_cast<size_t>(phys) * p.Hkv + hk) * R::kBytes;
      }
      if (failed) break;
    }
    for (int i = threadIdx.x; i < kGroup * D; i += kThreads) {
      const int t = i / D, c = i % D, row = t % kBlock;
      float kx = 0.f, vx = 0.f;
      if (t0 + t < lim) {
        if (own_rows) {
          kx = __bfloat162float(row_at(p.k_cur, b, t0 + t, hk)[c]);
          vx = __bfloat162float(row_at(p.v_cur, b, t0 + t, hk)[c]);
        } else if constexpr (KIND == LOOPKV_CELL_BF16) {
          kx = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(rec[t / 16] + R::kBfK)[row * D + c]);
          vx = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(rec[t / 16] + R::kBfV)[row * D + c]);
        } else {
          constexpr bool kSplit = KIND == LOOPKV_CELL_Q4;
          const uint8_t* rb = rec[t / 16];
          if (!complete) {
            kx = __bfloat162float(p.residual[((static_cast<size_t>(b) * p.Hkv + hk) * kGroup + t) * D + c]);
          } else {
            uint32_t code = (rb[R::kKHi + row * R::kRow + c / 4] >> (2 * (c % 4))) & 3;
            if (kSplit) code = (code << 2) | ((rb[R::kQ4KLo + row * R::kRow + c / 4] >> (2 * (c % 4))) & 3);
            const uint32_t w = *reinterpret_cast<const uint32_t*>(rec[c < D / 2 ? 0 : 1] + R::kKMetaOff + (c % (D / 2)) * 4);
            kx = fmaf(bf16_lo(w), static_cast<float>(code), bf16_hi(w));
          }
          uint32_t code = (rb[R::kVHi + (c / 4) * kBlock + row] >> (2 * (c % 4))) & 3;
          if (kSplit) code = (code << 2) | ((rb[R::kQ4VLo + row * R::kRow + c / 4] >> (2 * (c % 4))) & 3);
          const uint32_t w = *reinterpret_cast<const uint32_t*>(rb + R::kVMetaOff + (row * (D / kGroup) + c / kGroup) * 4);
          vx = fmaf(bf16_lo(w), static_cast<float>(code), bf16_hi(w));
        }
      }
      ks[t][c] = kx;
      vs[t][c] = vx;
    }
    __syncthreads();
    for (int r = 0; r < kRowsPerWarp; ++r) {
      const int lr = warp * kRowsPerWarp + r, row = row_first + lr;
      const int token = row >> p.g_log2;
      const int last = own_rows ? token : current ? stored - 1 : sc.start + token;
      float s = 0.f;
      for (int c = 0; c < D; ++c) s = fmaf(qs[lr][c], ks[lane][c], s);
      s *= p.sm_scale_log2;
      if (t0 + lane > last || t0 + lane >= lim) s = -INFINITY;
      float mx = s;
      for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float m_new = fmaxf(m[r], mx);
      const float scale = m_new == -INFINITY ? 1.f : exp2f(m[r] - m_new);
      const float e = m_new == -INFINITY ? 0.f : exp2f(s - m_new);
      m[r] = m_new;
      float sum = e;
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[r] = l[r] * scale + sum;
      for (int j = 0; j < CPL; ++j) o[r][j] *= scale;
      for (int k = 0; k < 32; ++k) {
        const float pk = __shfl_sync(0xffffffffu, e, k);
        for (int j = 0; j < CPL; ++j) o[r][j] = fmaf(pk, vs[k][lane + 32 * j], o[r][j]);
      }
    }
  }
  if (failed) {
    if (threadIdx.x == 0) flag_error(view.err, LOOPKV_DEVERR_BLOCK_ID);
    zero = true;
  }
  (void)seen;
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const int row = row_first + warp * kRowsPerWarp + r;
    if (row > row_last) continue;
    const int t = row >> p.g_log2, h = (hk << p.g_log2) + (row & (G - 1));
    const float inv = zero || l[r] == 0.f ? 0.f : 1.f / l[r];
    __nv_bfloat16* dst = p.out + ((static_cast<size_t>(b) * view.T + t) * p.H + h) * D;
    for (int j = 0; j < CPL; ++j) dst[lane + 32 * j] = __float2bfloat16_rn(zero ? 0.f : o[r][j] * inv);
  }
}

template <int KIND, int D>
cudaError_t launch_t(const ChunkAttnParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.chunk.T) << p.g_log2;
  const int tiles = static_cast<int>((rows + kRowsPerCta - 1) / kRowsPerCta);
  chunk_plain_kernel<KIND, D><<<static_cast<uint32_t>(p.chunk.B) * p.Hkv * tiles, kThreads, 0, stream>>>(p, tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_attention(int kind, int head_dim, const ChunkAttnParams& p, cudaStream_t stream) {
  switch (kind * 1000 + head_dim) {
    case LOOPKV_CELL_Q4 * 1000 + 128: return launch_t<LOOPKV_CELL_Q4, 128>(p, stream);
    case LOOPKV_CELL_Q4 * 1000 + 64: return launch_t<LOOPKV_CELL_Q4, 64>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 128: return launch_t<LOOPKV_CELL_Q2, 128>(p, stream);
    case LOOPKV_CELL_Q2 * 1000 + 64: return launch_t<LOOPKV_CELL_Q2, 64>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 128: return launch_t<LOOPKV_CELL_BF16, 128>(p, stream);
    case LOOPKV_CELL_BF16 * 1000 + 64: return launch_t<LOOPKV_CELL_BF16, 64>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace loopkv
