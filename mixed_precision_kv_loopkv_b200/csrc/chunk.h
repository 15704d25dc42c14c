// Launch interface of the prompt-side kernels (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "loopkv_chunk.h"

namespace loopkv {

// bf16 rows [batch][token][head][D] with strides in elements.
struct RowView {
  const __nv_bfloat16* p;
  int64_t sb, st, sh;
};

struct RotaryView {
  const float* cos_sin;          // [max_positions][rot]
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  double eps;
  int max_positions, rot, interleaved;  // rot 0: no rotation
};

// Which tokens of the chunk a sequence has, and how far its positions may go.
struct ChunkView {
  const int32_t* start_pos;
  const int32_t* new_lens;       // optional
  int32_t* err;                  // optional
  int B, T;
  int64_t max_end;               // start + len beyond this is a fault
};

// Norms and rotation of the heads of q (first) and k, one row each.
struct RotateParams {
  RotaryView rot;
  ChunkView chunk;
  RowView q, k;
  __nv_bfloat16 *q_out, *k_out;  // [B][T][H][D], [B][T][Hk][D]
  int H, Hk;                     // heads of q and k to do (0: none)
};

struct RopeAppendParams {
  RotateParams rows;             // the queries (Hk = 0)
  RowView k, v;
  uint8_t* arena;                // [num_blocks][Hkv][record]
  __nv_bfloat16* residual;       // [max_batch][Hkv][32][D], null for bf16 cells
  const int32_t* block_table;    // [B][max_blocks]
  int Hkv, max_blocks, num_blocks;
  int key_blocks;                // 32-token groups a sequence's chunk can touch
};

struct ReadParams {
  const uint8_t* arena;
  const __nv_bfloat16* residual;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* start_pos;
  __nv_bfloat16 *k_out, *v_out;  // [B][T][Hkv][D], each optional
  int32_t* err;
  int B, T, Hkv, max_blocks, num_blocks;
  int groups;                    // 32-token groups a sequence's range can touch
};

struct ChunkAttnParams {
  const uint8_t* arena;
  const __nv_bfloat16* residual;
  const int32_t* block_table;
  RowView q, k_cur, v_cur;       // k_cur.p null: the chunk is stored
  __nv_bfloat16* out;            // [B][T][H][D]
  ChunkView chunk;
  int H, Hkv, g_log2, max_blocks, num_blocks;
  int max_stored;                // host bound of the stored tokens
  float scale_mantissa;          // |sm_scale * log2(e)| = mantissa in [1, 2) times 2^exp
  int scale_exp, scale_negative;
};

cudaError_t launch_norm_rope(int head_dim, const RotateParams& p, cudaStream_t stream);
cudaError_t launch_rope_append(int kind, int head_dim, const RopeAppendParams& p, cudaStream_t stream);
cudaError_t launch_read(int kind, int head_dim, const ReadParams& p, cudaStream_t stream);
cudaError_t launch_chunk_attention(int kind, int head_dim, const ChunkAttnParams& p, cudaStream_t stream);

}  // namespace loopkv
