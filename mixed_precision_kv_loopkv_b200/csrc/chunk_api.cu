// C ABI of the prompt side: argument validation, plan resolution and kernel
// dispatch.  See include/loopkv_chunk.h for the contract of every call.
#include <math.h>
#include <stdint.h>

#include "api_checks.h"
#include "chunk.h"

namespace {

using namespace loopkv;

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;  // and tokens of a sequence
constexpr float kLog2e = 1.4426950408889634f;

bool rows_ok(const loopkv_rows* r) {
  return r->data && aligned16(r->data) && r->batch_stride >= 0 && r->token_stride >= 0 && r->head_stride >= 0 &&
         r->batch_stride % 8 == 0 && r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
}

RowView view(const loopkv_rows* r) {
  if (!r) return RowView{nullptr, 0, 0, 0};
  return RowView{static_cast<const __nv_bfloat16*>(r->data), r->batch_stride, r->token_stride, r->head_stride};
}

loopkv_status check_rotary(const loopkv_rotary* r, int head_dim) {
  if (!r) return LOOPKV_ERR_INVALID_ARG;
  if (r->cos_sin && (!aligned16(r->cos_sin) || r->max_positions <= 0 || r->rotary_dim <= 0 || r->rotary_dim % 16 != 0 ||
                     r->rotary_dim > head_dim))
    return LOOPKV_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return LOOPKV_ERR_INVALID_ARG;
  if ((r->q_weight && !aligned16(r->q_weight)) || (r->k_weight && !aligned16(r->k_weight))) return LOOPKV_ERR_INVALID_ARG;
  if ((r->q_weight || r->k_weight) && (!(r->eps >= 1e-30) || !isfinite(r->eps))) return LOOPKV_ERR_INVALID_ARG;
  return LOOPKV_OK;
}

RotaryView view(const loopkv_rotary* r) {
  if (!r) return RotaryView{nullptr, nullptr, nullptr, 0.0, 0, 0, 0};
  return RotaryView{r->cos_sin, static_cast<const __nv_bfloat16*>(r->q_weight),
                    static_cast<const __nv_bfloat16*>(r->k_weight), r->eps, r->max_positions, r->cos_sin ? r->rotary_dim : 0,
                    r->interleaved};
}

int64_t capacity(const loopkv_config* cfg) {
  return static_cast<int64_t>(cfg->max_blocks_per_seq) * cfg->block_size;
}

// Storage of a stored cell, or an error.
loopkv_status cell_storage(const loopkv_config* cfg, const loopkv_cells* cells, int cell, uint8_t** arena,
                           __nv_bfloat16** residual) {
  if (!cells || !cells->arena || !cells->key_residual) return LOOPKV_ERR_INVALID_ARG;
  *arena = static_cast<uint8_t*>(cells->arena[cell]);
  *residual = static_cast<__nv_bfloat16*>(cells->key_residual[cell]);
  if (!*arena || !aligned16(*arena)) return LOOPKV_ERR_INVALID_ARG;
  if (cfg->plan[cell] != LOOPKV_CELL_BF16 && (!*residual || !aligned16(*residual))) return LOOPKV_ERR_INVALID_ARG;
  return LOOPKV_OK;
}

loopkv_status result(cudaError_t e) { return e == cudaSuccess ? LOOPKV_OK : LOOPKV_ERR_CUDA; }

}  // namespace

extern "C" {

loopkv_status loopkv_norm_rope(const loopkv_rotary* rotary, int32_t head_dim, int32_t num_heads, int32_t num_kv_heads,
                               const loopkv_rows* q, const loopkv_rows* k, const int32_t* start_pos,
                               const int32_t* new_lens, int32_t batch, int32_t num_tokens, void* q_out, void* k_out,
                               int32_t* err_flag, void* stream) {
  if (head_dim != 64 && head_dim != 128) return LOOPKV_ERR_UNSUPPORTED;
  loopkv_status st = check_rotary(rotary, head_dim);
  if (st != LOOPKV_OK) return st;
  if (batch < 0 || num_tokens < 0 || (!q && !k)) return LOOPKV_ERR_INVALID_ARG;
  if ((q && num_heads <= 0) || (k && num_kv_heads <= 0)) return LOOPKV_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0) return LOOPKV_OK;
  if ((q && (!rows_ok(q) || !q_out || !aligned16(q_out))) || (k && (!rows_ok(k) || !k_out || !aligned16(k_out))))
    return LOOPKV_ERR_INVALID_ARG;
  if (!start_pos) return LOOPKV_ERR_INVALID_ARG;
  RotateParams p;
  p.rot = view(rotary);
  p.chunk = ChunkView{start_pos, new_lens, err_flag, batch, num_tokens,
                      rotary->cos_sin ? int64_t{rotary->max_positions} : INT64_MAX};
  p.q = view(q);
  p.k = view(k);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.H = q ? num_heads : 0;
  p.Hk = k ? num_kv_heads : 0;
  if (static_cast<double>(batch) * num_tokens * (static_cast<double>(p.H) + p.Hk) > static_cast<double>(kMaxRows))
    return LOOPKV_ERR_UNSUPPORTED;
  return result(launch_norm_rope(head_dim, p, static_cast<cudaStream_t>(stream)));
}

loopkv_status loopkv_rope_append(const loopkv_config* cfg, const loopkv_cells* cells, int32_t loop, int32_t layer,
                                 const loopkv_rotary* rotary, const loopkv_rows* q, const loopkv_rows* k_new,
                                 const loopkv_rows* v_new, const int32_t* block_table, const int32_t* start_pos,
                                 const int32_t* new_lens, int32_t batch, int32_t num_tokens, void* q_out,
                                 int32_t* err_flag, void* stream) {
  loopkv_status st = check_config(cfg);
  if (st != LOOPKV_OK) return st;
  int cell;
  if ((st = cell_index(cfg, loop, layer, &cell)) != LOOPKV_OK) return st;
  const int kind = cfg->plan[cell];
  if (kind == LOOPKV_CELL_REUSE) return LOOPKV_ERR_INVALID_ARG;  // reuse cells store nothing
  if (batch < 0 || batch > cfg->max_batch || num_tokens < 0) return LOOPKV_ERR_INVALID_ARG;
  if (!rotary && q) return LOOPKV_ERR_INVALID_ARG;
  if (rotary && (st = check_rotary(rotary, cfg->head_dim)) != LOOPKV_OK) return st;
  if (!cells || !cells->arena || !cells->key_residual) return LOOPKV_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0) return LOOPKV_OK;
  RopeAppendParams p;
  if ((st = cell_storage(cfg, cells, cell, &p.arena, &p.residual)) != LOOPKV_OK) return st;
  if (!k_new || !v_new || !rows_ok(k_new) || !rows_ok(v_new) || !block_table || !start_pos)
    return LOOPKV_ERR_INVALID_ARG;
  if (q && (!rows_ok(q) || !q_out || !aligned16(q_out))) return LOOPKV_ERR_INVALID_ARG;
  int64_t max_end = capacity(cfg);
  if (rotary && rotary->cos_sin && rotary->max_positions < max_end) max_end = rotary->max_positions;
  p.rows.rot = view(rotary);
  p.rows.chunk = ChunkView{start_pos, new_lens, err_flag, batch, num_tokens, max_end};
  p.rows.q = view(q);
  p.rows.k = view(static_cast<const loopkv_rows*>(nullptr));
  p.rows.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.rows.k_out = nullptr;
  p.rows.H = q ? cfg->num_heads : 0;
  p.rows.Hk = 0;
  p.k = view(k_new);
  p.v = view(v_new);
  p.block_table = block_table;
  p.Hkv = kv_heads(cfg);
  p.max_blocks = cfg->max_blocks_per_seq;
  p.num_blocks = cfg->num_blocks;
  // tokens of one call touch at most this many groups, wherever it starts
  p.key_blocks = static_cast<int>((int64_t{num_tokens} + 30) / 32 + 1);
  const int64_t cap_groups = (capacity(cfg) + 31) / 32;
  if (p.key_blocks > cap_groups) p.key_blocks = static_cast<int>(cap_groups);
  if (capacity(cfg) > kMaxRows || static_cast<double>(batch) * num_tokens * cfg->num_heads > static_cast<double>(kMaxRows) ||
      static_cast<double>(batch) * p.key_blocks * p.Hkv > static_cast<double>(kMaxRows / 2))
    return LOOPKV_ERR_UNSUPPORTED;
  return result(launch_rope_append(kind, cfg->head_dim, p, static_cast<cudaStream_t>(stream)));
}

loopkv_status loopkv_read_tokens(const loopkv_config* cfg, const loopkv_cells* cells, int32_t loop, int32_t layer,
                                 const int32_t* block_table, const int32_t* seq_lens, const int32_t* start_pos,
                                 int32_t batch, int32_t num_tokens, void* k_out, void* v_out, int32_t* err_flag,
                                 void* stream) {
  loopkv_status st = check_config(cfg);
  if (st != LOOPKV_OK) return st;
  int cell;
  if ((st = cell_index(cfg, loop, layer, &cell)) != LOOPKV_OK) return st;
  cell = source_cell(cfg, cell);
  if (batch < 0 || batch > cfg->max_batch || num_tokens < 0) return LOOPKV_ERR_INVALID_ARG;
  if (!cells || !cells->arena || !cells->key_residual) return LOOPKV_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0) return LOOPKV_OK;
  uint8_t* arena;
  __nv_bfloat16* residual;
  if ((st = cell_storage(cfg, cells, cell, &arena, &residual)) != LOOPKV_OK) return st;
  if (!block_table || !seq_lens || !start_pos || (!k_out && !v_out)) return LOOPKV_ERR_INVALID_ARG;
  if ((k_out && !aligned16(k_out)) || (v_out && !aligned16(v_out))) return LOOPKV_ERR_INVALID_ARG;
  ReadParams p;
  p.arena = arena;
  p.residual = residual;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.start_pos = start_pos;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.err = err_flag;
  p.B = batch;
  p.T = num_tokens;
  p.Hkv = kv_heads(cfg);
  p.max_blocks = cfg->max_blocks_per_seq;
  p.num_blocks = cfg->num_blocks;
  p.groups = static_cast<int>((int64_t{num_tokens} + 30) / 32 + 1);
  const int64_t cap_groups = (capacity(cfg) + 31) / 32;
  if (p.groups > cap_groups) p.groups = static_cast<int>(cap_groups);
  if (capacity(cfg) > kMaxRows || static_cast<double>(batch) * p.groups * p.Hkv > static_cast<double>(kMaxRows)) return LOOPKV_ERR_UNSUPPORTED;
  return result(launch_read(cfg->plan[cell], cfg->head_dim, p, static_cast<cudaStream_t>(stream)));
}

loopkv_status loopkv_chunk_attention(const loopkv_config* cfg, const loopkv_cells* cells, int32_t loop, int32_t layer,
                                     const loopkv_rows* q, const loopkv_rows* k_cur, const loopkv_rows* v_cur,
                                     const int32_t* block_table, const int32_t* start_pos, const int32_t* new_lens,
                                     int32_t batch, int32_t num_tokens, int32_t max_seq_len, float sm_scale, void* out,
                                     int32_t* err_flag, void* stream) {
  loopkv_status st = check_config(cfg);
  if (st != LOOPKV_OK) return st;
  int cell;
  if ((st = cell_index(cfg, loop, layer, &cell)) != LOOPKV_OK) return st;
  cell = source_cell(cfg, cell);
  if (batch < 0 || batch > cfg->max_batch || num_tokens < 0 || !isfinite(sm_scale * kLog2e)) return LOOPKV_ERR_INVALID_ARG;
  if (max_seq_len < 0 || max_seq_len > capacity(cfg)) return LOOPKV_ERR_INVALID_ARG;
  if ((k_cur == nullptr) != (v_cur == nullptr)) return LOOPKV_ERR_INVALID_ARG;  // both or neither
  if (!cells || !cells->arena || !cells->key_residual) return LOOPKV_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0) return LOOPKV_OK;
  uint8_t* arena;
  __nv_bfloat16* residual;
  if ((st = cell_storage(cfg, cells, cell, &arena, &residual)) != LOOPKV_OK) return st;
  if (!q || !rows_ok(q) || (k_cur && (!rows_ok(k_cur) || !rows_ok(v_cur)))) return LOOPKV_ERR_INVALID_ARG;
  if (!out || !aligned16(out) || !block_table || !start_pos) return LOOPKV_ERR_INVALID_ARG;
  if (capacity(cfg) > kMaxRows || static_cast<double>(batch) * num_tokens * cfg->num_heads > static_cast<double>(kMaxRows))
    return LOOPKV_ERR_UNSUPPORTED;
  ChunkAttnParams p;
  p.arena = arena;
  p.residual = residual;
  p.block_table = block_table;
  p.q = view(q);
  p.k_cur = view(k_cur);
  p.v_cur = view(v_cur);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.max_stored = max_seq_len ? max_seq_len : static_cast<int>(capacity(cfg));
  p.chunk = ChunkView{start_pos, new_lens, err_flag, batch, num_tokens, p.max_stored};
  const int group = cfg->num_heads / kv_heads(cfg);
  p.H = cfg->num_heads;
  p.Hkv = kv_heads(cfg);
  p.g_log2 = group == 8 ? 3 : group == 4 ? 2 : group == 2 ? 1 : 0;
  p.max_blocks = cfg->max_blocks_per_seq;
  p.num_blocks = cfg->num_blocks;
  const double scale = fabs(sm_scale * 1.4426950408889634);
  p.scale_mantissa = static_cast<float>(2.0 * frexp(scale, &p.scale_exp));
  p.scale_exp -= 1;
  if (scale == 0.0) p.scale_mantissa = 1.f, p.scale_exp = -10000;  // far below anything
  if (p.scale_mantissa == 2.f) p.scale_mantissa = 1.f, p.scale_exp += 1;  // rounded up
  p.scale_negative = sm_scale < 0.f;
  return result(launch_chunk_attention(cfg->plan[cell], cfg->head_dim, p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
