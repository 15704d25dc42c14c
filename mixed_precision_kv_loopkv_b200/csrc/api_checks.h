// Argument checks shared by the C-ABI layers (host, internal).
#pragma once

#include <stdint.h>

#include "loopkv.h"

namespace loopkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// KV heads of a config (0 in num_kv_heads: one per query head).
inline int kv_heads(const loopkv_config* cfg) { return cfg->num_kv_heads ? cfg->num_kv_heads : cfg->num_heads; }

inline bool stored_kind(int k) {
  return k == LOOPKV_CELL_Q4 || k == LOOPKV_CELL_Q2 || k == LOOPKV_CELL_BF16;
}

inline loopkv_status check_config(const loopkv_config* cfg) {
  if (!cfg || !cfg->plan) return LOOPKV_ERR_INVALID_ARG;
  if (cfg->num_loops <= 0 || cfg->num_layers <= 0 || cfg->num_heads <= 0 || cfg->num_blocks < 0 ||
      cfg->max_batch < 0 || cfg->max_blocks_per_seq <= 0)
    return LOOPKV_ERR_INVALID_ARG;
  if (cfg->num_kv_heads < 0 || cfg->num_heads % kv_heads(cfg) != 0) return LOOPKV_ERR_INVALID_ARG;
  const int group = cfg->num_heads / kv_heads(cfg);  // query heads per KV head: 1, 2, 4 or 8
  if (group != 1 && group != 2 && group != 4 && group != 8) return LOOPKV_ERR_UNSUPPORTED;
  if (cfg->head_dim != 64 && cfg->head_dim != 128) return LOOPKV_ERR_UNSUPPORTED;
  if (cfg->block_size != 16) return LOOPKV_ERR_UNSUPPORTED;
  if ((cfg->flags & LOOPKV_FLAG_SELECT_BLOCK) && (cfg->flags & LOOPKV_FLAG_SELECT_GROUP))
    return LOOPKV_ERR_INVALID_ARG;
  const int s = cfg->decode_splits;
  if (s != 0 && s != 1 && s != 2 && s != 4 && s != 8) return LOOPKV_ERR_INVALID_ARG;
  const int L = cfg->num_loops, N = cfg->num_layers;
  for (int c = 0; c < L * N; ++c) {
    const int k = cfg->plan[c];
    if (k != LOOPKV_CELL_REUSE && !stored_kind(k)) return LOOPKV_ERR_BAD_PLAN;
    if (k == LOOPKV_CELL_REUSE && c / N == L - 1) return LOOPKV_ERR_BAD_PLAN;
  }
  return LOOPKV_OK;
}

inline loopkv_status cell_index(const loopkv_config* cfg, int loop, int layer, int* cell) {
  if (loop < 0 || loop >= cfg->num_loops || layer < 0 || layer >= cfg->num_layers)
    return LOOPKV_ERR_INVALID_ARG;
  *cell = loop * cfg->num_layers + layer;
  return LOOPKV_OK;
}

// A reuse cell reads the final loop's cell of the same layer.
inline int source_cell(const loopkv_config* cfg, int cell) {
  return cfg->plan[cell] == LOOPKV_CELL_REUSE ? (cfg->num_loops - 1) * cfg->num_layers + cell % cfg->num_layers : cell;
}

}  // namespace loopkv
