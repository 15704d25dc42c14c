/*
 * loopkv_chunk.h -- C ABI of the LoopKV prompt side on B200 (sm_100a): a chunk
 * of new tokens (a prompt, a part of one, a few drafted tokens) through the
 * (loop, layer) cells that loopkv.h defines.
 *
 * For every cell of the looped model, in (loop, layer) order:
 *   a stored cell   loopkv_rope_append (norms, position rotation and store of
 *                   the chunk's keys and values, rotated queries), then
 *                   loopkv_chunk_attention over what is stored;
 *   a reuse cell    loopkv_norm_rope (its own keys are stored nowhere), then
 *                   loopkv_chunk_attention over the final loop's tokens of the
 *                   earlier chunks and the chunk's own exact rows.
 * loopkv_read_tokens gives a cell's tokens back as values.
 *
 * The conventions of loopkv.h hold (caller-owned memory, no allocation, no
 * synchronisation, the caller's stream, argument errors before any launch,
 * device faults as LOOPKV_DEVERR_* bits), with these additions:
 *   - a chunk is [batch][num_tokens] rows; sequence b has new_lens[b] of them
 *     (new_lens NULL: num_tokens for every sequence), at positions
 *     start_pos[b] .. start_pos[b] + new_lens[b] - 1.  The rows behind them are
 *     neither read nor written;
 *   - start_pos[b] < 0 skips the sequence, new_lens[b] = 0 has nothing to do;
 *   - a sequence with new_lens[b] outside [0, num_tokens], or whose tokens do
 *     not fit the block table, max_seq_len or the rotation table, sets
 *     LOOPKV_DEVERR_SEQ_LEN and is skipped;
 *   - input rows may be strided (views of one fused projection), see loopkv_rows;
 *     outputs are contiguous.  An output must not overlap an input, except that
 *     q_out (k_out) may be q (k) itself where that is contiguous;
 *   - a cell can go back (be appended to, or attended over, at fewer tokens than
 *     it holds) to any place if it is bf16, and not below the last multiple of 32
 *     tokens if it is 4-bit or 2-bit: behind that lie completed key groups, whose
 *     exact keys are gone.  Drafted tokens that may be rejected are therefore
 *     not appended but given as k_cur, v_cur, and the accepted ones appended
 *     afterwards;
 *   - the launches are ordinary ones, in stream order (LOOPKV_FLAG_PDL changes
 *     nothing here).  A loopkv_decode_attention with that flag reads old cache
 *     blocks before it waits, so it must not directly follow an append of
 *     several tokens: see LOOPKV_FLAG_PDL.
 */
#ifndef LOOPKV_CHUNK_H
#define LOOPKV_CHUNK_H

#include "loopkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bf16 rows [batch][num_tokens][heads][D] with strides in elements; the last
 * dimension is contiguous.  data 16-byte aligned, strides >= 0 and multiples
 * of 8 (a stride may be 0). */
typedef struct {
  const void* data;
  int64_t batch_stride, token_stride, head_stride;
} loopkv_rows;

/*
 * Norms and position rotation of queries and keys.  For a head's row x at
 * position p, with every fp32 step one correctly rounded operation:
 *   a = x                                   without a weight, else
 *   a = (x * r) * w,   r = fp32(1 / sqrt(mean(x^2) + eps)), mean in 64 bits
 *   y1 = a1 * cos[p] - a2 * sin[p],  y2 = a2 * cos[p] + a1 * sin[p]
 *   rounded once to bf16
 * over the pairs (a1, a2) = (a[i], a[i + rotary_dim / 2]) or, interleaved,
 * (a[2 i], a[2 i + 1]); channels from rotary_dim on are not rotated.
 */
typedef struct {
  const float* cos_sin;     /* device fp32 [max_positions][rotary_dim]: the cosines, then the sines,
                               of a position's rotary_dim / 2 angles; NULL: no rotation */
  int32_t max_positions;
  int32_t rotary_dim;       /* a multiple of 16, at most head_dim */
  int32_t interleaved;      /* 0: pairs half of rotary_dim apart, 1: neighbours */
  const void* q_weight;     /* device bf16 [head_dim], or NULL: queries not normed */
  const void* k_weight;     /* the same for keys */
  double eps;               /* at least 1e-30 where there is a weight (a row of zeros has a norm then) */
} loopkv_rotary;

/*
 * Norms and rotation of a chunk's queries and keys in one pass.
 *   q, k         : rows of num_heads and num_kv_heads heads; either may be NULL
 *                  (then its output is ignored)
 *   start_pos    : device int32 [batch];  new_lens: optional device int32 [batch]
 *   q_out, k_out : device bf16 [batch][num_tokens][heads][D]
 * Errors: INVALID_ARG for null or misaligned pointers, bad strides, a bad
 * rotary (rotary_dim, max_positions <= 0, eps below 1e-30 or not finite), negative sizes;
 * UNSUPPORTED for head_dim other than 64 and 128 or 2^31 rows or more.
 */
LOOPKV_API loopkv_status loopkv_norm_rope(const loopkv_rotary* rotary, int32_t head_dim, int32_t num_heads,
                                          int32_t num_kv_heads, const loopkv_rows* q, const loopkv_rows* k,
                                          const int32_t* start_pos, const int32_t* new_lens, int32_t batch,
                                          int32_t num_tokens, void* q_out, void* k_out, int32_t* err_flag,
                                          void* stream);

/*
 * Append a chunk to the stored cell (loop, layer), norms and rotation on the
 * way: the cell then holds the bytes that loopkv_norm_rope of the keys followed
 * by loopkv_quantize_append of them and the values would have stored, for
 * ragged chunks in one launch.  The queries (optional) are normed, rotated and
 * written to q_out in the same launch.
 *   rotary       : NULL stores the keys as they are, any NaN as 0x7FFF (q must
 *                  then be NULL)
 *   q            : optional rows of num_heads heads, q_out as for loopkv_norm_rope
 *   k_new, v_new : rows of num_kv_heads heads
 * Errors: as loopkv_quantize_append and loopkv_norm_rope.
 */
LOOPKV_API loopkv_status loopkv_rope_append(const loopkv_config* cfg, const loopkv_cells* cells, int32_t loop,
                                            int32_t layer, const loopkv_rotary* rotary, const loopkv_rows* q,
                                            const loopkv_rows* k_new, const loopkv_rows* v_new,
                                            const int32_t* block_table, const int32_t* start_pos,
                                            const int32_t* new_lens, int32_t batch, int32_t num_tokens, void* q_out,
                                            int32_t* err_flag, void* stream);

/*
 * Tokens start_pos[b] .. start_pos[b] + num_tokens - 1 of a cell that holds
 * seq_lens[b] tokens, as the values that they stand for: min + scale * code in
 * fp32, rounded to bf16; keys of the unfinished group and bf16 cells exactly.
 * A reuse cell reads the final loop's cell of its layer.  Rows of tokens from
 * seq_lens[b] on are left as they are; a bad block leaves its tokens' rows as
 * they are and sets LOOPKV_DEVERR_BLOCK_ID.
 *   seq_lens     : device int32 [batch]
 *   k_out, v_out : device bf16 [batch][num_tokens][Hkv][D]; either may be NULL
 */
LOOPKV_API loopkv_status loopkv_read_tokens(const loopkv_config* cfg, const loopkv_cells* cells, int32_t loop,
                                            int32_t layer, const int32_t* block_table, const int32_t* seq_lens,
                                            const int32_t* start_pos, int32_t batch, int32_t num_tokens, void* k_out,
                                            void* v_out, int32_t* err_flag, void* stream);

/*
 * Attention of a chunk of new tokens over the paged cell (loop, layer); a
 * reuse cell reads the final loop's cell of its layer.  Row i of sequence b is
 * the query at position start_pos[b] + i:
 *   k_cur, v_cur NULL : it attends the stored tokens 0 .. start_pos[b] + i (the
 *                       chunk itself is in the cell, which holds start_pos[b] +
 *                       new_lens[b] tokens);
 *   k_cur, v_cur given: it attends the stored tokens 0 .. start_pos[b] - 1 (the
 *                       cell holds start_pos[b]) and the chunk's rows 0 .. i of
 *                       k_cur, v_cur, exactly.
 * Stored tokens are dequantised at the cell's full precision: a chunk's queries
 * share one read of the low value plane, so the threshold tau of single-token
 * decoding has nothing to save here (as tau = 0 there).  Softmax weights and
 * dequantised rows enter the tensor cores in fp16 (11 bits) under powers of two
 * that follow the data, a block of 16 (or group of 32) tokens at a time; sums
 * and statistics are fp32.  Entries less than 2^-8 of the largest finite one of
 * their block, whether the row sees that or not, lose bits by the same factor
 * (exact keys, and bf16 cells: 2^-22); between blocks a row's precision follows
 * what it sees and weighs.  A row with a logit of NaN or +infinity, or none above
 * -infinity, is NaN; a value that is not finite shows in its channel of the rows
 * that see it, and in no others.
 *   q            : rows of num_heads heads (queries already rotated)
 *   k_cur, v_cur : optional rows of num_kv_heads heads (both or neither)
 *   max_seq_len  : host upper bound of the stored tokens; 0: the block table's
 *                  capacity.  It sizes the split of the context: results under
 *                  different bounds may differ in their last bits
 *   out          : device bf16 [batch][num_tokens][num_heads][D]; rows of a
 *                  sequence skipped by start_pos[b] < 0 or by a device fault (any
 *                  bad block of it) are zeros up to new_lens[b] (nothing where
 *                  that is out of range)
 * Errors: INVALID_ARG as for loopkv_decode_attention and loopkv_rows; BAD_PLAN;
 * UNSUPPORTED for 2^31 rows or more.
 */
LOOPKV_API loopkv_status loopkv_chunk_attention(const loopkv_config* cfg, const loopkv_cells* cells, int32_t loop,
                                                int32_t layer, const loopkv_rows* q, const loopkv_rows* k_cur,
                                                const loopkv_rows* v_cur, const int32_t* block_table,
                                                const int32_t* start_pos, const int32_t* new_lens, int32_t batch,
                                                int32_t num_tokens, int32_t max_seq_len, float sm_scale, void* out,
                                                int32_t* err_flag, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOPKV_CHUNK_H */
