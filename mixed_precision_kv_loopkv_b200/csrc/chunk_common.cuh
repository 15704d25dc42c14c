// Device helpers shared by the prompt-side kernels.
#pragma once

#include "chunk.h"
#include "device_common.cuh"

namespace loopkv {

// Sequence b's part of a chunk: len new tokens from position start on.
struct SeqChunk {
  int start, len;
};

// len = 0 where there is nothing to do: a skipped sequence, no tokens, or
// lengths that do not fit (then *bad is set and, if asked, the error flagged).
__device__ __forceinline__ SeqChunk seq_chunk(const ChunkView& c, int b, bool report, bool* bad = nullptr) {
  SeqChunk s;
  s.start = c.start_pos[b];
  s.len = c.new_lens ? c.new_lens[b] : c.T;
  if (bad) *bad = false;
  if (s.start < 0) {
    s.len = 0;
  } else if (s.len < 0 || s.len > c.T || (s.len > 0 && static_cast<int64_t>(s.start) + s.len > c.max_end)) {
    if (report) flag_error(c.err, LOOPKV_DEVERR_SEQ_LEN);
    if (bad) *bad = true;
    s.len = 0;
  }
  return s;
}

__device__ __forceinline__ const __nv_bfloat16* row_at(const RowView& v, int b, int t, int h) {
  return v.p + b * v.sb + t * v.st + h * v.sh;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(u[i]);
    x[2 * i + 1] = bf16_hi(u[i]);
  }
}

// Two floats as bf16, to nearest even, in one conversion (that of a single one
// runs at an eighth of its rate).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Minimum and maximum that are NaN where an operand is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 numbers side by side, each operation rounded as its plain form.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
}  // namespace loopkv
