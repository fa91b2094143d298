// What the units of the 8-bit cache share: its parameters, conversions and the checks of a
// sequence's row range and length.
#pragma once

#include <cuda_fp16.h>

#include <climits>

#include "kernels.cuh"

namespace lilicorr {

// The cache as the kernels take it.
struct Kv8 {
  uint8_t *k, *v;   // [n_pages, heads, page, D]
  float *ks, *vs;   // [n_pages, heads]
  int64_t n_pages;
  int heads, page;
};

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
// Two floats to e4m3 codes (a in the low byte), to nearest even, magnitudes above 448 to 448.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// One sequence's rows, or n = 0 where its row range or length is out of range (recorded).
struct SeqRange {
  int64_t q0;  // first row
  int n, len;  // new rows; cached tokens, the new ones among them
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* __restrict__ q_start,
                                              const int32_t* __restrict__ kv_len, int64_t b,
                                              int64_t total, int max_new, int64_t capacity,
                                              uint32_t* err) {
  SeqRange r;
  const int a = __ldg(q_start + b), e = __ldg(q_start + b + 1);
  r.q0 = a;
  r.n = e - a;
  r.len = __ldg(kv_len + b);
  if (a < 0 || e < a || e > total || r.n > max_new || r.len < 0 || r.len > capacity) {
    atomicOr(err, ERR_KV8_LENGTH);
    r.n = 0;
    r.len = 0;
  }
  return r;
}

// ---- host
// Null where the cache's description is in order, else what is wrong with it.
const char* kv8_cache_error(const lilicorr_kv8_cache* c);
struct Kv8Attention {
  Kv8 c;
  const __nv_bfloat16* q;
  int64_t q_tok, q_head;  // elements
  int64_t total;
  int q_heads, group, D;
  const int32_t *q_start, *kv_len, *table;
  int64_t batch, table_stride;
  int cols, max_new;
  float scale;
  __nv_bfloat16* out;
  float* lse;
  void* workspace;
};
size_t kv8_attention_workspace(int max_new, int group, int D);
cudaError_t kv8_attention_launch(const Kv8Attention& a, cudaStream_t stream);
cudaError_t kv8_attention_read_device_error(uint32_t* code);

}  // namespace lilicorr
