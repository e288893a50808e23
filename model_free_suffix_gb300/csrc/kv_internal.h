// kv_internal.h -- the paged 8-bit cache as its kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sgd.h"

namespace sgd {

// A cache of one layer: keys and values [num_pages][heads][page][dim] e4m3,
// scales [num_pages][heads].  One (page, head) block is page * dim contiguous
// bytes.  Value = byte as e4m3 * scale; a scale is 2^e, e in [-48, 48].
struct KvView {
  uint8_t *k, *v;
  float *ks, *vs;
  int num_pages, heads, page, dim;
  int page_bits;  // log2 of page
};

// Which tokens a call means: row b's tokens are packed q_start[b] ..
// q_start[b + 1] of the call's N, the last ones of its seq_lens[b] tokens.
struct KvRows {
  const int32_t *table;  // [B, max_pages]
  const int32_t *q_start, *seq_lens;
  int B, N, max_pages;
};

struct KvWriteArgs {
  KvView c;
  KvRows r;
  const void *k, *v;
  long long k_token, k_head, v_token, v_head;  // strides in elements
  int vec;                                     // 16-byte loads allowed
  int team;                                    // warps of a block (chosen at the launch)
  uint32_t *err;
};

struct KvReadArgs {
  KvView c;
  const int32_t *table, *from, *out_start;
  int B, N, max_pages;
  void *k, *v;  // [N, heads, dim]
  uint32_t *err;
};

struct KvAttendArgs {
  KvView c;
  KvRows r;
  const void *q;
  long long q_token, q_head;
  int q_vec;  // 16-byte loads allowed
  void *out;  // [N, q_heads, dim]
  int q_heads, group;  // group = q_heads / heads
  int max_q;
  float scale;
  int window, sinks;
  int sms;              // SMs of the device
  unsigned char *work;  // kv_attend_workspace bytes, 0 at creation
  uint32_t *err;
};

cudaError_t launch_kv_write(const KvWriteArgs &a, int dtype, cudaStream_t st);
cudaError_t launch_kv_read(const KvReadArgs &a, int dtype, cudaStream_t st);
size_t kv_attend_workspace();
cudaError_t kv_attend_set_limits();
cudaError_t launch_kv_attend(KvAttendArgs a, int dtype, cudaStream_t st, int *launches);

#ifdef __CUDACC__
// Two e4m3 bytes (the low 16 bits) as two f16: exact, every e4m3 value is one.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(two));
  return r;
}
// Four: the low two, the high two.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t &lo, uint32_t &hi) {
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
// Two floats as e4m3, to nearest even, saturated (NaN stays NaN).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{.reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %1, %2; cvt.u32.u16 %0, t;}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
#endif

}  // namespace sgd
