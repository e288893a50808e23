// kv_attend.cuh -- the attention's references, and where parts of units lie.
#pragma once

#include <cuda.h>
#include <math_constants.h>

#include "async_copy.cuh"
#include "kv_internal.h"
#include "kv_sched.cuh"
#include "num_types.cuh"

namespace sgd {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int MAX_CTAS = 152 * 4;  // what the workspace is laid out for

// Token j adds 2^z_j, z its scaled product in units of log 2, to l and
// 2^(z_j + log2 V_j) q_j to o, V_j the scale of its block of values and q_j what
// is stored.  Both are kept relative to one reference per row, the running
// maximum of z + log2 V (not of z: f16 probabilities have 11 bits down to 2^-14,
// and below that an absolute error, which has to be small against the largest
// share in o; a block of much larger values than the one that the softmax
// favours would show it otherwise).  Scales reach from 2^-48 to 2^48, so l stays
// far within 32 bits.  The reference moves, and o and l are scaled, only once
// the maximum has grown by 2^LAZY; probabilities are taken 2^LIFT times as large
// (the quotient is the same), so that they use f16's range up to its end: 2^15.99
// is 65082 of 65504.  (A larger LAZY saves little: at 4, a row that has seen a
// few tiles of common logits meets such a maximum once in hundreds of tiles.)
constexpr float LAZY = 4.f;
constexpr float LIFT = 11.99f;

// log2 of a block's scale (a power of two when sgd_kv_write made it), and its inverse
__device__ __forceinline__ float log2_scale(float s) { return __log2f(s); }
__device__ __forceinline__ float inverse_scale(float s) { return __fdividef(1.f, s); }

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Where the parts of split units lie in the workspace, after the counters (one
// per CTA): [M][D] sums, [M] maxima, [M] sums of probabilities.
template <int M, int D>
__device__ __forceinline__ float *part_of(const KvAttendArgs &a, int slot) {
  return reinterpret_cast<float *>(a.work + MAX_CTAS * 8) + (long long)slot * (M * (D + 2));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The queries of a unit's rows, R of them (beyond nrows: 0), by all warps, as
// the matrix instructions take them: [row / 16][D / 16 steps][lane] 16 bytes.
// f: what a product with a row counts in units of log 2.
template <typename T, int D, int R, int WARPS, class Walk>
__device__ __forceinline__ void kv_queries(const KvAttendArgs &a, const Walk &w, uint32_t q_at, float *s_f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool mine = lane * 4 < D;
  constexpr int BATCH = 4;  // rows of a warp with their loads in flight
  constexpr int DPT = D / 4;  // dims of a lane
  const int qc = lane * 4 / DPT, s = lane * 4 % DPT / 4;
#pragma unroll 1
  for (int r0 = warp; r0 < R && r0 < (w.nrows + 15) / 16 * 16; r0 += WARPS * BATCH) {
    uint2 raw[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int r = r0 + i * WARPS;
      raw[i] = make_uint2(0, 0);
      if (r < w.nrows && mine) {
        const T *q = static_cast<const T *>(a.q) + w.token(r) * a.q_token + w.q_head(r) * a.q_head + lane * 4;
        if (a.q_vec) {
          raw[i] = *reinterpret_cast<const uint2 *>(q);
        } else {
          const unsigned short *s = reinterpret_cast<const unsigned short *>(q);
          raw[i] = make_uint2(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int r = r0 + i * WARPS;
      const uint32_t to = q_at + (((r / 16) * (D / 16) + s) * 32 + (r % 8) * 4 + qc) * 16 + (r % 16) / 8 * 4;
      uint32_t pair[2] = {0, 0};
      if (r < w.nrows) {
        T in[4];
        *reinterpret_cast<uint2 *>(in) = raw[i];
        float x[4], top = 0.f;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = to_f32(in[e]);
          top = fmaxf(top, fabsf(x[e]));
          bad = bad || !(fabsf(x[e]) < CUDART_INF_F);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
        const bool poison = __any_sync(FULL, bad);  // (a bad element makes its row NaN)
        const int e2 = max((int)(__float_as_uint(top) >> 23) - 127, -100);
        const float inv = poison ? CUDART_NAN_F : pow2(-min(e2, 126));
        if (lane == 0) s_f[r] = a.scale * LOG2E * pow2(min(e2, 126));
        pair[0] = pack2<__half>(x[0] * inv, x[1] * inv);
        pair[1] = pack2<__half>(x[2] * inv, x[3] * inv);
      } else if (lane == 0) {
        s_f[r] = 0.f;
      }
      if (mine) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(pair[0]) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + 8), "r"(pair[1]) : "memory");
      }
    }
  }
}

// The parts of a unit that cuts go through, by all threads of the CTAs that hold
// them, once each has stored its part: the last joins them.  JOIN_ROWS rows at a
// time: the parts' weights 2^(m - max) first, then the sums with the loads of
// several parts in flight.  scratch: kv_join_floats() of shared memory.
constexpr int JOIN_ROWS = 8;
constexpr int kv_join_floats() { return MAX_CTAS * JOIN_ROWS * 2 + JOIN_ROWS; }

template <typename T, class K, int D, int THREADS>
__device__ __forceinline__ void kv_join(const KvAttendArgs &a, const KvShare &share, const KvWalk<K> &w, float *scratch,
                                        int *s_last) {
  constexpr int M = K::M, R = JOIN_ROWS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g0 = share.cta_of(w.u_begin), g1 = share.cta_of(w.u_end - 1);
  unsigned *count = reinterpret_cast<unsigned *>(a.work) + g0;
  __threadfence();
  __syncthreads();
  if (tid == 0) *s_last = atomicAdd(count, 1) == (unsigned)(g1 - g0);
  __syncthreads();
  if (!*s_last) return;
  __threadfence();
  if (tid == 0) *count = 0;
  const int parts = g1 - g0 + 1;
  float *w_inv = scratch, *w_m = scratch + R, *w_l = w_m + parts * R;
  auto slot = [&](int p) { return part_of<M, D>(a, 2 * (g0 + p) + (p == 0 ? 1 : 0)); };
#pragma unroll 1
  for (int r0 = 0; r0 < w.nrows; r0 += R) {
    const int rows = min(R, w.nrows - r0);
#pragma unroll 1
    for (int i = tid; i < parts * R; i += THREADS) {
      const float *from = slot(i / R) + M * D + r0 + i % R;
      const bool on = i % R < rows;
      w_m[i] = on ? __ldcg(from) : -CUDART_INF_F;
      w_l[i] = on ? __ldcg(from + M) : 0.f;
    }
    __syncthreads();
#pragma unroll 1
    for (int r = warp; r < rows; r += THREADS / 32) {
      float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll 1
      for (int p = lane; p < parts; p += 32) top = fmaxf(top, w_m[p * R + r]);
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
      const float base = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll 1
      for (int p = lane; p < parts; p += 32) {
        const float k = ex2_approx(w_m[p * R + r] - base);
        w_m[p * R + r] = k;
        if (w_l[p * R + r] != 0.f) sum += w_l[p * R + r] * k;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
      if (lane == 0) w_inv[r] = sum == 0.f ? 0.f : 1.f / sum;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < rows * (D / 4); i += THREADS) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int p = 0; p < parts; ++p) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(slot(p) + (r0 + r) * D + d));
        const float k = w_m[p * R + r];
        x.x += v.x * k;
        x.y += v.y * k;
        x.z += v.z * k;
        x.w += v.w * k;
      }
      const float inv = w_inv[r];
      T *dst = static_cast<T *>(a.out) + ((long long)w.token(r0 + r) * a.q_heads + w.q_head(r0 + r)) * D + d;
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(x.x * inv, x.y * inv), pack2<T>(x.z * inv, x.w * inv));
    }
    __syncthreads();
  }
}

// ---- host --------------------------------------------------------------------

// Keys or values as lines of 128 bytes (one token, or two of 64 bytes), in
// boxes of `tokens`, with the 128-byte swizzle.
bool kv_make_map(CUtensorMap *map, const KvView &c, void *base, int tokens);

// 16-bit tensors [N, heads, dim] of the caller, in boxes of `tokens` x 64 elements
// of one head, with the 128-byte swizzle.  Strides in elements, multiples of 8.
bool kv_make_token_map(CUtensorMap *map, const void *base, int dim, int heads, int N, long long head_stride,
                       long long token_stride, int tokens);

// Attention for units of more than 16 rows, up to KV_MANY_ROWS.
constexpr int KV_MANY_ROWS = 32;
cudaError_t attend_many_limits();
cudaError_t launch_attend_many(const KvAttendArgs &a, int dtype, cudaStream_t st);

}  // namespace sgd
