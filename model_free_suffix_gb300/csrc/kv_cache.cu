// kv_cache.cu -- writing keys and values into the paged 8-bit cache, and
// reading them back.
//
// A block is the tokens of one page for one head; x is held as q s with q in
// e4m3 and s = 2^e the smallest power of two that brings the block's largest
// magnitude to at most 448, e4m3's largest.  A power of two, because then
//   - x / s is exact, so the only rounding is the one to e4m3 (to nearest
//     even, relative error 2^-4 at most in its normal range, 2^-10 s below it);
//   - a block whose scale changes as tokens join it is re-encoded exactly, but
//     for magnitudes that become subnormal; a larger mantissa in the scale
//     would gain at most one bit of headroom and round every old entry again.
// The scale is made anew at each write from the entries that count (those
// before the write's first token, and the new ones): a rejected draft's values
// leave nothing behind.  Infinities do not count towards the scale and
// saturate, NaN is stored as 0; both set an error bit.
#include <math_constants.h>

#include "kv_internal.h"
#include "num_types.cuh"
#include "sgd_internal.h"

namespace sgd {
namespace {

constexpr int THREADS = 128;
constexpr int EXP_MIN = -48, EXP_MAX = 48;

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of the smallest power of two s with amax <= 448 s, by amax's
// bits: 448 = 1.75 * 2^8, so e = exponent - 8, one more above 1.75.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0);
  return min(max(e, EXP_MIN), EXP_MAX);
}

// Eight values of a token: a 16-byte load (two for floats) where alignment
// allows, else one by one.
template <typename T>
struct Eight {
  uint32_t w[8 * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T *p, int vec) {
    constexpr int NV = (int)sizeof(T) / 2;
    if (vec) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
      T x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[i];
      memcpy(w, x, sizeof(w));
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    T t[8];
    memcpy(t, w, sizeof(w));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(t[i]);
  }
};

__device__ __forceinline__ void decode8(uint2 r, float (&x)[8]) {
  const uint32_t w[2] = {r.x, r.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(w[i >> 1] >> (16 * (i & 1)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint2 r;
  r.x = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
  r.y = f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16;
  return r;
}

// One CTA takes the blocks whose first new token lies among `chunk` packed
// tokens, for one head, keys or values.  A block's entries stay in registers
// (PASSES groups of eight per thread) between the maximum and the encoding, so
// each is read once.
template <typename T, int PASSES>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(KvWriteArgs a) {
  __shared__ float sh[THREADS / 32];
  const int h = blockIdx.y, tid = threadIdx.x;
  const bool value = blockIdx.z != 0;
  const int D = a.c.dim, P = a.c.page;
  const int per = D / 8;                 // threads of a token
  const int slot_step = THREADS / per;   // tokens per pass
  const int sub = tid % per, slot_at = tid / per;
  const T *src = static_cast<const T *>(value ? a.v : a.k) +
                 (long long)h * (value ? a.v_head : a.k_head) + sub * 8;
  const long long src_token = value ? a.v_token : a.k_token;
  uint8_t *cache = value ? a.c.v : a.c.k;
  float *scales = value ? a.c.vs : a.c.ks;
  int i = blockIdx.x * a.chunk;
  const int end = min(i + a.chunk, a.r.N);
  int b = row_of_token(a.r.q_start, a.r.B, i);
  uint32_t bits = 0;
  while (b < a.r.B && i < end) {
    const int q0 = __ldg(a.r.q_start + b), q1 = min(__ldg(a.r.q_start + b + 1), a.r.N);
    if (i >= q1) {
      ++b;
      continue;
    }
    const int n = __ldg(a.r.seq_lens + b);
    const int pos = n - (q1 - q0) + (i - q0);
    if (q0 < 0 || q0 > i || n < q1 - q0) {
      bits |= SGD_KV_ERR_LENGTH;
      i = q1;
      ++b;
      continue;
    }
    const int slot0 = pos % P;
    const int stop = min(q1, i + P - slot0);
    const bool head = i == q0 || slot0 == 0;
    const int first = i;
    i = stop;
    if (!head) continue;  // the CTA of the block's first new token takes it
    const int block = pos / P;
    const int page = block < a.r.max_pages ? __ldg(a.r.table + (long long)b * a.r.max_pages + block) : -1;
    if (page < 0 || page >= a.c.num_pages) {
      bits |= SGD_KV_ERR_PAGE;
      continue;
    }
    const int cnt = stop - first, used = slot0 + cnt;
    uint8_t *base = cache + ((long long)page * a.c.heads + h) * P * D + sub * 8;
    float *scale = scales + (long long)page * a.c.heads + h;
    const float old = slot0 > 0 ? *scale : 1.f;
    Eight<T> fresh[PASSES];
    uint2 was[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int s = p * slot_step + slot_at;
      if (s < slot0)
        was[p] = *reinterpret_cast<const uint2 *>(base + s * D);
      else if (s < used)
        fresh[p].load(src + (long long)(first + s - slot0) * src_token, a.vec);
    }
    float amax = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int s = p * slot_step + slot_at;
      float x[8];
      if (s < slot0) {
        decode8(was[p], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]) * old);  // (a NaN is dropped)
      } else if (s < used) {
        fresh[p].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float m = fabsf(x[e]);
          if (!(m < CUDART_INF_F))
            bits |= SGD_KV_ERR_NONFINITE;
          else
            amax = fmaxf(amax, m);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o));
    __syncthreads();  // (the previous block's maxima are read)
    if ((tid & 31) == 0) sh[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, sh[w]);
    const int e = scale_exp(amax);
    const float s_new = pow2(e), inv = pow2(-e);
    const bool redo = slot0 > 0 && s_new != old;
    if (tid == 0) *scale = s_new;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int s = p * slot_step + slot_at;
      float x[8];
      if (s < slot0) {
        if (!redo) continue;
        decode8(was[p], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= old;
      } else if (s < used) {
        fresh[p].get(x);
      } else {
        continue;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] == x[j] ? x[j] : 0.f;
      *reinterpret_cast<uint2 *>(base + s * D) = encode8(x, inv);
    }
  }
  if (bits) atomicOr(a.err, bits);
}

// A thread takes 16 bytes of one token and head at a time and writes 16
// values; bound by the bytes written.  Tokens of a page and head are
// contiguous in the cache, heads of a token in the output: a CTA takes 64
// tokens of one head, so both sides move whole 32-byte sectors.
constexpr int READ_TOKENS = 64;
template <typename T>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(KvReadArgs a) {
  const int h = blockIdx.y, tid = threadIdx.x, D = a.c.dim, P = a.c.page;
  const bool value = blockIdx.z != 0;
  const uint8_t *cache = value ? a.c.v : a.c.k;
  const float *scales = value ? a.c.vs : a.c.ks;
  T *out = static_cast<T *>(value ? a.v : a.k);
  const int i0 = blockIdx.x * READ_TOKENS;
  int b = row_of_token(a.out_start, a.B, i0);
  const int per = D / 16, step = THREADS / per, sub = tid % per;
  uint32_t bits = 0;
#pragma unroll 4
  for (int t = tid / per; t < READ_TOKENS; t += step) {
    const int i = i0 + t;
    if (i >= a.N) break;
    while (b < a.B && i >= __ldg(a.out_start + b + 1)) ++b;
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
    if (b < a.B) {
      const int pos = __ldg(a.from + b) + i - __ldg(a.out_start + b);
      const int block = pos / P;
      const int page = pos >= 0 && block < a.max_pages ? __ldg(a.table + (long long)b * a.max_pages + block) : -1;
      if (page >= 0 && page < a.c.num_pages) {
        const long long at = (long long)page * a.c.heads + h;
        const uint4 raw = *reinterpret_cast<const uint4 *>(cache + (at * P + pos % P) * D + sub * 16);
        const float s = scales[at];
        float y[8];
        decode8(make_uint2(raw.x, raw.y), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e] * s;
        decode8(make_uint2(raw.z, raw.w), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 + e] = y[e] * s;
      } else {
        bits |= SGD_KV_ERR_PAGE;  // (zeros are returned for it)
      }
    } else {
      bits |= SGD_KV_ERR_LENGTH;
    }
    T *o = out + ((long long)i * a.c.heads + h) * D + sub * 16;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        reinterpret_cast<float4 *>(o)[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        reinterpret_cast<uint4 *>(o)[e] =
            make_uint4(pack2<T>(x[8 * e], x[8 * e + 1]), pack2<T>(x[8 * e + 2], x[8 * e + 3]),
                       pack2<T>(x[8 * e + 4], x[8 * e + 5]), pack2<T>(x[8 * e + 6], x[8 * e + 7]));
    }
  }
  if (bits) atomicOr(a.err, bits);
}

template <typename T>
cudaError_t write(const KvWriteArgs &a, cudaStream_t st) {
  const dim3 grid((a.r.N + a.chunk - 1) / a.chunk, a.c.heads, 2);
  switch (a.c.page * a.c.dim / (8 * THREADS)) {
    case 1: kv_write_kernel<T, 1><<<grid, THREADS, 0, st>>>(a); break;
    case 2: kv_write_kernel<T, 2><<<grid, THREADS, 0, st>>>(a); break;
    case 4: kv_write_kernel<T, 4><<<grid, THREADS, 0, st>>>(a); break;
    case 8: kv_write_kernel<T, 8><<<grid, THREADS, 0, st>>>(a); break;
    case 16: kv_write_kernel<T, 16><<<grid, THREADS, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write(KvWriteArgs a, int dtype, cudaStream_t st) {
  // Few tokens: one per CTA, so that every block has its own; many: up to a
  // page per CTA, so that few CTAs find that their tokens begin no block.
  const long long want = 152 * 16;
  a.chunk = 1;
  while (a.chunk < a.c.page && (long long)a.r.N * a.c.heads * 2 / (2 * a.chunk) >= want) a.chunk *= 2;
  if (dtype == SGD_F32) return write<float>(a, st);
  if (dtype == SGD_F16) return write<__half>(a, st);
  return write<__nv_bfloat16>(a, st);
}

cudaError_t launch_kv_read(KvReadArgs a, int dtype, cudaStream_t st) {
  const dim3 grid((a.N + READ_TOKENS - 1) / READ_TOKENS, a.c.heads, 2);
  if (dtype == SGD_F32)
    kv_read_kernel<float><<<grid, THREADS, 0, st>>>(a);
  else if (dtype == SGD_F16)
    kv_read_kernel<__half><<<grid, THREADS, 0, st>>>(a);
  else
    kv_read_kernel<__nv_bfloat16><<<grid, THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sgd
