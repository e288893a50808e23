// kv_prompt.cu -- attention of whole prompts, and of chunks over the paged cache.
#include <math_constants.h>

#include "async_copy.cuh"
#include "kv_internal.h"
#include "num_types.cuh"
#include "sgd_internal.h"

namespace sgd {
namespace {

constexpr float LOG2E = 1.4426950408889634f;

// One warp per (new token, query head), a running maximum and sum: the plainest
// form, one key at a time.
template <typename T, int D>
__global__ void __launch_bounds__(128) new_kernel(KvNewArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.r.B; b += 128) {
      const int q0 = __ldg(a.r.q_start + b), q1 = __ldg(a.r.q_start + b + 1);
      if (q0 < 0 || q1 > a.r.N || q1 < q0) atomicOr(a.err, SGD_KV_ERR_LENGTH);
    }
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(unit / a.q_heads), hq = (int)(unit % a.q_heads), h = hq / a.group;
  if (t >= a.r.N || t >= __ldg(a.r.q_start + a.r.B)) return;
  int lo = 0, hi = a.r.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.r.q_start + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int b = lo, q0 = __ldg(a.r.q_start + b), q1 = __ldg(a.r.q_start + b + 1);
  uint32_t bits = 0;
  if (q0 < 0 || q1 > a.r.N || t < q0 || t >= q1) {
    if (lane == 0) atomicOr(a.err, SGD_KV_ERR_LENGTH);
    return;
  }
  const int ql = q1 - q0, n = a.r.seq_lens ? __ldg(a.r.seq_lens + b) : ql, old = n < ql ? -1 : n - ql, p = old + t - q0;
  T *out = static_cast<T *>(a.out) + ((long long)t * a.q_heads + hq) * D + lane * E;
  if (old < 0 || (a.r.seq_lens && n > (long long)a.r.max_pages * a.c.page)) {
    for (int e = 0; e < E; ++e) out[e] = from_f32<T>(0.f);
    if (lane == 0) atomicOr(a.err, SGD_KV_ERR_LENGTH);
    return;
  }
  float q[E], o[E] = {}, m = -CUDART_INF_F, l = 0.f;
  const T *qp = static_cast<const T *>(a.q) + t * a.q_token + hq * a.q_head + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = to_f32(qp[e]);
  for (int j = 0; j <= p; ++j) {
    if (a.window > 0 && j <= p - a.window && j >= a.sinks) continue;
    float k[E], v[E];
    if (j < old) {
      const int pg = __ldg(a.r.table + (long long)b * a.r.max_pages + (j >> a.c.page_bits));
      if (pg < 0 || pg >= a.c.num_pages) {
        bits |= SGD_KV_ERR_PAGE;
        continue;
      }
      const long long block = (long long)pg * a.c.heads + h;
      const long long at = (block * a.c.page + (j & (a.c.page - 1))) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t k2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(a.c.k + at + e));
        const uint32_t v2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(a.c.v + at + e));
        const float2 kf = __half22float2(*reinterpret_cast<const __half2 *>(&k2));
        const float2 vf = __half22float2(*reinterpret_cast<const __half2 *>(&v2));
        k[e] = kf.x * a.c.ks[block];
        k[e + 1] = kf.y * a.c.ks[block];
        v[e] = vf.x * a.c.vs[block];
        v[e + 1] = vf.y * a.c.vs[block];
      }
    } else {
      const T *kp = static_cast<const T *>(a.k) + (q0 + j - old) * a.k_token + h * a.k_head + lane * E;
      const T *vp = static_cast<const T *>(a.v) + (q0 + j - old) * a.v_token + h * a.v_head + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = to_f32(kp[e]);
        v[e] = to_f32(vp[e]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(FULL, s, x);
    s *= a.scale * LOG2E;
    const float top = fmaxf(m, s), base = top == -CUDART_INF_F ? 0.f : top;
    const float keep = ex2_approx(m - base), w = ex2_approx(s - base);
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * v[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_f32<T>(o[e] / l);
  if (bits && lane == 0) atomicOr(a.err, bits);
}

template <typename T>
cudaError_t launch(const KvNewArgs &a, cudaStream_t st) {
  const unsigned blocks = (unsigned)(((long long)a.r.N * a.q_heads + 3) / 4);
  if (a.c.dim == 128) new_kernel<T, 128><<<blocks, 128, 0, st>>>(a);
  else new_kernel<T, 64><<<blocks, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv_new_workspace(int sms) { return 0; }
cudaError_t kv_new_set_limits() { return cudaSuccess; }

cudaError_t launch_kv_new(const KvNewArgs &a, int dtype, cudaStream_t st, int *launches) {
  *launches = 1;
  return dtype == SGD_F16 ? launch<__half>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace sgd
