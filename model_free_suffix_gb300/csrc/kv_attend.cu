// kv_attend.cu -- attention of each row's new tokens over the paged 8-bit cache.
//
//   o_r = sum_j softmax_j(scale q_r . k_j) v_j   over the positions j that row
//   r's token, at position p, sees: j <= p, and with a window j > p - window or
//   j < sinks.
#include <math_constants.h>

#include "kv_internal.h"
#include "num_types.cuh"
#include "sgd_internal.h"

namespace sgd {
namespace {

constexpr int THREADS = 128;

// One CTA per new token and query head; its warps take every fourth position.
template <typename T>
__global__ void __launch_bounds__(THREADS) kv_attend_kernel(KvAttendArgs a) {
  __shared__ float so[THREADS / 32][128];
  __shared__ float sm[THREADS / 32], sl[THREADS / 32];
  const int i = blockIdx.x, hq = blockIdx.y, h = hq / a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.c.dim, P = a.c.page, per = D / 32;
  const int b = row_of_token(a.r.q_start, a.r.B, i);
  T *out = static_cast<T *>(a.out) + ((long long)i * a.q_heads + hq) * D;
  int p = -1;
  if (b < a.r.B) {
    const int q0 = a.r.q_start[b], q1 = a.r.q_start[b + 1], n = a.r.seq_lens[b];
    p = n - (q1 - q0) + (i - q0);
    if (n < q1 - q0 || (long long)n > (long long)a.r.max_pages * P) p = -1;
  }
  if (p < 0 && threadIdx.x == 0) atomicOr(a.err, SGD_KV_ERR_LENGTH);
  const T *q = static_cast<const T *>(a.q) + i * a.q_token + hq * a.q_head;
  float qr[4], o[4];
  for (int e = 0; e < per; ++e) {
    qr[e] = to_f32(q[lane * per + e]);
    o[e] = 0.f;
  }
  float m = -CUDART_INF_F, l = 0.f;
  const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  for (int j = warp; j <= p; j += THREADS / 32) {
    if (j < lo && j >= a.sinks) continue;
    const int page = a.r.table[(long long)b * a.r.max_pages + j / P];
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) atomicOr(a.err, SGD_KV_ERR_PAGE);
      continue;
    }
    const long long at = (long long)page * a.c.heads + h;
    const uint8_t *k = a.c.k + (at * P + j % P) * D + lane * per;
    const uint8_t *v = a.c.v + (at * P + j % P) * D + lane * per;
    float s = 0.f, x[4];
    for (int e = 0; e < per; e += 2) {
      const uint32_t w = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(k + e));
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
      s += qr[e] * f.x + qr[e + 1] * f.y;
      const uint32_t u = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(v + e));
      const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&u));
      x[e] = g.x;
      x[e + 1] = g.y;
    }
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(FULL, s, d);
    s *= a.scale * a.c.ks[at];
    const float m2 = fmaxf(m, s), c = __expf(m - m2), w = __expf(s - m2);
    l = l * c + w;
    const float wv = w * a.c.vs[at];
    for (int e = 0; e < per; ++e) o[e] = o[e] * c + wv * x[e];
    m = m2;
  }
  for (int e = 0; e < per; ++e) so[warp][lane * per + e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float M = -CUDART_INF_F;
  for (int w = 0; w < THREADS / 32; ++w) M = fmaxf(M, sm[w]);
  for (int d = threadIdx.x; d < D; d += THREADS) {
    float L = 0.f, x = 0.f;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (sl[w] == 0.f) continue;
      const float c = __expf(sm[w] - M);
      L += sl[w] * c;
      x += so[w][d] * c;
    }
    out[d] = from_f32<T>(L == 0.f ? 0.f : x / L);
  }
}

}  // namespace

size_t kv_attend_workspace(const sgd_kv_config &) { return 256; }

cudaError_t kv_attend_set_limits() { return cudaSuccess; }

cudaError_t launch_kv_attend(KvAttendArgs a, int dtype, cudaStream_t st, int *launches) {
  const dim3 grid(a.r.N, a.q_heads);
  if (dtype == SGD_F16)
    kv_attend_kernel<__half><<<grid, THREADS, 0, st>>>(a);
  else
    kv_attend_kernel<__nv_bfloat16><<<grid, THREADS, 0, st>>>(a);
  *launches = 1;
  return cudaGetLastError();
}

}  // namespace sgd
