// verify.cu -- verification of drafted tokens against the target's probabilities.
//
// Row b has num_valid[b] drafts x_0 .. x_{v-1} and v + 1 rows of the target's
// logits, one per position.  With l a position's logits and t the row's
// temperature,
//     m = max l,  e_j = exp((l_j - m) / t),  Z = sum e_j,  p_j = e_j / Z,
// draft i is accepted iff u_i q_i(x_i) < p_i(x_i) and all before it were (q =
// 1 where the drafter proposed x_i outright), and at the first position that
// is not accepted, or after the last draft, one more token is drawn as
//     argmax_j w_j / noise_j,   noise_j ~ Exp(1) given,
// which picks j with probability w_j / sum w: w = p after the last draft, else
// the residual max(p - q, 0), which for a plain draft is p without x_i.  The
// accepted prefix and that token are together distributed as the target's own
// samples.  Temperatures below 1e-5 take the largest logit instead.
//
// Two launches.  The first makes (m, Z, argmax) of each position in one pass
// over its logits, a running maximum and sum per thread; a position is split
// over several CTAs and the last one to finish joins them in a fixed order, so
// that the result does not depend on which CTA that is.  The second draws at
// the one position per row where the drafts end, again split and joined.
// Statistics are held in 32 bits.  Both are bound by reading the logits (and
// the noise) once.
#include <math_constants.h>

#include "num_types.cuh"
#include "sgd_internal.h"

namespace sgd {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;                 // 16-byte loads in flight per thread
constexpr float LOG2E = 1.4426950408889634f;
constexpr float GREEDY_BELOW = 1e-5f;
constexpr float NOISE_MIN = 8.673617379884035e-19f;  // 2^-60: w / noise stays finite

struct Stat {
  float m, z;
  int arg;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp((l - m) / t) with c = log2(e) / t.  The difference is taken before the
// scaling, so logits of any size lose nothing; a NaN counts as -inf (the
// maximum with a number drops it).
__device__ __forceinline__ float weight(float l, float m, float c) {
  return ex2(fmaxf((l - m) * c, -1e30f));
}
// the same where m may be +inf: then only the +inf logits weigh, 1 each
__device__ __forceinline__ float weight_any(float l, float m, float c) {
  return m == CUDART_INF_F ? (l == CUDART_INF_F ? 1.f : 0.f) : weight(l, m, c);
}

__device__ __forceinline__ Stat join(const Stat &a, const Stat &b, float c) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  const float sa = a.m == r.m ? 1.f : weight(a.m, r.m, c);
  const float sb = b.m == r.m ? 1.f : weight(b.m, r.m, c);
  r.z = (a.z == 0.f ? 0.f : a.z * sa) + (b.z == 0.f ? 0.f : b.z * sb);
  r.arg = a.m > b.m ? a.arg : b.m > a.m ? b.arg : min(a.arg, b.arg);
  return r;
}

__device__ __forceinline__ Stat join_warp(Stat s, float c) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Stat t;
    t.m = __shfl_xor_sync(FULL, s.m, o);
    t.z = __shfl_xor_sync(FULL, s.z, o);
    t.arg = __shfl_xor_sync(FULL, s.arg, o);
    s = join(s, t, c);
  }
  return s;
}

// What a row's CTAs need to know of it.
struct Row {
  int nv;          // drafts
  long long first; // its first row of logits
  float t, c;      // temperature (1 for a greedy row), log2(e) / t
  bool greedy, on;
};

__device__ __forceinline__ Row row_of(const VerifyArgs &a, int b, bool report) {
  Row r;
  const int nv = a.num_valid[b];
  r.nv = min(max(nv, 0), a.k);
  r.first = a.row_start ? (long long)a.row_start[b] : (long long)b * (a.k + 1);
  const bool fits = r.first >= 0 && r.first + r.nv < a.rows;
  r.on = fits && (a.active == nullptr || a.active[b]);
  float t = a.temp ? a.temp[b] : 1.f;
  r.greedy = !(t >= GREEDY_BELOW);
  if (report) {
    uint32_t bits = 0;
    if (nv != r.nv || !fits) bits |= SGD_ERR_VERIFY_ROWS;
    if (!(t >= 0.f)) bits |= SGD_ERR_TEMPERATURE;
    if (bits) atomicOr(a.err, bits);
  }
  r.t = r.greedy ? 1.f : t;
  r.c = fmaxf(LOG2E * (1.f / r.t), 1e-37f);  // (positive: -inf logits keep weight 0)
  return r;
}

// Splits [lo, hi) of a row of T at `base` into elements before the first
// 16-byte boundary, whole 16-byte vectors, and what is left.
template <typename T>
struct Span {
  const T *base;
  int lo, hi, v0, nvec;  // vector i covers elements v0 + i * VN ..
  static constexpr int VN = 16 / sizeof(T);
  __device__ Span(const T *row, int lo_, int hi_) : base(row), lo(lo_), hi(hi_) {
    const int mis = (int)(((uintptr_t)(row + lo) & 15) / sizeof(T));
    v0 = min(hi, lo + (mis ? VN - mis : 0));
    nvec = (hi - v0) / VN;
  }
  // ordinal of a thread's edge element: head elements first, then the tail's
  __device__ int edge(int i) const {
    const int head = v0 - lo;
    if (i < head) return lo + i;
    const int e = v0 + nvec * VN + (i - head);
    return e < hi ? e : -1;
  }
};

template <typename T>
__global__ void __launch_bounds__(THREADS) verify_stats_kernel(VerifyArgs a) {
  __shared__ Stat sh[THREADS / 32];
  __shared__ int last;
  const int split = blockIdx.x % a.splits;
  const int pb = blockIdx.x / a.splits;
  const int i = pb / a.B, b = pb % a.B;
  const Row r = row_of(a, b, i == 0 && split == 0 && threadIdx.x == 0);
  if (!r.on || i > r.nv) return;
  const T *row = static_cast<const T *>(a.logits) + (r.first + i) * a.stride;
  const int chunk = (a.V + a.splits - 1) / a.splits;
  const int lo = min(a.V, split * chunk), hi = min(a.V, lo + chunk);
  const Span<T> sp(row, lo, hi);
  constexpr int VN = Span<T>::VN;
  const int tid = threadIdx.x;
  Stat s{-CUDART_INF_F, 0.f, 0x7fffffff};
  // (edge elements: at most 2 (VN - 1) of them)
  if (tid < 2 * VN) {
    const int e = sp.edge(tid);
    if (e >= 0) {
      const float l = to_f32(row[e]);
      if (l > s.m) {
        s.m = l;
        s.arg = e;
        s.z = 1.f;
      }
    }
  }
  const uint4 *vec = reinterpret_cast<const uint4 *>(row + sp.v0);
  for (int v = tid; v < sp.nvec; v += UNROLL * THREADS) {
    uint4 raw[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j)
      raw[j] = v + j * THREADS < sp.nvec ? __ldcs(vec + v + j * THREADS) : lowest_vec<T>();
    float x[UNROLL][VN];
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      unpack<T>(raw[j], x[j]);
#pragma unroll
      for (int e = 0; e < VN; ++e) mx = fmaxf(mx, x[j][e]);
    }
    if (mx >= s.m) {
      int at = 0x7fffffff;
#pragma unroll
      for (int j = UNROLL - 1; j >= 0; --j)
#pragma unroll
        for (int e = VN - 1; e >= 0; --e)
          if (x[j][e] == mx) at = sp.v0 + (v + j * THREADS) * VN + e;
      if (mx > s.m) {
        s.z = s.z == 0.f ? 0.f : s.z * weight(s.m, mx, r.c);
        s.m = mx;
        s.arg = at;
      } else {
        s.arg = min(s.arg, at);  // (a tail element of the same value may come first)
      }
    }
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < UNROLL; ++j)
#pragma unroll
      for (int e = 0; e < VN; ++e) z += weight(x[j][e], s.m, r.c);
    s.z += z;
  }
  if (s.m == CUDART_INF_F) {  // +inf logits: they alone weigh; count this thread's
    s.z = 0.f;
    if (tid < 2 * VN) {
      const int e = sp.edge(tid);
      if (e >= 0 && to_f32(row[e]) == CUDART_INF_F) s.z += 1.f;
    }
    for (int v = tid; v < sp.nvec; v += THREADS)
      for (int e = 0; e < VN; ++e)
        if (to_f32(row[sp.v0 + v * VN + e]) == CUDART_INF_F) s.z += 1.f;
  }
  s = join_warp(s, r.c);
  if ((tid & 31) == 0) sh[tid >> 5] = s;
  __syncthreads();
  if (tid >= 32) return;
  s = tid < THREADS / 32 ? sh[tid] : Stat{-CUDART_INF_F, 0.f, 0x7fffffff};
  s = join_warp(s, r.c);
  const int pos = b * (a.k + 1) + i;
  if (a.splits > 1) {
    if (tid == 0) {
      float4 *part = a.part + (long long)pb * a.splits;
      part[split] = make_float4(s.m, s.z, __int_as_float(s.arg), 0.f);
      __threadfence();
      last = atomicInc(a.count + pos, (unsigned)a.splits - 1) == (unsigned)a.splits - 1;
    }
    __syncwarp();
    if (!last) return;
    __threadfence();
    const float4 *part = a.part + (long long)pb * a.splits;
    s = Stat{-CUDART_INF_F, 0.f, 0x7fffffff};
    for (int j = tid; j < a.splits; j += 32) {
      const float4 p = __ldcg(part + j);
      s = join(s, Stat{p.x, p.y, __float_as_int(p.z)}, r.c);
    }
    s = join_warp(s, r.c);
  }
  if (tid != 0) return;
  a.stat[pos] = make_float4(s.m, s.z, __int_as_float(s.arg), 0.f);
  if (i == r.nv) return;
  // draft i: accepted, or the row ends here at the latest
  const int x = a.drafts[(long long)b * a.k + i];
  bool ok = false;
  if (x >= 0 && x < a.V && s.z > 0.f) {
    if (r.greedy) {
      ok = x == s.arg;
    } else {
      float u = a.uniform[(long long)b * a.k + i];
      if (a.q) u *= fmaxf(a.q[(r.first + i) * a.q_stride + x], 0.f);
      ok = u < weight_any(to_f32(row[x]), s.m, r.c) / s.z;
    }
  }
  if (!ok) atomicMin(a.stop + b, i);
}

struct Best {
  float w;  // the largest weight over noise, 0 if there is none
  int arg;
};
__device__ __forceinline__ Best better(const Best &x, const Best &y) {
  return x.w > y.w || (x.w == y.w && x.arg < y.arg) ? x : y;
}
__device__ __forceinline__ Best better_warp(Best s) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    s = better(s, Best{__shfl_xor_sync(FULL, s.w, o), __shfl_xor_sync(FULL, s.arg, o)});
  return s;
}
// The product with the noise is compared before the quotient is made: the
// division is reached a few times per thread only.
__device__ __forceinline__ void take(Best &s, float w, float noise, int j) {
  const float n = fmaxf(noise, NOISE_MIN);
  if (w >= s.w * n && w > 0.f) {
    const float q = w / n;
    if (q > s.w || (q == s.w && j < s.arg)) s = Best{q, j};
  }
}

// Row b's outputs: the accepted drafts and `token` (-1: none), the log
// probability of each.  One warp or more; `n` threads take part.
template <typename T>
__device__ void emit(const VerifyArgs &a, const Row &r, int b, int acc, int token, int tid, int n) {
  const T *first = static_cast<const T *>(a.logits) + r.first * a.stride;
  for (int i = tid; i <= a.k; i += n) {
    int x = -1;
    if (i < acc) x = a.drafts[(long long)b * a.k + i];
    if (i == acc) x = token;
    a.sampled[(long long)b * (a.k + 1) + i] = x;
    if (a.logprobs) {
      float lp = 0.f;
      if (x >= 0) {
        const float4 st = a.stat[b * (a.k + 1) + i];
        const float l = to_f32(first[i * a.stride + x]);
        lp = (l == st.x ? 0.f : (l - st.x) * (1.f / r.t)) - logf(st.y);
      }
      a.logprobs[(long long)b * (a.k + 1) + i] = lp;
    }
  }
  if (tid == 0) a.accepted[b] = acc;
}

template <typename T, bool Q>
__global__ void __launch_bounds__(THREADS) verify_draw_kernel(VerifyArgs a) {
  __shared__ Best sh[2][THREADS / 32];
  __shared__ int last;
  const int split = blockIdx.x % a.draw_splits, b = blockIdx.x / a.draw_splits;
  const int tid = threadIdx.x;
  const Row r = row_of(a, b, false);
  if (!r.on) {
    if (split == 0) {
      for (int i = tid; i <= a.k; i += THREADS) {
        a.sampled[(long long)b * (a.k + 1) + i] = -1;
        if (a.logprobs) a.logprobs[(long long)b * (a.k + 1) + i] = 0.f;
      }
      if (tid == 0) a.accepted[b] = 0;
    }
    return;
  }
  if (r.greedy && split != 0) return;
  const int acc = min(__ldcg(a.stop + b), r.nv);
  const float4 st = a.stat[b * (a.k + 1) + acc];
  const float m = st.x, z = st.y;
  int token = -1;
  if (r.greedy) {
    __syncthreads();
    if (z > 0.f) token = __float_as_int(st.z);
  } else {
    const long long at = r.first + acc;
    const T *row = static_cast<const T *>(a.logits) + at * a.stride;
    const float *noise = a.noise + (long long)b * a.noise_stride;
    const bool rejected = acc < r.nv;
    const int x = rejected ? a.drafts[(long long)b * a.k + acc] : -1;
    const float *q = Q && rejected ? a.q + at * a.q_stride : nullptr;
    const int chunk = (a.V + a.draw_splits - 1) / a.draw_splits;
    const int lo = min(a.V, split * chunk), hi = min(a.V, lo + chunk);
    const Span<T> sp(row, lo, hi);
    constexpr int VN = Span<T>::VN;
    Best s{0.f, 0x7fffffff}, f{0.f, 0x7fffffff};  // of the residual; of p, should that be empty
    const float inv_z = 1.f / z;
    auto one = [&](int j, float l, float nz, float qj) {
      const float e = weight_any(l, m, r.c);
      if (Q && q) {
        take(s, fmaxf(e * inv_z - fmaxf(qj, 0.f), 0.f), nz, j);
        take(f, e, nz, j);
      } else {
        take(s, j == x ? 0.f : e, nz, j);
      }
    };
    if (tid < 2 * VN) {
      const int e = sp.edge(tid);
      if (e >= 0) one(e, to_f32(row[e]), noise[e], Q && q ? q[e] : 0.f);
    }
    const uint4 *vec = reinterpret_cast<const uint4 *>(row + sp.v0);
    const bool nz16 = (((uintptr_t)(noise + sp.v0)) & 15) == 0;
    const bool q16 = Q && q && (((uintptr_t)(q + sp.v0)) & 15) == 0;
    for (int v = tid; v < sp.nvec; v += THREADS) {
      const int j0 = sp.v0 + v * VN;
      const uint4 raw = __ldcs(vec + v);
      float nz[VN], qv[VN];
      load_f32<VN>(noise + j0, nz16, nz);
      if (Q && q) load_f32<VN>(q + j0, q16, qv);
      float l[VN];
      unpack<T>(raw, l);
#pragma unroll
      for (int e = 0; e < VN; ++e) one(j0 + e, l[e], nz[e], Q && q ? qv[e] : 0.f);
    }
    s = better_warp(s);
    if (Q) f = better_warp(f);
    if ((tid & 31) == 0) {
      sh[0][tid >> 5] = s;
      if (Q) sh[1][tid >> 5] = f;
    }
    __syncthreads();
    if (tid >= 32) return;
    s = tid < THREADS / 32 ? sh[0][tid] : Best{0.f, 0x7fffffff};
    s = better_warp(s);
    if (Q) {
      f = tid < THREADS / 32 ? sh[1][tid] : Best{0.f, 0x7fffffff};
      f = better_warp(f);
    }
    if (a.draw_splits > 1) {
      float4 *part = a.draw_part + (long long)b * a.draw_splits;
      if (tid == 0) {
        part[split] = make_float4(s.w, __int_as_float(s.arg), f.w, __int_as_float(f.arg));
        __threadfence();
        last = atomicInc(a.draw_count + b, (unsigned)a.draw_splits - 1) == (unsigned)a.draw_splits - 1;
      }
      __syncwarp();
      if (!last) return;
      __threadfence();
      s = f = Best{0.f, 0x7fffffff};
      for (int j = tid; j < a.draw_splits; j += 32) {
        const float4 p = __ldcg(part + j);
        s = better(s, Best{p.x, __float_as_int(p.y)});
        f = better(f, Best{p.z, __float_as_int(p.w)});
      }
      s = better_warp(s);
      f = better_warp(f);
    }
    if (s.w > 0.f) {
      token = s.arg;
    } else if (Q && q && f.w > 0.f) {
      token = f.arg;  // nothing left of the residual (by rounding, or u >= 1): p itself
    } else if (rejected && x >= 0 && x < a.V && weight_any(to_f32(row[x]), m, r.c) > 0.f) {
      token = x;
    }
  }
  emit<T>(a, r, b, acc, token, tid, r.greedy ? THREADS : 32);
  if (tid == 0) {
    if (token < 0) atomicOr(a.err, SGD_ERR_NO_TOKEN);
    a.stop[b] = 0x7fffffff;  // for the next call
  }
}

template <typename T>
cudaError_t launch(const VerifyArgs &a, cudaStream_t st) {
  const unsigned stats = (unsigned)((long long)a.B * (a.k + 1) * a.splits);
  verify_stats_kernel<T><<<stats, THREADS, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned draws = (unsigned)(a.B * a.draw_splits);
  if (a.q)
    verify_draw_kernel<T, true><<<draws, THREADS, 0, st>>>(a);
  else
    verify_draw_kernel<T, false><<<draws, THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// CTAs that a launch is split into where there are fewer rows than that.
constexpr long long VERIFY_CTAS = 152 * 64;
constexpr int VERIFY_MAX_SPLITS = 64;

int verify_splits(long long rows, int V) {
  long long s = (VERIFY_CTAS + rows - 1) / rows;
  s = s < VERIFY_MAX_SPLITS ? s : VERIFY_MAX_SPLITS;
  const long long most = (V + 2047) / 2048;  // 2048 elements: one 16-byte load per thread
  s = s < most ? s : most;
  return s < 1 ? 1 : (int)s;
}

VerifyLayout verify_layout(int max_batch, int k) {
  VerifyLayout l;
  const size_t pos = (size_t)max_batch * (k + 1);
  l.part = 0;
  l.draw_part = l.part + (VERIFY_CTAS + pos) * 16;
  l.stat = l.draw_part + (VERIFY_CTAS + (size_t)max_batch) * 16;
  l.count = l.stat + pos * 16;
  l.draw_count = l.count + pos * 4;
  l.stop = l.draw_count + (size_t)max_batch * 4;
  l.bytes = l.stop + (size_t)max_batch * 4;
  return l;
}

cudaError_t launch_verify(const VerifyArgs &args, int dtype, cudaStream_t st) {
  VerifyArgs a = args;
  a.splits = verify_splits((long long)a.B * (a.k + 1), a.V);
  a.draw_splits = verify_splits(a.B, a.V);
  if (dtype == SGD_F32) return launch<float>(a, st);
  if (dtype == SGD_F16) return launch<__half>(a, st);
  return launch<__nv_bfloat16>(a, st);
}

}  // namespace sgd
