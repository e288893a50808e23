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
// over the CTAs of a cluster, whose first CTA joins their parts, in order,
// from its shared memory.  The second draws at the one position per row where
// the drafts end, split and joined alike.  Statistics are held in 32 bits.
// Both are bound by reading the logits (and the noise) once: at V = 151936, 256
// rows of up to 17 positions in bf16, 142 us, 5.7 TB/s (positions after the first
// rejected one are not drawn at); at V = 128256, 48 rows of 6 positions in 32 bits
// with draft probabilities, too little to fill the GPU for long, 41 us, 3.3 TB/s;
// 10 us at 4 rows of V = 32000, where two launches and the joins are most of it.
#include <math_constants.h>

#include "num_types.cuh"
#include "sgd_internal.h"
#include "verify.h"

namespace sgd {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;                 // 16-byte loads in flight per thread
constexpr int PER_SM = 4;                 // CTAs of an SM
constexpr int MAX_SPLITS = 8;             // CTAs of a cluster, everywhere allowed
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float GREEDY_BELOW = 1e-5f;
constexpr float NOISE_MIN = 8.673617379884035e-19f;  // 2^-60: w / noise stays finite

struct Stat {
  float m, z;
  int arg;
};

// A cluster's CTAs give their parts to the first one's shared memory:
// started() before anything else, then, when a part is ready, reached() (every
// CTA is running, so its memory may be written), the stores, done(), and in
// the first CTA all_done().
__device__ __forceinline__ void started() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void reached() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void done() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void all_done() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void give(void *slot, float4 v) {  // to `slot` in CTA 0
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"((uint32_t)__cvta_generic_to_shared(slot)));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(there), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp((l - m) / t) as 2^x, c = log2(e) / t.  With the reference r = m c rounded
// once, x = l c - r is one multiply-add that rounds only its small result, and
// the error of r (half a unit of its last place) is the same factor in every
// weight and in Z, and cancels.  That factor has to stay near 1: from |r| = 2^20
// on, where it would pass 2^(2^-4) and, ever larger, leave the type's range, the
// difference is taken first, x = (l - m) c.  A NaN logit or +inf - +inf weighs 0.
constexpr float LARGE_REF = 1048576.f;  // 2^20
__device__ __forceinline__ bool small_ref(float r) { return fabsf(r) < LARGE_REF; }
__device__ __forceinline__ float log2_weight(float l, float m, float c) {
  const float r = m * c;
  const float x = small_ref(r) ? fmaf(l, c, -r) : (l - m) * c;
  return fmaxf(x, -1e30f);
}
__device__ __forceinline__ float weight(float l, float m, float c) { return ex2(log2_weight(l, m, c)); }
// the same where m may be +inf: then only the +inf logits weigh, 1 each
__device__ __forceinline__ float weight_any(float l, float m, float c) {
  return m == CUDART_INF_F ? (l == CUDART_INF_F ? 1.f : 0.f) : weight(l, m, c);
}
// From one maximum to a larger one: the difference of what weight() took away,
// each maximum's product with c rounded where it is small, else exact.
__device__ __forceinline__ float reweight(float from, float to, float c) {
  const float x = from * c, y = to * c;
  float d = x - y;
  if (__builtin_expect(!(small_ref(x) && small_ref(y)), 0))
    d = small_ref(x) ? fmaf(-to, c, x) : small_ref(y) ? fmaf(from, c, -y) : (from - to) * c;
  return ex2(fmaxf(d, -1e30f));
}

__device__ __forceinline__ Stat join(const Stat &a, const Stat &b, float c) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  const float k = a.m == b.m ? 1.f : reweight(fminf(a.m, b.m), r.m, c);
  r.z = a.m == r.m ? fmaf(b.z, k, a.z) : fmaf(a.z, k, b.z);
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

// The largest of N vectors' elements (NaN counts as -inf).
template <typename T, int N>
__device__ __forceinline__ float max_of(const uint4 (&raw)[N]) {
  if constexpr (sizeof(T) == 4) {
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float x[4];
      unpack<float>(raw[j], x);
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, x[e]);
    }
    return mx;
  } else {  // two at a time
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const uint32_t low = lowest_vec<T>().x;
    T2 mx = *reinterpret_cast<const T2 *>(&low);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = __hmax2(mx, *reinterpret_cast<const T2 *>(&w[e]));
    }
    return fmaxf(to_f32(mx.x), to_f32(mx.y));
  }
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
__global__ void __launch_bounds__(THREADS, PER_SM) verify_stats_kernel(VerifyArgs a) {
  __shared__ Stat sh[THREADS / 32];
  __shared__ float4 parts[MAX_SPLITS];
  cudaTriggerProgrammaticLaunchCompletion();  // (the draw's CTAs may take their places and wait)
  const int split = blockIdx.x % a.splits;
  const int pb = blockIdx.x / a.splits;
  const int i = pb / a.B, b = pb % a.B;
  const Row r = row_of(a, b, i == 0 && split == 0 && threadIdx.x == 0);
  if (!r.on || i > r.nv) return;
  // A position after one that was not accepted decides nothing: its logits are
  // not read.  Positions come in order, all rows' first ones first, so this is
  // often known by now; where it is not, the work is done and not used.
  started();
  const bool moot = __syncthreads_or(__ldcg(a.stop + b) < i);
  const T *row = static_cast<const T *>(a.logits) + (r.first + i) * a.stride;
  const int chunk = (a.V + a.splits - 1) / a.splits;
  const int lo = min(a.V, split * chunk), hi = moot ? lo : min(a.V, lo + chunk);
  const Span<T> sp(row, lo, hi);
  constexpr int VN = Span<T>::VN;
  const int tid = threadIdx.x;
  // what the decision needs, on its way while the logits are read
  const bool decides = split == 0 && tid == 0 && i < r.nv;
  int draft = -1;
  float u = 0.f, l_draft = 0.f;
  if (decides) {
    draft = a.drafts[(long long)b * a.k + i];
    if (draft >= 0 && draft < a.V) {
      l_draft = to_f32(row[draft]);
      if (!r.greedy) {
        u = a.uniform[(long long)b * a.k + i];
        if (a.q) u *= fmaxf(a.q[(r.first + i) * a.q_stride + draft], 0.f);
      }
    }
  }
  Stat s{-CUDART_INF_F, 0.f, 0x7fffffff};
  int best = -1;  // the group of vectors that holds the largest logit (-1: an edge element)
  // (edge elements: at most 2 (VN - 1) of them)
  if (tid < 2 * VN) {
    const int e = sp.edge(tid);
    if (e >= 0) {
      const float l = to_f32(row[e]);
      if (l > s.m) {
        s.m = l;
        s.arg = e;
        s.z = weight(l, l, r.c);
      }
    }
  }
  const float edge_m = s.m;
  const uint4 *vec = reinterpret_cast<const uint4 *>(row + sp.v0);
  uint4 raw[UNROLL], ahead[UNROLL];  // the next group is on its way while one is worked on
  auto fetch = [&](int v) {
#pragma unroll
    for (int j = 0; j < UNROLL; ++j)
      ahead[j] = v + j * THREADS < sp.nvec ? __ldcs(vec + v + j * THREADS) : lowest_vec<T>();
  };
  fetch(tid);
  for (int v = tid; v < sp.nvec; v += UNROLL * THREADS) {
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) raw[j] = ahead[j];
    if (v + UNROLL * THREADS < sp.nvec) fetch(v + UNROLL * THREADS);
    const float mx = max_of<T, UNROLL>(raw);
    if (mx > s.m) {
      s.z *= reweight(s.m, mx, r.c);  // (0 and finite, or a finite product)
      s.m = mx;
      best = v;
    } else if (mx == s.m && best < 0) {
      best = v;  // (an edge element of the same value may be the row's last)
    }
    const float ref = s.m * r.c;
    float z = 0.f;
    if (__builtin_expect(small_ref(ref), 1)) {
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        float x[VN];
        unpack<T>(raw[j], x);
#pragma unroll
        for (int e = 0; e < VN; ++e) z += ex2(fmaf(x[e], r.c, -ref));
      }
    } else {
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        float x[VN];
        unpack<T>(raw[j], x);
#pragma unroll
        for (int e = 0; e < VN; ++e) z += ex2((x[e] - s.m) * r.c);
      }
    }
    if (!(z < CUDART_INF_F)) {  // NaN logits, an infinite maximum, or nothing but -inf so far
      z = 0.f;
#pragma unroll 1
      for (int j = 0; j < UNROLL; ++j)
        for (int e = 0; e < VN && v + j * THREADS < sp.nvec && s.m != -CUDART_INF_F; ++e)
          z += weight(to_f32(row[sp.v0 + (v + j * THREADS) * VN + e]), s.m, r.c);
    }
    s.z += z;
  }
  if (r.greedy && best >= 0) {  // its lowest index (an earlier group of this thread has none)
    if (edge_m != s.m) s.arg = 0x7fffffff;
    for (int j = UNROLL - 1; j >= 0; --j)
      for (int e = VN - 1; e >= 0; --e) {
        const int g = best + j * THREADS, at = sp.v0 + g * VN + e;
        if (g < sp.nvec && to_f32(row[at]) == s.m) s.arg = min(s.arg, at);
      }
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
  if (!moot) {
    s = join_warp(s, r.c);
    if ((tid & 31) == 0) sh[tid >> 5] = s;
    __syncthreads();
  }
  reached();
  if (tid < 32 && !moot) {
    s = tid < THREADS / 32 ? sh[tid] : Stat{-CUDART_INF_F, 0.f, 0x7fffffff};
    s = join_warp(s, r.c);
  }
  if (tid == 0) give(parts + split, make_float4(s.m, s.z, __int_as_float(s.arg), moot ? 1.f : 0.f));
  done();
  if (split != 0) return;
  all_done();
  if (tid >= 32) return;
  s = Stat{-CUDART_INF_F, 0.f, 0x7fffffff};
  bool missing = false;
  if (tid < a.splits) {
    const float4 p = parts[tid];
    s = Stat{p.x, p.y, __float_as_int(p.z)};
    missing = p.w != 0.f;
  }
  if (__any_sync(FULL, missing)) return;
  s = join_warp(s, r.c);
  if (tid != 0) return;
  a.stat[b * (a.k + 1) + i] = make_float4(s.m, s.z, __int_as_float(s.arg), 0.f);
  if (i == r.nv) return;
  // draft i: accepted, or the row ends here at the latest
  bool ok = false;
  if (draft >= 0 && draft < a.V && s.m != -CUDART_INF_F)
    ok = r.greedy ? draft == s.arg : u < weight_any(l_draft, s.m, r.c) / s.z;
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
// A weight over its noise.
__device__ __forceinline__ float ratio(float w, float noise) {
  return __fdividef(w, fmaxf(noise, NOISE_MIN));
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
        const float4 st = __ldcg(a.stat + b * (a.k + 1) + i);
        const float l = to_f32(first[i * a.stride + x]);
        lp = ((l == st.x && fabsf(l) == CUDART_INF_F ? 0.f : log2_weight(l, st.x, r.c)) - log2f(st.y)) * LN2;
      }
      a.logprobs[(long long)b * (a.k + 1) + i] = lp;
    }
  }
  if (tid == 0) a.accepted[b] = acc;
}

template <typename T, bool Q>
__global__ void __launch_bounds__(THREADS, Q ? 3 : 4) verify_draw_kernel(VerifyArgs a) {
  __shared__ Best sh[2][THREADS / 32];
  __shared__ float4 parts[MAX_SPLITS];
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
  if (!r.greedy) started();
  else if (split != 0) return;
  cudaGridDependencySynchronize();
  const int acc = min(__ldcg(a.stop + b), r.nv);
  const float4 st = __ldcg(a.stat + b * (a.k + 1) + acc);
  const float m = st.x, z = st.y;
  int token = -1;
  if (r.greedy) {
    __syncthreads();
    if (m != -CUDART_INF_F) token = __float_as_int(st.z);
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
    const float inv_z = 1.f / z, ref = m * r.c;
    const bool plain = small_ref(ref);  // (m is finite, so only a NaN logit needs more)
    // weight over noise: of the residual, and of p
    auto pair = [&](int j, float l, float nz, float qj, float &of_s, float &of_f) {
      const float e = plain ? ex2(fmaf(l, r.c, -ref)) : weight_any(l, m, r.c);
      if (Q && q) {
        of_s = ratio(fmaxf(__fmaf_rn(e, inv_z, -fmaxf(qj, 0.f)), 0.f), nz);
        of_f = ratio(e, nz);
      } else {
        of_s = j == x ? 0.f : ratio(e, nz);
        of_f = 0.f;
      }
    };
    if (tid < 2 * VN) {
      const int e = sp.edge(tid);
      if (e >= 0) {
        float u, w;
        pair(e, to_f32(row[e]), noise[e], Q && q ? q[e] : 0.f, u, w);
        if (u > 0.f) s = Best{u, e};
        if (w > 0.f) f = Best{w, e};
      }
    }
    const uint4 *vec = reinterpret_cast<const uint4 *>(row + sp.v0);
    const bool nz16 = (((uintptr_t)(noise + sp.v0)) & 15) == 0;
    const bool q16 = Q && q && (((uintptr_t)(q + sp.v0)) & 15) == 0;
    int at_s = -1, at_f = -1;  // the vectors that hold the best
    auto load = [&](int v, uint4 &raw, float (&nz)[VN], float (&qv)[VN]) {
      raw = __ldcs(vec + v);
      load_f32<VN>(noise + sp.v0 + v * VN, nz16, nz);
      if (Q && q) load_f32<VN>(q + sp.v0 + v * VN, q16, qv);
    };
    auto take = [&](int v, const uint4 &raw, const float (&nz)[VN], const float (&qv)[VN]) {
      const int j0 = sp.v0 + v * VN;
      float l[VN], top_s = 0.f, top_f = 0.f;
      unpack<T>(raw, l);
#pragma unroll
      for (int e = 0; e < VN; ++e) {
        float u, w;
        pair(j0 + e, l[e], nz[e], Q && q ? qv[e] : 0.f, u, w);
        top_s = fmaxf(top_s, u);
        if (Q) top_f = fmaxf(top_f, w);
      }
      if (top_s > s.w || (top_s == s.w && s.arg != 0x7fffffff && j0 < s.arg)) {
        s = Best{top_s, j0};
        at_s = v;
      }
      if (Q && (top_f > f.w || (top_f == f.w && f.arg != 0x7fffffff && j0 < f.arg))) {
        f = Best{top_f, j0};
        at_f = v;
      }
    };
    for (int v = tid; v < sp.nvec; v += 2 * THREADS) {
      uint4 raw[2];
      float nz[2][VN], qv[2][VN];
      const bool more = v + THREADS < sp.nvec;
      load(v, raw[0], nz[0], qv[0]);
      if (more) load(v + THREADS, raw[1], nz[1], qv[1]);
      take(v, raw[0], nz[0], qv[0]);
      if (more) take(v + THREADS, raw[1], nz[1], qv[1]);
    }
    // the best's own index: the lowest of its vector that has its value
    auto index = [&](int v, bool residual, Best &best) {
      for (int e = VN - 1; e >= 0; --e) {
        const int j = sp.v0 + v * VN + e;
        float u, w;
        pair(j, to_f32(row[j]), noise[j], Q && q ? q[j] : 0.f, u, w);
        if ((residual ? u : w) == best.w) best.arg = j;
      }
    };
    if (at_s >= 0) index(at_s, true, s);
    if (Q && at_f >= 0) index(at_f, false, f);
    s = better_warp(s);
    if (Q) f = better_warp(f);
    if ((tid & 31) == 0) {
      sh[0][tid >> 5] = s;
      if (Q) sh[1][tid >> 5] = f;
    }
    __syncthreads();
    reached();
    if (tid < 32) {
      s = better_warp(tid < THREADS / 32 ? sh[0][tid] : Best{0.f, 0x7fffffff});
      if (Q) f = better_warp(tid < THREADS / 32 ? sh[1][tid] : Best{0.f, 0x7fffffff});
    }
    if (tid == 0) give(parts + split, make_float4(s.w, __int_as_float(s.arg), f.w, __int_as_float(f.arg)));
    done();
    if (split != 0) return;
    all_done();
    if (tid >= 32) return;
    const float4 p = tid < a.draw_splits ? parts[tid] : make_float4(0.f, __int_as_float(0x7fffffff), 0.f, __int_as_float(0x7fffffff));
    s = better_warp(Best{p.x, __float_as_int(p.y)});
    f = better_warp(Best{p.z, __float_as_int(p.w)});
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

template <typename K>
cudaError_t launch_clusters(K *kernel, const VerifyArgs &a, long long rows, int splits, bool early, cudaStream_t st) {
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * splits));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T>
cudaError_t launch(const VerifyArgs &a, cudaStream_t st) {
  const cudaError_t e =
      launch_clusters(verify_stats_kernel<T>, a, (long long)a.B * (a.k + 1), a.splits, false, st);
  if (e != cudaSuccess) return e;
  return launch_clusters(a.q ? verify_draw_kernel<T, true> : verify_draw_kernel<T, false>, a, a.B, a.draw_splits,
                         true, st);
}

// CTAs of a row of logits: a power of two, until there are three CTAs per SM,
// in pieces of more than 1024 elements (a 16-byte load for each thread at 32
// bits, for half of them at 16).  Measured
// at V = 151936, B = 256, k = 16: 1 piece 142 us, 2 150, 4 182, 8 269 (each CTA
// costs its start and its joining); at V = 128256, B = 48, k = 5, 32-bit logits:
// 1 piece 48 us, 2 41, 8 44; at V = 32000, B = 4, k = 8: 1 piece 11.5 us, 8 10.5.
int splits_of(long long rows, int V) {
  int s = 1;
  while (s < MAX_SPLITS && rows * s < 152 * 3 && V > 2048 * s) s *= 2;
  return s;
}

}  // namespace

VerifyLayout verify_layout(int max_batch, int k) {
  VerifyLayout l;
  l.stat = 0;
  l.stop = (size_t)max_batch * (k + 1) * 16;
  l.bytes = l.stop + (size_t)max_batch * 4;
  return l;
}

cudaError_t launch_verify(const VerifyArgs &args, int dtype, cudaStream_t st) {
  VerifyArgs a = args;
  a.splits = splits_of((long long)a.B * (a.k + 1), a.V);
  a.draw_splits = splits_of(a.B, a.V);
  if (dtype == SGD_F32) return launch<float>(a, st);
  if (dtype == SGD_F16) return launch<__half>(a, st);
  return launch<__nv_bfloat16>(a, st);
}

}  // namespace sgd
