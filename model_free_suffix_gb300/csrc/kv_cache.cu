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
// before the write's first token, and the new ones), so a rejected draft's
// values do not stay in it.  What they may have cost the block's other entries
// does: while the draft was there they were held at its scale s, each within
// 2^-10 s of what it was, and those of up to 2^-10 s as 0.
// Infinities do not count towards the scale and saturate, NaN is stored as 0;
// both set an error bit.
#include <math_constants.h>

#include "kv_internal.h"
#include "num_types.cuh"
#include "sgd_internal.h"

namespace sgd {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int EXP_MIN = -48, EXP_MAX = 48;
constexpr int PAST = 1 << 30;  // a position that no table reaches

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
        const uint4 v = *(reinterpret_cast<const uint4 *>(p) + i);
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
  // The largest magnitude so far (NaN once there is one): two values at a time
  // where they have 16 bits.
  using Top = typename std::conditional<sizeof(T) == 4, float, uint32_t>::type;
  __device__ __forceinline__ void top(Top &m) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(__uint_as_float(w[i]))));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value)
          asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
        else
          asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
      }
    }
  }
  __device__ __forceinline__ static float top_value(Top m) {
    if constexpr (sizeof(T) == 4) {
      return m;
    } else {
      T t[2];
      memcpy(t, &m, 4);
      const float a = to_f32(t[0]), b = to_f32(t[1]);
      return a != a ? a : fmaxf(b, a == a && b == b ? a : b);
    }
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

// Some tokens of one row in one page: what a CTA takes, its warps sharing out
// the heads of keys and values.
struct Segment {
  int b;      // row (B: none)
  int first;  // packed token
  int count;
  int page, slot;  // where the first one lives; page -1: nowhere
};

// The s-th segment of a call whose row b has the packed tokens starts[b] ..
// starts[b + 1] at positions from pos0(b) on (below 0: a row that must not be
// touched).  Every CTA counts the rows' segments, which costs about as much as
// the search for a token's row would and leaves no CTA without work but those
// past the end.  Up to 32 rows each warp counts for itself, without a barrier.
template <typename Pos>
__device__ Segment segment_of(const int32_t *starts, int B, int N, const int32_t *table, int max_pages, int num_pages,
                              int P, long long s, Pos pos0, uint32_t *bits) {
  __shared__ int warp_sum[WARPS];
  __shared__ int found[5];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool alone = B <= 32;
  int row = B, t0 = 0, t1 = 0, p = 0, j = 0;
  long long before = 0;
  if (!alone && tid == 0) found[0] = B;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + (alone ? lane : tid);
    int n = 0;
    t0 = t1 = p = 0;
    if (b < B) {
      t0 = __ldg(starts + b);
      t1 = __ldg(starts + b + 1);
      p = pos0(b, t1 - t0);
      if (t0 < 0 || t1 < t0 || t1 > N || (p < 0 && t1 > t0))
        *bits |= SGD_KV_ERR_LENGTH;
      else if (t1 > t0)
        n = (p % P + (t1 - t0) + P - 1) / P;
    }
    int scan = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(FULL, scan, o);
      if (lane >= o) scan += x;
    }
    long long at = before + scan - n;
    if (alone) {
      const bool mine = at <= s && s < at + n;
      const uint32_t who = __ballot_sync(FULL, mine);
      if (who == 0) return Segment{B, 0, 0, -1, 0};
      const int src = __ffs(who) - 1;
      row = src;
      t0 = __shfl_sync(FULL, t0, src);
      t1 = __shfl_sync(FULL, t1, src);
      p = __shfl_sync(FULL, p, src);
      j = __shfl_sync(FULL, (int)(s - at), src);
      break;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) at += warp_sum[w];
      before += warp_sum[w];
    }
    if (at <= s && s < at + n) {
      found[0] = b;
      found[1] = t0;
      found[2] = t1;
      found[3] = p;
      found[4] = (int)(s - at);
    }
    if (before > s) break;
  }
  if (!alone) {
    __syncthreads();
    row = found[0];
    t0 = found[1];
    t1 = found[2];
    p = found[3];
    j = found[4];
  }
  Segment g{row, 0, 0, -1, 0};
  if (row == B) return g;
  const int block = p / P + j, from = j == 0 ? p : block * P;
  g.slot = from - block * P;
  g.first = t0 + (from - p);
  g.count = min(t1 - g.first, P - g.slot);
  if (block < max_pages) g.page = __ldg(table + (long long)row * max_pages + block);
  if (g.page < 0 || g.page >= num_pages) {
    g.page = -1;
    *bits |= SGD_KV_ERR_PAGE;
  }
  return g;
}

// The larger magnitudes of 16 e4m3 bytes and what is there (NaN codes drop out).
__device__ __forceinline__ __half2 top_of(__half2 top, const uint4 &v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x, y;
    e4m3x4_to_f16x4(w[i], x, y);
    top = __hmax2(top, __habs2(*reinterpret_cast<const __half2 *>(&x)));
    top = __hmax2(top, __habs2(*reinterpret_cast<const __half2 *>(&y)));
  }
  return top;
}

// A team of warps (one, or as many as keep a page's new entries in registers)
// takes one head's keys or values of a segment: the largest magnitude first, of
// the new entries and the block's older ones, then the encoding.  Bound by
// latency at the few tokens of a verification step (256 rows of 1 to 17 tokens,
// 8 heads of 128, 31 MB with the entries already there: 12 us, 2.5 TB/s; 4 tokens
// of one row: 4 us), by the bytes and the conversions at prompts (8 rows, 30620
// tokens, 188 MB: 46 us, 4.1 TB/s).  A page and head is one team's, since the
// scale needs every entry before any is encoded.  A warp keeps 1024 new entries
// in registers; where its share of a page is larger (single warps at prompts) it
// reads them a second time, from L2, to encode them.  (Eight loads of old entries
// in flight instead of four, or wider ones, cost more registers than they gain:
// 36 us for that step and its read back against 32.)
template <typename T, int D>
__global__ void __launch_bounds__(THREADS, sizeof(T) == 4 ? 3 : 4) kv_write_kernel(KvWriteArgs a) {
  __shared__ float team_max[2][WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = a.c.page;
  uint32_t bits = 0;
  const Segment g = segment_of(
      a.r.q_start, a.r.B, a.r.N, a.r.table, a.r.max_pages, a.c.num_pages, P, blockIdx.x,
      [&](int b, int ql) { return min(__ldg(a.r.seq_lens + b) - ql, PAST); }, &bits);
  constexpr int PER = D / 8, STEP = 32 / PER, UNROLL = 4;  // lanes of a token, tokens of a round
  constexpr int ROUND = STEP * UNROLL;
  const int sub = lane % PER, at = lane / PER;
  const int teams = WARPS / a.team, mate = warp % a.team;
  int turn = 0;
  for (int hv0 = blockIdx.y * teams; g.count > 0 && hv0 < 2 * a.c.heads; hv0 += gridDim.y * teams, turn ^= 1) {
    const int hv = hv0 + warp / a.team;
    const bool idle = hv >= 2 * a.c.heads;  // (its warps only keep the others' barriers)
    const bool value = hv >= a.c.heads;
    const int h = idle ? 0 : value ? hv - a.c.heads : hv;
    const int count = idle ? 0 : g.count;
    const long long token = value ? a.v_token : a.k_token;
    const T *src = static_cast<const T *>(value ? a.v : a.k) + (long long)h * (value ? a.v_head : a.k_head) +
                   (long long)g.first * token + sub * 8;
    Eight<T> x[UNROLL];
    auto fetch = [&](int t0) {
#pragma unroll
      for (int i = 0; i < UNROLL; ++i)
        if (t0 + i * STEP + at < count) x[i].load(src + (t0 + i * STEP + at) * token, a.vec);
    };
    fetch(mate * ROUND);  // (on its way before the page is known)
    if (g.page < 0) break;
    const long long block = (long long)g.page * a.c.heads + h;
    uint8_t *base = (value ? a.c.v : a.c.k) + block * P * D;
    float *scale = (value ? a.c.vs : a.c.ks) + block;
    const float old = g.slot > 0 ? *scale : 1.f;
    __half2 top = __float2half2_rn(0.f);
    const int n_old = idle ? 0 : g.slot * D / 16;
    for (int i0 = mate * 32 * 4; i0 < n_old; i0 += a.team * 32 * 4) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (i0 + i * 32 + lane < n_old) v[i] = *reinterpret_cast<const uint4 *>(base + (i0 + i * 32 + lane) * 16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) top = top_of(top, v[i]);
    }
    float amax = fmaxf(__low2float(top), __high2float(top)) * old;
    typename Eight<T>::Top all = 0;
    for (int t0 = mate * ROUND; t0 < count; t0 += a.team * ROUND) {
      if (t0 != mate * ROUND) fetch(t0);
#pragma unroll
      for (int i = 0; i < UNROLL; ++i)
        if (t0 + i * STEP + at < count) x[i].top(all);
    }
    const float new_max = Eight<T>::top_value(all);
    const bool finite = new_max < CUDART_INF_F;
    if (finite) {
      amax = fmaxf(amax, new_max);
    } else {  // without what is not
      bits |= SGD_KV_ERR_NONFINITE;
      for (int t = mate * ROUND + at; t < count; t += t % ROUND + STEP < ROUND ? STEP : (a.team - 1) * ROUND + STEP)
        for (int e = 0; e < 8; ++e) {
          const float m = fabsf(to_f32(src[t * token + e]));
          if (m < CUDART_INF_F) amax = fmaxf(amax, m);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o));
    if (a.team > 1) {
      if (lane == 0) team_max[turn][warp] = amax;
      __syncthreads();
      for (int w = warp - mate; w < warp - mate + a.team; ++w) amax = fmaxf(amax, team_max[turn][w]);
    }
    const int e = scale_exp(amax);
    const float s_new = pow2(e), inv = pow2(-e);
    if (lane == 0 && mate == 0 && !idle) *scale = s_new;
    for (int t0 = mate * ROUND; t0 < count; t0 += a.team * ROUND) {
      if (count > a.team * ROUND) fetch(t0);
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        const int t = t0 + i * STEP + at;
        if (t >= count) continue;
        float v[8];
        x[i].get(v);
        if (!finite) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = v[j] == v[j] ? v[j] : 0.f;
        }
        *reinterpret_cast<uint2 *>(base + (g.slot + t) * D + sub * 8) = encode8(v, inv);
      }
    }
    if (g.slot > 0 && !idle && s_new != old) {
      const int n = g.slot * D / 8;
      for (int i0 = mate * 32 * 4; i0 < n; i0 += a.team * 32 * 4) {
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i0 + i * 32 + lane < n) w[i] = *reinterpret_cast<const uint2 *>(base + (i0 + i * 32 + lane) * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i0 + i * 32 + lane >= n) continue;
          float v[8];
          decode8(w[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = v[j] == v[j] ? v[j] * old : 0.f;
          *reinterpret_cast<uint2 *>(base + (i0 + i * 32 + lane) * 8) = encode8(v, inv);
        }
      }
    }
  }
  if (bits) atomicOr(a.err, bits);
}

// A warp takes one head's keys or values of a segment, 16 bytes a lane, four
// loads in flight; bound by the bytes, two thirds of them written: 64 rows of 1024
// to 8192 tokens, 8 heads of 128, 1.8 GB in all: 291 us, 6.2 TB/s.
template <int D>
constexpr int READ_ROUND = 4 * 32 * 16 / D;  // tokens of a warp's round
template <typename T, int D>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(KvReadArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = a.c.page;
  uint32_t bits = 0;
  const Segment g = segment_of(
      a.out_start, a.B, a.N, a.table, a.max_pages, a.c.num_pages, P, blockIdx.x,
      [&](int b, int count) {
        const int from = __ldg(a.from + b);
        if (from < 0 && count > 0) bits |= SGD_KV_ERR_LENGTH;  // reads as what lies past the table: 0
        return from < 0 ? PAST : min(from, PAST);
      },
      &bits);
  // outputs that no row claims
  const int claimed = min(max(__ldg(a.out_start + a.B), 0), a.N);
  if (claimed < a.N) {
    bits |= SGD_KV_ERR_LENGTH;
    const long long width = (long long)a.c.heads * D;
    for (long long i = claimed * width + ((long long)(blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * THREADS + threadIdx.x;
         i < a.N * width; i += (long long)gridDim.x * gridDim.y * gridDim.z * THREADS)
      static_cast<T *>(a.k)[i] = static_cast<T *>(a.v)[i] = from_f32<T>(0.f);
  }
  constexpr int PER = D / 16, STEP = 32 / PER, UNROLL = READ_ROUND<D> / STEP;  // 4
  const int sub = lane % PER, at = lane / PER;
  for (int hv = blockIdx.y * WARPS + warp; hv < 2 * a.c.heads; hv += gridDim.y * WARPS) {
    const bool value = hv >= a.c.heads;
    const int h = value ? hv - a.c.heads : hv;
    const long long block = (long long)max(g.page, 0) * a.c.heads + h;
    const uint8_t *base = (value ? a.c.v : a.c.k) + (block * P + g.slot) * D + sub * 16;
    const float s = g.page >= 0 ? (value ? a.c.vs : a.c.ks)[block] : 0.f;
    T *out = static_cast<T *>(value ? a.v : a.k) + ((long long)g.first * a.c.heads + h) * D + sub * 16;
    for (int t0 = blockIdx.z * READ_ROUND<D>; t0 < g.count; t0 += gridDim.z * READ_ROUND<D>) {
      uint4 raw[UNROLL];
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        const int t = t0 + i * STEP + at;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (t < g.count && g.page >= 0) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(base + t * D));
      }
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        const int t = t0 + i * STEP + at;
        if (t >= g.count) continue;
        float x[16], y[8];
        decode8(make_uint2(raw[i].x, raw[i].y), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e] * s;
        decode8(make_uint2(raw[i].z, raw[i].w), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 + e] = y[e] * s;
        T *o = out + (long long)t * a.c.heads * D;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            __stcs(reinterpret_cast<float4 *>(o) + e, make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]));
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            __stcs(reinterpret_cast<uint4 *>(o) + e,
                   make_uint4(pack2<T>(x[8 * e], x[8 * e + 1]), pack2<T>(x[8 * e + 2], x[8 * e + 3]),
                              pack2<T>(x[8 * e + 4], x[8 * e + 5]), pack2<T>(x[8 * e + 6], x[8 * e + 7])));
        }
      }
    }
  }
  if (bits) atomicOr(a.err, bits);
}

// CTAs for B rows of N tokens: a row of n tokens touches at most n / page + 2
// pages, and 1 if it is one token.
unsigned segments(int B, int N, const KvView &c) {
  const long long few = (long long)N, many = (long long)N / c.page + 2LL * B;
  return (unsigned)(few < many ? few : many);
}

template <typename T>
cudaError_t write(KvWriteArgs a, cudaStream_t st) {
  // Rows of a page's tokens or more on average, and fewer warps than the GPU holds:
  // as many warps a page and head as keep it in their registers.  Measured, teams
  // against single warps (8 heads of 128): one row of 512 tokens, pages of 128: 4.7
  // us, 17.1; of 2048, pages of 64: 4.5, 9.1; of 8192, pages of 128: 12.3, 24.5; at
  // 8 rows of up to 8192 there are warps enough without: 52, 46.  Fewer tokens than
  // a page leave most of a team idle: a step of 1 to 17 tokens with its read back
  // takes 32 us with single warps, 40 with teams of two.
  const unsigned x = segments(a.r.B, a.r.N, a.c);
  a.team = 1;
  if (a.r.N / a.r.B >= a.c.page)
    while (a.team < WARPS && a.team * 1024 < a.c.page * a.c.dim && (long long)x * 2 * a.c.heads * a.team < 152 * 32)
      a.team *= 2;
  const unsigned teams = WARPS / a.team;
  const dim3 grid(x, (2 * a.c.heads + teams - 1) / teams);
  if (a.c.dim == 128)
    kv_write_kernel<T, 128><<<grid, THREADS, 0, st>>>(a);
  else
    kv_write_kernel<T, 64><<<grid, THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t read(const KvReadArgs &a, cudaStream_t st) {
  const unsigned x = segments(a.B, a.N, a.c), y = (2 * a.c.heads + WARPS - 1) / WARPS;
  // Each CTA finds its segment first: a segment's tokens are split over CTAs
  // only where the GPU would not be full otherwise.  Measured, split against
  // whole, at pages of 128: one row of 4096 tokens, 8 heads: 7.7 us, 11.3; two of
  // 1000, 4 heads: 3.7, 10.2; at 64 rows of 1024 to 8192 there are segments enough.
  const unsigned rounds = x * y < 152 * 4 ? (a.c.page + READ_ROUND<D> - 1) / READ_ROUND<D> : 1;
  kv_read_kernel<T, D><<<dim3(x, y, rounds), THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t read(const KvReadArgs &a, cudaStream_t st) {
  return a.c.dim == 128 ? read<T, 128>(a, st) : read<T, 64>(a, st);
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs &a, int dtype, cudaStream_t st) {
  if (dtype == SGD_F32) return write<float>(a, st);
  if (dtype == SGD_F16) return write<__half>(a, st);
  return write<__nv_bfloat16>(a, st);
}

cudaError_t launch_kv_read(const KvReadArgs &a, int dtype, cudaStream_t st) {
  if (dtype == SGD_F32) return read<float>(a, st);
  if (dtype == SGD_F16) return read<__half>(a, st);
  return read<__nv_bfloat16>(a, st);
}

}  // namespace sgd
