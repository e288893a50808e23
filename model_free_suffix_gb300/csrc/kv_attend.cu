// kv_attend.cu -- attention of each row's new tokens over the paged 8-bit cache.
//
//   o_r = sum_j softmax_j(scale q_r . k_j) v_j   over the positions j that row
//   r's token, at position p, sees: j <= p, and with a window j > p - window or
//   j < sinks.
//
// One pass over keys and values with a running maximum m and sum l per row: a
// tile's products s give m' = max(m, max s), and l and o are scaled by
// 2^(m - m') before the tile's 2^(s - m') are added (kv_attend.cuh has the
// scales of the blocks, and when this scaling is due).
// Rows of the query heads that share a head of keys and values go together, so
// that each byte of the cache is read once for all rows of a unit (16 here).
//
// Bound by reading the cache: at 256 batch rows of one token over 1024 to 4096
// cached ones, 8 heads of 128, 1.35 GB: 228 us, 5.9 TB/s, with 8 query heads a
// head of keys; 232 us with 4 new tokens and 4 query heads (16 rows).  At a dim
// of 64 and pages of 16, 1.08 GB: 197 us, 5.5 TB/s (a tile is half the bytes for
// the same softmax, and comes from two pages).  A window of 2048 over up to 16k
// tokens, 128 batch rows: 69 us, 3.9 TB/s.  One row of 2000 tokens: 17 us, of
// which the work is 1; the rest is a chain of loads, and joining the parts.
// The work is cut into equal shares wherever a cut falls since whole units leave
// the last ones running alone; 4 warps a CTA have rings of their own since they
// then never wait for one another, 3 CTAs an SM (64 KB of loads in flight each),
// at a dim of 64, where registers allow it, 4 (before a later gain: 203 and 72 us
// against 207 and 76; with tiles of 64 tokens there instead, 200 and 84: fewer,
// larger pieces to share).
#include <math_constants.h>

#include <type_traits>

#include "async_copy.cuh"
#include "kv_attend.cuh"
#include "kv_internal.h"
#include "kv_sched.cuh"
#include "num_types.cuh"
#include "sgd_internal.h"

namespace sgd {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int KV_TILE = 32;  // tokens
template <int D>
constexpr int PER_SM = D == 128 ? 3 : 4;  // CTAs
constexpr int M = 16;        // rows of a unit

struct KvFew {
  static constexpr int M = 16, TILE = KV_TILE;
  __host__ __device__ static constexpr int cost(int) { return 1; }
};

// Each warp keeps m, l and o of the unit's 16 rows in registers and streams its
// own 32-token tiles through its own ring of TMA loads; the warps meet where a
// unit ends.
//
// e4m3 is taken to f16, exactly, on the way into the registers that feed the
// matrix instructions, so the products carry no rounding of the cache's.  q goes
// to f16 after each row is scaled by a power of two that brings its largest
// element to [1, 2): exact down to 2^-17 of it for bf16 and 2^-14 for f16, where
// f16's last place is 2^-24; smaller elements move by 2^-25 at most.  The
// probabilities go to f16 (relative 2^-12 each; the sum l is taken before that
// rounding).
//
// The order of the elements of a product's long axis is free as long as both
// sides use the same: a lane takes 2 (D = 128) or 1 (D = 64) whole 16-byte
// chunks of a key, so all shared-memory reads are 16 bytes wide and, with the
// 128-byte swizzle of the TMA load, without bank conflicts.
template <typename T, int D, int S>
__global__ void __launch_bounds__(THREADS, PER_SM<D>)
    attend_kernel(KvAttendArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int HALF = KV_TILE * D;          // bytes of a tile's keys (or values)
  constexpr int NJ = D / 16;                 // 16-dim groups of the output
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  __shared__ __align__(8) unsigned long long bars[WARPS * S];
  __shared__ float s_f[M];
  __shared__ float s_m[WARPS][16], s_l[WARPS][16];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  uint32_t bits = 0;
  const KvShare share = kv_share<KvFew, THREADS>(a, WARPS, &bits);
  if (share.begin >= share.end) {
    if (bits) atomicOr(a.err, bits);  // (each thread looked at rows of its own)
    return;
  }
  const uint32_t q_at = smem_addr(smem) + WARPS * S * 2 * HALF;
  const uint32_t ring = smem_addr(smem) + warp * S * 2 * HALF, bar0 = smem_addr(bars) + warp * S * 8;
  if (tid == 0) {
    for (int i = 0; i < WARPS * S; ++i) bar_init(smem_addr(bars) + 8 * i, 1);
    bar_init_fence();
  }
  __syncthreads();

  const int P = a.c.page, H = a.c.heads;
  const int halves = P < KV_TILE ? 2 : 1;  // pages of a tile
  uint32_t phases = 0;  // of the ring's slots, a bit each
  KvWalk<KvFew> w(a, share);
#pragma unroll 1
  while (w.next(&bits)) {
    const KvJob &job = w.job;
    const int h = w.h, nrows = w.nrows, t0 = w.t0, t1 = w.t1;

    int in_slot = 0, out_slot = 0;  // to load, to consume

    // ---- tiles t0 + warp, + WARPS, ..., 32 at a time: lane i holds
    // what the i-th of them needs.  Those that no row of the unit sees are
    // passed over.
    struct Ahead {
      int y[2];   // lines of the tile's page(s) in the maps
      bool on;    // some row sees it
    };
    constexpr int PACK = 128 / D;  // tokens of a 128-byte line
    auto look = [&](int j, Ahead &t) {
      t.on = w.seen(j);
      t.y[0] = t.y[1] = 0;
      if (t.on) {
        const int x = job.tile(j) * KV_TILE;
        t.y[0] = ((max(w.page(x, 0, &bits), 0) * H + h) * P + (x & (P - 1))) / PACK;
        if (halves == 2) t.y[1] = (max(w.page(x, 1, &bits), 0) * H + h) * P / PACK;
      }
      return __ballot_sync(FULL, t.on);
    };
    Ahead ahead;
    int next = t0 + warp;  // the first tile of the batch being loaded
    uint32_t to_load = look(next + WARPS * lane, ahead);
    auto advance = [&]() {  // loads the next tile that is seen, if any
#pragma unroll 1
      while (to_load == 0) {
        next += 32 * WARPS;
        if (next >= t1) return;
        to_load = look(next + WARPS * lane, ahead);
      }
      const int i = __ffs(to_load) - 1;
      to_load &= to_load - 1;
      if (lane == i) {
        const uint32_t dst = ring + in_slot * 2 * HALF, bar = bar0 + 8 * in_slot;
        bar_expect(bar, 2 * HALF);
        tma_load_2d(dst, &kmap, 0, ahead.y[0], bar);
        tma_load_2d(dst + HALF, &vmap, 0, ahead.y[0], bar);
        if (halves == 2) {
          tma_load_2d(dst + HALF / 2, &kmap, 0, ahead.y[1], bar);
          tma_load_2d(dst + HALF + HALF / 2, &vmap, 0, ahead.y[1], bar);
        }
      }
      in_slot = in_slot + 1 == S ? 0 : in_slot + 1;
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) advance();

    kv_queries<T, D, M, WARPS>(a, w, q_at, s_f);
    __syncthreads();

    float o[2 * NJ][4];
    float m[2], l[2], f[2];
    int pos[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = x * 8 + g;
      m[x] = -CUDART_INF_F;
      l[x] = 0.f;
      f[x] = s_f[r];
      pos[x] = r < nrows ? job.n - job.ql + (w.r0 + r) / a.group : -1;
    }
#pragma unroll
    for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

#pragma unroll 1
    for (int j0 = t0 + warp; j0 < t1; j0 += 32 * WARPS) {
    float ks[2] = {0.f, 0.f};           // (a scale of 0: no such page)
    float lv[2] = {0.f, 0.f}, iv[2] = {1.f, 1.f};  // log2 V, 1 / V
    bool on = w.seen(j0 + WARPS * lane);
    if (on) {
      const int x = job.tile(j0 + WARPS * lane) * KV_TILE;
      for (int i = 0; i < halves; ++i) {
        const int pg = w.page(x, i, &bits);
        if (pg >= 0) {
          ks[i] = __ldg(a.c.ks + (long long)pg * H + h);
          const float vs = __ldg(a.c.vs + (long long)pg * H + h);
          lv[i] = log2_scale(vs);
          iv[i] = inverse_scale(vs);
        }
      }
      if (halves == 1) {
        ks[1] = ks[0];
        lv[1] = lv[0];
        iv[1] = iv[0];
      }
    }
#pragma unroll 1
    for (uint32_t todo = __ballot_sync(FULL, on); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int x0 = job.tile(j0 + WARPS * src) * KV_TILE;
      const float kh[2] = {__shfl_sync(FULL, ks[0], src), __shfl_sync(FULL, ks[1], src)};
      const float lh[2] = {__shfl_sync(FULL, lv[0], src), __shfl_sync(FULL, lv[1], src)};
      const float ih[2] = {__shfl_sync(FULL, iv[0], src), __shfl_sync(FULL, iv[1], src)};
      const uint32_t kt = ring + out_slot * 2 * HALF, vt = kt + HALF;
      if (!bar_wait(bar0 + 8 * out_slot, phases >> out_slot & 1)) bits |= SGD_KV_ERR_WAIT;
      // ---- s = q . k: rows g, g + 8; tokens 8 nt + 2 c, + 1
      float s[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
        uint4 kw[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int t = nt * 8 + g;
          if (D == 128)
            kw[nt] = lds128(kt + t * 128 + (((2 * c + ch) ^ (t & 7)) << 4));
          else
            kw[nt] = lds128(kt + (t >> 1) * 128 + ((((t & 1) * 4 + c) ^ ((t >> 1) & 7)) << 4));
        }
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const uint4 v = lds128(q_at + ((ch * 4 + q4) * 32 + lane) * 16);
          const uint32_t qa[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const uint32_t four = q4 == 0 ? kw[nt].x : q4 == 1 ? kw[nt].y : q4 == 2 ? kw[nt].z : kw[nt].w;
            uint32_t b0, b1;
            e4m3x4_to_f16x4(four, b0, b1);
            mma(s[nt], qa, b0, b1);
          }
        }
      }
      // ---- scales and masks: s becomes the exponent of the probability
      const bool missing = kh[0] == 0.f || kh[1] == 0.f;
      float limit[2];  // beyond it the row's maximum has moved
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool fresh = m[x] == -CUDART_INF_F;
        const float base = LIFT - (fresh ? 0.f : m[x]);
        limit[x] = fresh ? -CUDART_INF_F : LIFT + LAZY;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            s[nt][2 * x + e] = fmaf(s[nt][2 * x + e], f[x] * kh[nt >> 1], lh[nt >> 1] + base);
      }
      if (__builtin_expect(missing || w.edge(x0), 0)) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = x0 + nt * 8 + 2 * c + (e & 1), p = pos[e >> 1];
            const bool vis = x <= p && kh[nt >> 1] != 0.f && (a.window == 0 || x > p - a.window || x < a.sinks);
            if (!vis) s[nt][e] = -CUDART_INF_F;
          }
      }
      // ---- maxima
      float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[nt][e]);
      if (__builtin_expect(__any_sync(FULL, top[0] > limit[0] || top[1] > limit[1]), 0)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = fmaxf(top[x], __shfl_xor_sync(FULL, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(FULL, top[x], 2));
          if (top[x] > limit[x]) {
            const bool fresh = m[x] == -CUDART_INF_F;
            const float by = LIFT - top[x];  // what the exponents change by
            const float k = fresh ? 0.f : ex2_approx(by);
            m[x] = (fresh ? 0.f : m[x]) - by;
            l[x] *= k;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
              s[nt][2 * x] += by;
              s[nt][2 * x + 1] += by;
            }
#pragma unroll
            for (int n = 0; n < 2 * NJ; ++n) {
              o[n][2 * x] *= k;
              o[n][2 * x + 1] *= k;
            }
          }
        }
      }
      // ---- probabilities
      uint32_t pa[2][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] = ex2_approx(s[nt][e]);
          l[e >> 1] = fmaf(s[nt][e], ih[nt >> 1], l[e >> 1]);
        }
        pa[nt >> 1][(nt & 1) * 2] = pack2<__half>(s[nt][0], s[nt][1]);
        pa[nt >> 1][(nt & 1) * 2 + 1] = pack2<__half>(s[nt][2], s[nt][3]);
      }
      // ---- o += p v: dims 16 j + 4 c .. + 3 of rows g, g + 8.  Slots that no
      // token has reached may hold anything, NaN among it: they count as 0.
      if (__builtin_expect(missing || x0 + KV_TILE > job.n, 0)) {
        __syncwarp();
        const bool gone = (lane < 16 ? kh[0] : kh[1]) == 0.f || x0 + lane >= job.n;
        if (gone) {
          const uint32_t line = D == 128 ? vt + lane * 128 : vt + (lane >> 1) * 128;
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch) {
            const int at16 = D == 128 ? ch : (((lane & 1) * 4 + ch) ^ ((lane >> 1) & 7));
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(line + at16 * 16), "r"(0) : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
      }
#pragma unroll
      for (int jd = 0; jd < NJ; ++jd) {
        const int t = (lane >> 3) * 8 + (lane & 7);
        uint32_t x[4];
        if (D == 128)
          ldmatrix_x4_trans(x, vt + t * 128 + ((jd ^ (t & 7)) << 4));
        else
          ldmatrix_x4_trans(x, vt + (t >> 1) * 128 + ((((t & 1) * 4 + jd) ^ ((t >> 1) & 7)) << 4));
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) {
          uint32_t even[2], odd[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) e4m3x4_to_f16x4(__byte_perm(x[2 * kc + i], 0, 0x3120), even[i], odd[i]);
          mma(o[2 * jd], pa[kc], even[0], even[1]);
          mma(o[2 * jd + 1], pa[kc], odd[0], odd[1]);
        }
      }
      phases ^= 1u << out_slot;
      out_slot = out_slot + 1 == S ? 0 : out_slot + 1;
      __syncwarp();
      advance();
    }
    }

    // ---- the warps' parts together
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float sum = l[x];
      sum += __shfl_xor_sync(FULL, sum, 1);
      sum += __shfl_xor_sync(FULL, sum, 2);
      if (c == 0) {
        s_m[warp][x * 8 + g] = m[x];
        s_l[warp][x * 8 + g] = sum;
      }
    }
    __syncthreads();  // (every ring is drained)
    float *so = reinterpret_cast<float *>(smem) + warp * 16 * D;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = x * 8 + g;
      if (r < nrows) {
#pragma unroll
        for (int jd = 0; jd < NJ; ++jd)
          *reinterpret_cast<float4 *>(so + r * D + jd * 16 + 4 * c) = make_float4(
              o[2 * jd][2 * x], o[2 * jd + 1][2 * x], o[2 * jd][2 * x + 1], o[2 * jd + 1][2 * x + 1]);
      }
    }
    __syncthreads();
    const bool whole = w.whole();
    T *out = static_cast<T *>(a.out);
    float *part = part_of<M, D>(a, 2 * blockIdx.x + (w.starts() ? 1 : 0));
    const float *all = reinterpret_cast<const float *>(smem);
#pragma unroll 1
    for (int i = tid; i < nrows * (D / 4); i += THREADS) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int i2 = 0; i2 < WARPS; ++i2) top = fmaxf(top, s_m[i2][r]);
      const float base = top == -CUDART_INF_F ? 0.f : top;
      float sum = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i2 = 0; i2 < WARPS; ++i2) {
        const float k = ex2_approx(s_m[i2][r] - base);
        const float4 v = *reinterpret_cast<const float4 *>(all + (i2 * 16 + r) * D + d);
        if (s_l[i2][r] != 0.f) {
          sum += s_l[i2][r] * k;
          x.x += v.x * k;
          x.y += v.y * k;
          x.z += v.z * k;
          x.w += v.w * k;
        }
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        T *dst = out + ((long long)w.token(r) * a.q_heads + w.q_head(r)) * D + d;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(x.x * inv, x.y * inv), pack2<T>(x.z * inv, x.w * inv));
      } else {
        *reinterpret_cast<float4 *>(part + r * D + d) = x;
        if (d == 0) {
          part[M * D + r] = top;
          part[M * D + M + r] = sum;
        }
      }
    }
    if (!whole) {
      kv_join<T, KvFew, D, THREADS>(a, share, w, reinterpret_cast<float *>(smem), &s_last);
    }
    // (generic reads and writes of the ring's memory come before the next copies into it)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  if (bits) atomicOr(a.err, bits);
}

// ---- host --------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return (EncodeTiled) nullptr;
    }
    return (EncodeTiled)p;
  }();
  return fn;
}

}  // namespace

bool kv_make_map(CUtensorMap *map, const KvView &c, void *base, int tokens) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t lines = (cuuint64_t)c.num_pages * c.heads * c.page * c.dim / 128;
  const cuuint64_t dims[2] = {128, lines}, strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)(tokens * c.dim / 128)}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool kv_make_token_map(CUtensorMap *map, const void *base, int dim, int heads, int N, long long head_stride,
                       long long token_stride, int tokens) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  // (of one head, or one token, the stride means nothing and may be anything)
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)N};
  const cuuint64_t strides[2] = {(cuuint64_t)(heads == 1 ? dim : head_stride) * 2, (cuuint64_t)(N == 1 ? dim : token_stride) * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)tokens}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

template <int D, int S>
constexpr int smem_bytes() {
  static_assert(WARPS * S * 2 * KV_TILE * D >= kv_join_floats() * 4, "the parts' weights fit the ring");
  return 1024 + WARPS * S * 2 * KV_TILE * D + D / 16 * 512;
}

template <typename T, int D, int S>
cudaError_t launch(const KvAttendArgs &a, cudaStream_t st) {
  CUtensorMap k, v;
  const int tokens = a.c.page < KV_TILE ? a.c.page : KV_TILE;
  if (!kv_make_map(&k, a.c, a.c.k, tokens) || !kv_make_map(&v, a.c, a.c.v, tokens)) return cudaErrorInvalidValue;
  const int sms = a.sms < MAX_CTAS / PER_SM<D> ? a.sms : MAX_CTAS / PER_SM<D>;
  attend_kernel<T, D, S><<<sms * PER_SM<D>, THREADS, smem_bytes<D, S>(), st>>>(a, k, v);
  return cudaGetLastError();
}

template <typename T, int D, int S>
cudaError_t limit() {
  return cudaFuncSetAttribute(attend_kernel<T, D, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D, S>());
}

template <typename T>
cudaError_t attend(const KvAttendArgs &a, cudaStream_t st) {
  return a.c.dim == 128 ? launch<T, 128, 2>(a, st) : launch<T, 64, 3>(a, st);
}

}  // namespace

size_t kv_attend_workspace() { return (size_t)MAX_CTAS * 8 + (size_t)MAX_CTAS * 2 * KV_MANY_ROWS * (128 + 2) * 4; }

cudaError_t kv_attend_set_limits() {
  cudaError_t e = limit<__half, 128, 2>();
  if (e == cudaSuccess) e = limit<__half, 64, 3>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 128, 2>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 64, 3>();
  if (e == cudaSuccess) e = attend_many_limits();
  return e;
}

cudaError_t launch_kv_attend(KvAttendArgs a, int dtype, cudaStream_t st, int *launches) {
  *launches = 1;
  // Up to 16 rows a batch row and head, a tile a warp (this file); beyond, a tile
  // a CTA.  Measured, this against the other, at up to 16 rows: at a dim of 64 with
  // pages of 16 197 us, 271, with a window of 2048 69, 90; at 128, a window of 2048
  // over pages of 16 186, 207; without a window 1 to 3% apart either way (one row
  // of 2000 tokens 17, 17, 256 rows of one token and 8 query heads 228, 224), a
  // window of 256 over pages of 64 67, 60.  At 32 rows two warps to a tile took 411
  // against 279.  (max_q only chooses: each takes any number of rows.)
  if ((long long)a.max_q * a.group > M) return launch_attend_many(a, dtype, st);
  return dtype == SGD_F16 ? attend<__half>(a, st) : attend<__nv_bfloat16>(a, st);
}

}  // namespace sgd
