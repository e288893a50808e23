// kv_attend_many.cu -- attention where a batch row may have more than 16 rows
// (new tokens times the query heads that share a head of keys and values), in
// units of up to 32.
//
// The mathematics is that of kv_attend.cu.  Here the 4 warps of a CTA take every
// 64-token tile together: each has 16 of its tokens for s = q . k, of all rows,
// and a quarter of the dims for o += p v, of all rows and all tokens, so that
// each byte of the cache is taken from e4m3 to f16 by one lane once for all rows
// of the unit.  The probabilities cross over through shared memory.
// Two barriers a tile: one that also tells whether any row's maximum has moved
// (else there is nothing to exchange), one before the probabilities are read.
//
// What bounds it: neither the memory nor one unit alone.  At 256 batch rows of up
// to 8 new tokens, 8 heads of 128, 4 query heads each, 1.36 GB of keys and values:
// 279 us, 4.9 TB/s.  With up to 17 new tokens, 3 units that read the same tiles:
// 430 us; ncu shows the instruction slots 46% busy and the mma.sync units 42%, with
// 16 warps an SM that wait for results of their own and, a sixth of the time, at
// the barriers.
// Measured against it, in us at 8 new tokens, 17, and 33 over 8k to 32k tokens
// (279, 430, 669 here; 280, 438, 667 before shares were cut without divisions):
//   two warps to a tile, 16 rows each, every warp converting all of it   411 611 837
//   32 rows a warp (245 registers, 8 warps an SM)                        430 670 785
//   units of 64 rows, 3 CTAs an SM (the code outgrows the instruction
//     cache; 740 for the second before cold code was moved out of the way) 309 637 722
//   units of 48 rows, 3 CTAs an SM                                       337 505 724
//   units of 32, values with no place more than keys                     323 480 725
//   one barrier a tile, its products beside the sums of the tile before  314 481 719
//   exponents relative to the maximum taken after the barrier            291 448 682
//   tcgen05 with the tiles converted into shared memory                  573 745 836
#include <math_constants.h>

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
constexpr int PER_SM = 4;  // CTAs

// A tile's cost for a warp, in about 100 instructions: the bytes to convert, and
// each 16 rows' products and probabilities.
struct KvMany {
  static constexpr int M = KV_MANY_ROWS, TILE = 64;
  __host__ __device__ static constexpr int cost(int rows) { return 1 + (rows + 15) / 16; }
};

template <int D>
struct Layout {  // of the dynamic shared memory, from a multiple of 1024
  static constexpr int HALF = KvMany::TILE * D;  // bytes of a tile's keys (or values)
  static constexpr int STAGES = 2 * 128 / D;
  static constexpr int V = STAGES * HALF;                     // values: read later, so one place more
  static constexpr int P = V + (STAGES + 1) * HALF;           // probabilities, [row][token] f16
  static constexpr int Q = P + KvMany::M * KvMany::TILE * 2;  // queries
  static constexpr int BYTES = 1024 + Q + KvMany::M * D * 2;
  static_assert(Q + KvMany::M * D * 2 >= kv_join_floats() * 4, "the parts' weights fit");
};

// The ring of tiles, loaded by warp 0, 32 looked up at a time; tiles that no row
// of the unit sees are passed over.
template <int D>
struct Ring {
  using L = Layout<D>;
  const KvAttendArgs &a;
  const KvWalk<KvMany> &w;
  const CUtensorMap *kmap, *vmap;
  uint32_t tiles, bars, &bits;
  int slot, in_slot;      // to read, to load: places of keys
  int v_slot, in_v_slot;  // of values
  uint32_t phases;        // of the places, a bit each
  int next;           // tile of the list of lane 0
  uint32_t to_load;   // of the 32, those still to load
  int y[4];           // the lane's: lines of the tile's pages in the maps

  __device__ __forceinline__ void look() {
    constexpr int PACK = 128 / D;  // tokens of a 128-byte line
    const int P = a.c.page, pages = KvMany::TILE >> a.c.page_bits;
    const bool on = w.seen(next + lane_id());
    if (on) {
      const int x = w.job.tile(next + lane_id()) * KvMany::TILE;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < pages || i == 0)
          y[i] = ((max(w.page(x, i, &bits), 0) * a.c.heads + w.h) * P + (i == 0 ? x & (P - 1) : 0)) / PACK;
    }
    to_load = __ballot_sync(FULL, on);
  }
  __device__ __forceinline__ void advance() {  // loads the next tile that is seen, if any
#pragma unroll 1
    while (to_load == 0) {
      next += 32;
      if (next >= w.t1) return;
      look();
    }
    const int i = __ffs(to_load) - 1;
    to_load &= to_load - 1;
    if (lane_id() == i) {
      const int page = min(a.c.page, KvMany::TILE), pages = KvMany::TILE >> __popc(page - 1);
      const uint32_t bar = bars + 8 * in_slot;
      bar_expect(bar, 2 * L::HALF);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (p < pages) {
          tma_load_2d(tiles + in_slot * L::HALF + p * page * D, kmap, 0, y[p], bar);
          tma_load_2d(tiles + L::V + in_v_slot * L::HALF + p * page * D, vmap, 0, y[p], bar);
        }
      }
    }
    in_slot = in_slot + 1 == L::STAGES ? 0 : in_slot + 1;
    in_v_slot = in_v_slot == L::STAGES ? 0 : in_v_slot + 1;
  }
  __device__ __forceinline__ void fill() {  // where a segment begins
    next = w.t0 - 32;
    to_load = 0;
#pragma unroll 1
    for (int i = 0; i < L::STAGES; ++i) advance();
  }
  __device__ static int lane_id() { return threadIdx.x & 31; }
};

struct Shared {
  float f[KvMany::M];
  int token[KvMany::M];  // of the row, counted from the batch row's first new one; very negative: no such row
  float of_warp[WARPS][KvMany::M];  // maxima of a tile; in the end sums
  int last;
};

// One segment of a unit with 16 MT rows at most.
template <typename T, int D, int MT>
__device__ __forceinline__ void segment(const KvAttendArgs &a, const KvWalk<KvMany> &w, Shared &sh, Ring<D> &ring) {
  using L = Layout<D>;
  constexpr int M = KvMany::M, TILE = KvMany::TILE, HALF = L::HALF;
  constexpr int KS = D / 16;  // k steps of q . k
  constexpr int NJ = D / 64;  // 16-dim groups of a warp's part of the output
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const KvJob &job = w.job;
  const int H = a.c.heads;
  const uint32_t p_at = ring.tiles + L::P, q_at = ring.tiles + L::Q;

  float o[MT][2 * NJ][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      m[mt][x] = -CUDART_INF_F;
      l[mt][x] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
  }

#pragma unroll 1
  for (int j0 = w.t0; j0 < w.t1; j0 += 32) {
    float ks = 0.f, lv = 0.f, iv = 1.f;  // of the warp's 16 tokens: scale of keys (0: no such page), log2 V, 1 / V
    const bool on = w.seen(j0 + lane);
    if (on) {
      const int pg = w.page(job.tile(j0 + lane) * TILE + 16 * warp, 0, &ring.bits);
      if (pg >= 0) {
        ks = __ldg(a.c.ks + (long long)pg * H + w.h);
        const float vs = __ldg(a.c.vs + (long long)pg * H + w.h);
        lv = log2_scale(vs);
        iv = inverse_scale(vs);
      }
    }
#pragma unroll 1
    for (uint32_t todo = __ballot_sync(FULL, on); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int x0 = job.tile(j0 + src) * TILE, mine = x0 + 16 * warp;
      const float kh = __shfl_sync(FULL, ks, src), lh = __shfl_sync(FULL, lv, src), ih = __shfl_sync(FULL, iv, src);
      const uint32_t kt = ring.tiles + ring.slot * HALF, vt = ring.tiles + L::V + ring.v_slot * HALF;
      if (!bar_wait(ring.bars + 8 * ring.slot, ring.phases >> ring.slot & 1)) ring.bits |= SGD_KV_ERR_WAIT;
      // ---- s = q . k: rows g, g + 8 of each 16; tokens 16 warp + 8 nt + 2 c, + 1
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
        uint4 kw[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int t = warp * 16 + nt * 8 + g;
          if (D == 128)
            kw[nt] = lds128(kt + t * 128 + (((2 * c + ch) ^ (t & 7)) << 4));
          else
            kw[nt] = lds128(kt + (t >> 1) * 128 + ((((t & 1) * 4 + c) ^ ((t >> 1) & 7)) << 4));
        }
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t b[2][2];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            e4m3x4_to_f16x4(q4 == 0 ? kw[nt].x : q4 == 1 ? kw[nt].y : q4 == 2 ? kw[nt].z : kw[nt].w, b[nt][0], b[nt][1]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 v = lds128(q_at + ((mt * KS + ch * 4 + q4) * 32 + lane) * 16);
            const uint32_t qa[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) mma(s[mt][nt], qa, b[nt][0], b[nt][1]);
          }
        }
      }
      // ---- scales and masks: s becomes the exponent of the probability
      float limit[MT][2];  // beyond it the row's maximum has moved
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool fresh = m[mt][x] == -CUDART_INF_F;
          const float f = sh.f[mt * 16 + x * 8 + g] * kh, plus = lh + (LIFT - (fresh ? 0.f : m[mt][x]));
          limit[mt][x] = fresh ? -CUDART_INF_F : LIFT + LAZY;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[mt][nt][2 * x + e] = fmaf(s[mt][nt][2 * x + e], f, plus);
        }
      const bool missing = kh == 0.f;
      if (__builtin_expect(missing || w.edge(x0), 0)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int p = missing ? -1 : job.n - job.ql + sh.token[mt * 16 + x * 8 + g];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int t = mine + nt * 8 + 2 * c + e;
                const bool vis = t <= p && (a.window == 0 || t > p - a.window || t < a.sinks);
                if (!vis) s[mt][nt][2 * x + e] = -CUDART_INF_F;
              }
          }
        }
      }
      // Values of slots that no token has reached may be anything, NaN among it:
      // they count as 0.
      if (__builtin_expect(missing || mine + 16 > job.n, 0)) {
        const int t = 16 * warp + (lane >> 1);
        if (missing || x0 + t >= job.n) {
          const uint32_t line = D == 128 ? vt + t * 128 : vt + (t >> 1) * 128;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int ch = (lane & 1) * (D / 32) + i;
            const int at16 = D == 128 ? ch : (((t & 1) * 4 + ch) ^ ((t >> 1) & 7));
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(line + at16 * 16), "r"(0) : "memory");
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      // ---- maxima
      float top[MT][2];
      bool moves = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[mt][x] = fmaxf(fmaxf(s[mt][0][2 * x], s[mt][0][2 * x + 1]), fmaxf(s[mt][1][2 * x], s[mt][1][2 * x + 1]));
          moves = moves || top[mt][x] > limit[mt][x];
        }
      if (__builtin_expect(__syncthreads_or(moves), 0)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float v = top[mt][x];
            v = fmaxf(v, __shfl_xor_sync(FULL, v, 1));
            v = fmaxf(v, __shfl_xor_sync(FULL, v, 2));
            if (c == 0) sh.of_warp[warp][mt * 16 + x * 8 + g] = v;
          }
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = mt * 16 + x * 8 + g;
            const float v = fmaxf(fmaxf(sh.of_warp[0][r], sh.of_warp[1][r]), fmaxf(sh.of_warp[2][r], sh.of_warp[3][r]));
            if (v > limit[mt][x]) {
              const bool fresh = m[mt][x] == -CUDART_INF_F;
              const float by = LIFT - v;  // what the exponents change by
              const float k = fresh ? 0.f : ex2_approx(by);
              m[mt][x] = (fresh ? 0.f : m[mt][x]) - by;
              l[mt][x] *= k;
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                s[mt][nt][2 * x] += by;
                s[mt][nt][2 * x + 1] += by;
              }
#pragma unroll
              for (int n = 0; n < 2 * NJ; ++n) {
                o[mt][n][2 * x] *= k;
                o[mt][n][2 * x + 1] *= k;
              }
            }
          }
      }
      // (all warps have read the keys, and the values of the tile before: their places are free)
      if (warp == 0) ring.advance();
      // ---- probabilities, to where all warps read them
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t line = p_at + (mt * 16 + x * 8 + g) * 128 + 4 * c;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const float p0 = ex2_approx(s[mt][nt][2 * x]), p1 = ex2_approx(s[mt][nt][2 * x + 1]);
            l[mt][x] = fmaf(p0 + p1, ih, l[mt][x]);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(line + (((2 * warp + nt) ^ g) << 4)), "r"(pack2<__half>(p0, p1))
                         : "memory");
          }
        }
      __syncthreads();
      // ---- o += p v: dims 16 (NJ warp + j) + 4 c .. + 3 of rows g, g + 8
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t x[NJ][4];
        const int t = half * 32 + lane;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int jd = warp * NJ + j;
          if (D == 128)
            ldmatrix_x4_trans(x[j], vt + t * 128 + ((jd ^ (t & 7)) << 4));
          else
            ldmatrix_x4_trans(x[j], vt + (t >> 1) * 128 + ((((t & 1) * 4 + jd) ^ ((t >> 1) & 7)) << 4));
        }
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) {
          uint32_t even[NJ][2], odd[NJ][2];
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              e4m3x4_to_f16x4(__byte_perm(x[j][2 * kc + i], 0, 0x3120), even[j][i], odd[j][i]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int r = mt * 16 + (lane & 15), ch = half * 4 + kc * 2 + (lane >> 4);
            uint32_t pa[4];
            ldmatrix_x4(pa, p_at + r * 128 + ((ch ^ (r & 7)) << 4));
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              mma(o[mt][2 * j], pa, even[j][0], even[j][1]);
              mma(o[mt][2 * j + 1], pa, odd[j][0], odd[j][1]);
            }
          }
        }
      }
      ring.phases ^= 1u << ring.slot;
      ring.slot = ring.slot + 1 == L::STAGES ? 0 : ring.slot + 1;
      ring.v_slot = ring.v_slot == L::STAGES ? 0 : ring.v_slot + 1;
    }
  }

  // ---- the sums of the warps' tokens together
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float v = l[mt][x];
      v += __shfl_xor_sync(FULL, v, 1);
      v += __shfl_xor_sync(FULL, v, 2);
      if (c == 0) sh.of_warp[warp][mt * 16 + x * 8 + g] = v;
    }
  __syncthreads();  // (the ring is drained)
  const bool whole = w.whole();
  float *part = part_of<M, D>(a, 2 * blockIdx.x + (w.starts() ? 1 : 0));
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = mt * 16 + x * 8 + g;
      if (r < w.nrows) {
        const float sum = (sh.of_warp[0][r] + sh.of_warp[1][r]) + (sh.of_warp[2][r] + sh.of_warp[3][r]);
        const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        const int token = sh.token[r];
        const long long row = (long long)(job.q0 + token) * a.q_heads + w.h * a.group + (w.r0 + r - token * a.group);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int d = (warp * NJ + j) * 16 + 4 * c;
          const float4 v = make_float4(o[mt][2 * j][2 * x] * inv, o[mt][2 * j + 1][2 * x] * inv,
                                       o[mt][2 * j][2 * x + 1] * inv, o[mt][2 * j + 1][2 * x + 1] * inv);
          if (whole)
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * D + d) =
                make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
          else
            *reinterpret_cast<float4 *>(part + r * D + d) = v;
        }
        if (!whole && warp == 0 && c == 0) {
          part[M * D + r] = m[mt][x];
          part[M * D + M + r] = sum;
        }
      }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, PER_SM)
    attend_many_kernel(KvAttendArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using L = Layout<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) unsigned long long bars[L::STAGES];
  __shared__ Shared sh;
  uint32_t bits = 0;
  const KvShare share = kv_share<KvMany, THREADS>(a, 2 * KvMany::cost(KvMany::M), &bits);
  if (share.begin >= share.end) {
    if (bits) atomicOr(a.err, bits);  // (each thread looked at rows of its own)
    return;
  }
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::STAGES; ++i) bar_init(smem_addr(bars) + 8 * i, 1);
    bar_init_fence();
  }
  __syncthreads();
  KvWalk<KvMany> w(a, share);
  Ring<D> ring = {a, w, &kmap, &vmap, smem_addr(smem), smem_addr(bars), bits, 0, 0, 0, 0, 0, 0, 0, {0, 0, 0, 0}};
#pragma unroll 1
  while (w.next(&bits)) {
    if (threadIdx.x < 32) ring.fill();
    kv_queries<T, D, KvMany::M, WARPS>(a, w, ring.tiles + L::Q, sh.f);
    const int r = threadIdx.x;
    if (r < KvMany::M) sh.token[r] = r < w.nrows ? (w.r0 + r) / a.group : -(1 << 30);
    __syncthreads();
    if (w.nrows > 16)
      segment<T, D, 2>(a, w, sh, ring);
    else
      segment<T, D, 1>(a, w, sh, ring);
    if (!w.whole()) kv_join<T, KvMany, D, THREADS>(a, share, w, reinterpret_cast<float *>(smem), &sh.last);
    // (generic reads and writes of the ring's memory come before the next copies into it)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  if (bits) atomicOr(a.err, bits);
}

// ---- host --------------------------------------------------------------------

template <typename T, int D>
cudaError_t launch(const KvAttendArgs &a, cudaStream_t st) {
  CUtensorMap k, v;
  const int tokens = a.c.page < KvMany::TILE ? a.c.page : KvMany::TILE;
  if (!kv_make_map(&k, a.c, a.c.k, tokens) || !kv_make_map(&v, a.c, a.c.v, tokens)) return cudaErrorInvalidValue;
  const int sms = a.sms < MAX_CTAS / PER_SM ? a.sms : MAX_CTAS / PER_SM;
  attend_many_kernel<T, D><<<sms * PER_SM, THREADS, Layout<D>::BYTES, st>>>(a, k, v);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t limit() {
  return cudaFuncSetAttribute(attend_many_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::BYTES);
}

}  // namespace

cudaError_t attend_many_limits() {
  cudaError_t e = limit<__half, 128>();
  if (e == cudaSuccess) e = limit<__half, 64>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 64>();
  return e;
}

cudaError_t launch_attend_many(const KvAttendArgs &a, int dtype, cudaStream_t st) {
  if (a.c.dim == 128) return dtype == SGD_F16 ? launch<__half, 128>(a, st) : launch<__nv_bfloat16, 128>(a, st);
  return dtype == SGD_F16 ? launch<__half, 64>(a, st) : launch<__nv_bfloat16, 64>(a, st);
}

}  // namespace sgd
