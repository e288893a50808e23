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
// that each byte of the cache is read once for all of them.
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

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Few rows (M = 16 MT <= 32 a unit), bound by reading the cache.  Each warp
// streams its own 32-token tiles through a ring of TMA loads, S deep, and keeps
// m, l and o of all the unit's rows in registers; warps meet only where a unit
// ends.  e4m3 is taken to f16, exactly, on the way into the registers that
// feed the matrix instructions, so the products carry no rounding of the
// cache's; q goes to f16 after each row is scaled to [1, 2) by a power of two
// (bf16 has fewer bits than f16: only elements 2^-24 times the row's largest
// lose any), and the probabilities to f16 (relative 2^-12 each; the sum l is
// taken before that rounding).
//
// The order of the elements of a product's long axis is free as long as both
// sides use the same: a lane takes 2 (D = 128) or 1 (D = 64) whole 16-byte
// chunks of a key, so all shared-memory reads are 16 bytes wide and, with the
// 128-byte swizzle of the TMA load, without bank conflicts.
template <typename T, int D, int MT, int S>
__global__ void __launch_bounds__(THREADS) attend_few_kernel(KvAttendArgs a, const __grid_constant__ CUtensorMap kmap,
                                                             const __grid_constant__ CUtensorMap vmap) {
  constexpr int M = 16 * MT;
  constexpr int KS = D / 16;                 // k steps of q . k
  constexpr int HALF = KV_TILE * D;          // bytes of a tile's keys (or values)
  constexpr int NJ = D / 16;                 // 16-dim groups of the output
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  __shared__ __align__(8) unsigned long long bars[WARPS * S];
  __shared__ float s_f[M];
  __shared__ float s_m[WARPS][M], s_l[WARPS][M];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  uint32_t bits = 0;
  const KvShare share = kv_share<THREADS, M, KV_TILE>(a, WARPS, &bits);
  if (share.begin >= share.end) {
    if (bits && tid == 0) atomicOr(a.err, bits);
    return;
  }
  const uint32_t ring = smem_addr(smem) + warp * S * 2 * HALF;
  const uint32_t q_at = smem_addr(smem) + WARPS * S * 2 * HALF;
  const uint32_t bar0 = smem_addr(bars) + warp * S * 8;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) bar_init(bar0 + 8 * i, 1);
    bar_init_fence();
  }
  __syncwarp();
  uint32_t in_slot = 0, out_slot = 0, parity = 0;  // of the ring: to load, to consume

  const int P = a.c.page, H = a.c.heads;
  const int halves = P < KV_TILE ? 2 : 1;  // pages of a tile
  KvWalk<M, KV_TILE> w(a, share, &bits);
  while (w.next(&bits)) {
    const KvJob &job = w.job;
    const int h = w.h, nrows = w.nrows, t0 = w.t0, t1 = w.t1, p_first = w.p_first, p_last = w.p_last;

    // ---- this warp's tiles, t0 + warp, + WARPS, ..., 32 at a time: lane i holds
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
    for (int i = 0; i < S; ++i) advance();

    // ---- the unit's queries, as the matrix instructions take them
    for (int r = warp; r < M; r += WARPS) {
      const bool on = r < nrows;
      const T *q = static_cast<const T *>(a.q) + w.token(r) * a.q_token + w.q_head(r) * a.q_head;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      const bool mine = lane * 4 < D;
      if (on && mine) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = to_f32(q[lane * 4 + e]);
      }
      float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
      bool bad = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) bad = bad || !(fabsf(x[e]) < CUDART_INF_F);
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
      const bool poison = __any_sync(FULL, bad);  // (a bad element makes its row NaN)
      const int e2 = max((int)(__float_as_uint(top) >> 23) - 127, -100);
      const float inv = poison ? CUDART_NAN_F : pow2(-min(e2, 126));
      if (lane == 0) s_f[r] = a.scale * LOG2E * pow2(min(e2, 126));
      if (mine) {
        constexpr int DPT = D / 4;  // dims of a lane
        const int d = lane * 4, qc = d / DPT, s = d % DPT / 4;
        const uint32_t to = q_at + (((r / 16) * KS + s) * 32 + (r % 8) * 4 + qc) * 16 + (r % 16) / 8 * 4;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(pack2<__half>(x[0] * inv, x[1] * inv)) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + 8), "r"(pack2<__half>(x[2] * inv, x[3] * inv)) : "memory");
      }
    }
    __syncthreads();

    float o[MT][2 * NJ][4];
    float m[MT][2], l[MT][2], f[MT][2];
    int pos[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = mt * 16 + x * 8 + g;
        m[mt][x] = -CUDART_INF_F;
        l[mt][x] = 0.f;
        f[mt][x] = s_f[r];
        pos[mt][x] = r < nrows ? job.n - job.ql + (w.r0 + r) / a.group : -1;
      }
#pragma unroll
      for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
    }

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
          iv[i] = 1.f / vs;
        }
      }
      if (halves == 1) {
        ks[1] = ks[0];
        lv[1] = lv[0];
        iv[1] = iv[0];
      }
    }
    for (uint32_t todo = __ballot_sync(FULL, on); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int x0 = job.tile(j0 + WARPS * src) * KV_TILE;
      const float kh[2] = {__shfl_sync(FULL, ks[0], src), __shfl_sync(FULL, ks[1], src)};
      const float lh[2] = {__shfl_sync(FULL, lv[0], src), __shfl_sync(FULL, lv[1], src)};
      const float ih[2] = {__shfl_sync(FULL, iv[0], src), __shfl_sync(FULL, iv[1], src)};
      const uint32_t kt = ring + out_slot * 2 * HALF, vt = kt + HALF;
      if (!bar_wait(bar0 + 8 * out_slot, parity)) bits |= SGD_KV_ERR_WAIT;
      // ---- s = q . k: rows g, g + 8; tokens 8 nt + 2 c, + 1
      float s[MT][4][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
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
          uint32_t qa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 v = lds128(q_at + ((mt * KS + ch * 4 + q4) * 32 + lane) * 16);
            qa[mt][0] = v.x;
            qa[mt][1] = v.y;
            qa[mt][2] = v.z;
            qa[mt][3] = v.w;
          }
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const uint32_t w = q4 == 0 ? kw[nt].x : q4 == 1 ? kw[nt].y : q4 == 2 ? kw[nt].z : kw[nt].w;
            uint32_t b0, b1;
            e4m3x4_to_f16x4(w, b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              if (mt == 0 || mt * 16 < nrows) mma(s[mt][nt], qa[mt], b0, b1);
          }
        }
      }
      // ---- masks, maxima, probabilities
      const bool missing = kh[0] == 0.f || kh[1] == 0.f;
      const bool edge = missing || w.edge(x0);
      uint32_t pa[MT][2][4];
      float scale_o[MT][2];
      bool rescale = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
        const float fk[2][2] = {{f[mt][0] * kh[0], f[mt][0] * kh[1]}, {f[mt][1] * kh[0], f[mt][1] * kh[1]}};
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = fmaf(s[mt][nt][e], fk[e >> 1][nt >> 1], lh[nt >> 1]);
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = x0 + nt * 8 + 2 * c + (e & 1), p = pos[mt][e >> 1];
              const bool vis = x <= p && kh[nt >> 1] != 0.f && (a.window == 0 || x > p - a.window || x < a.sinks);
              if (!vis) s[mt][nt][e] = -CUDART_INF_F;
            }
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[mt][nt][e]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = fmaxf(top[x], __shfl_xor_sync(FULL, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(FULL, top[x], 2));
          scale_o[mt][x] = 1.f;
          if (top[x] > m[mt][x] + LAZY || (m[mt][x] == -CUDART_INF_F && top[x] > m[mt][x])) {
            const float k = m[mt][x] == -CUDART_INF_F ? 0.f : ex2_approx(m[mt][x] - top[x]);
            l[mt][x] *= k;
            scale_o[mt][x] *= k;
            m[mt][x] = top[x];
            rescale = true;
          }
        }
      }
      if (__any_sync(FULL, rescale)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][n][e] *= scale_o[mt][e >> 1];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float p[4][4];
        const float base[2] = {(m[mt][0] == -CUDART_INF_F ? 0.f : m[mt][0]) - LIFT,
                               (m[mt][1] == -CUDART_INF_F ? 0.f : m[mt][1]) - LIFT};
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = ex2_approx(s[mt][nt][e] - base[e >> 1]);
            l[mt][e >> 1] = fmaf(y, ih[nt >> 1], l[mt][e >> 1]);
            p[nt][e] = y;
          }
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) {
          pa[mt][kc][0] = pack2<__half>(p[2 * kc][0], p[2 * kc][1]);
          pa[mt][kc][1] = pack2<__half>(p[2 * kc][2], p[2 * kc][3]);
          pa[mt][kc][2] = pack2<__half>(p[2 * kc + 1][0], p[2 * kc + 1][1]);
          pa[mt][kc][3] = pack2<__half>(p[2 * kc + 1][2], p[2 * kc + 1][3]);
        }
      }
      // ---- o += p v: dims 16 j + 4 c .. + 3 of rows g, g + 8.  Slots that no
      // token has reached may hold anything, NaN among it: they count as 0.
      if (missing || x0 + KV_TILE > job.n) {
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
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (mt != 0 && mt * 16 >= nrows) continue;
            mma(o[mt][2 * jd], pa[mt][kc], even[0], even[1]);
            mma(o[mt][2 * jd + 1], pa[mt][kc], odd[0], odd[1]);
          }
        }
      }
      out_slot = out_slot + 1 == S ? 0 : out_slot + 1;
      parity ^= out_slot == 0;
      __syncwarp();
      advance();
    }
    }

    // ---- the warps' parts together
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float t = l[mt][x];
        t += __shfl_xor_sync(FULL, t, 1);
        t += __shfl_xor_sync(FULL, t, 2);
        const int r = mt * 16 + x * 8 + g;
        if (c == 0) {
          s_m[warp][r] = m[mt][x];
          s_l[warp][r] = t;
        }
      }
    __syncthreads();  // (every warp's ring is drained)
    float *so = reinterpret_cast<float *>(smem) + warp * M * D;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = mt * 16 + x * 8 + g;
        if (r < nrows) {
#pragma unroll
          for (int jd = 0; jd < NJ; ++jd)
            *reinterpret_cast<float4 *>(so + r * D + jd * 16 + 4 * c) =
                make_float4(o[mt][2 * jd][2 * x], o[mt][2 * jd + 1][2 * x],
                            o[mt][2 * jd][2 * x + 1], o[mt][2 * jd + 1][2 * x + 1]);
        }
      }
    __syncthreads();
    const bool whole = w.whole(), starts = t0 == 0;
    T *out = static_cast<T *>(a.out);
    float *part = part_of<M, D>(a, 2 * blockIdx.x + (starts ? 1 : 0));
    const float *all = reinterpret_cast<const float *>(smem);
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
        const float4 v = *reinterpret_cast<const float4 *>(all + (i2 * M + r) * D + d);
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
      // ---- the unit's parts together, by the CTA that is last
      const int g0 = kv_cta_of(share.total, share.ctas, w.u_begin);
      const int g1 = kv_cta_of(share.total, share.ctas, w.u_end - 1);
      unsigned *count = reinterpret_cast<unsigned *>(a.work) + g0;
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(count, 1) == (unsigned)(g1 - g0);
      __syncthreads();
      if (s_last) {
        // the parts' weights 2^(m - max) / l first, all loads in flight at once
        __threadfence();
        if (tid == 0) *count = 0;
        const int parts = g1 - g0 + 1;
        float *w_m = reinterpret_cast<float *>(smem), *w_l = w_m + parts * M;
        auto slot = [&](int p) { return part_of<M, D>(a, 2 * (g0 + p) + (p == 0 ? 1 : 0)); };
        for (int i = tid; i < parts * M; i += THREADS) {
          const float *from = slot(i / M) + M * D + i % M;
          const bool on = i % M < nrows;
          w_m[i] = on ? __ldcg(from) : -CUDART_INF_F;
          w_l[i] = on ? __ldcg(from + M) : 0.f;
        }
        __syncthreads();
        for (int r = warp; r < nrows; r += WARPS) {
          float top = -CUDART_INF_F, sum = 0.f;
          for (int p = lane; p < parts; p += 32) top = fmaxf(top, w_m[p * M + r]);
#pragma unroll
          for (int o2 = 16; o2; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o2));
          const float base = top == -CUDART_INF_F ? 0.f : top;
          for (int p = lane; p < parts; p += 32) {
            const float k = ex2_approx(w_m[p * M + r] - base);
            w_m[p * M + r] = k;
            if (w_l[p * M + r] != 0.f) sum += w_l[p * M + r] * k;
          }
#pragma unroll
          for (int o2 = 16; o2; o2 >>= 1) sum += __shfl_xor_sync(FULL, sum, o2);
          if (lane == 0) s_f[r] = sum == 0.f ? 0.f : 1.f / sum;
        }
        __syncthreads();
        for (int i = tid; i < nrows * (D / 4); i += THREADS) {
          const int r = i / (D / 4), d = i % (D / 4) * 4;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int p = 0; p < parts; ++p) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(slot(p) + r * D + d));
            const float k = w_m[p * M + r];
            x.x += v.x * k;
            x.y += v.y * k;
            x.z += v.z * k;
            x.w += v.w * k;
          }
          const float inv = s_f[r];
          T *dst = out + ((long long)w.token(r) * a.q_heads + w.q_head(r)) * D + d;
          *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(x.x * inv, x.y * inv), pack2<T>(x.z * inv, x.w * inv));
        }
      }
    }
    // (generic reads and writes of the ring's memory come before the next copies into it)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  if (bits) atomicOr(a.err, bits);
}

// ---- host --------------------------------------------------------------------

}  // namespace

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
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

namespace {

template <int D, int MT, int S>
constexpr int few_smem() {
  return 1024 + WARPS * S * 2 * KV_TILE * D + MT * D / 16 * 512;
}

template <typename T, int D, int MT, int S, int PER_SM>
cudaError_t launch_few(const KvAttendArgs &a, cudaStream_t st) {
  CUtensorMap k, v;
  const int tokens = a.c.page < KV_TILE ? a.c.page : KV_TILE;
  if (!kv_make_map(&k, a.c, a.c.k, tokens) || !kv_make_map(&v, a.c, a.c.v, tokens)) return cudaErrorInvalidValue;
  attend_few_kernel<T, D, MT, S><<<a.sms * PER_SM, THREADS, few_smem<D, MT, S>(), st>>>(a, k, v);
  return cudaGetLastError();
}

template <typename T, int D, int MT, int S>
cudaError_t limit_few() {
  return cudaFuncSetAttribute(attend_few_kernel<T, D, MT, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              few_smem<D, MT, S>());
}

template <typename T>
cudaError_t limits() {
  cudaError_t e = limit_few<T, 128, 1, 2>();
  if (e == cudaSuccess) e = limit_few<T, 128, 2, 3>();
  if (e == cudaSuccess) e = limit_few<T, 64, 1, 4>();
  if (e == cudaSuccess) e = limit_few<T, 64, 2, 6>();
  return e;
}

template <typename T>
cudaError_t attend(const KvAttendArgs &a, cudaStream_t st) {
  const long long rows = (long long)a.max_q * a.group;
  if (kv_many_rows(a)) return launch_attend_many(a, std::is_same<T, __half>::value ? SGD_F16 : SGD_BF16, st);
  const bool one = rows <= 16;
  if (a.c.dim == 128) return one ? launch_few<T, 128, 1, 2, 3>(a, st) : launch_few<T, 128, 2, 3, 2>(a, st);
  return one ? launch_few<T, 64, 1, 4, 3>(a, st) : launch_few<T, 64, 2, 6, 2>(a, st);
}

}  // namespace

size_t kv_attend_workspace() {
  // (the larger of 456 CTAs' parts of up to 32 rows and 152 CTAs' of 128)
  return (size_t)MAX_CTAS * 8 + (size_t)(MAX_CTAS / 3) * 2 * 128 * (128 + 2) * 4;
}

cudaError_t kv_attend_set_limits() {
  cudaError_t e = limits<__half>();
  if (e == cudaSuccess) e = limits<__nv_bfloat16>();
  if (e == cudaSuccess) e = attend_many_limits();
  return e;
}

cudaError_t launch_kv_attend(KvAttendArgs a, int dtype, cudaStream_t st, int *launches) {
  if (a.sms > MAX_CTAS / 3) a.sms = MAX_CTAS / 3;
  *launches = 1;
  return dtype == SGD_F16 ? attend<__half>(a, st) : attend<__nv_bfloat16>(a, st);
}

}  // namespace sgd
