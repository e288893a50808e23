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
constexpr int PER_SM = 3;    // CTAs

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
// A unit has up to M = 16 GROUPS rows.  A warp keeps m, l and o of 16 of them in
// registers and streams 32-token tiles through a ring of TMA loads.  Where a
// unit has 16 rows or fewer each of the 4 warps has tiles of its own; where it
// has more, two warps take the same tiles, 16 rows each, so that a byte of the
// cache is still loaded once for all.  Warps meet only over a shared tile's
// release and where a unit ends.
//
// e4m3 is taken to f16, exactly, on the way into the registers that feed the
// matrix instructions, so the products carry no rounding of the cache's; q goes
// to f16 after each row is scaled to [1, 2) by a power of two (bf16 has fewer
// bits than f16: only elements 2^-24 times the row's largest lose any), and the
// probabilities to f16 (relative 2^-12 each; the sum l is taken before that
// rounding).
//
// The order of the elements of a product's long axis is free as long as both
// sides use the same: a lane takes 2 (D = 128) or 1 (D = 64) whole 16-byte
// chunks of a key, so all shared-memory reads are 16 bytes wide and, with the
// 128-byte swizzle of the TMA load, without bank conflicts.
template <typename T, int D, int GROUPS, int S>
__global__ void __launch_bounds__(THREADS, PER_SM)
    attend_kernel(KvAttendArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int M = 16 * GROUPS;
  constexpr int KS = D / 16;                 // k steps of q . k
  constexpr int HALF = KV_TILE * D;          // bytes of a tile's keys (or values)
  constexpr int NJ = D / 16;                 // 16-dim groups of the output
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  __shared__ __align__(8) unsigned long long bars[WARPS * S];
  __shared__ float s_f[M];
  __shared__ float s_m[WARPS][16], s_l[WARPS][16];
  __shared__ uint32_t s_phase[WARPS];  // of the ring's slots, a bit each, by the warp whose own they are
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  uint32_t bits = 0;
  const KvShare share = kv_share<THREADS, M, KV_TILE>(a, WARPS, &bits);
  if (share.begin >= share.end) {
    if (bits && tid == 0) atomicOr(a.err, bits);
    return;
  }
  const uint32_t ring0 = smem_addr(smem), q_at = ring0 + WARPS * S * 2 * HALF;
  if (tid == 0) {
    for (int i = 0; i < WARPS * S; ++i) bar_init(smem_addr(bars) + 8 * i, 1);
    bar_init_fence();
  }
  if (lane == 0) s_phase[warp] = 0;
  __syncthreads();

  const int P = a.c.page, H = a.c.heads;
  const int halves = P < KV_TILE ? 2 : 1;  // pages of a tile
  KvWalk<M, KV_TILE> w(a, share);
#pragma unroll 1
  while (w.next(&bits)) {
    const KvJob &job = w.job;
    const int h = w.h, nrows = w.nrows, t0 = w.t0, t1 = w.t1, p_first = w.p_first, p_last = w.p_last;

    // the warp's rows, tiles and slots of the ring
    const bool pair = GROUPS == 2 && nrows > 16;
    const int rows16 = pair ? warp & 1 : 0, stream = pair ? warp >> 1 : warp, streams = pair ? WARPS / 2 : WARPS;
    const int slots = pair ? 2 * S : S;
    const uint32_t ring = ring0 + stream * slots * 2 * HALF, bar0 = smem_addr(bars) + stream * slots * 8;
    uint32_t phases = pair ? s_phase[2 * stream] | s_phase[2 * stream + 1] << S : s_phase[warp];
    int in_slot = 0, out_slot = 0;  // to load, to consume

    // ---- tiles t0 + stream, + streams, ..., 32 at a time: lane i holds
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
    int next = t0 + stream;  // the first tile of the batch being loaded
    uint32_t to_load = look(next + streams * lane, ahead);
    auto advance = [&]() {  // loads the next tile that is seen, if any
#pragma unroll 1
      while (to_load == 0) {
        next += 32 * streams;
        if (next >= t1) return;
        to_load = look(next + streams * lane, ahead);
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
      in_slot = in_slot + 1 == slots ? 0 : in_slot + 1;
    };
    if (rows16 == 0) {  // (one of a pair loads)
#pragma unroll 1
      for (int i = 0; i < slots; ++i) advance();
    }

    // ---- the unit's queries, as the matrix instructions take them
#pragma unroll 1
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

    float o[2 * NJ][4];
    float m[2], l[2], f[2];
    int pos[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rows16 * 16 + x * 8 + g;
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
    for (int j0 = t0 + stream; j0 < t1; j0 += 32 * streams) {
    float ks[2] = {0.f, 0.f};           // (a scale of 0: no such page)
    float lv[2] = {0.f, 0.f}, iv[2] = {1.f, 1.f};  // log2 V, 1 / V
    bool on = w.seen(j0 + streams * lane);
    if (on) {
      const int x = job.tile(j0 + streams * lane) * KV_TILE;
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
      const int x0 = job.tile(j0 + streams * src) * KV_TILE;
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
          const uint4 v = lds128(q_at + ((rows16 * KS + ch * 4 + q4) * 32 + lane) * 16);
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
      // ---- masks, maxima, probabilities
      const bool missing = kh[0] == 0.f || kh[1] == 0.f;
      {
        const float fk[2][2] = {{f[0] * kh[0], f[0] * kh[1]}, {f[1] * kh[0], f[1] * kh[1]}};
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = fmaf(s[nt][e], fk[e >> 1][nt >> 1], lh[nt >> 1]);
      }
      if (missing || w.edge(x0)) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = x0 + nt * 8 + 2 * c + (e & 1), p = pos[e >> 1];
            const bool vis = x <= p && kh[nt >> 1] != 0.f && (a.window == 0 || x > p - a.window || x < a.sinks);
            if (!vis) s[nt][e] = -CUDART_INF_F;
          }
      }
      float top[2] = {-CUDART_INF_F, -CUDART_INF_F}, scale_o[2] = {1.f, 1.f};
      bool rescale = false;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[nt][e]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = fmaxf(top[x], __shfl_xor_sync(FULL, top[x], 1));
        top[x] = fmaxf(top[x], __shfl_xor_sync(FULL, top[x], 2));
        if (top[x] > m[x] + LAZY || (m[x] == -CUDART_INF_F && top[x] > m[x])) {
          scale_o[x] = m[x] == -CUDART_INF_F ? 0.f : ex2_approx(m[x] - top[x]);
          l[x] *= scale_o[x];
          m[x] = top[x];
          rescale = true;
        }
      }
      if (__any_sync(FULL, rescale)) {
#pragma unroll
        for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= scale_o[e >> 1];
      }
      uint32_t pa[2][4];
      {
        const float base[2] = {(m[0] == -CUDART_INF_F ? 0.f : m[0]) - LIFT, (m[1] == -CUDART_INF_F ? 0.f : m[1]) - LIFT};
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nt][e] = ex2_approx(s[nt][e] - base[e >> 1]);
            l[e >> 1] = fmaf(s[nt][e], ih[nt >> 1], l[e >> 1]);
          }
          pa[nt >> 1][(nt & 1) * 2] = pack2<__half>(s[nt][0], s[nt][1]);
          pa[nt >> 1][(nt & 1) * 2 + 1] = pack2<__half>(s[nt][2], s[nt][3]);
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
          mma(o[2 * jd], pa[kc], even[0], even[1]);
          mma(o[2 * jd + 1], pa[kc], odd[0], odd[1]);
        }
      }
      phases ^= 1u << out_slot;
      out_slot = out_slot + 1 == slots ? 0 : out_slot + 1;
      __syncwarp();
      if (pair) {
        if (stream == 0)
          asm volatile("bar.sync 1, 64;" ::: "memory");
        else
          asm volatile("bar.sync 2, 64;" ::: "memory");
      }
      if (rows16 == 0) advance();
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
    if (lane == 0 && (!pair || rows16 == 0)) {
      s_phase[pair ? 2 * stream : warp] = phases & ((1u << S) - 1);
      if (pair) s_phase[2 * stream + 1] = phases >> S;
    }
    float *so = reinterpret_cast<float *>(smem) + warp * 16 * D;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = x * 8 + g;
      if (rows16 * 16 + r < nrows) {
#pragma unroll
        for (int jd = 0; jd < NJ; ++jd)
          *reinterpret_cast<float4 *>(so + r * D + jd * 16 + 4 * c) = make_float4(
              o[2 * jd][2 * x], o[2 * jd + 1][2 * x], o[2 * jd][2 * x + 1], o[2 * jd + 1][2 * x + 1]);
      }
    }
    __syncthreads();
    const bool whole = w.whole(), starts = t0 == 0;
    T *out = static_cast<T *>(a.out);
    float *part = part_of<M, D>(a, 2 * blockIdx.x + (starts ? 1 : 0));
    const float *all = reinterpret_cast<const float *>(smem);
#pragma unroll 1
    for (int i = tid; i < nrows * (D / 4); i += THREADS) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float top = -CUDART_INF_F;
      const int r16 = r % 16, skip = pair ? r / 16 ^ 1 : -1;  // (of a pair's warps the other has other rows)
#pragma unroll
      for (int i2 = 0; i2 < WARPS; ++i2)
        if ((i2 & 1) != skip) top = fmaxf(top, s_m[i2][r16]);
      const float base = top == -CUDART_INF_F ? 0.f : top;
      float sum = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i2 = 0; i2 < WARPS; ++i2) {
        if ((i2 & 1) == skip) continue;
        const float k = ex2_approx(s_m[i2][r16] - base);
        const float4 v = *reinterpret_cast<const float4 *>(all + (i2 * 16 + r16) * D + d);
        if (s_l[i2][r16] != 0.f) {
          sum += s_l[i2][r16] * k;
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
#pragma unroll 1
        for (int i = tid; i < parts * M; i += THREADS) {
          const float *from = slot(i / M) + M * D + i % M;
          const bool on = i % M < nrows;
          w_m[i] = on ? __ldcg(from) : -CUDART_INF_F;
          w_l[i] = on ? __ldcg(from + M) : 0.f;
        }
        __syncthreads();
#pragma unroll 1
        for (int r = warp; r < nrows; r += WARPS) {
          float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll 1
          for (int p = lane; p < parts; p += 32) top = fmaxf(top, w_m[p * M + r]);
#pragma unroll
          for (int o2 = 16; o2; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o2));
          const float base = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll 1
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
#pragma unroll 1
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

// Keys or values as lines of 128 bytes (one token, or two of 64 bytes), in
// boxes of `tokens`, with the 128-byte swizzle.
bool make_map(CUtensorMap *map, const KvView &c, void *base, int tokens) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t lines = (cuuint64_t)c.num_pages * c.heads * c.page * c.dim / 128;
  const cuuint64_t dims[2] = {128, lines}, strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)(tokens * c.dim / 128)}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int GROUPS, int S>
constexpr int smem_bytes() {
  return 1024 + WARPS * S * 2 * KV_TILE * D + GROUPS * D / 16 * 512;
}

template <typename T, int D, int GROUPS, int S>
cudaError_t launch(const KvAttendArgs &a, cudaStream_t st) {
  CUtensorMap k, v;
  const int tokens = a.c.page < KV_TILE ? a.c.page : KV_TILE;
  if (!make_map(&k, a.c, a.c.k, tokens) || !make_map(&v, a.c, a.c.v, tokens)) return cudaErrorInvalidValue;
  attend_kernel<T, D, GROUPS, S><<<a.sms * PER_SM, THREADS, smem_bytes<D, GROUPS, S>(), st>>>(a, k, v);
  return cudaGetLastError();
}

template <typename T, int D, int GROUPS, int S>
cudaError_t limit() {
  return cudaFuncSetAttribute(attend_kernel<T, D, GROUPS, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_bytes<D, GROUPS, S>());
}

template <typename T>
cudaError_t limits() {
  cudaError_t e = limit<T, 128, 1, 2>();
  if (e == cudaSuccess) e = limit<T, 128, 2, 2>();
  if (e == cudaSuccess) e = limit<T, 64, 1, 4>();
  if (e == cudaSuccess) e = limit<T, 64, 2, 4>();
  return e;
}

template <typename T>
cudaError_t attend(const KvAttendArgs &a, cudaStream_t st) {
  const bool one = (long long)a.max_q * a.group <= 16;
  if (a.c.dim == 128) return one ? launch<T, 128, 1, 2>(a, st) : launch<T, 128, 2, 2>(a, st);
  return one ? launch<T, 64, 1, 4>(a, st) : launch<T, 64, 2, 4>(a, st);
}

}  // namespace

size_t kv_attend_workspace() { return (size_t)MAX_CTAS * 8 + (size_t)MAX_CTAS * 2 * 32 * (128 + 2) * 4; }

cudaError_t kv_attend_set_limits() {
  cudaError_t e = limits<__half>();
  if (e == cudaSuccess) e = limits<__nv_bfloat16>();
  return e;
}

cudaError_t launch_kv_attend(KvAttendArgs a, int dtype, cudaStream_t st, int *launches) {
  if (a.sms > MAX_CTAS / PER_SM) a.sms = MAX_CTAS / PER_SM;
  *launches = 1;
  return dtype == SGD_F16 ? attend<__half>(a, st) : attend<__nv_bfloat16>(a, st);
}

}  // namespace sgd
