// kv_attend_many.cu -- the attention of kv_attend.cu for many rows a unit: up to
// 128 (new token, query head) rows share each pass over a head's keys and
// values, on the 5th-generation tensor cores.
//
// One persistent CTA per SM, its warps in roles that run ahead of one another
// through barriers, over all segments of the CTA's share without a stop:
//   a producer    loads 64-token tiles of keys and values by TMA, S deep;
//   4 converters  take e4m3 to f16 (exactly) in shared memory, in the 128-byte
//                 swizzled lines that the products read;
//   4 loaders     scale each row of q by a power of two into [1, 2), round it to
//                 f16 (see kv_attend.cu) and leave it in tensor memory;
//   one thread    issues s = q k^T and o += p v, 128 rows x 64 tokens and 128
//                 rows x D, accumulators in tensor memory;
//   4 softmax     warps, a row per thread, turn s into p: running maximum and sum
//                 in registers, p as f16 in tensor memory, where the second
//                 product takes it from.  o is scaled there, and only when the
//                 maximum has moved far enough.
// q and p come from tensor memory so that shared memory serves only the
// conversion and one operand: 96 KB a tile of 16 KB at D = 128, 768 cycles at
// 128 bytes, where the tile's loading takes about 700 at the measured copy
// bandwidth, the products 512 and the exponentials (128 rows) 512.
#include <math_constants.h>

#include "kv_attend.cuh"
#include "num_types.cuh"
#include "sgd_internal.h"
#include "tensor_core.cuh"

namespace sgd {
namespace {

constexpr int M = 128;
constexpr int TILE = 64;
constexpr int WARPS = 16, THREADS = 32 * WARPS;
// warps by role (tensor-memory lanes: rank modulo 4)
constexpr int W_PRODUCER = 0, W_ISSUER = 1, W_SOFTMAX = 4, W_CONVERT = 8, W_QUERY = 12;
constexpr int META = 32, FACTORS = 8;  // rings that outlast how far a role can run ahead

struct Meta {
  float ks, lv, iv;  // the tile's key scale (0: no such page), log2 V, 1 / V
};

template <int D>
struct Plan {
  static constexpr int RAW = 2 * TILE * D;     // bytes of a loaded tile
  static constexpr int HALF = TILE * D * 2;    // bytes of its keys (or values) as f16
  static constexpr int STAGES = D == 128 ? 9 : 12;
  static constexpr int SMEM = 1024 + STAGES * RAW + 4 * HALF;
  // tensor memory columns
  static constexpr int O = 0, S = 128, P = S + 2 * TILE, Q = P + TILE, COLS = 512;
};

enum Bar {
  RAW_FULL = 0, RAW_EMPTY = 16, KF_FULL = 32, KF_EMPTY = 34, VF_FULL = 36, VF_EMPTY = 38, S_FULL = 40,
  S_EMPTY = 42, P_FULL = 44, PV_DONE = 46, Q_FULL = 48, Q_EMPTY = 50, O_EMPTY = 52, PART = 53, LAST = 54, BARS = 55
};

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 1)
    attend_many_kernel(KvAttendArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using L = Plan<D>;
  using Walk = KvWalk<M, TILE>;
  constexpr int S = L::STAGES, PACK = 128 / D;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  __shared__ __align__(8) unsigned long long bars[BARS];
  __shared__ Meta meta[META];
  __shared__ float factor[FACTORS][M];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_last, s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t bits = 0;
  const KvShare share = kv_share<THREADS, M, TILE>(a, 4, &bits);
  if (share.begin >= share.end) {
    if (bits) atomicOr(a.err, bits);
    return;
  }
  const uint32_t raw0 = smem_addr(smem), kf0 = raw0 + S * L::RAW, vf0 = kf0 + 2 * L::HALF;
  auto bar = [&](int which, int i = 0) { return smem_addr(bars + which + i); };
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      bar_init(bar(RAW_FULL, i), 1);
      bar_init(bar(RAW_EMPTY, i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bar(KF_FULL, i), 4);
      bar_init(bar(KF_EMPTY, i), 1);
      bar_init(bar(VF_FULL, i), 4);
      bar_init(bar(VF_EMPTY, i), 1);
      bar_init(bar(S_FULL, i), 1);
      bar_init(bar(S_EMPTY, i), 4);
      bar_init(bar(P_FULL, i), 4);
      bar_init(bar(PV_DONE, i), 1);
      bar_init(bar(Q_FULL, i), 4);
      bar_init(bar(Q_EMPTY, i), 1);
    }
    bar_init(bar(O_EMPTY), 4);
    bar_init(bar(PART), 4);
    bar_init(bar(LAST), 1);
    bar_init_fence();
    s_abort = 0;
  }
  if (warp == W_ISSUER) tmem_alloc(smem_addr(&tmem_slot), L::COLS);
  tmem_before_sync();
  __syncthreads();
  tmem_after_sync();
  const uint32_t tmem = tmem_slot;
  // A wait that runs out, in any role, ends the others' as well; each role then
  // leaves its loops.
  auto wait = [&](uint32_t b, uint32_t parity) {
    for (int i = 0; i < (1 << 22); ++i) {
      if (bar_try(b, parity)) return true;
      if ((i & 63) == 63 && *reinterpret_cast<volatile int *>(&s_abort)) return false;
    }
    *reinterpret_cast<volatile int *>(&s_abort) = 1;
    bits |= SGD_KV_ERR_WAIT;
    return false;
  };
  // the g-th use of one of two buffers: wait for what filled it, or for its
  // (g - 2)-th use to be over
  auto full = [&](int which, uint32_t g) { return wait(bar(which, g & 1), (g >> 1) & 1); };
  auto over = [&](int which, uint32_t g) { return g < 2 || wait(bar(which, g & 1), ((g >> 1) - 1) & 1); };
  auto warp_arrive = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) bar_arrive(b);
  };

  if (warp == W_PRODUCER) {
    Walk w(a, share, &bits);
    uint32_t slot = 0, lap = 0, g = 0;
    bool ok = true;
    while (ok && w.next(&bits)) {
      for (int j0 = w.t0; ok && j0 < w.t1; j0 += 32) {
        // lane i: what the tile j0 + i needs
        const bool on = w.seen(j0 + lane);
        Meta mt{0.f, 0.f, 1.f};
        int y = 0;
        if (on) {
          const int x = w.job.tile(j0 + lane) * TILE, pg = w.page(x, 0, &bits);
          y = ((max(pg, 0) * a.c.heads + w.h) * a.c.page + x % a.c.page) / PACK;
          if (pg >= 0) {
            mt.ks = __ldg(a.c.ks + (long long)pg * a.c.heads + w.h);
            const float vs = __ldg(a.c.vs + (long long)pg * a.c.heads + w.h);
            mt.lv = log2_scale(vs);
            mt.iv = 1.f / vs;
          }
        }
        for (uint32_t todo = __ballot_sync(FULL, on); ok && todo; todo &= todo - 1) {
          if (lap > 0) ok = wait(bar(RAW_EMPTY, slot), (lap - 1) & 1);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
          if (lane == __ffs(todo) - 1) {
            meta[g % META] = mt;
            const uint32_t dst = raw0 + slot * L::RAW, b = bar(RAW_FULL, slot);
            bar_expect(b, L::RAW);
            tma_load_2d(dst, &kmap, 0, y, b);
            tma_load_2d(dst + L::RAW / 2, &vmap, 0, y, b);
          }
          __syncwarp();
          ++g;
          if (++slot == S) {
            slot = 0;
            ++lap;
          }
        }
      }
    }
    if (!ok) {  // (copies in flight land before the CTA ends, or a bound runs out)
      for (int i = 0; i < S; ++i)
        for (int n = 0; n < (1 << 16) && !bar_try(bar(RAW_FULL, i), lap & 1) && !bar_try(bar(RAW_FULL, i), (lap & 1) ^ 1); ++n) {
        }
    }
  } else if (warp == W_ISSUER) {
    if (lane == 0) {
      Walk w(a, share, &bits);
      uint32_t g = 0, units = 0, firsts = 0;
      bool pending = false, pending_first = false, ok = true;
      // o (+)= p v of tile g, the first of its segment or not
      auto second = [&](uint32_t t, bool first) {
        ok = full(P_FULL, t) && full(VF_FULL, t);
        if (ok && first) {
          if (firsts > 0) ok = wait(bar(O_EMPTY), (firsts - 1) & 1);
          ++firsts;
        }
        if (!ok) return;
        tmem_after_sync();
        const uint32_t v = vf0 + (t & 1) * L::HALF, p = tmem + L::P + (t & 1) * (TILE / 2);
#pragma unroll
        for (int k = 0; k < TILE / 16; ++k)
          mma_ts(tmem + L::O, p + k * 8, smem_operand(v + k * 2048, 1024, TILE * 128), f16_product(D, true),
                 !first || k > 0);
        mma_commit(bar(VF_EMPTY, t & 1));
        mma_commit(bar(PV_DONE, t & 1));
      };
      while (ok && w.next(&bits)) {
        bool first = true;
        for (int j = w.t0; ok && j < w.t1; ++j) {
          if (!w.seen(j)) continue;
          if (first) ok = full(Q_FULL, units);
          ok = ok && full(KF_FULL, g) && over(S_EMPTY, g);
          if (!ok) break;
          tmem_after_sync();
          const uint32_t k = kf0 + (g & 1) * L::HALF, q = tmem + L::Q + (units & 1) * (D / 2);
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_ts(tmem + L::S + (g & 1) * TILE, q + i * 8,
                   smem_operand(k + (i / 4) * TILE * 128 + (i % 4) * 32, 1024, 16), f16_product(TILE, false), i > 0);
          mma_commit(bar(KF_EMPTY, g & 1));
          mma_commit(bar(S_FULL, g & 1));
          if (pending) second(g - 1, pending_first);
          pending = true;
          pending_first = first;
          first = false;
          ++g;
        }
        if (!first) {
          mma_commit(bar(Q_EMPTY, units & 1));
          ++units;
        }
      }
      if (ok && pending) second(g - 1, pending_first);
    }
    __syncwarp();
  } else if (warp >= W_SOFTMAX && warp < W_SOFTMAX + 4) {
    const int r = tid - 32 * W_SOFTMAX;               // the thread's row of a unit
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // its warp's lanes, in an address
    Walk w(a, share, &bits);
    uint32_t g = 0, units = 0, cuts = 0;
    bool ok = true;
    while (ok && w.next(&bits)) {
      const bool on = (warp & 3) * 32 < w.nrows;  // the warp has rows of this unit
      const int pos = r < w.nrows ? w.job.n - w.job.ql + (w.r0 + r) / a.group : -1;
      float m = -CUDART_INF_F, l = 0.f, f = 0.f;
      bool first = true;
      for (int j = w.t0; ok && j < w.t1; ++j) {
        if (!w.seen(j)) continue;
        ok = full(S_FULL, g);
        if (!ok) break;
        tmem_after_sync();
        const Meta mt = meta[g % META];
        if (first) f = factor[units % FACTORS][r];
        float s[TILE];
        if (on) {
          const uint32_t from = tmem + lanes + L::S + (g & 1) * TILE;
          tmem_ld32(from, reinterpret_cast<uint32_t *>(s));
          tmem_ld32(from + 32, reinterpret_cast<uint32_t *>(s) + 32);
          tmem_wait_ld();
        }
        tmem_before_sync();
        warp_arrive(bar(S_EMPTY, g & 1));
        if (on) {
          const int x0 = w.job.tile(j) * TILE;
          if (mt.ks == 0.f || w.edge(x0)) {
            const int lim = mt.ks == 0.f ? -1 : pos - x0;  // the row sees slots up to lim
            const int from = a.window > 0 ? lim - a.window + 1 : -1, sink = a.sinks - x0;
#pragma unroll
            for (int i = 0; i < TILE; ++i)
              if (i > lim || (i < from && i >= sink)) s[i] = -CUDART_INF_F;
          }
          float top0 = s[0], top1 = s[1];
#pragma unroll
          for (int i = 2; i < TILE; i += 2) {
            top0 = fmaxf(top0, s[i]);
            top1 = fmaxf(top1, s[i + 1]);
          }
          const float fk = fmaxf(f * (mt.ks == 0.f ? 1.f : mt.ks), 1e-37f), top = fmaf(fmaxf(top0, top1), fk, mt.lv);
          float o_scale = 1.f;
          if (top > m + LAZY || (m == -CUDART_INF_F && top > m)) {
            const float k = m == -CUDART_INF_F ? 0.f : ex2_approx(m - top);
            l *= k;
            o_scale *= k;
            m = top;
          }
          if (__any_sync(FULL, o_scale != 1.f) && !first) {
            ok = full(PV_DONE, g - 1);  // (the products so far are in o)
            if (!__all_sync(FULL, ok)) break;
            tmem_after_sync();
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              uint32_t o[32];
              tmem_ld32(tmem + lanes + L::O + d, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * o_scale);
              tmem_st32(tmem + lanes + L::O + d, o);
            }
          }
          const float base = (m == -CUDART_INF_F ? 0.f : m) - LIFT - mt.lv;
          float sum0 = 0.f, sum1 = 0.f;
          uint32_t p[TILE / 2];
#pragma unroll
          for (int i = 0; i < TILE; i += 2) {
            const float x = ex2_approx(fmaf(s[i], fk, -base)), y = ex2_approx(fmaf(s[i + 1], fk, -base));
            sum0 += x;
            sum1 += y;
            p[i / 2] = pack2<__half>(x, y);
          }
          l = fmaf(sum0 + sum1, mt.iv, l);
          ok = over(PV_DONE, g);  // (the product two tiles ago has read this buffer)
          if (!__all_sync(FULL, ok)) break;
          tmem_after_sync();
          tmem_st32(tmem + lanes + L::P + (g & 1) * (TILE / 2), p);
          tmem_wait_st();
        }
        tmem_before_sync();
        warp_arrive(bar(P_FULL, g & 1));
        first = false;
        ++g;
      }
      ok = __all_sync(FULL, ok);
      if (!ok) break;
      // ---- the segment's result
      if (!first) {
        ok = full(PV_DONE, g - 1);
        if (!__all_sync(FULL, ok)) break;
        tmem_after_sync();
        ++units;
      }
      const bool whole = w.whole(), starts = w.t0 == 0, mine = r < w.nrows;
      float *part = part_of<M, D>(a, 2 * blockIdx.x + (starts ? 1 : 0));
      T *out = static_cast<T *>(a.out) + ((long long)w.token(r) * a.q_heads + w.q_head(r)) * D;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (on) {
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          if (first) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          } else {
            tmem_ld32(tmem + lanes + L::O + d, o);
            tmem_wait_ld();
          }
          if (!mine) continue;
          float x[32];
          // (nothing seen: whatever the products left does not count)
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = l == 0.f ? 0.f : whole ? __uint_as_float(o[i]) * inv : __uint_as_float(o[i]);
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4 *>(out + d)[i] =
                  make_uint4(pack2<T>(x[8 * i], x[8 * i + 1]), pack2<T>(x[8 * i + 2], x[8 * i + 3]),
                             pack2<T>(x[8 * i + 4], x[8 * i + 5]), pack2<T>(x[8 * i + 6], x[8 * i + 7]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4 *>(part + r * D + d)[i] =
                  make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
      }
      if (!first) {
        tmem_before_sync();
        warp_arrive(bar(O_EMPTY));
      }
      if (!whole) {
        // the unit's parts together, by the CTA that is last
        if (mine) {
          part[M * D + r] = m;
          part[M * D + M + r] = l;
        }
        const int g0 = kv_cta_of(share.total, share.ctas, w.u_begin);
        const int g1 = kv_cta_of(share.total, share.ctas, w.u_end - 1);
        unsigned *count = reinterpret_cast<unsigned *>(a.work) + g0;
        __threadfence();
        warp_arrive(bar(PART));
        if (warp == W_SOFTMAX) {
          ok = wait(bar(PART), cuts & 1);
          if (ok && lane == 0) {
            s_last = atomicAdd(count, 1) == (unsigned)(g1 - g0);
            bar_arrive(bar(LAST));
          }
        }
        ok = ok && wait(bar(LAST), cuts & 1);
        if (!__all_sync(FULL, ok)) break;
        ++cuts;
        if (s_last) {
          __threadfence();
          if (r == 0) *count = 0;
          auto slot = [&](int p) { return part_of<M, D>(a, 2 * p + (p == g0 ? 1 : 0)); };
          T *all = static_cast<T *>(a.out);
          for (int i = r; i < w.nrows * (D / 4); i += 128) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            float top = -CUDART_INF_F, sum = 0.f;
            for (int p = g0; p <= g1; ++p) top = fmaxf(top, __ldcg(slot(p) + M * D + row));
            const float base = top == -CUDART_INF_F ? 0.f : top;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int p = g0; p <= g1; ++p) {
              const float *from = slot(p);
              const float4 v = __ldcg(reinterpret_cast<const float4 *>(from + row * D + d));
              const float k = ex2_approx(__ldcg(from + M * D + row) - base);
              sum += __ldcg(from + M * D + M + row) * k;
              x.x += v.x * k;
              x.y += v.y * k;
              x.z += v.z * k;
              x.w += v.w * k;
            }
            const float n = sum == 0.f ? 0.f : 1.f / sum;
            T *dst = all + ((long long)w.token(row) * a.q_heads + w.q_head(row)) * D + d;
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(x.x * n, x.y * n), pack2<T>(x.z * n, x.w * n));
          }
        }
      }
    }
  } else if (warp >= W_CONVERT && warp < W_CONVERT + 4) {
    const int i = tid - 32 * W_CONVERT;
    const int t = i & (TILE - 1), side = i >> 6;  // the thread's token, which half of its dims
    constexpr int CHUNKS = D / 32;                // 16-byte chunks of e4m3 per thread
    const uint32_t line = D == 128 ? t : t >> 1, odd = D == 128 ? 0 : (t & 1) * 4;
    Walk w(a, share, &bits);
    uint32_t g = 0, slot = 0, lap = 0;
    bool ok = true;
    while (ok && w.next(&bits)) {
      for (int j = w.t0; ok && j < w.t1; ++j) {
        if (!w.seen(j)) continue;
        const int x0 = w.job.tile(j) * TILE;
        ok = wait(bar(RAW_FULL, slot), lap & 1);
        const bool gone = ok && (meta[g % META].ks == 0.f || x0 + t >= w.job.n);
        const uint32_t raw = raw0 + slot * L::RAW;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && over(kv == 0 ? KF_EMPTY : VF_EMPTY, g);
          if (!__all_sync(FULL, ok)) break;
          const uint32_t from = raw + kv * (L::RAW / 2) + line * 128;
          const uint32_t to = (kv == 0 ? kf0 : vf0) + (g & 1) * L::HALF + t * 128;
          uint4 v[CHUNKS];
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            const uint32_t at = from + (((odd + side * CHUNKS + c) ^ (line & 7)) << 4);
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w)
                         : "r"(at));
          }
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            uint32_t h[8];
            e4m3x4_to_f16x4(v[c].x, h[0], h[1]);
            e4m3x4_to_f16x4(v[c].y, h[2], h[3]);
            e4m3x4_to_f16x4(v[c].z, h[4], h[5]);
            e4m3x4_to_f16x4(v[c].w, h[6], h[7]);
            // slots that no token has reached may hold anything, NaN among it
            if (kv == 1 && gone) {
#pragma unroll
              for (int e = 0; e < 8; ++e) h[e] = 0;
            }
            const int chunk = side * CHUNKS + c;  // of 16 elements: two of 16 bytes as f16
            const uint32_t panel = to + chunk / 4 * (TILE * 128);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                               panel + (((chunk % 4 * 2 + e) ^ (t & 7)) << 4)),
                           "r"(h[4 * e]), "r"(h[4 * e + 1]), "r"(h[4 * e + 2]), "r"(h[4 * e + 3])
                           : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          warp_arrive(bar(kv == 0 ? KF_FULL : VF_FULL, g & 1));
        }
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        warp_arrive(bar(RAW_EMPTY, slot));
        ++g;
        if (++slot == S) {
          slot = 0;
          ++lap;
        }
      }
    }
  } else if (warp >= W_QUERY) {
    const int r = tid - 32 * W_QUERY;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    Walk w(a, share, &bits);
    uint32_t units = 0;
    while (w.next(&bits)) {
      bool any = false;
      for (int j = w.t0; !any && j < w.t1; ++j) any = w.seen(j);
      if (!any) continue;
      const bool on = (warp & 3) * 32 < w.nrows;
      uint32_t x[D / 2];  // the row: pairs of T, then of f16
#pragma unroll
      for (int i = 0; i < D / 2; ++i) x[i] = 0;
      float f = 0.f;
      if (r < w.nrows) {
        const T *q = static_cast<const T *>(a.q) + w.token(r) * a.q_token + w.q_head(r) * a.q_head;
        if (a.q_vec) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(q) + i);
            x[4 * i] = v.x;
            x[4 * i + 1] = v.y;
            x[4 * i + 2] = v.z;
            x[4 * i + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) {
            const T two[2] = {q[2 * i], q[2 * i + 1]};
            memcpy(&x[i], two, 4);
          }
        }
        float top = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < D / 2; ++i) {
          T two[2];
          memcpy(two, &x[i], 4);
          const float u = fabsf(to_f32(two[0])), v = fabsf(to_f32(two[1]));
          bad = bad || !(u < CUDART_INF_F) || !(v < CUDART_INF_F);
          top = fmaxf(top, fmaxf(u, v));
        }
        const int e2 = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 126);
        // a bad element makes its row NaN; the sign of the scale goes with q
        const float inv = bad ? CUDART_NAN_F : a.scale == 0.f ? 0.f : copysignf(pow2(-e2), a.scale);
        f = a.scale == 0.f ? 1.f : fabsf(a.scale) * LOG2E * pow2(e2);
#pragma unroll
        for (int i = 0; i < D / 2; ++i) {
          T two[2];
          memcpy(two, &x[i], 4);
          x[i] = pack2<__half>(to_f32(two[0]) * inv, to_f32(two[1]) * inv);
        }
      }
      const bool ok = over(Q_EMPTY, units);
      if (!__all_sync(FULL, ok)) break;
      tmem_after_sync();
      if (on) {
        const uint32_t to = tmem + lanes + L::Q + (units & 1) * (D / 2);
#pragma unroll
        for (int i = 0; i < D / 2; i += 32) tmem_st32(to + i, x + i);
        tmem_wait_st();
      }
      factor[units % FACTORS][r] = f;
      tmem_before_sync();
      warp_arrive(bar(Q_FULL, units & 1));
      ++units;
    }
  }
  if (bits) atomicOr(a.err, bits);
  tmem_before_sync();
  __syncthreads();
  tmem_after_sync();
  if (warp == W_ISSUER) tmem_free(tmem, L::COLS);
}

template <typename T, int D>
cudaError_t launch(const KvAttendArgs &a, cudaStream_t st) {
  CUtensorMap k, v;
  if (!kv_make_map(&k, a.c, a.c.k, TILE) || !kv_make_map(&v, a.c, a.c.v, TILE)) return cudaErrorInvalidValue;
  attend_many_kernel<T, D><<<a.sms, THREADS, Plan<D>::SMEM, st>>>(a, k, v);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t limit() {
  return cudaFuncSetAttribute(attend_many_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<D>::SMEM);
}

}  // namespace

// More than 16 rows, a tile within a page (one scale), and units enough that
// few of them are cut in many parts.
bool kv_many_rows(const KvAttendArgs &a) {
  return (long long)a.max_q * a.group > 16 && a.c.page >= TILE && a.r.B * a.c.heads >= a.sms / 4;
}

cudaError_t launch_attend_many(const KvAttendArgs &a, int dtype, cudaStream_t st) {
  if (a.c.dim == 128) return dtype == SGD_F16 ? launch<__half, 128>(a, st) : launch<__nv_bfloat16, 128>(a, st);
  return dtype == SGD_F16 ? launch<__half, 64>(a, st) : launch<__nv_bfloat16, 64>(a, st);
}

cudaError_t attend_many_limits() {
  cudaError_t e = limit<__half, 128>();
  if (e == cudaSuccess) e = limit<__half, 64>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 64>();
  return e;
}

}  // namespace sgd
