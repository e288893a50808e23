// kv_prompt.cu -- attention of rows of many new tokens: whole prompts, and chunks
// over the paged cache.
//
// A unit is up to 256 rows (new token, query head of the group) of one batch row
// and one head of keys and values, in two tiles of 128.  Its work is a list of
// 128-token tiles: those of the cache that its rows see, then those of the new
// tokens.  Per tile and 128 rows the tensor cores form s = q k^T into tensor
// memory (TMEM), a warpgroup turns s into p = 2^(z - m) with a running maximum
// and sum, a row per thread, and writes p over s, and o += p v accumulates in
// TMEM.  The two row tiles take turns: one's products run beside the other's
// exponentials.
//
// One persistent CTA per SM, its warps in roles that run ahead of one another
// through barriers:
//   8 softmax warps   a warpgroup per row tile;
//   4 loading warps   queries, then keys and values through a ring: the caller's
//                     by TMA, the cache's converted from e4m3 in registers;
//   1 thread          issues the products.
// The tiles of all units, one after the other, are cut into equal shares, one
// per CTA; a unit that a cut goes through leaves parts, which a second kernel
// joins in their order (no atomics: the result does not depend on timing).
//
// Numbers.  Products of 16-bit values and p, sums, maxima and outputs in 32 bits; p is
// rounded to the values' type for the second product (2^-8 of it for bf16, 2^-11 for f16:
// the tensor cores take both operands in one type), the sum of p before that.  Cached keys
// and values go to 16 bits exactly (see `widen`).
//
// What bounds it.  Per tile and two row tiles the products take 2048 cycles at a dim of
// 128, 1024 at 64, and the exponentials 1024; from p to the next scores of a row tile lie
// both products (1024 cycles) and some 300 of latency, and its exponentials, alone, take the
// thread of a row some 1600 to 2000.  That is 2900 to 3300 cycles a tile; measured 3800 with all that
// a unit costs: 32768 tokens, 32 query heads of 128 in groups of four, 6.3 ms at 2070 MHz, 1390
// TFLOP/s; calls one after the other, which the power limit holds at some 1980 MHz, 6.6 ms, 1330.  At a
// dim of 64 5.6 ms, 780.  A tile of the cache takes 1.8 times as long: without its conversion
// a chunk of 1391 tokens over 31377 took 0.79 ms, not 0.97.
// Tried and slower or no faster, the same 32768 tokens in ms, 6.5 then: two threads a row, half of
// a tile's tokens each, meeting once a tile (6.6, chunks over the cache 30% slower: 16
// softmax warps leave the loading ones few registers and turns) or finishing in turn (9.6);
// all p of a tile at once (6.5, short prompts and chunks 10% slower); s read twice, for its
// maximum and for p (8.1); the first half of the next scores before the products with p (7.3: N =
// 64 reads the queries from shared memory twice as often); the issuing thread alone in a
// divergent branch (8.1: operands go through vector registers).
#include <float.h>
#include <math_constants.h>

#include "kv_attend.cuh"
#include "num_types.cuh"
#include "sgd_internal.h"
#include "tensor_core.cuh"

namespace sgd {
namespace {

constexpr int M = 128, ROWS = 2 * M, TILE = 128;
constexpr int WARPS = 16, THREADS = 32 * WARPS;
// (warps 0 to W_LOAD - 1: softmax)
constexpr int W_LOAD = 8, W_ISSUE = 12, W_JOIN = 13;
constexpr int LOADERS = 4;
// Registers a thread by role: together what 512 threads are launched with (128 each).  With
// 168 and 88 chunks of a step took 1.59 ms against 1.27 (the loading warps spill), with 152 and 104
// 1.29 and a step's prompts 1.37 against 1.33, with 136 and 120 chunks 1.39 (the softmax ones do).
constexpr int REGS_SOFTMAX = 144, REGS_OTHER = 112;
static_assert(32 * W_LOAD * REGS_SOFTMAX + 32 * (WARPS - W_LOAD) * REGS_OTHER <= THREADS * 128, "the pool of the launch");
// p and o are relative to a reference, the maximum as it was when it was last set, for which p
// is 2^UP.  It is set anew, and o scaled to it, only where the types' range asks for it:
// bf16 has the range of 32 bits, but values may be up to 2^128.  o is at most the sum l of p
// (and 2^-8 of it) times the largest value, so l stays below 1.  p is that much smaller, and so
// is o, which loses bits of values below 2^-111 (2^-97 in rows whose reference rose for the sake of l).
// f16: p is up to 2^15.99 (< 65504) before that, 2^UP for the maximum as it was; it has all its
// bits down to 2^-21 of that, and below an error of 2^-33 of it.  (o is within 2^63.)
template <typename T>
struct Range;
template <>
struct Range<__nv_bfloat16> {
  static constexpr float UP = -15.f, THRESHOLD = 0.f;  // (l tells)
};
template <>
struct Range<__half> {
  static constexpr float THRESHOLD = 8.f, UP = 15.99f - THRESHOLD;
};
// bf16: the largest l, and by how much the reference rises where l is of many tokens rather than of
// a larger one, as a power of 2.  Either type: how much larger one makes other references of the
// warp rise as well (so that fewer tiles are done twice).
constexpr float L_MOST = 0.98f, RISE = 14.f, WITH = 1.f;
// References of this size on (as powers of 2) are far: 32 bits hold them too coarsely (2^-12 here),
// and p is made from the difference of the scores, for which a half of a tile is gone over twice: with
// such rows in every warp a step's prompts take 3.4 ms, not 1.34.
constexpr float FAR = 4096.f;
// A row's reference: the score (with the scale that its tile's keys were brought to; -inf: none yet) and what
// is added to its exponent (log2 of the values' scale, RISEs).
struct __align__(16) Reference {
  float s, add;
  int far;
};
// What a unit costs beside its tiles, in tiles; the fewest tiles of a part; the least work that
// is worth a CTA.  Measured: a step's prompts 1.33 ms, 1.36 with 2 or 5 in the first place; one
// prompt of 200 tokens 18.6 us, 18.9 with 3 in the last and 24.7 with 5, a chunk of 68 over 2032
// 32.0, 33.5 and 36.7.
constexpr int OVERHEAD = 3, LEAST_PART = 2, LEAST_SHARE = 2;
constexpr int META = 16;      // outlasts how far the loaders run ahead
constexpr int BAD_SEGMENTS = 4, BAD_TILES = 8;

template <int D>
struct Plan {
  static constexpr int HALF = TILE * D * 2;  // bytes of a tile of keys, or of values
  static constexpr int Q = ROWS * D * 2;
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int SMEM = 1024 + Q + STAGES * HALF;
  // TMEM columns: s of a row tile and a key tile (p over it), in turn; then o of either row tile
  static constexpr int BUFFERS = D == 128 ? 2 : 3, S = 0, O = BUFFERS * TILE;
  static constexpr int CHUNKS = D / 8;       // 16-byte chunks of a token
};

// What the loaders know of a tile and the softmax needs.
struct __align__(8) Meta {
  int edge;       // some row does not see some token; then:
  int x, last;    // the tile's first position, the last one that it holds
  uint32_t gone;  // 16-token groups whose page is not there
  float k, v;     // f16: the scales that the tile's keys and values were brought to
};
// Tokens of a tile whose values are not finite (see `spoil`).
struct BadTile {
  int x;                   // the tile's first token, from q0
  uint32_t word[LOADERS];  // of warp w: bits of the tokens that it loaded
};

// ---- the work --------------------------------------------------------------------

struct BatchRow {
  int q0, ql, old;  // first packed token, new tokens, tokens before them
  bool bad;         // its lengths make no sense: the result is 0
};

__device__ __forceinline__ BatchRow batch_row(const KvNewArgs &a, int b, uint32_t *bits) {
  BatchRow r;
  const int q0 = __ldg(a.r.q_start + b), q1 = __ldg(a.r.q_start + b + 1);
  r.q0 = q0;
  r.ql = q1 - q0;
  r.old = 0;
  r.bad = false;
  if (q0 < 0 || q1 > a.r.N || q1 < q0) {
    *bits |= SGD_KV_ERR_LENGTH;
    r.ql = 0;
  } else if (a.r.seq_lens) {
    const int n = __ldg(a.r.seq_lens + b);
    if (r.ql > 0 && (n < r.ql || (long long)n > ((long long)a.r.max_pages << a.c.page_bits))) {
      *bits |= SGD_KV_ERR_LENGTH;
      r.bad = true;
    } else {
      r.old = n - r.ql;
    }
  }
  return r;
}
__device__ __forceinline__ int blocks_of(const KvNewArgs &a, const BatchRow &r) {
  return (r.ql * a.group + ROWS - 1) / ROWS;
}

struct Unit {
  int r0, nrows;               // its rows among the batch row's ql * group
  int p_first, p_last;         // positions of the first and the last row's token
  int c_sink, c_lo, c_tiles;   // of the cache: tiles of first tokens, then from c_lo on
  int f_sink, f_lo, tiles;     // of the new tokens likewise; all tiles
};

__device__ __forceinline__ Unit unit_of(const KvNewArgs &a, const BatchRow &r, int i) {
  Unit u;
  u.r0 = i * ROWS;
  u.nrows = min(ROWS, r.ql * a.group - u.r0);
  const int t_last = (u.r0 + u.nrows - 1) / a.group;
  u.p_first = r.old + u.r0 / a.group;
  u.p_last = r.old + t_last;
  u.c_sink = u.c_lo = u.c_tiles = u.f_sink = u.f_lo = u.tiles = 0;
  if (r.bad) return u;
  const int lo = a.window > 0 ? max(0, u.p_first - a.window + 1) : 0;
  const int c_end = (r.old + TILE - 1) / TILE, f_end = t_last / TILE + 1;
  if (lo > 0) {
    u.c_lo = lo >= r.old ? c_end : lo / TILE;
    u.c_sink = min((min(a.sinks, r.old) + TILE - 1) / TILE, u.c_lo);
    u.f_lo = max(0, lo - r.old) / TILE;
    u.f_sink = min((max(0, a.sinks - r.old) + TILE - 1) / TILE, u.f_lo);
  }
  u.c_tiles = u.c_sink + c_end - u.c_lo;
  u.tiles = u.c_tiles + u.f_sink + f_end - u.f_lo;
  return u;
}

// Where a share begins or ends: before tile t of unit u, or past it.
struct Cut {
  long long u;
  int b, i, h, t;
  bool past;
};
struct Share {
  Cut begin, end;
  long long all;   // weight of all units
  long long u_at;  // weight before the unit of `end`
  int end_tiles;   // its tiles
  int ctas;
};

__device__ __forceinline__ long long block_scan(long long x, long long *s, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long scan = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(FULL, scan, o);
    if (lane >= o) scan += t;
  }
  __syncthreads();
  if (lane == 31) s[warp] = scan;
  __syncthreads();
  long long before = scan - x, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s[w];
    all += s[w];
  }
  *total = all;
  return before;
}

// A cut at `into` of a unit's weight, moved to the unit's ends where a part would
// be too small to be worth its join.
__device__ __forceinline__ void place_cut(Cut &c, long long into, int tiles) {
  const long long t = into - OVERHEAD;
  c.t = t < LEAST_PART ? 0 : (int)t;
  c.past = t >= LEAST_PART && tiles - t < LEAST_PART;
  if (c.past) c.t = 0;
}

// By all threads of the block.  first: [B + 1] ints of shared memory.
__device__ const Share &share_of(const KvNewArgs &a, int *first, uint32_t *bits) {
  __shared__ long long s_sum[WARPS];
  __shared__ Share s;
  const int tid = threadIdx.x, B = a.r.B;
  const int per = (B + THREADS - 1) / THREADS, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long mine = 0, total;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += blocks_of(a, batch_row(a, b, bits));
  long long at = block_scan(mine, s_sum, &total);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    first[b] = (int)at;
    at += blocks_of(a, batch_row(a, b, bits));
  }
  if (tid == 0) {
    first[B] = (int)total;
    s.ctas = 0;
  }
  __syncthreads();
  const long long blocks = total;
  // Rows that overlap may claim any number of units, with what counts them beyond 32 bits; those that
  // do not have no more than this many.  (The same for all threads.)
  if (blocks > ((long long)a.r.N * a.group + (long long)(ROWS - 1) * B) / ROWS) {
    *bits |= SGD_KV_ERR_LENGTH;
    return s;
  }
  const int c0 = (int)(blocks * tid / THREADS), c1 = (int)(blocks * (tid + 1) / THREADS);
  int b_from = 0;
  mine = 0;
  if (c0 < c1) {
    int hi = B;
    while (hi - b_from > 1) {
      const int mid = (b_from + hi) >> 1;
      if (first[mid] <= c0) b_from = mid;
      else hi = mid;
    }
    int b = b_from;
    BatchRow r = batch_row(a, b, bits);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      while (c >= first[b + 1]) r = batch_row(a, ++b, bits);
      mine += OVERHEAD + unit_of(a, r, c - first[b]).tiles;
    }
  }
  const long long before = block_scan(mine, s_sum, &total);
  const long long all = total * a.c.heads;
  const long long most = (all + LEAST_SHARE - 1) / LEAST_SHARE;
  const int ctas = (int)(most < (long long)gridDim.x ? most : (long long)gridDim.x), g = blockIdx.x;
  if (g < ctas) {
    if (tid == 0) {
      s.ctas = ctas;
      s.all = all;
      s.end.u = a.c.heads * blocks;  // (where it is the end of all)
      s.end.t = 0;
      s.end.past = false;
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const long long pos = quotient(all * (g + k), ctas);
      const int h = (int)quotient(pos, total);
      const long long in = pos - h * total;
      if (h < a.c.heads && c0 < c1 && before <= in && in < before + mine) {
        int b = b_from, c = c0;
        long long w = before;
        BatchRow r = batch_row(a, b, bits);
        Unit u;
        for (;; ++c) {
          while (c >= first[b + 1]) r = batch_row(a, ++b, bits);
          u = unit_of(a, r, c - first[b]);
          if (in < w + OVERHEAD + u.tiles) break;
          w += OVERHEAD + u.tiles;
        }
        Cut &cut = k ? s.end : s.begin;
        cut.u = h * blocks + c;
        cut.b = b;
        cut.i = c - first[b];
        cut.h = h;
        place_cut(cut, in - w, u.tiles);
        if (k) {
          s.u_at = h * total + w;
          s.end_tiles = u.tiles;
        }
      }
    }
  }
  __syncthreads();
  return s;
}

// A share's segments: the units that it holds or cuts, each with its range of tiles.
struct Walk {
  const KvNewArgs &a;
  const Share &s;
  BatchRow row;
  Unit unit;
  long long u;
  int b, i, h, blocks;
  int t0, t1, shift = 0;
  bool begun = false;

  __device__ Walk(const KvNewArgs &a_, const Share &s_) : a(a_), s(s_), u(s_.begin.u), b(s_.begin.b), i(s_.begin.i), h(s_.begin.h) {}

  __device__ __forceinline__ bool done() const { return u > s.end.u || (u == s.end.u && s.end.t == 0 && !s.end.past); }
  __device__ __forceinline__ bool next(uint32_t *bits) {
    t0 = 0;
    if (!begun) {
      begun = true;
      row = batch_row(a, b, bits);
      blocks = blocks_of(a, row);
      if (!s.begin.past) {
        if (done()) return false;
        t0 = s.begin.t;
        return shape();
      }
    }
    ++u;
    if (done()) return false;
    if (++i == blocks) {
      i = 0;
      do {
        if (++b == a.r.B) {
          b = 0;
          ++h;
        }
        row = batch_row(a, b, bits);
        blocks = blocks_of(a, row);
      } while (blocks == 0);
    }
    return shape();
  }
  __device__ __forceinline__ bool shape() {
    unit = unit_of(a, row, i);
    shift = a.window > 0 ? unit.tiles / 2 : 0;
    t1 = u == s.end.u && !s.end.past ? s.end.t : unit.tiles;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == unit.tiles; }
  // The list from its middle on where there is a window: a row may see next to nothing of
  // the tiles at its ends, and its maximum would grow, and o be scaled, after them (a
  // window of 2048 took 0.65 ms where 0.48 was the time without tiles of first tokens).
  __device__ __forceinline__ int turned(int j) const {
    j += shift;
    return j < unit.tiles ? j : j - unit.tiles;
  }
  __device__ __forceinline__ bool cached(int j) const { return turned(j) < unit.c_tiles; }
  // first position of tile j
  __device__ __forceinline__ int at(int j) const {
    j = turned(j);
    if (j < unit.c_tiles) return (j < unit.c_sink ? j : unit.c_lo + j - unit.c_sink) * TILE;
    j -= unit.c_tiles;
    return row.old + (j < unit.f_sink ? j : unit.f_lo + j - unit.f_sink) * TILE;
  }
  // whether some row does not see some token of the tile at x
  __device__ __forceinline__ bool edge(int j, int x) const {
    return x + TILE - 1 > (cached(j) ? row.old - 1 : unit.p_first) ||
           (a.window > 0 && x <= unit.p_last - a.window && x + TILE > a.sinks);
  }
};

// Parts: [D / 4][ROWS] results (four dims each) and what they weigh, 2^(s c + add): [ROWS] s,
// [ROWS] add; two for each CTA, of the unit that its share begins within (0) and ends within (1).
struct Join {
  int parts, q0, r0, nrows, h;
};
__device__ __forceinline__ Join *join_of(const KvNewArgs &a, int g) {
  return reinterpret_cast<Join *>(a.work + MAX_CTAS * 8) + g;
}
template <int D>
__device__ __forceinline__ float *new_part(const KvNewArgs &a, int slot) {
  return reinterpret_cast<float *>(a.work + MAX_CTAS * 8 + MAX_CTAS * 32) + (long long)slot * (ROWS * (D + 2));
}

// ---- pieces of the roles ---------------------------------------------------------

__device__ __forceinline__ void st_shared16(uint32_t to, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A 16-byte chunk (c-th of its token or row) of line `line` of an operand.
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int line, int c) {
  return base + (c >> 3) * (TILE * 128) + line * 128 + (((c & 7) ^ (line & 7)) << 4);
}

// Two e4m3 bytes, each in the high byte of a half, as two T of 2^-120 (bf16) or 2^-8
// (f16) times their value: sign, exponent and fraction keep their order, so moving
// the bits is exact, for subnormals too; `f` brings the values to their size (a power
// of two: exact).
template <typename T>
__device__ __forceinline__ uint32_t widen(uint32_t pair, uint32_t f);
template <>
__device__ __forceinline__ uint32_t widen<__nv_bfloat16>(uint32_t pair, uint32_t f) {
  const uint32_t w = (pair & 0x80008000u) | ((pair >> 4) & 0x07f007f0u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(f));
  return r;
}
template <>
__device__ __forceinline__ uint32_t widen<__half>(uint32_t pair, uint32_t f) {
  const uint32_t w = (pair & 0x80008000u) | ((pair >> 1) & 0x3f803f80u);
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(f));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t twice(float x) {
  return pack2<T>(x, x);
}

// 2^60, twice: a scale of up to 2^48 times 2^120 is beyond bf16.
constexpr float BF16_STEP = 1.152921504606847e18f;

template <typename T>
struct Is;
template <>
struct Is<__nv_bfloat16> {
  static constexpr bool bf16 = true;
};
template <>
struct Is<__half> {
  static constexpr bool bf16 = false;
};

// Whether a chunk of 16-bit values holds one that is not finite.
template <typename T>
__device__ __forceinline__ bool not_finite(uint4 v) {
  constexpr uint32_t E = Is<T>::bf16 ? 0x7f807f80u : 0x7c007c00u, LOW = Is<T>::bf16 ? 0x00800080u : 0x04000400u;
  // (all ones in an exponent: adding its lowest bit carries into the sign's place)
  const uint32_t x = ((v.x & E) + LOW) | ((v.y & E) + LOW) | ((v.z & E) + LOW) | ((v.w & E) + LOW);
  return (x & 0x80008000u) != 0;
}
// The word with 0 in place of such values.
template <typename T>
__device__ __forceinline__ uint32_t finite_word(uint32_t w) {
  constexpr uint32_t E = Is<T>::bf16 ? 0x7f80u : 0x7c00u;
  if ((w & E) == E) w &= 0xffff0000u;
  if ((w >> 16 & E) == E) w &= 0xffffu;
  return w;
}

__device__ __forceinline__ uint4 load16(const unsigned short *p, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const uint4 *>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A tile of the caller's keys or values by the loading warps themselves, where TMA does not take it
// (off 16 bytes: 8192 tokens, 32 query heads of 128 in groups of four, 2.07 ms against 0.48):
// `tokens` of them, 0 behind.  CHECK: values that are not finite are taken out; returns
// the bits of this warp's tokens that had some.
template <typename T, int D, bool CHECK>
__device__ __forceinline__ uint32_t copy_tile(uint32_t to, const void *base, long long stride, int tokens, int tid) {
  constexpr int C = Plan<D>::CHUNKS, PER = TILE * C / (32 * LOADERS), STEP = 32 * LOADERS / C, IN_WARP = 32 / C;
  const int c = tid % C, line0 = tid / C;
  const unsigned short *p = static_cast<const unsigned short *>(base) + line0 * stride + c * 8;
  uint32_t bad = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < PER; i0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (line0 + (i0 + i) * STEP < tokens) v[i] = load16(p + (long long)(i0 + i) * STEP * stride, false);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (CHECK) {
        const uint32_t votes = __ballot_sync(FULL, not_finite<T>(v[i]));
        if (votes) {
          v[i] = make_uint4(finite_word<T>(v[i].x), finite_word<T>(v[i].y), finite_word<T>(v[i].z), finite_word<T>(v[i].w));
#pragma unroll
          for (int k = 0; k < IN_WARP; ++k)
            if (votes >> (k * C) & ((1u << C) - 1)) bad |= 1u << ((i0 + i) * IN_WARP + k);
        }
      }
      st_shared16(chunk_at(to, line0 + (i0 + i) * STEP, c), v[i].x, v[i].y, v[i].z, v[i].w);
    }
  }
  return bad;
}

// What copy_tile<.., true> does, for a tile that TMA has brought.
template <typename T, int D>
__device__ __forceinline__ uint32_t check_tile(uint32_t at, int tokens, int tid) {
  constexpr int C = Plan<D>::CHUNKS, PER = TILE * C / (32 * LOADERS), STEP = 32 * LOADERS / C, IN_WARP = 32 / C;
  const int c = tid % C, line0 = tid / C;
  uint32_t bad = 0;
#pragma unroll 4
  for (int i = 0; i < PER; ++i) {
    const int line = line0 + i * STEP;
    const uint32_t from = chunk_at(at, line, c);
    const uint4 v = lds128(from);
    const uint32_t votes = __ballot_sync(FULL, not_finite<T>(v));
    if (votes) {
      st_shared16(from, finite_word<T>(v.x), finite_word<T>(v.y), finite_word<T>(v.z), finite_word<T>(v.w));
#pragma unroll
      for (int k = 0; k < IN_WARP; ++k)  // (tokens behind the row's are others', and not its concern)
        if (votes >> (k * C) & ((1u << C) - 1) && (tid & ~31) / C + k + i * STEP < tokens) bad |= 1u << (i * IN_WARP + k);
    }
  }
  return bad;
}

// The queries of a unit's rows.
template <typename T, int D>
__device__ __forceinline__ void copy_queries(const KvNewArgs &a, const Walk &w, uint32_t to, int tid) {
  constexpr int C = Plan<D>::CHUNKS, STEP = 32 * LOADERS / C;
  const int c = tid % C;
  // (token and head of a row, and by how much they go on: no division a row)
  int t = (w.unit.r0 + tid / C) / a.group, h = (w.unit.r0 + tid / C) % a.group;
  const int dt = STEP / a.group, dh = STEP % a.group;
  const unsigned short *q = static_cast<const unsigned short *>(a.q) + c * 8 + w.row.q0 * a.q_token + w.h * a.group * a.q_head;
  const bool direct = a.q_vec && a.scale >= 0.f;
  const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0;  // (the scale is taken without its sign)
#pragma unroll 4
  for (int r = tid / C; r < w.unit.nrows; r += STEP) {
    const unsigned short *from = q + t * a.q_token + h * a.q_head;
    const uint32_t at = chunk_at(to + (r >> 7) * (M * D * 2), r & 127, c);
    if (direct) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    } else {
      const uint4 v = load16(from, a.q_vec);
      st_shared16(at, v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign);
    }
    t += dt;
    h += dh;
    if (h >= a.group) {
      h -= a.group;
      ++t;
    }
  }
  if (direct) asm volatile("cp.async.wait_all;" ::: "memory");
}

// Values that are not finite meet p = 0 in rows that do not see their tokens, and 0
// times them is NaN; so tiles that some row does not see in full hold 0 in their
// place, and what they do to the rows that see them is done afterwards, here: a row's
// result plus the value (an infinity, or NaN).  Rare, and out of the way.
template <typename T, int D>
__device__ __noinline__ void spoil(const KvNewArgs &a, const BadTile *bad, int n, int q0, int old, int h, int p, T *out,
                                   float *part) {
  constexpr int C = Plan<D>::CHUNKS, STEP = 32 * LOADERS / C, IN_WARP = 32 / C;
  for (int k = 0; k < n; ++k)
    for (int w = 0; w < LOADERS; ++w)
      for (uint32_t m = bad[k].word[w]; m; m &= m - 1) {
        const int bit = __ffs(m) - 1, t = bad[k].x + bit / IN_WARP * STEP + w * IN_WARP + bit % IN_WARP, j = old + t;
        if (j > p || (a.window > 0 && j <= p - a.window && j >= a.sinks)) continue;
        const T *v = static_cast<const T *>(a.v) + (long long)(q0 + t) * a.v_token + h * a.v_head;
        for (int d = 0; d < D; ++d) {
          const float x = to_f32(v[d]);
          if (fabsf(x) < CUDART_INF_F) continue;
          if (out) out[d] = from_f32<T>(to_f32(out[d]) + x);
          else part[(d >> 2) * (ROWS * 4) + (d & 3)] += x;
        }
      }
}

// A barrier's phases are told apart by their parity alone: whoever waits for one knows
// that the one before it is complete and that the next one cannot be.  Those of the row
// tiles' scores and products: BUFFERS each, in turn, since so many may be ahead.
enum Bar {
  FULL_AT = 0, EMPTY_AT = 8, Q_FULL = 16, Q_EMPTY = 17,
  S_FULL = 18,             // [row tile][BUFFERS]
  P_HALF = 24, P_FULL = 27,  // [buffer]: p of the first half of the tile's tokens, of the second
  PV_HALF = 30, PV_DONE = 36,  // [row tile][BUFFERS]: the products with them are done
  O_EMPTY = 42,
  RAW_AT = 44,             // [slot]: values that came to be checked (see `settle`)
  SEGMENT_OVER = 52, BARS = SEGMENT_OVER + BAD_SEGMENTS
};

template <int REGS>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// the lowest n bits, n clamped to 0 .. 32
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1; }

__device__ __forceinline__ uint64_t pair64(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
// the largest of three, as fmaxf (NaN only where all are)
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// 1 / x of a power of two within 2^+-126: exact
__device__ __forceinline__ float inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

// Rows' 64 scores at s_at less `at` and `less`.  (Out of the way: inlined it slowed down what is
// around it, by up to 3%.)
__device__ __noinline__ void lift(uint32_t s_at, float at, float less) {
#pragma unroll 1
  for (int e0 = 0; e0 < 64; e0 += 16) {
    uint32_t s[16];
    tmem_ld16(s_at + e0, s);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) - at - less);
    tmem_st16(s_at + e0, s);
  }
  tmem_wait_st();
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 1)
    new_kernel(const __grid_constant__ KvNewArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using L = Plan<D>;
  constexpr bool BF16 = Is<T>::bf16;
  constexpr int STAGES = L::STAGES;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  __shared__ __align__(8) unsigned long long bars[BARS];
  __shared__ Meta meta[META];
  __shared__ BadTile bad_tiles[BAD_SEGMENTS][BAD_TILES];
  __shared__ int bad_count[BAD_SEGMENTS];
  __shared__ Reference references[ROWS];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(FULL, tid >> 5, 0);
  uint32_t bits = 0;
  const Share &share = share_of(a, reinterpret_cast<int *>(smem), &bits);
  if (share.ctas == 0) {
    if (tid == 0) join_of(a, blockIdx.x)->parts = 0;
    if (bits) atomicOr(a.err, bits);
    return;
  }
  const uint32_t q_at = smem_addr(smem), ring = q_at + L::Q;
  auto bar = [&](int which) { return smem_addr(bars + which); };
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      bar_init(bar(FULL_AT + i), LOADERS);
      bar_init(bar(EMPTY_AT + i), 1);
      bar_init(bar(RAW_AT + i), 1);
    }
    bar_init(bar(Q_FULL), LOADERS);
    bar_init(bar(Q_EMPTY), 1);
    for (int i = 0; i < 2 * L::BUFFERS; ++i) {
      bar_init(bar(S_FULL + i), 1);
      bar_init(bar(PV_HALF + i), 1);
      bar_init(bar(PV_DONE + i), 1);
    }
    for (int i = 0; i < L::BUFFERS; ++i) {
      bar_init(bar(P_HALF + i), 4);
      bar_init(bar(P_FULL + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bar(O_EMPTY + i), 4);
    }
    for (int i = 0; i < BAD_SEGMENTS; ++i) bar_init(bar(SEGMENT_OVER + i), W_LOAD);
    bar_init_fence();
    s_abort = 0;
  }
  if (warp == W_ISSUE) tmem_alloc(smem_addr(&tmem_slot), 512);
  tmem_before_sync();
  __syncthreads();
  tmem_after_sync();
  const uint32_t tmem = tmem_slot;
  // A wait that runs out, in any role, ends the others' as well; each role then
  // leaves its loops.
  auto wait = [&](int which, uint32_t parity) {
    const uint32_t b = bar(which);
    if (bar_try(b, parity & 1)) return true;
#pragma unroll 1
    for (int i = 0; i < (1 << 20); ++i) {
      if (bar_try(b, parity & 1)) return true;
      if ((i & 15) == 15 && *reinterpret_cast<volatile int *>(&s_abort)) return false;
    }
    *reinterpret_cast<volatile int *>(&s_abort) = 1;
    bits |= SGD_KV_ERR_WAIT;
    return false;
  };
  auto warp_arrive = [&](int which) {
    __syncwarp();
    if (lane == 0) bar_arrive(bar(which));
  };

  if (warp >= W_LOAD && warp < W_LOAD + LOADERS) {
    fewer_registers<REGS_OTHER>();
    const int me = tid - 32 * W_LOAD, wl = warp - W_LOAD;
    constexpr int CHUNKS8 = D / 16, PER = TILE * CHUNKS8 / (32 * LOADERS);  // 16-byte chunks of e4m3: of a token, of a thread
    constexpr int STEP = 32 * LOADERS / CHUNKS8;
    const int c8 = me % CHUNKS8, line0 = me / CHUNKS8;
    const int per_tile = TILE >> a.c.page_bits;
    Walk w(a, share);
    uint32_t item = 0, segments = 0, g = 0;
    bool ok = true;
    auto slot_free = [&]() {
      if (item >= STAGES) ok = ok && wait(EMPTY_AT + item % STAGES, item / STAGES - 1);
      ok = __all_sync(FULL, ok);
      return ok;
    };
    // the cached tile in hand: of page `lane` of it, the block and what its keys and values
    // are multiplied by (packed), and whether that is done in two steps
    int block = -1;
    uint32_t k_by = 0, v_by = 0;
    bool twice_k = false, twice_v = false;
    Meta mt{0, 0, 0, 0u, 1.f, 1.f};
    auto pages = [&](int j) {
      const int x = w.at(j), index = (x >> a.c.page_bits) + lane;
      const bool in = lane < per_tile && index << a.c.page_bits < w.row.old;
      block = -1;
      float ks = 0.f, vs = 0.f;
      if (in) {
        const int pg = __ldg(a.r.table + (long long)w.b * a.r.max_pages + index);
        if (pg >= 0 && pg < a.c.num_pages) {
          block = pg * a.c.heads + w.h;
          ks = __ldg(a.c.ks + block);
          vs = __ldg(a.c.vs + block);
        } else {
          bits |= SGD_KV_ERR_PAGE;
        }
      }
      const uint32_t lost = __ballot_sync(FULL, in && block < 0);
      mt.gone = 0;
      if (lost)
        for (int i = 0; i < per_tile; ++i)
          if (lost >> i & 1) mt.gone |= ((1u << ((1 << a.c.page_bits) / 16)) - 1) << (i << (a.c.page_bits - 4));
      if (BF16) {
        // 2^120 times a scale above 2^7 is beyond bf16
        twice_k = __any_sync(FULL, ks > 128.f);
        twice_v = __any_sync(FULL, vs > 128.f);
        k_by = twice<T>(ks * (twice_k ? BF16_STEP : BF16_STEP * BF16_STEP));
        v_by = twice<T>(vs * (twice_v ? BF16_STEP : BF16_STEP * BF16_STEP));
      } else {
        // f16 has not the range of the scales: keys and values are brought to the largest
        // scale of the tile (those of much smaller ones lose bits below 2^-24 of it)
        float km = ks, vm = vs;
#pragma unroll
        for (int o = 4; o; o >>= 1) {
          km = fmaxf(km, __shfl_xor_sync(FULL, km, o));
          vm = fmaxf(vm, __shfl_xor_sync(FULL, vm, o));
        }
        km = __shfl_sync(FULL, km, 0);
        vm = __shfl_sync(FULL, vm, 0);
        mt.k = km > 0.f ? km : 1.f;
        mt.v = vm > 0.f ? vm : 1.f;
        k_by = twice<T>(ks * (256.f / mt.k));
        v_by = twice<T>(vs * (256.f / mt.v));
      }
    };
    uint4 raw[PER];  // what the thread has of the item in hand, then of the next
    auto load8 = [&](const uint8_t *base, int i) {
      const int t = line0 + i * STEP, blk = __shfl_sync(FULL, block, t >> a.c.page_bits);
      raw[i] = make_uint4(0, 0, 0, 0);
      if (blk >= 0)
        raw[i] = __ldg(reinterpret_cast<const uint4 *>(base + ((long long)blk * a.c.page + (t & (a.c.page - 1))) * D) + c8);
    };
    // the i-th chunk into the ring
    const int swap = D == 128 ? c8 >> 2 & 1 : 0;  // (lanes of a token's second half store in the other order: no bank twice)
    auto store8 = [&](uint32_t to, int i, uint32_t by_lane, bool twice_by) {
      const int t = line0 + i * STEP;
      const uint32_t by = __shfl_sync(FULL, by_lane, t >> a.c.page_bits);
      const uint4 v = swap ? make_uint4(raw[i].z, raw[i].w, raw[i].x, raw[i].y) : raw[i];
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[2 * e] = widen<T>(__byte_perm(in[e], 0, 0x1404), by);
        h[2 * e + 1] = widen<T>(__byte_perm(in[e], 0, 0x3424), by);
      }
      if (BF16 && twice_by) {
#pragma unroll
        for (int e = 0; e < 8; ++e) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(twice<T>(BF16_STEP)));
      }
      st_shared16(chunk_at(to, t, 2 * c8 + swap), h[0], h[1], h[2], h[3]);
      st_shared16(chunk_at(to, t, 2 * c8 + 1 - swap), h[4], h[5], h[6], h[7]);
    };
    // hands the slot in hand to the products
    auto done = [&]() {
      async_fence();
      warp_arrive(FULL_AT + item % STAGES);
      ++item;
    };
    auto by_tma = [&](const CUtensorMap *map, int token) {
      if (wl == 0 && lane == 0) {
        const uint32_t to = ring + item % STAGES * L::HALF, b = bar(FULL_AT + item % STAGES);
        bar_expect(b, L::HALF);
#pragma unroll
        for (int d = 0; d < D; d += 64) tma_load_3d(to + d * (TILE * 2), map, d, w.h, token, b);
      } else if (lane == 0) {
        bar_arrive(bar(FULL_AT + item % STAGES));
      }
      __syncwarp();
      ++item;
    };
    // A tile of values with an edge, on its way: checked once the loads behind it are under
    // way too.  Its slot, tokens, first token, and where what is found goes.
    bool late = false;
    // (Its barrier is its slot's: one warp may be several tiles ahead of another, but not a
    // whole round of slots.  parities: of the slots' next uses.)
    uint32_t raw_slot = 0, parities = 0, raw_segment = 0;
    int raw_tokens = 0, raw_from = 0, raw_index = 0;
    auto note = [&](uint32_t segment, int index, int from, uint32_t bad) {
      BadTile &e = bad_tiles[segment % BAD_SEGMENTS][index];
      if (lane == 0) e.word[wl] = bad;
      if (wl == 0 && lane == 0) {
        e.x = from;
        bad_count[segment % BAD_SEGMENTS] = index + 1;
      }
    };
    auto settle = [&]() {
      if (!late) return;
      late = false;
      ok = ok && wait(RAW_AT + raw_slot, parities >> raw_slot);
      parities ^= 1u << raw_slot;
      ok = __all_sync(FULL, ok);
      if (!ok) return;
      note(raw_segment, raw_index, raw_from, check_tile<T, D>(ring + raw_slot * L::HALF, raw_tokens, me));
      async_fence();
      warp_arrive(FULL_AT + raw_slot);
    };
    while (ok && w.next(&bits)) {
      if (w.t0 == w.t1) continue;
      if (segments >= BAD_SEGMENTS) {
        ok = wait(SEGMENT_OVER + segments % BAD_SEGMENTS, segments / BAD_SEGMENTS - 1);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
      }
      if (w.cached(w.t0)) {
        pages(w.t0);
#pragma unroll
        for (int i = 0; i < PER; ++i) load8(a.c.k, i);
      }
      int bads = 0;
      for (int j = w.t0; j < w.t1; ++j) {
        const int x = w.at(j);
        const bool cached = w.cached(j);
        const int from = x - w.row.old, tokens = w.row.ql - from;  // (of a tile of new ones: its first, and how many there are)
        if (wl == 0 && lane == 0) {
          if (j == w.t0) bad_count[segments % BAD_SEGMENTS] = 0;
          Meta &to = meta[g % META];
          to.edge = w.edge(j, x) || (cached && mt.gone);
          to.x = x;
          to.last = cached ? w.row.old - 1 : w.row.old + w.row.ql - 1;
          to.gone = cached ? mt.gone : 0u;
          to.k = cached ? mt.k : 1.f;
          to.v = cached ? mt.v : 1.f;
        }
        ++g;
        if (!slot_free()) break;
        if (cached) {
          // (a chunk's registers take the next item's, with as long as this item takes to arrive)
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            store8(ring + item % STAGES * L::HALF, i, k_by, twice_k);
            load8(a.c.v, i);
          }
          done();
        } else if (a.k_vec) {
          by_tma(&kmap, w.row.q0 + from);
        } else {
          copy_tile<T, D, false>(ring + item % STAGES * L::HALF,
                                 static_cast<const T *>(a.k) + (w.row.q0 + from) * a.k_token + w.h * a.k_head, a.k_token,
                                 tokens, me);
          done();
        }
        settle();
        if (!ok) break;
        if (j == w.t0) {
          if (segments > 0) ok = wait(Q_EMPTY, segments - 1);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
          copy_queries<T, D>(a, w, q_at, me);
          async_fence();
          warp_arrive(Q_FULL);
        }
        if (!slot_free()) break;
        if (cached) {
          const uint32_t by = v_by;
          const bool two_steps = twice_v, more = j + 1 < w.t1 && w.cached(j + 1);
          if (more) pages(j + 1);
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            store8(ring + item % STAGES * L::HALF, i, by, two_steps);
            if (more) load8(a.c.k, i);
          }
          done();
        } else if (a.v_vec && !w.edge(j, x)) {
          by_tma(&vmap, w.row.q0 + from);
        } else if (!w.edge(j, x)) {
          copy_tile<T, D, false>(ring + item % STAGES * L::HALF,
                                 static_cast<const T *>(a.v) + (w.row.q0 + from) * a.v_token + w.h * a.v_head, a.v_token,
                                 tokens, me);
          done();
        } else {
          // (at most 7 tiles of a unit have an edge: 3 where its rows' tokens are, 3 where
          // their windows begin, 1 where the first tokens end)
          const int index = min(bads++, BAD_TILES - 1);
          if (a.v_vec) {
            late = true;
            raw_slot = item % STAGES;
            raw_segment = segments;
            raw_tokens = tokens;
            raw_from = from;
            raw_index = index;
            if (wl == 0 && lane == 0) {
              const uint32_t to = ring + raw_slot * L::HALF, b = bar(RAW_AT + raw_slot);
              bar_expect(b, L::HALF);
#pragma unroll
              for (int d = 0; d < D; d += 64) tma_load_3d(to + d * (TILE * 2), &vmap, d, w.h, w.row.q0 + from, b);
            }
            __syncwarp();
            ++item;
          } else {
            note(segments, index, from,
                 copy_tile<T, D, true>(ring + item % STAGES * L::HALF,
                                       static_cast<const T *>(a.v) + (w.row.q0 + from) * a.v_token + w.h * a.v_head, a.v_token,
                                       tokens, me));
            done();
          }
        }
        if (!cached && j + 1 < w.t1 && w.cached(j + 1)) {
          pages(j + 1);
#pragma unroll
          for (int i = 0; i < PER; ++i) load8(a.c.k, i);
        }
      }
      ++segments;
    }
    settle();
    if (!ok) {
      // (Copies in flight land before the CTA ends: they take microseconds.  Their barriers
      // may never complete, since other warps arrive at them too.)
      for (int n = 0; n < (1 << 12); ++n) __nanosleep(256);
    }
  } else if (warp >= W_ISSUE) {
    fewer_registers<REGS_OTHER>();
    if (warp == W_ISSUE) {
      // The whole warp walks, so that addresses and counters are the warp's (in its
      // uniform registers, where the products take them from); one thread issues.  What it
      // executes from one p to the next scores adds to every tile's time: little.
      constexpr uint32_t QK = product16(BF16, TILE, false), PV = product16(BF16, D, true), HIGH = operand_high(1024);
      constexpr uint32_t SLOT = L::HALF / 16;
      Walk w(a, share);
      const uint32_t bars0 = smem_addr(bars);
      auto ready = [&](uint32_t at, uint32_t parity) {
        if (__all_sync(FULL, bar_try(bars0 + at * 8, parity))) return true;
        return (bool)__all_sync(FULL, wait(at, parity));
      };
      const uint32_t q_low = operand_low(q_at, 0), k_low = operand_low(ring, 0), v_low = operand_low(ring, TILE * 128);
      // (half of a tile's tokens at a time: the products with the first run while p of the second is made)
      // the next keys' and values' slots, and the parity of their barriers
      uint32_t ks = 0, k_par = 0, vs = 1, v_par = 0;
      // of the products in turn: the buffer of the next scores, of the next p, and its parity
      uint32_t s_buf = 0, p_buf = 0, p_par = 0;
      // of either row tile: the barriers of its next scores and of its next products with p
      uint32_t s_bar0 = 0, s_bar1 = 0, p_bar0 = 0, p_bar1 = 0;
      uint32_t segments = 0, segs1 = 0;
      bool ok = true;
      while (ok && w.next(&bits)) {
        const int n = __reduce_max_sync(FULL, w.t1 - w.t0);
        if (n == 0) continue;
        const uint32_t two = __reduce_max_sync(FULL, (uint32_t)(w.unit.nrows > M));
        ok = ready(Q_FULL, segments & 1);
        // scores: row tile qi, key tile qj
        uint32_t qi = 0;
        int qj = 0;
        auto scores = [&]() {
          if (qi == 0) ok = ok && ready(FULL_AT + ks, k_par);
          if (!ok) return;
          tmem_after_sync();
          if (elect_one()) {
            const uint32_t q = q_low + qi * (M * D * 2 / 16), k = k_low + ks * SLOT, to = tmem + L::S + s_buf * TILE;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
              const uint32_t off = ((e / 4) * (TILE * 128) + (e % 4) * 32) / 16;
              mma_ss(to, q + off, k + off, HIGH, QK, e > 0);
            }
            mma_commit(bars0 + (S_FULL + (qi ? L::BUFFERS + s_bar1 : s_bar0)) * 8);
            if (qi == two) {
              mma_commit(bars0 + (EMPTY_AT + ks) * 8);
              if (qj + 1 == n) mma_commit(bars0 + Q_EMPTY * 8);
            }
          }
          __syncwarp();
          if (qi) s_bar1 = s_bar1 + 1 == L::BUFFERS ? 0 : s_bar1 + 1;
          else s_bar0 = s_bar0 + 1 == L::BUFFERS ? 0 : s_bar0 + 1;
          s_buf = s_buf + 1 == L::BUFFERS ? 0 : s_buf + 1;
          if (qi == two) {
            qi = 0;
            ++qj;
            ks += 2;
            if (ks >= STAGES) {
              ks = 0;
              k_par ^= 1;
            }
          } else {
            qi = 1;
          }
        };
#pragma unroll 1
        for (int x = 0; x < L::BUFFERS && qj < n; ++x) scores();
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j) {
          ok = ready(FULL_AT + vs, v_par);
#pragma unroll 1
          for (uint32_t i = 0; ok && i <= two; ++i) {
            if (j == 0) {
              const uint32_t before = i ? segs1 : segments;
              if (before > 0) ok = ready(O_EMPTY + i, (before - 1) & 1);
            }
            ok = ok && ready(P_HALF + p_buf, p_par);
            if (!ok) break;
            const uint32_t v = v_low + vs * SLOT, p = tmem + L::S + p_buf * TILE, o = tmem + L::O + i * D;
            const uint32_t of = (i ? L::BUFFERS + p_bar1 : p_bar0) * 8;
            tmem_after_sync();
            if (elect_one()) {
              mma_ts(o, p, v, HIGH, PV, j > 0);
#pragma unroll
              for (int e = 1; e < 4; ++e) mma_ts(o, p + e * 8, v + e * (2048 / 16), HIGH, PV, true);
              mma_commit(bars0 + PV_HALF * 8 + of);
            }
            __syncwarp();
            ok = ready(P_FULL + p_buf, p_par);
            if (!ok) break;
            tmem_after_sync();
            if (elect_one()) {
#pragma unroll
              for (int e = 4; e < TILE / 16; ++e) mma_ts(o, p + e * 8, v + e * (2048 / 16), HIGH, PV, true);
              mma_commit(bars0 + PV_DONE * 8 + of);
              if (i == two) mma_commit(bars0 + (EMPTY_AT + vs) * 8);
            }
            __syncwarp();
            if (i) p_bar1 = p_bar1 + 1 == L::BUFFERS ? 0 : p_bar1 + 1;
            else p_bar0 = p_bar0 + 1 == L::BUFFERS ? 0 : p_bar0 + 1;
            if (++p_buf == L::BUFFERS) {
              p_buf = 0;
              p_par ^= 1;
            }
            if (qj < n) scores();
          }
          vs += 2;
          if (vs >= STAGES) {
            vs = 1;
            v_par ^= 1;
          }
        }
        ++segments;
        segs1 += two;
      }
    } else if (warp == W_JOIN && lane == 0) {
      // the unit that this share ends within, if it begins here: how many shares hold it
      Join join{0, 0, 0, 0, 0};
      if (share.end.t > 0 && (share.end.u > share.begin.u || (share.begin.t == 0 && !share.begin.past))) {
        const BatchRow r = batch_row(a, share.end.b, &bits);
        const Unit u = unit_of(a, r, share.end.i);
        join.parts = 2;
        for (int g = blockIdx.x + 2; g < share.ctas; ++g) {
          const long long into = quotient(share.all * g, share.ctas) - share.u_at;
          if (into >= OVERHEAD + share.end_tiles) break;
          Cut c;
          place_cut(c, into, share.end_tiles);
          if (c.past) break;
          ++join.parts;
        }
        join.q0 = r.q0;
        join.r0 = u.r0;
        join.nrows = u.nrows;
        join.h = share.end.h;
      }
      *join_of(a, blockIdx.x) = join;
    }
    __syncwarp();
  } else {
    more_registers<REGS_SOFTMAX>();
    const int i = warp >> 2, r = tid & 127, R = i * M + r;  // the warpgroup's row tile, the thread's row of it, of the unit
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t o_at = tmem + lanes + L::O + i * D;
    const float c0 = fmaxf(fabsf(a.scale) * LOG2E, 1e-37f);
    constexpr float UP = Range<T>::UP, THRESHOLD = Range<T>::THRESHOLD;
    Reference &reference = references[R];
    Walk w(a, share);
    uint32_t g = 0, segments = 0;
    uint32_t buf = 0;            // of the next segment's first scores
    uint32_t turn = 0, use = 0;  // of the row tile's next scores: their barriers, and how often those were used before
    bool ok = true;
    while (ok && w.next(&bits)) {
      const int tiles = w.t1 - w.t0, two = w.unit.nrows > M;
      const int t = (w.unit.r0 + R) / a.group, p = w.row.old + t;
      T *out = static_cast<T *>(a.out) + ((long long)(w.row.q0 + t) * a.q_heads + w.h * a.group + (w.unit.r0 + R) % a.group) * D;
      if (tiles == 0) {
        if (R < w.unit.nrows)
          for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4 *>(out + d) = make_uint4(0, 0, 0, 0);
        continue;
      }
      uint32_t s_buf = (buf + i) % L::BUFFERS;
      buf = (buf + ((uint32_t)tiles << two)) % L::BUFFERS;
      if (i > two) {
        // (no rows here.  Not further ahead than the phase before, or this warpgroup would
        // arrive in the other's place)
        if (segments >= BAD_SEGMENTS) ok = wait(SEGMENT_OVER + segments % BAD_SEGMENTS, segments / BAD_SEGMENTS - 1);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        g += tiles;
        warp_arrive(SEGMENT_OVER + segments % BAD_SEGMENTS);
        ++segments;
        continue;
      }
      const bool live = R < w.unit.nrows;
      // the reference's exponent; -inf: there is none yet, or a far one
      float m = live ? -CUDART_INF_F : 0.f, l = 0.f;  // (what rows that are not there hold does not matter)
      uint32_t turn_before = 0, use_before = 0;
#pragma unroll 1
      for (int j = 0; j < tiles; ++j, ++g) {
        ok = wait(S_FULL + i * L::BUFFERS + turn, use);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        tmem_after_sync();
        const uint32_t s_at = tmem + lanes + L::S + s_buf * TILE;
        uint32_t sa[32], sb[32], pk[32];
        if (j > 0) tmem_ld32(s_at, sa);
        const Meta &mt = meta[g % META];
        const int edge = mt.edge;
        // z = s c; m is that of z + log2 V, V the scale that the tile's values were brought to
        const float c = BF16 ? c0 : fmaxf(c0 * mt.k, 1e-37f), lv = BF16 ? 0.f : __log2f(mt.v);
        const uint64_t c2 = pair64(c, c), one = pair64(1.f, 1.f);
        // -inf in place of what the row does not see, of 32 tokens from e0 on
        auto mask = [&](uint32_t (&s)[32], int e0) {
          const int x = mt.x + e0;
          uint32_t see = low_bits(min(p, mt.last) - x + 1);
          if (a.window > 0) see &= ~low_bits(p - a.window + 1 - x) | low_bits(a.sinks - x);
          const uint32_t gone = mt.gone >> (e0 / 16);
          if (gone & 1) see &= 0xffff0000u;
          if (gone & 2) see &= 0xffffu;
          if (__all_sync(FULL, see == 0xffffffffu)) return;  // (half of an edge's tile, mostly)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(see >> e & 1)) s[e] = 0xff800000u;
          __syncwarp();
        };
        // Half of the tokens at a time, so that the products with the first run beside the
        // exponentials of the second.  (Loops rather than straight code: what 16 warps in
        // three roles run has to stay in the instruction cache.)
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          bool first = j + half == 0;  // (of a segment: there is no reference yet)
          bool lifted = false;         // scores of rows with a far reference are relative to it
          float sum = 0.f;
          while (true) {
            bool grown = first;
            if (!first) {
              const float base = (m == -CUDART_INF_F ? 0.f : m) - UP - lv;
              const uint64_t b2 = pair64(-base, -base);
              uint64_t sum0 = 0, sum1 = 0;
              float top0 = -CUDART_INF_F, top1 = -CUDART_INF_F;
              // 32 tokens' p relative to m as it is, and their sum
              auto exps = [&](const uint32_t (&s)[32], uint32_t *to) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  float y[4];
                  if (!BF16) {
                    top0 = max3(top0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    top1 = max3(top1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
                  }
                  unpair(fma2(pair64(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, b2), y[0], y[1]);
                  unpair(fma2(pair64(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), c2, b2), y[2], y[3]);
#pragma unroll
                  for (int q = 0; q < 4; ++q) y[q] = ex2_approx(y[q]);
                  sum0 = fma2(pair64(y[0], y[1]), one, sum0);
                  sum1 = fma2(pair64(y[2], y[3]), one, sum1);
                  to[e / 2] = pack2<T>(y[0], y[1]);
                  to[e / 2 + 1] = pack2<T>(y[2], y[3]);
                }
              };
              tmem_wait_ld();
              tmem_ld32(s_at + half * 64 + 32, sb);
              if (edge) mask(sa, half * 64);
              exps(sa, pk);
              tmem_wait_ld();
              if (half == 0) tmem_ld32(s_at + 64, sa);
              if (edge) mask(sb, half * 64 + 32);
              exps(sb, pk + 16);
              float u0, u1;
              unpair(fma2(sum0, one, sum1), u0, u1);
              sum = u0 + u1;
              if (BF16) {
                grown = live && (l + sum > L_MOST || m == -CUDART_INF_F);
              } else {
                const float top = fmaf(fmaxf(top0, top1), c, lv);
                grown = live && (top > m + THRESHOLD || (m == -CUDART_INF_F && top > m));
              }
            }
            if (!__any_sync(FULL, grown)) break;
            if (lifted) break;  // (NaN, or nothing seen so far)
            // p would be too large for the reference as it is (rarely but for a segment's first half):
            // the reference rises, o and l are scaled to it, and p is made anew.
            tmem_wait_ld();
            float largest = -CUDART_INF_F;
#pragma unroll 1
            for (int e0 = half * 64 + 32; e0 >= half * 64; e0 -= 32) {
              tmem_ld32(s_at + e0, sb);
              tmem_wait_ld();
              if (edge) mask(sb, e0);
#pragma unroll
              for (int e = 0; e < 32; e += 2) largest = max3(largest, __uint_as_float(sb[e]), __uint_as_float(sb[e + 1]));
            }
            Reference ref{-CUDART_INF_F, 0.f, 0};
            if (live && !first) ref = reference;
            const bool none = ref.s == -CUDART_INF_F;
            // the exponent of the largest p
            const float y = ref.far ? fmaf(largest - (BF16 ? ref.s : ref.s * inverse(mt.k)), c, lv - ref.add + UP) : fmaf(largest, c, UP - m + lv);
            const bool must = !none && (BF16 ? l + (ref.far ? 64.f * ex2_approx(y) : sum) > L_MOST : y > UP + THRESHOLD);
            const bool rising = __any_sync(FULL, must && largest < CUDART_INF_F);
            const bool up = must || (live && (none ? largest > -CUDART_INF_F : rising && y > UP + WITH));
            if (!first && !__any_sync(FULL, up || ref.far)) break;  // (NaN, or nothing seen so far)
            float o_scale = 1.f;
            if (up) {
              if (none || !BF16 || y > UP + 1.f) {
                o_scale = none ? 0.f : ex2_approx(UP - y);
                m = fmaxf(fmaf(largest, c, lv), -FLT_MAX);
                ref = Reference{BF16 ? largest : largest * mt.k, lv, fabsf(m) >= FAR};
                if (ref.far) m = -CUDART_INF_F;
              } else {
                o_scale = ex2_approx(-RISE);
                ref.add += RISE;
                m += RISE;
              }
              l *= o_scale;
            }
            if (live) reference = ref;
            __syncwarp();
            if (!first && __any_sync(FULL, up)) {
              if (j > 0) ok = wait(PV_DONE + i * L::BUFFERS + turn_before, use_before);
              if (half > 0) ok = ok && wait(PV_HALF + i * L::BUFFERS + turn, use);
              ok = __all_sync(FULL, ok);
              if (!ok) break;
              tmem_after_sync();
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                tmem_ld16(o_at + d, sa);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) sa[e] = __float_as_uint(__uint_as_float(sa[e]) * o_scale);
                tmem_st16(o_at + d, sa);
              }
              tmem_wait_st();
            }
            first = false;
            if (__any_sync(FULL, ref.far)) {
              // scores relative to such references, so that m does not matter
              const float at = ref.far ? (BF16 ? ref.s : ref.s * inverse(mt.k)) : 0.f, less = ref.far ? __fdividef(ref.add, c) : 0.f;
              lift(s_at + half * 64, at, less);
              lifted = true;
            }
            tmem_ld32(s_at + half * 64, sa);
          }
          if (!ok) break;
          l = BF16 ? l + sum : fmaf(sum, __fdividef(1.f, mt.v), l);
          tmem_st32(s_at + half * 32, pk);
          tmem_wait_st();
          tmem_before_sync();
          warp_arrive((half ? P_FULL : P_HALF) + s_buf);
        }
        if (!ok) break;
        if ((s_buf += 1 + two) >= L::BUFFERS) s_buf -= L::BUFFERS;
        turn_before = turn;
        use_before = use;
        if (++turn == L::BUFFERS) {
          turn = 0;
          ++use;
        }
      }
      if (!ok) break;
      // ---- the segment's result
      ok = wait(PV_DONE + i * L::BUFFERS + turn_before, use_before);
      ok = __all_sync(FULL, ok);
      if (!ok) break;
      tmem_after_sync();
      const bool whole = w.whole();
      const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      float *part = new_part<D>(a, slot) + R * 4;
      const bool nothing = !whole && live && reference.s == -CUDART_INF_F;
      // (a row sees itself: 0 only where its scores are all -inf, and then the result is NaN)
      const float inv = nothing ? 0.f : 1.f / l;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        tmem_ld32(o_at + d, o);
        tmem_wait_ld();
        if (R >= w.unit.nrows) {
          // (nowhere to go)
        } else if (whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(o[8 * e + q]) * inv;
            reinterpret_cast<uint4 *>(out + d)[e] =
                make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4 *>(part + (d / 4 + e) * (ROWS * 4)) =
                make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv, __uint_as_float(o[4 * e + 2]) * inv,
                            __uint_as_float(o[4 * e + 3]) * inv);
        }
        __syncwarp();  // (a warp's rows may end within it, and the next load is the whole warp's)
      }
      tmem_before_sync();
      warp_arrive(O_EMPTY + i);
      if (R < w.unit.nrows) {
        if (!whole) {
          float *ml = new_part<D>(a, slot) + ROWS * D + R;
          ml[0] = reference.s;
          ml[ROWS] = nothing ? 0.f : reference.add + __log2f(l);
        }
        const int n = bad_count[segments % BAD_SEGMENTS];
        uint32_t any = 0;
        for (int k = 0; k < n; ++k)
          for (int q = 0; q < LOADERS; ++q) any |= bad_tiles[segments % BAD_SEGMENTS][k].word[q];
        if (any)
          spoil<T, D>(a, bad_tiles[segments % BAD_SEGMENTS], n, w.row.q0, w.row.old, w.h, p, whole ? out : nullptr, part);
      }
      warp_arrive(SEGMENT_OVER + segments % BAD_SEGMENTS);
      ++segments;
    }
  }
  if (bits) atomicOr(a.err, bits);
  tmem_before_sync();
  __syncthreads();
  tmem_after_sync();
  if (warp == W_ISSUE) tmem_free(tmem, 512);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The parts of the units that cuts went through: 32 rows a block, lanes along rows, a
// warp's share of the dims each.  The parts' weights first, then the sums with all of a
// warp's dims of several parts in flight (with one load after the other a chunk of 68
// tokens over 2032, in five parts, took 15 us here, half of its attention).
constexpr int JOIN_THREADS = 256;
template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ KvNewArgs a) {
  constexpr int W = JOIN_THREADS / 32, E = D / 4 / W;  // float4s of a warp
  extern __shared__ float s_w[];                       // [parts][32] each of the parts' s and add
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join join = *join_of(a, blockIdx.x);
  const int R = blockIdx.y * 32 + lane;
  if (join.parts == 0 || (int)blockIdx.y * 32 >= join.nrows) return;
  auto slot = [&](int p) { return new_part<D>(a, 2 * (blockIdx.x + p) + (p == 0 ? 1 : 0)); };
  float *s_add = s_w + join.parts * 32;
  for (int p = warp; p < join.parts; p += W) {
    const float *weight = slot(p) + ROWS * D + R;
    s_w[p * 32 + lane] = weight[0];
    s_add[p * 32 + lane] = weight[ROWS];
  }
  __syncthreads();
  // relative to the largest, by differences (see FAR)
  const float c0 = fmaxf(fabsf(a.scale) * LOG2E, 1e-37f);
  float s0 = s_w[lane], add0 = s_add[lane], all = 0.f;
  for (int p = 1; p < join.parts; ++p) {
    const float s = s_w[p * 32 + lane], add = s_add[p * 32 + lane];
    if (fmaf(s - s0, c0, add - add0) > 0.f) {
      s0 = s;
      add0 = add;
    }
  }
  auto weight = [&](int p) { return ex2_approx(fmaf(s_w[p * 32 + lane] - s0, c0, s_add[p * 32 + lane] - add0)); };
  for (int p = 0; p < join.parts; ++p) all += weight(p);
  // (weights that add up to 1: no sum beyond the largest value)
  const float inv = 1.f / all;
  float4 x[E] = {};
#pragma unroll 4
  for (int p = 0; p < join.parts; ++p) {
    const float *from = slot(p) + (warp * E * ROWS + R) * 4;
    const float k = weight(p) * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float4 v = *reinterpret_cast<const float4 *>(from + e * (ROWS * 4));
      x[e].x = fmaf(v.x, k, x[e].x);
      x[e].y = fmaf(v.y, k, x[e].y);
      x[e].z = fmaf(v.z, k, x[e].z);
      x[e].w = fmaf(v.w, k, x[e].w);
    }
  }
  if (R >= join.nrows) return;
  const int row = join.r0 + R;
  T *out = static_cast<T *>(a.out) +
           ((long long)(join.q0 + row / a.group) * a.q_heads + join.h * a.group + row % a.group) * D + warp * E * 4;
#pragma unroll
  for (int e = 0; e < E; ++e)
    *reinterpret_cast<uint2 *>(out + e * 4) = make_uint2(pack2<T>(x[e].x, x[e].y), pack2<T>(x[e].z, x[e].w));
}
// (a unit has at most as many parts as there are CTAs)
constexpr int join_smem(int ctas) { return ctas * 32 * 2 * 4; }

// Within what the workspace and the join's shared memory are laid out for.
constexpr int NEW_MAX_CTAS = 190;
static_assert(join_smem(NEW_MAX_CTAS) <= 48 * 1024 && NEW_MAX_CTAS <= MAX_CTAS, "the parts' weights");
int new_ctas(int sms) { return sms < NEW_MAX_CTAS ? sms : NEW_MAX_CTAS; }

template <typename T, int D>
cudaError_t launch(KvNewArgs a, cudaStream_t st, int *launches) {
  CUtensorMap k = {}, v = {};
  // (strides that a map does not take: the loading warps copy the tiles)
  a.k_vec = a.k_vec && kv_make_token_map(&k, a.k, D, a.c.heads, a.r.N, a.k_head, a.k_token, TILE);
  a.v_vec = a.v_vec && kv_make_token_map(&v, a.v, D, a.c.heads, a.r.N, a.v_head, a.v_token, TILE);
  const int ctas = new_ctas(a.sms);
  new_kernel<T, D><<<ctas, THREADS, Plan<D>::SMEM, st>>>(a, k, v);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  *launches = 2;
  // (launched while the first kernel ends, it waits there for its results)
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = dim3(ctas, ROWS / 32);
  c.blockDim = dim3(JOIN_THREADS);
  c.dynamicSmemBytes = join_smem(ctas);
  c.stream = st;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, join_kernel<T, D>, a);
}

template <typename T, int D>
cudaError_t limit() {
  return cudaFuncSetAttribute(new_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<D>::SMEM);
}

}  // namespace

size_t kv_new_workspace(int sms) {
  const size_t ctas = new_ctas(sms);
  return (size_t)MAX_CTAS * 8 + MAX_CTAS * 32 + ctas * 2 * (ROWS * (128 + 2) * 4);
}

cudaError_t kv_new_set_limits() {
  cudaError_t e = limit<__half, 128>();
  if (e == cudaSuccess) e = limit<__half, 64>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = limit<__nv_bfloat16, 64>();
  return e;
}

cudaError_t launch_kv_new(const KvNewArgs &a, int dtype, cudaStream_t st, int *launches) {
  *launches = 1;
  if (a.c.dim == 128) return dtype == SGD_F16 ? launch<__half, 128>(a, st, launches) : launch<__nv_bfloat16, 128>(a, st, launches);
  return dtype == SGD_F16 ? launch<__half, 64>(a, st, launches) : launch<__nv_bfloat16, 64>(a, st, launches);
}

}  // namespace sgd
