// kv_sched.cuh -- how the attention's work is cut: rows, units, tiles, shares.
//
// A unit is up to M rows (new token, query head of the group) of one batch row
// and one head of keys and values; its work is the list of key tiles that the
// batch row's new tokens see, each weighted by what the unit's rows make it cost.
// All tiles of all units, one after the other, are cut into equal shares, one
// per CTA, wherever the cut falls (within a tile: before it): rows of very
// unequal length keep every SM busy to the end.  A unit that a cut goes through
// is joined from its parts by the CTA that finishes last, in the order of the
// parts, so that the result does not depend on which CTA that is.
#pragma once

#include "kv_internal.h"
#include "sgd_internal.h"

namespace sgd {

// What one batch row asks for.
struct KvJob {
  int q0, ql, n;       // first packed token, new tokens, cached tokens
  int sink_tiles;      // tiles of first tokens before the others
  int lo_tile, tiles;  // the others start at lo_tile; all tiles
  int units;           // of one head: all but the last have M rows
  int cost, cost_last; // of a tile of the units before the last; of the last

  // the token tile of the j-th tile of the list
  __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : lo_tile + j - sink_tiles; }
};

// The kernel's M: rows of a unit; TILE: tokens of a tile; cost(rows): of a tile.
template <class K>
__device__ __forceinline__ KvJob kv_job(const KvAttendArgs &a, int b, uint32_t *bits) {
  constexpr int TILE = K::TILE;
  KvJob r;
  const int q0 = __ldg(a.r.q_start + b), q1 = __ldg(a.r.q_start + b + 1);
  r.n = __ldg(a.r.seq_lens + b);
  r.q0 = q0;
  r.ql = q1 - q0;
  if (q0 < 0 || q1 > a.r.N || r.ql < 0) {
    *bits |= SGD_KV_ERR_LENGTH;
    r.ql = 0;
  }
  r.units = (int)(((long long)r.ql * a.group + K::M - 1) / K::M);
  r.cost = K::cost(K::M);
  r.cost_last = K::cost(r.ql * a.group - (r.units - 1) * K::M);
  r.sink_tiles = r.lo_tile = 0;
  if (r.ql > 0 && (r.n < r.ql || (long long)r.n > (long long)a.r.max_pages * a.c.page)) {
    *bits |= SGD_KV_ERR_LENGTH;  // sees nothing: one tile, which no token sees
    r.n = 0;
    r.tiles = 1;
    return r;
  }
  const int first = r.n - r.ql;  // position of the first new token
  int lo = 0;
  if (a.window > 0) lo = max(0, first - a.window + 1);
  r.lo_tile = lo / TILE;
  r.sink_tiles = min((int)(((long long)min(a.sinks, r.n) + TILE - 1) / TILE), r.lo_tile);
  r.tiles = r.sink_tiles + (r.n + TILE - 1) / TILE - r.lo_tile;
  return r;
}

__device__ __forceinline__ long long kv_head_work(const KvJob &j) {
  return j.units ? ((long long)(j.units - 1) * j.cost + j.cost_last) * j.tiles : 0;
}
__device__ __forceinline__ long long kv_work(const KvJob &j, int heads) { return kv_head_work(j) * heads; }

// (A 64-bit division takes about a hundred instructions, and at one token of one
// row the scheduling is most of what a warp executes.)
static __device__ __noinline__ long long wide_quotient(long long x, long long y) { return x / y; }
__device__ __forceinline__ long long quotient(long long x, long long y) {
  return (x | y) >> 31 ? wide_quotient(x, y) : (long long)((unsigned)x / (unsigned)y);
}

// A CTA's share [begin, end) of the work, and the batch row where it begins.  The
// first `more` shares are of each + 1, the others of each.
struct KvShare {
  long long begin, end;
  long long each;
  int ctas, more;
  int b;                // batch row of `begin`
  long long b_begin;    // the work before row b

  __device__ __forceinline__ long long cut(int g) const { return each * g + min(g, more); }
  // the CTA whose share holds `at`
  __device__ __forceinline__ int cta_of(long long at) const {
    const long long large = (each + 1) * more;
    return at < large ? (int)quotient(at, each + 1) : more + (int)quotient(at - large, each);
  }
};

// By all threads of the block.  `least`: work that makes a share worth a CTA.
template <class K, int THREADS>
__device__ KvShare kv_share(const KvAttendArgs &a, int least, uint32_t *bits) {
  __shared__ long long s_warp[THREADS / 32];
  __shared__ long long s_before;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.r.B + THREADS - 1) / THREADS;
  const int b0 = min(a.r.B, tid * per), b1 = min(a.r.B, b0 + per);
  long long mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += kv_work(kv_job<K>(a, b, bits), a.c.heads);
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(FULL, scan, o);
    if (lane >= o) scan += t;
  }
  if (lane == 31) s_warp[warp] = scan;
  __syncthreads();
  long long before = scan - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  KvShare s;
  const long long most = quotient(total + least - 1, least);
  s.ctas = (int)(most < (long long)gridDim.x ? most : (long long)gridDim.x);
  const int g = blockIdx.x;
  if (g >= s.ctas) {
    s.begin = s.end = s.each = s.b_begin = 0;
    s.more = 0;
    s.b = a.r.B;
    return s;
  }
  s.each = quotient(total, s.ctas);
  s.more = (int)(total - s.each * s.ctas);
  s.begin = s.cut(g);
  s.end = s.cut(g + 1);
  if (before <= s.begin && s.begin < before + mine) {
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const long long w = kv_work(kv_job<K>(a, b, bits), a.c.heads);
      if (s.begin < before + w) {
        s_b = b;
        s_before = before;
        break;
      }
      before += w;
    }
  }
  __syncthreads();
  s.b = s_b;
  s.b_begin = s_before;
  return s;
}

// A share's segments: the units it holds or cuts, each with its range of tiles.
template <class K>
struct KvWalk {
  static constexpr int M = K::M, TILE = K::TILE;
  const KvAttendArgs &a;
  const KvShare &share;
  long long at, b_begin;
  int b;
  KvJob job;
  // of the current segment
  long long u_begin, u_end;  // its unit's place in all the work
  int h, r0, nrows;          // head, first row of the unit, rows
  int t0, t1;                // tiles of the list
  int p_first, p_last;       // positions of the first and the last row's token

  __device__ KvWalk(const KvAttendArgs &a_, const KvShare &s)
      : a(a_), share(s), at(s.begin), b_begin(s.b_begin), b(s.b) {
    job.units = -1;
  }

  __device__ __forceinline__ bool next(uint32_t *bits) {
    if (at >= share.end) return false;
    if (job.units < 0) job = kv_job<K>(a, b, bits);
#pragma unroll 1
    while (at >= b_begin + kv_work(job, a.c.heads)) {
      b_begin += kv_work(job, a.c.heads);
      ++b;
      job = kv_job<K>(a, b, bits);
    }
    const long long into = at - b_begin, head = kv_head_work(job), unit = (long long)job.cost * job.tiles;
    h = (int)quotient(into, head);
    const long long in_head = into - h * head;
    const int u = min((int)quotient(in_head, unit), job.units - 1);
    const int cost = u == job.units - 1 ? job.cost_last : job.cost;
    u_begin = at - in_head + u * unit;
    u_end = u_begin + (long long)cost * job.tiles;
    t0 = (int)quotient(at - u_begin, cost);
    at = min(u_end, share.end);
    t1 = (int)quotient(at - u_begin, cost);
    r0 = u * M;  // (a head's units follow one another: the later ones find its tiles in L2)
    nrows = min(M, job.ql * a.group - r0);
    p_first = job.n - job.ql + r0 / a.group;
    p_last = job.n - job.ql + (r0 + nrows - 1) / a.group;
    return true;
  }
  // whether the share holds the whole unit, or its begin
  __device__ bool whole() const { return u_begin >= share.begin && u_end <= share.end; }
  __device__ bool starts() const { return u_begin >= share.begin; }
  // whether some row of the unit sees some token of tile j of the list
  __device__ bool seen(int j) const {
    if (j >= t1) return false;
    const int x = job.tile(j) * TILE;
    return x <= p_last && (a.window == 0 || x + TILE - 1 > p_first - a.window || x < a.sinks);
  }
  // whether some row does not see some token of the tile at x
  __device__ bool edge(int x) const {
    return x + TILE - 1 > p_first || (a.window > 0 && x <= p_last - a.window && x + TILE > a.sinks);
  }
  // the page of the tile at x, its i-th; -1: none (reported where it should be there)
  __device__ int page(int x, int i, uint32_t *bits) const {
    const int block = (x >> a.c.page_bits) + i;
    if (block >= a.r.max_pages || block << a.c.page_bits >= job.n) return -1;
    const int pg = __ldg(a.r.table + (long long)b * a.r.max_pages + block);
    if (pg >= 0 && pg < a.c.num_pages) return pg;
    *bits |= SGD_KV_ERR_PAGE;
    return -1;
  }
  // token and query head of row r of the unit
  __device__ int token(int r) const { return job.q0 + (r0 + r) / a.group; }
  __device__ int q_head(int r) const { return h * a.group + (r0 + r) % a.group; }
};

}  // namespace sgd
