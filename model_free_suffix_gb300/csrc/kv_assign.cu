// kv_assign.cu -- pages of a step's tokens: which pages each row gives back or
// gets, and for the packed new tokens their rows, positions and slots.
//
// Row b keeps keep[b] tokens and gets new[b]: need = ceil((keep + new) / P) pages.
// With held pages so far, the held - need beyond them go to the end of the free
// list, row by row; then want = need - held come from its end, row by row.  All of
// it is prefix sums over the rows (new tokens, pages back, pages wanted), so the
// result does not depend on the order in which threads run.
//
// One cluster of eight CTAs, every one of which computes all the sums (rows are few: 12
// bytes each), keeps the rows' places in shared memory and takes its share of the rows'
// pages and of the tokens.  Two cluster barriers: nothing is written before all
// CTAs have read the state, nothing taken before all given pages are on the list.
// Many tokens (prompts) get a second kernel, of as many CTAs as they fill.
//
// Nothing here is bound by bytes but the places of prompts' tokens (12 bytes each): a call
// of a serving step is a chain of launch, one read of the rows, four prefix sums, two
// cluster barriers and the reads of tables and list.  Measured, a call: 4 rows 5 us, 256
// rows of 1..17 tokens 8 to 9, 1024 rows of which 256 give up or get 8192 tokens'
// pages (half of the calls place a million tokens) 26.  One CTA of 1024 threads took 28 and 616
// for the latter two; clusters of four CTAs 9 and 34, of 256 threads a CTA 9 and 34, of 1024
// 10 and 24.
#include <cooperative_groups.h>

#include "kv_internal.h"
#include "sgd_internal.h"

namespace cg = cooperative_groups;

namespace sgd {
namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int CTAS = 8;            // of the cluster
// Tokens that the cluster places itself: at some 20000 a step a second kernel took 8.8 us
// a call against 7.8, at 96000 its own 16 against 9.
constexpr int OWN_TOKENS = 32768;

struct Row {
  int keep, held, fresh;  // tokens that stay, pages so far, new tokens
  bool good;
};

__device__ __forceinline__ Row row_of(const KvAssignArgs &a, int b) {
  Row r;
  r.keep = a.keep[b];
  r.fresh = a.fresh[b];
  r.held = a.held[b];
  const long long room = (long long)a.max_pages << a.page_bits;
  r.good = r.held >= 0 && r.held <= a.max_pages && r.keep >= 0 && r.fresh >= 0 &&
           r.keep <= ((long long)r.held << a.page_bits) && (long long)r.keep + r.fresh <= room;
  if (!r.good) r.fresh = 0;
  return r;
}
__device__ __forceinline__ int pages_of(const KvAssignArgs &a, int tokens) {
  return (int)(((long long)tokens + (1 << a.page_bits) - 1) >> a.page_bits);
}

// Exclusive prefix sum over the block's threads, and the total.
__device__ __forceinline__ long long block_scan(long long x, long long *s, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long scan = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(FULL, scan, o);
    if (lane >= o) scan += t;
  }
  __syncthreads();  // (the sums of the scan before have been read)
  if (lane == 31) s[warp] = scan;
  __syncthreads();
  long long w = lane < WARPS ? s[lane] : 0;
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const long long t = __shfl_up_sync(FULL, w, o);
    if (lane >= o) w += t;
  }
  *total = __shfl_sync(FULL, w, WARPS - 1);
  const long long before = __shfl_sync(FULL, w, max(warp - 1, 0));
  return scan - x + (warp ? before : 0);
}

__global__ void __launch_bounds__(THREADS, 1) assign_kernel(KvAssignArgs a) {
  extern __shared__ int s_rows[];
  int *s_start = s_rows;               // [B + 1] first packed token
  int *s_keep = s_start + a.B + 1;     // [B]
  int *s_held = s_keep + a.B;          // [B] pages before
  int *s_need = s_held + a.B;          // [B] pages after (-1: a row passed over)
  int *s_place = s_need + a.B;         // [B] pages before its own: of those given back, or of those taken
  __shared__ long long s_sum[32];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  uint32_t bits = 0;
  int count = *a.free_count;
  if (count < 0 || count > a.num_pages) {
    bits |= SGD_KV_ERR_PAGE;
    count = min(max(count, 0), a.num_pages);
  }
  // what fits the packed tokens
  long long total, mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Row r = row_of(a, b);
    s_keep[b] = r.keep;
    s_held[b] = r.held;
    s_need[b] = r.good ? 0 : -1;
    s_start[b] = r.fresh;
    mine += r.fresh;
    if (!r.good) bits |= SGD_KV_ERR_LENGTH;
  }
  long long at = block_scan(mine, s_sum, &total);
  const bool packed = total <= a.N;
  // pages back, pages wanted
  long long back = 0, want = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    if (s_need[b] < 0) continue;
    const int fresh = s_start[b];
    at += fresh;
    if (!packed && fresh > 0 && at > a.N) {
      s_start[b] = 0;
      bits |= SGD_KV_ERR_ROOM;
    }
    const int need = pages_of(a, s_keep[b] + s_start[b]), held = s_held[b];
    s_need[b] = need;
    if (need < held) back += held - need;
    else want += need - held;
  }
  long long back_total, want_total;
  long long back_at = block_scan(back, s_sum, &back_total);
  long long want_at = block_scan(want, s_sum, &want_total);
  const long long have = count + back_total;
  // the tokens of the rows that get their pages
  long long taken = 0;
  mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    if (s_need[b] < 0) continue;
    const int more = s_need[b] - s_held[b];
    if (more > 0) {
      s_place[b] = (int)want_at;
      want_at += more;
      if (want_at > have) {
        s_start[b] = 0;
        s_need[b] = s_held[b];
        bits |= SGD_KV_ERR_ROOM;
      } else {
        taken += more;
      }
    } else {
      s_place[b] = (int)min(back_at, (long long)a.num_pages);  // (more are only where held is wrong, and go nowhere)
      back_at -= more;
    }
    mine += s_start[b];
  }
  long long new_total, taken_total;
  at = block_scan(mine, s_sum, &new_total);
  block_scan(taken, s_sum, &taken_total);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int fresh = s_start[b];
    s_start[b] = (int)at;
    at += fresh;
  }
  if (tid == 0) s_start[a.B] = (int)new_total;
  cluster.sync();  // (all have read the state)

  const int rank = cta * WARPS + warp, warps = ctas * WARPS;
  for (int b = cta * THREADS + tid; b <= a.B; b += ctas * THREADS) {
    a.q_start[b] = s_start[b];
    if (b == a.B) break;
    a.seq_lens[b] = s_need[b] < 0 ? 0 : s_keep[b] + s_start[b + 1] - s_start[b];
    if (s_need[b] >= 0) a.held[b] = s_need[b];
  }
  const long long left = have - taken_total;
  if (cta == 0 && tid == 0) *a.free_count = (int)min(left, (long long)a.num_pages);
  if (back_total > 0) {
#pragma unroll 1
    for (int b = rank; b < a.B; b += warps) {
      if (s_need[b] < 0) continue;
      int *row = a.table + (long long)b * a.max_pages;
      for (int j = s_need[b] + lane; j < s_held[b]; j += 32) {
        const int page = row[j];
        const long long to = (long long)count + s_place[b] + j - s_need[b];
        row[j] = -1;
        if (page < 0 || page >= a.num_pages) bits |= SGD_KV_ERR_PAGE;
        if (to < a.num_pages) a.free[to] = page;
        else bits |= SGD_KV_ERR_PAGE;
      }
    }
    cluster.sync();  // (all given pages are on the list)
  }
  // page j of row b: one that it held, or one off the end of the list
  auto taken_page = [&](int b, int j) {
    const long long from = have - 1 - s_place[b] - (j - s_held[b]);
    return from < a.num_pages ? a.free[from] : -1;
  };
#pragma unroll 1
  for (int b = rank; b < a.B; b += warps) {
    if (s_need[b] < 0) continue;  // (what it holds may be below 0, and no place of the table)
    for (int j = s_held[b] + lane; j < s_need[b]; j += 32) {
      const int page = taken_page(b, j);
      if (page < 0 || page >= a.num_pages) bits |= SGD_KV_ERR_PAGE;
      a.table[(long long)b * a.max_pages + j] = page;
    }
  }
  if (a.N > OWN_TOKENS) {
    if (bits) atomicOr(a.err, bits);
    return;
  }
  // the packed tokens
#pragma unroll 1
  for (int i = cta * THREADS + tid; i < a.N; i += ctas * THREADS) {
    int row = -1, position = 0, slot = -1;
    if (i < s_start[a.B]) {
      int lo = 0, hi = a.B;  // the last row that starts at or before i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= i) lo = mid;
        else hi = mid;
      }
      row = lo;
      position = s_keep[row] + i - s_start[row];
      if (a.slots) {
        const int j = position >> a.page_bits;
        const int page = j < s_held[row] ? a.table[(long long)row * a.max_pages + j] : taken_page(row, j);
        if (page < 0 || page >= a.num_pages) bits |= SGD_KV_ERR_PAGE;
        else slot = (page << a.page_bits) + (position & ((1 << a.page_bits) - 1));
      }
    }
    if (a.rows) a.rows[i] = row;
    if (a.positions) a.positions[i] = position;
    if (a.slots) a.slots[i] = slot;
  }
  if (bits) atomicOr(a.err, bits);
}

// The places of many packed tokens, after assign_kernel: a thread's four in a row, the
// row found for the first of them.
constexpr int PLACE_THREADS = 256, PLACE_TOKENS = 4 * PLACE_THREADS;
__global__ void __launch_bounds__(PLACE_THREADS) place_kernel(KvAssignArgs a) {
  __shared__ int s_row;  // that of the block's first token
  const int first = blockIdx.x * PLACE_TOKENS, total = __ldg(a.q_start + a.B);
  const int tid = threadIdx.x;
  // (a warp's lanes look at 32 starts at a time)
  if (tid < 32) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + tid * step;
      const uint32_t below = __ballot_sync(FULL, at < hi && __ldg(a.q_start + at) <= first);
      const int last = 31 - __clz(below | 1);
      const int from = lo + last * step;
      hi = min(hi, from + step);
      lo = from;
    }
    if (tid == 0) s_row = lo;
  }
  __syncthreads();
  int i = first + tid * 4, row = s_row;
  if (i >= a.N) return;
  if (i < total) {
    int hi = a.B;
    // (far from the block's first row only where rows are short: doubling steps, then halving)
    int step = 1;
    while (row + step < hi && __ldg(a.q_start + row + step) <= i) {
      row += step;
      step <<= 1;
    }
    hi = min(hi, row + step);
    while (hi - row > 1) {
      const int mid = (row + hi) >> 1;
      if (__ldg(a.q_start + mid) <= i) row = mid;
      else hi = mid;
    }
  }
  int rows[4], positions[4], slots[4];
  uint32_t bits = 0;
  int start = 0, end = 0, keep = 0, at = -1, page = -1;
  if (i < total) {
    start = __ldg(a.q_start + row);
    end = __ldg(a.q_start + row + 1);
    keep = a.seq_lens[row] - (end - start);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e, ++i) {
    rows[e] = slots[e] = -1;
    positions[e] = 0;
    if (i >= total) continue;
    while (i >= end) {
      start = end;
      end = __ldg(a.q_start + ++row + 1);
      keep = a.seq_lens[row] - (end - start);
      at = -1;
    }
    rows[e] = row;
    positions[e] = keep + i - start;
    if (at != positions[e] >> a.page_bits) {
      at = positions[e] >> a.page_bits;
      page = __ldg(a.table + (long long)row * a.max_pages + at);
    }
    if (page < 0 || page >= a.num_pages) bits |= SGD_KV_ERR_PAGE;
    else slots[e] = (page << a.page_bits) + (positions[e] & ((1 << a.page_bits) - 1));
  }
  i -= 4;
  auto put = [&](int32_t *to, const int (&x)[4]) {
    if (!to) return;
    if (i + 4 <= a.N && ((uintptr_t)to & 15) == 0) {
      *reinterpret_cast<int4 *>(to + i) = make_int4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < a.N) to[i + e] = x[e];
    }
  };
  put(a.rows, rows);
  put(a.positions, positions);
  if (a.slots) {
    put(a.slots, slots);
    if (bits) atomicOr(a.err, bits);
  }
}

constexpr size_t smem_bytes(int B) { return ((size_t)B * 5 + 1) * sizeof(int); }

}  // namespace

cudaError_t kv_assign_set_limits() {
  return cudaFuncSetAttribute(assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem_bytes(SGD_KV_ASSIGN_MAX_ROWS));
}

cudaError_t launch_kv_assign(const KvAssignArgs &a, cudaStream_t st, int *launches) {
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {CTAS, 1, 1};
  c.gridDim = {CTAS, 1, 1};
  c.blockDim = {THREADS, 1, 1};
  c.dynamicSmemBytes = smem_bytes(a.B);
  c.stream = st;
  c.attrs = at;
  c.numAttrs = 1;
  *launches = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, assign_kernel, a);
  if (e != cudaSuccess || a.N <= OWN_TOKENS || !(a.positions || a.slots || a.rows)) return e;
  *launches = 2;
  place_kernel<<<(unsigned)(((long long)a.N + PLACE_TOKENS - 1) / PLACE_TOKENS), PLACE_THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sgd
