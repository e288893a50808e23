// kv_assign.cu -- pages of a step's tokens: which pages each row gives back or
// gets, and for the packed new tokens their rows, positions and slots.
//
// Row b keeps keep[b] tokens and gets new[b]: need = ceil((keep + new) / P) pages.
// With held pages so far, the held - need beyond them go to the end of the free
// list, row by row; then want = need - held come from its end, row by row.  All of
// it is prefix sums over the rows (new tokens, pages back, pages wanted), so the
// result does not depend on the order in which threads run.
//
// One cluster: every CTA computes all the sums (rows are few: 16 bytes each) and
// keeps the rows' places in shared memory, then takes its share of the rows'
// pages and of the tokens.  Two cluster barriers: nothing is written before all
// CTAs have read the state, nothing taken before all given pages are on the list.
#include <cooperative_groups.h>

#include "kv_internal.h"
#include "sgd_internal.h"

namespace cg = cooperative_groups;

namespace sgd {
namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;

struct Row {
  int keep, held, need;  // tokens that stay; pages before and after
  int fresh;             // new tokens
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
  long long w = s[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(FULL, w, o);
    if (lane >= o) w += t;
  }
  *total = __shfl_sync(FULL, w, 31);
  const long long before = __shfl_sync(FULL, w, max(warp - 1, 0));
  return scan - x + (warp ? before : 0);
}

__global__ void __launch_bounds__(THREADS, 1) assign_kernel(KvAssignArgs a) {
  extern __shared__ int s_rows[];
  int *s_start = s_rows;               // [B + 1] first packed token
  int *s_keep = s_start + a.B + 1;     // [B]
  int *s_held = s_keep + a.B;          // [B] pages before
  int *s_need = s_held + a.B;          // [B] pages after (-1 - held: a row passed over)
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
  for (int b = b0; b < b1; ++b) mine += row_of(a, b).fresh;
  long long at = block_scan(mine, s_sum, &total);
  const bool packed = total <= a.N;
  // pages back, pages wanted
  long long back = 0, want = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    Row r = row_of(a, b);
    if (!r.good) bits |= SGD_KV_ERR_LENGTH;
    at += r.fresh;
    if (!packed && r.fresh > 0 && at > a.N) {
      r.fresh = 0;
      bits |= SGD_KV_ERR_ROOM;
    }
    r.need = r.good ? pages_of(a, r.keep + r.fresh) : r.held;
    s_keep[b] = r.keep;
    s_held[b] = r.held;
    s_need[b] = r.good ? r.need : -1;
    s_start[b] = r.fresh;
    if (r.need < r.held) back += r.held - r.need;
    else want += r.need - r.held;
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
      s_place[b] = (int)back_at;
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
  for (int b = rank; b < a.B; b += warps)
    for (int j = s_held[b] + lane; j < s_need[b]; j += 32) {
      const int page = taken_page(b, j);
      if (page < 0 || page >= a.num_pages) bits |= SGD_KV_ERR_PAGE;
      a.table[(long long)b * a.max_pages + j] = page;
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

constexpr size_t smem_bytes(int B) { return ((size_t)B * 5 + 1) * sizeof(int); }

}  // namespace

cudaError_t kv_assign_set_limits() {
  return cudaFuncSetAttribute(assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem_bytes(SGD_KV_ASSIGN_MAX_ROWS));
}

cudaError_t launch_kv_assign(const KvAssignArgs &a, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {1, 1, 1};
  c.gridDim = {1, 1, 1};
  c.blockDim = {THREADS, 1, 1};
  c.dynamicSmemBytes = smem_bytes(a.B);
  c.stream = st;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, assign_kernel, a);
}

}  // namespace sgd
