// kv_attend.cuh -- the attention's references, and where parts of units lie.
#pragma once

#include <cuda.h>

#include "async_copy.cuh"
#include "kv_internal.h"
#include "kv_sched.cuh"

namespace sgd {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int MAX_CTAS = 152 * 3;  // what the workspace is laid out for

// Token j adds 2^z_j, z its scaled product in units of log 2, to l and
// 2^(z_j + log2 V_j) q_j to o, V_j the scale of its block of values and q_j what
// is stored.  Both are kept relative to one reference per row, the running
// maximum of z + log2 V (not of z: f16 probabilities have 11 bits down to 2^-14,
// and below that an absolute error, which has to be small against the largest
// share in o; a block of much larger values than the one that the softmax
// favours would show it otherwise).  Scales reach from 2^-48 to 2^48, so l stays
// far within 32 bits.  The reference moves, and o and l are scaled, only once
// the maximum has grown by 2^LAZY; probabilities are taken 2^LIFT times as large
// (the quotient is the same), so that they use f16's range up to its end: 2^15.99
// is 65082 of 65504.  (A larger LAZY saves little: at 4, a row that has seen a
// few tiles of common logits meets such a maximum once in hundreds of tiles.)
constexpr float LAZY = 4.f;
constexpr float LIFT = 11.99f;

// log2 of a block's scale (a power of two when sgd_kv_write made it), and its inverse
__device__ __forceinline__ float log2_scale(float s) { return __log2f(s); }
__device__ __forceinline__ float inverse_scale(float s) { return __fdividef(1.f, s); }

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Where the parts of split units lie in the workspace, after the counters (one
// per CTA): [M][D] sums, [M] maxima, [M] sums of probabilities.
template <int M, int D>
__device__ __forceinline__ float *part_of(const KvAttendArgs &a, int slot) {
  return reinterpret_cast<float *>(a.work + MAX_CTAS * 8) + (long long)slot * (M * (D + 2));
}

}  // namespace sgd
