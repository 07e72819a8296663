// Packed sequences seen from fixed windows of rows: helpers of the kernels that take
// seq_offsets.
//
// Rows are cut into windows of R rows at multiples of R.  Window w and sequence s overlap
// in one run of rows, and w + s numbers these pairs without a gap in order of their rows
// and without a collision (going on along the rows, w or s grows), so pair (w, s) owns slot
// w + s of a table of ceil(T / R) + S - 1 slots and nothing has to be counted first.
#pragma once

#include "common.cuh"

namespace moe {

// Number of i in [0, n) with key(i) <= x, for keys that do not decrease; run by every
// thread of the block, which probes blockDim.x places at a time (one round up to
// blockDim.x keys).  Any keys give a result in [0, n].
template <class Key>
__device__ __forceinline__ int block_count_le(int n, long long x, Key key) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = (hi - lo + (int)blockDim.x - 1) / (int)blockDim.x;
    const long long i = lo + ((long long)threadIdx.x + 1) * step - 1;
    const bool le = i < hi && key((int)i) <= x;
    lo += __syncthreads_count(le) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Offsets that decrease or leave [0, T] are reported; every block looks at a share.
__device__ __forceinline__ void check_offsets(const int32_t* off, int S, int64_t T, int* err) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < S;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int a = off[i], b = off[i + 1];
    if (a < 0 || b < a || b > T) report_error(err, MOE_ERR_DEVICE_INDEX);
  }
}

}  // namespace moe
