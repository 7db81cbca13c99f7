// A sequence's rows of a ragged batch, from two neighbouring starts.  Plain C++,
// so that it also compiles for the host.
#pragma once

#ifdef __CUDACC__
#define VQKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define VQKV_HOST_DEVICE inline
#endif

namespace vqkv {

struct RowRange {
  int first, n;   // n == 0: first is 0, a row that may be read whatever the starts hold
};

// Of rows [0, n_rows): those from start up to end, at most max_queries; none where
// the starts do not ascend within [0, n_rows].  *fine: they do, and the rows are all there.
VQKV_HOST_DEVICE RowRange rows_of_starts(int start, int end, int n_rows, int max_queries, bool* fine) {
  // (differences in 64 bits: starts of any bits must not overflow on the way to the comparisons)
  const long long lo = start, hi = end, n = hi - lo;
  const bool ascend = lo >= 0 && n >= 0 && hi <= n_rows;
  *fine = ascend && n <= max_queries;
  if (!ascend || n == 0) return {0, 0};
  return {start, n < max_queries ? (int)n : max_queries};
}

}  // namespace vqkv
