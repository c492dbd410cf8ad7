// How an expert's rows are shared out over its tiles.  Plain arithmetic, for the host too.
#pragma once
#ifdef __CUDACC__
#define GMMFR_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define GMMFR_HOST_DEVICE inline
#endif

namespace gmmfr {

// Rows `first` .. first + count - 1 are tile i of an expert's `rows` (1 and more), whose n tiles are each ceil(rows / n) rows rounded
// up to 32.  n = ceil(rows / bn) with bn = 256, or n = 1: then (n - 1) of that width are below `rows`, and no tile is empty.
// Every step stays below 2^31 for rows up to 2^31 - 1024.
GMMFR_HOST_DEVICE void row_tile(int rows, int n, int i, int& first, int& count) {
  const int w = ((rows - 1) / n + 32) / 32 * 32;
  first = i * w;
  count = w < rows - first ? w : rows - first;
}

}  // namespace gmmfr
