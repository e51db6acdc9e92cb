// Runs of rows that a sequence is cut into.  Row numbers go up to 2^31 - 256 and a run
// may be as long as the tensor, so nothing here forms the sum of a row and a run's
// length in 32 bits.  Plain C++ too: tests compile it for the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PRISM_HD __host__ __device__ __forceinline__
#else
#define PRISM_HD inline
#endif

namespace prism {

// Rows [r0, r1) of run `piece` of the sequence at rows [begin, begin + len), cut into runs of
// `unit`; false if the sequence has no such run.
PRISM_HD bool run_rows(int begin, int len, int64_t piece, int unit, int &r0, int &r1) {
  if (piece < 0 || piece * unit >= len) return false;
  const int at = (int)(piece * unit);
  r0 = begin + at;
  r1 = r0 + (unit < len - at ? unit : len - at);
  return true;
}

// Runs of a sequence of `len` rows.
PRISM_HD int run_count(int len, int unit) { return len / unit + (len % unit != 0); }

}  // namespace prism
