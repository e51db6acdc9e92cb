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

// Rows of a run: a share of the rows for each of `ctas` CTAs.  A sequence's last run may be
// short, so the share is that of one CTA less per sequence, but never of fewer than three
// quarters: with many sequences the longest would be left to a few CTAs, or to one.
// (61440 x 1536, one sequence with half of the rows: in 150 sequences the forward took
// 6680 us with the share falling to one CTA's, 147 now; in 1000 the backward 36.9 ms,
// 0.89 now; one sequence 143 and 307.)
PRISM_HD int64_t run_length(int64_t rows, int seqs, int ctas, int64_t least) {
  const int64_t wave = ctas - seqs > ctas * 3 / 4 ? ctas - seqs : ctas * 3 / 4;
  const int64_t unit = (rows + wave - 1) / wave;
  return unit > least ? unit : least;
}

// Runs of a sequence of `len` rows.
PRISM_HD int run_count(int len, int unit) { return len / unit + (len % unit != 0); }

}  // namespace prism
