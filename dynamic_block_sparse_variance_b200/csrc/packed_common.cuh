// Packed sequences: `seqs` sequences stored one behind the other in the rows
// of one tensor, sequence b at rows [off[b], off[b+1]) (no offsets: the rows
// are split evenly).  The offsets live on the device, so no launch waits for
// the host; grids are sized by an upper bound of the work instead.
//
// Work slots.  Cutting sequence b (rows s..e, counted in `scale` units per row)
// into pieces of `unit` takes ceil((e - s) / unit) slots.  Giving it the slots
// from f(b) = floor(s / unit) + b on leaves room for them all, because
// floor(e / unit) - floor(s / unit) + 1 >= ceil((e - s) / unit), and f grows with b,
// so a CTA finds its sequence by searching f for its slot: no prefix sum over
// the lengths, no work list, at most one idle slot per sequence.
#pragma once

#include "common.cuh"

namespace prism {

// What the kernel before this one on the stream wrote is there from here on (see
// launch_behind); every thread calls it before its first access to global memory.  That
// kernel may still write while this one is resident, so no load here is a non-coherent
// one (__ldg, __restrict__), which promises that nobody writes during the kernel's life.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct Offsets {
  const int32_t *off;   // [seqs + 1], or nullptr: `even` rows each
  int seqs;
  int even;
  int rows;             // rows of the tensor
  __device__ __forceinline__ int64_t at(int b) const { return off ? (int64_t)off[b] : (int64_t)b * even; }
};

// Rows [begin, begin + len) of sequence b; false (and a latched PRISM_EBOUNDS)
// if the offsets leave the tensor or run backwards.
__device__ __forceinline__ bool sequence_rows(const Offsets &o, int b, int &begin, int &len) {
  const int64_t s = o.at(b), e = o.at(b + 1);
  if (s < 0 || e < s || e > o.rows) {
    set_status(PRISM_EBOUNDS);
    begin = len = 0;
    return false;
  }
  begin = (int)s;
  len = (int)(e - s);
  return true;
}

// Offsets that run backwards can hide a sequence from every slot's search, so
// slot b also looks at sequence b itself (there are at least `seqs` slots).
__device__ __forceinline__ void check_sequence(const Offsets &o, int64_t slot) {
  int begin, len;
  if (threadIdx.x == 0 && slot < o.seqs) sequence_rows(o, (int)slot, begin, len);
}

// The sequence of work slot `slot` and the piece of it (0, 1, ...) that the
// slot stands for.  Called by whole warps; 32 candidates per step, so up to
// 1024 sequences take two dependent loads.
__device__ __forceinline__ int find_sequence(const Offsets &o, int64_t slot, int scale, int unit, int64_t &piece) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = o.seqs;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool below = b < lo + n && o.at(b) * scale / unit + b <= slot;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int hit = m ? 31 - __clz(m) : 0;
    const int nlo = lo + hit * step;
    n = min(step, lo + n - nlo);
    lo = nlo;
  }
  piece = slot - (o.at(lo) * scale / unit + lo);
  return lo;
}

inline int64_t slot_bound(int64_t rows, int seqs, int scale, int unit) { return rows * scale / unit + seqs; }

}  // namespace prism
