// Dense attention over packed sequences: what its kernels share.  The query
// rows of a key/value head are flattened to (token, head of the group): row r
// of a sequence is token r / group, head r % group.  Every kernel tiles these
// flattened rows, so the heads of a group share each key and value that is
// read, whatever the group's size, and a causal tile's rows are neighbours.
#pragma once

#include "attn_common.cuh"
#include "tc_common.cuh"
#include "packed_common.cuh"

namespace prism {

struct PackedArgs {
  Offsets qs, ks;
  const int32_t *k_used;
  int heads, kv_heads, group, causal;
  int debug_stall;                  // test knob (PRISM_OPT_DEBUG_STALL): the first P or dS is never signalled
  float scale, scale_log2;
  const __nv_bfloat16 *q, *k, *v, *dout;
  __nv_bfloat16 *o, *o_res, *dq, *dk, *dv;
  float *lse;
  const float *lse2, *delta;        // backward: LSE log2e and rowsum(dO o O), [kv_heads][q_rows][group]
  int64_t sq[2], sk[2], sv[2], so[2], sdo[2], sdq[2], sdk[2], sdv[2];
};

struct PackedSeq {
  int q0, lq, k0, lk, room;   // lk keys in use of `room` rows
  __device__ __forceinline__ bool load(const PackedArgs &a, int b) {
    if (!sequence_rows(a.qs, b, q0, lq) || !sequence_rows(a.ks, b, k0, room)) return false;
    lk = room;
    if (a.k_used) {
      lk = a.k_used[b];
      if (lk < 0 || lk > room) {
        set_status(PRISM_EBOUNDS);
        lk = 0;
      }
    }
    return true;
  }
  // What a kernel's slot does first: offsets and lengths checked (see check_sequence).
  __device__ __forceinline__ static void check(const PackedArgs &a, int64_t slot) {
    PackedSeq s;
    if (threadIdx.x == 0 && slot < a.qs.seqs) s.load(a, (int)slot);
  }
  // Keys 0 .. visible - 1 are what token `tok` sees.
  __device__ __forceinline__ int visible(const PackedArgs &a, int tok) const {
    return a.causal ? max(0, min(lk, tok + lk - lq + 1)) : lk;
  }
};

// Per query row and head (8 or 16 lanes, 8 columns each; two rows at a time, so that
// six 16-byte loads are in flight): D = rowsum(dO o (O + residual)) and LSE log2e; a
// row that sees nothing (LSE -inf) gets +inf, so that its probabilities 2^(x - inf) are zero.
// Written in flattened order.
template <int D>
__global__ void __launch_bounds__(256) packed_stats_kernel(const PackedArgs a, const __nv_bfloat16 *o, float *delta,
                                                           float *lse2) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes;      // (row, head) pairs of a CTA and pass
  after_previous();
  const int sub = threadIdx.x % kLanes;
  const int64_t total = (int64_t)a.qs.rows * a.heads;
  uint4 uo[2], ug[2], ur[2];
  int64_t row[2];
  int h[2];
  float L[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int64_t i = (int64_t)blockIdx.x * (2 * kRows) + p * kRows + threadIdx.x / kLanes;   // row * heads + head
    row[p] = i / a.heads;
    h[p] = (int)(i - row[p] * a.heads);
    uo[p] = ug[p] = ur[p] = make_uint4(0u, 0u, 0u, 0u);
    if (i < total) {
      uo[p] = *reinterpret_cast<const uint4 *>(o + row[p] * a.so[0] + h[p] * a.so[1] + sub * 8);
      ug[p] = *reinterpret_cast<const uint4 *>(a.dout + row[p] * a.sdo[0] + h[p] * a.sdo[1] + sub * 8);
      if (a.o_res) ur[p] = *reinterpret_cast<const uint4 *>(a.o_res + i * D + sub * 8);
      L[p] = a.lse[(int64_t)h[p] * a.qs.rows + row[p]];
    } else {
      row[p] = -1;
    }
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t wo[4] = {uo[p].x, uo[p].y, uo[p].z, uo[p].w}, wg[4] = {ug[p].x, ug[p].y, ug[p].z, ug[p].w},
                   wr[4] = {ur[p].x, ur[p].y, ur[p].z, ur[p].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(bf16_lo(wo[e]) + bf16_lo(wr[e]), bf16_lo(wg[e]), s);
      s = fmaf(bf16_hi(wo[e]) + bf16_hi(wr[e]), bf16_hi(wg[e]), s);
    }
#pragma unroll
    for (int w = kLanes / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    if (row[p] >= 0 && sub == 0) {
      const int kvh = h[p] / a.group;
      const int64_t at = ((int64_t)kvh * a.qs.rows + row[p]) * a.group + h[p] - kvh * a.group;
      delta[at] = s;
      lse2[at] = L[p] == -INFINITY ? INFINITY : L[p] * kLog2e;
    }
  }
}

}  // namespace prism
