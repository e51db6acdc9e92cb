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

// Per query row and head (half a warp for head_dim 64, a warp for 128): D =
// rowsum(dO o (O + residual)) and LSE log2e; a row that sees nothing gets +inf,
// so that its probabilities 2^(x - inf) are zero.  Written in flattened order.
template <int D>
__global__ void __launch_bounds__(256) packed_stats_kernel(const PackedArgs a, const __nv_bfloat16 *__restrict__ o,
                                                           float *__restrict__ delta, float *__restrict__ lse2) {
  constexpr int kLanes = D / 4;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kLanes;   // row * heads + head
  const int sub = threadIdx.x % kLanes;
  float s = 0.f;
  const bool in = i < (int64_t)a.qs.rows * a.heads;
  const int64_t row = i / a.heads;
  const int h = (int)(i - row * a.heads);
  if (in) {
    const uint2 uo = *reinterpret_cast<const uint2 *>(o + row * a.so[0] + h * a.so[1] + sub * 4);
    const uint2 ug = *reinterpret_cast<const uint2 *>(a.dout + row * a.sdo[0] + h * a.sdo[1] + sub * 4);
    float o0 = bf16_lo(uo.x), o1 = bf16_hi(uo.x), o2 = bf16_lo(uo.y), o3 = bf16_hi(uo.y);
    if (a.o_res) {
      const uint2 ur = *reinterpret_cast<const uint2 *>(a.o_res + i * D + sub * 4);
      o0 += bf16_lo(ur.x); o1 += bf16_hi(ur.x); o2 += bf16_lo(ur.y); o3 += bf16_hi(ur.y);
    }
    s = (o0 * bf16_lo(ug.x) + o1 * bf16_hi(ug.x)) + (o2 * bf16_lo(ug.y) + o3 * bf16_hi(ug.y));
  }
#pragma unroll
  for (int w = kLanes / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
  if (in && sub == 0) {
    const float L = a.lse[(int64_t)h * a.qs.rows + row];
    const int kvh = h / a.group;
    const int64_t at = ((int64_t)kvh * a.qs.rows + row) * a.group + h - kvh * a.group;
    delta[at] = s;
    lse2[at] = isfinite(L) ? L * kLog2e : INFINITY;
  }
}

}  // namespace prism
