// Dense attention over packed sequences, one warp per query (or key) row on
// the CUDA cores: the simplest form of the operator.
#pragma once

#include "packed_attn.cuh"

namespace prism {

template <int D>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float (&f)[D / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) f[e] = __bfloat162float(p[lane * (D / 32) + e]);
}
template <int D>
__device__ __forceinline__ float dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) s = fmaf(a[e], b[e], s);
  return warp_sum(s);
}

template <int D>
__global__ void __launch_bounds__(256) packed_dq_simple_kernel(const PackedArgs a) {
  const int lane = threadIdx.x & 31;
  const int kvh = blockIdx.y;
  int64_t piece;
  PackedSeq::check(a, blockIdx.x);
  const int b = find_sequence(a.qs, blockIdx.x, a.group, 8, piece);
  PackedSeq s;
  if (!s.load(a, b)) return;
  const int64_t fr = piece * 8 + (threadIdx.x >> 5);
  if (piece < 0 || fr >= (int64_t)s.lq * a.group) return;
  const int tok = (int)(fr / a.group), head = kvh * a.group + (int)(fr % a.group);
  float q[D / 32], k[D / 32], v[D / 32], g[D / 32], dq[D / 32];
  load_row<D>(a.q + (int64_t)(s.q0 + tok) * a.sq[0] + head * a.sq[1], q);
  load_row<D>(a.dout + (int64_t)(s.q0 + tok) * a.sdo[0] + head * a.sdo[1], g);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) dq[e] = 0.f;
  const int64_t st = (int64_t)head * a.qs.rows + s.q0 + tok;
  const float lse2 = a.lse2[st], delta = a.delta[st];
  const int n = s.visible(a, tok);
  for (int j = 0; j < n; ++j) {
    load_row<D>(a.k + (int64_t)(s.k0 + j) * a.sk[0] + kvh * a.sk[1], k);
    load_row<D>(a.v + (int64_t)(s.k0 + j) * a.sv[0] + kvh * a.sv[1], v);
    const float p = exp2f(dot<D>(q, k) * a.scale_log2 - lse2);
    const float ds = p * (dot<D>(g, v) - delta) * a.scale;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) dq[e] = fmaf(ds, k[e], dq[e]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    a.dq[(int64_t)(s.q0 + tok) * a.sdq[0] + head * a.sdq[1] + lane * (D / 32) + e] = __float2bfloat16_rn(dq[e]);
}

template <int D>
__global__ void __launch_bounds__(256) packed_dkdv_simple_kernel(const PackedArgs a) {
  const int lane = threadIdx.x & 31;
  const int kvh = blockIdx.y;
  int64_t piece;
  PackedSeq::check(a, blockIdx.x);
  const int b = find_sequence(a.ks, blockIdx.x, 1, 8, piece);
  PackedSeq s;
  if (!s.load(a, b)) return;
  const int64_t j = piece * 8 + (threadIdx.x >> 5);
  if (piece < 0 || j >= s.room) return;
  float q[D / 32], k[D / 32], v[D / 32], g[D / 32], dk[D / 32], dv[D / 32];
  load_row<D>(a.k + (s.k0 + j) * a.sk[0] + kvh * a.sk[1], k);
  load_row<D>(a.v + (s.k0 + j) * a.sv[0] + kvh * a.sv[1], v);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) dk[e] = dv[e] = 0.f;
  for (int tok = 0; tok < s.lq; ++tok) {
    if (j >= s.visible(a, tok)) continue;
    for (int h = kvh * a.group; h < (kvh + 1) * a.group; ++h) {
      load_row<D>(a.q + (int64_t)(s.q0 + tok) * a.sq[0] + h * a.sq[1], q);
      load_row<D>(a.dout + (int64_t)(s.q0 + tok) * a.sdo[0] + h * a.sdo[1], g);
      const int64_t st = (int64_t)h * a.qs.rows + s.q0 + tok;
      const float p = exp2f(dot<D>(q, k) * a.scale_log2 - a.lse2[st]);
      const float ds = p * (dot<D>(g, v) - a.delta[st]) * a.scale;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) dk[e] = fmaf(ds, q[e], dk[e]), dv[e] = fmaf(p, g[e], dv[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    a.dk[(s.k0 + j) * a.sdk[0] + kvh * a.sdk[1] + lane * (D / 32) + e] = __float2bfloat16_rn(dk[e]);
    a.dv[(s.k0 + j) * a.sdv[0] + kvh * a.sdv[1] + lane * (D / 32) + e] = __float2bfloat16_rn(dv[e]);
  }
}

}  // namespace prism
