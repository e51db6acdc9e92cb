// Dense attention forward for few query rows per sequence (a token over a cache):
// 16 flattened rows (tokens x heads of the group) of one kv head per CTA, on the
// warp-level m16n8k16 MMA.  Bound by reading K and V once: one flop a byte and row,
// 16 with all rows in use, so the tensor rate does not matter, the bytes in flight do.
//
// The keys are split over blockIdx.z and, in a CTA, over its four warps, which
// take 32 keys in turn and never wait for one another: each fills a ring of its
// own with cp.async (3 stages of 16 KB, 192 KB of loads in flight per SM for
// head_dim 128), keeps its own running maximum, sum and O, and the four are joined
// at the end.  Rows past the keys in use are not read: zeros take their place.
// Measured (48 sequences of up to 8192 cached keys, 32 / 8 heads of 128): 174
// to 181 us by board, 6.0 TB/s, 0.90 to 0.94 of the measured copy rate.
#pragma once

#include "packed_fwd_tc.cuh"

namespace prism {

constexpr int kPrWarps = 4, kPrStages = 3, kPrKeys = 32;
template <int D>
constexpr int kPrSmem = 16 * D * 2 + kPrWarps * kPrStages * 2 * kPrKeys * D * 2;

template <int D>
__global__ void __launch_bounds__(kPrWarps * 32) packed_fwd_rows_kernel(const PackedArgs a, const PackedSplit sp) {
  constexpr int CH = D / 8, kTile = kPrKeys * D * 2;
  extern __shared__ __align__(128) uint8_t pr_smem[];
  __shared__ float sm[kPrWarps][16], sl[kPrWarps][16], sn[kPrWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = (int)(blockIdx.x % a.kv_heads);
  const int64_t slot = blockIdx.x / a.kv_heads;
  after_previous();
  PackedSeq::check(a, slot);
  int64_t piece;
  const int b = find_sequence(a.qs, slot, a.group, 16, piece);
  PackedSeq s;
  if (!s.load(a, b)) return;
  const int64_t nrows = (int64_t)s.lq * a.group;
  if (piece < 0 || piece * 16 >= nrows) return;
  const int r0 = (int)(piece * 16), rows = (int)min((int64_t)16, nrows - r0);
  // the share's keys: tiles of 32 in [t0, t1), seen by some row
  const int all = (s.visible(a, (r0 + rows - 1) / a.group) + kPrKeys - 1) / kPrKeys;
  const int t0 = (int)((int64_t)all * blockIdx.z / sp.splits), t1 = (int)((int64_t)all * (blockIdx.z + 1) / sp.splits);

  const uint32_t sQ = smem_u32(pr_smem);
  const uint32_t ring = sQ + 16 * D * 2 + (uint32_t)warp * kPrStages * 2 * kTile;
  const int ch = lane % CH, rr = lane / CH;            // this lane's piece and first row of a tile
  constexpr int kRowStep = 32 / CH;
  const __nv_bfloat16 *gk = a.k + (int64_t)s.k0 * a.sk[0] + (int64_t)kvh * a.sk[1] + ch * 8;
  const __nv_bfloat16 *gv = a.v + (int64_t)s.k0 * a.sv[0] + (int64_t)kvh * a.sv[1] + ch * 8;
  auto fetch = [&](int t, int st) {
    if (t < t1) {
      const uint32_t dk = ring + (uint32_t)st * 2 * kTile, dv = dk + kTile;
#pragma unroll
      for (int i = 0; i < kPrKeys / kRowStep; ++i) {
        const int r = rr + i * kRowStep;
        const int64_t key = (int64_t)t * kPrKeys + r;
        const bool have = key < s.lk;
        const int64_t kk = have ? key : 0;
        cp_async16_or_zero(dk + tile_off<D>(r, ch), gk + kk * a.sk[0], have);
        cp_async16_or_zero(dv + tile_off<D>(r, ch), gv + kk * a.sv[0], have);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kPrStages - 1; ++i) fetch(t0 + warp + i * kPrWarps, i);
  // Q: 16 rows, zeros past the end (every warp needs them all)
  for (int i = threadIdx.x; i < 16 * CH; i += kPrWarps * 32) {
    const int r = i / CH, c = i % CH;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const int fr = r0 + r, tok = fr / a.group;
      w = *reinterpret_cast<const uint4 *>(a.q + (int64_t)(s.q0 + tok) * a.sq[0] +
                                           (int64_t)(kvh * a.group + fr - tok * a.group) * a.sq[1] + c * 8);
    }
    *reinterpret_cast<uint4 *>(pr_smem + tile_off<D>(r, c)) = w;
  }
  __syncthreads();
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) load_a_frag<D>(qf[k], sQ, 0, k * 16);
  // this thread's rows: lane / 4 and lane / 4 + 8
  int vis[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = (lane >> 2) + 8 * r;
    vis[r] = row < rows ? s.visible(a, (r0 + row) / a.group) : 0;
  }
  float acc[D / 8][4];
#pragma unroll
  for (int t = 0; t < D / 8; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, nr[2] = {0.f, 0.f};   // nr: sum of P as rounded
  const float sl2 = a.scale_log2;
  int st = 0;
  for (int t = t0 + warp; t < t1; t += kPrWarps) {
    fetch(t + (kPrStages - 1) * kPrWarps, (st + kPrStages - 1) % kPrStages);
    cp_async_wait<kPrStages - 1>();
    __syncwarp();
    const uint32_t tK = ring + (uint32_t)st * 2 * kTile, tV = tK + kTile;
    float x[kPrKeys / 8][4];
#pragma unroll
    for (int n = 0; n < kPrKeys / 8; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int n = 0; n < kPrKeys / 16; ++n) {
        uint32_t f[4];
        load_b_nk<D>(f, tK, n * 16, k * 16);
        mma16816(x[2 * n], qf[k], f[0], f[1]);
        mma16816(x[2 * n + 1], qf[k], f[2], f[3]);
      }
    const int k0 = t * kPrKeys + (lane & 3) * 2;
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < kPrKeys / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[n][e] = k0 + 8 * n + (e & 1) < vis[e >> 1] ? x[n][e] * sl2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], x[n][e]);
      }
    float c[2], mm[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      mx[r] = fmaxf(mx[r], m[r]);
      mm[r] = mx[r] == -INFINITY ? 0.f : mx[r];     // nothing seen yet: 2^(-inf - 0) = 0
      c[r] = tc::ex2(m[r] - mm[r]);
      m[r] = mx[r];
      l[r] *= c[r];
      nr[r] *= c[r];
    }
    uint32_t p[kPrKeys / 16][4];
#pragma unroll
    for (int n = 0; n < kPrKeys / 8; ++n) {
      const float p0 = tc::ex2(x[n][0] - mm[0]), p1 = tc::ex2(x[n][1] - mm[0]);
      const float p2 = tc::ex2(x[n][2] - mm[1]), p3 = tc::ex2(x[n][3] - mm[1]);
      l[0] += p0 + p1;
      l[1] += p2 + p3;
      // P enters the product as bf16, and what divides O sums it after that
      // rounding, as in the other forward kernel
      const uint32_t a01 = pack_bf16(p0, p1), a23 = pack_bf16(p2, p3);
      p[n >> 1][(n & 1) * 2] = a01;
      p[n >> 1][(n & 1) * 2 + 1] = a23;
      nr[0] += bf16_lo(a01) + bf16_hi(a01);
      nr[1] += bf16_lo(a23) + bf16_hi(a23);
    }
#pragma unroll
    for (int d = 0; d < D / 8; ++d) {
      acc[d][0] *= c[0]; acc[d][1] *= c[0];
      acc[d][2] *= c[1]; acc[d][3] *= c[1];
    }
#pragma unroll
    for (int k = 0; k < kPrKeys / 16; ++k)
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t f[4];
        load_b_kn<D>(f, tV, k * 16, d * 16);
        mma16816(acc[2 * d], p[k], f[0], f[1]);
        mma16816(acc[2 * d + 1], p[k], f[2], f[3]);
      }
    __syncwarp();       // the stage may be filled again
    st = (st + 1) % kPrStages;
  }
  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    nr[r] += __shfl_xor_sync(0xffffffffu, nr[r], 1);
    nr[r] += __shfl_xor_sync(0xffffffffu, nr[r], 2);
    if ((lane & 3) == 0) {
      sm[warp][(lane >> 2) + 8 * r] = m[r];
      sl[warp][(lane >> 2) + 8 * r] = l[r];
      sn[warp][(lane >> 2) + 8 * r] = nr[r];
    }
  }
  __syncthreads();      // all rings are idle: they hold the four warps' O next, fp32 [warp][16][D]
  float *const so = reinterpret_cast<float *>(pr_smem + 16 * D * 2);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = (lane >> 2) + 8 * r;
    float top = sm[0][row];
#pragma unroll
    for (int w = 1; w < kPrWarps; ++w) top = fmaxf(top, sm[w][row]);
    const float f = top == -INFINITY ? 0.f : tc::ex2(m[r] - top);
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
      *reinterpret_cast<float2 *>(so + (warp * 16 + row) * D + d * 8 + (lane & 3) * 2) =
          make_float2(acc[d][2 * r] * f, acc[d][2 * r + 1] * f);
  }
  __syncthreads();
  constexpr int kPieces = D / 4;
  for (int i = threadIdx.x; i < rows * kPieces; i += kPrWarps * 32) {
    const int row = i / kPieces, c4 = (i % kPieces) * 4;
    float top = sm[0][row], sum = 0.f, nsum = 0.f;
#pragma unroll
    for (int w = 1; w < kPrWarps; ++w) top = fmaxf(top, sm[w][row]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPrWarps; ++w) {
      const float f = top > -INFINITY ? tc::ex2(sm[w][row] - top) : 1.f;      // 1: the sums are 0 or NaN
      sum += sl[w][row] * f;
      nsum += sn[w][row] * f;
      const float4 q = *reinterpret_cast<const float4 *>(so + (w * 16 + row) * D + c4);
      o.x += q.x; o.y += q.y; o.z += q.z; o.w += q.w;
    }
    const float inv = nsum == 0.f ? 0.f : 1.f / nsum;      // 0: saw no key; NaN stays NaN
    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    const int fr = r0 + row, tok = fr / a.group, head = kvh * a.group + fr - tok * a.group;
    const int64_t at = s.q0 + tok;
    const float l2 = sum == 0.f ? -INFINITY : top + log2f(sum);
    if (sp.splits > 1) {
      *reinterpret_cast<float4 *>(sp.o + (((int64_t)blockIdx.z * a.qs.rows + at) * a.heads + head) * D + c4) =
          make_float4(v[0], v[1], v[2], v[3]);
      if (c4 == 0) sp.lse2[((int64_t)blockIdx.z * a.heads + head) * a.qs.rows + at] = l2;
    } else {
      const uint2 u = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      *reinterpret_cast<uint2 *>(a.o + at * a.so[0] + head * a.so[1] + c4) = u;
      if (a.o_res)
        *reinterpret_cast<uint2 *>(a.o_res + (at * a.heads + head) * D + c4) =
            make_uint2(pack_bf16(v[0] - bf16_lo(u.x), v[1] - bf16_hi(u.x)), pack_bf16(v[2] - bf16_lo(u.y), v[3] - bf16_hi(u.y)));
      if (c4 == 0) a.lse[(int64_t)head * a.qs.rows + at] = l2 * kLn2;
    }
  }
}

}  // namespace prism
