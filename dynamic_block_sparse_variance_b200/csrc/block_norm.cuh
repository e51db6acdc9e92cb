// The norms around a block, fused with its gate and the residual stream
// (a diffusion transformer's adaptive norm, a language model's sandwich norm):
//   x_out = alpha x + gate (N_post(y) w_post)          y: the block's output
//   h     = N_pre(x_out) w (1 + scale) + shift          the next block's input
// N is the identity, x / sqrt(mean(x^2) + eps), or that of x - mean(x); gate,
// scale and shift belong to the packed sequence of the row.
//
// Both directions are bound by HBM: a row is read once, kept in registers
// while its statistics are reduced, and written once.  A thread owns the same
// 8 (or 16) columns of every row of its CTA's run of rows, so the column
// parameters, folded to w (1 + scale), shift and gate w_post in fp32, stay in
// registers too, and so do the backward's column sums, which leave the CTA
// once per run.
#pragma once

#include <type_traits>

#include "packed_common.cuh"

namespace prism {

constexpr int kBnMaxChannels = 8192;
constexpr int kBnMaxThreads = 512;

struct BlockNormArgs {
  Offsets seq;
  int C, unit;               // channels, rows per slot
  int post, pre;             // PRISM_NORM_*
  int param_f32;
  float eps, alpha;
  int64_t sx, sy, sxo, sh, sdh, sdxo, sdx, sdy;   // row strides (elements)
  const void *x, *y, *post_weight, *gate, *weight, *scale, *shift, *dh, *dx_out;
  int64_t sgate, sscale, sshift;                  // elements from one sequence to the next
  void *x_out, *h, *dx, *dy;
  float *y_norms;
  float *part;               // backward: [slots * rows per pass][3][C] column sums
};

// Eight consecutive elements as loaded, and as fp32.
template <typename T>
struct BnVec8;
template <>
struct BnVec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void get(float *f) const {
    f[0] = bf16_lo(a.x); f[1] = bf16_hi(a.x); f[2] = bf16_lo(a.y); f[3] = bf16_hi(a.y);
    f[4] = bf16_lo(a.z); f[5] = bf16_hi(a.z); f[6] = bf16_lo(a.w); f[7] = bf16_hi(a.w);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16 *p, const float *f) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                    pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
  }
};
template <>
struct BnVec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void get(float *f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ static void store(float *p, const float *f) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  }
};

__device__ __forceinline__ float param_at(const void *p, int64_t i, int f32) {
  return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
// Eight parameters from element i on (i a multiple of 8).
__device__ __forceinline__ void param8(const void *p, int64_t i, int f32, float *f) {
  if (f32) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    BnVec8<__nv_bfloat16> v;
    v.a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i));
    v.get(f);
  }
}

// Sums K values over the threads of one row (`wpr` warps), the same on every
// thread: a butterfly in each warp, then the warps' sums in warp order.  Rows
// of a CTA use barriers of their own (1 + row slot); `buf` alternates between
// two halves of `red`, so one barrier per reduction is enough.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float *red, int &buf, int wpr, int warp_in_row, int sub) {
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = warp_sum(v[i]);
  if (wpr == 1) return;
  float *half = red + buf * (kBnMaxThreads / 32) * 4 + sub * wpr * 4;
  buf ^= 1;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < K; ++i) half[warp_in_row * 4 + i] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(wpr * 32) : "memory");
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = 0.f;
  for (int w = 0; w < wpr; ++w) {
    const float4 t = *reinterpret_cast<const float4 *>(half + 4 * w);
    const float tv[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += tv[i];
  }
}

// Column parameters of sequence b for this thread's columns.
template <int V>
struct BnColumns {
  float A[8 * V], B[8 * V], G[8 * V];
  __device__ __forceinline__ void load(const BlockNormArgs &a, int b, int t, int tpr) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * tpr + t) * 8;
      float w[8], s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) A[8 * v + e] = 1.f, B[8 * v + e] = 0.f, G[8 * v + e] = 1.f;
      if (c >= a.C) continue;
      if (a.weight) {
        param8(a.weight, c, a.param_f32, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) A[8 * v + e] = w[e];
      }
      if (a.scale) {
        param8(a.scale, b * a.sscale + c, a.param_f32, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) A[8 * v + e] *= 1.f + s[e];
      }
      if (a.shift) param8(a.shift, b * a.sshift + c, a.param_f32, B + 8 * v);
      if (a.post_weight) param8(a.post_weight, c, a.param_f32, G + 8 * v);
      if (a.gate) {
        param8(a.gate, b * a.sgate + c, a.param_f32, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) G[8 * v + e] *= s[e];
      }
    }
  }
};

template <typename TX, typename TY, int V>
__global__ void __launch_bounds__(kBnMaxThreads) block_norm_fwd_kernel(const BlockNormArgs a, int wpr) {
  __shared__ __align__(16) float red[2 * (kBnMaxThreads / 32) * 4];
  const int warp = threadIdx.x >> 5;
  const int sub = warp / wpr, wir = warp - sub * wpr;    // row slot of the CTA, warp within the row
  const int rpc = (blockDim.x >> 5) / wpr;
  const int tpr = wpr * 32, t = threadIdx.x - sub * tpr;
  int64_t piece;
  check_sequence(a.seq, blockIdx.x);
  const int b = find_sequence(a.seq, blockIdx.x, 1, a.unit, piece);
  int begin, len;
  if (!sequence_rows(a.seq, b, begin, len)) return;
  if (piece < 0 || piece * a.unit >= len) return;
  const int r0 = begin + (int)piece * a.unit, r1 = min(begin + len, r0 + a.unit);

  BnColumns<V> col;
  col.load(a, b, t, tpr);
  const TX *x = static_cast<const TX *>(a.x);
  const TY *y = static_cast<const TY *>(a.y);
  TX *xo = static_cast<TX *>(a.x_out);
  TY *h = static_cast<TY *>(a.h);
  const float inv_c = 1.f / (float)a.C;
  int buf = 0;

  BnVec8<TX> xv[V];
  BnVec8<TY> yv[V];
  auto fetch = [&](int r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c < a.C) {
        xv[v].load(x + (int64_t)r * a.sx + c);
        if (y) yv[v].load(y + (int64_t)r * a.sy + c);
      }
    }
  };
  int r = r0 + sub;
  if (r < r1) fetch(r);
  for (; r < r1; r += rpc) {   // the rows of one slot run on their own barrier
    float res[8 * V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if ((v * tpr + t) * 8 < a.C) {
        xv[v].get(res + 8 * v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) res[8 * v + e] = 0.f;
      }
    }
    if (y) {
      float f[8 * V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if ((v * tpr + t) * 8 < a.C) {
          yv[v].get(f + 8 * v);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[8 * v + e] = 0.f;
        }
      }
      if (r + rpc < r1) fetch(r + rpc);
      float mu = 0.f, rs = 1.f;
      float s2[2] = {0.f, 0.f};
      if (a.post != PRISM_NORM_NONE || a.y_norms) {
#pragma unroll
        for (int e = 0; e < 8 * V; ++e) s2[0] += f[e], s2[1] = fmaf(f[e], f[e], s2[1]);
        row_sums(s2, red, buf, wpr, wir, sub);
        if (a.y_norms && t == 0) a.y_norms[r] = sqrtf(s2[1]);
      }
      if (a.post == PRISM_NORM_RMS) {
        rs = rsqrtf(s2[1] * inv_c + a.eps);
      } else if (a.post == PRISM_NORM_LAYER) {
        mu = s2[0] * inv_c;
        float q[1] = {0.f};
#pragma unroll
        for (int v = 0; v < V; ++v)
          if ((v * tpr + t) * 8 < a.C) {
#pragma unroll
            for (int e = 0; e < 8; ++e) q[0] = fmaf(f[8 * v + e] - mu, f[8 * v + e] - mu, q[0]);
          }
        row_sums(q, red, buf, wpr, wir, sub);
        rs = rsqrtf(q[0] * inv_c + a.eps);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * tpr + t) * 8;
        if (c < a.C) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            res[8 * v + e] = fmaf(col.G[8 * v + e], (f[8 * v + e] - mu) * rs, a.alpha * res[8 * v + e]);
          if (xo) BnVec8<TX>::store(xo + (int64_t)r * a.sxo + c, res + 8 * v);
        }
      }
    } else if (r + rpc < r1) {
      fetch(r + rpc);
    }
    if (!h) continue;
    float mu = 0.f;
    if (a.pre == PRISM_NORM_LAYER) {
      float s[1] = {0.f};
#pragma unroll
      for (int e = 0; e < 8 * V; ++e) s[0] += res[e];
      row_sums(s, red, buf, wpr, wir, sub);
      mu = s[0] * inv_c;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((v * tpr + t) * 8 < a.C) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[0] = fmaf(res[8 * v + e] - mu, res[8 * v + e] - mu, q[0]);
      }
    row_sums(q, red, buf, wpr, wir, sub);
    const float rs = rsqrtf(q[0] * inv_c + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c < a.C) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e] = fmaf((res[8 * v + e] - mu) * rs, col.A[8 * v + e], col.B[8 * v + e]);
        BnVec8<TY>::store(h + (int64_t)r * a.sh + c, o);
      }
    }
  }
}

// Backward.  With r = x_out, u = r - mean, xhat = u rs and d = dh w (1 + scale):
//   dr = rs (d - mean(d) - xhat mean(d xhat)) + dx_out   (mean(d): only with a mean)
//   dx = alpha dr,  e = dr gate w_post,  dy = rs_y (e - mean(e) - yhat mean(e yhat))
// and the column sums sum(dh xhat), sum(dh), sum(dr yhat), from which the
// parameters' gradients follow (block_norm_params_kernel).  The statistics
// are formed again from x_out and y, which the pass reads anyway: keeping
// them would cost the forward a write and this pass a read.
template <typename TX, typename TY, int V>
__global__ void __launch_bounds__(kBnMaxThreads) block_norm_bwd_kernel(const BlockNormArgs a, int wpr) {
  __shared__ __align__(16) float red[2 * (kBnMaxThreads / 32) * 4];
  const int warp = threadIdx.x >> 5;
  const int sub = warp / wpr, wir = warp - sub * wpr;
  const int rpc = (blockDim.x >> 5) / wpr;
  const int tpr = wpr * 32, t = threadIdx.x - sub * tpr;
  int64_t piece;
  check_sequence(a.seq, blockIdx.x);
  const int b = find_sequence(a.seq, blockIdx.x, 1, a.unit, piece);
  int begin, len;
  if (!sequence_rows(a.seq, b, begin, len)) return;
  if (piece < 0 || piece * a.unit >= len) return;
  const int r0 = begin + (int)piece * a.unit, r1 = min(begin + len, r0 + a.unit);

  BnColumns<V> col;
  col.load(a, b, t, tpr);
  const TX *xo = static_cast<const TX *>(a.x_out), *dxo = static_cast<const TX *>(a.dx_out);
  const TY *y = static_cast<const TY *>(a.y), *dh = static_cast<const TY *>(a.dh);
  TX *dx = static_cast<TX *>(a.dx);
  TY *dy = static_cast<TY *>(a.dy);
  const float inv_c = 1.f / (float)a.C;
  int buf = 0;
  float p1[8 * V], p2[8 * V], p3[8 * V];
#pragma unroll
  for (int e = 0; e < 8 * V; ++e) p1[e] = p2[e] = p3[e] = 0.f;

  BnVec8<TX> xv[V], gv[V];
  BnVec8<TY> yv[V], hv[V];
  auto fetch = [&](int r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c < a.C) {
        if (dh) {
          xv[v].load(xo + (int64_t)r * a.sxo + c);
          hv[v].load(dh + (int64_t)r * a.sdh + c);
        }
        if (dxo) gv[v].load(dxo + (int64_t)r * a.sdxo + c);
        if (y) yv[v].load(y + (int64_t)r * a.sy + c);
      }
    }
  };
  int r = r0 + sub;
  if (r < r1) fetch(r);
  for (; r < r1; r += rpc) {
    float dr[8 * V], f[8 * V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool in = (v * tpr + t) * 8 < a.C;
      if (in && dxo) {
        gv[v].get(dr + 8 * v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dr[8 * v + e] = 0.f;
      }
      if (in && y) {
        yv[v].get(f + 8 * v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[8 * v + e] = 0.f;
      }
    }
    float u[8 * V], g[8 * V];
    if (dh) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if ((v * tpr + t) * 8 < a.C) {
          xv[v].get(u + 8 * v);
          hv[v].get(g + 8 * v);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[8 * v + e] = g[8 * v + e] = 0.f;
        }
      }
    }
    if (r + rpc < r1) fetch(r + rpc);
    // means
    float mu = 0.f, muy = 0.f;
    const bool lx = dh && a.pre == PRISM_NORM_LAYER, ly = y && a.post == PRISM_NORM_LAYER;
    if (lx || ly) {
      float s[2] = {0.f, 0.f};
      if (lx) {
#pragma unroll
        for (int e = 0; e < 8 * V; ++e) s[0] += u[e];
      }
      if (ly) {
#pragma unroll
        for (int e = 0; e < 8 * V; ++e) s[1] += f[e];
      }
      row_sums(s, red, buf, wpr, wir, sub);
      mu = s[0] * inv_c;
      muy = s[1] * inv_c;
    }
    // centred squares, and the sums of the pre-norm's gradient
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((v * tpr + t) * 8 < a.C) {
        if (dh) {
#pragma unroll
          for (int e = 8 * v; e < 8 * v + 8; ++e) {
            u[e] -= mu;
            const float d = g[e] * col.A[e];
            s4[0] = fmaf(u[e], u[e], s4[0]);
            s4[1] += d;
            s4[2] = fmaf(d, u[e], s4[2]);
          }
        }
        if (y) {
#pragma unroll
          for (int e = 8 * v; e < 8 * v + 8; ++e) {
            f[e] -= muy;
            s4[3] = fmaf(f[e], f[e], s4[3]);
          }
        }
      }
    row_sums(s4, red, buf, wpr, wir, sub);
    if (dh) {
      const float rs = rsqrtf(s4[0] * inv_c + a.eps);
      const float c1 = a.pre == PRISM_NORM_LAYER ? s4[1] * inv_c : 0.f;
      const float c2 = s4[2] * rs * inv_c;    // mean(d xhat)
#pragma unroll
      for (int e = 0; e < 8 * V; ++e) {
        const float xh = u[e] * rs, d = g[e] * col.A[e];
        dr[e] += rs * (d - c1 - xh * c2);
        p1[e] = fmaf(g[e], xh, p1[e]);
        p2[e] += g[e];
      }
    }
    float dxs[8 * V];
    const float al = y ? a.alpha : 1.f;
#pragma unroll
    for (int e = 0; e < 8 * V; ++e) dxs[e] = al * dr[e];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c < a.C) BnVec8<TX>::store(dx + (int64_t)r * a.sdx + c, dxs + 8 * v);
    }
    if (!y) continue;
    float m1 = 0.f, m2 = 0.f, rsy = 1.f;
    if (a.post != PRISM_NORM_NONE) {
      rsy = rsqrtf(s4[3] * inv_c + a.eps);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int v = 0; v < V; ++v)
        if ((v * tpr + t) * 8 < a.C) {
#pragma unroll
          for (int e = 8 * v; e < 8 * v + 8; ++e) {
            f[e] *= rsy;
            const float de = dr[e] * col.G[e];
            s[0] += de;
            s[1] = fmaf(de, f[e], s[1]);
          }
        }
      row_sums(s, red, buf, wpr, wir, sub);
      m1 = a.post == PRISM_NORM_LAYER ? s[0] * inv_c : 0.f;
      m2 = s[1] * inv_c;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c < a.C) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = 8 * v + e;
          p3[k] = fmaf(dr[k], f[k], p3[k]);
          o[e] = rsy * (dr[k] * col.G[k] - m1 - f[k] * m2);
        }
        BnVec8<TY>::store(dy + (int64_t)r * a.sdy + c, o);
      }
    }
  }
  if (a.part) {
    float *out = a.part + ((int64_t)blockIdx.x * rpc + sub) * 3 * a.C;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c < a.C) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          *reinterpret_cast<float4 *>(out + c + 4 * k) =
              make_float4(p1[8 * v + 4 * k], p1[8 * v + 4 * k + 1], p1[8 * v + 4 * k + 2], p1[8 * v + 4 * k + 3]);
          *reinterpret_cast<float4 *>(out + a.C + c + 4 * k) =
              make_float4(p2[8 * v + 4 * k], p2[8 * v + 4 * k + 1], p2[8 * v + 4 * k + 2], p2[8 * v + 4 * k + 3]);
          *reinterpret_cast<float4 *>(out + 2 * a.C + c + 4 * k) =
              make_float4(p3[8 * v + 4 * k], p3[8 * v + 4 * k + 1], p3[8 * v + 4 * k + 2], p3[8 * v + 4 * k + 3]);
        }
      }
    }
  }
}

// Parameter gradients from the column sums, in two steps with a fixed order
// of additions.  Step 1, one CTA per (32 columns, sequence): the sums of the
// sequence's slots; per-sequence gradients leave here.
struct BnParamArgs {
  Offsets seq;
  int C, unit, rpc, param_f32;
  const float *part;         // [slots * rpc][3][C]
  float *sums;               // [seqs][3][C]
  const void *weight, *post_weight, *gate, *scale;
  int64_t sgate, sscale;
  void *dweight, *dpost_weight;               // [C]
  void *dgate, *dscale, *dshift;              // [seqs, C], or [C] where the parameter is shared
  int per_gate, per_scale, per_shift;         // one gradient row per sequence
};
__device__ __forceinline__ void put_param(void *p, int64_t i, float v, int f32) {
  if (f32) static_cast<float *>(p)[i] = v;
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__global__ void __launch_bounds__(1024) block_norm_sums_kernel(const BnParamArgs a) {
  __shared__ float sh[32][3][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, b = blockIdx.y;
  int begin, len;
  const bool ok = sequence_rows(a.seq, b, begin, len);
  const int64_t first = ((int64_t)begin / a.unit + b) * a.rpc;
  const int64_t n = ok ? (int64_t)((len + a.unit - 1) / a.unit) * a.rpc : 0;
  float s[3] = {0.f, 0.f, 0.f};
  if (c < a.C) {
    for (int64_t i = w; i < n; i += 32) {
      const float *p = a.part + (first + i) * 3 * a.C + c;
      s[0] += p[0];
      s[1] += p[a.C];
      s[2] += p[2 * (int64_t)a.C];
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) sh[w][k][lane] = s[k];
  __syncthreads();
  if (w < 3) {
    float v = 0.f;
    for (int i = 0; i < 32; ++i) v += sh[i][w][lane];
    if (c < a.C) {
      a.sums[((int64_t)b * 3 + w) * a.C + c] = v;
      const int64_t at = (int64_t)b * a.C + c;
      if (w == 0 && a.dscale && a.per_scale)
        put_param(a.dscale, at, a.weight ? v * param_at(a.weight, c, a.param_f32) : v, a.param_f32);
      if (w == 1 && a.dshift && a.per_shift) put_param(a.dshift, at, v, a.param_f32);
      if (w == 2 && a.dgate && a.per_gate)
        put_param(a.dgate, at, a.post_weight ? v * param_at(a.post_weight, c, a.param_f32) : v, a.param_f32);
    }
  }
}

// Step 2, one thread per column: what is summed over the sequences.
__global__ void __launch_bounds__(128) block_norm_params_kernel(const BnParamArgs a) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= a.C) return;
  float dw = 0.f, dpw = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  for (int b = 0; b < a.seq.seqs; ++b) {
    const float *p = a.sums + (int64_t)b * 3 * a.C + c;
    const float q1 = p[0], q2 = p[a.C], q3 = p[2 * (int64_t)a.C];
    s1 += q1;
    s2 += q2;
    s3 += q3;
    dw = fmaf(a.scale ? 1.f + param_at(a.scale, b * a.sscale + c, a.param_f32) : 1.f, q1, dw);
    dpw = fmaf(a.gate ? param_at(a.gate, b * a.sgate + c, a.param_f32) : 1.f, q3, dpw);
  }
  if (a.dweight) put_param(a.dweight, c, dw, a.param_f32);
  if (a.dpost_weight) put_param(a.dpost_weight, c, dpw, a.param_f32);
  if (a.dscale && !a.per_scale)
    put_param(a.dscale, c, a.weight ? s1 * param_at(a.weight, c, a.param_f32) : s1, a.param_f32);
  if (a.dshift && !a.per_shift) put_param(a.dshift, c, s2, a.param_f32);
  if (a.dgate && !a.per_gate)
    put_param(a.dgate, c, a.post_weight ? s3 * param_at(a.post_weight, c, a.param_f32) : s3, a.param_f32);
}

}  // namespace prism
