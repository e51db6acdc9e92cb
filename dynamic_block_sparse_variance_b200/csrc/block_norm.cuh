// The norms around a block, fused with its gate and the residual stream
// (a diffusion transformer's adaptive norm, a language model's sandwich norm):
//   x_out = alpha x + gate (N_post(y) w_post)          y: the block's output
//   h     = N_pre(x_out) w (1 + scale) + shift          the next block's input
// N is the identity, x / sqrt(mean(x^2) + eps), or that of x - mean(x); gate,
// scale and shift belong to the packed sequence of the row.
//
// Both directions are bound by HBM: a row is read once and written once.  A
// CTA works through a run of rows of one sequence.  The rows come in through
// bulk copies into a ring in shared memory, issued ahead by one thread, so the
// bytes in flight do not depend on registers.  What sets the time otherwise is
// the reductions: with a row spread over a whole CTA (8 columns a thread) every
// statistic is a butterfly, a barrier and a table, about 1000 cycles of
// dependent latency, and most instructions (61440 x 1536 forward: 208 us, 143 us as
// it is now, 5.3 TB/s, 0.81 of the measured copy rate).  So
//   forward   a row belongs to one warp (2 to 4 beyond 2048 channels), which
//             keeps it in registers; warps run on their own, without barriers
//   backward  the column sums, three per column, want to stay in registers, so
//             a row is spread over the CTA all the same, two rows at a time
// (The backward with rows by warps for the statistics and columns by threads for
// the results reads each row three times and was slower: 331 us against 233 then at
// 30011 x 2048.  204 us now, 3.6 TB/s: what is left is the two exchanges of sums per
// pair of rows, whose barriers 16 warps per SM hide only in part.)
#pragma once

#include "packed_common.cuh"
#include "packed_runs.cuh"
#include "tc_common.cuh"

namespace prism {

constexpr int kBnWarps = 16;          // forward
constexpr int kBnMaxThreads = 512;    // backward
constexpr int kBnMaxGroups = 8;       // rows of a CTA at a time, backward
constexpr int kBnMaxStages = 4;

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
  float *part;               // backward: [slots * groups][3][C] column sums
  int need;                  // backward: bit k, column sum k is wanted
  int wpr, groups, stages;   // warps per row, row groups of a CTA, stages of a ring
  int vecs;                  // forward: 256-column vectors per warp
  uint32_t wait_limit;
};

// Eight consecutive elements as four fp32 pairs: sums and products run on
// register pairs (tc::fma2 and its kin), two lanes an instruction.
template <typename T>
struct BnVec8;
template <>
struct BnVec8<__nv_bfloat16> {
  __device__ __forceinline__ static void unpack(const uint4 &a, float2 *f) {
    f[0] = tc::f2(bf16_lo(a.x), bf16_hi(a.x));
    f[1] = tc::f2(bf16_lo(a.y), bf16_hi(a.y));
    f[2] = tc::f2(bf16_lo(a.z), bf16_hi(a.z));
    f[3] = tc::f2(bf16_lo(a.w), bf16_hi(a.w));
  }
  __device__ __forceinline__ static void load(const __nv_bfloat16 *p, float2 *f) {
    unpack(*reinterpret_cast<const uint4 *>(p), f);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16 *p, const float2 *f) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y),
                                                    pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y)));
  }
};
template <>
struct BnVec8<float> {
  __device__ __forceinline__ static void load(const float *p, float2 *f) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = tc::f2(a.x, a.y);
    f[1] = tc::f2(a.z, a.w);
    f[2] = tc::f2(b.x, b.y);
    f[3] = tc::f2(b.z, b.w);
  }
  __device__ __forceinline__ static void store(float *p, const float2 *f) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
  }
};
__device__ __forceinline__ float2 both(float x) { return tc::f2(x, x); }
// (a, b) + (c, d) as one packed instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float param_at(const void *p, int64_t i, int f32) {
  return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
// Eight parameters from element i on (i a multiple of 8).
__device__ __forceinline__ void param8(const void *p, int64_t i, int f32, float2 *f) {
  if (f32) BnVec8<float>::load(static_cast<const float *>(p) + i, f);
  else BnVec8<__nv_bfloat16>::load(static_cast<const __nv_bfloat16 *>(p) + i, f);
}

// Folded parameters of 8 columns from c on: w (1 + scale), shift, gate w_post.
__device__ __forceinline__ void fold_params(const BlockNormArgs &a, int b, int c, float2 (&A)[4], float2 (&B)[4], float2 (&G)[4]) {
  float2 s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] = both(1.f), B[e] = both(0.f), G[e] = both(1.f);
  if (a.weight) param8(a.weight, c, a.param_f32, A);
  if (a.scale) {
    param8(a.scale, b * a.sscale + c, a.param_f32, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) A[e] = tc::mul2(A[e], add2(s[e], both(1.f)));
  }
  if (a.shift) param8(a.shift, b * a.sshift + c, a.param_f32, B);
  if (a.post_weight) param8(a.post_weight, c, a.param_f32, G);
  if (a.gate) {
    param8(a.gate, b * a.sgate + c, a.param_f32, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) G[e] = tc::mul2(G[e], s[e]);
  }
}
__device__ __forceinline__ float sum8(const float2 (&x)[4]) {
  const float2 s = add2(add2(x[0], x[1]), add2(x[2], x[3]));
  return s.x + s.y;
}
__device__ __forceinline__ void shift8(float2 (&x)[4], float m) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = add2(x[e], both(-m));
}
__device__ __forceinline__ float2 dot8(const float2 (&x)[4], const float2 (&y)[4], float2 q) {
#pragma unroll
  for (int e = 0; e < 4; ++e) q = tc::fma2(x[e], y[e], q);
  return q;
}

// The run of rows [r0, r1) of sequence b that slot blockIdx.x stands for.
__device__ __forceinline__ bool bn_rows(const BlockNormArgs &a, int &b, int &r0, int &r1) {
  int64_t piece;
  check_sequence(a.seq, blockIdx.x);
  b = find_sequence(a.seq, blockIdx.x, 1, a.unit, piece);
  int begin, len;
  if (!sequence_rows(a.seq, b, begin, len)) return false;
  if (!run_rows(begin, len, piece, a.unit, r0, r1)) return false;
  // The two as plain numbers: where the compiler sees how r1 follows from r0, it orders the
  // backward's loop otherwise (30011 x 2048: 219 us against 203).
  asm volatile("" : "+r"(r0), "+r"(r1));
  return true;
}

// ---- forward -------------------------------------------------------------------
// Row group `sub` of the CTA: wpr warps, a ring of single rows and, for wpr > 1,
// named barrier 1 + sub and a table for sums.  V: vectors of 8 columns a thread
// holds at most (a.vecs of them are used); vector v of a warp's lane covers
// columns (warp vecs + v) 256 + 8 lane ...
template <int V>
struct BnRow {
  int wpr, sub, warp, n, buf;
  float *red;          // [2][wpr][2]
  __device__ __forceinline__ void sync() const {
    if (wpr == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(wpr * 32) : "memory");
  }
  __device__ __forceinline__ float sum(float x) {
    x = warp_sum(x);
    if (wpr == 1) return x;
    float *h = red + buf * wpr;
    buf ^= 1;          // two halves used in turn: one barrier per sum
    if ((threadIdx.x & 31) == 0) h[warp] = x;
    sync();
    float s = h[0];
    for (int w = 1; w < wpr; ++w) s += h[w];
    return s;
  }
};

template <typename TX, typename TY, int V>
__global__ void __launch_bounds__(kBnWarps * 32) block_norm_fwd_kernel(const BlockNormArgs a) {
  extern __shared__ __align__(16) uint8_t bn_smem[];     // [A | B | G][C] fp32, rings
  __shared__ uint64_t mbars[kBnWarps * kBnMaxStages];
  __shared__ float red[2 * kBnWarps];
  __shared__ int abort_flag;
  int b, r0, r1;
  after_previous();
  if (!bn_rows(a, b, r0, r1)) return;
  const int lane = threadIdx.x & 31;
  const TX *x = static_cast<const TX *>(a.x);
  const TY *y = static_cast<const TY *>(a.y);
  BnRow<V> g;
  g.wpr = a.wpr;
  g.sub = (threadIdx.x >> 5) / a.wpr;
  g.warp = (threadIdx.x >> 5) - g.sub * a.wpr;
  g.red = red + 2 * g.sub * a.wpr;
  g.buf = 0;
  const int c0 = g.warp * a.vecs * 256 + lane * 8;
  g.n = min(a.vecs, max(0, (a.C - c0 + 255) / 256));
  const int bx = a.C * (int)sizeof(TX), stage_bytes = bx + (y ? a.C * (int)sizeof(TY) : 0);
  uint8_t *ring = bn_smem + 12 * a.C + (size_t)g.sub * a.stages * stage_bytes;
  const uint32_t ring_addr = smem_u32(ring), bars = smem_u32(mbars + g.sub * a.stages);
  volatile int *abort = &abort_flag;
  const bool lead = g.warp == 0 && lane == 0 && g.sub < a.groups;
  if (lead) {
    for (int i = 0; i < a.stages; ++i) tc::mbar_init(bars + 8u * i, 1);
    tc::fence_barrier_init();
  }
  if (threadIdx.x == 0) *abort = 0;
  __syncthreads();
  const int first = r0 + g.sub, rows = g.sub < a.groups && first < r1 ? (r1 - first + a.groups - 1) / a.groups : 0;
  int st_put = 0, st = 0;
  uint32_t ph = 0;
  auto fetch = [&](int it) {
    const int64_t r = first + (int64_t)it * a.groups;
    const uint32_t dst = ring_addr + st_put * stage_bytes, bar = bars + 8u * st_put;
    tc::mbar_expect_tx(bar, stage_bytes);
    tc::bulk_load(dst, x + r * a.sx, bx, bar);
    if (y) tc::bulk_load(dst + bx, y + r * a.sy, stage_bytes - bx, bar);
    if (++st_put == a.stages) st_put = 0;
  };
  if (lead)
    for (int it = 0; it < min(rows, a.stages); ++it) fetch(it);
  float *const pA = reinterpret_cast<float *>(bn_smem), *const pB = pA + a.C, *const pG = pB + a.C;
  for (int c = threadIdx.x * 8; c < a.C; c += blockDim.x * 8) {
    float2 A[4], B[4], G[4];
    fold_params(a, b, c, A, B, G);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *reinterpret_cast<float2 *>(pA + c + 2 * e) = A[e];
      *reinterpret_cast<float2 *>(pB + c + 2 * e) = B[e];
      *reinterpret_cast<float2 *>(pG + c + 2 * e) = G[e];
    }
  }
  __syncthreads();
  const float inv_c = 1.f / (float)a.C;
  TX *xo = static_cast<TX *>(a.x_out) + first * a.sxo + c0;
  TY *h = a.h ? static_cast<TY *>(a.h) + first * a.sh + c0 : nullptr;

  for (int it = 0; it < rows; ++it) {
    // A wait that runs out latches PRISM_ETIMEOUT; the warps go on (with whatever
    // the ring holds), so that every barrier still sees all of its threads.
    tc::mbar_wait(bars + 8u * st, ph, abort, a.wait_limit);
    const TX *sx = reinterpret_cast<const TX *>(ring + st * stage_bytes) + c0;
    const TY *sy = reinterpret_cast<const TY *>(ring + st * stage_bytes + bx) + c0;
    if (++st == a.stages) st = 0, ph ^= 1;
    float2 res[V][4];
    if (y) {
      float mu = 0.f, rs = 1.f;
      if (a.y_norms) {
        float2 q = both(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v < g.n) {
            float2 f[4];
            BnVec8<TY>::load(sy + v * 256, f);
            q = dot8(f, f, q);
          }
        const float z = g.sum(q.x + q.y);
        if (lead) a.y_norms[first + (int64_t)it * a.groups] = sqrtf(z);
      }
      if (a.post != PRISM_NORM_NONE) {
        if (a.post == PRISM_NORM_LAYER) {
          float t = 0.f;
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (v < g.n) {
              float2 f[4];
              BnVec8<TY>::load(sy + v * 256, f);
              t += sum8(f);
            }
          mu = g.sum(t) * inv_c;
        }
        float2 q = both(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v < g.n) {
            float2 f[4];
            BnVec8<TY>::load(sy + v * 256, f);
            shift8(f, mu);
            q = dot8(f, f, q);
          }
        rs = rsqrtf(g.sum(q.x + q.y) * inv_c + a.eps);
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < g.n) {
          float2 f[4], G[4];
          BnVec8<TX>::load(sx + v * 256, res[v]);
          BnVec8<TY>::load(sy + v * 256, f);
          BnVec8<float>::load(pG + c0 + v * 256, G);
          shift8(f, mu);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            res[v][e] = tc::fma2(tc::mul2(f[e], both(rs)), G[e], tc::mul2(res[v][e], both(a.alpha)));
          BnVec8<TX>::store(xo + v * 256, res[v]);
        }
      xo += a.groups * a.sxo;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < g.n) BnVec8<TX>::load(sx + v * 256, res[v]);
    }
    // the row is in registers: the next one may land in its stage
    g.sync();
    if (lead && it + a.stages < rows) fetch(it + a.stages);
    if (h) {
      float mu = 0.f;
      if (a.pre == PRISM_NORM_LAYER) {
        float t = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v < g.n) t += sum8(res[v]);
        mu = g.sum(t) * inv_c;
      }
      float2 q = both(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < g.n) {
          shift8(res[v], mu);
          q = dot8(res[v], res[v], q);
        }
      const float rs = rsqrtf(g.sum(q.x + q.y) * inv_c + a.eps);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < g.n) {
          float2 A[4], o[4];
          BnVec8<float>::load(pA + c0 + v * 256, A);
          BnVec8<float>::load(pB + c0 + v * 256, o);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = tc::fma2(tc::mul2(res[v][e], both(rs)), A[e], o[e]);
          BnVec8<TY>::store(h + v * 256, o);
        }
      h += a.groups * a.sh;
    }
  }
  if (lead && *abort) {      // after a wait ran out: the copies still in flight land before the CTA exits
    volatile int no_abort = 0;
    for (int it = max(0, rows - a.stages); it < rows; ++it)
      tc::mbar_wait(bars + 8u * (it % a.stages), (uint32_t)(it / a.stages) & 1u, &no_abort, a.wait_limit);
  }
}

// ---- backward --------------------------------------------------------------------
// With r = x_out, u = r - mean, xhat = u rs and d = dh w (1 + scale):
//   dr = rs (d - mean(d) - xhat mean(d xhat)) + dx_out   (mean(d): only with a mean)
//   dx = alpha dr,  e = dr gate w_post,  dy = rs_y (e - mean(e) - yhat mean(e yhat))
// and the column sums sum(dh xhat), sum(dh), sum(dr yhat), from which the
// parameters' gradients follow (block_norm_params_kernel).  The statistics
// are formed again from x_out and y, which the pass reads anyway: keeping
// them would cost the forward a write and this pass a read.
//
// R rows at a time (2; 1 beyond 4096 channels): a thread owns the same 8 (or 16)
// columns of every row and sums the R rows' statistics together, so one butterfly
// and one barrier serve several values.  Registers: at 16 columns a thread
// (V = 2) the accumulators of the column sums and a row of values fill them, so
// there the folded parameters live in shared memory.
//
// Sums over a warp of K values (a power of two) with few shuffles: lanes that
// pair up keep half of the values each, so 4 values take 6 shuffles, not 20.
// Lane 32 i / K returns the sum of value i.
template <int K>
__device__ __forceinline__ float warp_sums(float (&v)[K]) {
  int n = K;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool hi = threadIdx.x & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float keep = hi ? v[i + n] : v[i], send = hi ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return v[0];
}

// Row group `sub` of the CTA: its threads, its ring (stages of R rows) and its
// barrier, and the sums over a row.
template <int V, int R>
struct BnGroup {
  int wpr, sub, warp, t, tpr;          // warps per row, group, warp of the group, thread of the group, threads
  int n;                               // vectors of a row that this thread owns
  int row_bytes[4], off[4], bytes_per_row, stage_bytes, stages;
  uint8_t *ring;
  uint32_t ring_addr, bars;
  float *red;                          // [2][wpr][8]
  int buf, st_get, st_put, ph;         // stage to read and its phase, stage to fill
  bool issues;                         // this thread issues a copy per batch: see plan_copies
  int copy_row, copy_bytes, copy_off;
  const uint8_t *copy_src;
  int64_t copy_step;
  volatile int *abort;
  uint32_t limit;

  // bytes[k]: of a row of the k-th tensor of the ring, 0 for none.
  __device__ __forceinline__ void init(const BlockNormArgs &a, const int (&bytes)[4], uint8_t *smem, uint64_t *mbars,
                                       float *reds, volatile int *ab) {
    wpr = a.wpr;
    sub = (threadIdx.x >> 5) / wpr;
    warp = (threadIdx.x >> 5) - sub * wpr;
    tpr = wpr * 32;
    t = threadIdx.x - sub * tpr;
    n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) n += column(v) < a.C ? 1 : 0;
    bytes_per_row = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      row_bytes[k] = bytes[k];
      off[k] = bytes_per_row * R;
      bytes_per_row += bytes[k];
    }
    stage_bytes = bytes_per_row * R;
    stages = a.stages;
    ring = smem + (size_t)sub * stages * stage_bytes;
    ring_addr = smem_u32(ring);
    bars = smem_u32(mbars + sub * stages);
    red = reds + sub * 2 * wpr * 8;
    buf = st_get = st_put = ph = 0;
    abort = ab;
    limit = a.wait_limit;
    if (t == 0) {
      for (int i = 0; i < stages; ++i) tc::mbar_init(bars + 8u * i, 4 * R);      // one arrival per copy
      tc::fence_barrier_init();
    }
    if (threadIdx.x == 0) *abort = 0;
    __syncthreads();
  }
  __device__ __forceinline__ int column(int v) const { return (warp * V + v) * 256 + (threadIdx.x & 31) * 8; }
  // All threads of the group: what they did before is visible after.
  __device__ __forceinline__ void sync() const {
    if (wpr == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(tpr) : "memory");
  }
  // Which copies of a batch this thread issues: copy c is tensor c % 4 of row c / 4,
  // warp c % wpr's lane c / wpr has it (issuing takes a thread some 200 cycles; eight
  // copies by one thread held the others up at the next barrier for 1900 of 9000
  // cycles).  src: the first row of each tensor, step: bytes from a row to the next.
  __device__ __forceinline__ void plan_copies(const uint8_t *s0, const uint8_t *s1, const uint8_t *s2, const uint8_t *s3,
                                              int64_t d0, int64_t d1, int64_t d2, int64_t d3) {
    const int c = warp + wpr * (threadIdx.x & 31), k = c & 3;
    issues = c < 4 * R;
    copy_row = c >> 2;
    const int64_t d = k == 0 ? d0 : k == 1 ? d1 : k == 2 ? d2 : d3;
    copy_bytes = k == 0 ? row_bytes[0] : k == 1 ? row_bytes[1] : k == 2 ? row_bytes[2] : row_bytes[3];
    copy_off = (k == 0 ? off[0] : k == 1 ? off[1] : k == 2 ? off[2] : off[3]) + copy_row * copy_bytes;
    copy_src = (k == 0 ? s0 : k == 1 ? s1 : k == 2 ? s2 : s3) + copy_row * d;
    copy_step = R * d;
  }
  // The next batch, of `rows` rows, into the next stage; called by the whole group.
  __device__ __forceinline__ void fetch(int rows) {
    const uint32_t bar = bars + 8u * st_put;
    if (issues) {
      if (copy_row < rows && copy_bytes) {
        tc::mbar_expect_tx(bar, copy_bytes);
        tc::bulk_load(ring_addr + st_put * stage_bytes + copy_off, copy_src, copy_bytes, bar);
      } else {
        tc::mbar_arrive(bar);
      }
      copy_src += copy_step;
    }
    __syncwarp();
    if (++st_put == stages) st_put = 0;
  }
  // The next stage.  A wait that runs out latches PRISM_ETIMEOUT; the group goes on
  // (with whatever the ring holds), so that every barrier still sees all threads.
  __device__ __forceinline__ const uint8_t *next() {
    const int st = st_get;
    tc::mbar_wait(bars + 8u * st, (uint32_t)ph, abort, limit);
    if (++st_get == stages) st_get = 0, ph ^= 1;
    return ring + st * stage_bytes;
  }
  // After a wait ran out: the copies still in flight land before the CTA exits.
  __device__ __forceinline__ void drain(int batches) const {
    if (t != 0 || !*abort) return;
    volatile int no_abort = 0;
    for (int it = max(0, batches - stages); it < batches; ++it)
      tc::mbar_wait(bars + 8u * (it % stages), (uint32_t)(it / stages) & 1u, &no_abort, limit);
  }
  // This thread's elements of row i of tensor k of a stage, zeros past the end.
  template <typename T>
  __device__ __forceinline__ void read(const uint8_t *stage, int k, int i, float2 (&f)[V][4]) const {
    const T *p = reinterpret_cast<const T *>(stage + off[k] + i * row_bytes[k]) + column(0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v < n) {
        BnVec8<T>::load(p + v * 256, f[v]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[v][e] = both(0.f);
      }
    }
  }
  __device__ __forceinline__ float total(const float2 (&x)[V][4]) const {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += sum8(x[v]);
    return s;
  }
  __device__ __forceinline__ float squares(const float2 (&x)[V][4]) const {
    float2 q = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) q = dot8(x[v], x[v], q);
    return q.x + q.y;
  }
  // x - m where this thread owns columns (0 stays 0 past the end).
  __device__ __forceinline__ void subtract(float2 (&x)[V][4], float m) const {
#pragma unroll
    for (int v = 0; v < V; ++v) shift8(x[v], v < n ? m : 0.f);
  }
  // Sums of K values over the group, the same on every thread, in a fixed order: a
  // butterfly in each warp, then the warps in order.  The table has two halves
  // used in turn, so one barrier per exchange is enough.
  template <int K>
  __device__ __forceinline__ void sums(float (&v)[K]) {
    const int lane = threadIdx.x & 31;
    const float x = warp_sums(v);
    if (wpr == 1) {
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] = __shfl_sync(0xffffffffu, x, i * (32 / K));
      return;
    }
    float *h = red + buf * wpr * 8;
    buf ^= 1;
    if (lane % (32 / K) == 0) h[warp * 8 + lane / (32 / K)] = x;
    sync();
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = 0.f;
    for (int w = 0; w < wpr; ++w, h += 8) {
#pragma unroll
      for (int i = 0; i < K; i += 2) {
        const float2 y = *reinterpret_cast<const float2 *>(h + i);
        v[i] += y.x;
        v[i + 1] += y.y;
      }
    }
  }
};

// Rows per batch: registers hold R rows of values beside the column sums.
constexpr int bn_bwd_rows(int V) { return V == 1 ? 2 : 1; }

// kThreads: the most threads it is launched with (fewer leave it more registers).
template <typename TX, typename TY, int V, int kThreads>
__global__ void __launch_bounds__(kThreads) block_norm_bwd_kernel(const BlockNormArgs a) {
  constexpr int R = bn_bwd_rows(V);
  extern __shared__ __align__(16) uint8_t bn_smem[];
  __shared__ uint64_t mbars[kBnMaxGroups * kBnMaxStages];
  __shared__ __align__(16) float red[2 * (kBnMaxThreads / 32) * 8];
  __shared__ int ab;
  int b, r0, r1;
  after_previous();
  if (!bn_rows(a, b, r0, r1)) return;

  const TX *xo = static_cast<const TX *>(a.x_out), *dxo = static_cast<const TX *>(a.dx_out);
  const TY *y = static_cast<const TY *>(a.y), *dh = static_cast<const TY *>(a.dh);
  TX *dx = static_cast<TX *>(a.dx);
  TY *dy = static_cast<TY *>(a.dy);
  BnGroup<V, R> g;
  const int rx = a.C * (int)sizeof(TX), ry = a.C * (int)sizeof(TY);
  const int bytes[4] = {dh ? rx : 0, dh ? ry : 0, dxo ? rx : 0, y ? ry : 0};
  float *const params = reinterpret_cast<float *>(bn_smem);      // V = 2: [A | G][C]
  g.init(a, bytes, bn_smem + (V == 2 ? 8 * a.C : 0), mbars, red, &ab);
  // the group's rows are consecutive
  const int per = (r1 - r0 + a.groups - 1) / a.groups;
  const int first = r0 + g.sub * per, rows = max(0, min(per, r1 - first)), batches = (rows + R - 1) / R;
  g.plan_copies(reinterpret_cast<const uint8_t *>(xo + first * a.sxo), reinterpret_cast<const uint8_t *>(dh + first * a.sdh),
                reinterpret_cast<const uint8_t *>(dxo + first * a.sdxo), reinterpret_cast<const uint8_t *>(y + first * a.sy),
                a.sxo * (int64_t)sizeof(TX), a.sdh * (int64_t)sizeof(TY), a.sdxo * (int64_t)sizeof(TX),
                a.sy * (int64_t)sizeof(TY));
  for (int it = 0; it < min(batches, a.stages); ++it) g.fetch(min(R, rows - it * R));
  float2 A1[4], G1[4];      // V = 1
#pragma unroll
  for (int e = 0; e < 4; ++e) A1[e] = G1[e] = both(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v < g.n) {
      float2 A[4], B[4], G[4];
      fold_params(a, b, g.column(v), A, B, G);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (V == 1) {
          A1[e] = A[e];
          G1[e] = G[e];
        } else {            // a thread reads only what it wrote
          *reinterpret_cast<float2 *>(params + g.column(v) + 2 * e) = A[e];
          *reinterpret_cast<float2 *>(params + a.C + g.column(v) + 2 * e) = G[e];
        }
      }
    }
  auto parameter = [&](int which, int v, float2 (&p)[4]) {
    if constexpr (V == 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = which ? G1[e] : A1[e];
    } else {
      BnVec8<float>::load(params + which * a.C + g.column(v), p);
    }
  };
  const float inv_c = 1.f / (float)a.C;
  const bool cx = dh && a.pre == PRISM_NORM_LAYER, cy = y && a.post == PRISM_NORM_LAYER;
  const bool py = y && a.post != PRISM_NORM_NONE;
  const float al = y ? a.alpha : 1.f;
  float2 p1[V][4], p2[V][4], p3[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) p1[v][e] = p2[v][e] = p3[v][e] = both(0.f);
  dx += first * a.sdx + g.column(0);
  if (y) dy += first * a.sdy + g.column(0);

  for (int it = 0; it < batches; ++it) {
    const uint8_t *stage = g.next();
    const int m = min(R, rows - it * R);     // rows of this batch; what is computed of others is not used
    float2 u[R][V][4], f[R][V][4];           // x_out - mean, then dr; y - mean, then yhat
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (y) g.template read<TY>(stage, 3, i, f[i]);
      if (dh) g.template read<TX>(stage, 0, i, u[i]);
    }
    if (cx || cy) {
      float s[2 * R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        s[2 * i] = cx ? g.total(u[i]) : 0.f;
        s[2 * i + 1] = cy ? g.total(f[i]) : 0.f;
      }
      g.sums(s);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (cx) g.subtract(u[i], s[2 * i] * inv_c);
        if (cy) g.subtract(f[i], s[2 * i + 1] * inv_c);
      }
    }
    float rs[R], c1[R], c2[R], rsy[R];
    if (dh || py) {
      float s[4 * R];       // squares of x_out - mean, of y - mean; sum(d), sum(d u)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        s[4 * i] = s[4 * i + 2] = s[4 * i + 3] = 0.f;
        s[4 * i + 1] = py ? g.squares(f[i]) : 0.f;
        if (dh) {
          s[4 * i] = g.squares(u[i]);
          float2 d8[V][4], sd = both(0.f), sdu = both(0.f);
          g.template read<TY>(stage, 1, i, d8);
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (V == 1 || v < g.n) {
              float2 A[4];
              parameter(0, v, A);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                d8[v][e] = tc::mul2(d8[v][e], A[e]);
                sd = add2(d8[v][e], sd);
              }
              sdu = dot8(d8[v], u[i][v], sdu);
            }
          s[4 * i + 2] = sd.x + sd.y;
          s[4 * i + 3] = sdu.x + sdu.y;
        }
      }
      g.sums(s);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        rs[i] = rsqrtf(s[4 * i] * inv_c + a.eps);
        rsy[i] = py ? rsqrtf(s[4 * i + 1] * inv_c + a.eps) : 1.f;
        c1[i] = cx ? s[4 * i + 2] * inv_c : 0.f;
        c2[i] = s[4 * i + 3] * rs[i] * inv_c;        // mean(d xhat)
        if (py) {
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[i][v][e] = tc::mul2(f[i][v][e], both(rsy[i]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) rs[i] = c1[i] = c2[i] = 0.f, rsy[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < m) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v < g.n) {
            float2 o[4];
            if (dxo) {
              BnVec8<TX>::load(reinterpret_cast<const TX *>(stage + g.off[2] + i * g.row_bytes[2]) + g.column(v), o);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = both(0.f);
            }
            if (dh) {
              float2 A[4], d8[4];
              parameter(0, v, A);
              BnVec8<TY>::load(reinterpret_cast<const TY *>(stage + g.off[1] + i * g.row_bytes[1]) + g.column(v), d8);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 xh = tc::mul2(u[i][v][e], both(rs[i]));
                const float2 in = tc::fma2(xh, both(-c2[i]), tc::fma2(d8[e], A[e], both(-c1[i])));
                o[e] = tc::fma2(both(rs[i]), in, o[e]);
                p1[v][e] = tc::fma2(d8[e], xh, p1[v][e]);
                p2[v][e] = add2(d8[e], p2[v][e]);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              u[i][v][e] = o[e];
              o[e] = tc::mul2(o[e], both(al));
            }
            BnVec8<TX>::store(dx + v * 256, o);
          }
        dx += a.sdx;
      }
    float s[2 * R];        // sum(e), sum(e yhat)
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) s[i] = 0.f;
    if (py) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v < g.n) {
            float2 G[4];
            parameter(1, v, G);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 de = tc::mul2(u[i][v][e], G[e]);
              s0 = add2(de, s0);
              s1 = tc::fma2(de, f[i][v][e], s1);
            }
          }
        s[2 * i] = s0.x + s0.y;
        s[2 * i + 1] = s1.x + s1.y;
      }
      g.sums(s);
    }
    if (!py || g.wpr == 1) g.sync();
    // every thread of the group has read the stage: its next rows may land there
    if (it + a.stages < batches) g.fetch(min(R, rows - (it + a.stages) * R));
    if (y) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < m) {
          const float m1 = cy ? s[2 * i] * inv_c : 0.f, m2 = s[2 * i + 1] * inv_c;
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (v < g.n) {
              float2 o[4], G[4];
              parameter(1, v, G);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                p3[v][e] = tc::fma2(u[i][v][e], f[i][v][e], p3[v][e]);
                const float2 de = tc::fma2(u[i][v][e], G[e], both(-m1));
                o[e] = tc::mul2(tc::fma2(f[i][v][e], both(-m2), de), both(rsy[i]));
              }
              BnVec8<TY>::store(dy + v * 256, o);
            }
          dy += a.sdy;
        }
    }
  }
  g.drain(batches);
  if (a.need) {
    float *out = a.part + ((int64_t)blockIdx.x * a.groups + g.sub) * 3 * a.C;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v < g.n) {
        float *o = out + g.column(v);
        if (a.need & 1) BnVec8<float>::store(o, p1[v]);
        if (a.need & 2) BnVec8<float>::store(o + a.C, p2[v]);
        if (a.need & 4) BnVec8<float>::store(o + 2 * a.C, p3[v]);
      }
  }
}

// Parameter gradients from the column sums, one CTA per 32 columns and
//   blockIdx.y = 0       what is summed over all sequences: the weights, and gate,
//                        scale and shift where the sequences share them
//   blockIdx.y = 1 + b   gate, scale and shift of sequence b
// The warps' sums are added in order: the additions have a fixed order.
struct BnParamArgs {
  Offsets seq;
  int C, unit, groups, param_f32, need;
  const float *part;         // [slots * groups][3][C]
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

constexpr int kBnParamWarps = 16;
__global__ void __launch_bounds__(kBnParamWarps * 32) block_norm_params_kernel(const BnParamArgs a) {
  after_previous();
  __shared__ float sh[kBnParamWarps][5][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const bool in = c < a.C;
  const bool all = blockIdx.y == 0;
  const int b0 = all ? 0 : (int)blockIdx.y - 1, b1 = all ? a.seq.seqs : (int)blockIdx.y;
  // few sequences have many runs of rows each, which the warps share out; many
  // have few, and a warp takes a sequence
  const int over = b1 - b0 > kBnParamWarps ? kBnParamWarps : 1, each = kBnParamWarps / over;
  // plain sums of the three kinds, and the sums that the weights' gradients take
  float s[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
  for (int b = b0 + w / each; b < b1; b += over) {
    int begin, len;
    if (!in || !sequence_rows(a.seq, b, begin, len)) continue;
    const float ws = all && a.dweight && a.scale ? 1.f + param_at(a.scale, b * a.sscale + c, a.param_f32) : 1.f;
    const float wg = all && a.dpost_weight && a.gate ? param_at(a.gate, b * a.sgate + c, a.param_f32) : 1.f;
    const float *p = a.part + ((int64_t)begin / a.unit + b) * a.groups * 3 * a.C + c;
    const int64_t n = (int64_t)run_count(len, a.unit) * a.groups;
    const bool k0 = a.need & 1, k1 = a.need & 2, k2 = a.need & 4;
    float t[3] = {0.f, 0.f, 0.f};
#pragma unroll 4
    for (int64_t i = w % each; i < n; i += each) {
      const float *q = p + i * 3 * a.C;
      if (k0) t[0] += q[0];
      if (k1) t[1] += q[a.C];
      if (k2) t[2] += q[2 * (int64_t)a.C];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += t[k];
    s[3] = fmaf(ws, t[0], s[3]);
    s[4] = fmaf(wg, t[2], s[4]);
  }
#pragma unroll
  for (int k = 0; k < 5; ++k) sh[w][k][lane] = s[k];
  __syncthreads();
  if (w >= 5 || !in) return;
  float v = 0.f;
  for (int i = 0; i < kBnParamWarps; ++i) v += sh[i][w][lane];
  const int64_t at = all ? c : (int64_t)b0 * a.C + c;
  if (w == 0 && a.dscale && (a.per_scale != 0) != all)
    put_param(a.dscale, at, a.weight ? v * param_at(a.weight, c, a.param_f32) : v, a.param_f32);
  if (w == 1 && a.dshift && (a.per_shift != 0) != all) put_param(a.dshift, at, v, a.param_f32);
  if (w == 2 && a.dgate && (a.per_gate != 0) != all)
    put_param(a.dgate, at, a.post_weight ? v * param_at(a.post_weight, c, a.param_f32) : v, a.param_f32);
  if (w == 3 && all && a.dweight) put_param(a.dweight, c, v, a.param_f32);
  if (w == 4 && all && a.dpost_weight) put_param(a.dpost_weight, c, v, a.param_f32);
}

}  // namespace prism
