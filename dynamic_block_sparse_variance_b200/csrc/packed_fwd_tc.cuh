// Dense attention forward over packed sequences on the tcgen05 tensor cores.
//
// One CTA per (128 or 256 flattened query rows, kv head, share of the keys); with
// 256, two 128-row tiles A and B share every key/value tile.
//   S = Q K^T (tensor memory), running maximum m and sum l per row,
//   P = 2^(scale log2e S - m), O += P V (P as bf16 from tensor memory over S).
// Warps: 0 TMA producer, 1 MMA issuer and tensor-memory owner, 2-5 and 6-9
// softmax of tile A and B, one thread per row (its tensor-memory lane).
//
// K and V come in through TMA tiles of a 3-D map (head_dim, head, row), Q likewise
// where the group's size divides 128 (boxes of 128 / group tokens of the group's
// heads), otherwise through cp.async, row by row.  A key tile that reaches past its sequence's
// keys holds other rows: their scores are replaced by -inf before they are
// used, and their values by zeros in shared memory (0 x NaN would not be 0).
//
// What bounds it is a tile's chain, not one unit: of about 4000 cycles per pair of
// 128 x 128 tiles the products take 2048 and the special-function unit's
// exponentials 2048, and with S, P and O of two tiles in all 512 columns of tensor
// memory the next S of a tile waits for its P V.  Measured (8 heads of 128, 16384
// causal rows, bursts): 484 us, 1136 TFLOP/s, 0.69 of the bf16 rate measured with a
// library product; under the power cap of a long run 560 us.  Slower, each against
// the form of its time: eight softmax warps per tile (527 against 512 us), three of
// eight exponentials as polynomials on the FMA pipe (598 against 512: the products
// themselves then run at 70% of their rate), 208 registers for the softmax warps,
// which then spill nothing (497 against 490), and a whole warp that walks the issuer's
// loop in uniform registers (479 against 474).
//
// With few rows the keys are split over blockIdx.z; a share writes its O in
// fp32 and its log2-sum-exp, and packed_combine_kernel joins them.
#pragma once

#include "packed_attn.cuh"
#include "tc_common.cuh"

namespace prism {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(have ? 16 : 0));
}

// One arrival for a whole warp, after what all of its lanes did (their tensor-memory
// stores have been waited for and fenced).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

// A [128][D] bf16 tile of 128-byte-swizzled atoms of 64 columns.
template <int D>
struct Tile {
  static constexpr int kBytes = 128 * D * 2;
  static constexpr int kAtom = 128 * 128;       // bytes of one 64-column atom
  static constexpr int kAtoms = D / 64;
  // byte offset of 16-byte piece ch (8 columns) of row r
  __device__ __forceinline__ static uint32_t off(int r, int ch) {
    return (uint32_t)(ch >> 3) * kAtom + (uint32_t)r * 128u + (uint32_t)(((ch & 7) ^ (r & 7)) << 4);
  }
  // operand offset of the k-th 16-column step of a K-major operand
  __device__ __forceinline__ static uint32_t kstep(int k) { return (uint32_t)(k >> 2) * kAtom + (uint32_t)(k & 3) * 32u; }
  __device__ __forceinline__ static void load(uint32_t dst, const CUtensorMap *map, int head, int row, uint32_t bar) {
#pragma unroll
    for (int c = 0; c < kAtoms; ++c) tma_load_3d(dst + c * kAtom, map, 64 * c, head, row, bar);
  }
  // Zeroes rows [from, 128); called by a whole warp.
  __device__ __forceinline__ static void zero_rows(uint8_t *tile, int from) {
    const int lane = threadIdx.x & 31;
    for (int i = from * 8 + lane; i < 128 * 8; i += 32) {
#pragma unroll
      for (int c = 0; c < kAtoms; ++c) *reinterpret_cast<uint4 *>(tile + c * kAtom + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

// Loads `rows` flattened query rows of a kv head (rows from r0 of a sequence whose first
// row is q0) into a tile, zeros behind them; `threads` threads, this one being `t`.
// A thread keeps one 16-byte piece of every (threads / (D / 8))-th row and steps from
// row to row by additions: row r is token r / group, head r % group.
template <int D>
__device__ __forceinline__ void load_rows_async(uint32_t tile, const __nv_bfloat16 *x, const int64_t (&stride)[2], int q0,
                                                int head0, int group, int r0, int rows, int tile_rows, int t, int threads) {
  constexpr int CH = D / 8;
  const int step = threads / CH, dt = step / group, dg = step - dt * group;
  const int ch = t % CH;
  int r = t / CH, tok = (r0 + r) / group, g = r0 + r - tok * group;
  const __nv_bfloat16 *const base = x + (int64_t)q0 * stride[0] + (int64_t)head0 * stride[1] + ch * 8;
  for (; r < tile_rows; r += step) {
    const bool have = r < rows;
    cp_async16_or_zero(tile + (uint32_t)(r >> 7) * Tile<D>::kBytes + Tile<D>::off(r & 127, ch),
                       have ? base + tok * stride[0] + g * stride[1] : base, have);
    tok += dt;
    g += dg;
    if (g >= group) {
      g -= group;
      ++tok;
    }
  }
}

// A warp's 32 rows of COLS bf16, which it has put into rows [row0, row0 + 32) of a tile
// of D columns in shared memory, from 16-byte piece ch0 on, to their places in global
// memory, whole rows at a time (straight from the registers, a row per lane, every
// store would touch 32 rows).  dst: where this lane's row goes, nullptr for none.
template <int D, int COLS = D>
__device__ __forceinline__ void flush_rows(const uint8_t *tile, int row0, __nv_bfloat16 *dst, int ch0 = 0) {
  constexpr int CH = COLS / 8;
  const int lane = threadIdx.x & 31, ch = lane % CH;
  __syncwarp();
#pragma unroll 4
  for (int i = 0; i < CH; ++i) {      // 32 / CH rows at a time
    const int r = i * (32 / CH) + lane / CH;
    __nv_bfloat16 *const p = reinterpret_cast<__nv_bfloat16 *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
    const uint4 w = *reinterpret_cast<const uint4 *>(tile + Tile<D>::off(row0 + r, ch0 + ch));
    if (p) *reinterpret_cast<uint4 *>(p + ch * 8) = w;
  }
  __syncwarp();
}

// The two probabilities of a packed pair as they enter the product.
__device__ __forceinline__ float2 rounded_pair(uint32_t w) { return tc::f2(bf16_lo(w), bf16_hi(w)); }

struct PackedSplit {
  int splits;
  float *o;     // [split][q_rows][heads][D]
  float *lse2;  // [split][heads][q_rows]
};

// NG query tiles of 128 rows: 2, which share each key/value tile, one CTA per SM;
// or 1, two CTAs per SM, whose fixed costs (Q, the first tiles, the epilogue)
// overlap each other's work.
template <int D, int NG>
struct PfCfg {
  static constexpr int kStages = (D == 128 ? 1 : 2) * NG;
  static constexpr int kThreads = 64 + 128 * NG;
  static constexpr int kSmem = Tile<D>::kBytes * (NG + 2 * kStages) + 512 + 1024;
};

template <int D, int NG>
__global__ void __launch_bounds__(64 + 128 * NG, 3 - NG)
    packed_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const PackedArgs a, const PackedSplit sp, const uint32_t limit) {
  using T = Tile<D>;
  constexpr int kStages = PfCfg<D, NG>::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *sgen = smem_raw + (sbase - smem_u32(smem_raw));
  auto sQ = [&](int g) { return sbase + (uint32_t)g * T::kBytes; };
  auto sK = [&](int s) { return sbase + (uint32_t)(NG + 2 * s) * T::kBytes; };
  auto sV = [&](int s) { return sbase + (uint32_t)(NG + 1 + 2 * s) * T::kBytes; };
  const uint32_t sBar = sbase + (uint32_t)(NG + 2 * kStages) * T::kBytes;
  auto b_kfull = [&](int s) { return sBar + 8u * s; };
  auto b_vfull = [&](int s) { return sBar + 8u * (4 + s); };
  auto b_kempty = [&](int s) { return sBar + 8u * (8 + s); };
  auto b_vempty = [&](int s) { return sBar + 8u * (12 + s); };
  auto b_sfull = [&](int g) { return sBar + 8u * (16 + g); };
  auto b_pfull = [&](int g) { return sBar + 8u * (18 + g); };
  const uint32_t b_edge = sBar + 8u * 20;    // the edge tile of V landed
  const uint32_t b_drain = sBar + 8u * 21;
  const uint32_t b_q = sBar + 8u * 22;       // Q is in shared memory (the copy, or an arrival per softmax warp)
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sgen + (sBar - sbase) + 8 * 24);
  volatile int *abort = reinterpret_cast<volatile int *>(sgen + (sBar - sbase) + 8 * 24 + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool q_copy = 128 % a.group == 0;
  const auto setup = [&] {
    if (threadIdx.x == 64) {
      tc::prefetch_tmap(&tmQ);
      tc::prefetch_tmap(&tmK);
      tc::prefetch_tmap(&tmV);
    }
    if (threadIdx.x == 0) {
      for (int i = 0; i < kStages; ++i) {
        tc::mbar_init(b_kfull(i), 1);
        tc::mbar_init(b_vfull(i), 1);
        tc::mbar_init(b_kempty(i), 1);
        tc::mbar_init(b_vempty(i), 1);
      }
      for (int g = 0; g < NG; ++g) {
        tc::mbar_init(b_sfull(g), 1);
        tc::mbar_init(b_pfull(g), 4);      // one arrival per warp
      }
      tc::mbar_init(b_edge, 1);
      tc::mbar_init(b_drain, 1);
      tc::mbar_init(b_q, q_copy ? 1 : 4 * NG);
      *abort = 0;
      tc::fence_barrier_init();
    }
    if (warp == 1) {
      tc::tmem_alloc(smem_u32(tmem_slot), 256 * NG);
      tc::tmem_relinquish();
    }
  };
  // Barriers and tensor memory take about as long as the loads by which the CTA finds
  // its rows; with single tiles, whose walks are short, they come first (7680 queries
  // of 12 heads of 64 over 1111 keys in 4 sequences: 31.3 -> 29.9 us; pairs: 3% slower).
  constexpr bool kEarly = NG == 1;
  if constexpr (kEarly) setup();
  const auto leave = [&] {      // without work (all threads): the tensor memory goes back
    if constexpr (kEarly) {
      tc::tc_fence_before();
      __syncthreads();
      tc::tc_fence_after();
      if (warp == 1) tc::tmem_dealloc(*tmem_slot, 256 * NG);
    }
  };
  after_previous();
  // later tiles of a causal sequence see more keys: they start first
  const int slots = (int)(gridDim.x / a.kv_heads);
  const int kvh = (int)(blockIdx.x % a.kv_heads), slot = slots - 1 - (int)(blockIdx.x / a.kv_heads);
  PackedSeq::check(a, slot);
  int64_t piece;
  const int b = find_sequence(a.qs, slot, a.group, 128 * NG, piece);
  PackedSeq s;
  if (!s.load(a, b)) return leave();
  const int64_t nrows = (int64_t)s.lq * a.group;
  if (piece < 0 || piece * (128 * NG) >= nrows) return leave();
  const int r0 = (int)(piece * (128 * NG));            // first flattened row
  const int rows = (int)min((int64_t)(128 * NG), nrows - r0);
  // key tiles [t0, t1[g]) of tile g
  int t0, t1[NG];
  {
    int top[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int last = min(rows, 128 * (g + 1)) - 1;    // tile g's last row
      top[g] = last >= 128 * g ? (s.visible(a, (r0 + last) / a.group) + 127) >> 7 : 0;
    }
    const int all = max(top[0], top[NG - 1]);
    t0 = (int)((int64_t)all * blockIdx.z / sp.splits);
    const int te = (int)((int64_t)all * (blockIdx.z + 1) / sp.splits);
#pragma unroll
    for (int g = 0; g < NG; ++g) t1[g] = max(t0, min(te, top[g]));
  }
  const int tend = max(t1[0], t1[NG - 1]);
  if constexpr (!kEarly) setup();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int g) { return tmem + 256u * (uint32_t)g; };
  auto tO = [&](int g) { return tmem + 256u * (uint32_t)g + 128u; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && q_copy && t0 < tend) {
      // rows behind the sequence's last one are whatever lies there: no other row's
      // result depends on them, and theirs are not stored
      tc::mbar_expect_tx(b_q, NG * T::kBytes);
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int c = 0; c < T::kAtoms; ++c)
          tma_load_3d(sQ(g) + c * T::kAtom, &tmQ, 64 * c, kvh * a.group, s.q0 + (r0 + 128 * g) / a.group, b_q);
    }
    int nk = 0, nv = 0, edge = 0;
    bool ok = true;
    for (int t = t0; t < tend; ++t) {
      const int st = nk % kStages;
      const uint32_t ph = (uint32_t)(nk / kStages) & 1u;
      if (!__all_sync(0xffffffffu, tc::mbar_wait(b_kempty(st), ph ^ 1u, abort, limit))) break;
      if (lane == 0) {
        tc::mbar_expect_tx(b_kfull(st), T::kBytes);
        T::load(sK(st), &tmK, kvh, s.k0 + 128 * t, b_kfull(st));
      }
      ++nk;
      if (!__all_sync(0xffffffffu, tc::mbar_wait(b_vempty(st), ph ^ 1u, abort, limit))) break;
      const int valid = s.lk - 128 * t;
      const uint32_t bar = valid < 128 ? b_edge : b_vfull(st);
      if (lane == 0) {
        tc::mbar_expect_tx(bar, T::kBytes);
        T::load(sV(st), &tmV, kvh, s.k0 + 128 * t, bar);
      }
      if (valid < 128) {   // the sequence's last tile
        edge = 1;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(b_edge, 0, abort, limit));
        if (!ok) break;
        T::zero_rows(sgen + (sV(st) - sbase), valid);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(b_vfull(st));
      } else {
        ++nv;
      }
    }
    // Every copy lands before the CTA exits.  At most one fill per stage is
    // outstanding, so each parity wait is unambiguous; the edge tile took the
    // stage of the oldest V fill, which had been read by then.
    if (lane == 0) {
      volatile int no_abort = 0;
      for (int k = max(0, nk - kStages); k < nk; ++k)
        tc::mbar_wait(b_kfull(k % kStages), (uint32_t)(k / kStages) & 1u, &no_abort, limit);
      for (int k = max(0, nv - kStages + edge); k < nv; ++k)
        tc::mbar_wait(b_vfull(k % kStages), (uint32_t)(k / kStages) & 1u, &no_abort, limit);
      if (edge) tc::mbar_wait(b_edge, 0, &no_abort, limit);
      if (q_copy && t0 < tend) tc::mbar_wait(b_q, 0, &no_abort, limit);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t idO = tc::idesc_bf16(128, D, false, true);
      const int n_all = tend - t0, n_g[2] = {t1[0] - t0, t1[NG - 1] - t0};
      const uint64_t dQ[2] = {tc::sw128_desc(sQ(0), 16, 1024), tc::sw128_desc(sQ(NG - 1), 16, 1024)};
      const uint64_t dK0 = tc::sw128_desc(sK(0), 16, 1024), dV0 = tc::sw128_desc(sV(0), T::kAtom, 1024);
      auto issue_s = [&](int n, int g) {
        const uint64_t dK = dK0 + (uint64_t)((uint32_t)(n % kStages) * (2u * T::kBytes >> 4)), dQg = dQ[g];
        const uint32_t tSg = tS(g);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tSg, tc::desc_adv(dQg, T::kstep(k)), tc::desc_adv(dK, T::kstep(k)), idS, k > 0);
        tc::mma_commit(b_sfull(g));
      };
      auto issue_pv = [&](int n, int g) {
        const uint64_t dV = dV0 + (uint64_t)((uint32_t)(n % kStages) * (2u * T::kBytes >> 4));
        const uint32_t tOg = tO(g), tPg = tS(g);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc::mma_ts(tOg, tPg + 8u * k, tc::desc_adv(dV, 2048u * k), idO, (n > 0 || k > 0) ? 1u : 0u);
      };
      auto wait_full = [&](uint32_t bar, int n) {
        const bool r = tc::mbar_wait(bar, (uint32_t)(n / kStages) & 1u, abort, limit);
        tc::tc_fence_after();
        return r;
      };
      // S of step 0, then per step PV_A S_A(+1) PV_B S_B(+1): one tile's softmax
      // runs while the other tile's products execute
      bool ok = n_all == 0 || (tc::mbar_wait(b_q, 0, abort, limit) && wait_full(b_kfull(0), 0));
      if (ok && n_all > 0) {
        for (int g = 0; g < NG; ++g)
          if (n_g[g] > 0) issue_s(0, g);
        tc::mma_commit(b_kempty(0));
      }
      for (int n = 0; ok && n < n_all; ++n) {
        const int st = n % kStages;
        const bool more = n + 1 < n_all;
        bool have_k = false;
        if (!wait_full(b_vfull(st), n)) break;
        for (int g = 0; g < NG && ok; ++g) {
          if (n < n_g[g]) {
            if (!tc::mbar_wait(b_pfull(g), (uint32_t)n & 1u, abort, limit)) { ok = false; break; }
            tc::tc_fence_after();
            issue_pv(n, g);
          }
          if (g == NG - 1) tc::mma_commit(b_vempty(st));
          if (n + 1 < n_g[g]) {
            if (!have_k && !wait_full(b_kfull((n + 1) % kStages), n + 1)) { ok = false; break; }
            have_k = true;
            issue_s(n + 1, g);
          }
          if (g == NG - 1 && more) tc::mma_commit(b_kempty((n + 1) % kStages));
        }
      }
      tc::mma_commit(b_drain);
      volatile int no_abort = 0;
      tc::mbar_wait(b_drain, 0, &no_abort, limit);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int g = (warp - 2) >> 2;
    const int q = warp & 3;                      // tensor-memory lane quadrant
    const int row = 128 * g + 32 * q + lane;     // of the CTA's rows
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const bool have = row < rows;
    const int fr = r0 + row, tok = have ? fr / a.group : 0;
    const int vis = have ? s.visible(a, tok) : 0;
    const float sl2 = a.scale_log2;
    // Q while the first tiles of K and V are on their way
    if (t0 < tend && !q_copy)
      load_rows_async<D>(sQ(0), a.q, a.sq, s.q0, kvh * a.group, a.group, r0, rows, 128 * NG, (int)threadIdx.x - 64, 128 * NG);
    if (!q_copy) {
      cp_async_commit();
      cp_async_wait<0>();
      fence_async_smem();
      warp_arrive(b_q);
    }
    float m_run = -INFINITY, l_run = 0.f, n_run = 0.f;
    bool ok = true;
    const int steps = t1[g] - t0;
    for (int n = 0; n < steps; ++n) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(b_sfull(g), (uint32_t)n & 1u, abort, limit))) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      uint32_t raw[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS(g) + lane_off + 32u * c, raw[c]);
      tc::tmem_ld_wait();
      const int seen = vis - 128 * (t0 + n);       // keys of this tile that the row sees
      if (__any_sync(0xffffffffu, seen < 128)) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e >= seen) raw[c][e] = __float_as_uint(-INFINITY);
      }
      float m8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) m8[e] = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e) m8[e & 7] = fmaxf(m8[e & 7], __uint_as_float(raw[c][e]));
      float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
      mx *= sl2;
      // the maximum moves only when it grew by more than 2^8 (P stays far below
      // the range of bf16 and fp32), so most steps leave O alone
      const bool grow = mx > m_run + 8.f;
      float alpha = 1.f;
      if (grow) {
        alpha = tc::ex2(m_run - mx);
        l_run *= alpha;
        n_run *= alpha;
        m_run = mx;
      }
      const float mm = m_run == -INFINITY ? 0.f : m_run;   // a row that has seen nothing: 2^(-inf - 0) = 0
      float2 r2[2], n2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) r2[e] = n2[e] = tc::f2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = tc::fma2(tc::f2u(raw[c][2 * e], raw[c][2 * e + 1]), tc::f2(sl2, sl2), tc::f2(-mm, -mm));
          const float2 p = tc::f2(tc::ex2(x.x), tc::ex2(x.y));
          // P enters the product as bf16 (V's type: both operands of one product
          // have one type).  l, of which LSE is made, sums it in fp32 before that
          // rounding; what divides O sums it after: O is then an average of the
          // values whatever the rounding did (with l it would carry their common
          // part times the rounding's sum, and D = rowsum(dO o O) with it)
          pk[e] = pack_bf16(p.x, p.y);
          r2[e & 1] = tc::fma2(p, tc::f2(1.f, 1.f), r2[e & 1]);
          n2[e & 1] = tc::fma2(rounded_pair(pk[e]), tc::f2(1.f, 1.f), n2[e & 1]);
        }
        tc::tmem_st16(tS(g) + lane_off + 16u * c, pk);
      }
      if (n > 0 && __any_sync(0xffffffffu, grow)) {
        // rare: S_g(n) was issued after PV_g(n-1), so O has settled; PV_g(n) waits for
        // this step's P
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tc::tmem_ld32(tO(g) + lane_off + 32u * c, ov);
          tc::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          tc::tmem_st32(tO(g) + lane_off + 32u * c, ov);
        }
      }
      l_run += (r2[0].x + r2[0].y) + (r2[1].x + r2[1].y);
      n_run += (n2[0].x + n2[0].y) + (n2[1].x + n2[1].y);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      if (!(a.debug_stall && n == 0)) warp_arrive(b_pfull(g));
    }
    // epilogue
    if (__all_sync(0xffffffffu, ok && !*abort)) {
      if (steps > 0) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(b_drain, 0, abort, limit))) ok = false;
        tc::tc_fence_after();
      } else if (t0 < tend) {
        // no key for this tile, some for the other: Q comes in for both, and the zeros
        // below go into its place
        if (!__all_sync(0xffffffffu, tc::mbar_wait(b_q, 0, abort, limit))) ok = false;
      }
      if (ok) {
        const float inv = n_run == 0.f ? 0.f : 1.f / n_run;      // 0: saw no key; NaN stays NaN
        const int head = kvh * a.group + fr - tok * a.group;
        const int64_t grow_ = s.q0 + tok;
        const auto load_o = [&](int c, uint32_t (&v)[32]) {
          if (steps > 0) {
            tc::tmem_ld32(tO(g) + lane_off + 32u * c, v);
            tc::tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
        };
        if (sp.splits > 1) {
          float *const prow = sp.o + (((int64_t)blockIdx.z * a.qs.rows + grow_) * a.heads + head) * D;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            load_o(c, ov);
            if (have) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4 *>(prow + 32 * c + e) =
                    make_float4(__uint_as_float(ov[e]) * inv, __uint_as_float(ov[e + 1]) * inv,
                                __uint_as_float(ov[e + 2]) * inv, __uint_as_float(ov[e + 3]) * inv);
            }
            __syncwarp();
          }
        } else {
          // every product that reads this tile of Q is done: its memory takes the rows of
          // O, then those of its rounding residual
          uint8_t *const tile = sgen + (sQ(g) - sbase);
          for (int pass = 0; pass < (a.o_res ? 2 : 1); ++pass) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              load_o(c, ov);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint4 w;
                uint32_t *const wp = &w.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float x0 = __uint_as_float(ov[8 * j + 2 * e]) * inv, x1 = __uint_as_float(ov[8 * j + 2 * e + 1]) * inv;
                  const uint32_t u = pack_bf16(x0, x1);
                  wp[e] = pass ? pack_bf16(x0 - bf16_lo(u), x1 - bf16_hi(u)) : u;
                }
                *reinterpret_cast<uint4 *>(tile + T::off(32 * q + lane, 4 * c + j)) = w;
              }
            }
            __nv_bfloat16 *const dst = pass ? a.o_res + (grow_ * a.heads + head) * D : a.o + grow_ * a.so[0] + head * a.so[1];
            flush_rows<D>(tile, 32 * q, have ? dst : nullptr);
          }
        }
        if (have) {
          const float l2 = l_run == 0.f ? -INFINITY : m_run + log2f(l_run);
          if (sp.splits > 1) sp.lse2[((int64_t)blockIdx.z * a.heads + head) * a.qs.rows + grow_] = l2;
          else a.lse[(int64_t)head * a.qs.rows + grow_] = l2 * kLn2;
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 256 * NG);
  }
}

// Joins the shares of split keys: O = sum_s 2^(L_s - L) O_s with L = log2 sum_s 2^(L_s).
// D / 4 threads per (row, head), shares summed in order.  A share that saw no key of the row
// has L_s = -inf and O_s = 0, one with a NaN has both NaN, and so has the row.
template <int D>
__global__ void __launch_bounds__(256) packed_combine_kernel(const PackedArgs a, const PackedSplit sp) {
  constexpr int kLanes = D / 4;
  after_previous();
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kLanes;   // row * heads + head
  const int sub = threadIdx.x % kLanes;
  if (i >= (int64_t)a.qs.rows * a.heads) return;
  const int64_t row = i / a.heads;
  const int h = (int)(i - row * a.heads);
  // rows outside the sequences were not written by any share
  const int64_t first = a.qs.at(0), last = a.qs.at(a.qs.seqs);
  if (row < first || row >= last) return;
  const float *L = sp.lse2 + (int64_t)h * a.qs.rows + row;
  const int64_t ls = (int64_t)a.heads * a.qs.rows;
  float m = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < sp.splits; ++s) m = fmaxf(m, L[s * ls]);
  if (m == -INFINITY) m = 0.f;                    // no share saw a number: weights of 0 or NaN
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < sp.splits; ++s) {
    const float w = exp2f(L[s * ls] - m);
    const float4 p = *reinterpret_cast<const float4 *>(sp.o + (s * (int64_t)a.qs.rows * a.heads + i) * D + sub * 4);
    l += w;
    o.x = fmaf(w, p.x, o.x); o.y = fmaf(w, p.y, o.y); o.z = fmaf(w, p.z, o.z); o.w = fmaf(w, p.w, o.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  const uint2 u = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  *reinterpret_cast<uint2 *>(a.o + row * a.so[0] + h * a.so[1] + sub * 4) = u;
  if (a.o_res)
    *reinterpret_cast<uint2 *>(a.o_res + i * D + sub * 4) =
        make_uint2(pack_bf16(x[0] - bf16_lo(u.x), x[1] - bf16_hi(u.x)), pack_bf16(x[2] - bf16_lo(u.y), x[3] - bf16_hi(u.y)));
  if (sub == 0) a.lse[(int64_t)h * a.qs.rows + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace prism
