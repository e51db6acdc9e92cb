// Dense attention backward over packed sequences on the tcgen05 tensor cores:
//   P = 2^(scale log2e S - LSE log2e),  dP = dO V^T,  dS = P (dP - D),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Two kinds of CTA, neither of which shares a sum with another, so results do
// not depend on their order:
//   keys     128 keys of one kv head; walks the query tiles that see them (the
//            heads of the group are rows of the same tiles) and keeps dK and dV
//            in tensor memory:  S^T = K Q^T, dP^T = V dO^T, dV += P^T dO,
//            dK += dS^T Q with P^T and dS^T as operands from tensor memory
//   queries  128 flattened query rows; walks their key tiles and keeps dQ:
//            S = Q K^T, dP = dO V^T, dQ += dS K
// That is 7 products for the algorithm's 5 and the exponentials twice.  The
// other way, one kind that adds its part of dQ to an fp32 array with atomics,
// saves two products but writes 64 KB of reductions per tile pair and gives dQ
// whose last bits change from run to run.
//
// Measured (8192 tokens, 8 heads of 128, all pairs, bursts): 882 us, 779 TFLOP/s of
// the algorithm's 5 products, 1091 of the 7, 0.66 of the bf16 rate measured with a
// library product; 172 us at 7 packed causal sequences of 6144 tokens in all, 16 / 4
// heads.  What bounds it is a tile's chain again (S, P, its product, dP, dS, its
// product, in all 512 columns of tensor memory), and the operands that the products
// read from shared memory (S and dP both of theirs, 64 KB per 128 x 128 x 128).
//
// P and dS enter their products rounded once to bf16, the type of dO, Q and K
// (a product's operands have one type); everything else is fp32.  A row of dS sums
// to zero, so dQ has nothing of what the keys have in common; a row of rounded dS
// does not, and dQ would take its sum times that common part, which in keys with a
// bias is many times the rest (13 times, 1024 causal tokens: dQ off by 2.7% of its norm,
// where 0.24% is what the roundings explain).  The queries kind therefore sums each row of the dS that enter
// the product and takes the sum times the keys' common part (common_key) away at the
// end: right for any vector in its place, since the true sum is zero.  It is not where
// o and lse belong to a softmax over more keys than this call's (shares of the keys
// joined by their LSE): such a row is known by its P, which do not sum to one, and
// keeps its sum.  (The sums cost the two cases above 25 and 8 us.)
//
// Warps of either kind: 0 TMA producer, 1 MMA issuer and tensor-memory owner,
// 2-9 elementwise, a row of the tile per thread (its tensor-memory lane), warps
// 2-5 for columns [0, 64) and 6-9 for [64, 128).  A thread writes its 16-bit
// operand over the first 32 of its own 64 columns, so k-step k (16 rows of the
// sum) sits at column 8k + (k >= 4 ? 32 : 0).
#pragma once

#include "packed_fwd_tc.cuh"

namespace prism {

constexpr int kPbThreads = 320;
// Two resident tiles, three stages of one streamed tensor, two of the other,
// two floats per row for two stages, barriers.  The window has no slack for
// alignment: the kernel checks that it starts on 1024 bytes.
template <int D>
constexpr int kPbSmem = Tile<D>::kBytes * 7 + 2 * 1024 + 256;
static_assert(kPbSmem<128> <= 232448, "backward shared memory");

__device__ __forceinline__ uint32_t operand_col(int k) { return 8u * (uint32_t)k + (k >= 4 ? 32u : 0u); }

// Waits of a whole warp: all lanes go on or none does.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t limit) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort, limit));
}

// dS = P (dP - D) over 64 columns of dP starting at `src`, packed to bf16 at `dst`
// in chunks of 16 columns; chunk c + 1 is loaded while chunk c is computed.
// delta(j): D of column j (a multiple of 4) .. j + 3.  kSum: sum, the rounded dS are
// added to it.
template <bool kSum, typename F>
__device__ __forceinline__ void form_ds(uint32_t src, uint32_t dst, const uint32_t (&p)[64], F delta, float2 &sum) {
  uint32_t a[16], b[16];
  tc::tmem_ld16(src, a);
  tc::tmem_ld_wait_regs(a);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t(&cur)[16] = (c & 1) ? b : a;
    uint32_t(&nxt)[16] = (c & 1) ? a : b;
    if (c < 3) tc::tmem_ld16(src + 16u * (c + 1), nxt);
    uint32_t w[8];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int j = 16 * c + 4 * g;
      const float4 d = delta(j);
      const float2 x = tc::mul2(tc::f2u(p[j], p[j + 1]), tc::sub2(tc::f2u(cur[4 * g], cur[4 * g + 1]), tc::f2(d.x, d.y)));
      const float2 y = tc::mul2(tc::f2u(p[j + 2], p[j + 3]), tc::sub2(tc::f2u(cur[4 * g + 2], cur[4 * g + 3]), tc::f2(d.z, d.w)));
      w[2 * g] = pack_bf16(x.x, x.y);
      w[2 * g + 1] = pack_bf16(y.x, y.y);
      if constexpr (kSum) {
        sum = tc::fma2(rounded_pair(w[2 * g]), tc::f2(1.f, 1.f), sum);
        sum = tc::fma2(rounded_pair(w[2 * g + 1]), tc::f2(1.f, 1.f), sum);
      }
    }
    if (c < 3) tc::tmem_ld_wait_regs(nxt);
    tc::tmem_st8(dst + 8u * c, w);   // dst may be src: columns below 16 (c + 1) have been read
  }
}

// COLS columns of an accumulator row (zeros where `zero`), times `mul`, as bf16 into row
// `row` of a tile in shared memory, from piece ch0 on.  kLess: less `sum` times the vector
// `common` (of these columns).
template <int D, int COLS, bool kLess = false>
__device__ __forceinline__ void put_row(uint32_t taddr, bool zero, float mul, uint8_t *tile, int row, int ch0,
                                        float sum = 0.f, const float *common = nullptr) {
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) {
    uint32_t v[32];
    tc::tmem_ld32(taddr + 32u * c, v);
    tc::tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 w;
      uint32_t *const wp = &w.x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 x = tc::f2u(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
        if constexpr (kLess) x = tc::fma2(tc::f2(-sum, -sum), *reinterpret_cast<const float2 *>(common + 32 * c + 8 * j + 2 * e), x);
        wp[e] = zero ? 0u : pack_bf16(x.x * mul, x.y * mul);
      }
      *reinterpret_cast<uint4 *>(tile + Tile<D>::off(row, ch0 + 4 * c + j)) = w;
    }
  }
}

// COLS columns of an accumulator row in fp32 to the layout of PackedParts, zeros where not `keep`; out: the
// row's place for the first of the columns.
template <int COLS>
__device__ __forceinline__ void store_part(uint32_t taddr, bool keep, float *out) {
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) {
    uint32_t v[32];
    tc::tmem_ld32(taddr + 32u * c, v);
    tc::tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      *reinterpret_cast<uint4 *>(out + (8 * c + e / 4) * 512) =
          keep ? make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// The query tiles (of tt tokens) that see keys from key0 on, and how they are cut.
// A keys CTA walks 4 products per tile, 2 us, and with grouped heads or few CTAs the
// longest walk can take longer than all the rest: `splits` CTAs share it, each writes
// its dK and dV in fp32, and packed_sum_kernel adds them in order.  A share has at
// least 6 tiles, so short walks stay whole and are written at once.
struct KeyWalk {
  int tt, behind, first, steps, chunk, shares;
  __device__ __forceinline__ KeyWalk(const PackedArgs &a, const PackedSeq &s, int key0, int splits) {
    tt = 128 / a.group;
    behind = a.causal ? s.lk - s.lq : 0x40000000;     // token t sees key j iff t >= j - behind
    const int ntile = (s.lq + tt - 1) / tt;
    first = key0 < s.lk ? min(ntile, max(0, key0 - behind) / tt) : ntile;
    steps = ntile - first;
    chunk = max(6, (steps + splits - 1) / splits);
    shares = max(1, (steps + chunk - 1) / chunk);
  }
};
struct PackedParts {
  int splits;
  int64_t tiles;      // key tiles times kv heads
  float *dk, *dv;     // [split][tile][D / 4][128 rows][4]: a warp's 32 rows of 4 columns are consecutive
};

// The kind that keeps dK and dV; `block`: its number among the CTAs of its kind.
template <int D>
__device__ __forceinline__ void packed_keys_cta(const CUtensorMap &tmQ, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                                const CUtensorMap &tmO, const PackedArgs &a, const PackedParts &parts,
                                                const uint32_t limit, int block) {
  using T = Tile<D>;
  extern __shared__ __align__(1024) uint8_t sgen[];
  const uint32_t sbase = smem_u32(sgen);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) set_status(PRISM_EBOUNDS);
    return;
  }
  const uint32_t sK = sbase, sV = sbase + T::kBytes;
  auto sQ = [&](int i) { return sbase + (uint32_t)(2 + i) * T::kBytes; };
  auto sO = [&](int i) { return sbase + (uint32_t)(5 + i) * T::kBytes; };
  auto stat = [&](int i) { return reinterpret_cast<float *>(sgen + 7 * T::kBytes + 1024 * i); };   // [lse2 | D][128]
  const uint32_t sBar = sbase + 7 * T::kBytes + 2 * 1024;
  auto b_qfull = [&](int i) { return sBar + 8u * i; };
  auto b_qempty = [&](int i) { return sBar + 8u * (3 + i); };
  auto b_ofull = [&](int i) { return sBar + 8u * (6 + i); };
  auto b_oempty = [&](int i) { return sBar + 8u * (8 + i); };
  const uint32_t b_kv = sBar + 8u * 10;
  const uint32_t b_s = sBar + 8u * 11;      // S^T_n done
  const uint32_t b_dp = sBar + 8u * 12;     // dP^T_n done
  const uint32_t b_p = sBar + 8u * 13;      // P^T_n written
  const uint32_t b_ds = sBar + 8u * 14;     // dS^T_n written
  const uint32_t b_qedge = sBar + 8u * 15;  // the last tile of Q, of dO landed
  const uint32_t b_oedge = sBar + 8u * 16;
  const uint32_t b_drain = sBar + 8u * 17;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sgen + (sBar - sbase) + 8 * 20);
  volatile int *abort = reinterpret_cast<volatile int *>(sgen + (sBar - sbase) + 8 * 20 + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int share = block % parts.splits, kvh = block / parts.splits % a.kv_heads, slot = block / parts.splits / a.kv_heads;
  if (a.qs.rows == 0) PackedSeq::check(a, slot);      // there is no other kind to look
  int64_t piece;
  const int b = find_sequence(a.ks, slot, 1, 128, piece);
  PackedSeq s;
  if (!s.load(a, b)) return;
  if (piece < 0 || piece * 128 >= s.room) return;
  const int key0 = (int)piece * 128;
  const KeyWalk walk(a, s, key0, parts.splits);
  if (share >= walk.shares) return;
  const int tt = walk.tt, behind = walk.behind;
  const int first = walk.first + share * walk.chunk, nsteps = min(walk.chunk, walk.steps - share * walk.chunk);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(b_qfull(i), 33);     // the copy, and each producer lane's rows of LSE and D
      tc::mbar_init(b_qempty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(b_ofull(i), 1);
      tc::mbar_init(b_oempty(i), 1);
    }
    tc::mbar_init(b_kv, 1);
    tc::mbar_init(b_s, 1);
    tc::mbar_init(b_dp, 1);
    tc::mbar_init(b_p, 8);           // one arrival per elementwise warp
    tc::mbar_init(b_ds, 8);
    tc::mbar_init(b_qedge, 1);
    tc::mbar_init(b_oedge, 1);
    tc::mbar_init(b_drain, 1);
    *abort = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  if (tt * a.group < 128 && warp >= 2 && warp < 7) {   // rows of the streamed tiles that no copy fills
    T::zero_rows(sgen + (2 + warp - 2) * T::kBytes, tt * a.group);
    fence_async_smem();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tdK = tmem, tdV = tmem + 128, tS = tmem + 256, tDP = tmem + 384;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int nq = 0, no = 0, qedge = 0, oedge = 0;
    const int tile_bytes = tt * a.group * D * 2;
    auto fetch = [&](uint32_t dst, const CUtensorMap *map, int tok, uint32_t bar) {
      tc::mbar_expect_tx(bar, tile_bytes);
#pragma unroll
      for (int c = 0; c < T::kAtoms; ++c) tma_load_3d(dst + c * T::kAtom, map, 64 * c, kvh * a.group, s.q0 + tok, bar);
    };
    if (lane == 0 && nsteps > 0) {
      tc::mbar_expect_tx(b_kv, 2 * T::kBytes);
      T::load(sK, &tmK, kvh, s.k0 + key0, b_kv);
      T::load(sV, &tmV, kvh, s.k0 + key0, b_kv);
    }
    const float *glse = a.lse2 + (int64_t)kvh * a.qs.rows * a.group, *gd = a.delta + (int64_t)kvh * a.qs.rows * a.group;
    for (int n = 0; n < nsteps; ++n) {
      const int tok = (first + n) * tt;
      const int valid = min(tt, s.lq - tok) * a.group;     // rows of the tile
      const bool last = s.lq - tok < tt;
      const int qi = n % 3, oi = n & 1;
      // both copies first: what follows (rows of LSE and D, the last tile's zeros) waits
      // for more
      if (!warp_wait(b_qempty(qi), ((uint32_t)(n / 3) & 1u) ^ 1u, abort, limit)) break;
      if (lane == 0) fetch(sQ(qi), &tmQ, tok, last ? b_qedge : b_qfull(qi));
      (last ? qedge : nq) += 1;
      if (!warp_wait(b_oempty(oi), ((uint32_t)(n >> 1) & 1u) ^ 1u, abort, limit)) break;
      if (lane == 0) fetch(sO(oi), &tmO, tok, last ? b_oedge : b_ofull(oi));
      (last ? oedge : no) += 1;
      {
        const int64_t r = (int64_t)(s.q0 + tok) * a.group;
        float L[4], Dr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = lane + 32 * i;
          L[i] = c < valid ? glse[r + c] : INFINITY;       // rows without a query: P = 0
          Dr[i] = c < valid ? gd[r + c] : 0.f;
        }
        // dK_{n-2} follows the last use of that tile's rows of LSE and D
        if (n >= 2 && !warp_wait(b_qempty((n - 2) % 3), (uint32_t)((n - 2) / 3) & 1u, abort, limit)) break;
        float *st = stat(n & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st[lane + 32 * i] = L[i];
          st[128 + lane + 32 * i] = Dr[i];
        }
      }
      if (last) {
        if (!warp_wait(b_qedge, 0, abort, limit)) break;
        T::zero_rows(sgen + (sQ(qi) - sbase), valid);
        if (!warp_wait(b_oedge, 0, abort, limit)) break;
        T::zero_rows(sgen + (sO(oi) - sbase), valid);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(b_qfull(qi));
          tc::mbar_arrive(b_ofull(oi));
        }
      }
      tc::mbar_arrive(b_qfull(qi));
    }
    // Every copy lands before the CTA exits (the last tile took the stage of the
    // oldest fill, which had been read; each remaining parity is unambiguous).
    if (lane == 0 && nsteps > 0) {
      volatile int no_abort = 0;
      tc::mbar_wait(b_kv, 0, &no_abort, limit);
      for (int k = max(0, nq - 3 + qedge); k < nq; ++k)
        tc::mbar_wait(b_qfull(k % 3), (uint32_t)(k / 3) & 1u, &no_abort, limit);
      for (int k = max(0, no - 2 + oedge); k < no; ++k)
        tc::mbar_wait(b_ofull(k & 1), (uint32_t)(k >> 1) & 1u, &no_abort, limit);
      if (qedge) tc::mbar_wait(b_qedge, 0, &no_abort, limit);
      if (oedge) tc::mbar_wait(b_oedge, 0, &no_abort, limit);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t idG = tc::idesc_bf16(128, D, false, true);
      const uint64_t dK = tc::sw128_desc(sK, 16, 1024), dV = tc::sw128_desc(sV, 16, 1024);
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool r = tc::mbar_wait(bar, parity, abort, limit);
        tc::tc_fence_after();
        return r;
      };
      auto rows_by_rows = [&](uint32_t d, uint64_t x, uint32_t saddr, uint32_t bar) {   // d = x y^T, both K-major
        const uint64_t y = tc::sw128_desc(saddr, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(d, tc::desc_adv(x, T::kstep(k)), tc::desc_adv(y, T::kstep(k)), idS, k > 0);
        tc::mma_commit(bar);
      };
      auto accumulate = [&](uint32_t d, uint32_t x, uint32_t saddr, bool begun) {       // d += x y
        const uint64_t y = tc::sw128_desc(saddr, T::kAtom, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc::mma_ts(d, x + operand_col(k), tc::desc_adv(y, 2048u * k), idG, (begun || k > 0) ? 1u : 0u);
      };
      bool ok = nsteps > 0 && wait(b_kv, 0) && wait(b_qfull(0), 0);
      if (ok) {
        rows_by_rows(tS, dK, sQ(0), b_s);
        ok = wait(b_ofull(0), 0);
        if (ok) rows_by_rows(tDP, dV, sO(0), b_dp);
      }
      for (int n = 0; ok && n < nsteps; ++n) {
        const int m = n + 1;
        const bool more = m < nsteps;
        // the copies were asked for long ago: seeing here that they landed keeps it off the
        // way from P and dS to their products
        if (more && !(wait(b_qfull(m % 3), (uint32_t)(m / 3) & 1u) && wait(b_ofull(m & 1), (uint32_t)(m >> 1) & 1u))) break;
        if (!wait(b_p, (uint32_t)n & 1u)) break;
        accumulate(tdV, tS, sO(n & 1), n > 0);
        tc::mma_commit(b_oempty(n & 1));
        if (more) rows_by_rows(tS, dK, sQ(m % 3), b_s);
        if (!wait(b_ds, (uint32_t)n & 1u)) break;
        accumulate(tdK, tDP, sQ(n % 3), n > 0);
        tc::mma_commit(b_qempty(n % 3));
        if (more) rows_by_rows(tDP, dV, sO(m & 1), b_dp);
      }
      tc::mma_commit(b_drain);
      volatile int no_abort = 0;
      tc::mbar_wait(b_drain, 0, &no_abort, limit);
    }
  } else {
    // ------------------------------------------------------------ elementwise
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int row = 32 * q + lane;
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const uint32_t colS = tS + lane_off + 64u * half, colDP = tDP + lane_off + 64u * half;
    const float cS = a.scale_log2;
    // the tile's rows from (j - behind - token) group on see key j
    const int64_t from0 = (int64_t)(key0 + row - behind) * a.group - 64 * half;
    bool ok = true;
    for (int n = 0; n < nsteps; ++n) {
      const int qi = n % 3;
      if (!warp_wait(b_qfull(qi), (uint32_t)(n / 3) & 1u, abort, limit) || !warp_wait(b_s, (uint32_t)n & 1u, abort, limit)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const float4 *st = reinterpret_cast<const float4 *>(stat(n & 1)) + 16 * half;
      uint32_t p[64];
      {
        uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(p);
        uint32_t(&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(p + 32);
        tc::tmem_ld32(colS, lo);
        tc::tmem_ld32(colS + 32u, hi);
        tc::tmem_ld_wait();
      }
      // first column of this half that sees the key
      const int from = (int)max((int64_t)0, min((int64_t)64, from0 - (int64_t)(first + n) * tt * a.group));
      const bool mask = __any_sync(0xffffffffu, from > 0);
#pragma unroll
      for (int j = 0; j < 64; j += 4) {
        const float4 L = st[j / 4];
        float2 x = tc::fma2(tc::f2u(p[j], p[j + 1]), tc::f2(cS, cS), tc::f2(-L.x, -L.y));
        float2 y = tc::fma2(tc::f2u(p[j + 2], p[j + 3]), tc::f2(cS, cS), tc::f2(-L.z, -L.w));
        if (mask) {
          if (j + 0 < from) x.x = -INFINITY;
          if (j + 1 < from) x.y = -INFINITY;
          if (j + 2 < from) y.x = -INFINITY;
          if (j + 3 < from) y.y = -INFINITY;
        }
        p[j] = __float_as_uint(tc::ex2(x.x));
        p[j + 1] = __float_as_uint(tc::ex2(x.y));
        p[j + 2] = __float_as_uint(tc::ex2(y.x));
        p[j + 3] = __float_as_uint(tc::ex2(y.y));
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack_bf16(__uint_as_float(p[32 * c + 2 * e]), __uint_as_float(p[32 * c + 2 * e + 1]));
        tc::tmem_st16(colS + 16u * c, w);
      }
      tc::tmem_st_wait();
      tc::tc_fence_before();
      if (!(a.debug_stall && n == 0)) warp_arrive(b_p);
      if (!warp_wait(b_dp, (uint32_t)n & 1u, abort, limit)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      float2 none = tc::f2(0.f, 0.f);
      form_ds<false>(colDP, colDP, p, [&](int j) { return st[32 + j / 4]; }, none);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      warp_arrive(b_ds);
    }
    if (__all_sync(0xffffffffu, ok && !*abort)) {
      if (nsteps > 0) ok = warp_wait(b_drain, 0, abort, limit);
      if (ok) {
        tc::tc_fence_after();
        const int key = key0 + row;
        const bool have = key < s.room;
        const bool zero = nsteps == 0;
        const bool keep = key < s.lk;                 // rows with room but not in use: zero
        const int64_t r = s.k0 + key;
        constexpr int kCols = D / 2;                  // of each half's warps
        const uint32_t co = lane_off + (uint32_t)(half * kCols);
        if (walk.shares > 1) {
          const int64_t at = (((int64_t)share * parts.tiles + slot * a.kv_heads + kvh) * (D / 4) + half * (kCols / 4)) * 512 + row * 4;
          store_part<kCols>(tdK + co, keep, parts.dk + at);
          store_part<kCols>(tdV + co, keep, parts.dv + at);
        } else {
          // every product that reads K and V is done: their memory takes the rows (zeros
          // for rows with room but not in use, whatever their accumulators hold)
          uint8_t *const tk = sgen + (sK - sbase), *const tv = sgen + (sV - sbase);
          const int ch0 = half * (kCols / 8);
          put_row<D, kCols>(tdK + co, zero || !keep, a.scale, tk, row, ch0);
          put_row<D, kCols>(tdV + co, zero || !keep, 1.f, tv, row, ch0);
          flush_rows<D, kCols>(tk, 32 * q, have ? a.dk + r * a.sdk[0] + kvh * a.sdk[1] + half * kCols : nullptr, ch0);
          flush_rows<D, kCols>(tv, 32 * q, have ? a.dv + r * a.sdv[0] + kvh * a.sdv[1] + half * kCols : nullptr, ch0);
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// A barrier of the eight elementwise warps.
__device__ __forceinline__ void elementwise_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// What the first n keys of a sequence (kv head's keys at `k`) have in common, into the first
// D floats of `room`, 2 KB of shared memory, by the elementwise warps (t: 0 .. 255): the
// mean of 64 keys spread evenly over them, in the columns where it is beyond four of its
// standard errors, and zero in the others, whose mean is chance and would only add to dQ's
// error.  The partial sums pass through bf16: any vector will do, as long as every row of
// the tile takes the same.
template <int D>
__device__ __forceinline__ void common_key(const __nv_bfloat16 *k, int64_t row_stride, int n, uint8_t *room, int t) {
  constexpr int kPairs = D / 2, kParts = 256 / kPairs, kKeys = 64;
  uint32_t *const part = reinterpret_cast<uint32_t *>(room);      // [sums | squares][kParts][kPairs]
  const int col = t % kPairs, first = t / kPairs;
  float2 m = tc::f2(0.f, 0.f), q = tc::f2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kKeys / kParts; ++i) {
    const int64_t key = (int64_t)(2 * (first + i * kParts) + 1) * n / (2 * kKeys);      // < n
    const float2 x = rounded_pair(*reinterpret_cast<const uint32_t *>(k + key * row_stride + 2 * col));
    m = tc::fma2(x, tc::f2(1.f / kKeys, 1.f / kKeys), m);
    q = tc::fma2(tc::mul2(x, tc::f2(1.f / kKeys, 1.f / kKeys)), x, q);
  }
  part[t] = pack_bf16(m.x, m.y);
  part[256 + t] = pack_bf16(q.x, q.y);
  elementwise_sync();
  m = q = tc::f2(0.f, 0.f);
  if (t < kPairs)
    for (int i = 0; i < kParts; ++i) {
      m = tc::fma2(rounded_pair(part[i * kPairs + t]), tc::f2(1.f, 1.f), m);
      q = tc::fma2(rounded_pair(part[256 + i * kPairs + t]), tc::f2(1.f, 1.f), q);
    }
  elementwise_sync();
  const float least = 16.f / (float)min(n, kKeys);      // mean^2 > 16 variance / keys
  if (t < kPairs)
    reinterpret_cast<float2 *>(room)[t] = tc::f2(m.x * m.x > least * (q.x - m.x * m.x) ? m.x : 0.f,
                                                 m.y * m.y > least * (q.y - m.y * m.y) ? m.y : 0.f);
}

// The kind that keeps dQ, `block` of `blocks`.
template <int D>
__device__ __forceinline__ void packed_queries_cta(const CUtensorMap &tmQ, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                                   const CUtensorMap &tmO, const PackedArgs &a,
                                                   const uint32_t limit, int block, int blocks) {
  using T = Tile<D>;
  extern __shared__ __align__(1024) uint8_t sgen[];
  const uint32_t sbase = smem_u32(sgen);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) set_status(PRISM_EBOUNDS);
    return;
  }
  const uint32_t sQ = sbase, sO = sbase + T::kBytes;
  auto sK = [&](int i) { return sbase + (uint32_t)(2 + i) * T::kBytes; };
  auto sV = [&](int i) { return sbase + (uint32_t)(5 + i) * T::kBytes; };
  const uint32_t sBar = sbase + 7 * T::kBytes + 2 * 1024;
  auto b_kfull = [&](int i) { return sBar + 8u * i; };
  auto b_kempty = [&](int i) { return sBar + 8u * (3 + i); };
  auto b_vfull = [&](int i) { return sBar + 8u * (6 + i); };
  auto b_vempty = [&](int i) { return sBar + 8u * (8 + i); };
  auto b_s = [&](int i) { return sBar + 8u * (10 + i); };     // S_n done
  const uint32_t b_dp = sBar + 8u * 12;     // dP_n done
  const uint32_t b_ds = sBar + 8u * 13;     // dS_n written
  const uint32_t b_kedge = sBar + 8u * 14;  // the last tile of K, of V landed
  const uint32_t b_vedge = sBar + 8u * 15;
  const uint32_t b_drain = sBar + 8u * 16;
  const uint32_t b_qo = sBar + 8u * 17;     // Q and dO landed (the copies, or an arrival per elementwise warp)
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sgen + (sBar - sbase) + 8 * 20);
  volatile int *abort = reinterpret_cast<volatile int *>(sgen + (sBar - sbase) + 8 * 20 + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = block % a.kv_heads, slot = blocks / a.kv_heads - 1 - block / a.kv_heads;   // long ones first
  PackedSeq::check(a, slot);
  int64_t piece;
  const int b = find_sequence(a.qs, slot, a.group, 128, piece);
  PackedSeq s;
  if (!s.load(a, b)) return;
  const int64_t nrows = (int64_t)s.lq * a.group;
  if (piece < 0 || piece * 128 >= nrows) return;
  const int r0 = (int)(piece * 128);
  const int rows = (int)min((int64_t)128, nrows - r0);
  const int keys = s.visible(a, (r0 + rows - 1) / a.group), nsteps = (keys + 127) >> 7;
  const bool q_copy = 128 % a.group == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(b_kfull(i), 1);
      tc::mbar_init(b_kempty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(b_vfull(i), 1);
      tc::mbar_init(b_vempty(i), 1);
      tc::mbar_init(b_s(i), 1);
    }
    tc::mbar_init(b_dp, 1);
    tc::mbar_init(b_ds, 8);
    tc::mbar_init(b_kedge, 1);
    tc::mbar_init(b_vedge, 1);
    tc::mbar_init(b_drain, 1);
    tc::mbar_init(b_qo, q_copy ? 1 : 8);
    *abort = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int i) { return tmem + 128u * (uint32_t)i; };
  const uint32_t tDP = tmem + 256, tdQ = tmem + 384;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && q_copy && nsteps > 0) {
      // (rows behind the sequence's last one: as in the forward)
      tc::mbar_expect_tx(b_qo, 2 * T::kBytes);
#pragma unroll
      for (int c = 0; c < T::kAtoms; ++c) {
        tma_load_3d(sQ + c * T::kAtom, &tmQ, 64 * c, kvh * a.group, s.q0 + r0 / a.group, b_qo);
        tma_load_3d(sO + c * T::kAtom, &tmO, 64 * c, kvh * a.group, s.q0 + r0 / a.group, b_qo);
      }
    }
    int nk = 0, nv = 0, kedge = 0, vedge = 0;
    for (int n = 0; n < nsteps; ++n) {
      const int valid = s.lk - 128 * n, ki = n % 3, vi = n & 1;
      const bool last = valid < 128;
      if (!warp_wait(b_kempty(ki), ((uint32_t)(n / 3) & 1u) ^ 1u, abort, limit)) break;
      if (lane == 0) {
        const uint32_t bar = last ? b_kedge : b_kfull(ki);
        tc::mbar_expect_tx(bar, T::kBytes);
        T::load(sK(ki), &tmK, kvh, s.k0 + 128 * n, bar);
      }
      if (last) {   // other rows' keys would meet dS = 0 in the product for dQ: they must be numbers
        kedge = 1;
        if (!warp_wait(b_kedge, 0, abort, limit)) break;
        T::zero_rows(sgen + (sK(ki) - sbase), valid);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(b_kfull(ki));
      } else {
        ++nk;
      }
      if (!warp_wait(b_vempty(vi), ((uint32_t)(n >> 1) & 1u) ^ 1u, abort, limit)) break;
      if (lane == 0) {
        const uint32_t bar = last ? b_vedge : b_vfull(vi);
        tc::mbar_expect_tx(bar, T::kBytes);
        T::load(sV(vi), &tmV, kvh, s.k0 + 128 * n, bar);
      }
      if (last) {
        vedge = 1;
        if (!warp_wait(b_vedge, 0, abort, limit)) break;
        T::zero_rows(sgen + (sV(vi) - sbase), valid);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(b_vfull(vi));
      } else {
        ++nv;
      }
    }
    if (lane == 0) {
      volatile int no_abort = 0;
      for (int k = max(0, nk - 3 + kedge); k < nk; ++k)
        tc::mbar_wait(b_kfull(k % 3), (uint32_t)(k / 3) & 1u, &no_abort, limit);
      for (int k = max(0, nv - 2 + vedge); k < nv; ++k)
        tc::mbar_wait(b_vfull(k & 1), (uint32_t)(k >> 1) & 1u, &no_abort, limit);
      if (kedge) tc::mbar_wait(b_kedge, 0, &no_abort, limit);
      if (vedge) tc::mbar_wait(b_vedge, 0, &no_abort, limit);
      if (q_copy && nsteps > 0) tc::mbar_wait(b_qo, 0, &no_abort, limit);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && nsteps > 0) {
      constexpr uint32_t idS = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t idG = tc::idesc_bf16(128, D, false, true);
      const uint64_t dQ = tc::sw128_desc(sQ, 16, 1024), dO = tc::sw128_desc(sO, 16, 1024);
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool r = tc::mbar_wait(bar, parity, abort, limit);
        tc::tc_fence_after();
        return r;
      };
      auto rows_by_rows = [&](uint32_t d, uint64_t x, uint32_t saddr, uint32_t bar) {
        const uint64_t y = tc::sw128_desc(saddr, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(d, tc::desc_adv(x, T::kstep(k)), tc::desc_adv(y, T::kstep(k)), idS, k > 0);
        tc::mma_commit(bar);
      };
      auto scores = [&](int n) {
        if (!wait(b_kfull(n % 3), (uint32_t)(n / 3) & 1u)) return false;
        rows_by_rows(tS(n & 1), dQ, sK(n % 3), b_s(n & 1));
        return true;
      };
      auto landed_v = [&](int n) { return wait(b_vfull(n & 1), (uint32_t)(n >> 1) & 1u); };
      auto dprob = [&](int n) {
        rows_by_rows(tDP, dO, sV(n & 1), b_dp);
        tc::mma_commit(b_vempty(n & 1));
      };
      bool ok = wait(b_qo, 0) && scores(0) && landed_v(0);
      if (ok) {
        dprob(0);
        ok = nsteps < 2 || scores(1);
      }
      for (int n = 0; ok && n < nsteps; ++n) {
        if (n + 1 < nsteps && !landed_v(n + 1)) break;
        if (!wait(b_ds, (uint32_t)n & 1u)) break;
        if (n + 1 < nsteps) dprob(n + 1);
        const uint64_t y = tc::sw128_desc(sK(n % 3), T::kAtom, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc::mma_ts(tdQ, tS(n & 1) + operand_col(k), tc::desc_adv(y, 2048u * k), idG, (n > 0 || k > 0) ? 1u : 0u);
        tc::mma_commit(b_kempty(n % 3));
        if (n + 2 < nsteps && !scores(n + 2)) break;
      }
      tc::mma_commit(b_drain);
      volatile int no_abort = 0;
      tc::mbar_wait(b_drain, 0, &no_abort, limit);
    }
  } else {
    // ------------------------------------------------------------ elementwise
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int row = 32 * q + lane;
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const bool have = row < rows;
    const int fr = r0 + row, tok = have ? fr / a.group : 0, head = kvh * a.group + fr - tok * a.group;
    const int vis = have ? s.visible(a, tok) : 0;
    const int64_t st = (int64_t)kvh * a.qs.rows * a.group + (int64_t)s.q0 * a.group + fr;
    const float nl = have ? -a.lse2[st] : -INFINITY, delta = have ? a.delta[st] : 0.f;
    const float4 d4 = make_float4(delta, delta, delta, delta);
    const float cS = a.scale_log2;
    bool ok = true;
    if (!q_copy) {
      const int t = (int)threadIdx.x - 64;
      if (nsteps > 0) {
        load_rows_async<D>(sQ, a.q, a.sq, s.q0, kvh * a.group, a.group, r0, rows, 128, t, 256);
        load_rows_async<D>(sO, a.dout, a.sdo, s.q0, kvh * a.group, a.group, r0, rows, 128, t, 256);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_async_smem();
      warp_arrive(b_qo);
    }
    // `room`: D floats, the common part of the keys; at the end, from 512 bytes on, the rows' sums of dS that
    // count, and from 1 KB on the sums of dS and of P over the second half of the columns
    uint8_t *const room = sgen + 7 * T::kBytes;
    if (nsteps > 0)
      common_key<D>(a.k + (int64_t)s.k0 * a.sk[0] + (int64_t)kvh * a.sk[1], a.sk[0], keys, room, (int)threadIdx.x - 64);
    float2 ds_sum = tc::f2(0.f, 0.f), p_sum = ds_sum;
    for (int n = 0; n < nsteps; ++n) {
      if (!warp_wait(b_s(n & 1), (uint32_t)(n >> 1) & 1u, abort, limit)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const uint32_t colS = tS(n & 1) + lane_off + 64u * half;
      uint32_t p[64];
      {
        uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(p);
        uint32_t(&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(p + 32);
        tc::tmem_ld32(colS, lo);
        tc::tmem_ld32(colS + 32u, hi);
        tc::tmem_ld_wait();
      }
      const int seen = vis - 128 * n - 64 * half;
      const bool mask = __any_sync(0xffffffffu, seen < 64);
#pragma unroll
      for (int j = 0; j < 64; j += 2) {
        float2 x = tc::fma2(tc::f2u(p[j], p[j + 1]), tc::f2(cS, cS), tc::f2(nl, nl));
        if (mask) {
          if (j + 0 >= seen) x.x = -INFINITY;
          if (j + 1 >= seen) x.y = -INFINITY;
        }
        p[j] = __float_as_uint(tc::ex2(x.x));
        p[j + 1] = __float_as_uint(tc::ex2(x.y));
        p_sum = tc::fma2(tc::f2u(p[j], p[j + 1]), tc::f2(1.f, 1.f), p_sum);
      }
      if (!warp_wait(b_dp, (uint32_t)n & 1u, abort, limit)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      form_ds<true>(tDP + lane_off + 64u * half, colS, p, [&](int) { return d4; }, ds_sum);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      if (!(a.debug_stall && n == 0)) warp_arrive(b_ds);
    }
    float *const counts = reinterpret_cast<float *>(room + 512);
    float2 *const second = reinterpret_cast<float2 *>(room + 1024);
    if (half) second[row] = make_float2(ds_sum.x + ds_sum.y, p_sum.x + p_sum.y);
    elementwise_sync();      // (after a wait that ran out too)
    if (!half) {
      // (the fp32 LSE leaves P's sum off by some 2^-22 of its size)
      const float whole = p_sum.x + p_sum.y + second[row].y;
      counts[row] = fabsf(whole - 1.f) <= fmaf(fabsf(nl), 0x1p-20f, 0x1p-12f) ? ds_sum.x + ds_sum.y + second[row].x : 0.f;
    }
    elementwise_sync();
    if (__all_sync(0xffffffffu, ok && !*abort)) {
      if (nsteps > 0) ok = warp_wait(b_drain, 0, abort, limit);
      if (ok) {
        tc::tc_fence_after();
        constexpr int kCols = D / 2;
        const float sum = counts[row];
        uint8_t *const tile = sgen + (sQ - sbase);      // every product that reads Q is done
        const int ch0 = half * (kCols / 8);
        put_row<D, kCols, true>(tdQ + lane_off + (uint32_t)(half * kCols), nsteps == 0, a.scale, tile, row, ch0, sum,
                                reinterpret_cast<const float *>(room) + half * kCols);
        flush_rows<D, kCols>(tile, 32 * q, have ? a.dq + (int64_t)(s.q0 + tok) * a.sdq[0] + (int64_t)head * a.sdq[1] + half * kCols : nullptr, ch0);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Both kinds in one launch: the first `key_blocks` CTAs keep dK and dV (their loops
// are longer), the others dQ, which fill the SMs as the first kind runs out (8192
// tokens, 8 heads: 512 CTAs of either kind on 148 SMs).
template <int D>
__global__ void __launch_bounds__(kPbThreads, 1)
    packed_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                         const PackedArgs a, const PackedParts parts, const uint32_t limit, const int key_blocks) {
  const int block = (int)blockIdx.x;
  after_previous();
  if (block < key_blocks) packed_keys_cta<D>(tmQ, tmK, tmV, tmO, a, parts, limit, block);
  else packed_queries_cta<D>(tmQ, tmK, tmV, tmO, a, limit, block - key_blocks, (int)gridDim.x - key_blocks);
}

// Adds the shares of walks that were cut (see KeyWalk), in order: one CTA per (128
// keys, kv head, 32 columns).
template <int D>
__global__ void __launch_bounds__(256) packed_sum_kernel(const PackedArgs a, const PackedParts parts) {
  const int kvh = (int)(blockIdx.x % a.kv_heads), slot = (int)(blockIdx.x / a.kv_heads);
  after_previous();
  int64_t piece;
  const int b = find_sequence(a.ks, slot, 1, 128, piece);
  PackedSeq s;
  if (!s.load(a, b)) return;
  if (piece < 0 || piece * 128 >= s.room) return;
  const int key0 = (int)piece * 128;
  const KeyWalk walk(a, s, key0, parts.splits);
  if (walk.shares == 1) return;
  const int row = threadIdx.x & 127, rows = min(128, s.room - key0);
  const int64_t step = parts.tiles * (D * 128);
  const float *const base = (threadIdx.x < 128 ? parts.dk : parts.dv) + ((int64_t)blockIdx.x * (D / 4) + blockIdx.y * 8) * 512 + row * 4;
  float4 x[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int n = 0; n < walk.shares; ++n) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 p = *reinterpret_cast<const float4 *>(base + n * step + c * 512);
      x[c].x += p.x; x[c].y += p.y; x[c].z += p.z; x[c].w += p.w;
    }
  }
  if (row >= rows) return;
  const int64_t r = s.k0 + key0 + row;
  const float mul = threadIdx.x < 128 ? a.scale : 1.f;
  __nv_bfloat16 *const out = (threadIdx.x < 128 ? a.dk + r * a.sdk[0] + kvh * a.sdk[1] : a.dv + r * a.sdv[0] + kvh * a.sdv[1]) + blockIdx.y * 32;
#pragma unroll
  for (int c = 0; c < 8; c += 2)
    *reinterpret_cast<uint4 *>(out + 4 * c) =
        make_uint4(pack_bf16(x[c].x * mul, x[c].y * mul), pack_bf16(x[c].z * mul, x[c].w * mul),
                   pack_bf16(x[c + 1].x * mul, x[c + 1].y * mul), pack_bf16(x[c + 1].z * mul, x[c + 1].w * mul));
}

}  // namespace prism
