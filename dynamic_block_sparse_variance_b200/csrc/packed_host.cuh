// Entry points of the packed-sequence operators: argument checks, workspace
// layout and launches (included by prism.cu, whose helpers it uses).
#pragma once

#include "block_norm.cuh"
#include "packed_bwd_tc.cuh"
#include "packed_fwd_rows.cuh"

namespace prism {

// A launch that is made ready while the kernel before it on the stream runs out; the
// kernel itself waits for that one's results (after_previous()).  About 2 us per launch
// in a row of them, both sides on one machine: the training pass over 777 tokens 50.3 ->
// 47.6 us (on one with a faster host 46 -> 41), over 6144 packed tokens 251 -> 245,
// 61440 x 1536 block norms 145 -> 142.9.  A go-ahead from the kernel's
// own start (griddepcontrol.launch_dependents), so that the next one's blocks wait on the
// SMs as they come free, was slower: those 6144 tokens 267.
template <typename... P, typename... A>
static void launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, kernel, args...);
}

static bool strides_ok(const int64_t s[2]) {
  return (s[0] == 0 && s[1] == 0) || (s[0] > 0 && s[1] > 0 && s[0] % 8 == 0 && s[1] % 8 == 0);
}
// Strides of a [rows, heads, D] tensor; for a written one, no two elements may coincide.
static bool fill_strides(const int64_t in[2], int64_t rows, int heads, int D, bool written, int64_t out[2]) {
  if (!strides_ok(in)) return false;
  out[0] = in[0] ? in[0] : (int64_t)heads * D;
  out[1] = in[1] ? in[1] : D;
  if (out[0] >= ((int64_t)1 << 36) || out[1] >= ((int64_t)1 << 36)) return false;
  if (!written) return true;
  const bool rows_outer = (heads == 1 || out[1] >= D) && (rows <= 1 || out[0] >= (heads - 1) * out[1] + D);
  const bool heads_outer = (rows <= 1 || out[0] >= D) && (heads == 1 || out[1] >= (rows - 1) * out[0] + D);
  return rows_outer || heads_outer;
}

// Whether a written tensor begins where another one does (what else overlaps is the caller's to see: slices
// of one buffer interleave without sharing an element).
static bool same_start(std::initializer_list<const void *> written, std::initializer_list<const void *> read) {
  for (auto w = written.begin(); w != written.end(); ++w) {
    if (!*w) continue;
    for (auto v = written.begin(); v != w; ++v)
      if (*v == *w) return true;
    for (const void *r : read)
      if (r == *w) return true;
  }
  return false;
}

static bool even_split(int64_t rows, int seqs) { return rows % seqs == 0; }

static int check_packed(const prism_packed_params *p) {
  if (!p) return fail(PRISM_EINVAL, "packed params is NULL");
  if (p->seqs < 1) return fail(PRISM_EINVAL, "packed: seqs must be positive");
  if (p->heads < 1 || p->kv_heads < 1 || p->heads % p->kv_heads)
    return fail(PRISM_EINVAL, "packed: heads must be a positive multiple of kv_heads");
  if (p->heads / p->kv_heads > 128) return fail(PRISM_EINVAL, "packed: at most 128 query heads per kv head");
  if (p->kv_heads > 65535) return fail(PRISM_EINVAL, "packed: at most 65535 kv heads");
  if (p->head_dim != 64 && p->head_dim != 128) return fail(PRISM_EINVAL, "packed: head_dim must be 64 or 128");
  if (p->q_rows < 0 || p->k_rows < 0 || p->q_rows > 0x7fffff00LL || p->k_rows > 0x7fffff00LL)
    return fail(PRISM_EINVAL, "packed: row counts must be in [0, 2^31 - 256]");
  if (p->q_rows * (p->heads / p->kv_heads) > 0x7fffff00LL)
    return fail(PRISM_EINVAL, "packed: q_rows * heads / kv_heads must stay below 2^31 - 256");
  if (!(p->scale >= 0.f) || std::isinf(p->scale)) return fail(PRISM_EINVAL, "packed: scale must be finite and >= 0");
  return PRISM_OK;
}

static Offsets make_offsets(const int32_t *off, int seqs, int64_t rows) {
  return Offsets{off, seqs, (int)(rows / seqs), (int)rows};
}

// Common part of the kernel arguments; the caller has checked p.
static int packed_args(const prism_packed_params *p, const void *q, const void *k, const void *v, const int32_t *q_off,
                       const int32_t *k_off, const int32_t *k_used, PackedArgs *a) {
  if ((p->q_rows && !q) || (p->k_rows && (!k || !v))) return fail(PRISM_EINVAL, "packed: NULL tensor");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return fail(PRISM_EINVAL, "packed: tensors must be 16-byte aligned");
  if ((!q_off && !even_split(p->q_rows, p->seqs)) || (!k_off && !even_split(p->k_rows, p->seqs)))
    return fail(PRISM_EINVAL, "packed: without offsets the rows must split evenly over the sequences");
  if (!fill_strides(p->q_stride, p->q_rows, p->heads, p->head_dim, false, a->sq) ||
      !fill_strides(p->k_stride, p->k_rows, p->kv_heads, p->head_dim, false, a->sk) ||
      !fill_strides(p->v_stride, p->k_rows, p->kv_heads, p->head_dim, false, a->sv) ||
      !fill_strides(p->o_stride, p->q_rows, p->heads, p->head_dim, true, a->so))
    return fail(PRISM_EINVAL, "packed: strides must be positive multiples of 8, and outputs must not overlap themselves");
  a->qs = make_offsets(q_off, p->seqs, p->q_rows);
  a->ks = make_offsets(k_off, p->seqs, p->k_rows);
  a->k_used = k_used;
  a->heads = p->heads;
  a->kv_heads = p->kv_heads;
  a->group = p->heads / p->kv_heads;
  a->causal = p->causal != 0;
  a->debug_stall = g_debug_stall;
  a->scale = p->scale > 0.f ? p->scale : 1.f / std::sqrt((float)p->head_dim);
  a->scale_log2 = a->scale * kLog2e;
  a->q = static_cast<const __nv_bfloat16 *>(q);
  a->k = static_cast<const __nv_bfloat16 *>(k);
  a->v = static_cast<const __nv_bfloat16 *>(v);
  return PRISM_OK;
}

// The backward's cut of long walks over the queries (see KeyWalk): the longest walk
// is brought down to an even share of all products on 148 SMs, the walks of several
// sequences, whose lengths the host does not know, to twice that with the longest
// sequence taken as three times the average.  Whole against cut and added: 7 / 1 heads,
// 500 tokens 69 us / 27 + 8; 8 / 1, 4096 517 / 135 + 12; 5 / 1 of 64, 5000 over 2000 keys
// 132 / 38 + 14; 14 / 2, 3000 160 / 108 + 10; 16 / 4, 7 sequences of 6144 in all, which the
// rule leaves whole, 178 / 215 + 45.
struct PackedBwdWs {
  int splits;
  int64_t tiles;
  size_t delta, lse2, dk, dv, total;
  explicit PackedBwdWs(const prism_packed_params *p) {
    const size_t n = (size_t)p->q_rows * p->heads;
    const double seqs = p->seqs, qt = (double)p->q_rows / seqs * (p->heads / p->kv_heads) / 128, kt = (double)p->k_rows / seqs / 128;
    const double share = 7.0 * seqs * p->kv_heads * std::max(qt, 1.0) * std::max(kt, 1.0) * (p->causal ? 0.5 : 1.0) / 148;
    const double longest = 4.0 * qt * (p->seqs > 1 ? 1.5 : 1.0);
    splits = (int)std::max(1.0, std::min({8.0, std::floor(longest / share), std::floor(longest / 4 / 6)}));
    tiles = slot_bound(p->k_rows, p->seqs, 1, 128) * p->kv_heads;
    delta = 0;
    lse2 = align256(n * 4);
    dk = lse2 + align256(n * 4);
    const size_t part = splits > 1 ? align256((size_t)tiles * splits * 128 * p->head_dim * 4) : 0;
    dv = dk + part;
    total = dv + part;
  }
};

// 3-D map (head_dim, head, row) over a strided tensor: boxes of 64 columns of
// one head of 128 rows, 128-byte swizzle; rows past the end read as zero.
static bool make_head_map(CUtensorMap *map, const void *base, int D, int heads, int64_t rows, const int64_t s[2],
                          cuuint32_t box_heads = 1, cuuint32_t box_rows = 128) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)s[1] * 2, (cuuint64_t)s[0] * 2};
  cuuint32_t box[3] = {64, box_heads, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static uint32_t wait_limit() { return g_wait_limit ? g_wait_limit : kDefaultWaitLimit; }

// Which forward kernel runs and how the keys are split.  The host knows the rows,
// not the sequences' lengths, and goes by their average; either kernel is right for
// any.  Up to 16 flattened rows per sequence: the 16-row kernel (32 sequences, 32 / 8
// heads, 4096 keys: 4 rows 100 us against 144 with the other kernel, 16 rows 108
// against 145; with 32 rows it would read the keys twice).  Keys are split when
// the query rows alone give fewer CTAs than the SMs take (two of the 16-row
// kernel's waves, one of the others), in shares of at least 128 or 512 keys: one
// token over 32768 keys 41 us split, 250 whole, over 8192 25 / 68; 64 tokens over
// 16384 keys 33 / 259, 300 over 6000 (4 heads) 31 / 102; but over 1500 keys, where
// the second launch costs the host what the split saves, 17.5 / 17.0.
struct PackedFwdWs {
  bool few;
  int splits;
  size_t o, lse2, total;
  explicit PackedFwdWs(const prism_packed_params *p) {
    const int64_t group = p->heads / p->kv_heads;
    few = p->q_rows * group <= (int64_t)16 * p->seqs;
    const int64_t ctas = std::max<int64_t>(1, std::max<int64_t>(p->seqs, p->q_rows * group / 256) * p->kv_heads);
    const int64_t keys = p->k_rows / p->seqs;
    splits = (int)std::max<int64_t>(1, few ? std::min<int64_t>({(296 + ctas - 1) / ctas, keys / 128, 64})
                                           : std::min<int64_t>({148 / ctas, keys / 512, 64}));
    const size_t n = (size_t)p->q_rows * p->heads;
    o = 0;
    lse2 = splits > 1 ? align256(n * splits * p->head_dim * 4) : 0;
    total = splits > 1 ? lse2 + align256(n * splits * 4) : 0;
  }
};

template <int D>
static int launch_packed_fwd_rows(const prism_packed_params *p, const PackedArgs &a, const PackedSplit &sp, cudaStream_t st) {
  cudaFuncSetAttribute(packed_fwd_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrSmem<D>);
  const int64_t grid = slot_bound(p->q_rows, p->seqs, a.group, 16) * a.kv_heads;
  if (grid > 0x7fffffffLL) return fail(PRISM_EINVAL, "packed: too many query rows");
  PRISM_TRACED("packed_fwd_rows_kernel", st, launch_behind(packed_fwd_rows_kernel<D>, dim3((unsigned)grid, 1, sp.splits), kPrWarps * 32, kPrSmem<D>, st, a, sp));
  return PRISM_OK;
}

template <int D, int NG>
static int launch_packed_fwd_tc(const prism_packed_params *p, const PackedArgs &a, const PackedSplit &sp, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  // without keys nothing is loaded: the maps then only need to be well formed
  const bool keys = p->k_rows > 0;
  const int64_t dummy[2] = {D, D};
  if (!make_head_map(&tk, keys ? (const void *)a.k : a.q, D, keys ? a.kv_heads : 1, keys ? p->k_rows : 1, keys ? a.sk : dummy) ||
      !make_head_map(&tv, keys ? (const void *)a.v : a.q, D, keys ? a.kv_heads : 1, keys ? p->k_rows : 1, keys ? a.sv : dummy))
    return fail(PRISM_ECUDA, "cuTensorMapEncodeTiled failed");
  if (!make_head_map(&tq, a.q, D, a.heads, p->q_rows, a.sq, 128 % a.group ? 1 : a.group, 128 % a.group ? 128 : 128 / a.group))
    return fail(PRISM_ECUDA, "cuTensorMapEncodeTiled failed");
  using Cfg = PfCfg<D, NG>;
  cudaFuncSetAttribute(packed_fwd_tc_kernel<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  const int64_t slots = slot_bound(p->q_rows, p->seqs, a.group, 128 * NG);
  if (slots * a.kv_heads > 0x7fffffffLL) return fail(PRISM_EINVAL, "packed: too many query rows");
  const dim3 grid((unsigned)(slots * a.kv_heads), 1, sp.splits);
  PRISM_TRACED("packed_fwd_tc_kernel", st, launch_behind(packed_fwd_tc_kernel<D, NG>, grid, (int)Cfg::kThreads, Cfg::kSmem, st, tq, tk, tv, a, sp, wait_limit()));
  return PRISM_OK;
}

template <int D>
static int launch_packed_fwd(const prism_packed_params *p, const PackedArgs &a, uint8_t *ws, cudaStream_t st) {
  const PackedFwdWs w(p);
  PackedSplit sp{w.splits, reinterpret_cast<float *>(ws + w.o), reinterpret_cast<float *>(ws + w.lse2)};
  // Pairs of tiles from 512 keys per sequence on, single tiles below.  Pairs against
  // single, 16 / 4 heads of 128, 8192 causal rows in equal sequences: of 256 keys 45.5
  // against 43.2 us, of 512 53.3 / 52.7, of 1024 68.0 / 69.6, of 4096 140 / 162; 9
  // sequences of 119 to 3540, 99 / 107.
  const int rc = w.few ? launch_packed_fwd_rows<D>(p, a, sp, st) : p->k_rows / p->seqs < 512 ? launch_packed_fwd_tc<D, 1>(p, a, sp, st) : launch_packed_fwd_tc<D, 2>(p, a, sp, st);
  if (rc) return rc;
  if (w.splits > 1) {
    const int64_t threads = p->q_rows * p->heads * (D / 4);
    PRISM_TRACED("packed_combine_kernel", st, launch_behind(packed_combine_kernel<D>, dim3((unsigned)((threads + 255) / 256)), 256, 0, st, a, sp));
  }
  return PRISM_OK;
}

template <int D>
static int launch_packed_bwd(const prism_packed_params *p, const PackedArgs &a, const PackedParts &parts, float *delta,
                             float *lse2, cudaStream_t st) {
  const int64_t dummy[2] = {D, D};
  const bool keys = p->k_rows > 0, rows = p->q_rows > 0;
  if (!keys && !rows) return PRISM_OK;
  const int tt = 128 / a.group;     // tokens per streamed query tile
  const void *any = rows ? (const void *)a.q : a.k;
  CUtensorMap tq, to, tk, tv;
  if (!make_head_map(&tk, keys ? (const void *)a.k : any, D, keys ? a.kv_heads : 1, keys ? p->k_rows : 1, keys ? a.sk : dummy) ||
      !make_head_map(&tv, keys ? (const void *)a.v : any, D, keys ? a.kv_heads : 1, keys ? p->k_rows : 1, keys ? a.sv : dummy) ||
      !make_head_map(&tq, any, D, rows ? a.heads : 1, rows ? p->q_rows : 1, rows ? a.sq : dummy, a.group, tt) ||
      !make_head_map(&to, rows ? (const void *)a.dout : any, D, rows ? a.heads : 1, rows ? p->q_rows : 1, rows ? a.sdo : dummy, a.group, tt))
    return fail(PRISM_ECUDA, "cuTensorMapEncodeTiled failed");
  if (rows) {
    const int64_t threads = p->q_rows * p->heads * (D / 8);
    PRISM_TRACED("packed_stats_kernel", st, launch_behind(packed_stats_kernel<D>, dim3((unsigned)((threads + 511) / 512)), 256, 0, st, a, (const __nv_bfloat16 *)a.o, delta, lse2));
  }
  const int64_t key_tiles = keys ? parts.tiles : 0, key_blocks = key_tiles * parts.splits;
  const int64_t blocks = key_blocks + (rows ? slot_bound(p->q_rows, p->seqs, a.group, 128) * a.kv_heads : 0);
  if (blocks > 0x7fffffffLL) return fail(PRISM_EINVAL, "packed: too many rows");
  cudaFuncSetAttribute(packed_bwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPbSmem<D>);
  PRISM_TRACED("packed_bwd_tc_kernel", st, launch_behind(packed_bwd_tc_kernel<D>, dim3((unsigned)blocks), kPbThreads, kPbSmem<D>, st, tq, tk, tv, to, a, parts, wait_limit(), (int)key_blocks));
  if (parts.splits > 1 && keys)
    PRISM_TRACED("packed_sum_kernel", st, launch_behind(packed_sum_kernel<D>, dim3((unsigned)key_tiles, D / 32), 256, 0, st, a, parts));
  return PRISM_OK;
}

// ---- block norms -----------------------------------------------------------------

static bool norm_row_stride(int64_t in, int C, int64_t *out) {
  *out = in ? in : C;
  return in == 0 || (in >= C && in % 8 == 0 && in < ((int64_t)1 << 40));
}
// A row's copies have landed before the row is written, so an output may begin where an input does if its
// rows lie the same way: the same type and row stride.
struct NormInput {
  const void *p;
  int64_t stride;
  bool same_type;
};
static bool in_place(const void *out, int64_t stride, std::initializer_list<NormInput> in) {
  for (const NormInput &i : in)
    if (i.p == out && !(i.same_type && i.stride == stride)) return false;
  return true;
}
static bool is_float_type(int t) { return t == PRISM_BF16 || t == PRISM_F32; }

static int check_norm(const prism_norm_params *p) {
  if (!p) return fail(PRISM_EINVAL, "norm params is NULL");
  if (p->rows < 0 || p->rows > 0x7fffff00LL) return fail(PRISM_EINVAL, "block_norm: rows must be in [0, 2^31 - 256]");
  if (p->seqs < 1) return fail(PRISM_EINVAL, "block_norm: seqs must be positive");
  if (p->seqs > 65534) return fail(PRISM_EINVAL, "block_norm: at most 65534 sequences");
  if (p->channels < 8 || p->channels % 8 || p->channels > PRISM_NORM_MAX_CHANNELS)
    return fail(PRISM_EINVAL, "block_norm: channels must be a multiple of 8 in [8, 8192]");
  if (!is_float_type(p->stream_dtype) || !is_float_type(p->branch_dtype) || !is_float_type(p->param_dtype))
    return fail(PRISM_EINVAL, "block_norm: dtypes must be bf16 or f32");
  if (p->post_norm < PRISM_NORM_NONE || p->post_norm > PRISM_NORM_LAYER) return fail(PRISM_EINVAL, "block_norm: unknown post_norm");
  if (p->pre_norm != PRISM_NORM_RMS && p->pre_norm != PRISM_NORM_LAYER) return fail(PRISM_EINVAL, "block_norm: pre_norm must be RMS or LAYER");
  if (!(p->eps >= 0.f) || std::isinf(p->eps) || !std::isfinite(p->alpha)) return fail(PRISM_EINVAL, "block_norm: eps must be finite and >= 0, alpha finite");
  for (int64_t s : {p->gate_stride, p->scale_stride, p->shift_stride})
    if (s != 0 && (s < p->channels || s % 8 || s >= ((int64_t)1 << 40)))
      return fail(PRISM_EINVAL, "block_norm: parameter strides must be 0 or a multiple of 8 of at least channels");
  return PRISM_OK;
}

static int norm_args(const prism_norm_params *p, const int32_t *off, const void *post_weight, const void *gate,
                     const void *weight, const void *scale, const void *shift, BlockNormArgs *a) {
  if (!off && !even_split(p->rows, p->seqs))
    return fail(PRISM_EINVAL, "block_norm: without offsets the rows must split evenly over the sequences");
  for (const void *q : {post_weight, gate, weight, scale, shift})
    if (!aligned16(q)) return fail(PRISM_EINVAL, "block_norm: parameters must be 16-byte aligned");
  if (!norm_row_stride(p->x_row_stride, p->channels, &a->sx) || !norm_row_stride(p->y_row_stride, p->channels, &a->sy) ||
      !norm_row_stride(p->x_out_row_stride, p->channels, &a->sxo) || !norm_row_stride(p->h_row_stride, p->channels, &a->sh) ||
      !norm_row_stride(p->dh_row_stride, p->channels, &a->sdh) || !norm_row_stride(p->dx_out_row_stride, p->channels, &a->sdxo) ||
      !norm_row_stride(p->dx_row_stride, p->channels, &a->sdx) || !norm_row_stride(p->dy_row_stride, p->channels, &a->sdy))
    return fail(PRISM_EINVAL, "block_norm: row strides must be 0 or a multiple of 8 of at least channels");
  a->seq = make_offsets(off, p->seqs, p->rows);
  a->C = p->channels;
  a->post = p->post_norm;
  a->pre = p->pre_norm;
  a->param_f32 = p->param_dtype == PRISM_F32;
  a->eps = p->eps;
  a->alpha = p->alpha;
  a->post_weight = post_weight;
  a->gate = gate;
  a->weight = weight;
  a->scale = scale;
  a->shift = shift;
  a->sgate = p->gate_stride;
  a->sscale = p->scale_stride;
  a->sshift = p->shift_stride;
  a->wait_limit = wait_limit();
  return PRISM_OK;
}

// Launch shapes: one CTA per SM, whose rings take what shared memory the folded
// parameters leave, and about as many runs of rows as there are SMs.
constexpr int kBnSmem = 216 * 1024;
static int type_bytes(int t) { return t == PRISM_F32 ? 4 : 2; }
// Forward: a row in the registers of one warp up to 2048 channels (8 vectors of
// 8 columns a thread), of 2 to 4 warps beyond.
struct NormFwdShape {
  int wpr, groups, vecs, V, stages, unit, threads;
  size_t smem;
  int64_t slots;
  NormFwdShape(const prism_norm_params *p, bool with_y) {
    const int C = p->channels;
    wpr = (C + 2047) / 2048;
    vecs = (C + 256 * wpr - 1) / (256 * wpr);
    V = vecs <= 1 ? 1 : vecs <= 2 ? 2 : vecs <= 4 ? 4 : 8;
    const int row = C * (type_bytes(p->stream_dtype) + (with_y ? type_bytes(p->branch_dtype) : 0));
    groups = std::max(1, std::min(kBnWarps / wpr, (kBnSmem - 12 * C) / row));
    unit = (int)run_length(p->rows, p->seqs, 148, 1);
    groups = std::min(groups, unit);
    stages = std::max(1, std::min({kBnMaxStages, (kBnSmem - 12 * C) / (groups * row), (unit + groups - 1) / groups}));
    smem = (size_t)12 * C + (size_t)groups * stages * row;
    // more warps than rows need still share the folding of the parameters
    threads = std::max(groups * wpr, std::min(kBnWarps, C / 256)) * 32;
    slots = slot_bound(p->rows, p->seqs, 1, unit);
  }
};
// Backward: 8 columns a thread up to 4096 channels, 16 beyond; narrow rows share
// a CTA of about 256 threads.  The kernel's registers let an SM hold 16 warps,
// which with the rings gives the CTAs per SM and, one wave of them, the rows
// per CTA.  The stages have room for all four tensors, whichever a call gives.
struct NormBwdShape {
  int V, wpr, groups, threads, stages, unit;
  size_t smem;
  int64_t slots;
  explicit NormBwdShape(const prism_norm_params *p) {
    const int C = p->channels;
    V = C > 8 * kBnMaxThreads ? 2 : 1;
    wpr = (C + 256 * V - 1) / (256 * V);
    groups = std::max(1, 8 / wpr);
    threads = wpr * groups * 32;
    const int batch = bn_bwd_rows(V);
    const int stage = C * 2 * (type_bytes(p->stream_dtype) + type_bytes(p->branch_dtype)) * groups * batch;
    const int fixed = V == 2 ? 8 * C : 0;
    const int ctas = std::max(1, std::min(16 / (wpr * groups), 200 * 1024 / (2 * stage + fixed + 2048)));
    stages = std::max(1, std::min(kBnMaxStages, (200 * 1024 / ctas - fixed - 2048) / stage));
    smem = (size_t)stages * stage + fixed;
    unit = (int)run_length(p->rows, p->seqs, 148 * ctas, 2 * groups);
    const int whole = batch * groups;      // whole batches, unless the rows are few
    if (unit >= whole) unit = (unit + whole - 1) / whole * whole;
    slots = slot_bound(p->rows, p->seqs, 1, unit);
  }
};

template <typename TX, typename TY, int V>
static int launch_norm_fwd_v(const NormFwdShape &s, const BlockNormArgs &a, cudaStream_t st) {
  cudaFuncSetAttribute(block_norm_fwd_kernel<TX, TY, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBnSmem);
  PRISM_TRACED("block_norm_fwd_kernel", st, launch_behind(block_norm_fwd_kernel<TX, TY, V>, dim3((unsigned)s.slots), s.threads, s.smem, st, a));
  return PRISM_OK;
}
template <typename TX, typename TY>
static int launch_norm_fwd(const prism_norm_params *p, BlockNormArgs &a, cudaStream_t st) {
  const NormFwdShape s(p, a.y != nullptr);
  a.unit = s.unit;
  a.wpr = s.wpr;
  a.groups = s.groups;
  a.stages = s.stages;
  a.vecs = s.vecs;
  switch (s.V) {
    case 1: return launch_norm_fwd_v<TX, TY, 1>(s, a, st);
    case 2: return launch_norm_fwd_v<TX, TY, 2>(s, a, st);
    case 4: return launch_norm_fwd_v<TX, TY, 4>(s, a, st);
    default: return launch_norm_fwd_v<TX, TY, 8>(s, a, st);
  }
}
template <typename TX, typename TY, int V, int kThreads>
static int launch_norm_bwd_v(const NormBwdShape &s, const BlockNormArgs &a, cudaStream_t st) {
  void (*const kernel)(const BlockNormArgs) = block_norm_bwd_kernel<TX, TY, V, kThreads>;
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBnSmem);
  PRISM_TRACED("block_norm_bwd_kernel", st, launch_behind(kernel, dim3((unsigned)s.slots), s.threads, s.smem, st, a));
  return PRISM_OK;
}
// Two vectors a thread need 156 to 168 registers, which 384 threads (6144 channels) leave
// each of them; beyond, the form of 512 threads has 128 and spills (6144 channels, bf16,
// 7500 rows: 150 us against 205 with that form).
template <typename TX, typename TY>
static int launch_norm_bwd(const NormBwdShape &s, const BlockNormArgs &a, cudaStream_t st) {
  return s.V == 1 ? launch_norm_bwd_v<TX, TY, 1, 512>(s, a, st)
                  : s.threads <= 384 ? launch_norm_bwd_v<TX, TY, 2, 384>(s, a, st) : launch_norm_bwd_v<TX, TY, 2, 512>(s, a, st);
}

}  // namespace prism

extern "C" {

int prism_packed_workspace_size(const prism_packed_params *p, int kind, size_t *bytes) {
  int rc = check_packed(p);
  if (rc) return rc;
  if (!bytes) return fail(PRISM_EINVAL, "bytes is NULL");
  switch (kind) {
    case PRISM_WS_PACKED_FWD: *bytes = PackedFwdWs(p).total; break;
    case PRISM_WS_PACKED_BWD: *bytes = PackedBwdWs(p).total; break;
    default: return fail(PRISM_EINVAL, "unknown workspace kind");
  }
  return PRISM_OK;
}

int prism_packed_attn_fwd(const prism_packed_params *p, const void *q, const void *k, const void *v,
                          const int32_t *q_off, const int32_t *k_off, const int32_t *k_used, void *o, void *o_res,
                          float *lse, void *workspace, size_t ws_bytes, prism_stream stream) {
  int rc = check_packed(p);
  if (rc) return rc;
  PackedArgs a = {};
  rc = packed_args(p, q, k, v, q_off, k_off, k_used, &a);
  if (rc) return rc;
  if (p->q_rows == 0) return PRISM_OK;
  if (!o || !lse) return fail(PRISM_EINVAL, "packed: NULL output");
  if (!aligned16(o) || !aligned16(o_res)) return fail(PRISM_EINVAL, "packed: tensors must be 16-byte aligned");
  a.o = static_cast<__nv_bfloat16 *>(o);
  a.o_res = static_cast<__nv_bfloat16 *>(o_res);
  a.lse = lse;
  const size_t need = PackedFwdWs(p).total;
  if (need && (!workspace || ws_bytes < need || !aligned16(workspace)))
    return fail(PRISM_EINVAL, "packed: workspace missing, misaligned or below prism_packed_workspace_size");
  if (same_start({o, o_res, lse}, {q, p->k_rows ? k : nullptr, p->k_rows ? v : nullptr}))
    return fail(PRISM_EINVAL, "packed: an output must not take the place of an input or of another output");
  cudaStream_t st = as_stream(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  return p->head_dim == 128 ? launch_packed_fwd<128>(p, a, ws, st) : launch_packed_fwd<64>(p, a, ws, st);
}

int prism_packed_attn_bwd(const prism_packed_params *p, const void *q, const void *k, const void *v, const void *o,
                          const void *o_res, const void *dout, const float *lse, const int32_t *q_off,
                          const int32_t *k_off, const int32_t *k_used, void *dq, void *dk, void *dv, void *workspace,
                          size_t ws_bytes, prism_stream stream) {
  int rc = check_packed(p);
  if (rc) return rc;
  PackedArgs a = {};
  rc = packed_args(p, q, k, v, q_off, k_off, k_used, &a);
  if (rc) return rc;
  if ((p->q_rows && (!o || !dout || !lse || !dq)) || (p->k_rows && (!dk || !dv)))
    return fail(PRISM_EINVAL, "packed: NULL tensor");
  for (const void *t : {o, o_res, dout, (const void *)dq, (const void *)dk, (const void *)dv})
    if (!aligned16(t)) return fail(PRISM_EINVAL, "packed: tensors must be 16-byte aligned");
  if (!fill_strides(p->dout_stride, p->q_rows, p->heads, p->head_dim, false, a.sdo) ||
      !fill_strides(p->dq_stride, p->q_rows, p->heads, p->head_dim, true, a.sdq) ||
      !fill_strides(p->dk_stride, p->k_rows, p->kv_heads, p->head_dim, true, a.sdk) ||
      !fill_strides(p->dv_stride, p->k_rows, p->kv_heads, p->head_dim, true, a.sdv))
    return fail(PRISM_EINVAL, "packed: strides must be positive multiples of 8, and outputs must not overlap themselves");
  const PackedBwdWs w(p);
  if (w.total && (!workspace || ws_bytes < w.total || !aligned16(workspace)))
    return fail(PRISM_EINVAL, "packed: workspace missing, misaligned or below prism_packed_workspace_size");
  if (p->q_rows && p->k_rows ? same_start({dq, dk, dv}, {q, k, v, o, o_res, dout, lse})
                             : p->q_rows ? same_start({dq}, {q, o, o_res, dout, lse}) : p->k_rows && same_start({dk, dv}, {k, v}))
    return fail(PRISM_EINVAL, "packed: an output must not take the place of an input or of another output");
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  float *delta = reinterpret_cast<float *>(ws + w.delta), *lse2 = reinterpret_cast<float *>(ws + w.lse2);
  a.o = static_cast<__nv_bfloat16 *>(const_cast<void *>(o));
  a.o_res = static_cast<__nv_bfloat16 *>(const_cast<void *>(o_res));
  a.dout = static_cast<const __nv_bfloat16 *>(dout);
  a.lse = const_cast<float *>(lse);
  a.delta = delta;
  a.lse2 = lse2;
  a.dq = static_cast<__nv_bfloat16 *>(dq);
  a.dk = static_cast<__nv_bfloat16 *>(dk);
  a.dv = static_cast<__nv_bfloat16 *>(dv);
  cudaStream_t st = as_stream(stream);
  const PackedParts parts{w.splits, w.tiles, reinterpret_cast<float *>(ws + w.dk), reinterpret_cast<float *>(ws + w.dv)};
  return p->head_dim == 128 ? launch_packed_bwd<128>(p, a, parts, delta, lse2, st)
                            : launch_packed_bwd<64>(p, a, parts, delta, lse2, st);
}

int prism_block_norm_fwd(const prism_norm_params *p, const void *x, const void *y, const int32_t *off,
                         const void *post_weight, const void *gate, const void *weight, const void *scale,
                         const void *shift, void *x_out, void *h, float *y_norms, prism_stream stream) {
  int rc = check_norm(p);
  if (rc) return rc;
  BlockNormArgs a = {};
  rc = norm_args(p, off, post_weight, gate, weight, scale, shift, &a);
  if (rc) return rc;
  if (p->rows == 0) return PRISM_OK;
  if (!x || (y && !x_out) || (!y && !h)) return fail(PRISM_EINVAL, "block_norm: NULL tensor");
  if (!y && y_norms) return fail(PRISM_EINVAL, "block_norm: y_norms needs y");
  for (const void *t : {x, y, (const void *)x_out, (const void *)h})
    if (!aligned16(t)) return fail(PRISM_EINVAL, "block_norm: tensors must be 16-byte aligned");
  const bool xt = p->stream_dtype == p->branch_dtype;      // x and x_out have the types of y and h
  if ((y && h && same_start({x_out, h}, {})) || (y && !in_place(x_out, a.sxo, {{x, a.sx, true}, {y, a.sy, xt}})) ||
      (h && !in_place(h, a.sh, {{x, a.sx, xt}, {y, a.sy, true}})))
    return fail(PRISM_EINVAL, "block_norm: an output takes an input's place only with its type and row stride, and never another output's");
  a.x = x;
  a.y = y;
  a.x_out = y ? x_out : nullptr;
  a.h = h;
  a.y_norms = y_norms;
  cudaStream_t st = as_stream(stream);
  if (p->stream_dtype == PRISM_BF16)
    return p->branch_dtype == PRISM_BF16 ? launch_norm_fwd<__nv_bfloat16, __nv_bfloat16>(p, a, st)
                                         : launch_norm_fwd<__nv_bfloat16, float>(p, a, st);
  return p->branch_dtype == PRISM_BF16 ? launch_norm_fwd<float, __nv_bfloat16>(p, a, st)
                                       : launch_norm_fwd<float, float>(p, a, st);
}

int prism_block_norm_workspace_size(const prism_norm_params *p, size_t *bytes) {
  int rc = check_norm(p);
  if (rc) return rc;
  if (!bytes) return fail(PRISM_EINVAL, "bytes is NULL");
  const NormBwdShape s(p);
  *bytes = align256((size_t)s.slots * s.groups * 3 * p->channels * 4);
  return PRISM_OK;
}

int prism_block_norm_bwd(const prism_norm_params *p, const void *x_out, const void *y, const int32_t *off,
                         const void *post_weight, const void *gate, const void *weight, const void *scale,
                         const void *dh, const void *dx_out, void *dx, void *dy, void *dpost_weight, void *dgate,
                         void *dweight, void *dscale, void *dshift, void *workspace, size_t ws_bytes,
                         prism_stream stream) {
  int rc = check_norm(p);
  if (rc) return rc;
  BlockNormArgs a = {};
  rc = norm_args(p, off, post_weight, gate, weight, scale, nullptr, &a);
  if (rc) return rc;
  if (p->rows && ((!dh && !dx_out) || (dh && !x_out) || !dx || (y && !dy)))
    return fail(PRISM_EINVAL, "block_norm: NULL tensor");
  if (!y && (dpost_weight || dgate)) return fail(PRISM_EINVAL, "block_norm: dpost_weight and dgate need y");
  for (const void *t : {x_out, y, dh, dx_out, (const void *)dx, (const void *)dy})
    if (!aligned16(t)) return fail(PRISM_EINVAL, "block_norm: tensors must be 16-byte aligned");
  const NormBwdShape w(p);
  const size_t need_ws = (size_t)w.slots * w.groups * 3 * p->channels * 4;
  if (!workspace || ws_bytes < need_ws || !aligned16(workspace))
    return fail(PRISM_EINVAL, "block_norm: workspace missing, misaligned or below prism_block_norm_workspace_size");
  const bool xt = p->stream_dtype == p->branch_dtype;
  if (p->rows && (same_start({dx, y ? dy : nullptr}, {}) ||
                  !in_place(dx, a.sdx, {{x_out, a.sxo, true}, {dx_out, a.sdxo, true}, {dh, a.sdh, xt}, {y, a.sy, xt}}) ||
                  (y && !in_place(dy, a.sdy, {{x_out, a.sxo, xt}, {dx_out, a.sdxo, xt}, {dh, a.sdh, true}, {y, a.sy, true}}))))
    return fail(PRISM_EINVAL, "block_norm: an output takes an input's place only with its type and row stride, and never another output's");
  a.unit = w.unit;
  a.wpr = w.wpr;
  a.groups = w.groups;
  a.stages = w.stages;
  a.y = y;
  a.x_out = const_cast<void *>(x_out);
  a.dh = dh;
  a.dx_out = dx_out;
  a.dx = dx;
  a.dy = dy;
  a.need = (dweight || dscale ? 1 : 0) | (dshift ? 2 : 0) | (dgate || dpost_weight ? 4 : 0);
  a.part = static_cast<float *>(workspace);
  cudaStream_t st = as_stream(stream);
  if (p->rows) {
    if (p->stream_dtype == PRISM_BF16)
      rc = p->branch_dtype == PRISM_BF16 ? launch_norm_bwd<__nv_bfloat16, __nv_bfloat16>(w, a, st)
                                         : launch_norm_bwd<__nv_bfloat16, float>(w, a, st);
    else
      rc = p->branch_dtype == PRISM_BF16 ? launch_norm_bwd<float, __nv_bfloat16>(w, a, st)
                                         : launch_norm_bwd<float, float>(w, a, st);
    if (rc) return rc;
  }
  if (!a.need) return PRISM_OK;
  BnParamArgs q = {};
  q.seq = a.seq;
  q.C = a.C;
  q.unit = w.unit;
  q.groups = w.groups;
  q.param_f32 = a.param_f32;
  q.need = a.need;
  q.part = a.part;
  q.weight = weight;
  q.post_weight = post_weight;
  q.gate = gate;
  q.scale = scale;
  q.sgate = a.sgate;
  q.sscale = a.sscale;
  q.dweight = dweight;
  q.dpost_weight = dpost_weight;
  q.dgate = dgate;
  q.dscale = dscale;
  q.dshift = dshift;
  q.per_gate = p->gate_stride != 0;
  q.per_scale = p->scale_stride != 0;
  q.per_shift = p->shift_stride != 0;
  const bool per = (dgate && q.per_gate) || (dscale && q.per_scale) || (dshift && q.per_shift);
  PRISM_TRACED("block_norm_params_kernel", st, launch_behind(block_norm_params_kernel, dim3((unsigned)((a.C + 31) / 32), per ? 1 + p->seqs : 1), kBnParamWarps * 32, 0, st, q));
  return PRISM_OK;
}

}  // extern "C"
