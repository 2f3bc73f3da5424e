// ops_api.cuh — entry points of the operators around attention (include/fa.h): the norm with the
// position rotation, the decode steps over pieces of the cache, and the eviction.  Included by
// fa_api.cu, whose helpers (alignment, TMA descriptors, launches) it uses.
#pragma once
#ifndef FA_ROPE_PERSM
#define FA_ROPE_PERSM 32
#endif
#ifndef FA_ROPE_BWD_PERSM
#define FA_ROPE_BWD_PERSM 32
#endif
#ifndef FA_ROPE_BWD_C
#define FA_ROPE_BWD_C 2
#endif

namespace {

// Rotation arguments that every rotary entry point shares: sizes, then one of `out` launches.
fa_status rope_check(const int* positions, const double* inv_freq, int B, int Hq, int Hkv, int N, int d, int rotary_dim,
                     const int* sections, int n_axes, int interleaved, float eps, fa_dtype dtype) {
  if (!positions || !inv_freq || !sections) return FA_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0 || rotary_dim <= 0) return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return FA_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > 3 || (interleaved != 0 && interleaved != 1)) return FA_ERR_INVALID_ARG;
  if (rotary_dim > d || rotary_dim % 2 != 0) return FA_ERR_INVALID_ARG;
  long sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0) return FA_ERR_INVALID_ARG;
    sum += sections[a];
  }
  if (sum != rotary_dim / 2) return FA_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_F32 && dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
  if ((d != 64 && d != 96 && d != 128 && d != 256) || rotary_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (Hq > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Rows of 16-byte pieces at any (batch, head, token): base and strides (elements) are multiples of 16 bytes.
bool rope_rows(const void* p, const int64_t* strides, fa_dtype dtype) {
  const int64_t per = dtype == FA_DTYPE_F32 ? 4 : 8;
  if (!p || !strides || !aligned(p, 16)) return false;
  for (int i = 0; i < 3; ++i)
    if (strides[i] < 0 || strides[i] % per != 0) return false;
  return true;
}

// Heads per unit of work: 16, halved until every SM has `per_sm` units (or a head is a unit),
// and spread evenly over the heads.
int rope_chunk(int64_t rows, int tokens_per_warp, int H, int per_sm, int sms) {
  int c = rope::MAX_CHUNK;
  while (c > 1 && rows / (int64_t(tokens_per_warp) * c) < int64_t(per_sm) * sms) c /= 2;
  const int chunks = (H + c - 1) / c;
  return (H + chunks - 1) / chunks;
}

template <typename T, int D, bool PAGED>
fa_status rope_launch(RopeParams& prm, bool inter, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const int64_t tokens = int64_t(prm.B) * prm.N;
  constexpr int TOKENS = rope::Cfg<D>::TOKENS;
  const int heads = prm.Hq + (PAGED ? 2 : 1) * prm.Hkv;
  prm.chunk = rope_chunk(tokens * heads, TOKENS, prm.Hq, FA_ROPE_PERSM, sms);
  prm.chunks_q = (prm.Hq + prm.chunk - 1) / prm.chunk;
  prm.chunks_k = (prm.Hkv + prm.chunk - 1) / prm.chunk;
  const int64_t units = (tokens + TOKENS - 1) / TOKENS * (prm.chunks_q + (PAGED ? 2 : 1) * prm.chunks_k);
  const int64_t grid = (units + rope::THREADS / 32 - 1) / (rope::THREADS / 32);
  if (tokens > 0x7fffff00 || grid > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  auto kern = inter ? fa_qk_norm_rope_kernel<T, D, true, PAGED> : fa_qk_norm_rope_kernel<T, D, false, PAGED>;
  constexpr int SMEM = rope::STAGES * rope::Slot<T, sizeof(T) == 4>::BYTES;
  if (set_smem(kern, SMEM) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_pdl(kern, dim3(unsigned(grid)), dim3(rope::THREADS), SMEM, st, prm) != cudaSuccess) return FA_ERR_CUDA;
  return launched();
}

constexpr int kRopeBwdCtas = 148 * FA_ROPE_BWD_C;  // CTAs of the backward kernel, at most

template <typename T, typename TG, typename TO, int D>
fa_status rope_bwd_launch(RopeBwdParams& prm, bool inter, float* dwq, float* dwk, cudaStream_t st) {
  const int64_t tokens = int64_t(prm.B) * prm.N;
  if (tokens > 0x7fffff00) return FA_ERR_UNSUPPORTED;
  constexpr int TOKENS = rope::Cfg<D>::TOKENS, WARPS = rope::THREADS / 32;
  const int heads = prm.H[0] + prm.H[1];
  prm.chunk = rope_chunk(tokens * heads, TOKENS, prm.H[0], FA_ROPE_BWD_PERSM, kRopeBwdCtas / FA_ROPE_BWD_C);
  int ctas[2];
  for (int k = 0; k < 2; ++k) {
    prm.chunks[k] = (prm.H[k] + prm.chunk - 1) / prm.chunk;
    // CTAs in proportion to the rows, no more than there are units
    const int64_t units = (tokens + TOKENS - 1) / TOKENS * prm.chunks[k];
    const int64_t share = std::max<int64_t>(1, int64_t(kRopeBwdCtas) * prm.H[k] / heads);
    ctas[k] = int(std::min<int64_t>(std::min<int64_t>(share, kRopeBwdCtas - 1), (units + WARPS - 1) / WARPS));
  }
  prm.ctas_q = ctas[0];
  auto kern = inter ? fa_qk_norm_rope_bwd_kernel<T, TG, TO, D, true> : fa_qk_norm_rope_bwd_kernel<T, TG, TO, D, false>;
  constexpr int SMEM = rope::BWD_STAGES * rope::THREADS * 16 * int(sizeof(T) + sizeof(TG));
  static_assert(SMEM >= WARPS * D * 4, "the weight-gradient sums reuse the slots");
  if (set_smem(kern, SMEM) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_pdl(kern, dim3(unsigned(ctas[0] + ctas[1])), dim3(rope::THREADS), SMEM, st, prm) != cudaSuccess)
    return FA_ERR_CUDA;
  if (prm.w[0] && launch_pdl(fa_qk_norm_rope_dw_kernel, dim3(D / 8, 2), dim3(512), 0, st,
                             static_cast<const float*>(prm.part), dwq, dwk, D, ctas[0], ctas[0] + ctas[1]) != cudaSuccess)
    return FA_ERR_CUDA;
  return launched();
}

template <typename T, typename TG, typename TO>
fa_status rope_bwd_by_d(RopeBwdParams& prm, int d, bool inter, float* dwq, float* dwk, cudaStream_t st) {
  switch (d) {
    case 64: return rope_bwd_launch<T, TG, TO, 64>(prm, inter, dwq, dwk, st);
    case 96: return rope_bwd_launch<T, TG, TO, 96>(prm, inter, dwq, dwk, st);
    case 128: return rope_bwd_launch<T, TG, TO, 128>(prm, inter, dwq, dwk, st);
    default: return rope_bwd_launch<T, TG, TO, 256>(prm, inter, dwq, dwk, st);
  }
}

template <typename T>
fa_status rope_by_d(RopeParams& prm, int d, bool inter, cudaStream_t st) {
  switch (d) {
    case 64: return rope_launch<T, 64, false>(prm, inter, st);
    case 96: return rope_launch<T, 96, false>(prm, inter, st);
    case 128: return rope_launch<T, 128, false>(prm, inter, st);
    default: return rope_launch<T, 256, false>(prm, inter, st);
  }
}

// ---- decode over pieces

// Blocks of a piece: enough pieces for a few CTAs on each of 148 SMs when `sets` sets of rows
// walk `blocks` blocks each, at least part::MIN_CHUNK blocks a piece and at most 64 pieces.
int part_chunk(int64_t sets, int64_t blocks) {
  const int64_t want = std::max<int64_t>(1, (148 * 4 + sets - 1) / sets);
  const int64_t pieces = std::min<int64_t>(64, want);
  const int64_t c = std::max<int64_t>(part::MIN_CHUNK, (blocks + pieces - 1) / pieces);
  return int((c + part::WARPS - 1) / part::WARPS * part::WARPS);
}

struct PartPlan {
  int chunk, prefix_chunk, own_parts, prefix_parts, row_tiles;
  size_t off_lse, off_scores, bytes;
};

PartPlan part_plan(int R, int Hq, int Hkv, int d, int max_blocks, int prefix_blocks, bool scored) {
  PartPlan n = {};
  n.chunk = part_chunk(int64_t(R) * Hkv, max_blocks);
  n.own_parts = (max_blocks + n.chunk - 1) / n.chunk;
  if (prefix_blocks > 0) {
    n.row_tiles = int((int64_t(R) * (Hq / Hkv) + part::ROWS - 1) / part::ROWS);
    n.prefix_chunk = part_chunk(int64_t(n.row_tiles) * Hkv, prefix_blocks);
    n.prefix_parts = (prefix_blocks + n.prefix_chunk - 1) / n.prefix_chunk;
  }
  const size_t rows = size_t(R) * Hq * (n.own_parts + n.prefix_parts);
  n.off_lse = align256(rows * d * sizeof(float));
  n.off_scores = n.off_lse + align256(rows * sizeof(float));
  n.bytes = n.off_scores + (scored ? align256(size_t(R) * Hq * max_blocks * part::BS * sizeof(float)) : 0);
  return n;
}

bool part_sizes(int R, int Hq, int Hkv, int d, int max_blocks, int block_size) {
  return R > 0 && Hq > 0 && Hkv > 0 && d > 0 && max_blocks > 0 && block_size > 0 && Hq % Hkv == 0;
}

template <int D, bool PREFIX, bool SCORED>
fa_status part_launch(const CUtensorMap& mk, const CUtensorMap& mv, const PartParams& prm, dim3 grid, cudaStream_t st) {
  auto kern = fa_decode_part_kernel<D, PREFIX, SCORED>;
  if (set_smem(kern, part::Cfg<D>::SMEM) != cudaSuccess) return FA_ERR_CUDA;
  if (launch_pdl(kern, grid, dim3(part::WARPS * 32), part::Cfg<D>::SMEM, st, mk, mv, prm) != cudaSuccess)
    return FA_ERR_CUDA;
  return FA_OK;
}

template <int D>
fa_status part_run(const CUtensorMap& mk, const CUtensorMap& mv, const PartParams& prm, const PartPlan& n, bool scored,
                   cudaStream_t st) {
  fa_status s = FA_OK;
  if (prm.pbt) s = part_launch<D, true, false>(mk, mv, prm, dim3(n.prefix_parts, prm.Hkv, n.row_tiles), st);
  if (s != FA_OK) return s;
  const dim3 own(n.own_parts, prm.Hkv, prm.R);
  s = scored ? part_launch<D, false, true>(mk, mv, prm, own, st) : part_launch<D, false, false>(mk, mv, prm, own, st);
  if (s != FA_OK) return s;
  if (scored && launch_pdl(fa_decode_weights_kernel, dim3((prm.max_blocks * part::BS + 255) / 256, prm.Hkv, prm.R),
                           dim3(256), 0, st, prm) != cudaSuccess)
    return FA_ERR_CUDA;
  if (launch_pdl(fa_decode_merge_kernel<D>, dim3(unsigned(prm.R * prm.Hq)), dim3(D), 0, st, prm) != cudaSuccess)
    return FA_ERR_CUDA;
  return launched();
}

fa_status part_check(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                     const int* ctx_lens, const void* o, const float* lse, int R, int Hq, int Hkv, int d, int block_size,
                     int max_blocks, int num_blocks, float scale, fa_dtype dtype) {
  if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !o) return FA_ERR_INVALID_ARG;
  if (!part_sizes(R, Hq, Hkv, d, max_blocks, block_size) || num_blocks <= 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
      !aligned(block_table, 4) || !aligned(ctx_lens, 4) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_BF16 || (d != 64 && d != 128) || block_size != part::BS) return FA_ERR_UNSUPPORTED;
  if (Hq / Hkv > part::ROWS || R > 65535 || Hkv > 65535 || int64_t(R) * Hq > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  if (int64_t(num_blocks) * Hkv * part::BS > 0x7fffffff || int64_t(max_blocks) * part::BS > 0x7fffffff)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status part_call(const void* q, const void* k_cache, const void* v_cache, const int* prefix_table,
                    const int* prefix_len, const int* block_table, const int* ctx_lens, float* weights, void* o,
                    float* lse, int R, int Hq, int Hkv, int d, int max_prefix_blocks, int max_blocks, int num_blocks,
                    float scale, void* workspace, size_t workspace_bytes, void* stream) {
  const PartPlan n = part_plan(R, Hq, Hkv, d, max_blocks, max_prefix_blocks, weights != nullptr);
  if (n.row_tiles > 65535) return FA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < n.bytes || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  PartParams prm{static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(o), lse,
                 reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + n.off_lse),
                 reinterpret_cast<float*>(ws + n.off_scores), weights, block_table, ctx_lens, prefix_table, prefix_len,
                 R, Hq, Hkv, max_blocks, max_prefix_blocks, num_blocks, n.own_parts + n.prefix_parts, n.prefix_parts,
                 n.chunk, n.prefix_chunk, scale * 1.4426950408889634f, g_wait_ns};
  CUtensorMap mk, mv;
  const long cache_rows = long(num_blocks) * Hkv * part::BS;
  if (!make_map_cache(&mk, k_cache, cache_rows, d) || !make_map_cache(&mv, v_cache, cache_rows, d)) return FA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 64 ? part_run<64>(mk, mv, prm, n, weights != nullptr, st)
                 : part_run<128>(mk, mv, prm, n, weights != nullptr, st);
}

// Rows that may move of one (request, kv head): min(keep, n - keep) for n up to max_blocks * 16.
int evict_cap(int max_blocks, int keep) {
  const int64_t M = int64_t(max_blocks) * evict::BS;
  return int(std::max<int64_t>(0, std::min<int64_t>(keep, M - keep)));
}

}  // namespace

extern "C" {

fa_status fa_qk_norm_rope(const void* q, const void* k, const int64_t* q_strides, const int64_t* k_strides,
                          const void* q_weight, const void* k_weight, const int* positions, int64_t pos_axis_stride,
                          int64_t pos_batch_stride, const double* inv_freq, void* q_out, void* k_out, int B, int Hq,
                          int Hkv, int N, int d, int rotary_dim, const int* sections, int n_axes, int interleaved,
                          float eps, fa_dtype dtype, void* stream) {
  const fa_status s = rope_check(positions, inv_freq, B, Hq, Hkv, N, d, rotary_dim, sections, n_axes, interleaved, eps,
                                 dtype);
  if (s != FA_OK) return s;
  if (!rope_rows(q, q_strides, dtype) || !rope_rows(k, k_strides, dtype)) return FA_ERR_INVALID_ARG;
  if (!q_out || !k_out || !aligned(q_out, 16) || !aligned(k_out, 16)) return FA_ERR_INVALID_ARG;
  if (!q_weight != !k_weight || !aligned(q_weight, 2) || !aligned(k_weight, 2)) return FA_ERR_INVALID_ARG;
  RopeParams prm{{q, k, nullptr},
                 {q_strides[0], k_strides[0], 0},
                 {q_strides[1], k_strides[1], 0},
                 {q_strides[2], k_strides[2], 0},
                 {q_weight, k_weight},
                 positions, inv_freq,
                 {q_out, k_out},
                 pos_axis_stride, pos_batch_stride, B, Hq, Hkv, N, rotary_dim, sections[0],
                 n_axes > 1 ? sections[0] + sections[1] : sections[0], eps, 1, 1, 1,
                 nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == FA_DTYPE_BF16 ? rope_by_d<__nv_bfloat16>(prm, d, interleaved, st)
                                : rope_by_d<float>(prm, d, interleaved, st);
}

fa_status fa_qk_norm_rope_append(const void* q, const void* k, const void* v, const int64_t* q_strides,
                                 const int64_t* k_strides, const int64_t* v_strides, const void* q_weight,
                                 const void* k_weight, const int* positions, int64_t pos_axis_stride,
                                 int64_t pos_batch_stride, const double* inv_freq, void* k_cache, void* v_cache,
                                 const int* block_table, const int* ctx_lens, const int* q_lens, void* q_out, int R,
                                 int Hq, int Hkv, int Nq_max, int d, int block_size, int max_blocks_per_seq,
                                 int num_blocks, int rotary_dim, const int* sections, int n_axes, int interleaved,
                                 float eps, fa_dtype dtype, void* stream) {
  const fa_status s = rope_check(positions, inv_freq, R, Hq, Hkv, Nq_max, d, rotary_dim, sections, n_axes, interleaved,
                                 eps, dtype);
  if (s != FA_OK) return s;
  if (block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_BF16 || d == 256 || block_size != 16) return FA_ERR_UNSUPPORTED;
  if (int64_t(max_blocks_per_seq) * 16 > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  if (!rope_rows(q, q_strides, dtype) || !rope_rows(k, k_strides, dtype) || !rope_rows(v, v_strides, dtype))
    return FA_ERR_INVALID_ARG;
  if (!q_out || !k_cache || !v_cache || !block_table || !ctx_lens || !q_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_table, 4) ||
      !aligned(ctx_lens, 4) || !aligned(q_lens, 4))
    return FA_ERR_INVALID_ARG;
  if (!q_weight != !k_weight || !aligned(q_weight, 2) || !aligned(k_weight, 2)) return FA_ERR_INVALID_ARG;
  RopeParams prm{{q, k, v},
                 {q_strides[0], k_strides[0], v_strides[0]},
                 {q_strides[1], k_strides[1], v_strides[1]},
                 {q_strides[2], k_strides[2], v_strides[2]},
                 {q_weight, k_weight},
                 positions, inv_freq,
                 {q_out, nullptr},
                 pos_axis_stride, pos_batch_stride, R, Hq, Hkv, Nq_max, rotary_dim, sections[0],
                 n_axes > 1 ? sections[0] + sections[1] : sections[0], eps, 1, 1, 1,
                 block_table, ctx_lens, q_lens, k_cache, v_cache, max_blocks_per_seq, num_blocks};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (d) {
    case 64: return rope_launch<__nv_bfloat16, 64, true>(prm, interleaved, st);
    case 96: return rope_launch<__nv_bfloat16, 96, true>(prm, interleaved, st);
    default: return rope_launch<__nv_bfloat16, 128, true>(prm, interleaved, st);
  }
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  return d <= 0 ? 0 : align256(size_t(kRopeBwdCtas) * d * sizeof(float));
}

fa_status fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, fa_dtype dout_dtype, const void* q, const void* k,
                              const int64_t* q_strides, const int64_t* k_strides, const void* q_weight,
                              const void* k_weight, const int* positions, int64_t pos_axis_stride,
                              int64_t pos_batch_stride, const double* inv_freq, void* dq, void* dk,
                              const int64_t* dq_strides, const int64_t* dk_strides, fa_dtype grad_dtype, float* dq_weight,
                              float* dk_weight, int B, int Hq, int Hkv, int N, int d, int rotary_dim,
                              const int* sections, int n_axes, int interleaved, float eps, fa_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const fa_status s = rope_check(positions, inv_freq, B, Hq, Hkv, N, d, rotary_dim, sections, n_axes, interleaved, eps,
                                 dtype);
  if (s != FA_OK) return s;
  if (!dq_out || !dk_out || !aligned(dq_out, 16) || !aligned(dk_out, 16)) return FA_ERR_INVALID_ARG;
  if (!q_weight != !k_weight || !aligned(q_weight, 2) || !aligned(k_weight, 2)) return FA_ERR_INVALID_ARG;
  if (dout_dtype != FA_DTYPE_F32 && dout_dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
  if (grad_dtype != FA_DTYPE_F32 && grad_dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_DTYPE_F32 && (dout_dtype != FA_DTYPE_F32 || grad_dtype != FA_DTYPE_F32)) return FA_ERR_UNSUPPORTED;
  if (!rope_rows(q, q_strides, dtype) || !rope_rows(k, k_strides, dtype) || !rope_rows(dq, dq_strides, grad_dtype) ||
      !rope_rows(dk, dk_strides, grad_dtype))
    return FA_ERR_INVALID_ARG;
  // no two rows of a gradient may share memory
  const int n[2][3] = {{B, Hq, N}, {B, Hkv, N}};
  for (int t = 0; t < 2; ++t)
    for (int i = 0; i < 3; ++i)
      if (n[t][i] > 1 && (t ? dk_strides : dq_strides)[i] < d) return FA_ERR_INVALID_ARG;
  if (q_weight) {
    if (!dq_weight || !dk_weight || !aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return FA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < fa_qk_norm_rope_bwd_workspace_size(d) || !aligned(workspace, 256))
      return FA_ERR_WORKSPACE;
  }
  RopeBwdParams prm{{dq_out, dk_out},
                    {q, k},
                    {q_strides[0], k_strides[0]},
                    {q_strides[1], k_strides[1]},
                    {q_strides[2], k_strides[2]},
                    {q_weight, k_weight},
                    positions, inv_freq,
                    {dq, dk},
                    {dq_strides[0], dk_strides[0]},
                    {dq_strides[1], dk_strides[1]},
                    {dq_strides[2], dk_strides[2]},
                    static_cast<float*>(workspace),
                    pos_axis_stride, pos_batch_stride, B, {Hq, Hkv}, N, rotary_dim, sections[0],
                    n_axes > 1 ? sections[0] + sections[1] : sections[0], eps, 1, {1, 1}, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == FA_DTYPE_F32) return rope_bwd_by_d<float, float, float>(prm, d, interleaved, dq_weight, dk_weight, st);
  using bf = __nv_bfloat16;
  if (dout_dtype == FA_DTYPE_F32)
    return grad_dtype == FA_DTYPE_F32 ? rope_bwd_by_d<bf, float, float>(prm, d, interleaved, dq_weight, dk_weight, st)
                                      : rope_bwd_by_d<bf, float, bf>(prm, d, interleaved, dq_weight, dk_weight, st);
  return grad_dtype == FA_DTYPE_F32 ? rope_bwd_by_d<bf, bf, float>(prm, d, interleaved, dq_weight, dk_weight, st)
                                    : rope_bwd_by_d<bf, bf, bf>(prm, d, interleaved, dq_weight, dk_weight, st);
}

size_t fa_paged_decode_shared_workspace_size(int R, int Hq, int Hkv, int d, int max_prefix_blocks,
                                             int max_blocks_per_seq, int block_size) {
  if (!part_sizes(R, Hq, Hkv, d, max_blocks_per_seq, block_size) || max_prefix_blocks <= 0) return 0;
  return part_plan(R, Hq, Hkv, d, max_blocks_per_seq, max_prefix_blocks, false).bytes;
}

fa_status fa_paged_decode_shared(const void* q, const void* k_cache, const void* v_cache, const int* prefix_table,
                                 const int* prefix_len, const int* block_table, const int* ctx_lens, void* o, float* lse,
                                 int R, int Hq, int Hkv, int d, int block_size, int max_prefix_blocks,
                                 int max_blocks_per_seq, int num_blocks, float scale, fa_dtype dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!prefix_table || !prefix_len || max_prefix_blocks <= 0 || !aligned(prefix_table, 4) || !aligned(prefix_len, 4))
    return FA_ERR_INVALID_ARG;
  const fa_status s = part_check(q, k_cache, v_cache, block_table, ctx_lens, o, lse, R, Hq, Hkv, d, block_size,
                                 max_blocks_per_seq, num_blocks, scale, dtype);
  if (s != FA_OK) return s;
  if (int64_t(max_prefix_blocks) * part::BS > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  return part_call(q, k_cache, v_cache, prefix_table, prefix_len, block_table, ctx_lens, nullptr, o, lse, R, Hq, Hkv, d,
                   max_prefix_blocks, max_blocks_per_seq, num_blocks, scale, workspace, workspace_bytes, stream);
}

size_t fa_paged_decode_scored_workspace_size(int R, int Hq, int Hkv, int d, int max_blocks_per_seq, int block_size) {
  if (!part_sizes(R, Hq, Hkv, d, max_blocks_per_seq, block_size)) return 0;
  return part_plan(R, Hq, Hkv, d, max_blocks_per_seq, 0, true).bytes;
}

fa_status fa_paged_decode_scored(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                                 const int* ctx_lens, float* weights, void* o, float* lse, int R, int Hq, int Hkv,
                                 int d, int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                                 fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!weights || !aligned(weights, 4)) return FA_ERR_INVALID_ARG;
  const fa_status s = part_check(q, k_cache, v_cache, block_table, ctx_lens, o, lse, R, Hq, Hkv, d, block_size,
                                 max_blocks_per_seq, num_blocks, scale, dtype);
  if (s != FA_OK) return s;
  return part_call(q, k_cache, v_cache, nullptr, nullptr, block_table, ctx_lens, weights, o, lse, R, Hq, Hkv, d, 0,
                   max_blocks_per_seq, num_blocks, scale, workspace, workspace_bytes, stream);
}

size_t fa_paged_evict_workspace_size(int R, int Hkv, int max_blocks_per_seq, int keep) {
  if (R <= 0 || Hkv <= 0 || max_blocks_per_seq <= 0 || keep <= 0) return 0;
  const size_t n = size_t(R) * Hkv;
  return align256(n * sizeof(int)) + align256(n * 2 * evict_cap(max_blocks_per_seq, keep) * sizeof(int));
}

fa_status fa_paged_evict(void* k_cache, void* v_cache, const int* block_table, const int* ctx_lens, const int* seq_lens,
                         const float* weights, const int* slot_pos, float* weights_out, int* slot_pos_out, int* new_ctx,
                         int R, int Hkv, int d, int block_size, int max_blocks_per_seq, int num_blocks, int keep,
                         int recent, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!k_cache || !v_cache || !block_table || !ctx_lens || !seq_lens || !weights || !slot_pos || !weights_out ||
      !slot_pos_out || !new_ctx)
    return FA_ERR_INVALID_ARG;
  if (R <= 0 || Hkv <= 0 || d <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
    return FA_ERR_INVALID_ARG;
  if (keep <= 0 || recent < 0 || recent > keep) return FA_ERR_INVALID_ARG;
  const void* small[] = {block_table, ctx_lens, seq_lens, weights, slot_pos, weights_out, slot_pos_out, new_ctx};
  for (const void* p : small)
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return FA_ERR_INVALID_ARG;
  // the selection reads its inputs while it writes its outputs
  if (weights_out == weights || slot_pos_out == slot_pos || new_ctx == ctx_lens || new_ctx == seq_lens)
    return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_BF16 || (d != 64 && d != 96 && d != 128 && d != 256) || block_size != evict::BS)
    return FA_ERR_UNSUPPORTED;
  if (R > 65535 || Hkv > 65535 || int64_t(max_blocks_per_seq) * evict::BS > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < fa_paged_evict_workspace_size(R, Hkv, max_blocks_per_seq, keep) ||
      !aligned(workspace, 256))
    return FA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  EvictParams prm{block_table, ctx_lens, seq_lens, weights, slot_pos, weights_out, slot_pos_out, new_ctx,
                  reinterpret_cast<int*>(ws + align256(size_t(R) * Hkv * sizeof(int))), reinterpret_cast<int*>(ws),
                  static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), R, Hkv, max_blocks_per_seq, num_blocks,
                  keep, recent, evict_cap(max_blocks_per_seq, keep), d * 2 / 16};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pdl(fa_evict_select_kernel, dim3(Hkv, R), dim3(evict::THREADS), 0, st, prm) != cudaSuccess)
    return FA_ERR_CUDA;
  if (prm.cap > 0) {
    const int64_t pieces = int64_t(prm.cap) * 2 * prm.row16;
    const int64_t want = std::max<int64_t>(1, 148 * 8 / (int64_t(R) * Hkv));
    const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(want, (pieces + 255) / 256)));
    if (launch_pdl(fa_evict_move_kernel, dim3(grid, Hkv, R), dim3(256), 0, st, prm) != cudaSuccess) return FA_ERR_CUDA;
  }
  return launched();
}

}  // extern "C"
