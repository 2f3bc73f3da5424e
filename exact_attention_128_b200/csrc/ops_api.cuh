// ops_api.cuh — entry points of the operators around attention (include/fa.h): the norm with the
// position rotation, the decode steps over pieces of the cache, and the eviction.  Included by
// fa_api.cu, whose helpers (alignment, TMA descriptors, launches) it uses.
#pragma once

namespace {

// A kernel whose launches need attributes (dynamic shared memory past 48 KB, the SM's memory as
// shared memory): they are set at its first launch on each device, and again should a launch need
// more memory or fail (a reset device has forgotten them).  Never to less than before: threads may
// launch at once.
class Prepared {
 public:
  template <typename... KArgs, typename... Args>
  cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t st, const Args&... args) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    std::atomic<int>& have = smem_[dev & 63];
    if (have.load(std::memory_order_acquire) >= smem) {
      if (launch_pdl(kernel, grid, block, smem, st, args...) == cudaSuccess) return cudaSuccess;
      cudaGetLastError();
    }
    std::lock_guard<std::mutex> lock(setting_);
    const int most = std::max(smem, have.load(std::memory_order_relaxed));
    if (cudaError_t e = set_smem(kernel, most)) return e;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             cudaSharedmemCarveoutMaxShared))
      return e;
    have.store(most, std::memory_order_release);
    return launch_pdl(kernel, grid, block, smem, st, args...);
  }

 private:
  std::atomic<int> smem_[64] = {};  // of each device; 0: not launched yet
  std::mutex setting_;
};

constexpr int kSms = 148;  // SMs that work is divided for
constexpr int kMaxTokens = 1 << 30;  // of a table, so that token indexes plus a grid's stride stay below 2^31

// Rotation arguments that every rotary entry point shares: sizes, then one of `out` launches.
fa_status rope_check(const int* positions, const double* inv_freq, int B, int Hq, int Hkv, int N, int d, int rotary_dim,
                     const int* sections, int n_axes, int interleaved, float eps, int dtype) {
  if (!positions || !inv_freq) return FA_ERR_INVALID_ARG;
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

// Both weights, or neither.
bool rope_weights(const void* q, const void* k, int dtype) {
  const size_t size = dtype == FA_DTYPE_F32 ? 4 : 2;
  return !q == !k && aligned(q, size) && aligned(k, size);
}

// Rows of 16-byte pieces at any (batch, head, token): base and strides (elements) are multiples of 16 bytes.
bool rope_rows(const void* p, const int64_t* strides, int dtype) {
  const int64_t per = dtype == FA_DTYPE_F32 ? 4 : 8;
  if (!p || !aligned(p, 16)) return false;
  for (int i = 0; i < 3; ++i)
    if (strides[i] < 0 || strides[i] % per != 0) return false;
  return true;
}

// Whether rows of d values at these strides may share memory: each dimension's step has to clear all that the
// dimensions of smaller steps cover, as in any permuted slice of a dense array.
bool rows_overlap(const int64_t* strides, int B, int H, int N, int d) {
  std::pair<int64_t, int> dims[3] = {{strides[0], B}, {strides[1], H}, {strides[2], N}};
  std::sort(dims, dims + 3);
  __int128 covered = d;
  for (const auto& [step, n] : dims) {
    if (n <= 1) continue;
    if (step < covered) return true;
    covered += __int128(step) * (n - 1);
  }
  return false;
}

template <typename T, int D, bool PAGED>
fa_status rope_launch(RopeParams& prm, bool inter, cudaStream_t st) {
  const int64_t tokens = int64_t(prm.B) * prm.N;
  constexpr int TOKENS = rope::Cfg<D>::TOKENS;
  const int heads = prm.Hq + (PAGED ? 2 : 1) * prm.Hkv;
  // Warps that share a token group: about 10 heads each, and all eight while that leaves
  // SMs without a CTA.
  const int64_t tgroups = (tokens + TOKENS - 1) / TOKENS;
  int sharers = 8;
  while (sharers > 1 && heads < 10 * sharers && tgroups * (sharers / 2) >= int64_t(8) * 4 * kSms) sharers /= 2;
  prm.groups = 8 / sharers;
  const int64_t grid = (tgroups + prm.groups - 1) / prm.groups;
  if (tokens > 0x7fffff00 || grid > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  auto kern = inter ? fa_qk_norm_rope_kernel<T, D, true, PAGED> : fa_qk_norm_rope_kernel<T, D, false, PAGED>;
  const int smem = (sizeof(T) == 4 ? rope::FWD_STAGES_F32 : rope::FWD_STAGES) * rope::Slot<T, sizeof(T) == 4>::BYTES +
                   (prm.groups * rope::TABLE + 8 * rope::Cfg<D>::L) * 16;
  static Prepared prepared[2];
  if (prepared[inter].launch(kern, dim3(unsigned(grid)), dim3(rope::THREADS), smem, st, prm) != cudaSuccess)
    return FA_ERR_CUDA;
  return launched();
}

constexpr int kRopeBwdCtas = kSms * 2;  // CTAs of the backward kernel, at most

template <typename T, typename TG, typename TO, int D>
fa_status rope_bwd_launch(RopeBwdParams& prm, bool inter, float* dwq, float* dwk, cudaStream_t st) {
  const int64_t tokens = int64_t(prm.B) * prm.N;
  if (tokens > 0x7fffff00) return FA_ERR_UNSUPPORTED;
  constexpr int TOKENS = rope::Cfg<D>::TOKENS, WARPS = rope::THREADS / 32;
  // Heads per unit and CTAs of q and of k: units go to warps in turn, so the slowest warp has
  // ceil(units / warps) of them, each worth its heads and about two more for its cosines.  Of all
  // ways to cut the heads, the one whose slowest warp is the fastest.  The CTAs are shared out as if a
  // unit cost four heads more: k's units have few heads, and a unit's first rows arrive with nothing
  // else to do (12 + 3 heads of 256, 4 x 8192 tokens: 144 us with two, 136 with four; 24 + 6 heads of 128:
  // 133 and 130; of 2 x 2305 tokens 27.5 and 28.9).
  const int64_t tgroups = (tokens + TOKENS - 1) / TOKENS;
  int64_t best = INT64_MAX;
  int ctas[2] = {1, 1};
  for (int cq = rope::MAX_CHUNK; cq >= 1; cq /= 2)
    for (int ck = rope::MAX_CHUNK; ck >= 1; ck /= 2) {
      const int most[2] = {cq, ck};
      int chunk[2], chunks[2], n[2];
      int64_t units[2], work[2], time = 0;
      for (int k = 0; k < 2; ++k) {
        chunks[k] = (prm.H[k] + most[k] - 1) / most[k];
        chunk[k] = (prm.H[k] + chunks[k] - 1) / chunks[k];
        units[k] = tgroups * chunks[k];
        work[k] = units[k] * (chunk[k] + 4);
      }
      for (int k = 0; k < 2; ++k) {
        const int64_t share = int64_t(double(kRopeBwdCtas) * double(work[k]) / double(work[0] + work[1]) + 0.5);
        n[k] = int(std::min<int64_t>(std::max<int64_t>(1, std::min<int64_t>(kRopeBwdCtas - 1, share)),
                                     (units[k] + WARPS - 1) / WARPS));
        time = std::max(time, (units[k] + n[k] * WARPS - 1) / (n[k] * WARPS) * (chunk[k] + 2));
      }
      if (n[0] + n[1] > kRopeBwdCtas) --n[n[0] > n[1] ? 0 : 1];  // (both shares rounded up)
      if (time < best) {
        best = time;
        for (int k = 0; k < 2; ++k) {
          prm.chunk[k] = chunk[k];
          prm.chunks[k] = chunks[k];
          ctas[k] = n[k];
        }
      }
    }
  prm.ctas_q = ctas[0];
  auto kern = inter ? fa_qk_norm_rope_bwd_kernel<T, TG, TO, D, true> : fa_qk_norm_rope_bwd_kernel<T, TG, TO, D, false>;
  constexpr int SMEM = rope::BWD_STAGES * rope::THREADS * 16 * int(sizeof(T) + sizeof(TG));
  static_assert(SMEM >= WARPS * D * 4, "the weight-gradient sums reuse the slots");
  static Prepared prepared[2];
  const dim3 grid(unsigned(ctas[0] + ctas[1]));
  if (prepared[inter].launch(kern, grid, dim3(rope::THREADS), SMEM, st, prm) != cudaSuccess) return FA_ERR_CUDA;
  if (prm.w[0] && launch_pdl(fa_qk_norm_rope_dw_kernel, dim3(D / 8, 2), dim3(512), 0, st,
                             static_cast<const float*>(prm.part), dwq, dwk, D, ctas[0], ctas[0] + ctas[1]) !=
                                 cudaSuccess)
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

// Blocks of a piece when `sets` sets of rows walk up to `blocks` blocks each: enough pieces for 12
// CTAs on each SM, which holds 3 (tables are wider than most contexts; 64 requests of 512 to 8192
// tokens, 2 kv heads: 6, 12 and 24 CTAs took 72, 67 and 69 us), at least MIN_CHUNK blocks a piece
// and at most MAX_PARTS pieces.
int part_chunk(int64_t sets, int64_t blocks) {
  const int64_t want = std::max<int64_t>(1, (kSms * 12 + sets - 1) / sets);
  const int64_t pieces = std::min<int64_t>(part::MAX_PARTS, want);
  const int64_t c = std::max<int64_t>(part::MIN_CHUNK, (blocks + pieces - 1) / pieces);
  return int((c + part::WARPS - 1) / part::WARPS * part::WARPS);
}

// Whether the prefix goes to the tensor-core kernel, whose CTAs work on 256 rows at a time, or to
// 16-row pieces, which read the prefix again for each 16 rows but need no kernel of their own.  By
// the rows of a kv head, the sets of 16 rows over all kv heads, the blocks of the prefix's table, and
// the work, sets x blocks.  A step with 1 to 64 own tokens a request, replayed from a graph, pieces /
// tensor cores in us (heads as query/kv; P tokens):
//   d = 128, few rows: 1 request of 4/1, P 2000 8.8 / 11.3, 16384 12.7 / 18.0; 2 of 48/8 (12 rows), P 3000
//     14.2 / 16.9, 32768 48.4 / 51.5
//   one kv head, up to 4 sets: 4 of 4/1, P 300 11.7 / 10.7, 700 13.3 / 10.6, 4000 13.1 / 12.2, 16384 16.3 / 18.0; 16 of
//     4/1, P 500 13.1 / 11.4, 6000 15.6 / 13.9
//   60 to 128 blocks: 4 of 4/1, P 2000 12.8 / 11.3; 4 of 32/8, P 1000 13.4 / 12.1, 2000 15.0 / 14.1; 64 of
//     8/2, P 1000 19.5 / 16.4; 8 of 12/2, P 2000 13.4 / 12.3
//   more blocks, less than 4 sets or 2000 of work: 8 of 8/2, P 3000 13.6 / 14.7, 4000 13.7 / 15.1; 4 of 8/2,
//     P 8000 14.6 / 16.3, 32768 20.1 / 23.0; 4 of 32/8, P 3000 15.7 / 17.6; but 8 of 8/2, P 6000 15.6 / 14.1
//   more blocks, more work: 16 of 8/2, P 4000 18.8 / 15.8; 4 of 32/8, P 4000 18.7 / 17.5, 6000 19.1 / 19.8,
//     16384 37.4 / 32.2; 64 of 32/8, P 16384 149 / 43.4
//   fewer blocks: 64 of 8/2, P 300 14.5 / 20.9, 700 16.7 / 20.9; 200 of 8/1, P 300 19.3 / 22.2; 24 of 32/8, P 700
//     20.0 / 17.6; 128 of 32/8, P 200 31.7 / 23.6; but 4 of 32/8, P 500 13.2 / 11.7; many
//     sets: 256 of 32/8, P 40 41.1 / 33.4, 100 43.0 / 33.7
//   d = 64 (pieces hold fewer registers): 4 of 32/8, P 32768 22.9 / 34.9; 16 of 8/2, P 8000 13.3 / 14.7; 8 of
//     32/8, P 2000 11.6 / 12.3, 4000 15.1 / 14.9, 16384 25.6 / 23.4; 24 of 32/8, P 1000 14.4 / 13.0; 64 of 32/8,
//     P 700 18.6 / 19.9, 2000 27.8 / 19.7, 16384 83.2 / 34.9; 64 of 8/2, P 3000 18.4 / 17.6; 256 of 32/8,
//     P 100 24.2 / 21.8, 300 34.9 / 24.4
bool prefix_on_tensor_cores(int64_t rows, int Hkv, int d, int blocks) {
  const int64_t sets = (rows + part::ROWS - 1) / part::ROWS * Hkv, work = sets * blocks;
  if (d == 64) return sets >= 512 || (sets >= 16 && work >= (blocks >= 60 ? 3000 : 8000));
  if (rows < part::ROWS) return false;
  if (Hkv == 1 && sets <= 4 && blocks >= 16 && blocks <= 400) return true;  // (no CTA works on two heads' tiles)
  return (blocks >= 60 && blocks <= 128) || (sets >= 4 && work >= 2000) || sets >= 256;
}

struct PartPlan {
  int chunk, prefix_chunk, own_parts, prefix_parts, row_tiles;
  int RT, pairs, pre_parts;  // tensor-core prefix: requests per row tile, tile pairs, results per item
  size_t off_lse, off_scores, off_pre_o, off_pre_lse, bytes;
};

PartPlan part_plan(int R, int Hq, int Hkv, int d, int max_blocks, int prefix_blocks, bool scored) {
  PartPlan n = {};
  const int G = Hq / Hkv;
  n.chunk = part_chunk(int64_t(R) * Hkv, max_blocks);
  n.own_parts = (max_blocks + n.chunk - 1) / n.chunk;
  const int64_t rows = int64_t(R) * G, row_tiles = (rows + part::ROWS - 1) / part::ROWS;
  if (prefix_blocks > 0 && G <= part::ROWS && prefix_on_tensor_cores(rows, Hkv, d, prefix_blocks)) {
    n.RT = 128 / G;
    n.pairs = (R + 2 * n.RT - 1) / (2 * n.RT);
    n.pre_parts = int((part::PREFIX_CTAS + int64_t(n.pairs) * Hkv - 1) / (int64_t(n.pairs) * Hkv)) + 1;
  } else if (prefix_blocks > 0) {
    n.row_tiles = int(row_tiles);
    n.prefix_chunk = part_chunk(int64_t(n.row_tiles) * Hkv, prefix_blocks);
    n.prefix_parts = (prefix_blocks + n.prefix_chunk - 1) / n.prefix_chunk;
  }
  const size_t results = size_t(R) * Hq * (n.own_parts + n.prefix_parts);
  n.off_lse = align256(results * d * sizeof(float));
  n.off_scores = n.off_lse + align256(results * sizeof(float));
  n.off_pre_o = n.off_scores + (scored ? align256(size_t(R) * Hq * max_blocks * part::BS * sizeof(float)) : 0);
  const size_t pre_rows = size_t(n.pairs) * Hkv * n.pre_parts * 256;
  n.off_pre_lse = n.off_pre_o + pre_rows * d * sizeof(float);
  n.bytes = n.off_pre_lse + pre_rows * sizeof(float);
  return n;
}

// 3-D map of q [R, Hq, d] with a box of one row tile's heads and requests.
bool make_map_rows(CUtensorMap* m, const void* q, int d, int Hq, int R, int G, int RT) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(Hq), cuuint64_t(R)};
  cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(d) * 2 * cuuint64_t(Hq)};
  cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(RT)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool part_sizes(int R, int Hq, int Hkv, int d, int max_blocks, int block_size) {
  return R > 0 && Hq > 0 && Hkv > 0 && d > 0 && max_blocks > 0 && block_size > 0 && Hq % Hkv == 0;
}

template <int D>
fa_status prefix_launch(const CUtensorMap& mk, const CUtensorMap& mv, const PartParams& prm, const PartPlan& n,
                        int withhold, cudaStream_t st) {
  using C = PrefixCfg<D>;
  CUtensorMap mq;
  const int G = prm.Hq / prm.Hkv;
  if (!make_map_rows(&mq, prm.q, D, prm.Hq, prm.R, G, n.RT)) return FA_ERR_CUDA;
  const PrefixParams pp{prm.pbt, prm.plen, const_cast<float*>(prm.pre_o), const_cast<float*>(prm.pre_lse), prm.R,
                        prm.Hkv, G, n.RT, n.pairs * prm.Hkv, n.pairs, n.pre_parts, prm.prefix_blocks, prm.num_blocks,
                        prm.scale_log2, prm.wait_ns, withhold};
  // (all of the SM's memory as shared memory: the CTA of the next grid has to find room beside this one)
  static Prepared prepared;
  if (prepared.launch(fa_prefix_kernel<D>, dim3(part::PREFIX_CTAS), dim3(C::THREADS), C::SMEM, st, mq, mk, mv, pp) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  return FA_OK;
}

template <int D>
fa_status part_run(const CUtensorMap& mk, const CUtensorMap& mv, PartParams& prm, const PartPlan& n, bool scored,
                   int withhold, cudaStream_t st) {
  if (prm.pre_o) {
    const fa_status s = prefix_launch<D>(mk, mv, prm, n, withhold, st);
    if (s != FA_OK) return s;
    prm.late_wait = true;
  }
  const int64_t pre = int64_t(n.prefix_parts) * prm.Hkv * n.row_tiles, own = int64_t(n.own_parts) * prm.Hkv * prm.R;
  if (pre + own > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  prm.n_prefix = int(pre);
  static Prepared prepared[2];
  auto kern = scored ? fa_decode_part_kernel<D, true> : fa_decode_part_kernel<D, false>;
  if (prepared[scored].launch(kern, dim3(unsigned(pre + own)), dim3(part::WARPS * 32), part::Cfg<D>::SMEM, st, mk, mv,
                              prm) != cudaSuccess)
    return FA_ERR_CUDA;
  // warps that share a row of the join: one for each 8 pieces it may have
  const int most = n.own_parts + n.prefix_parts + n.pre_parts;
  const int strands = most > 32 ? 8 : most > 16 ? 4 : most > 8 ? 2 : 1;
  const int64_t joins = (int64_t(prm.R) * prm.Hq * strands + 7) / 8;
  const int64_t sets = int64_t(prm.R) * prm.Hkv;
  // spans of weights: four CTAs for each SM in all, at most one per JOIN_TOKENS tokens
  const int64_t tokens = int64_t(prm.max_blocks) * part::BS;
  const int64_t spans = std::min<int64_t>((tokens + part::JOIN_TOKENS - 1) / part::JOIN_TOKENS,
                                          std::max<int64_t>(1, kSms * 4 / sets));
  const int64_t grid = joins + (scored ? sets * spans : 0);
  if (grid > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  auto join = scored ? fa_decode_join_kernel<D, true> : fa_decode_join_kernel<D, false>;
  if (launch_pdl(join, dim3(unsigned(grid)), dim3(256), 0, st, prm, int(joins), strands, int(spans)) != cudaSuccess)
    return FA_ERR_CUDA;
  return launched();
}

fa_status part_check(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                     const int* ctx_lens, const void* o, const float* lse, int R, int Hq, int Hkv, int d,
                     int block_size, int max_blocks, int num_blocks, float scale, int dtype) {
  if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !o) return FA_ERR_INVALID_ARG;
  if (!part_sizes(R, Hq, Hkv, d, max_blocks, block_size) || num_blocks <= 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
      !aligned(block_table, 4) || !aligned(ctx_lens, 4) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_BF16 || (d != 64 && d != 128) || block_size != part::BS) return FA_ERR_UNSUPPORTED;
  if (Hq / Hkv > part::ROWS || R > 65535 || Hkv > 65535 || int64_t(R) * Hq > 0x7fffffff) return FA_ERR_UNSUPPORTED;
  if (int64_t(num_blocks) * Hkv * part::BS > 0x7fffffff || int64_t(max_blocks) * part::BS > kMaxTokens)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status part_call(const void* q, const void* k_cache, const void* v_cache, const int* prefix_table,
                    const int* prefix_len, const int* block_table, const int* ctx_lens, float* weights, void* o,
                    float* lse, int R, int Hq, int Hkv, int d, int max_prefix_blocks, int max_blocks, int num_blocks,
                    float scale, void* workspace, size_t workspace_bytes, void* stream, int withhold = INT_MAX) {
  const PartPlan n = part_plan(R, Hq, Hkv, d, max_blocks, max_prefix_blocks, weights != nullptr);
  if (withhold != INT_MAX && n.pairs == 0) return FA_ERR_UNSUPPORTED;  // (the self-test is the tensor-core kernel's)
  if (!workspace || workspace_bytes < n.bytes || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  PartParams prm{static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(o), lse,
                 reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + n.off_lse),
                 reinterpret_cast<float*>(ws + n.off_scores), weights, block_table, ctx_lens, prefix_table, prefix_len,
                 R, Hq, Hkv, max_blocks, max_prefix_blocks, num_blocks, n.own_parts + n.prefix_parts,
                 n.prefix_parts, n.own_parts, 0, n.chunk, n.prefix_chunk,
                 n.pairs > 0 ? reinterpret_cast<const float*>(ws + n.off_pre_o) : nullptr,
                 n.pairs > 0 ? reinterpret_cast<const float*>(ws + n.off_pre_lse) : nullptr,
                 n.pre_parts, n.pairs, n.RT, false, scale * 1.4426950408889634f, g_wait_ns};
  CUtensorMap mk, mv;
  const long cache_rows = long(num_blocks) * Hkv * part::BS;
  if (!make_map_cache(&mk, k_cache, cache_rows, d) || !make_map_cache(&mv, v_cache, cache_rows, d)) return FA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 64 ? part_run<64>(mk, mv, prm, n, weights != nullptr, withhold, st)
                 : part_run<128>(mk, mv, prm, n, weights != nullptr, withhold, st);
}

fa_status shared_call(const fa_paged_decode_shared_args* args, int withhold, void* stream) {
  if (!args) return FA_ERR_INVALID_ARG;
  const fa_paged_decode_shared_args& a = *args;
  if (!a.prefix_table || !a.prefix_len || a.max_prefix_blocks <= 0 || !aligned(a.prefix_table, 4) ||
      !aligned(a.prefix_len, 4))
    return FA_ERR_INVALID_ARG;
  const fa_status s = part_check(a.q, a.k_cache, a.v_cache, a.block_table, a.ctx_lens, a.o, a.lse, a.R, a.Hq, a.Hkv,
                                 a.d, a.block_size, a.max_blocks_per_seq, a.num_blocks, a.scale, a.dtype);
  if (s != FA_OK) return s;
  if (int64_t(a.max_prefix_blocks) * part::BS > kMaxTokens) return FA_ERR_UNSUPPORTED;
  return part_call(a.q, a.k_cache, a.v_cache, a.prefix_table, a.prefix_len, a.block_table, a.ctx_lens, nullptr, a.o,
                   a.lse, a.R, a.Hq, a.Hkv, a.d, a.max_prefix_blocks, a.max_blocks_per_seq, a.num_blocks, a.scale,
                   a.workspace, a.workspace_bytes, stream, withhold);
}

struct EvictPlan {
  int cap;  // rows that may move of one (request, kv head): min(keep, n - keep) for n up to the table's width
  bool in_smem, fused;
  size_t off_moves, off_masks, bytes;
};

EvictPlan evict_plan(int R, int Hkv, int max_blocks, int keep) {
  EvictPlan n = {};
  const int64_t M = int64_t(max_blocks) * evict::BS, sets = int64_t(R) * Hkv;
  n.cap = int(std::max<int64_t>(0, std::min<int64_t>(keep, M - keep)));
  n.in_smem = M <= evict::MAX_KEYS;
  // The selecting CTAs move the rows themselves where few can move, which saves a launch.  Many
  // rows go to a second kernel, which spreads them evenly.  A call replayed from a graph, itself / second, us:
  //   128 rows move, sets of (request, kv head) 2, 64, 256, 512: 5.9 / 7.5, 8.9 / 10.8, 12.2 / 14.5, 21.9 / 24.6
  //   480 of 4096: 12.8 / 10.6, 14.9 / 14.3, 33.4 / 33.6, 67.0 / 65.7;  512 of 1024: 10.3 / 9.6, 10.7 / 10.8, 17.1 / 19.4,
  //     44.7 / 45.6
  //   750 of 1500: 12.2 / 9.6, 12.5 / 12.1, 29.2 / 29.2, 60.2 / 58.1 (128 sets 13.0 / 14.8)
  //   2048 of 4097 to 8192: 23.0 / 12.8, 42.2 / 29.1, 97.4 / 85.9, 180 / 169
  // The lengths are on the device, so the table's width decides: in one of 8192 tokens, steady contexts
  // of 2049 to 2176 with 2048 kept take the second kernel: 7.3 / 8.8, 9.6 / 11.2, 13.7 / 15.1, 24.9 / 27.3.
  n.fused = n.in_smem && n.cap <= 512;
  n.off_moves = n.fused ? 0 : align256(size_t(sets) * sizeof(int));
  n.off_masks = n.off_moves + (n.fused ? 0 : align256(size_t(sets) * 2 * n.cap * sizeof(int)));
  n.bytes = n.off_masks + (n.in_smem ? 0 : align256(size_t(sets) * 2 * ((M + 31) / 32) * sizeof(uint32_t)));
  return n;
}

}  // namespace

extern "C" {

fa_status fa_qk_norm_rope(const fa_qk_norm_rope_args* args, void* stream) {
  if (!args) return FA_ERR_INVALID_ARG;
  const fa_qk_norm_rope_args& a = *args;
  const fa_status s = rope_check(a.positions, a.inv_freq, a.B, a.Hq, a.Hkv, a.N, a.d, a.rotary_dim, a.sections,
                                 a.n_axes, a.interleaved, a.eps, a.dtype);
  if (s != FA_OK) return s;
  if (!rope_rows(a.q, a.q_strides, a.dtype) || !rope_rows(a.k, a.k_strides, a.dtype)) return FA_ERR_INVALID_ARG;
  if (!a.q_out || !a.k_out || !aligned(a.q_out, 16) || !aligned(a.k_out, 16)) return FA_ERR_INVALID_ARG;
  if (!rope_weights(a.q_weight, a.k_weight, a.dtype)) return FA_ERR_INVALID_ARG;
  RopeParams prm{{a.q, a.k, nullptr},
                 {a.q_strides[0], a.k_strides[0], 0},
                 {a.q_strides[1], a.k_strides[1], 0},
                 {a.q_strides[2], a.k_strides[2], 0},
                 {a.q_weight, a.k_weight},
                 a.positions, a.inv_freq,
                 {a.q_out, a.k_out},
                 a.pos_axis_stride, a.pos_batch_stride, a.B, a.Hq, a.Hkv, a.N, a.rotary_dim, a.sections[0],
                 a.n_axes > 1 ? a.sections[0] + a.sections[1] : a.sections[0], a.eps, 1,
                 nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.dtype == FA_DTYPE_BF16 ? rope_by_d<__nv_bfloat16>(prm, a.d, a.interleaved, st)
                                : rope_by_d<float>(prm, a.d, a.interleaved, st);
}

fa_status fa_qk_norm_rope_append(const fa_qk_norm_rope_append_args* args, void* stream) {
  if (!args) return FA_ERR_INVALID_ARG;
  const fa_qk_norm_rope_append_args& a = *args;
  const fa_status s = rope_check(a.positions, a.inv_freq, a.R, a.Hq, a.Hkv, a.Nq_max, a.d, a.rotary_dim, a.sections,
                                 a.n_axes, a.interleaved, a.eps, a.dtype);
  if (s != FA_OK) return s;
  if (a.block_size <= 0 || a.max_blocks_per_seq <= 0 || a.num_blocks <= 0) return FA_ERR_INVALID_ARG;
  if (a.dtype != FA_DTYPE_BF16 || a.d == 256 || a.block_size != 16) return FA_ERR_UNSUPPORTED;
  if (int64_t(a.max_blocks_per_seq) * 16 > kMaxTokens) return FA_ERR_UNSUPPORTED;
  if (!rope_rows(a.q, a.q_strides, a.dtype) || !rope_rows(a.k, a.k_strides, a.dtype) ||
      !rope_rows(a.v, a.v_strides, a.dtype))
    return FA_ERR_INVALID_ARG;
  if (!a.q_out || !a.k_cache || !a.v_cache || !a.block_table || !a.ctx_lens || !a.q_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(a.q_out, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.block_table, 4) ||
      !aligned(a.ctx_lens, 4) || !aligned(a.q_lens, 4))
    return FA_ERR_INVALID_ARG;
  if (!rope_weights(a.q_weight, a.k_weight, a.dtype)) return FA_ERR_INVALID_ARG;
  RopeParams prm{{a.q, a.k, a.v},
                 {a.q_strides[0], a.k_strides[0], a.v_strides[0]},
                 {a.q_strides[1], a.k_strides[1], a.v_strides[1]},
                 {a.q_strides[2], a.k_strides[2], a.v_strides[2]},
                 {a.q_weight, a.k_weight},
                 a.positions, a.inv_freq,
                 {a.q_out, nullptr},
                 a.pos_axis_stride, a.pos_batch_stride, a.R, a.Hq, a.Hkv, a.Nq_max, a.rotary_dim, a.sections[0],
                 a.n_axes > 1 ? a.sections[0] + a.sections[1] : a.sections[0], a.eps, 1,
                 a.block_table, a.ctx_lens, a.q_lens, a.k_cache, a.v_cache, a.max_blocks_per_seq, a.num_blocks};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (a.d) {
    case 64: return rope_launch<__nv_bfloat16, 64, true>(prm, a.interleaved, st);
    case 96: return rope_launch<__nv_bfloat16, 96, true>(prm, a.interleaved, st);
    default: return rope_launch<__nv_bfloat16, 128, true>(prm, a.interleaved, st);
  }
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  return d <= 0 ? 0 : align256(size_t(kRopeBwdCtas) * d * sizeof(float));
}

fa_status fa_qk_norm_rope_bwd(const fa_qk_norm_rope_bwd_args* args, void* stream) {
  if (!args) return FA_ERR_INVALID_ARG;
  const fa_qk_norm_rope_bwd_args& a = *args;
  const fa_status s = rope_check(a.positions, a.inv_freq, a.B, a.Hq, a.Hkv, a.N, a.d, a.rotary_dim, a.sections,
                                 a.n_axes, a.interleaved, a.eps, a.dtype);
  if (s != FA_OK) return s;
  if (!a.dq_out || !a.dk_out || !aligned(a.dq_out, 16) || !aligned(a.dk_out, 16)) return FA_ERR_INVALID_ARG;
  if (!rope_weights(a.q_weight, a.k_weight, a.dtype)) return FA_ERR_INVALID_ARG;
  if (a.dout_dtype != FA_DTYPE_F32 && a.dout_dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
  if (a.grad_dtype != FA_DTYPE_F32 && a.grad_dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
  if (a.dtype == FA_DTYPE_F32 && (a.dout_dtype != FA_DTYPE_F32 || a.grad_dtype != FA_DTYPE_F32))
    return FA_ERR_UNSUPPORTED;
  if (!rope_rows(a.q, a.q_strides, a.dtype) || !rope_rows(a.k, a.k_strides, a.dtype) ||
      !rope_rows(a.dq, a.dq_strides, a.grad_dtype) || !rope_rows(a.dk, a.dk_strides, a.grad_dtype))
    return FA_ERR_INVALID_ARG;
  if (rows_overlap(a.dq_strides, a.B, a.Hq, a.N, a.d) || rows_overlap(a.dk_strides, a.B, a.Hkv, a.N, a.d))
    return FA_ERR_INVALID_ARG;
  if (a.q_weight) {
    if (!a.dq_weight || !a.dk_weight || !aligned(a.dq_weight, 4) || !aligned(a.dk_weight, 4)) return FA_ERR_INVALID_ARG;
    if (!a.workspace || a.workspace_bytes < fa_qk_norm_rope_bwd_workspace_size(a.d) || !aligned(a.workspace, 256))
      return FA_ERR_WORKSPACE;
  }
  RopeBwdParams prm{{a.dq_out, a.dk_out},
                    {a.q, a.k},
                    {a.q_strides[0], a.k_strides[0]},
                    {a.q_strides[1], a.k_strides[1]},
                    {a.q_strides[2], a.k_strides[2]},
                    {a.q_weight, a.k_weight},
                    a.positions, a.inv_freq,
                    {a.dq, a.dk},
                    {a.dq_strides[0], a.dk_strides[0]},
                    {a.dq_strides[1], a.dk_strides[1]},
                    {a.dq_strides[2], a.dk_strides[2]},
                    static_cast<float*>(a.workspace),
                    a.pos_axis_stride, a.pos_batch_stride, a.B, {a.Hq, a.Hkv}, a.N, a.rotary_dim, a.sections[0],
                    a.n_axes > 1 ? a.sections[0] + a.sections[1] : a.sections[0], a.eps, {1, 1}, {1, 1}, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float *dwq = a.dq_weight, *dwk = a.dk_weight;
  if (a.dtype == FA_DTYPE_F32) return rope_bwd_by_d<float, float, float>(prm, a.d, a.interleaved, dwq, dwk, st);
  using bf = __nv_bfloat16;
  const bool out_f32 = a.grad_dtype == FA_DTYPE_F32;
  if (a.dout_dtype == FA_DTYPE_F32)
    return out_f32 ? rope_bwd_by_d<bf, float, float>(prm, a.d, a.interleaved, dwq, dwk, st)
                   : rope_bwd_by_d<bf, float, bf>(prm, a.d, a.interleaved, dwq, dwk, st);
  return out_f32 ? rope_bwd_by_d<bf, bf, float>(prm, a.d, a.interleaved, dwq, dwk, st)
                 : rope_bwd_by_d<bf, bf, bf>(prm, a.d, a.interleaved, dwq, dwk, st);
}

size_t fa_paged_decode_shared_workspace_size(int R, int Hq, int Hkv, int d, int max_prefix_blocks,
                                             int max_blocks_per_seq, int block_size) {
  if (!part_sizes(R, Hq, Hkv, d, max_blocks_per_seq, block_size) || max_prefix_blocks <= 0) return 0;
  return part_plan(R, Hq, Hkv, d, max_blocks_per_seq, max_prefix_blocks, false).bytes;
}

fa_status fa_paged_decode_shared(const fa_paged_decode_shared_args* args, void* stream) {
  return shared_call(args, INT_MAX, stream);
}

fa_status fa_selftest_shared_timeout(const fa_paged_decode_shared_args* args, int tiles, void* stream) {
  return tiles < 0 ? FA_ERR_INVALID_ARG : shared_call(args, tiles, stream);
}

size_t fa_paged_decode_scored_workspace_size(int R, int Hq, int Hkv, int d, int max_blocks_per_seq, int block_size) {
  if (!part_sizes(R, Hq, Hkv, d, max_blocks_per_seq, block_size)) return 0;
  return part_plan(R, Hq, Hkv, d, max_blocks_per_seq, 0, true).bytes;
}

fa_status fa_paged_decode_scored(const fa_paged_decode_scored_args* args, void* stream) {
  if (!args) return FA_ERR_INVALID_ARG;
  const fa_paged_decode_scored_args& a = *args;
  if (!a.weights || !aligned(a.weights, 16)) return FA_ERR_INVALID_ARG;
  const fa_status s = part_check(a.q, a.k_cache, a.v_cache, a.block_table, a.ctx_lens, a.o, a.lse, a.R, a.Hq, a.Hkv,
                                 a.d, a.block_size, a.max_blocks_per_seq, a.num_blocks, a.scale, a.dtype);
  if (s != FA_OK) return s;
  return part_call(a.q, a.k_cache, a.v_cache, nullptr, nullptr, a.block_table, a.ctx_lens, a.weights, a.o, a.lse, a.R,
                   a.Hq, a.Hkv, a.d, 0, a.max_blocks_per_seq, a.num_blocks, a.scale, a.workspace, a.workspace_bytes,
                   stream);
}

size_t fa_paged_evict_workspace_size(int R, int Hkv, int max_blocks_per_seq, int keep) {
  if (R <= 0 || Hkv <= 0 || max_blocks_per_seq <= 0 || keep <= 0) return 0;
  return evict_plan(R, Hkv, max_blocks_per_seq, keep).bytes;
}

fa_status fa_paged_evict(const fa_paged_evict_args* args, void* stream) {
  if (!args) return FA_ERR_INVALID_ARG;
  const fa_paged_evict_args& a = *args;
  if (!a.k_cache || !a.v_cache || !a.block_table || !a.ctx_lens || !a.seq_lens || !a.weights || !a.slot_pos ||
      !a.weights_out || !a.slot_pos_out || !a.new_ctx)
    return FA_ERR_INVALID_ARG;
  if (a.R <= 0 || a.Hkv <= 0 || a.d <= 0 || a.block_size <= 0 || a.max_blocks_per_seq <= 0 || a.num_blocks <= 0)
    return FA_ERR_INVALID_ARG;
  if (a.keep <= 0 || a.recent < 0 || a.recent > a.keep) return FA_ERR_INVALID_ARG;
  const void* small[] = {a.block_table, a.ctx_lens, a.seq_lens, a.weights, a.slot_pos, a.weights_out,
                         a.slot_pos_out, a.new_ctx};
  for (const void* p : small)
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  const void* large[] = {a.k_cache, a.v_cache, a.weights, a.slot_pos, a.weights_out, a.slot_pos_out};
  for (const void* p : large)
    if (!aligned(p, 16)) return FA_ERR_INVALID_ARG;
  // the selection reads its inputs while it writes its outputs
  if (a.weights_out == a.weights || a.slot_pos_out == a.slot_pos || a.new_ctx == a.ctx_lens || a.new_ctx == a.seq_lens)
    return FA_ERR_INVALID_ARG;
  if (a.dtype != FA_DTYPE_BF16 || (a.d != 64 && a.d != 96 && a.d != 128 && a.d != 256) || a.block_size != evict::BS)
    return FA_ERR_UNSUPPORTED;
  if (a.R > 65535 || a.Hkv > 65535 || int64_t(a.max_blocks_per_seq) * evict::BS > kMaxTokens ||
      int64_t(a.num_blocks) * a.Hkv * evict::BS > 0x7fffffff)
    return FA_ERR_UNSUPPORTED;
  const EvictPlan n = evict_plan(a.R, a.Hkv, a.max_blocks_per_seq, a.keep);
  if (n.bytes > 0 && (!a.workspace || a.workspace_bytes < n.bytes || !aligned(a.workspace, 256)))
    return FA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(a.workspace);
  const EvictParams prm{a.block_table, a.ctx_lens, a.seq_lens, a.weights, a.slot_pos, a.weights_out, a.slot_pos_out,
                        a.new_ctx, reinterpret_cast<int*>(ws + n.off_moves), reinterpret_cast<int*>(ws),
                        reinterpret_cast<uint32_t*>(ws + n.off_masks), static_cast<uint4*>(a.k_cache),
                        static_cast<uint4*>(a.v_cache), a.R, a.Hkv, a.max_blocks_per_seq, a.num_blocks, a.keep,
                        a.recent, n.cap, a.d * 2 / 16, n.in_smem, n.fused};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t M = int64_t(a.max_blocks_per_seq) * evict::BS;
  const int smem = n.in_smem ? int((M + 2 * ((M + 31) / 32)) * 4) : 0;
  static Prepared prepared;
  if (prepared.launch(fa_evict_select_kernel, dim3(a.Hkv, a.R), dim3(evict::THREADS), smem, st, prm) != cudaSuccess)
    return FA_ERR_CUDA;
  if (!n.fused && n.cap > 0) {
    const int64_t pieces = int64_t(n.cap) * 2 * prm.row16;
    const int64_t want = std::max<int64_t>(1, kSms * 16 / (int64_t(a.R) * a.Hkv));
    const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(want, (pieces + 1023) / 1024)));
    if (launch_pdl(fa_evict_move_kernel, dim3(grid, a.Hkv, a.R), dim3(256), 0, st, prm) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return launched();
}

}  // extern "C"
