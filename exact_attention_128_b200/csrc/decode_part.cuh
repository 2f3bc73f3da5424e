// decode_part.cuh — one decode step over pieces of a paged cache, left as partial results and
// merged: the decode that also adds up each cached token's attention weight, and the decode of a
// batch whose requests share a prefix.
//
// A piece is a run of cache blocks that a set of query rows attends to.  Its partial result is
// (u / l, lse) of those keys alone; the pieces of one row are joined by their unnormalised mass,
//   lse = ln sum_s e^{lse_s},  o = sum_s e^{lse_s - lse} o_s
// (block results are never simply averaged).  Two kinds of pieces share the kernel:
//   own     rows = the G = Hq / Hkv query heads of one request and kv head, keys = its own blocks;
//   prefix  rows = 16 consecutive ones of all R * G rows of a kv head, keys = the shared blocks,
//           so that a prefix block is read once for up to 16 rows.
//
// What bounds it: reading K and V once.  Four warps take every fourth block, each with its own
// ring of TMA stages and its own (m, l, u); rows sit in the 16 rows of mma.sync m16n8k16.
// P is multiplied as the sum of two bf16 parts, its rounding and the rest: the tensor cores idle
// here, and with it the output's only rounding is the last one.  64 requests of 512 to 8192 tokens, 2
// kv heads, d = 128 (286 MB): 56 us, 5.1 TB/s; with scores (13 MB more) 58 us.  The join takes 9 us
// behind it: it is a chain of four dependent loads (lengths, lse of the pieces, results, old weights).
#pragma once
#include "decode.cuh"

namespace fa {
namespace part {
constexpr int WARPS = 4;
constexpr int STAGES = 2;  // (3 and 4 leave fewer CTAs on an SM: 71 and 94 us where 2 take 67)
constexpr int BS = 16;
constexpr int ROWS = 16;       // query rows of a piece
constexpr int MIN_CHUNK = 8;   // blocks of a piece, at least: two for each warp
constexpr int MAX_PARTS = 64;  // pieces of a row, at most, of either kind
constexpr int PREFIX_CTAS = 148;  // CTAs of the tensor-core prefix kernel, at most
constexpr int JOIN_TOKENS = 1024;  // tokens whose weights one CTA adds up at a time

template <int D>
struct Cfg {
  static constexpr int SLAB = BS * D * 2;  // one (block, kv head) of K or V
  static constexpr int STAGE_BYTES = 2 * SLAB;
  static constexpr int OFF_BAR = WARPS * STAGES * STAGE_BYTES;
  static constexpr int SMEM = OFF_BAR + WARPS * STAGES * 8 + 1024;
  static constexpr int OP = D + 8;  // padded row of the warp merge (floats)
  static_assert(WARPS * ROWS * OP * 4 + 2 * WARPS * ROWS * 4 <= OFF_BAR, "merge buffer must fit the stages");
};
}  // namespace part

struct PartParams {
  const __nv_bfloat16* q;  // [R, Hq, D]
  __nv_bfloat16* o;        // [R, Hq, D]
  float* lse;              // [R, Hq], may be null
  float* part_o;           // [R * Hq][parts][D]
  float* part_lse;         // [R * Hq][parts], in base 2
  float* scores;           // [R, Hq, max_blocks * 16] scaled, base 2 (scored only)
  float* weights;          // [R, Hkv, max_blocks * 16] (scored only)
  const int* bt;           // own blocks [R, max_blocks]
  const int* ctx;          // own tokens [R]
  const int* pbt;          // prefix blocks [prefix_blocks] (shared only)
  const int* plen;         // prefix tokens [1] (shared only)
  int R, Hq, Hkv, max_blocks, prefix_blocks, num_blocks;
  int parts;               // partial results per row: prefix pieces, then own pieces
  int prefix_parts, own_parts;
  int n_prefix;            // CTAs that work on prefix pieces
  int chunk, prefix_chunk;  // blocks of a piece
  // the prefix part by the tensor-core kernel (shared_prefix.cuh): its results, else null
  const float *pre_o, *pre_lse;
  int pre_parts, pairs, RT;
  bool late_wait;  // the grid before this one is that kernel, and nothing of it is read here
  float scale_log2;
  uint64_t wait_ns;
};

// Tokens of the shared prefix / of request r, or -1 (flagged) where out of range.
__device__ __forceinline__ int part_len(const int* len, int i, int max_blocks, int where) {
  const int n = len[i];
  if (n >= 0 && n <= max_blocks * part::BS) return n;
  set_status(FA_ERR_INVALID_ARG, where);
  return -1;
}

// CTAs [0, n_prefix) take the prefix's pieces, the others the requests' own.
template <int D, bool SCORED>
__global__ void __launch_bounds__(part::WARPS * 32)
    fa_decode_part_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ PartParams p) {
  using namespace part;
  using C = Cfg<D>;
  constexpr int KS = D / 16, NT = D / 8, KB = D / 64;
  extern __shared__ uint8_t dsmem_raw[];
  uint8_t* dsmem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~uintptr_t(1023));
  const bool prefix = int(blockIdx.x) < p.n_prefix;
  const int parts = prefix ? p.prefix_parts : p.own_parts, at = prefix ? blockIdx.x : blockIdx.x - p.n_prefix;
  const int zg = at / parts, s = at - zg * parts;                // piece
  const int z = zg / p.Hkv, g = zg - z * p.Hkv, G = p.Hq / p.Hkv;  // request or row tile, kv head
  // late_wait: the prefix kernel let this grid start once it had waited for everything before it.
  // Its own results are read by the grid after this one, which waits for this grid alone: so one
  // CTA, the last to be started, holds this grid open until the prefix kernel is done.
  const bool hold = p.late_wait && blockIdx.x == gridDim.x - 1;
  auto finish = [&] {
    if (hold) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (!p.late_wait) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = prefix ? part_len(p.plen, 0, p.prefix_blocks, 302) : part_len(p.ctx, z, p.max_blocks, 300);
  const int chunk = prefix ? p.prefix_chunk : p.chunk;
  const int nblk = (n + BS - 1) / BS;
  const int b0 = s * chunk;
  if (n <= 0 || b0 >= nblk) return finish();
  const int b1 = min(nblk, b0 + chunk);
  const int* bt = prefix ? p.pbt : p.bt + size_t(z) * p.max_blocks;
  const int rows = prefix ? min(ROWS, p.R * G - z * ROWS) : G;
  // (request, head) of row i, as one index into [R * Hq]
  auto row_of = [&](int i) {
    if (!prefix) return z * p.Hq + g * G + i;
    const int j = z * ROWS + i;
    return (j / G) * p.Hq + g * G + j % G;
  };

  const int warp = warp_id(), lane = lane_id();
  const int gq = lane >> 2, t4 = lane & 3;
  const int nb = max(0, (b1 - b0 - warp + WARPS - 1) / WARPS);  // this warp's blocks
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsmem + C::OFF_BAR) + warp * STAGES;
  const uint32_t sbase = smem_u32(dsmem) + warp * STAGES * C::STAGE_BYTES;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0)
    for (int st = 0; st < STAGES; ++st) mbar_init(&bars[st], 1);
  fence_barrier_init();
  __syncthreads();

  // physical blocks of this warp's next 32 blocks, one per lane
  int my_phys = 0;
  auto fetch_table = [&](int i) {
    my_phys = 0;
    if (i + lane < nb) {
      my_phys = bt[b0 + warp + (i + lane) * WARPS];
      if (my_phys < 0 || my_phys >= p.num_blocks) {
        set_status(FA_ERR_INVALID_ARG, 301);
        my_phys = 0;  // never address an out-of-range block; the result is flagged invalid
      }
    }
  };
  // the whole warp calls issue(i), in order; lane 0 issues the loads
  auto issue = [&](int i) {
    if ((i & 31) == 0) fetch_table(i);
    const int phys = __shfl_sync(0xffffffffu, my_phys, i & 31);
    if (lane == 0) {
      const int row = (phys * p.Hkv + g) * BS;
      uint64_t* bar = &bars[i % STAGES];
      const uint32_t st = sbase + (i % STAGES) * C::STAGE_BYTES;
      mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        tma_load_2d(st + kb * 2048, &tmK, bar, kb * 64, row);
        tma_load_2d(st + C::SLAB + kb * 2048, &tmV, bar, kb * 64, row);
      }
    }
  };
  for (int i = 0; i < min(nb, STAGES); ++i) issue(i);

  // q fragments (A operand), rows past `rows` zero
  uint32_t qa[KS][4];
  {
    const bool v0 = gq < rows, v1 = gq + 8 < rows;
    const uint32_t* q0 = reinterpret_cast<const uint32_t*>(p.q + size_t(row_of(v0 ? gq : 0)) * D);
    const uint32_t* q1 = reinterpret_cast<const uint32_t*>(p.q + size_t(row_of(v1 ? gq + 8 : 0)) * D);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qa[ks][0] = v0 ? q0[8 * ks + t4] : 0u;
      qa[ks][1] = v1 ? q1[8 * ks + t4] : 0u;
      qa[ks][2] = v0 ? q0[8 * ks + 4 + t4] : 0u;
      qa[ks][3] = v1 ? q1[8 * ks + 4 + t4] : 0u;
    }
  }
  float* sc0 = nullptr;
  float* sc1 = nullptr;
  if constexpr (SCORED) {
    const size_t M = size_t(p.max_blocks) * BS;
    if (gq < rows) sc0 = p.scores + size_t(row_of(gq)) * M;
    if (gq + 8 < rows) sc1 = p.scores + size_t(row_of(gq + 8)) * M;
  }

  float m0 = -INFINITY, m1 = -INFINITY;  // running max (base 2) of rows gq, gq + 8
  float l0 = 0.f, l1 = 0.f;
  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
  const float sl2 = p.scale_log2;
  const int mi = lane >> 3, rr = lane & 7;  // ldmatrix: lane -> (matrix, row)
  const int k_tok = rr + 8 * (mi >> 1), k_chunk_lo = mi & 1;
  const int v_tok = rr + 8 * (mi & 1), v_chunk_hi = mi >> 1;

  bool ok = true;
  int consumed = 0;
  for (int i = 0; i < nb && ok; ++i) {
    ok = warp_wait(&bars[i % STAGES], (i / STAGES) & 1, p.wait_ns, &abort_flag, 303);
    if (!ok) break;
    consumed = i + 1;
    const uint32_t sk = sbase + (i % STAGES) * C::STAGE_BYTES, sv = sk + C::SLAB;
    const int lb = b0 + warp + i * WARPS;
    const int valid = min(BS, n - lb * BS);

    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t b00, b01, b10, b11;
      ldsm_x4(sk + slab_off(k_tok, 2 * ks + k_chunk_lo), b00, b01, b10, b11);
      mma_bf16_16816(sc[0], qa[ks], b00, b01);
      mma_bf16_16816(sc[1], qa[ks], b10, b11);
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] *= sl2;
    if constexpr (SCORED) {
      // (slots past the request's tokens in its last block get a score too; nobody reads it)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const size_t at = size_t(lb) * BS + nt * 8 + 2 * t4;
        if (sc0) *reinterpret_cast<float2*>(sc0 + at) = make_float2(sc[nt][0], sc[nt][1]);
        if (sc1) *reinterpret_cast<float2*>(sc1 + at) = make_float2(sc[nt][2], sc[nt][3]);
      }
    }
    if (valid < BS) {  // selection, so that nothing in unused slots can leak
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (nt * 8 + 2 * t4 + (e & 1) >= valid) sc[nt][e] = -INFINITY;
    }
    const float old0 = m0, old1 = m1;
    float mx0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
    float mx1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    m0 = fmaxf(m0, mx0);
    m1 = fmaxf(m1, mx1);
    // (scores of -inf alone so far, from keys with infinities: their mass is 0)
    const float n0 = m0 == -INFINITY ? 0.f : m0, n1 = m1 == -INFINITY ? 0.f : m1;
    const float a0 = ex2(old0 - n0), a1 = ex2(old1 - n1);
    float pr[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      pr[nt][0] = ex2(sc[nt][0] - n0);
      pr[nt][1] = ex2(sc[nt][1] - n0);
      pr[nt][2] = ex2(sc[nt][2] - n1);
      pr[nt][3] = ex2(sc[nt][3] - n1);
    }
    l0 = l0 * a0 + pr[0][0] + pr[0][1] + pr[1][0] + pr[1][1];
    l1 = l1 * a1 + pr[0][2] + pr[0][3] + pr[1][2] + pr[1][3];
    if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        acc[nt][0] *= a0; acc[nt][1] *= a0;
        acc[nt][2] *= a1; acc[nt][3] *= a1;
      }
    }
    // P = hi + lo, both bf16: hi is P rounded, lo the rest rounded (2^-16 of P is lost)
    uint32_t pa[4], pl[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = pr[k >> 1][2 * (k & 1)], y = pr[k >> 1][2 * (k & 1) + 1];
      pa[k] = pack_bf16x2(x, y);
      pl[k] = pack_bf16x2(x - __uint_as_float(pa[k] << 16), y - __uint_as_float(pa[k] & 0xffff0000u));
    }
    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
    if (valid < BS) {  // zero V of unused slots (P is 0 there; 0 * NaN would not be)
      keep0 = (2 * t4 < valid ? 0x0000ffffu : 0u) | (2 * t4 + 1 < valid ? 0xffff0000u : 0u);
      keep1 = (2 * t4 + 8 < valid ? 0x0000ffffu : 0u) | (2 * t4 + 9 < valid ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int nt = 0; nt < NT; nt += 2) {
      uint32_t v00, v01, v10, v11;
      ldsm_x4_t(sv + slab_off(v_tok, nt + v_chunk_hi), v00, v01, v10, v11);
      mma_bf16_16816(acc[nt], pa, v00 & keep0, v01 & keep1);
      mma_bf16_16816(acc[nt + 1], pa, v10 & keep0, v11 & keep1);
      mma_bf16_16816(acc[nt], pl, v00 & keep0, v01 & keep1);
      mma_bf16_16816(acc[nt + 1], pl, v10 & keep0, v11 & keep1);
    }
    __syncwarp();  // all lanes have read this stage: refill it
    if (i + STAGES < nb) {
      fence_proxy_async_smem();
      issue(i + STAGES);
    }
  }
  if (!ok) {
    // a bounded wait ran out: let the loads in flight land before the shared memory is given up
    if (lane == 0)
      for (int i = consumed; i < min(nb, consumed + STAGES); ++i)
        mbar_wait_bounded(&bars[i % STAGES], (i / STAGES) & 1, p.wait_ns);
    __syncwarp();
  }
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  __syncthreads();  // all warps are done with their stages: reuse shared memory
  const int part = prefix ? s : p.prefix_parts + s;
  if (abort_flag) {  // NaN, so that nothing merged from this piece looks valid
    for (int i = threadIdx.x; i < rows; i += WARPS * 32) p.part_lse[size_t(row_of(i)) * p.parts + part] = NAN;
    return finish();
  }
  float* so = reinterpret_cast<float*>(dsmem);  // [WARPS][ROWS][OP]
  float* sm = so + WARPS * ROWS * C::OP;        // [WARPS][ROWS]
  float* sl = sm + WARPS * ROWS;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int d0 = 8 * nt + 2 * t4;
    *reinterpret_cast<float2*>(&so[(warp * ROWS + gq) * C::OP + d0]) = make_float2(acc[nt][0], acc[nt][1]);
    *reinterpret_cast<float2*>(&so[(warp * ROWS + gq + 8) * C::OP + d0]) = make_float2(acc[nt][2], acc[nt][3]);
  }
  if (t4 == 0) {
    sm[warp * ROWS + gq] = m0;
    sm[warp * ROWS + gq + 8] = m1;
    sl[warp * ROWS + gq] = l0;
    sl[warp * ROWS + gq + 8] = l1;
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < rows * D; idx += WARPS * 32) {
    const int i = idx / D, d = idx % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm[w * ROWS + i]);
    float L = 0.f, U = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float mw = sm[w * ROWS + i];
      const float wt = (mw == -INFINITY) ? 0.f : ex2(mw - M);
      L += sl[w * ROWS + i] * wt;
      U += so[(w * ROWS + i) * C::OP + d] * wt;
    }
    const size_t pi = size_t(row_of(i)) * p.parts + part;
    p.part_o[pi * D + d] = L == 0.f ? 0.f : U / L;  // (no mass: lse = -inf)
    if (d == 0) p.part_lse[pi] = M + __log2f(L);
  }
  finish();
}

// How the tiles of a prefix of P tokens are dealt out by the tensor-core kernel: CTA c < ctas takes
// [begin(c), begin(c + 1)) of the items' tiles.
struct PrefixDeal {
  static constexpr int BN = 64;
  int nt, ctas;
  long long all;
  __device__ PrefixDeal(int P, int items) {
    nt = (P + BN - 1) / BN;
    all = (long long)(items)*nt;
    // at least two tiles per CTA: a single one does not pay for its partial result
    ctas = int(min((all + 1) / 2, (long long)(part::PREFIX_CTAS)));
  }
  __device__ long long begin(int c) const { return c * all / ctas; }
  __device__ int owner(long long x) const { return int(((x + 1) * ctas - 1) / all); }
};

// The pieces of the rows of (request r, kv head g): `np` of the prefix and `no` of its own tokens.
struct PartPieces {
  int np, no;
  size_t pre0;  // first row of the prefix kernel's results for these heads; 256 rows to the next piece
  __device__ PartPieces(const PartParams& p, int r, int g, int n) {
    using namespace part;
    const int P = p.plen ? p.plen[0] : 0;
    const bool bad = n < 0 || n > p.max_blocks * BS || P < 0 || P > p.prefix_blocks * BS;
    no = bad ? 0 : ((n + BS - 1) / BS + p.chunk - 1) / p.chunk;
    np = 0;
    pre0 = 0;
    if (bad || P == 0) return;
    if (p.pre_o) {
      const int tile = r / p.RT, it = g * p.pairs + tile / 2;
      const PrefixDeal deal(P, p.Hkv * p.pairs);
      np = deal.owner((long long)(it + 1) * deal.nt - 1) - deal.owner((long long)(it)*deal.nt) + 1;
      pre0 = (size_t(it) * p.pre_parts * 2 + (tile & 1)) * 128 + (r - tile * p.RT) * (p.Hq / p.Hkv);
    } else {
      np = ((P + BS - 1) / BS + p.prefix_chunk - 1) / p.prefix_chunk;
    }
  }
  // piece k of head h of the group, as a row of the prefix kernel's results or of the pieces
  __device__ bool in_pre(const PartParams& p, int k) const { return p.pre_o != nullptr && k < np; }
  __device__ size_t row(const PartParams& p, size_t row0, int h, int k) const {
    if (in_pre(p, k)) return pre0 + h + size_t(k) * 256;
    return (row0 + h) * p.parts + (k < np ? k : p.prefix_parts + k - np);
  }
};

// One warp: lse (base 2) of head h's row from its pieces; w[k] becomes piece k's share e^{lse_k - lse}.
__device__ __forceinline__ float part_lse_of(const PartParams& p, const PartPieces& x, size_t row0, int h, float* w) {
  const int lane = lane_id(), pieces = x.np + x.no;
  float M = -INFINITY, W = 0.f;
  for (int k = lane; k < pieces; k += 32) {
    const float v = (x.in_pre(p, k) ? p.pre_lse : p.part_lse)[x.row(p, row0, h, k)];
    w[k] = v;
    M = fmaxf(M, v);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
  for (int k = lane; k < pieces; k += 32) W += ex2(w[k] - M);  // (NaN where a wait ran out)
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) W += __shfl_xor_sync(0xffffffffu, W, m);
  const float lse = pieces > 0 ? M + __log2f(W) : -INFINITY;  // no key at all: o = 0, lse = -inf
  for (int k = lane; k < pieces; k += 32) w[k] = ex2(w[k] - lse);
  __syncwarp();
  return lse;
}

// The first `joins` CTAs write o and lse: `strands` of their eight warps share a row (request,
// head), each adding up every strands-th piece.  SCORED: the others, `spans` for each (request, kv
// head), add up the weights of JOIN_TOKENS tokens at a time,
//   weights[r, g, s] += sum over the heads of kv head g of e^{score - lse}.
template <int D, bool SCORED>
__global__ void __launch_bounds__(256) fa_decode_join_kernel(const __grid_constant__ PartParams p, int joins,
                                                             int strands, int spans) {
  using namespace part;
  constexpr int PIECES = MAX_PARTS + PREFIX_CTAS + 1;
  __shared__ float s_w[8][PIECES];
  __shared__ float s_lse[ROWS];
  __shared__ float4 s_u[8][D / 4];
  const int G = p.Hq / p.Hkv, warp = warp_id(), lane = lane_id();
  // Lengths and old weights are read before the grid before this one is waited for: it let this one
  // start after it had itself waited for everything before, and writes neither.
  if (int(blockIdx.x) < joins) {
    const int row = blockIdx.x * (8 / strands) + warp / strands, strand = warp % strands;
    const bool on = row < p.R * p.Hq;
    const int n = on ? p.ctx[row / p.Hq] : 0;
    const PartPieces x(p, on ? row / p.Hq : 0, on ? row % p.Hq / G : 0, n);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int Q = D / 4, PER = 32 / Q;  // lanes of a row, pieces a warp reads at a time
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
    float lse = 0.f;
    if (on) {
      const int r = row / p.Hq, h = row - r * p.Hq, g = h / G;
      const size_t row0 = size_t(r) * p.Hq + g * G;
      lse = part_lse_of(p, x, row0, h - g * G, s_w[warp]);
      const int pieces = x.np + x.no, c = (lane % Q) * 4;
#pragma unroll 8
      for (int k = strand * PER + lane / Q; k < pieces; k += strands * PER) {
        const float* src = (x.in_pre(p, k) ? p.pre_o : p.part_o) + x.row(p, row0, h - g * G, k) * D;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src + c));
        const float w = s_w[warp][k];
        u.x += w * v.x;
        u.y += w * v.y;
        u.z += w * v.z;
        u.w += w * v.w;
      }
      if constexpr (PER == 2) {
        u.x += __shfl_xor_sync(0xffffffffu, u.x, 16);
        u.y += __shfl_xor_sync(0xffffffffu, u.y, 16);
        u.z += __shfl_xor_sync(0xffffffffu, u.z, 16);
        u.w += __shfl_xor_sync(0xffffffffu, u.w, 16);
      }
    }
    if (strands > 1) {
      if (lane < Q) s_u[warp][lane] = u;
      __syncthreads();
      if (strand == 0 && lane < Q)
        for (int k = 1; k < strands; ++k) {
          const float4 v = s_u[warp + k][lane];
          u.x += v.x;
          u.y += v.y;
          u.z += v.z;
          u.w += v.w;
        }
    }
    if (on && strand == 0) {
      if (lane < Q)
        *reinterpret_cast<uint2*>(p.o + size_t(row) * D + lane * 4) =
            make_uint2(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w));
      if (lane == 0 && p.lse) p.lse[row] = lse * 0.69314718055994531f;
    }
    return;
  }
  if constexpr (SCORED) {
    const int at = blockIdx.x - joins, set = at / spans, span = at - set * spans;
    const int r = set / p.Hkv, g = set - r * p.Hkv;
    const int n = p.ctx[r];
    const PartPieces x(p, r, g, n);
    const bool any = x.no > 0 && span * JOIN_TOKENS < n;  // (no pieces: a length out of range)
    const size_t row0 = size_t(r) * p.Hq + g * G, M = size_t(p.max_blocks) * BS;
    float* const w0 = p.weights + (size_t(r) * p.Hkv + g) * M;
    int s = span * JOIN_TOKENS + threadIdx.x * 4;
    float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
    if (any && s < n) old = *reinterpret_cast<const float4*>(w0 + s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!any) return;
    for (int h = warp; h < G; h += 8) {
      const float lse = part_lse_of(p, x, row0, h, s_w[warp]);
      if (lane == 0) s_lse[h] = lse;
    }
    __syncthreads();
    for (; s < n; s += spans * JOIN_TOKENS) {
      float* out = w0 + s;
      const int next = s + spans * JOIN_TOKENS;
      const float4 cur = old;
      if (next < n) old = *reinterpret_cast<const float4*>(w0 + next);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int h = 0; h < G; ++h) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.scores + (row0 + h) * M + s));
        const float lse = s_lse[h];
        w.x += ex2(v.x - lse);
        w.y += ex2(v.y - lse);
        w.z += ex2(v.z - lse);
        w.w += ex2(v.w - lse);
      }
      if (s + 4 <= n) {
        *reinterpret_cast<float4*>(out) = make_float4(cur.x + w.x, cur.y + w.y, cur.z + w.z, cur.w + w.w);
      } else {
        out[0] = cur.x + w.x;
        if (s + 1 < n) out[1] = cur.y + w.y;
        if (s + 2 < n) out[2] = cur.z + w.z;
      }
    }
  }
}

}  // namespace fa
