// evict.cuh — eviction from a paged cache by accumulated attention weight.
//
// For each request r and kv head h, of the n = ctx_lens[r] cached tokens keep `keep`: every token
// among the `recent` newest positions of the sequence, then the heaviest of the others (ties: the
// lower slot).  Attention does not depend on the order of its keys, so kept tokens in slots below
// `keep` stay where they are and the i-th kept token at or past `keep` moves into the i-th freed
// slot below it: at most min(keep, n - keep) rows move, and no row is both read and written.
// A token's age is not its slot then; slot_pos carries each slot's sequence position (-1: not
// moved since it was appended, so its position is seq_len - n + slot).
//
// One CTA per (r, h).  Each token's key is its weight as an order-preserving 32-bit integer, all
// ones where it is protected, and is kept in shared memory (read again from the inputs past
// MAX_KEYS tokens).  The keep-th largest key is found in three digits of 9, 11 and 12 bits, from a
// histogram each.  The first digit is a weight's exponent, of which few differ: its histogram has
// 16 copies, one for every other lane, so that the lanes of a warp seldom add to one address (with
// one copy of an 11-bit digit the selection of 8192 tokens took 32 us, most of it there).  Which
// tokens are above the threshold, and which equal it, become bit masks of 32 tokens; prefix sums of
// their population counts give every freed slot and every moving token its number.
// The CTA then moves the rows itself, or, where min(keep, the table's tokens - keep) rows may be too many
// for that, a second kernel does (evict_plan in ops_api.cuh, with both sides measured).
//
// What bounds it: after long prompts, the rows that move (32 requests x 8 heads of 4097 to 8192 tokens,
// keep 2048: 22 us of selection, then 66 us for about 390 MB of rows read and written, 5.9 TB/s); in
// steady eviction of up to 128 tokens of 2176 (64 x 2 heads: 10 us), the selection's latency: two
// passes over the weights, five over shared memory, a dozen barriers.
#pragma once
#include "common.cuh"

namespace fa {
namespace evict {
constexpr int THREADS = 512;
constexpr int BS = 16;
constexpr int COPIES = 16;       // of the first digit's histogram
constexpr int BINS = 512 * COPIES;
constexpr int MAX_KEYS = 40960;  // tokens whose keys (and masks) fit in shared memory
}  // namespace evict

struct EvictParams {
  const int *bt, *ctx, *seq;
  const float* weights;  // [R, Hkv, M], M = max_blocks * 16
  const int* slot_pos;   // [R, Hkv, M]
  float* weights_out;
  int* slot_pos_out;
  int* new_ctx;    // [R]
  int* moves;      // [R * Hkv][2 * cap]: destinations, then sources, as cache rows (block * Hkv + h) * 16 + slot
  int* n_moves;    // [R * Hkv] (both for the second kernel)
  uint32_t* masks; // [R * Hkv][2][ceil(M / 32)], past MAX_KEYS only
  uint4 *kc, *vc;
  int R, Hkv, max_blocks, num_blocks, keep, recent, cap;
  int row16;       // 16-byte pieces of a cache row
  bool in_smem;    // keys, masks and lists in shared memory
  bool fused;      // this kernel moves the rows (in_smem only)
};

// Larger weight, larger key; -0 as +0; NaN below everything.
__device__ __forceinline__ uint32_t evict_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the CTA, and the total.
__device__ __forceinline__ int evict_scan(int v, int4* s_warp, int& total) {
  const int lane = lane_id(), warp = warp_id();
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the last call's readers are done
  if (lane == 31) reinterpret_cast<int*>(s_warp)[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < evict::THREADS / 32; w += 4) {
    const int4 t = s_warp[w / 4];
    before += (w < warp ? t.x : 0) + (w + 1 < warp ? t.y : 0) + (w + 2 < warp ? t.z : 0) + (w + 3 < warp ? t.w : 0);
    all += t.x + t.y + t.z + t.w;
  }
  total = all;
  return before + x - v;
}

// Copy `moves` key and value rows: a group of lanes a row, thread t of `threads`.  U rows are read
// before the first is written, so a thread has 2 U pieces of 16 bytes in flight.
__device__ __forceinline__ void evict_move_rows(const EvictParams& p, const int* dst, const int* src, int moves, int t,
                                                int threads) {
  const int lanes = p.row16 <= 8 ? 8 : p.row16 <= 16 ? 16 : 32;  // 96 columns: 12 of 16 work
  const int e = t & (lanes - 1), step = threads / lanes;
  if (e >= p.row16) return;
  constexpr int U = 2;
  for (int64_t i = t / lanes; i < moves; i += U * step) {
    uint4 k[U], v[U];
    int to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = i + u * step;
      to[u] = -1;
      if (at < moves) {
        const int a = src[at];
        to[u] = a < 0 ? -1 : dst[at];  // (a block id out of range was flagged)
        if (to[u] >= 0) {
          k[u] = p.kc[size_t(a) * p.row16 + e];
          v[u] = p.vc[size_t(a) * p.row16 + e];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0) {
        p.kc[size_t(to[u]) * p.row16 + e] = k[u];
        p.vc[size_t(to[u]) * p.row16 + e] = v[u];
      }
  }
}

__global__ void __launch_bounds__(evict::THREADS) fa_evict_select_kernel(const __grid_constant__ EvictParams p) {
  using namespace evict;
  extern __shared__ __align__(16) uint32_t evict_smem[];
  __shared__ __align__(16) int s_hist[BINS];
  __shared__ int4 s_warp[THREADS / 128];
  __shared__ int s_found[3];  // the digit's bin, how many of its tokens are needed, and how many it has
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (the second kernel's CTAs, held ready on the SMs, left it 10 us slower)
  if (p.fused) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = lane_id();
  const size_t rh = size_t(r) * p.Hkv + h;
  const int M = p.max_blocks * BS;
  const float* w = p.weights + rh * M;
  const int* sp = p.slot_pos + rh * M;
  float* wo = p.weights_out + rh * M;
  int* so = p.slot_pos_out + rh * M;
  const int* bt = p.bt + size_t(r) * p.max_blocks;
  const int n = p.ctx[r], seq = p.seq[r];
  const bool bad = n < 0 || n > M || seq < n;
  if (bad || n <= p.keep) {  // out of range: left as it is; nothing to evict: the positions are written down
    if (tid == 0) {
      if (bad) set_status(FA_ERR_INVALID_ARG, 400);
      if (!p.fused) p.n_moves[rh] = 0;
      if (h == 0) p.new_ctx[r] = n;
    }
    for (int s = tid; s < M; s += THREADS) {
      const int pos = sp[s];
      const float v = w[s];
      wo[s] = bad || s < n ? v : 0.f;
      so[s] = bad ? pos : s >= n ? -1 : pos >= 0 ? pos : seq - n + s;
    }
    return;
  }
  if (tid == 0 && h == 0) p.new_ctx[r] = p.keep;
  auto pos_of = [&](int s, int v) { return v >= 0 ? v : seq - n + s; };
  const int newest = seq - p.recent;
  auto key_from = [&](int s, float wt, int v) { return pos_of(s, v) >= newest ? 0xffffffffu : evict_key(wt); };
  const int words = (n + 31) / 32, MW = (M + 31) / 32;
  uint32_t* s_key = evict_smem;                                           // [n]
  uint32_t* above = p.in_smem ? evict_smem + M : p.masks + rh * 2 * MW;  // [words]: key above the threshold, kept
  uint32_t* equal = above + MW;                                           // [words]: key at it; then the words' numbers
  const float4* w4 = reinterpret_cast<const float4*>(w);
  const int4* sp4 = reinterpret_cast<const int4*>(sp);
  for (int i = tid; i < BINS / 4; i += THREADS) reinterpret_cast<int4*>(s_hist)[i] = make_int4(0, 0, 0, 0);
  __syncthreads();
  auto count_first = [&](int s, uint32_t k) {
    if (s < n) atomicAdd(&s_hist[int(k >> 23) * COPIES + (lane & (COPIES - 1))], 1);
  };
  if (p.in_smem) {
#pragma unroll 4
    for (int i = tid; 4 * i < n; i += THREADS) {  // (keys past n are not used)
      const float4 a = __ldg(w4 + i);
      const int4 v = __ldg(sp4 + i);
      const uint4 k = make_uint4(key_from(4 * i, a.x, v.x), key_from(4 * i + 1, a.y, v.y),
                                 key_from(4 * i + 2, a.z, v.z), key_from(4 * i + 3, a.w, v.w));
      reinterpret_cast<uint4*>(s_key)[i] = k;
      count_first(4 * i, k.x);
      count_first(4 * i + 1, k.y);
      count_first(4 * i + 2, k.z);
      count_first(4 * i + 3, k.w);
    }
  }
  auto key_of = [&](int s) { return p.in_smem ? s_key[s] : key_from(s, __ldg(w + s), __ldg(sp + s)); };

  // A threshold: keys above it are kept, and `need` of the tokens at it.  The keep-th largest key, digit
  // by digit, or the key below the last bin where that bin is kept whole.
  uint32_t thr = 0;
  int need = p.keep;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 23 : pass == 1 ? 12 : 0;
    const int bins = pass == 0 ? 512 : pass == 1 ? 2048 : 4096;
    if (pass > 0) {
      const uint32_t mask = 0xffffffffu << (pass == 1 ? 23 : 12);
#pragma unroll 4
      for (int s = tid; s < n; s += THREADS) {
        const uint32_t k = key_of(s);
        if ((k & mask) == thr) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1);
      }
    } else if (!p.in_smem) {
      for (int s = tid; s < n; s += THREADS) count_first(s, key_of(s));
    }
    __syncthreads();
    // a few bins a thread, the highest first
    const int per = bins / THREADS, top = bins - 1 - per * tid;
    int c[8], sum = 0, total;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      c[i] = 0;
      if (pass == 0) {
#pragma unroll
        for (int j = 0; j < COPIES / 4; ++j) {
          const int at = (top - i) * (COPIES / 4) + ((j + lane) & (COPIES / 4 - 1));
          const int4 t = reinterpret_cast<const int4*>(s_hist)[at];
          c[i] += t.x + t.y + t.z + t.w;
        }
      } else {
        c[i] = s_hist[top - i];
      }
      sum += c[i];
    }
    int before = evict_scan(sum, s_warp, total);
    if (before < need && need <= before + sum) {
#pragma unroll
      for (int i = 0; i < per; ++i) {
        if (before < need && need <= before + c[i]) {
          s_found[0] = top - i;
          s_found[1] = need - before;
          s_found[2] = c[i];
        }
        before += c[i];
      }
    }
    if (pass < 2)
      for (int i = tid; i < 1024; i += THREADS)  // (every thread has read its bins: evict_scan)
        reinterpret_cast<int4*>(s_hist)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    thr |= uint32_t(s_found[0]) << shift;
    need = s_found[1];
    if (need == s_found[2]) {  // all of the bin: the digits below it do not matter
      thr -= 1;                // (> 0: not every token is kept)
      need = 0;
      break;
    }
  }

#pragma unroll 4
  for (int s = tid; s - lane < n; s += THREADS) {  // (whole warps)
    const uint32_t k = s < n ? key_of(s) : 0u;
    const uint32_t a = __ballot_sync(0xffffffffu, s < n && k > thr), e = __ballot_sync(0xffffffffu, s < n && k == thr);
    if (lane == 0) {
      above[s >> 5] = a;
      equal[s >> 5] = e;
    }
  }
  __syncthreads();
  // kept = above, and the first `need` at the threshold; then each word's first number among the
  // freed slots (below keep) and the moving tokens (past it)
  int eq_done = 0, hole_done = 0, mover_done = 0;
  for (int b = 0; b < words; b += THREADS) {
    const int i = b + tid;
    const uint32_t a = i < words ? above[i] : 0u;
    uint32_t e = i < words ? equal[i] : 0u;
    int total;
    const int skip = need - (eq_done + evict_scan(__popc(e), s_warp, total));  // of this word's, so many are kept
    eq_done += total;
    int drop = __popc(e) - max(0, skip);
    for (; drop > 0; --drop) e &= ~(0x80000000u >> __clz(e));
    const uint32_t kept = a | e;
    // bits of slots below keep, and of slots below n
    const int lo = p.keep - 32 * i, hi = n - 32 * i;
    const uint32_t below = lo <= 0 ? 0u : lo >= 32 ? 0xffffffffu : (1u << lo) - 1;
    const uint32_t live = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1;
    const int holes = __popc(~kept & below & live), movers = __popc(kept & ~below);
    // (both sums of a round fit in 16 bits: 512 words of 32)
    const int first = evict_scan(holes | movers << 16, s_warp, total);
    const int hole = (first & 0xffff) + hole_done, mover = int(unsigned(first) >> 16) + mover_done;
    hole_done += total & 0xffff;
    mover_done += int(unsigned(total) >> 16);
    if (i < words) {
      above[i] = kept;
      equal[i] = uint32_t(lo > 0 ? hole : mover);  // (in the one word that may hold both, movers start at 0)
    }
  }
  __syncthreads();
  const int moves = mover_done;  // == hole_done
  // The moving tokens in order, in the keys' place once nothing reads a key (moves <= n / 2), and
  // the slots past keep emptied.
  const bool in_place = p.in_smem && p.fused;
  int* g_dst = p.moves + rh * 2 * p.cap;
  int* src = p.in_smem ? reinterpret_cast<int*>(s_key) : g_dst + p.cap;
  for (int i = p.keep / 4 + tid; 4 * i < M; i += THREADS) {
    if (4 * i < n) {
      const uint32_t kept = above[i >> 3];
      const int lo = p.keep - ((4 * i) & ~31);
      const uint32_t past = kept & (lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : ~((1u << lo) - 1));
      const int number = lo > 0 ? 0 : int(equal[i >> 3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t bit = 1u << ((4 * i + j) & 31);
        if (past & bit) src[number + __popc(past & (bit - 1))] = 4 * i + j;
      }
    }
    if (4 * i >= p.keep) {
      reinterpret_cast<float4*>(wo)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      reinterpret_cast<int4*>(so)[i] = make_int4(-1, -1, -1, -1);
    }
  }
  __syncthreads();
  if (tid == 0 && !p.fused) p.n_moves[rh] = moves;
  // The slots below keep: their own token, or the moving token of the freed slot's number, whose
  // weight and position are gathered here (scattered to the slots afterwards, 4 bytes of a sector
  // each, the selection of 32 x 8 x 8192 tokens took 24.3 us; gathered, 23.1 us).
  int* out_src = in_place ? src : g_dst + p.cap;
  int* out_dst = in_place ? src + M / 2 : g_dst;
#pragma unroll 2
  for (int i = tid; 4 * i < p.keep; i += THREADS) {
    const uint32_t kept = above[i >> 3];
    const int number = int(equal[i >> 3]);
    const float4 a = __ldg(w4 + i);
    const int4 v = __ldg(sp4 + i);
    float wt[4] = {a.x, a.y, a.z, a.w};
    int pos[4] = {v.x, v.y, v.z, v.w}, from[4], page[4], to = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the slot whose token comes here
      const int s = 4 * i + j;
      from[j] = s >= p.keep ? -1 : (kept >> (s & 31)) & 1 ? s : src[number + __popc(~kept & ((1u << (s & 31)) - 1))];
    }
    bool moved = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (from[j] < 0 || from[j] == 4 * i + j) continue;
      moved = true;
      wt[j] = __ldg(w + from[j]);
      pos[j] = __ldg(sp + from[j]);
      page[j] = __ldg(bt + from[j] / BS);
    }
    if (moved) to = __ldg(bt + i / (BS / 4));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = 4 * i + j;
      if (from[j] >= 0 && from[j] != s) {
        const bool ok = page[j] >= 0 && page[j] < p.num_blocks && to >= 0 && to < p.num_blocks;
        if (!ok) set_status(FA_ERR_INVALID_ARG, 401);
        const int at = number + __popc(~kept & ((1u << (s & 31)) - 1));
        out_src[at] = ok ? (page[j] * p.Hkv + h) * BS + from[j] % BS : -1;
        out_dst[at] = ok ? (to * p.Hkv + h) * BS + s % BS : -1;
      }
      wt[j] = from[j] >= 0 ? wt[j] : 0.f;
      pos[j] = from[j] >= 0 ? pos_of(from[j], pos[j]) : -1;
    }
    reinterpret_cast<float4*>(wo)[i] = make_float4(wt[0], wt[1], wt[2], wt[3]);
    reinterpret_cast<int4*>(so)[i] = make_int4(pos[0], pos[1], pos[2], pos[3]);
  }
  if (!p.fused) return;
  __syncthreads();
  evict_move_rows(p, out_dst, out_src, moves, tid, THREADS);
}

__global__ void __launch_bounds__(256) fa_evict_move_kernel(const __grid_constant__ EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const size_t rh = size_t(blockIdx.z) * p.Hkv + blockIdx.y;
  const int* dst = p.moves + rh * 2 * p.cap;
  evict_move_rows(p, dst, dst + p.cap, p.n_moves[rh], blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

}  // namespace fa
