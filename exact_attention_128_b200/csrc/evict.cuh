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
// Selection: each token's key is its weight as an order-preserving 32-bit integer, all ones where
// it is protected; the keep-th largest key is found digit by digit from histograms.  One CTA per
// (r, h) selects and writes the lists of moves, a second kernel moves the rows.
#pragma once
#include "common.cuh"

namespace fa {
namespace evict {
constexpr int THREADS = 512;
constexpr int BS = 16;
}  // namespace evict

struct EvictParams {
  const int *bt, *ctx, *seq;
  const float* weights;   // [R, Hkv, M], M = max_blocks * 16
  const int* slot_pos;    // [R, Hkv, M]
  float* weights_out;
  int* slot_pos_out;
  int* new_ctx;           // [R]
  int* moves;             // [R * Hkv][2 * cap]: destinations, then sources
  int* n_moves;           // [R * Hkv]
  uint4 *kc, *vc;
  int R, Hkv, max_blocks, num_blocks, keep, recent, cap;
  int row16;              // 16-byte pieces of a cache row
};

// Larger weight, larger key; -0 as +0; NaN below everything.
__device__ __forceinline__ uint32_t evict_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the CTA of v (two 16-bit halves), and the total.
__device__ __forceinline__ uint32_t evict_scan(uint32_t v, uint32_t* s_warp, uint32_t& total) {
  const int lane = lane_id(), warp = warp_id();
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the last call's readers are done
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < evict::THREADS / 32; ++w) {
    const uint32_t t = s_warp[w];
    before += w < warp ? t : 0u;
    all += t;
  }
  total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(evict::THREADS) fa_evict_select_kernel(const __grid_constant__ EvictParams p) {
  using namespace evict;
  __shared__ int s_hist[256];
  __shared__ uint32_t s_warp[THREADS / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int r = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  const size_t rh = size_t(r) * p.Hkv + h;
  const int M = p.max_blocks * BS;
  const float* w = p.weights + rh * M;
  const int* sp = p.slot_pos + rh * M;
  float* wo = p.weights_out + rh * M;
  int* so = p.slot_pos_out + rh * M;
  int n = p.ctx[r];
  const int seq = p.seq[r];
  if (n < 0 || n > M || seq < n) {
    if (tid == 0) {
      set_status(FA_ERR_INVALID_ARG, 400);
      p.n_moves[rh] = 0;
      if (h == 0) p.new_ctx[r] = n;
    }
    for (int s = tid; s < M; s += THREADS) {
      wo[s] = w[s];
      so[s] = sp[s];
    }
    return;
  }
  if (tid == 0 && h == 0) p.new_ctx[r] = min(n, p.keep);
  auto pos_of = [&](int s) {
    const int v = sp[s];
    return v >= 0 ? v : seq - n + s;
  };
  auto key_of = [&](int s) { return pos_of(s) >= seq - p.recent ? 0xffffffffu : evict_key(w[s]); };

  uint32_t thr = 0;  // the keep-th largest key; `ties` of the tokens that have it are kept
  int ties = n;
  if (n > p.keep) {
    if (tid == 0) {
      s_prefix = 0;
      s_need = p.keep;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += THREADS) s_hist[i] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int s = tid; s < n; s += THREADS) {
        const uint32_t k = key_of(s);
        if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int need = s_need, b = 255;
        for (; b > 0 && s_hist[b] < need; --b) need -= s_hist[b];
        s_need = need;
        s_prefix = prefix | (uint32_t(b) << shift);
      }
      __syncthreads();
    }
    thr = s_prefix;
    ties = s_need;
  }

  // slots in order: which are kept, the freed ones below `keep`, the kept ones past it
  const int lim = min(n, p.keep);
  int* dst = p.moves + rh * 2 * p.cap;
  int* src = dst + p.cap;
  int eq_before = 0, holes = 0, movers = 0;
  for (int base = 0; base < n; base += THREADS) {
    const int s = base + tid;
    uint32_t key = 0;
    int pos = -1;
    float wt = 0.f;
    if (s < n) {
      pos = pos_of(s);
      wt = w[s];
      key = pos >= seq - p.recent ? 0xffffffffu : evict_key(wt);
    }
    const bool eq = s < n && key == thr;
    uint32_t total;
    const uint32_t rank = evict_scan(eq ? 1u : 0u, s_warp, total);
    const bool kept = s < n && (n <= p.keep || key > thr || (eq && int(rank) + eq_before < ties));
    eq_before += total;
    const bool hole = s < lim && !kept, mover = kept && s >= p.keep;
    const uint32_t at = evict_scan((hole ? 1u : 0u) | (mover ? 0x10000u : 0u), s_warp, total);
    if (hole) dst[holes + (at & 0xffff)] = s;
    if (mover) src[movers + (at >> 16)] = s;
    holes += total & 0xffff;
    movers += total >> 16;
    if (s < n) {
      const bool stays = kept && s < p.keep;
      wo[s] = stays ? wt : 0.f;
      so[s] = stays ? pos : -1;
    }
  }
  for (int s = n + tid; s < M; s += THREADS) {
    wo[s] = 0.f;
    so[s] = -1;
  }
  __syncthreads();
  if (tid == 0) p.n_moves[rh] = movers;  // == holes
  for (int i = tid; i < movers; i += THREADS) {
    wo[dst[i]] = w[src[i]];
    so[dst[i]] = pos_of(src[i]);
  }
}

// 32 threads per move at 128 columns: 16 for the key's 16-byte pieces, 16 for the value's.
__global__ void __launch_bounds__(256) fa_evict_move_kernel(const __grid_constant__ EvictParams p) {
  using namespace evict;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int r = blockIdx.z, h = blockIdx.y;
  const size_t rh = size_t(r) * p.Hkv + h;
  const int moves = p.n_moves[rh];
  const int* dst = p.moves + rh * 2 * p.cap;
  const int* src = dst + p.cap;
  const int* bt = p.bt + size_t(r) * p.max_blocks;
  const int per = 2 * p.row16;
  const int64_t all = int64_t(moves) * per;
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < all; t += int64_t(gridDim.x) * 256) {
    const int i = int(t / per), piece = int(t % per);
    const int a = src[i], b = dst[i];
    const int pa = bt[a / BS], pb = bt[b / BS];
    if (pa < 0 || pa >= p.num_blocks || pb < 0 || pb >= p.num_blocks) {
      set_status(FA_ERR_INVALID_ARG, 401);
      continue;
    }
    uint4* c = piece < p.row16 ? p.kc : p.vc;
    const int e = piece < p.row16 ? piece : piece - p.row16;
    c[((size_t(pb) * p.Hkv + h) * BS + b % BS) * p.row16 + e] = c[((size_t(pa) * p.Hkv + h) * BS + a % BS) * p.row16 + e];
  }
}

}  // namespace fa
