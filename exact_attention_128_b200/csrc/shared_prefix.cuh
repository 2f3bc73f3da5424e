// shared_prefix.cuh — the prefix part of a decode step of many requests, on the tensor cores.
//
// Requests that share a prefix turn its attention into a matrix product: the R * G query rows of a
// kv head (request-major, G = Hq / Hkv heads each) against the prefix's P keys, with the
// online-softmax recurrence over tiles of BN keys (running maximum m, sum l, numerator u).  Each
// K/V block is read once per 256 rows.  What is left is one partial result (u / l, lse) per row
// and run of tiles, merged by their mass with the requests' own tokens (decode_part.cuh).
//
// Work: an item is (kv head, two row tiles); a row tile is the most whole requests that fit 128
// rows, so that one TMA box {64 columns, G heads, requests} fills it.  Items all have the same
// nt = ceil(P / BN) key tiles, and CTA c of C takes tiles [c W / C, (c + 1) W / C) of all W =
// items * nt: every CTA does the same work, whatever the batch and the prefix (P is read on the
// device), and an item's tiles fall to a few consecutive CTAs, one partial result each.
//   warp 0     producer of Q (by TMA, per item) and K: lane i < BN / 16 looks block i of a key tile
//              up in the prefix table and issues its 16-row boxes; warp V_WARP the same for V.
//   warp 1     MMA issuer: S_t = Q_t K^T into TMEM, then u_t += P_t V with P_t (two parts) read from TMEM.
//   warps 2-9  softmax of row tiles 0 and 1, one thread per row.
// Scores are double-buffered in TMEM and issued one key tile ahead, so a softmax warp goes from
// one tile to the next without waiting for its own P V (with one buffer, the chain S, softmax,
// P V of a 64-key tile took 3290 cycles a step of two row tiles where two took 2150, with one product).
// Only the rare step whose maximum rises waits for the P V before it, to rescale u.
// What bounds it: the chain S, P V of a row tile.  Its MMAs need 1540 cycles a step of two row tiles at
// the full rate, but S reads Q from shared memory again for every 64-key tile, 192 bytes a cycle where
// there are 128, and each hand-over between the MMA warp and the softmax costs some 200; the exponentials,
// 1024 cycles, run beside it.  A step takes 1.9 us (1.5 with one product).  256 requests of 32 heads, 8 kv heads,
// 16384 shared tokens: 107 us, 640 TFLOP/s, the tensor pipe 48 % busy; with the own tokens and the join
// 142 us in short runs, 165 to 167 power-capped.
// BN = 64 and two K/V stages keep the CTA at 150 KB of shared memory and 352 threads of at most
// 104 registers, so that a CTA of the requests' own (memory-bound) part runs on the SM beside it.
// P is multiplied as the sum of two bf16 parts, its rounding and the rest, as in the pieces
// (decode_part.cuh), so that a request's precision does not depend on its batch or its table: both
// parts fit the 64 columns of the scores they come from.  The second product costs 256 requests behind
// 16384 tokens 17 us (125 -> 142 us the step, the MMAs 14 of them), 8 behind 2000 tokens 0.6 us.
#pragma once
#include "decode_part.cuh"

namespace fa {

// All N phases: the barriers are looked at together, since a look takes some 200 cycles even where
// the phase is over (one after the other, six of them took half of a step's 2500 cycles).
template <int N>
__device__ __forceinline__ bool warp_wait_all(uint64_t* const (&bar)[N], const uint32_t (&parity)[N], uint64_t limit_ns,
                                              volatile int* abort_flag, int where) {
#pragma unroll 1
  for (int look = 0; look < 32; ++look) {
    bool over = true;
#pragma unroll
    for (int i = 0; i < N; ++i) over &= mbar_try_wait(bar[i], parity[i]);
    if (__all_sync(0xffffffffu, over)) return true;
  }
  bool ok = true;
#pragma unroll
  for (int i = 0; i < N; ++i) ok = ok && warp_wait(bar[i], parity[i], limit_ns, abort_flag, where + i);
  return ok;
}

template <int D>
struct PrefixCfg {
  static constexpr int BM = 128, BN = PrefixDeal::BN;
  static constexpr int KB = D / 64;
  static constexpr int Q_TILE = BM * D * 2, KV_TILE = BN * D * 2;
  static constexpr int NSTAGE = D == 128 ? 2 : 4;
  static constexpr int STG_WARP = 32 * 16 * 4;  // epilogue staging of a warp: 32 rows x 16 columns fp32
  static constexpr int OFF_Q = 0, OFF_K = 2 * Q_TILE, OFF_V = OFF_K + NSTAGE * KV_TILE;
  static constexpr int OFF_STG = OFF_V + NSTAGE * KV_TILE, OFF_BAR = OFF_STG + 8 * STG_WARP;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;  // + barriers, alignment of the base
  static constexpr int V_WARP = 10, THREADS = 352;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 4 * BN;  // S of row tile t, buffer b at (2 b + t) * BN; u_t at COL_O + t * D
  static_assert(4 * BN + 2 * D <= 512, "TMEM");
};

struct PrefixParams {
  const int *pbt, *plen;
  float* part_o;    // [items][parts][2 tiles][128 rows][D]
  float* part_lse;  // [items][parts][2][128], base 2
  int R, Hkv, G, RT;  // RT requests per row tile
  int items, pairs;   // items = Hkv * pairs, kv-head-major
  int parts;
  int prefix_blocks, num_blocks;
  float scale_log2;
  uint64_t wait_ns;
  int withhold;  // K tiles that a CTA loads at most (the self-test's; INT_MAX otherwise)
};

struct PrefixBars {
  uint64_t q_full, q_empty, k_full[4], v_full[4], k_empty[4], v_empty[4];
  uint64_t s_full[2][2], p_full[2][2];  // [row tile][buffer]
  uint64_t drained;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PrefixBars) <= 256, "barrier area");

// (104 registers, so that the register file holds a CTA of the requests' own part too.  With one product
// of P: 96 and 112 took the same time, with 120 it did not fit beside this one, 3 us more for 256
// requests.  With two, a few values spill: 36 bytes at d = 128.)
template <int D>
__global__ void __maxnreg__(104)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PrefixParams p) {
  using C = PrefixCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PrefixBars* bars = reinterpret_cast<PrefixBars*>(smem + C::OFF_BAR);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < C::NSTAGE; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->s_full[t][b], 1);
        mbar_init(&bars->p_full[t][b], 4);
      }
    }
    mbar_init(&bars->drained, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the grid after this one (the requests' own tokens) needs nothing of it and may start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int P = p.plen[0];
  if (P < 0 || P > p.prefix_blocks * 16) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(FA_ERR_INVALID_ARG, 302);
    P = 0;
  }
  const uint32_t tmem = bars->tmem_base;
  const uint32_t sQ = smem_u32(smem + C::OFF_Q), sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
  const PrefixDeal deal(P, p.items);
  const bool any = P > 0 && int(blockIdx.x) < deal.ctas;
  const long long x0 = any ? deal.begin(blockIdx.x) : 0, x1 = any ? deal.begin(blockIdx.x + 1) : 0;
  const int nblk = (P + 15) / 16;

  if (warp == 0 || warp == C::V_WARP) {
    // K (and Q) and V have a producer each: neither waits for the other's stage, so a load is
    // issued two steps before its tile is due.
    constexpr int NB = C::BN / 16;
    const bool is_v = warp != 0;
    const CUtensorMap* map = is_v ? &tmV : &tmK;
    uint64_t* full = is_v ? bars->v_full : bars->k_full;
    uint64_t* empty = is_v ? bars->v_empty : bars->k_empty;
    uint8_t* ring = smem + (is_v ? C::OFF_V : C::OFF_K);
    if (lane == 0) {
      prefetch_tmap(map);
      if (!is_v) prefetch_tmap(&tmQ);
    }
    int kv = 0, local = 0;  // tiles issued, items begun
    bool ok = true;
    for (long long x = x0; x < x1 && ok; ++local) {
      const int it = int(x / deal.nt), j0 = int(x - (long long)(it)*deal.nt);
      const int j1 = int(min((long long)(deal.nt), j0 + (x1 - x)));
      x += j1 - j0;
      const int hk = it / p.pairs, pair = it - hk * p.pairs;
      int ph = (lane < NB && j0 * NB + lane < nblk) ? __ldg(p.pbt + j0 * NB + lane) : 0;
      if (!is_v) {
        if (local > 0 && !(ok = warp_wait(&bars->q_empty, (local - 1) & 1, p.wait_ns, abort_flag, 311))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full, uint32_t(2 * C::KB * 128 * p.G * p.RT));
          for (int t = 0; t < 2; ++t)
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_3d(smem + C::OFF_Q + t * C::Q_TILE + kb * C::BM * 128, &tmQ, &bars->q_full, kb * 64, hk * p.G,
                          (2 * pair + t) * p.RT);
        }
      }
      for (int j = j0; j < j1; ++j, ++kv) {
        if (!is_v && kv >= p.withhold) {
          ok = false;
          break;
        }
        const int st = kv % C::NSTAGE, round = kv / C::NSTAGE;
        const int lb = j * NB + lane;
        const int ph_next = (lane < NB && j + 1 < j1 && lb + NB < nblk) ? __ldg(p.pbt + lb + NB) : 0;
        const int nload = min(NB, nblk - j * NB);  // >= 1
        int crow = 0;
        if (lane < nload) {
          int pb = ph;
          if (pb < 0 || pb >= p.num_blocks) {
            set_status(FA_ERR_INVALID_ARG, 301);
            pb = 0;
          }
          crow = (pb * p.Hkv + hk) * 16;
        }
        ph = ph_next;
        if (round > 0 && !(ok = warp_wait(&empty[st], (round - 1) & 1, p.wait_ns, abort_flag, 310 + 2 * is_v))) break;
        uint8_t* tile = ring + st * C::KV_TILE;
        if (is_v && nload < NB) {  // V rows of blocks past the prefix: zero (their P is 0; 0 * NaN would not be)
          for (int kb = 0; kb < C::KB; ++kb)
            for (int i = nload * 128 + lane; i < C::BN * 8; i += 32)
              *reinterpret_cast<uint4*>(tile + kb * C::BN * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[st], uint32_t(nload) * 16 * 128 * C::KB);
        __syncwarp();
        if (lane < nload)
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_2d(smem_u32(tile + kb * C::BN * 128 + lane * 16 * 128), map, &full[st], kb * 64, crow);
      }
    }
    if (!ok && lane == 0) {  // a wait ran out: let the loads in flight land before the CTA ends
      for (int i = max(0, kv - C::NSTAGE); i < kv; ++i)
        mbar_wait_bounded(&full[i % C::NSTAGE], (i / C::NSTAGE) & 1, p.wait_ns);
      if (!is_v && local > 0) mbar_wait_bounded(&bars->q_full, (local - 1) & 1, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t leader = elect_one();
    constexpr uint32_t idS = idesc_bf16_f32(128, C::BN, 0), idPV = idesc_bf16_f32(128, D, 1);
    const uint64_t dQ = sdesc_sw128(sQ, 16, 1024), dK = sdesc_sw128(sK, 16, 1024);
    const uint64_t dV = sdesc_sw128(sV, C::BN * 128, 1024);
    // scores of both row tiles against the K tile of ring position i, into the buffers of step g
    auto issue_S = [&](int i, int g) {
      const int st = i % C::NSTAGE;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int kb = ks >> 2, kin = ks & 3;
          mma_ss_p(tmem + (2 * (g & 1) + t) * C::BN, desc_add(dQ, t * C::Q_TILE + kb * C::BM * 128 + kin * 32),
                   desc_add(dK, st * C::KV_TILE + kb * C::BN * 128 + kin * 32), idS, ks > 0 ? 1u : 0u, leader);
        }
        mma_commit_p(&bars->s_full[t][g & 1], leader);
      }
      mma_commit_p(&bars->k_empty[st], leader);
    };
    auto issue_PV = [&](int t, int st, int g, bool first) {
#pragma unroll
      for (int ks = 0; ks < C::BN / 16; ++ks)
#pragma unroll
        for (int half = 0; half < 2; ++half)  // P rounded, then the rest
          mma_ts_p(tmem + C::COL_O + t * D, tmem + (2 * (g & 1) + t) * C::BN + half * (C::BN / 2) + ks * 8,
                   desc_add(dV, st * C::KV_TILE + ks * 16 * 128), idPV, (!first || ks + half > 0) ? 1u : 0u, leader);
    };
    int kv = 0, local = 0;  // kv: K/V tiles so far, which is also the step (every tile is one)
    bool ok = true;
    // The scores of a step go where P of two steps before was.  The tensor core keeps the order of
    // MMAs of one shape and accumulator only, so that step's P V must be waited for: v_empty tells
    // that P V of both row tiles is over (every commit costs some 100 cycles, so there is one).
    for (long long x = x0; x < x1 && ok; ++local) {
      const int it = int(x / deal.nt), j0 = int(x - (long long)(it)*deal.nt);
      const int j1 = int(min((long long)(deal.nt), j0 + (x1 - x)));
      x += j1 - j0;
      ok = warp_wait(&bars->q_full, local & 1, p.wait_ns, abort_flag, 320) &&
           warp_wait(&bars->k_full[kv % C::NSTAGE], (kv / C::NSTAGE) & 1, p.wait_ns, abort_flag, 321);
      if (!ok) break;
      tc_fence_after();
      issue_S(kv, kv);  // (over P of step kv - 2, which was waited for before step kv - 1)
      if (j1 - j0 == 1) mma_commit_p(&bars->q_empty, leader);
      for (int j = j0; j < j1; ++j, ++kv) {
        const int st = kv % C::NSTAGE;
        const int i = kv + 1, st2 = i % C::NSTAGE;
        // step kv - 1
        uint64_t* const last_pv = &bars->v_empty[(i + C::NSTAGE - 2) % C::NSTAGE];
        const uint32_t pk = (i / C::NSTAGE) & 1, pd = kv > 0 ? ((kv - 1) / C::NSTAGE) & 1 : 1;
        if (j + 1 < j1) {
          // (before the first step that barrier is in its first phase, whose predecessor counts as over)
          ok = warp_wait_all({&bars->k_full[st2], last_pv}, {pk, pd}, p.wait_ns, abort_flag, 324);
          if (!ok) break;
          tc_fence_after();
          issue_S(i, i);
          if (j + 2 == j1) mma_commit_p(&bars->q_empty, leader);  // the item's last scores
        } else if (!(ok = warp_wait(last_pv, pd, p.wait_ns, abort_flag, 326))) {
          break;
        }
        const uint32_t pp = (kv >> 1) & 1;
        ok = warp_wait_all({&bars->v_full[st], &bars->p_full[0][kv & 1], &bars->p_full[1][kv & 1]},
                           {uint32_t((kv / C::NSTAGE) & 1), pp, pp}, p.wait_ns, abort_flag, 327);
        if (!ok) break;
        if ((P & 15) != 0 && (P - 1) / C::BN == j) {  // V rows of the last block's unused slots: zero
          uint8_t* sv = smem + C::OFF_V + st * C::KV_TILE;
          const int r0 = P - j * C::BN, r1 = nblk * 16 - j * C::BN;
          for (int kb = 0; kb < C::KB; ++kb)
            for (int z = r0 * 8 + lane; z < r1 * 8; z += 32)
              *reinterpret_cast<uint4*>(sv + kb * C::BN * 128 + z * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        issue_PV(0, st, kv, j == j0);
        issue_PV(1, st, kv, j == j0);
        mma_commit_p(&bars->v_empty[st], leader);
      }
    }
    if (!ok) {  // likewise the MMAs, before TMEM is given back
      mma_commit_p(&bars->drained, leader);
      if (lane == 0) mbar_wait_bounded(&bars->drained, 0, p.wait_ns);
      __syncwarp();
    }
  } else {
    const int t = (warp - 2) >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t lane_off = uint32_t(wq * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::COL_O + t * D;
    const float sl2 = p.scale_log2;
    int g = 0, local = 0;
    bool ok = true;
    for (long long x = x0; x < x1 && ok; ++local) {
      const int it = int(x / deal.nt), j0 = int(x - (long long)(it)*deal.nt);
      const int j1 = int(min((long long)(deal.nt), j0 + (x1 - x)));
      x += j1 - j0;
      const int req = (2 * (it % p.pairs) + t) * p.RT + r / p.G;
      const bool idle = __all_sync(0xffffffffu, r >= p.G * p.RT || req >= p.R);
      float m = -INFINITY, l = 0.f;
      for (int j = j0; j < j1; ++j, ++g) {
        const uint32_t tS = tmem + lane_off + (2 * (g & 1) + t) * C::BN;
        if (!(ok = warp_wait(&bars->s_full[t][g & 1], (g >> 1) & 1, p.wait_ns, abort_flag, 330 + t))) break;
        if (!idle) {
          tc_fence_after();
          uint32_t sr[C::BN];
#pragma unroll
          for (int c = 0; c < C::BN / 32; ++c)
            tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
          tmem_wait_ld();
          float f[C::BN];
#pragma unroll
          for (int c = 0; c < C::BN; ++c) f[c] = __uint_as_float(sr[c]);
          const int lim = P - j * C::BN;
          if (lim < C::BN) {
#pragma unroll
            for (int c = 0; c < C::BN; ++c) f[c] = (c < lim) ? f[c] : -INFINITY;
          }
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(f[k], f[8 + k]);
#pragma unroll
          for (int c = 16; c < C::BN; c += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], f[c + k], f[c + 8 + k]);
          const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
          // the reference of l and u moves only when the maximum passes it by FA_RESCALE_LOG2 (see the forward kernel)
          const float m_cand = fmaxf(m, mx * sl2);
          const float m_new = (m_cand > m + FA_RESCALE_LOG2) ? m_cand : m;
          const float base = (m_new == -INFINITY) ? 0.f : m_new;
          const float alpha = (m_new == m) ? 1.f : ex2(m - base);
          const float2 sl2v = make_float2(sl2, sl2), nbase = make_float2(-base, -base);
          float2 rs2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < C::BN / 32; ++c) {
            uint32_t hi[16], lo[16];  // P = hi + lo, as in the pieces
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = __ffma2_rn(make_float2(f[c * 32 + 2 * i], f[c * 32 + 2 * i + 1]), sl2v, nbase);
              const float2 pv = make_float2(ex2(y.x), ex2(y.y));
              rs2[i & 3] = __fadd2_rn(rs2[i & 3], pv);
              hi[i] = pack_bf16x2(pv.x, pv.y);
              const float2 rest = __ffma2_rn(make_float2(__uint_as_float(hi[i] << 16), __uint_as_float(hi[i] & 0xffff0000u)),
                                             make_float2(-1.f, -1.f), pv);
              lo[i] = pack_bf16x2(rest.x, rest.y);
            }
            tmem_st16(tS + c * 16, hi);
            tmem_st16(tS + C::BN / 2 + c * 16, lo);
          }
          const float2 rsa = __fadd2_rn(__fadd2_rn(rs2[0], rs2[1]), __fadd2_rn(rs2[2], rs2[3]));
          l = l * alpha + (rsa.x + rsa.y);
          if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // u must hold the tile before this one, and no later one can have been added yet
            ok = warp_wait(&bars->v_empty[(g - 1) % C::NSTAGE], ((g - 1) / C::NSTAGE) & 1, p.wait_ns, abort_flag, 332 + t);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + c * 32, o);
            }
          }
          tmem_wait_st();
          m = m_new;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t][g & 1]);
      }
      // P V of the item's last step
      if (ok)
        ok = warp_wait(&bars->v_empty[(g - 1) % C::NSTAGE], ((g - 1) / C::NSTAGE) & 1, p.wait_ns, abort_flag, 340 + t);
      if (!ok) break;
      if (idle) continue;
      tc_fence_after();
      // u / l: 16 columns at a time through the warp's staging (16-byte pieces swizzled by the row),
      // so that four lanes write 64 consecutive bytes of a row
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (scores of -inf alone: lse = -inf, no share in the row)
      const int part = int(blockIdx.x) - deal.owner((long long)(it)*deal.nt);
      const size_t row0 = ((size_t(it) * p.parts + part) * 2 + t) * C::BM + wq * 32;
      uint8_t* stg = smem + C::OFF_STG + (warp - 2) * C::STG_WARP;
#pragma unroll 2
      for (int c = 0; c < D / 16; ++c) {
        uint32_t o[16];
        tmem_ld16(tO + c * 16, o);
        tmem_wait_ld();
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<float4*>(stg + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
              make_float4(__uint_as_float(o[4 * u]) * inv, __uint_as_float(o[4 * u + 1]) * inv,
                          __uint_as_float(o[4 * u + 2]) * inv, __uint_as_float(o[4 * u + 3]) * inv);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = k * 8 + (lane >> 2), u = lane & 3;
          *reinterpret_cast<float4*>(p.part_o + (row0 + rr) * D + c * 16 + u * 4) =
              *reinterpret_cast<const float4*>(stg + rr * 64 + ((u ^ ((rr >> 1) & 3)) << 4));
        }
      }
      p.part_lse[row0 + lane] = m + __log2f(l);
    }
    if (!ok) {  // NaN for the item in progress and those behind it, so that nothing merged from them looks valid
      int i = 0;
      for (long long x = x0; x < x1; ++i) {
        const int it = int(x / deal.nt);
        x = min(x1, (long long)(it + 1) * deal.nt);
        const int part = int(blockIdx.x) - deal.owner((long long)(it)*deal.nt);
        if (i >= local) p.part_lse[((size_t(it) * p.parts + part) * 2 + t) * C::BM + wq * 32 + lane] = NAN;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace fa
