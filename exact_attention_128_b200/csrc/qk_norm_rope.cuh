// qk_norm_rope.cuh — per-head RMS norm of q and k with the position rotation in one pass:
// forward (dense), the serving form that writes K and V into a paged cache, and backward.
//
// A head's row x [d] with weight w [d]:  r = (mean_c x_c^2 + eps)^(-1/2),  y = x r w  (y = x
// without weights), then each pair (a, b) of y is turned by its angle t = position * frequency:
//   a' = a cos t - b sin t,  b' = a sin t + b cos t.
// Backward, with R^T the turn by -t and n = x r:  g = R^T dy,  dw = sum over rows of g n,
// h = g w,  dx = r (h - n mean_c(h n)).
//
// What bounds it: device memory.  Each value is read once and written once (backward: dy and x
// read, dx written) for about 10 operations.  A row of d values is held by d/16 lanes, two
// 16-byte pieces each, chosen so that both members of every pair sit in one lane: no value moves
// between lanes but the row's sum of squares.  A CTA works on `tok` tokens and computes their
// cosines and sines once, for all heads, into shared memory.
//
// Angles: the position (up to 2^31) times the frequency is taken in turns in 64 bits and reduced
// to [-1/2, 1/2] before it is rounded to 32 bits, so far positions lose nothing; no table of
// cosines is read.  All arithmetic behind that is fp32 with one rounding at the end.
#pragma once
#include "common.cuh"

namespace fa {
namespace rope {
constexpr int THREADS = 256;
constexpr int MAX_TOK = 8;

// Lanes of one row: d / 16 rounded up to a power of two (d = 96: 6 of 8 lanes work).
template <int D>
struct Cfg {
  static constexpr int PAIRS = D / 16;  // lanes that hold values
  static constexpr int L = D == 96 ? 8 : D / 16;
  static constexpr int GROUPS = THREADS / L;  // rows a CTA holds at a time
};
}  // namespace rope

struct RopeParams {
  const void* x[3];       // q, k, v (v: paged only)
  int64_t sb[3], sh[3], sn[3];  // their strides, in elements
  const void* w[2];       // weights of q and k, or null
  const int* pos;         // [axes] x pos_sa, [B] x pos_sb, [N]
  const double* freq;     // [rd / 2], radians per position
  void* out[2];           // q', k' [B, H, N, d] (paged: q' only)
  int64_t pos_sa, pos_sb;
  int B, Hq, Hkv, N;
  int rd, sec0, sec1;     // rotary dims; frequencies below sec0 follow axis 0, below sec1 axis 1, then axis 2
  float eps;
  int tok;                // tokens per CTA
  // paged: cache rows of the tokens
  const int *bt, *ctx, *qlen;
  void *kc, *vc;
  int max_blocks, num_blocks;
};

struct RopeBwdParams {
  const void* dy[2];  // dq', dk' [B, H, N, d]
  const void* x[2];
  int64_t sb[2], sh[2], sn[2];
  const void* w[2];
  const int* pos;
  const double* freq;
  void* dx[2];
  int64_t dsb[2], dsh[2], dsn[2];
  float* part;  // [CTAs of q + CTAs of k][d] partial weight gradients
  int64_t pos_sa, pos_sb;
  int B, H[2], N;
  int rd, sec0, sec1;
  float eps;
  int tok;
  int ctas_q;  // CTAs [0, ctas_q) take the rows of q, the others those of k
};

namespace rope {

// Eight values as they are stored, and as fp32.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(a[i] << 16);
      f[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 u, v;
  __device__ __forceinline__ void load(const float* p) {
    u = __ldg(reinterpret_cast<const float4*>(p));
    v = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { u = v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
    f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *(reinterpret_cast<float4*>(p) + 1) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// The two 8-value pieces of lane c: piece c and its partner a half rotary width behind it; the
// pieces behind the rotary width are dealt out in the same way, to the lanes behind it.
template <int D>
__device__ __forceinline__ void pieces(int c, int rd, int& lo, int& hi) {
  const int p2 = rd / 16;
  lo = c < p2 ? c : p2 + c;
  hi = c < p2 ? c + p2 : D / 16 + c;
}

// A per-lane table of 8 values per lane is kept as two planes of [lane][4], so that a 16-byte
// read of neighbouring lanes touches neighbouring banks.
template <int D>
__device__ __forceinline__ int slot(int c, int e) {
  return ((e >> 2) * Cfg<D>::PAIRS + c) * 4 + (e & 3);
}
template <int D>
__device__ __forceinline__ void read8(const float* t, int c, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(t + c * 4);
  const float4 b = *reinterpret_cast<const float4*>(t + (Cfg<D>::PAIRS + c) * 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Cosine and sine of table entry i (lane i / 8, pair i % 8) of one token.  `pos` points at the
// token's position on axis 0.  Lanes behind the rotary width get (1, 0).
template <int D, bool INTER>
__device__ __forceinline__ void angle(int i, const int* pos, int64_t pos_sa, const double* freq, int rd, int sec0,
                                      int sec1, float& c, float& s) {
  const int lane = i >> 3, e = i & 7, p2 = rd / 16;
  c = 1.f;
  s = 0.f;
  if (lane >= p2) return;
  const int f = INTER ? (e < 4 ? 4 * lane + e : 4 * (lane + p2) + e - 4) : i;
  const int axis = f < sec0 ? 0 : f < sec1 ? 1 : 2;
  const double turns = double(__ldg(pos + axis * pos_sa)) * (__ldg(freq + f) * 0.15915494309189533577);
  sincospif(2.f * float(turns - rint(turns)), &s, &c);
}

template <bool INTER>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
  if constexpr (INTER) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x0 = a[2 * e], x1 = a[2 * e + 1], y0 = b[2 * e], y1 = b[2 * e + 1];
      a[2 * e] = x0 * c[e] - x1 * s[e];
      a[2 * e + 1] = x0 * s[e] + x1 * c[e];
      b[2 * e] = y0 * c[4 + e] - y1 * s[4 + e];
      b[2 * e + 1] = y0 * s[4 + e] + y1 * c[4 + e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = a[e], y = b[e];
      a[e] = x * c[e] - y * s[e];
      b[e] = x * s[e] + y * c[e];
    }
  }
}

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Weight tables of lane order: piece lo at [0], piece hi at [1].
template <typename T, int D>
__device__ __forceinline__ void fill_weights(float (*t)[D / 2], const void* w, int rd) {
  for (int i = threadIdx.x; i < D; i += THREADS) {
    const int half = i / (D / 2), j = i % (D / 2), c = j >> 3, e = j & 7;
    int lo, hi;
    pieces<D>(c, rd, lo, hi);
    t[half][slot<D>(c, e)] = to_f32(static_cast<const T*>(w)[(half ? hi : lo) * 8 + e]);
  }
}

}  // namespace rope

// One CTA: `tok` consecutive tokens (of the B x N), all their heads.  Rows run head-fastest, so
// the rows of a warp share a token's cosines and the reads of a fused projection are contiguous.
// PAGED (bf16): token (r, i) of request r is one of its last q_lens[r] positions; q' goes to
// [R, Hq, N, d], k' and v to cache position ctx_lens[r] - q_lens[r] + i; padding rows are left.
template <typename T, int D, bool INTER, bool PAGED>
__global__ void __launch_bounds__(rope::THREADS) fa_qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  using namespace rope;
  using C = Cfg<D>;
  __shared__ float s_cos[MAX_TOK][D / 2], s_sin[MAX_TOK][D / 2];
  __shared__ float s_w[2][2][D / 2];
  __shared__ int64_t s_row[MAX_TOK];  // paged: cache row (block * Hkv * 16 + slot) of the token, -1: not cached
  __shared__ int s_live[MAX_TOK];
  const int64_t tokens = int64_t(p.B) * p.N;
  const int64_t t0 = int64_t(blockIdx.x) * p.tok;
  const int nt = int(min(int64_t(p.tok), tokens - t0));
  const bool norm = p.w[0] != nullptr;
  const int heads = p.Hq + p.Hkv + (PAGED ? p.Hkv : 0);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  if constexpr (PAGED) {
    int live = 0;
    if (threadIdx.x < nt) {
      const int64_t t = t0 + threadIdx.x;
      const int r = int(t / p.N), i = int(t % p.N);
      const int L = p.ctx[r], ql = p.qlen[r];
      int64_t row = -1;
      if (ql < 0 || ql > p.N || L < ql || L > p.max_blocks * 16) {
        if (i == 0) set_status(FA_ERR_INVALID_ARG, 200);
      } else if (i < ql) {
        live = 1;
        const int at = L - ql + i;
        const int phys = p.bt[int64_t(r) * p.max_blocks + at / 16];
        if (phys < 0 || phys >= p.num_blocks)
          set_status(FA_ERR_INVALID_ARG, 201);
        else
          row = int64_t(phys) * p.Hkv * 16 + at % 16;
      }
      s_row[threadIdx.x] = row;
      s_live[threadIdx.x] = live;
    }
    if (!__syncthreads_or(live)) return;
  }
  for (int i = threadIdx.x; i < nt * (D / 2); i += THREADS) {
    const int tt = i / (D / 2), j = i % (D / 2);
    const int64_t t = t0 + tt;
    float c, s;
    angle<D, INTER>(j, p.pos + (t / p.N) * p.pos_sb + t % p.N, p.pos_sa, p.freq, p.rd, p.sec0, p.sec1, c, s);
    s_cos[tt][slot<D>(j >> 3, j & 7)] = c;
    s_sin[tt][slot<D>(j >> 3, j & 7)] = s;
  }
  if (norm) {
    fill_weights<T, D>(s_w[0], p.w[0], p.rd);
    fill_weights<T, D>(s_w[1], p.w[1], p.rd);
  }
  __syncthreads();

  const int c = threadIdx.x % C::L;
  const bool lane_on = c < C::PAIRS;
  int lo, hi;
  pieces<D>(c, p.rd, lo, hi);
  const int rows = nt * heads;
  const int first = threadIdx.x / C::L;
  const int warp_first = (threadIdx.x & ~31) / C::L;
  for (int base = 0; base + warp_first < rows; base += C::GROUPS) {
    const int row = base + first;
    const int tt = row / heads, h = row - tt * heads;
    bool on = lane_on && row < rows;
    if constexpr (PAGED) on = on && s_live[tt];
    const int64_t t = t0 + tt, b = t / p.N, n = t % p.N;
    const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
    Raw<T> ra, rb;
    ra.clear();
    rb.clear();
    if (on) {
      const T* src = static_cast<const T*>(p.x[kind]) + b * p.sb[kind] + hh * p.sh[kind] + n * p.sn[kind];
      ra.load(src + lo * 8);
      rb.load(src + hi * 8);
    }
    float a[8], bb[8];
    ra.get(a);
    rb.get(bb);
    if (norm) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq += a[e] * a[e] + bb[e] * bb[e];
      sq = row_sum<C::L>(sq);
      if (on && kind < 2) {
        const float r = rsqrtf(sq * (1.f / D) + p.eps);
        float wa[8], wb[8];
        read8<D>(s_w[kind][0], c, wa);
        read8<D>(s_w[kind][1], c, wb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] *= r * wa[e];
          bb[e] *= r * wb[e];
        }
      }
    }
    if (!on) continue;
    if (kind < 2) {
      float cs[8], sn[8];
      read8<D>(s_cos[tt], c, cs);
      read8<D>(s_sin[tt], c, sn);
      turn<INTER>(a, bb, cs, sn);
    }
    T* dst;
    if (kind == 0) {
      dst = static_cast<T*>(p.out[0]) + ((b * p.Hq + hh) * p.N + n) * D;
    } else if constexpr (PAGED) {
      if (s_row[tt] < 0) continue;
      dst = static_cast<T*>(kind == 1 ? p.kc : p.vc) + (s_row[tt] + int64_t(hh) * 16) * D;
    } else {
      dst = static_cast<T*>(p.out[1]) + ((b * p.Hkv + hh) * p.N + n) * D;
    }
    store8(dst + lo * 8, a);
    store8(dst + hi * 8, bb);
  }
}

// Backward.  CTAs [0, ctas_q) walk the tokens' q rows, the others the k rows, so that a thread
// keeps the 16 weight-gradient sums of its two pieces in registers over all its rows; the CTA's
// sums go to `part`, which the second kernel adds up in a fixed order (no atomics: the same call
// gives the same bits).
template <typename T, typename TG, typename TO, int D, bool INTER>
__global__ void __launch_bounds__(rope::THREADS) fa_qk_norm_rope_bwd_kernel(const __grid_constant__ RopeBwdParams p) {
  using namespace rope;
  using C = Cfg<D>;
  __shared__ float s_cos[MAX_TOK][D / 2], s_sin[MAX_TOK][D / 2];
  __shared__ float s_w[2][D / 2];
  __shared__ float s_sum[THREADS / 32][D];
  const int kind = int(blockIdx.x) < p.ctas_q ? 0 : 1;
  const int64_t first_tile = kind ? blockIdx.x - p.ctas_q : blockIdx.x;
  const int64_t n_cta = kind ? gridDim.x - p.ctas_q : p.ctas_q;
  const int64_t tokens = int64_t(p.B) * p.N;
  const bool norm = p.w[0] != nullptr;
  const int heads = p.H[kind];
  const T* x = static_cast<const T*>(p.x[kind]);
  const TG* dy = static_cast<const TG*>(p.dy[kind]);
  TO* dx = static_cast<TO*>(p.dx[kind]);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (norm) fill_weights<T, D>(s_w, p.w[kind], p.rd);
  const int c = threadIdx.x % C::L;
  const bool lane_on = c < C::PAIRS;
  int lo, hi;
  pieces<D>(c, p.rd, lo, hi);
  const int first = threadIdx.x / C::L;
  const int warp_first = (threadIdx.x & ~31) / C::L;
  float sa[8], sb[8];  // weight-gradient sums of the two pieces
#pragma unroll
  for (int e = 0; e < 8; ++e) sa[e] = sb[e] = 0.f;

  for (int64_t t0 = first_tile * p.tok; t0 < tokens; t0 += n_cta * p.tok) {
    const int nt = int(min(int64_t(p.tok), tokens - t0));
    __syncthreads();  // the last tile's readers are done with the tables
    for (int i = threadIdx.x; i < nt * (D / 2); i += THREADS) {
      const int tt = i / (D / 2), j = i % (D / 2);
      const int64_t t = t0 + tt;
      float cc, ss;
      angle<D, INTER>(j, p.pos + (t / p.N) * p.pos_sb + t % p.N, p.pos_sa, p.freq, p.rd, p.sec0, p.sec1, cc, ss);
      s_cos[tt][slot<D>(j >> 3, j & 7)] = cc;
      s_sin[tt][slot<D>(j >> 3, j & 7)] = -ss;
    }
    __syncthreads();
    const int rows = nt * heads;
    for (int base = 0; base + warp_first < rows; base += C::GROUPS) {
      const int row = base + first;
      const int tt = row / heads, h = row - tt * heads;
      const bool on = lane_on && row < rows;
      const int64_t t = t0 + tt, b = t / p.N, n = t % p.N;
      Raw<T> rxa, rxb;
      Raw<TG> rga, rgb;
      rxa.clear();
      rxb.clear();
      rga.clear();
      rgb.clear();
      if (on) {
        const TG* g = dy + ((b * heads + h) * p.N + n) * D;
        rga.load(g + lo * 8);
        rgb.load(g + hi * 8);
        if (norm) {
          const T* xs = x + b * p.sb[kind] + h * p.sh[kind] + n * p.sn[kind];
          rxa.load(xs + lo * 8);
          rxb.load(xs + hi * 8);
        }
      }
      float ga[8], gb[8], cs[8], sn[8];
      rga.get(ga);
      rgb.get(gb);
      if (on) {
        read8<D>(s_cos[tt], c, cs);
        read8<D>(s_sin[tt], c, sn);
        turn<INTER>(ga, gb, cs, sn);
      }
      if (norm) {
        float xa[8], xb[8];
        rxa.get(xa);
        rxb.get(xb);
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += xa[e] * xa[e] + xb[e] * xb[e];
        sq = row_sum<C::L>(sq);
        const float r = rsqrtf(sq * (1.f / D) + p.eps);
        float wa[8], wb[8];
        if (lane_on) {
          read8<D>(s_w[0], c, wa);
          read8<D>(s_w[1], c, wb);
        }
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xa[e] *= r;  // n
          xb[e] *= r;
          if (on) {
            sa[e] += ga[e] * xa[e];
            sb[e] += gb[e] * xb[e];
            ga[e] *= wa[e];  // h
            gb[e] *= wb[e];
            dot += ga[e] * xa[e] + gb[e] * xb[e];
          }
        }
        dot = row_sum<C::L>(dot) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ga[e] = r * (ga[e] - xa[e] * dot);
          gb[e] = r * (gb[e] - xb[e] * dot);
        }
      }
      if (on) {
        TO* dst = dx + b * p.dsb[kind] + h * p.dsh[kind] + n * p.dsn[kind];
        store8(dst + lo * 8, ga);
        store8(dst + hi * 8, gb);
      }
    }
  }
  if (!norm) return;
  // rows of a warp, then the warps
#pragma unroll
  for (int m = C::L; m < 32; m <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sa[e] += __shfl_xor_sync(0xffffffffu, sa[e], m);
      sb[e] += __shfl_xor_sync(0xffffffffu, sb[e], m);
    }
  if (lane_id() < C::L && lane_on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s_sum[warp_id()][lo * 8 + e] = sa[e];
      s_sum[warp_id()][hi * 8 + e] = sb[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += THREADS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) v += s_sum[w][i];
    p.part[int64_t(blockIdx.x) * D + i] = v;
  }
}

// dw of q (block 0) and k (block 1): the CTAs' partial sums, eight strands per column.
__global__ void __launch_bounds__(256) fa_qk_norm_rope_dw_kernel(const float* part, float* dwq, float* dwk, int D,
                                                                 int ctas_q, int ctas) {
  __shared__ float s[256];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int r0 = blockIdx.x ? ctas_q : 0, r1 = blockIdx.x ? ctas : ctas_q;
  float* dw = blockIdx.x ? dwk : dwq;
  const int col = threadIdx.x & 31, strand = threadIdx.x >> 5;
  for (int c0 = 0; c0 < D; c0 += 32) {
    float v = 0.f;
    for (int r = r0 + strand; r < r1; r += 8) v += part[int64_t(r) * D + c0 + col];
    s[threadIdx.x] = v;
    __syncthreads();
    if (strand == 0) {
      for (int k = 1; k < 8; ++k) v += s[k * 32 + col];
      dw[c0 + col] = v;
    }
    __syncthreads();
  }
}

}  // namespace fa
