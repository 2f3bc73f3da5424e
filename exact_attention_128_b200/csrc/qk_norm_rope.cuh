// qk_norm_rope.cuh — per-head RMS norm of q and k with the position rotation in one pass:
// forward (dense), the serving form that writes K and V into a paged cache, and backward.
//
// A head's row x [d] with weight w [d]:  r = (mean_c x_c^2 + eps)^(-1/2),  y = x r w  (y = x
// without weights), then each pair (a, b) of y is turned by its angle t = position * frequency:
//   a' = a cos t - b sin t,  b' = a sin t + b cos t.
// Backward, with R^T the turn by -t and n = x r:  g = R^T dy,  dw = sum over rows of g n,
// h = g w,  dx = r (h - n mean_c(h n)).
//
// What bounds it: device memory.  Each value is read once and written once (backward: dy and x read,
// dx written) for about 10 operations.  A row of d values is held by d/16 lanes, four runs of 4
// values each, chosen so that both members of every pair sit in one lane: no value moves between
// lanes but the row's sum of squares.  Forward: a CTA takes the tokens of 1 to 8 warps (a warp holds
// 32 / lanes tokens of one head) with all their heads.  Each thread computes one cosine and sine per
// token group, while the first rows are on their way; all heads' rows share them, from shared
// memory, as they share the weights.  (With the angles of a lane's 8 pairs computed by each warp for
// itself and kept in registers, 116 registers left 16 warps on an SM, and the prefill of 4 x 8192
// tokens, 32 + 8 heads of 128, took 4 us longer into reused outputs, the fp32 image layer 33 us instead
// of 29.)  A warp writes 1 KB of consecutive tokens of one head.  Measured: that prefill reads and
// writes 671 MB in 110 us into reused outputs, 6.1 TB/s (without norm 105), and in 118 to 125 us in
// calls in a row into fresh ones; the backward of 8 x 4096 tokens, 16 + 16 heads of 64 with fp32
// gradients in, 537 MB in 95 us with the weights' sums (without norm 65); in fp32 throughout, 805 MB in
// 133 us, 6.0 TB/s.
//
// Angles: the position (up to 2^31) times the frequency is taken in turns in 64 bits and reduced
// to [-1/2, 1/2] before it is rounded to 32 bits, so far positions lose nothing (and where the results
// have 32 bits, the rounded part is not lost either); no table of cosines is read.  All arithmetic
// behind that is fp32 with one rounding at the end.
#pragma once
#include "common.cuh"

namespace fa {
namespace rope {
constexpr int THREADS = 256;
constexpr int MAX_CHUNK = 16;  // backward: heads of a unit, at most
// Rows a thread has in flight, + 1.  Forward: 3 CTAs on an SM; more stages or a fourth CTA at 64
// registers were slower (prefill of 4 x 8192: 110 us; 7 stages 115, 4 CTAs 130).  Backward: 2 CTAs
// of 128 registers; the forward's form, with angles and weights read from shared memory, took 99 us
// on the training step (2 CTAs; 3 CTAs 142 to 149), this one 93.
constexpr int FWD_STAGES = 5, FWD_STAGES_F32 = 4, FWD_CTAS = 3;
constexpr int BWD_STAGES = 4, BWD_CTAS = 2;

// Lanes of one row: d / 16.  (d = 96: 5 rows of 6 lanes, 2 lanes idle.  4 rows of 8 lanes with 6 at
// work took 113 us forward and 160 backward for 4 x 8192 tokens of 32 + 8 heads, this way 101 and 149.)
template <int D>
struct Cfg {
  static constexpr int L = D / 16;
  static constexpr int TOKENS = 32 / L;       // tokens of a warp
  static constexpr int WORK = L * TOKENS;     // its lanes that hold values
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
  int groups;             // token groups of a CTA: 1, 2, 4 or 8; 8 / groups warps share one
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
  int chunk[2], chunks[2];  // of q and of k: heads per unit, units of a token group
  int ctas_q;  // CTAs [0, ctas_q) take the rows of q, the others those of k
};

namespace rope {

// Packed fp32 pairs: one instruction for two values.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

__device__ __forceinline__ float2 unpack(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Where a lane's four runs of 4 values lie in a row (in runs): two in the first half of the
// rotary width and their partners in the second; the runs behind the rotary width are dealt out
// to the lanes behind it in the same way.  SPREAD: neighbouring lanes hold neighbouring runs, so
// that an fp32 access of 16 bytes a lane fills its 32-byte sectors (with the bf16 layout, which
// keeps two runs side by side for 16-byte accesses, fp32 asked L2 for each sector twice).
template <int D, bool SPREAD>
struct Runs {
  int q[4];
  __device__ __forceinline__ Runs(int c, int rd) {
    const int p2 = rd / 16, m = D / 16 - p2;
    const int base = c < p2 ? 0 : 4 * p2, w = c < p2 ? p2 : m, j = c < p2 ? c : c - p2;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = base + (SPREAD ? i * w + j : (i >> 1) * 2 * w + 2 * j + (i & 1));
  }
};
// A thread's 16 values of a row on their way from device memory: pieces in shared memory that
// only this thread writes (cp.async) and reads, [piece][thread], so that rows in flight cost no
// registers and no barrier.  Values are kept as 8 pairs, pairs 2i and 2i + 1 of run i.
template <typename T, bool SPREAD>
struct Slot {
  static constexpr int N = SPREAD ? 4 : 2;                 // pieces
  static constexpr int PIECE = 16 * int(sizeof(T)) / N;    // their bytes: 8 or 16
  static constexpr int BYTES = N * PIECE * THREADS;        // of one row of every thread
  static_assert(SPREAD || sizeof(T) == 2, "fp32 rows are spread");
  // a row's values, or zeros
  template <int D>
  static __device__ __forceinline__ void fetch(uint32_t at, const T* row, const Runs<D, SPREAD>& r, bool on) {
    const int bytes = on ? PIECE : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const T* src = row + r.q[SPREAD ? i : 2 * i] * 4;
      if constexpr (PIECE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + i * THREADS * PIECE), "l"(src),
                     "r"(bytes)
                     : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at + i * THREADS * PIECE), "l"(src),
                     "r"(bytes)
                     : "memory");
    }
  }
  static __device__ __forceinline__ void read(uint32_t at, float2 (&f)[8]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint4 v;
      if constexpr (PIECE == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(at + i * THREADS * PIECE));
      else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at + i * THREADS * PIECE));
      if constexpr (sizeof(T) == 4) {
        f[2 * i] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[2 * i + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
      } else if constexpr (SPREAD) {
        f[2 * i] = unpack(v.x);
        f[2 * i + 1] = unpack(v.y);
      } else {
        f[4 * i] = unpack(v.x);
        f[4 * i + 1] = unpack(v.y);
        f[4 * i + 2] = unpack(v.z);
        f[4 * i + 3] = unpack(v.w);
      }
    }
  }
};
template <int D, bool SPREAD>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, const Runs<D, SPREAD>& r, const float2 (&f)[8]) {
  if constexpr (SPREAD) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(row + r.q[i] * 4) =
          make_uint2(pack_bf16x2(f[2 * i].x, f[2 * i].y), pack_bf16x2(f[2 * i + 1].x, f[2 * i + 1].y));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(row + r.q[2 * i] * 4) =
          make_uint4(pack_bf16x2(f[4 * i].x, f[4 * i].y), pack_bf16x2(f[4 * i + 1].x, f[4 * i + 1].y),
                     pack_bf16x2(f[4 * i + 2].x, f[4 * i + 2].y), pack_bf16x2(f[4 * i + 3].x, f[4 * i + 3].y));
  }
}
template <int D>
__device__ __forceinline__ void store_row(float* row, const Runs<D, true>& r, const float2 (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(row + r.q[i] * 4) = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
}
// A lane's 16 weights.
template <typename T, int D, bool SPREAD>
__device__ __forceinline__ void load_weights(const void* w, const Runs<D, SPREAD>& r, float2 (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const T* at = static_cast<const T*>(w) + r.q[i >> 1] * 4 + 2 * (i & 1);
    f[i] = make_float2(float(at[0]), float(at[1]));
  }
}
__device__ __forceinline__ void rows_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void rows_wait() {  // all but this thread's newest N rows are here
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Cosine and sine of a position times a frequency.  FINE (results of 32 bits): what the reduced angle
// loses when it is rounded, up to 2^-26 turns, is added back (the first term of the series); for a result
// of 16 bits it does not matter.
template <bool FINE>
__device__ __forceinline__ void turn_of(int pos, double freq, float& s, float& c) {
  const double turns = double(pos) * (freq * 0.15915494309189533577), part = turns - rint(turns);
  const float near = float(part);
  sincospif(2.f * near, &s, &c);
  if constexpr (FINE) {
    const float rest = float(part - double(near)) * 6.2831853f, s0 = s;
    s = fmaf(c, rest, s);
    c = fmaf(-s0, rest, c);
  }
}
// 1 / sqrt(v), for results of 32 bits rounded to the nearest (rsqrtf is off by up to two steps).
template <bool FINE>
__device__ __forceinline__ float inverse_root(float v) {
  return FINE ? __frsqrt_rn(v) : rsqrtf(v);
}

// Cosines and sines of a lane's 8 pairs for one token (lanes behind the rotary width: 1 and 0).
// `pos` points at the token's position on axis 0.
template <bool INTER, bool FINE, int D, bool SPREAD>
__device__ __forceinline__ void angles(const Runs<D, SPREAD>& r, const int* pos, int64_t pos_sa, const double* freq,
                                       int rd, int sec0, int sec1, float2 (&cs)[4], float2 (&sn)[4]) {
  const bool turns_at_all = r.q[0] * 4 < rd;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float s = 0.f, c = 1.f;
    if (turns_at_all) {
      // pair e: adjacent values of run e / 2, or value e % 4 of run e / 4 with its partner
      const int f = INTER ? r.q[e >> 1] * 2 + (e & 1) : r.q[e >> 2] * 4 + (e & 3);
      const int axis = f < sec0 ? 0 : f < sec1 ? 1 : 2;
      turn_of<FINE>(__ldg(pos + axis * pos_sa), __ldg(freq + f), s, c);
    }
    (e & 1 ? sn[e >> 1].y : sn[e >> 1].x) = s;
    (e & 1 ? cs[e >> 1].y : cs[e >> 1].x) = c;
  }
}

// Cosines and sines of the 8 pairs of every lane, for one token group, in shared memory: one
// float4 a lane in four planes (a 16-byte read of neighbouring lanes touches neighbouring banks),
// cosines of pairs 0-3 and 4-7, then sines.  Pairs behind the rotary width get 1 and 0.  `pos`
// points at the token's position on axis 0.
constexpr int TABLE = 4 * 32;  // float4 of a token group
template <bool INTER, int D, bool SPREAD>
__device__ __forceinline__ void table_entry(float4* table, int lane, int e, const Runs<D, SPREAD>& r, const int* pos,
                                            int64_t pos_sa, const double* freq, int rd, int sec0, int sec1, bool on) {
  float s = 0.f, c = 1.f;
  if (on && r.q[0] * 4 < rd) {
    const int f = INTER ? r.q[e >> 1] * 2 + (e & 1) : r.q[e >> 2] * 4 + (e & 3);
    const int axis = f < sec0 ? 0 : f < sec1 ? 1 : 2;
    turn_of<SPREAD>(__ldg(pos + axis * pos_sa), __ldg(freq + f), s, c);  // (forward: spread rows are fp32 ones)
  }
  float* at = reinterpret_cast<float*>(table + (e >> 2) * 32 + lane) + (e & 3);
  at[0] = c;
  at[2 * 32 * 4] = s;
}
// One kind's weights in the same form: [4][L].
template <typename T, int D, bool SPREAD>
__device__ __forceinline__ void fill_weights(float4* table, const void* w, int rd) {
  using C = Cfg<D>;
  for (int i = threadIdx.x; i < C::L * 16; i += THREADS) {  // value v of lane l
    const int l = i / 16, v = i % 16;
    const Runs<D, SPREAD> r(l, rd);
    reinterpret_cast<float*>(table + (v >> 2) * C::L + l)[v & 3] =
        float(static_cast<const T*>(w)[r.q[v >> 2] * 4 + (v & 3)]);
  }
}
// 8 pairs (16 values), or 4, from planes of float4.
template <int N>
__device__ __forceinline__ void read_planes(const float4* t, int stride, float2 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float4 v = t[i * stride];
    f[2 * i] = make_float2(v.x, v.y);
    f[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// Turn a lane's pairs: half-width pairs (runs 0, 1 with runs 2, 3) in packed form, adjacent ones
// one by one.
template <bool INTER>
__device__ __forceinline__ void turn(float2 (&f)[8], const float2 (&c)[4], const float2 (&s)[4]) {
  if constexpr (INTER) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float cc = e & 1 ? c[e >> 1].y : c[e >> 1].x, ss = e & 1 ? s[e >> 1].y : s[e >> 1].x;
      // (x, y) -> x (c, s) + y (-s, c)
      f[e] = fma2(both(f[e].x), make_float2(cc, ss), mul2(both(f[e].y), make_float2(-ss, cc)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = f[i], y = f[4 + i];
      f[i] = fma2(x, c[i], neg2(mul2(y, s[i])));
      f[4 + i] = fma2(x, s[i], mul2(y, c[i]));
    }
  }
}

// Sum over the lanes of a row, the same bits in each of them.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (L == 6) {
    const int lane = lane_id(), c = lane % 6, first = lane - c;
    v += __shfl_sync(0xffffffffu, v, first + (c < 3 ? c + 3 : c - 3));
    return __shfl_sync(0xffffffffu, v, first) + __shfl_sync(0xffffffffu, v, first + 1) +
           __shfl_sync(0xffffffffu, v, first + 2);
  } else {
#pragma unroll
    for (int m = 1; m < L; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
  }
}
// Sum over the rows of a warp, for each lane of the first row.
template <int L>
__device__ __forceinline__ float rows_sum(float v) {
  if constexpr (L == 6) {
    float sum = v;
#pragma unroll
    for (int k = 1; k < 5; ++k) sum += __shfl_down_sync(0xffffffffu, v, 6 * k);
    return sum;
  } else {
#pragma unroll
    for (int m = L; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
  }
}

}  // namespace rope

// PAGED (bf16): token (r, i) of request r is one of its last q_lens[r] positions; q' goes to
// [R, Hq, N, d], k' and v to cache position ctx_lens[r] - q_lens[r] + i; padding rows are left.
template <typename T, int D, bool INTER, bool PAGED>
__global__ void __launch_bounds__(rope::THREADS, rope::FWD_CTAS)
    fa_qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  using namespace rope;
  using C = Cfg<D>;
  constexpr bool SPREAD = sizeof(T) == 4, FINE = SPREAD;
  constexpr int STAGES = SPREAD ? FWD_STAGES_F32 : FWD_STAGES;
  using R = Slot<T, SPREAD>;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  float4* s_table = reinterpret_cast<float4*>(rope_smem + STAGES * R::BYTES);  // [groups][TABLE]
  float4* s_w = s_table + p.groups * TABLE;                                    // [q, k][4][L]
  const int tokens = p.B * p.N;
  const int lane = lane_id(), c = lane % C::L, warp = warp_id();
  const int sharers = 8 / p.groups, sub = warp / sharers;  // warps of a token group; this warp's group
  const int t = (int(blockIdx.x) * p.groups + sub) * C::TOKENS + lane / C::L;
  const int heads = p.Hq + p.Hkv + (PAGED ? p.Hkv : 0);
  bool on = lane < C::WORK && t < tokens;
  const int b = on ? t / p.N : 0, n = on ? t - b * p.N : 0;
  const Runs<D, SPREAD> runs(c, p.rd);
  const bool norm = p.w[0] != nullptr;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int phys = 0, at = 0;  // paged: cache block and position of the token
  if constexpr (PAGED) {
    if (on) {
      const int L = p.ctx[b], ql = p.qlen[b];
      if (ql < 0 || ql > p.N || L < ql || L > p.max_blocks * 16) {
        if (n == 0) set_status(FA_ERR_INVALID_ARG, 200);
        on = false;
      } else if (n >= ql) {
        on = false;
      } else {
        at = L - ql + n;
        phys = p.bt[int64_t(b) * p.max_blocks + at / 16];
      }
    }
  }
  const uint32_t slot = smem_u32(rope_smem) + threadIdx.x * R::PIECE;
  const int h0 = warp - sub * sharers;
  int64_t off[PAGED ? 3 : 2];
#pragma unroll
  for (int k = 0; k < (PAGED ? 3 : 2); ++k) off[k] = b * p.sb[k] + n * p.sn[k];
  // row i of this warp: head h0 + i * sharers of q, then k, then v
  auto fetch = [&](int i) {
    const int h = h0 + i * sharers;
    if (h < heads) {
      const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
      const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
      const T* src = static_cast<const T*>(p.x[kind]) + (kind == 0 ? off[0] : kind == 1 ? off[1] : off[PAGED ? 2 : 1]);
      R::template fetch<D>(slot + (i % STAGES) * R::BYTES, src + hh * p.sh[kind], runs, on);
    }
    rows_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  // meanwhile the tables: thread (pair warp, lane) of every token group
  for (int g = 0; g < p.groups; ++g) {
    const int tt = (int(blockIdx.x) * p.groups + g) * C::TOKENS + lane / C::L;
    const int bb = tt < tokens ? tt / p.N : 0, nn = tt < tokens ? tt - bb * p.N : 0;
    table_entry<INTER>(s_table + g * TABLE, lane, warp, runs, p.pos + bb * p.pos_sb + nn, p.pos_sa, p.freq, p.rd,
                       p.sec0, p.sec1, lane < C::WORK && tt < tokens);
  }
  if (norm) {
    fill_weights<T, D, SPREAD>(s_w, p.w[0], p.rd);
    fill_weights<T, D, SPREAD>(s_w + 4 * C::L, p.w[1], p.rd);
  }
  int64_t row = -1;  // cache row (block * Hkv * 16 + slot) of the token, -1: not cached
  if constexpr (PAGED) {
    if (on && (phys < 0 || phys >= p.num_blocks))
      set_status(FA_ERR_INVALID_ARG, 201);
    else
      row = int64_t(phys) * p.Hkv * 16 + at % 16;
    if (!__syncthreads_or(on)) {
      rows_wait<0>();
      return;
    }
  } else {
    __syncthreads();
  }
  const float4* table = s_table + sub * TABLE + lane;
  for (int i = 0; h0 + i * sharers < heads; ++i) {
    rows_wait<STAGES - 2>();
    float2 f[8];
    R::read(slot + (i % STAGES) * R::BYTES, f);
    fetch(i + STAGES - 1);  // into the slot of row i - 1
    const int h = h0 + i * sharers;
    const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
    if (kind < 2) {
      if (norm) {
        float2 sq = mul2(f[0], f[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) sq = fma2(f[e], f[e], sq);
        const float2 r = both(inverse_root<FINE>(row_sum<C::L>(sq.x + sq.y) * (1.f / D) + p.eps));
        float2 w[8];
        read_planes(s_w + kind * 4 * C::L + c, C::L, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = mul2(f[e], mul2(r, w[e]));
      }
      float2 cs[4], sn[4];
      read_planes(table, 32, cs);
      read_planes(table + 2 * 32, 32, sn);
      turn<INTER>(f, cs, sn);
    }
    if (on) {
      if (kind == 0) {
        store_row(static_cast<T*>(p.out[0]) + ((int64_t(b) * p.Hq + hh) * p.N + n) * D, runs, f);
      } else if constexpr (PAGED) {
        if (row >= 0) store_row(static_cast<T*>(kind == 1 ? p.kc : p.vc) + (row + hh * 16) * D, runs, f);
      } else {
        store_row(static_cast<T*>(p.out[1]) + ((int64_t(b) * p.Hkv + hh) * p.N + n) * D, runs, f);
      }
    }
  }
}

// Backward.  CTAs [0, ctas_q) walk the units of q, the others those of k, so that a thread keeps
// the 16 weight-gradient sums of its two pieces in registers over all its rows; the CTA's sums go
// to `part`, which the second kernel adds up in a fixed order (no atomics: the same call gives
// the same bits).
template <typename T, typename TG, typename TO, int D, bool INTER>
__global__ void __launch_bounds__(rope::THREADS, rope::BWD_CTAS)
    fa_qk_norm_rope_bwd_kernel(const __grid_constant__ RopeBwdParams p) {
  using namespace rope;
  using C = Cfg<D>;
  constexpr bool SPREAD = sizeof(T) + sizeof(TG) + sizeof(TO) > 6;  // any of them fp32
  constexpr bool FINE = sizeof(TO) == 4;
  using RX = Slot<T, SPREAD>;
  using RG = Slot<TG, SPREAD>;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  const uint32_t slot_x = smem_u32(rope_smem) + RG::BYTES + threadIdx.x * RX::PIECE;
  const uint32_t slot_g = smem_u32(rope_smem) + threadIdx.x * RG::PIECE;
  const int kind = int(blockIdx.x) < p.ctas_q ? 0 : 1;
  const int cta = kind ? blockIdx.x - p.ctas_q : blockIdx.x, n_cta = kind ? gridDim.x - p.ctas_q : p.ctas_q;
  const int tokens = p.B * p.N;
  const bool norm = p.w[0] != nullptr;
  const int H = p.H[kind], chunks = p.chunks[kind];
  const int64_t units = int64_t((tokens + C::TOKENS - 1) / C::TOKENS) * chunks;
  const int lane = lane_id(), c = lane % C::L;
  const Runs<D, SPREAD> runs(c, p.rd);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float2 w[8], sum[8];  // weights, and their gradients' sums
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = both(0.f);
  if (norm) load_weights<T>(p.w[kind], runs, w);

  constexpr int WARPS = THREADS / 32;
  for (int64_t unit = int64_t(cta) * WARPS + warp_id(); unit < units; unit += int64_t(n_cta) * WARPS) {
    const int tg = int(unit / chunks), h0 = int(unit - int64_t(tg) * chunks) * p.chunk[kind],
              h1 = min(H, h0 + p.chunk[kind]);
    const int t = tg * C::TOKENS + lane / C::L;
    const bool on = lane < C::WORK && t < tokens;
    const int b = on ? t / p.N : 0, n = on ? t - b * p.N : 0;
    const TG* dy = static_cast<const TG*>(p.dy[kind]) + (int64_t(b) * H * p.N + n) * D;
    const T* x = static_cast<const T*>(p.x[kind]) + b * p.sb[kind] + n * p.sn[kind];
    TO* dx = static_cast<TO*>(p.dx[kind]) + b * p.dsb[kind] + n * p.dsn[kind];
    const int64_t gh = int64_t(p.N) * D, xh = p.sh[kind], dh = p.dsh[kind];
    auto fetch = [&](int i) {
      if (h0 + i < h1) {
        const int at = (i % BWD_STAGES) * (RX::BYTES + RG::BYTES);
        RG::template fetch<D>(slot_g + at, dy + (h0 + i) * gh, runs, on);
        if (norm) RX::template fetch<D>(slot_x + at, x + (h0 + i) * xh, runs, on);
      }
      rows_commit();
    };
    rows_wait<0>();
#pragma unroll
    for (int i = 0; i < BWD_STAGES - 1; ++i) fetch(i);
    float2 cs[4], sn[4];
    if (on) {
      angles<INTER, FINE>(runs, p.pos + b * p.pos_sb + n, p.pos_sa, p.freq, p.rd, p.sec0, p.sec1, cs, sn);
#pragma unroll
      for (int e = 0; e < 4; ++e) sn[e] = neg2(sn[e]);
    }
    for (int i = 0; h0 + i < h1; ++i) {
      rows_wait<BWD_STAGES - 2>();
      const int at = (i % BWD_STAGES) * (RX::BYTES + RG::BYTES);
      float2 g[8];
      RG::read(slot_g + at, g);
      if (on) turn<INTER>(g, cs, sn);
      if (norm) {
        float2 xn[8];
        RX::read(slot_x + at, xn);
        fetch(i + BWD_STAGES - 1);  // into the slot of row i - 1
        float2 sq = mul2(xn[0], xn[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) sq = fma2(xn[e], xn[e], sq);
        const float2 r = both(inverse_root<FINE>(row_sum<C::L>(sq.x + sq.y) * (1.f / D) + p.eps));
        float2 dot2 = both(0.f);
        if (on) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            xn[e] = mul2(xn[e], r);  // n
            sum[e] = fma2(g[e], xn[e], sum[e]);
            g[e] = mul2(g[e], w[e]);  // h
            dot2 = fma2(g[e], xn[e], dot2);
          }
        }
        const float2 dot = both(-row_sum<C::L>(dot2.x + dot2.y) * (1.f / D));
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = mul2(r, fma2(xn[e], dot, g[e]));
      } else {
        fetch(i + BWD_STAGES - 1);
      }
      if (on) store_row(dx + (h0 + i) * dh, runs, g);
    }
  }
  if (!norm) return;
  // rows of a warp, then the warps
  float* s_sum = reinterpret_cast<float*>(rope_smem);  // [warps][D], over the slots
  rows_wait<0>();
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 v = make_float2(rows_sum<C::L>(sum[e].x), rows_sum<C::L>(sum[e].y));
    if (lane < C::L) *reinterpret_cast<float2*>(&s_sum[warp_id() * D + runs.q[e >> 1] * 4 + 2 * (e & 1)]) = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += THREADS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) v += s_sum[w * D + i];
    p.part[int64_t(blockIdx.x) * D + i] = v;
  }
}

// dw of q (blockIdx.y 0) and k (1), 8 columns a CTA: 64 strands per column add the CTAs' partial
// sums, then the strands are added pairwise (one CTA per 32 columns with 8 strands took 9 to 29 us).
__global__ void __launch_bounds__(512) fa_qk_norm_rope_dw_kernel(const float* part, float* dwq, float* dwk, int D,
                                                                 int ctas_q, int ctas) {
  __shared__ float s[512];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int r0 = blockIdx.y ? ctas_q : 0, r1 = blockIdx.y ? ctas : ctas_q;
  const int col = blockIdx.x * 8 + (threadIdx.x & 7), strand = threadIdx.x >> 3;
  float v = 0.f;
#pragma unroll 4
  for (int r = r0 + strand; r < r1; r += 64) v += part[int64_t(r) * D + col];
  s[threadIdx.x] = v;
  for (int k = 256; k >= 8; k >>= 1) {
    __syncthreads();
    if (int(threadIdx.x) < k) s[threadIdx.x] += s[threadIdx.x + k];
  }
  if (threadIdx.x < 8) (blockIdx.y ? dwk : dwq)[col] = s[threadIdx.x];
}

}  // namespace fa
