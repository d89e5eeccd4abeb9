// The walk over keys and values that attention over prompts and over the cache
// share.
//
// Stage: where the tiles come from.  next_k and next_v turn to the next tile of the
// keys or the values (from the first on; behind the last they load zeros or
// nothing), load_k and load_v start load i of LOADS of a tile, straight into LDS
// (DIRECT) or into registers, from where finish_k and finish_v take it there.  gap:
// no token of the step's tile is there; asked for once a step, in order (GAPS).
//
// A wave takes 32 query rows, a block NW waves of them, and the block goes over
// the keys and values 32 tokens at a time.  The transposed product S^T = K Q^T
// leaves one query row per lane (its other half in lane + 32), so the softmax's
// maximum and sum are taken within the lane and once across the halves, and
// exp(S^T) is the right operand of O^T = V^T P^T as it stands: k runs over the
// tokens in the order in which the lane holds them, and V^T is read from LDS in
// that order.
#pragma once

#include "gdn_mma.h"

namespace {

// Infinities and NaN of a tile of v that some row must not see (0 x inf would take
// them to it): they become 0 in LDS, and odd[e] the first token whose element e
// is one (odd[D] the first of all).  A row that sees that token sees all before
// it, so its element e is NaN in the end.
template <typename TK, int D, int ROWS, int THREADS>
__device__ __forceinline__ void set_aside(char* tile, int j0, int* odd, int tid) {
  using P = Plane<TK, D, ROWS>;
  constexpr int CPR = P::RB / 16;
#pragma unroll 1
  for (int c = tid; c < ROWS * CPR; c += THREADS) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(tile + 16 * c);
    bool bad = false;
#pragma unroll
    for (int w = 0; w < 4; ++w) bad |= (x[w] & 0x7f800000u) == 0x7f800000u || (x[w] & 0x7f80u) == 0x7f80u;
    if (!bad) continue;
    const int r = c / CPR, e0 = ((c % CPR) ^ swizzle<P::RB>(r)) * 8;
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      uint16_t* y = reinterpret_cast<uint16_t*>(tile + 16 * c) + e;
      if ((*y & 0x7f80u) != 0x7f80u) continue;
#pragma unroll
      for (int i = 0; i < P::N; ++i) y[i * (P::BYTES / 2)] = 0;
      atomicMin(&odd[e0 + e], j0 + r);
      atomicMin(&odd[D], j0 + r);
    }
  }
}

// What a wave has of its rows: O^T's sums, the running maximum and sum.
template <int D>
struct AttnState {
  v16f acc[D / 32];
  float m = -INFINITY, l = 0.0f;
  __device__ __forceinline__ AttnState() {
#pragma unroll
    for (int d = 0; d < D / 32; ++d) acc[d] = zero16();
  }
};
// The places of a wave's rows and of its block's.
struct AttnRows {
  int lim;       // the lane's row sees tokens up to here
  int lo, hi;    // the least and (for the gradient) the largest of the wave's rows
  int block_lo;  // the least of the block's
};

constexpr int kAttnStep = 32;             // tokens a step
constexpr int kAttnWaves = 4, kAttnRows = 32 * kAttnWaves;  // of a block
// Waves a SIMD that the walk's registers leave room for: two for bf16 heads up to 128
// (222 registers) and fp32 heads of 64, else one.
template <typename T, int D>
constexpr int kAttnOcc = sizeof(T) == 2 ? (D <= 128 ? 2 : 1) : (D <= 64 ? 2 : 1);

// Groups of waves that share a block's rows, each of which takes every second tile:
// two where two waves fit a SIMD and an fp32 step (2.6 times the products of a bf16
// one, and as much again to take tiles and weights into parts) leaves each waiting
// (1, 777, 2049 and 1003 tokens, 6 heads of 64: forward 98 us with one, 79 with two;
// dq 136 and 115).
template <typename T, int D>
constexpr int kAttnGroups = sizeof(T) == 4 && D <= 64 ? 2 : 1;

// Goes over tiles [j, end) of 32 tokens.  T: the rows' type, TK: the tiles'.  NG
// groups of NW waves, of which group grp takes the tiles j + grp, j + grp + NG, ..
// (the same number of each; what lies behind the end is masked); group 0 has the
// sums of all in the end.
//
// Step j: first half, the products S of tile j + 1 beside the first part of the
// softmax of tile j; then tile j + 2 of the keys and j + 1 of the values have
// arrived; second half, the products with the values of tile j beside the rest of
// the softmax and the loads of the tiles behind.  The halves are laid out in slots
// of one product each, with the LDS reads AHEAD slots before the products that
// take them (a product is 32 cycles, a read some 100), so that one wave a SIMD
// keeps the matrix cores busy.
//
// What bounds it: the matrix cores, at the clock that they leave (2.0 of 2.4 GHz).  32
// prompts of 128 to 8192 tokens, 16 and 2 heads of 256, bf16: 8.0 ms, 907 TFLOP/s,
// where a library product of 8192^3 reaches 1140; products fill 44% of the CUs'
// cycles, vector instructions 29%, LDS 22% without a bank conflict.  8x4096, 32 and 8
// heads of 128: 1.2 ms, 917 TFLOP/s.  Not faster: loads two tiles further ahead, tiles
// sorted over all sequences, two chains of products in the first half, the step once
// in a loop with its buffers by pointer (17.4 ms).
//
// The running maximum moves only where a row's grows by more than 2^kLazy: until
// then exp(s - m) is at most that, which costs no bits.  Its sum is taken in fp32.  For
// the product exp(s - m) of bf16 rows is rounded to bf16, 2^-8 of each weight: outputs
// are 2.1e-3 off (norms; over the cache 2.3e-3), where their own rounding is 1.65e-3.  In
// two parts they would be at that, for 8.0 -> 10.1 ms of the 32 prompts, 188 -> 238 us of
// 4x2048 and 307 -> 367 over the cache: the matrix cores are what bounds it.  Of fp32 rows
// all three parts go in.
constexpr float kLazy = 8.0f;

// x *= f for sums that stay in the accumulation registers.  Written out, because
// the compiler otherwise takes them to the others and back on every step (100
// moves), whether they change or not.  The waits cover a product's result before
// it is read (18 cycles at most) and a register before a product takes it.
__device__ __forceinline__ void scale_in_agprs(v16f& x, float f) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    float a = x[i], b = x[i + 1], c = x[i + 2], d = x[i + 3], t, u, v, w;
    asm volatile(
        "s_nop 15\n\ts_nop 7\n\t"
        "v_accvgpr_read_b32 %4, %0\n\tv_accvgpr_read_b32 %5, %1\n\tv_accvgpr_read_b32 %6, %2\n\tv_accvgpr_read_b32 %7, %3\n\t"
        "s_nop 1\n\t"
        "v_mul_f32 %4, %4, %8\n\tv_mul_f32 %5, %5, %8\n\tv_mul_f32 %6, %6, %8\n\tv_mul_f32 %7, %7, %8\n\t"
        "v_accvgpr_write_b32 %0, %4\n\tv_accvgpr_write_b32 %1, %5\n\tv_accvgpr_write_b32 %2, %6\n\tv_accvgpr_write_b32 %3, %7\n\t"
        "s_nop 7"
        : "+a"(a), "+a"(b), "+a"(c), "+a"(d), "=&v"(t), "=&v"(u), "=&v"(v), "=&v"(w)
        : "v"(f));
    x[i] = a; x[i + 1] = b; x[i + 2] = c; x[i + 3] = d;
  }
  asm volatile("" : "+a"(x));
}
template <typename T, typename TK, int D, int NW, int NG, class Stage>
__device__ __forceinline__ void attn_walk(Stage& st, int grp, const Held<T, D> (&q)[D / 16], int j, int end, const AttnRows& rows,
                                          float c, int lane, int* odd, AttnState<D>& a) {
  constexpr int BN = kAttnStep, KS = D / 16, ND = D / 32, AHEAD = sizeof(T) == 2 ? 4 : 2, TOP = KS / 4;
  using P = Plane<TK, D, BN>;
  // fp32 tiles at d = 256 have room for one of each, and take the step's parts one
  // after another
  constexpr bool ONE = 6 * P::TILE > 152 * 1024;
  constexpr int REST = ONE ? 16 : P::TILE;
  __shared__ __align__(1024) char kA_[NG * P::TILE], kB_[NG * REST], kC_[NG * REST], vA_[NG * P::TILE], vB_[NG * REST], vC_[NG * REST];
  char *kA = kA_ + grp * P::TILE, *vA = vA_ + grp * P::TILE;
  char *kB = kB_ + grp * REST, *kC = kC_ + grp * REST, *vB = vB_ + grp * REST, *vC = vC_ + grp * REST;
  for (int e = threadIdx.x; e < D + 1; e += NG * NW * 64) odd[e] = INT32_MAX;
  if (j >= end) {
    __syncthreads();
    return;
  }
  const int j_0 = j, own = grp * BN;
  end = j + (end - j + NG - 1) / NG;                               // steps, from here on
  auto place = [&](int j) { return (j_0 + (j - j_0) * NG) * BN; };  // of group 0's tile
  auto clean = [&](char* vb, int j) {
    if (place(j) + NG * BN - 1 > rows.block_lo) {  // some place is masked for some row of the block
      set_aside<TK, D, BN, NW * 64>(vb, place(j) + own, odd, threadIdx.x - grp * NW * 64);
      __syncthreads();
    }
  };
  v16f s, sn;
  auto hide = [&](int j0) {
    if (j0 + BN - 1 > rows.lo) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (j0 + c_row(i, lane) > rows.lim) s[i] = -INFINITY;
    }
    if constexpr (Stage::GAPS) {
      if (st.gap()) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = -INFINITY;
      }
    }
  };
  auto raise = [&](float top) {  // the maximum; what it is in log2 afterwards, 0 for none
    top = fmaxf(top, other_half(top));
    if (__any(top * c > a.m * c + kLazy)) {
      const bool move = top * c > a.m * c + kLazy;
      const float f = move ? __builtin_amdgcn_exp2f((a.m - top) * c) : 1.0f;  // 0 from m = -inf
      if (__any(a.m > -INFINITY)) {  // else the sums are 0
        a.l *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          if constexpr (kAttnOcc<T, D> == 1)
            scale_in_agprs(a.acc[d], f);
          else
            a.acc[d] *= f;
        }
      }
      a.m = move ? top : a.m;
    }
    return a.m == -INFINITY ? 0.0f : a.m * c;
  };
  auto weight = [&](int i, float mc) {
    float e = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc));
    asm volatile("" : "+v"(e));  // here, and not where it is used
    s[i] = e;
    a.l += e;
  };
  auto load = [&](bool keys, char* buf) {  // a whole tile
#pragma unroll
    for (int i = 0; i < Stage::LOADS; ++i) keys ? st.load_k(i, buf) : st.load_v(i, buf);
  };
  st.next_k();
  load(true, kA);
  st.next_v();
  load(false, vA);
  if constexpr (ONE) {
    for (; j < end; ++j) {
      st.finish_k(kA);
      st.finish_v(vA);
      __syncthreads();
      st.next_k();
      load(true, kA);
      st.next_v();
      load(false, vA);
      clean(vA, j);
      s = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) s = mma32(row_frag<TK, D, BN>(kA, 0, ks, lane), q[ks].get(), s);
      hide(place(j) + own);
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[i]);
      const float mc = raise(top);
#pragma unroll
      for (int i = 0; i < 16; ++i) weight(i, mc);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        Frag<T> p;
        p.pack(s, 8 * u);
#pragma unroll
        for (int d = 0; d < ND; ++d) a.acc[d] = mma32(col_frag<TK, D, BN>(vA, 16 * u, d, lane), p, a.acc[d]);
      }
      __syncthreads();
    }
  } else {
    Frag<TK> rf[KS], cf[2 * ND];
    // v0: values of tile j, k1 and v1: tile j + 1, k2: keys of tile j + 2; into k3 and
    // v2 go the next ones
    auto step = [&](char* v0, char* k1, char* v1, char* k2, char* v2, char* k3, int j) {
      hide(place(j) + own);
      sn = zero16();
      auto product = [&](int m) {
        if (m + AHEAD < KS) rf[m + AHEAD] = row_frag<TK, D, BN>(k1, 0, m + AHEAD, lane);
        if (m >= KS - AHEAD) cf[m - KS + AHEAD] = col_frag<TK, D, BN>(v0, 16 * ((m - KS + AHEAD) / ND), (m - KS + AHEAD) % ND, lane);
        sn = mma32(rf[m], q[m].get(), sn);
      };
      float top = -INFINITY;
#pragma unroll
      for (int m = 0; m < TOP; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        product(m);
#pragma unroll
        for (int i = 16 * m / TOP; i < 16 * (m + 1) / TOP; ++i) top = fmaxf(top, s[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      const float mc = raise(top);
      Frag<T> p[2];
#pragma unroll
      for (int m = TOP; m < KS; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        product(m);
#pragma unroll
        for (int i = 8 * (m - TOP) / (KS - TOP); i < 8 * (m - TOP + 1) / (KS - TOP); ++i) weight(i, mc);
        if constexpr (!Stage::DIRECT) {
          if (m == KS - 2) st.finish_k(k2);
          if (m == KS - 1) st.finish_v(v1);
        }
        if (m == KS - 1) p[0].pack(s, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      wait_loads();
      __syncthreads();
      if (j + 1 < end) clean(v1, j + 1);
      st.next_k();
      st.next_v();
#pragma unroll
      for (int f = 0; f < 2 * ND; ++f) {
        __builtin_amdgcn_sched_barrier(0);
        if (f + AHEAD < 2 * ND) cf[f + AHEAD] = col_frag<TK, D, BN>(v0, 16 * ((f + AHEAD) / ND), (f + AHEAD) % ND, lane);
        if (f >= 2 * ND - AHEAD) rf[f - 2 * ND + AHEAD] = row_frag<TK, D, BN>(k2, 0, f - 2 * ND + AHEAD, lane);
        a.acc[f % ND] = mma32(cf[f], p[f / ND], a.acc[f % ND]);
        constexpr int N = 2 * Stage::LOADS;
#pragma unroll
        for (int i = f * N / (2 * ND); i < (f + 1) * N / (2 * ND); ++i) i < N / 2 ? st.load_k(i, k3) : st.load_v(i - N / 2, v2);
        if (f < ND) {
#pragma unroll
          for (int i = 8 + 8 * f / ND; i < 8 + 8 * (f + 1) / ND; ++i) weight(i, mc);
        }
        if (f == ND - 1) p[1].pack(s, 8);
      }
      __builtin_amdgcn_sched_barrier(0);
      s = sn;
    };
    if constexpr (!Stage::DIRECT) {
      st.finish_k(kA);
      st.finish_v(vA);
    }
    st.next_k();
    load(true, kB);
    if constexpr (!Stage::DIRECT) st.finish_k(kB);
    st.next_k();
    load(true, kC);
    st.next_v();
    load(false, vB);
    if constexpr (Stage::DIRECT) wait_loads<2 * Stage::LOADS>();
    __syncthreads();
    clean(vA, j);
    s = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) s = mma32(row_frag<TK, D, BN>(kA, 0, ks, lane), q[ks].get(), s);
#pragma unroll
    for (int m = 0; m < AHEAD; ++m) rf[m] = row_frag<TK, D, BN>(kB, 0, m, lane);
    for (; j < end; j += 3) {
      step(vA, kB, vB, kC, vC, kA, j);
      if (j + 1 < end) step(vB, kC, vC, kA, vA, kB, j + 1);
      if (j + 2 < end) step(vC, kA, vA, kB, vB, kC, j + 2);
      if constexpr (kAttnOcc<T, D> == 1) {
#pragma unroll
        for (int d = 0; d < ND; ++d) in_agprs(a.acc[d]);
      }
    }
  }
  wait_loads();
  __syncthreads();
  if constexpr (NG == 2) {  // through LDS: half of the sums in kA_, half in kB_
    static_assert(NG * P::TILE >= D * NW * 64 && !ONE);
    const int at = threadIdx.x & (NW * 64 - 1);
    float *s0 = reinterpret_cast<float*>(kA_) + at, *s1 = reinterpret_cast<float*>(kB_) + at, *ml = reinterpret_cast<float*>(kC_) + at;
    constexpr int H = D / 4;
    if (grp == 1) {
#pragma unroll
      for (int i = 0; i < 2 * H; ++i) (i < H ? s0 + i * NW * 64 : s1 + (i - H) * NW * 64)[0] = a.acc[i / 16][i % 16];
      ml[0] = a.m;
      ml[NW * 64] = a.l;
    }
    __syncthreads();
    if (grp == 1) return;
    const float top = fmaxf(a.m, ml[0]);
    const float f0 = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((a.m - top) * c);
    const float f1 = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((ml[0] - top) * c);
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) a.acc[i / 16][i % 16] = a.acc[i / 16][i % 16] * f0 + (i < H ? s0 + i * NW * 64 : s1 + (i - H) * NW * 64)[0] * f1;
    a.m = top;
    a.l = a.l * f0 + ml[NW * 64] * f1;
  }
  a.l += other_half(a.l);
  // The maximum's own weight is exp2 of what m c lost when it was rounded, 2^-64 at
  // least up to scores of 2^30.  Of far larger ones, or where m c is infinite, all
  // weights may be 0: NaN, and not a row that sees nothing.
  if (a.l == 0.0f && a.m > -INFINITY) a.l = NAN;
  if (odd[D] != INT32_MAX) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (rows.lim >= odd[32 * d + c_row(i, lane)]) a.acc[d][i] = NAN;
  }
}

// Writes the lane's part of a row: its elements 32 d + 8 x + 4 (l / 32) .. + 3, times f.
template <int D, typename T>
__device__ __forceinline__ void store_row(T* o, const v16f (&acc)[D / 32], float f, int lane) {
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float y[4] = {acc[d][4 * x] * f, acc[d][4 * x + 1] * f, acc[d][4 * x + 2] * f, acc[d][4 * x + 3] * f};
      store4(o + 32 * d + 8 * x + 4 * (lane >> 5), y);
    }
}
// 1 / sum, 0 for a row that sees nothing; and its lse from the maximum in log2.
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.0f || l != l ? 1.0f / l : 0.0f; }
__device__ __forceinline__ float lse_of(float m2, float l) { return l > 0.0f ? (m2 + __log2f(l)) * kLn2 : l != l ? l : -INFINITY; }

}  // namespace
