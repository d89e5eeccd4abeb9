// The walk over keys and values that attention over prompts and over the cache
// share.
//
// A wave takes 32 query rows, a block NW waves of them, and the block goes over
// the keys and values BN tokens at a time.  The transposed product S^T = K Q^T
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
__device__ __forceinline__ void set_aside(char* tile, int j0, int* odd) {
  using P = Plane<TK, D, ROWS>;
  constexpr int CPR = P::RB / 16;
#pragma unroll 1
  for (int c = threadIdx.x; c < ROWS * CPR; c += THREADS) {
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
  int lo, hi;    // the least and the largest of the wave's rows
  int block_lo;  // the least of the block's
};

template <typename T, int D>
struct AttnTile {
  static constexpr int NW = 4, BM = 32 * NW;
  static constexpr int BN = sizeof(T) == 2 && D <= 128 ? 64 : 32;  // tokens a step
};

// Steps [j, end) of BN tokens.  T: the rows' type, TK: the tiles'.
template <typename T, typename TK, int D, int BN, int NW, class Stage>
__device__ __forceinline__ void attn_walk(Stage& st, const Held<T, D> (&q)[D / 16], int j, int end, const AttnRows& rows,
                                          float c, int lane, int* odd, AttnState<D>& a) {
  using P = Plane<TK, D, BN>;
  constexpr int NS = BN / 32, KS = D / 16, ND = D / 32;
  constexpr bool TWO = 4 * P::TILE <= 144 * 1024;  // buffers
  __shared__ __align__(1024) char kA[P::TILE], vA[P::TILE], kB[TWO ? P::TILE : 16], vB[TWO ? P::TILE : 16];
  for (int e = threadIdx.x; e < D + 1; e += NW * 64) odd[e] = INT32_MAX;
  auto step = [&](char* kb, char* vb, char* kn, char* vn, int j) {
    if constexpr (Stage::DIRECT) wait_loads();
    __syncthreads();
    if (j + 1 < end) st.start(j + 1, kn, vn);
    const int j0 = j * BN;
    if (j0 + BN - 1 > rows.block_lo) {  // some place is masked for some row of the block
      set_aside<TK, D, BN, NW * 64>(vb, j0, odd);
      __syncthreads();
    }
    if (j0 <= rows.hi) {
      v16f s[NS];
#pragma unroll
      for (int t = 0; t < NS; ++t) {
        s[t] = zero16();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) s[t] = mma32(row_frag<TK, D, BN>(kb, 32 * t, ks, lane), q[ks].get(), s[t]);
      }
      if (j0 + BN - 1 > rows.lo) {
#pragma unroll
        for (int t = 0; t < NS; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j0 + 32 * t + c_row(i, lane) > rows.lim) s[t][i] = -INFINITY;
      }
      if constexpr (Stage::GAPS) {
#pragma unroll
        for (int t = 0; t < NS; ++t)
          if (st.gap(t)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = -INFINITY;
          }
      }
      float top = a.m;
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
      top = fmaxf(top, other_half(top));
      if (__any(top > a.m)) {
        const float f = top > a.m ? __builtin_amdgcn_exp2f((a.m - top) * c) : 1.0f;  // 0 from m = -inf
        a.m = top;
        a.l *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) a.acc[d] *= f;
      }
      const float mc = a.m == -INFINITY ? 0.0f : a.m * c;
#pragma unroll
      for (int t = 0; t < NS; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -mc));
          a.l += s[t][i];
        }
      }
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          Frag<T> p;
          p.pack(s[t], 8 * u);
#pragma unroll
          for (int d = 0; d < ND; ++d) a.acc[d] = mma32(col_frag<TK, D, BN>(vb, 32 * t + 16 * u, d, lane), p, a.acc[d]);
        }
    }
    if constexpr (!Stage::DIRECT) {
      if constexpr (!TWO) __syncthreads();
      if (j + 1 < end) st.finish(kn, vn);
    }
  };
  if (j < end) {
    st.start(j, kA, vA);
    if constexpr (!Stage::DIRECT) st.finish(kA, vA);
  }
  if constexpr (TWO) {
    for (; j < end; j += 2) {
      step(kA, vA, kB, vB, j);
      if (j + 1 < end) step(kB, vB, kA, vA, j + 1);
    }
  } else {
    for (; j < end; ++j) step(kA, vA, kA, vA, j);
  }
  __syncthreads();
  a.l += other_half(a.l);
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
