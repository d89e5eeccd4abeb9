// Causal attention over packed sequences with grouped heads (include/gdn.h):
// kernels and C ABI.
#include "gdn_mma.h"

namespace {

struct AttnIO {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;           // [T_q][H_q], nullable forward
  const int32_t* cu_q;  // [N + 1]
  const int32_t* cu_k;
  int64_t T_q, T_k, ldq, ldk, ldv, ldo;
  int N, H_q, H_kv, G;
  float c;  // scale log2(e)
};

// The rows of one sequence, clamped to the buffers.
struct Span {
  int64_t q0, k0;
  int Lq, Lk;
};
__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }
__device__ __forceinline__ Span span_of(const int32_t* cu_q, const int32_t* cu_k, int64_t T_q, int64_t T_k, int n) {
  Span s;
  s.q0 = clamp64(cu_q[n], 0, T_q);
  s.Lq = static_cast<int>(clamp64(cu_q[n + 1], s.q0, T_q) - s.q0);
  s.k0 = clamp64(cu_k[n], 0, T_k);
  s.Lk = static_cast<int>(clamp64(cu_k[n + 1], s.k0, T_k) - s.k0);
  return s;
}

// The sequence that owns tile slot x, where sequence n's slots begin at cu[n] /
// rows + n (at least as many as it has tiles, whatever the lengths), and the
// tile within it.
__device__ __forceinline__ int tile_seq(const int32_t* __restrict__ cu, int N, int rows, int x, int* tile) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] / rows + mid <= x) lo = mid; else hi = mid - 1;
  }
  *tile = x - (cu[lo] / rows + lo);
  return lo;
}
inline int64_t tile_slots(int64_t T, int64_t N, int rows) { return T / rows + N; }

// ---- forward ------------------------------------------------------------------
//
// A wave takes 32 query rows of one head, a block NW waves of them, and the
// block goes over the keys and values BN tokens at a time.  The transposed
// product S^T = K Q^T leaves one query row per lane (its other half in lane +
// 32), so the softmax's maximum and sum are taken within the lane and once
// across the halves, and exp(S^T) is the right operand of O^T = V^T P^T as it
// stands: k runs over the tokens in the order in which the lane holds them, and
// V^T is read from LDS in that order.
template <typename T, int D>
struct FwdTile {
  static constexpr int BN = sizeof(T) == 2 && D <= 128 ? 64 : 32;  // keys a step
  static constexpr int NW = 4;
  static constexpr int BM = 32 * NW;
};

// Infinities and NaN of a tile of v that some row must not see (0 x inf would take
// them to it): they become 0 in LDS, and odd[e] the first token whose element e
// is one (odd[D] the first of all).  A row that sees that token sees all before
// it, so its element e is NaN in the end.
template <typename T, int D, int ROWS, int THREADS>
__device__ __forceinline__ void set_aside(char* tile, int j0, int* odd) {
  constexpr int RB = D * sizeof(T), CPR = RB / 16, E = 16 / sizeof(T);
#pragma unroll 1
  for (int c = threadIdx.x; c < ROWS * CPR; c += THREADS) {
    u32x4* at = reinterpret_cast<u32x4*>(tile) + c;
    const u32x4 x = *at;
    constexpr uint32_t lo = sizeof(T) == 2 ? 0x7f80u : 0, hi = 0x7f800000u;
    bool bad = false;
#pragma unroll
    for (int w = 0; w < 4; ++w) bad |= (x[w] & hi) == hi || (sizeof(T) == 2 && (x[w] & lo) == lo);
    if (!bad) continue;
    const int r = c / CPR, e0 = ((c % CPR) ^ swizzle<RB>(r)) * E;
    T* y = reinterpret_cast<T*>(at);
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
      uint32_t u = sizeof(T) == 2 ? static_cast<uint32_t>(reinterpret_cast<uint16_t*>(y)[e]) << 16 : reinterpret_cast<uint32_t*>(y)[e];
      if ((u & hi) != hi) continue;
      y[e] = 0;
      atomicMin(&odd[e0 + e], j0 + r);
      atomicMin(&odd[D], j0 + r);
    }
  }
}

template <typename T, int D>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void k_attn_fwd(AttnIO io) {
#ifdef GDN_DEVICE_PASS
  using Tile = FwdTile<T, D>;
  constexpr int BN = Tile::BN, BM = Tile::BM, NW = Tile::NW, NS = BN / 32, KS = D / 16, ND = D / 32;
  constexpr int RB = D * sizeof(T);
  __shared__ __align__(1024) char kA[BN * RB], vA[BN * RB], kB[BN * RB], vB[BN * RB];
  __shared__ int odd[D + 1];
  const int hk = blockIdx.x % io.H_kv;
  const int y = blockIdx.x / io.H_kv;
  const int hq = hk * io.G + y % io.G;
  int tile;
  const int n = tile_seq(io.cu_q, io.N, BM, y / io.G, &tile);
  const Span sp = span_of(io.cu_q, io.cu_k, io.T_q, io.T_k, n);
  const int tiles = (sp.Lq + BM - 1) / BM;
  if (tile < 0 || tile >= tiles) return;
  tile = tiles - 1 - tile;  // the longest first
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r0 = tile * BM + wave * 32, row = r0 + (lane & 31);
  const int off = sp.Lk - sp.Lq;  // row i sees keys up to i + off
  const int last = (tile + 1) * BM < sp.Lq ? (tile + 1) * BM - 1 : sp.Lq - 1;
  const int steps = last + off >= 0 ? (last + off) / BN + 1 : 0;
  const int lim = row < sp.Lq ? row + off : -1;
  const int wave_last = r0 + 31 < sp.Lq ? r0 + 31 : sp.Lq - 1;
  const int lim_hi = r0 < sp.Lq ? wave_last + off : -1, lim_lo = r0 + off;  // of the wave's rows

  Frag<T> q[KS];
  {
    const int rows = sp.Lq - r0 < 32 ? sp.Lq - r0 : 32;
    const brsrc_t rq = rows_rsrc<T, D>(io.q, sp.q0 + (rows > 0 ? r0 : 0), io.ldq, hq, rows);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks].load(rq, (lane & 31) * io.ldq * sizeof(T) + (16 * ks + 8 * (lane >> 5)) * sizeof(T));
  }
  const Stager<T, D, BN, NW> sk(io.ldk, wave, lane), sv(io.ldv, wave, lane);
  auto fetch = [&](char* kb, char* vb, int j) {
    const int rows = sp.Lk - j * BN < BN ? sp.Lk - j * BN : BN;
    sk.start(rows_rsrc<T, D>(io.k, sp.k0 + j * BN, io.ldk, hk, rows), kb);
    sv.start(rows_rsrc<T, D>(io.v, sp.k0 + j * BN, io.ldv, hk, rows), vb);
  };

  v16f acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = zero16();
  float m = -INFINITY, l = 0.0f;
  const int edge_lo = tile * BM + off;  // behind it places are masked for some row of the block
  for (int e = threadIdx.x; e < D + 1; e += NW * 64) odd[e] = INT32_MAX;
  __syncthreads();

  auto step = [&](char* kb, char* vb, char* kn, char* vn, int j) {
    wait_loads();
    __syncthreads();
    if (j + 1 < steps) fetch(kn, vn, j + 1);
    const int j0 = j * BN;
    if (j0 + BN - 1 > edge_lo) {
      set_aside<T, D, BN, NW * 64>(vb, j0, odd);
      __syncthreads();
    }
    if (j0 > lim_hi) return;
    v16f s[NS];
#pragma unroll
    for (int t = 0; t < NS; ++t) {
      s[t] = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) s[t] = mma32(row_frag<T, RB>(kb, 32 * t, ks, lane), q[ks], s[t]);
    }
    const bool edge = j0 + BN - 1 > lim_lo;  // some place is masked for some row
    if (edge) {
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j0 + 32 * t + c_row(i, lane) > lim) s[t][i] = -INFINITY;
    }
    float top = m;
#pragma unroll
    for (int t = 0; t < NS; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
    top = fmaxf(top, other_half(top));
    if (__any(top > m)) {
      const float f = top > m ? __builtin_amdgcn_exp2f((m - top) * io.c) : 1.0f;  // 0 from m = -inf
      m = top;
      l *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[d] *= f;
    }
    const float mc = m == -INFINITY ? 0.0f : m * io.c;
    Frag<T> p[NS][2];
#pragma unroll
    for (int t = 0; t < NS; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], io.c, -mc));
        l += s[t][i];
      }
      p[t][0].pack(s[t], 0);
      p[t][1].pack(s[t], 8);
    }
#pragma unroll
    for (int t = 0; t < NS; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = mma32(col_frag<T, RB>(vb, 32 * t + 16 * u, d, lane), p[t][u], acc[d]);
  };
  if (steps > 0) fetch(kA, vA, 0);
  for (int j = 0; j < steps; j += 2) {
    step(kA, vA, kB, vB, j);
    if (j + 1 < steps) step(kB, vB, kA, vA, j + 1);
  }

  l += other_half(l);
  __syncthreads();
  if (odd[D] != INT32_MAX) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (lim >= odd[32 * d + c_row(i, lane)]) acc[d][i] = NAN;
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;  // an empty row is 0
  if (row < sp.Lq) {
    T* o = static_cast<T*>(io.o) + (sp.q0 + row) * io.ldo + static_cast<int64_t>(hq) * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float x[4] = {acc[d][4 * a] * inv, acc[d][4 * a + 1] * inv, acc[d][4 * a + 2] * inv, acc[d][4 * a + 3] * inv};
        store4(o + 32 * d + 8 * a + 4 * (lane >> 5), x);
      }
    if (io.lse && lane < 32)
      io.lse[(sp.q0 + row) * io.H_q + hq] = l > 0.0f ? (m * io.c + __log2f(l)) * kLn2 : l != l ? l : -INFINITY;
  }
#endif
}

// ---- gradient -----------------------------------------------------------------
//
// Two kernels, no atomics.  k_attn_dq goes over the keys for 32 query rows a wave
// as the forward does (S^T and dP^T leave a query row per lane, whose lse and
// dO . o are then one number each) and keeps those two numbers for the second.
// k_attn_dkv goes over the queries of all heads of the group for 32 keys a wave,
// with S and dP in the other orientation (a key per lane), so that P and dS are
// right operands of dV^T = dO^T P and dK^T = Q^T dS as they stand.
struct GradIO {
  AttnIO a;  // o: the forward's output, read
  const void* dO;
  void* dq;
  void* dk;
  void* dv;
  float* stat;  // [H_q][T_q][2]: lse log2(e) and dO . o
  int64_t lddo, lddq, lddk, lddv;
  float scale;
};

template <typename T, int D>
__global__ __launch_bounds__(256, sizeof(T) == 2 && D <= 128 ? 2 : 1) void k_attn_dq(GradIO g) {
#ifdef GDN_DEVICE_PASS
  constexpr int BN = 32, NW = 4, BM = 32 * NW, KS = D / 16, ND = D / 32, RB = D * sizeof(T);
  __shared__ __align__(1024) char kA[BN * RB], vA[BN * RB], kB[BN * RB], vB[BN * RB];
  const AttnIO& io = g.a;
  const int hk = blockIdx.x % io.H_kv;
  const int y = blockIdx.x / io.H_kv;
  const int hq = hk * io.G + y % io.G;
  int tile;
  const int n = tile_seq(io.cu_q, io.N, BM, y / io.G, &tile);
  const Span sp = span_of(io.cu_q, io.cu_k, io.T_q, io.T_k, n);
  const int tiles = (sp.Lq + BM - 1) / BM;
  if (tile < 0 || tile >= tiles) return;
  tile = tiles - 1 - tile;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r0 = tile * BM + wave * 32, row = r0 + (lane & 31);
  const int off = sp.Lk - sp.Lq;
  const int last = (tile + 1) * BM < sp.Lq ? (tile + 1) * BM - 1 : sp.Lq - 1;
  const int steps = last + off >= 0 ? (last + off) / BN + 1 : 0;
  const int lim = row < sp.Lq ? row + off : -1;
  const int wave_last = r0 + 31 < sp.Lq ? r0 + 31 : sp.Lq - 1;
  const int lim_hi = r0 < sp.Lq ? wave_last + off : -1, lim_lo = r0 + off;

  Frag<T> q[KS], dO[KS];
  float lse2, dot = 0.0f;
  {
    const int rows = sp.Lq - r0 < 32 ? sp.Lq - r0 : 32;
    const int64_t at = sp.q0 + (rows > 0 ? r0 : 0);
    const brsrc_t rq = rows_rsrc<T, D>(io.q, at, io.ldq, hq, rows);
    const brsrc_t rd = rows_rsrc<T, D>(g.dO, at, g.lddo, hq, rows);
    const brsrc_t ro = rows_rsrc<T, D>(io.o, at, io.ldo, hq, rows);
    const uint32_t col = 8 * (lane >> 5) * sizeof(T), r = lane & 31;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks].load(rq, static_cast<uint32_t>(r * io.ldq * sizeof(T)) + col + 16 * ks * sizeof(T));
      dO[ks].load(rd, static_cast<uint32_t>(r * g.lddo * sizeof(T)) + col + 16 * ks * sizeof(T));
      Frag<T> o;
      o.load(ro, static_cast<uint32_t>(r * io.ldo * sizeof(T)) + col + 16 * ks * sizeof(T));
      dot += o.dot(dO[ks]);
    }
    dot += other_half(dot);
    lse2 = row < sp.Lq ? io.lse[(sp.q0 + row) * io.H_q + hq] * kLog2e : 0.0f;
    if (row < sp.Lq && lane < 32) {
      float* s = g.stat + 2 * (static_cast<int64_t>(hq) * io.T_q + sp.q0 + row);
      s[0] = lse2;
      s[1] = dot;
    }
  }
  const Stager<T, D, BN, NW> sk(io.ldk, wave, lane), sv(io.ldv, wave, lane);
  auto fetch = [&](char* kb, char* vb, int j) {
    const int rows = sp.Lk - j * BN < BN ? sp.Lk - j * BN : BN;
    sk.start(rows_rsrc<T, D>(io.k, sp.k0 + j * BN, io.ldk, hk, rows), kb);
    sv.start(rows_rsrc<T, D>(io.v, sp.k0 + j * BN, io.ldv, hk, rows), vb);
  };
  v16f acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = zero16();
  auto step = [&](char* kb, char* vb, char* kn, char* vn, int j) {
    wait_loads();
    __syncthreads();
    if (j + 1 < steps) fetch(kn, vn, j + 1);
    const int j0 = j * BN;
    if (j0 > lim_hi) return;
    v16f s = zero16(), dp = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      s = mma32(row_frag<T, RB>(kb, 0, ks, lane), q[ks], s);
      dp = mma32(row_frag<T, RB>(vb, 0, ks, lane), dO[ks], dp);
    }
    const bool edge = j0 + BN - 1 > lim_lo;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float p = __builtin_amdgcn_exp2f(fmaf(s[i], io.c, -lse2));
      s[i] = p * (dp[i] - dot);
      if (edge && j0 + c_row(i, lane) > lim) s[i] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Frag<T> ds;
      ds.pack(s, 8 * u);
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[d] = mma32(col_frag<T, RB>(kb, 16 * u, d, lane), ds, acc[d]);
    }
  };
  if (steps > 0) fetch(kA, vA, 0);
  for (int j = 0; j < steps; j += 2) {
    step(kA, vA, kB, vB, j);
    if (j + 1 < steps) step(kB, vB, kA, vA, j + 1);
  }
  if (row < sp.Lq) {
    T* o = static_cast<T*>(g.dq) + (sp.q0 + row) * g.lddq + static_cast<int64_t>(hq) * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float x[4] = {acc[d][4 * a] * g.scale, acc[d][4 * a + 1] * g.scale, acc[d][4 * a + 2] * g.scale,
                            acc[d][4 * a + 3] * g.scale};
        store4(o + 32 * d + 8 * a + 4 * (lane >> 5), x);
      }
  }
#endif
}

// WHAT: 3 both gradients, 1 dk, 2 dv (rows of 512 bytes and more, whose two sums
// and operands together pass the registers of a wave).
template <typename T, int D, int WHAT>
__global__ __launch_bounds__(256, 1) void k_attn_dkv(GradIO g) {
#ifdef GDN_DEVICE_PASS
  constexpr int BQ = 32, NW = 4, BK = 32 * NW, KS = D / 16, ND = D / 32, RB = D * sizeof(T);
  constexpr bool DK = WHAT & 1, DV = WHAT & 2;
  __shared__ __align__(1024) char qA[BQ * RB], oA[BQ * RB], qB[BQ * RB], oB[BQ * RB];
  __shared__ __align__(1024) float sA[2 * BQ], sB[2 * BQ];
  const AttnIO& io = g.a;
  const int hk = blockIdx.x % io.H_kv;
  int tile;
  const int n = tile_seq(io.cu_k, io.N, BK, blockIdx.x / io.H_kv, &tile);
  const Span sp = span_of(io.cu_q, io.cu_k, io.T_q, io.T_k, n);
  if (tile < 0 || tile * BK >= sp.Lk) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j0 = tile * BK + wave * 32, key = j0 + (lane & 31);
  const int off = sp.Lk - sp.Lq;
  // query tiles from the first that sees one of the block's keys on
  const int first = tile * BK - off > 0 ? (tile * BK - off) / BQ : 0;
  const int per = (sp.Lq + BQ - 1) / BQ - first, steps = per > 0 ? per * io.G : 0;

  Frag<T> k[KS], v[DK ? KS : 1];
  {
    const int rows = sp.Lk - j0 < 32 ? sp.Lk - j0 : 32;
    const int64_t at = sp.k0 + (rows > 0 ? j0 : 0);
    const brsrc_t rk = rows_rsrc<T, D>(io.k, at, io.ldk, hk, rows), rv = rows_rsrc<T, D>(io.v, at, io.ldv, hk, rows);
    const uint32_t col = 8 * (lane >> 5) * sizeof(T), r = lane & 31;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      k[ks].load(rk, static_cast<uint32_t>(r * io.ldk * sizeof(T)) + col + 16 * ks * sizeof(T));
      if constexpr (DK) v[ks].load(rv, static_cast<uint32_t>(r * io.ldv * sizeof(T)) + col + 16 * ks * sizeof(T));
    }
  }
  const Stager<T, D, BQ, NW> sq(io.ldq, wave, lane), so(g.lddo, wave, lane);
  auto fetch = [&](char* qb, char* ob, float* sb, int x) {
    const int h = hk * io.G + x / per, i0 = (first + x % per) * BQ;
    const int rows = sp.Lq - i0 < BQ ? sp.Lq - i0 : BQ;
    sq.start(rows_rsrc<T, D>(io.q, sp.q0 + i0, io.ldq, h, rows), qb);
    so.start(rows_rsrc<T, D>(g.dO, sp.q0 + i0, g.lddo, h, rows), ob);
    if (wave == 0) {
      float* st = g.stat + 2 * (static_cast<int64_t>(h) * io.T_q + sp.q0 + i0);
      const brsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(st, static_cast<short>(0), rows * 8, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GDN_LDS void*)sb, 4, lane * 4, 0, 0, 0);
    }
  };
  v16f ak[DK ? ND : 1], av[DV ? ND : 1];
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    if constexpr (DK) ak[d] = zero16();
    if constexpr (DV) av[d] = zero16();
  }
  auto step = [&](char* qb, char* ob, float* sb, char* qn, char* on, float* sn, int x) {
    wait_loads();
    __syncthreads();
    if (x + 1 < steps) fetch(qn, on, sn, x + 1);
    const int i0 = (first + x % per) * BQ;
    if (i0 + BQ - 1 + off < j0) return;  // the wave's keys are all behind the tile's queries
    v16f s = zero16(), dp = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      s = mma32(row_frag<T, RB>(qb, 0, ks, lane), k[ks], s);
      if constexpr (DK) dp = mma32(row_frag<T, RB>(ob, 0, ks, lane), v[ks], dp);
    }
    const bool edge = i0 + off < j0 + 31;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float* st = sb + 2 * (8 * a + 4 * (lane >> 5));
      const v4f s0 = *reinterpret_cast<const v4f*>(st), s1 = *reinterpret_cast<const v4f*>(st + 4);
      const float lse2[4] = {s0[0], s0[2], s1[0], s1[2]}, dot[4] = {s0[1], s0[3], s1[1], s1[3]};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i = 4 * a + b;
        float p = __builtin_amdgcn_exp2f(fmaf(s[i], io.c, -lse2[b]));
        float ds = p * (dp[i] - dot[b]);
        if (edge && i0 + c_row(i, lane) + off < key) p = ds = 0.0f;
        s[i] = p;
        dp[i] = ds;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Frag<T> p, ds;
      p.pack(s, 8 * u);
      ds.pack(dp, 8 * u);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        if constexpr (DV) av[d] = mma32(col_frag<T, RB>(ob, 16 * u, d, lane), p, av[d]);
        if constexpr (DK) ak[d] = mma32(col_frag<T, RB>(qb, 16 * u, d, lane), ds, ak[d]);
      }
    }
  };
  if (steps > 0) fetch(qA, oA, sA, 0);
  for (int x = 0; x < steps; x += 2) {
    step(qA, oA, sA, qB, oB, sB, x);
    if (x + 1 < steps) step(qB, oB, sB, qA, oA, sA, x + 1);
  }
  if (key < sp.Lk) {
    T* dk = static_cast<T*>(g.dk) + (sp.k0 + key) * g.lddk + static_cast<int64_t>(hk) * D;
    T* dv = static_cast<T*>(g.dv) + (sp.k0 + key) * g.lddv + static_cast<int64_t>(hk) * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int e = 32 * d + 8 * a + 4 * (lane >> 5);
        if constexpr (DK) {
          const float x[4] = {ak[d][4 * a] * g.scale, ak[d][4 * a + 1] * g.scale, ak[d][4 * a + 2] * g.scale,
                              ak[d][4 * a + 3] * g.scale};
          store4(dk + e, x);
        }
        if constexpr (DV) {
          const float x[4] = {av[d][4 * a], av[d][4 * a + 1], av[d][4 * a + 2], av[d][4 * a + 3]};
          store4(dv + e, x);
        }
      }
  }
#endif
}

// ---- host side ----------------------------------------------------------------

template <typename T, int D>
void launch_dkv(const GradIO& g, unsigned blocks, hipStream_t st) {
  constexpr bool split = D * sizeof(T) >= 512;
  hipLaunchKernelGGL((k_attn_dkv<T, D, split ? 1 : 3>), dim3(blocks), dim3(256), 0, st, g);
  if constexpr (split) hipLaunchKernelGGL((k_attn_dkv<T, D, 2>), dim3(blocks), dim3(256), 0, st, g);
}

template <typename F>
int attn_dispatch(const gdn_attn_shape_t* s, F&& f) {
  if (s->in_dtype == GDN_BF16) {
    if (s->d == 64) return f.template operator()<bf16_t, 64>();
    if (s->d == 128) return f.template operator()<bf16_t, 128>();
    return f.template operator()<bf16_t, 256>();
  }
  if (s->d == 64) return f.template operator()<float, 64>();
  if (s->d == 128) return f.template operator()<float, 128>();
  return f.template operator()<float, 256>();
}

// Checks what the two calls share and fills io.
int attn_common(const gdn_attn_shape_t* s, int32_t N, const int32_t* cu_q, const int32_t* cu_k, int64_t T_q, int64_t T_k,
                const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv, AttnIO* io) {
  int rc = gdn::check_attn_shape(s);
  if (rc != GDN_OK) return rc;
  if (N < 0 || T_q < 0 || T_k < 0) return GDN_ERR_INVALID_ARG;
  if (!cu_q || (N == 0 && T_q > 0)) return GDN_ERR_INVALID_ARG;
  if (!cu_k) {
    if (T_k != T_q) return GDN_ERR_INVALID_ARG;
    cu_k = cu_q;
  }
  if (!gdn::aligned16({cu_q, cu_k, q, k, v})) return GDN_ERR_INVALID_ARG;
  if ((T_q > 0 && !q) || (T_k > 0 && (!k || !v))) return GDN_ERR_INVALID_ARG;
  if (T_q > INT32_MAX || T_k > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  const int64_t wq = static_cast<int64_t>(s->H_q) * s->d, wk = static_cast<int64_t>(s->H_kv) * s->d;
  rc = gdn::attn_rows({{ldq, wq, &io->ldq}, {ldk, wk, &io->ldk}, {ldv, wk, &io->ldv}});
  if (rc != GDN_OK) return rc;
  io->q = q; io->k = k; io->v = v; io->cu_q = cu_q; io->cu_k = cu_k;
  io->T_q = T_q; io->T_k = T_k; io->N = N; io->H_q = s->H_q; io->H_kv = s->H_kv; io->G = s->H_q / s->H_kv;
  io->c = s->scale * kLog2e;
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_attn_prefill(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_q, const int32_t* cu_k,
                     int64_t T_q, int64_t T_k, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                     int64_t ldv, void* o, int64_t ldo, float* lse, void* stream) {
  AttnIO io{};
  int rc = attn_common(shape, n_seqs, cu_q, cu_k, T_q, T_k, q, ldq, k, ldk, v, ldv, &io);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({o, lse}) || (T_q > 0 && !o)) return GDN_ERR_INVALID_ARG;
  rc = gdn::attn_rows({{ldo, static_cast<int64_t>(shape->H_q) * shape->d, &io.ldo}});
  if (rc != GDN_OK) return rc;
  if (T_q == 0) return GDN_OK;
  io.o = o; io.lse = lse;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return attn_dispatch(shape, [&]<typename T, int D>() {
    using Tile = FwdTile<T, D>;
    const int64_t blocks = tile_slots(T_q, n_seqs, Tile::BM) * io.H_q;
    if (blocks * Tile::NW * 64 >= gdn::kLaunchThreads) return static_cast<int>(GDN_ERR_UNSUPPORTED);
    Timed t_("k_attn_fwd", st);
    hipLaunchKernelGGL((k_attn_fwd<T, D>), dim3(static_cast<unsigned>(blocks)), dim3(Tile::NW * 64), 0, st, io);
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}

size_t gdn_attn_workspace_bytes(const gdn_attn_shape_t* shape, int64_t T_q, int64_t T_k) {
  if (gdn::check_attn_shape(shape) != GDN_OK || T_q < 0 || T_k < 0 || T_q > INT32_MAX || T_k > INT32_MAX) return 0;
  const size_t bytes = static_cast<size_t>(T_q) * shape->H_q * 2 * sizeof(float);
  return (bytes + gdn::kAlign) / gdn::kAlign * gdn::kAlign;
}

int gdn_attn_bwd(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_q, const int32_t* cu_k, int64_t T_q,
                 int64_t T_k, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                 const void* o, int64_t ldo, const float* lse, const void* dO, int64_t lddo, void* dq, int64_t lddq,
                 void* dk, int64_t lddk, void* dv, int64_t lddv, void* ws, size_t ws_bytes, void* stream) {
  GradIO g{};
  int rc = attn_common(shape, n_seqs, cu_q, cu_k, T_q, T_k, q, ldq, k, ldk, v, ldv, &g.a);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({o, lse, dO, dq, dk, dv, ws})) return GDN_ERR_INVALID_ARG;
  if ((T_q > 0 && (!o || !lse || !dO || !dq)) || (T_k > 0 && (!dk || !dv))) return GDN_ERR_INVALID_ARG;
  const int64_t wq = static_cast<int64_t>(shape->H_q) * shape->d, wk = static_cast<int64_t>(shape->H_kv) * shape->d;
  rc = gdn::attn_rows({{ldo, wq, &g.a.ldo}, {lddo, wq, &g.lddo}, {lddq, wq, &g.lddq}, {lddk, wk, &g.lddk}, {lddv, wk, &g.lddv}});
  if (rc != GDN_OK) return rc;
  if (!ws || ws_bytes < gdn_attn_workspace_bytes(shape, T_q, T_k)) return GDN_ERR_WORKSPACE;
  if (n_seqs == 0) return GDN_OK;
  g.a.o = const_cast<void*>(o); g.a.lse = const_cast<float*>(lse);
  g.dO = dO; g.dq = dq; g.dk = dk; g.dv = dv;
  g.stat = static_cast<float*>(ws);
  g.scale = shape->scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return attn_dispatch(shape, [&]<typename T, int D>() {
    const int64_t nq = tile_slots(T_q, n_seqs, 128) * g.a.H_q, nk = tile_slots(T_k, n_seqs, 128) * g.a.H_kv;
    if (nq * 256 >= gdn::kLaunchThreads || nk * 256 >= gdn::kLaunchThreads) return static_cast<int>(GDN_ERR_UNSUPPORTED);
    if (T_q > 0) {
      Timed t_("k_attn_dq", st);
      hipLaunchKernelGGL((k_attn_dq<T, D>), dim3(static_cast<unsigned>(nq)), dim3(256), 0, st, g);
    }
    if (T_k > 0) {
      Timed t_("k_attn_dkv", st);
      launch_dkv<T, D>(g, static_cast<unsigned>(nk), st);
    }
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}

}  // extern "C"
