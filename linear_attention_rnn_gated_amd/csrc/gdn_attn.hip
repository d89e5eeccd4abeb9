// Causal attention over packed sequences with grouped heads (include/gdn.h):
// kernels and C ABI.
#include "gdn_attn_walk.h"

#include <type_traits>

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

// The query rows of a block: 32 for each wave.
struct QueryTile {
  Span sp;
  int hk, hq;
  int r0, row;  // the wave's first row, the lane's
  int rows;     // of the wave that there are (0 or fewer: none)
  int last;     // the last token that the block's rows see
  AttnRows at;
};
template <int BM>
__device__ __forceinline__ bool query_tile(const AttnIO& io, int wave, int lane, QueryTile* x) {
  x->hk = blockIdx.x % io.H_kv;
  const int y = blockIdx.x / io.H_kv;
  x->hq = x->hk * io.G + y % io.G;
  int tile;
  const int n = tile_seq(io.cu_q, io.N, BM, y / io.G, &tile);
  const Span sp = x->sp = span_of(io.cu_q, io.cu_k, io.T_q, io.T_k, n);
  const int tiles = (sp.Lq + BM - 1) / BM;
  if (tile < 0 || tile >= tiles) return false;
  tile = tiles - 1 - tile;  // the longest first
  const int off = sp.Lk - sp.Lq;  // row i sees keys up to i + off
  x->r0 = tile * BM + wave * 32;
  x->row = x->r0 + (lane & 31);
  x->rows = sp.Lq - x->r0 < 32 ? sp.Lq - x->r0 : 32;
  x->last = ((tile + 1) * BM < sp.Lq ? (tile + 1) * BM - 1 : sp.Lq - 1) + off;
  x->at.lim = x->row < sp.Lq ? x->row + off : -1;
  x->at.lo = x->r0 + off;
  x->at.hi = x->rows > 0 ? x->r0 + x->rows - 1 + off : -1;
  x->at.block_lo = tile * BM + off;
  return true;
}

// Keys and values of one head as rows in memory, from tile `first` on every NG-th.
template <typename T, int D, int BN, int NW, int NG>
struct RowStage {
  using Move = Stager<T, D, BN, NW>;
  static constexpr bool DIRECT = sizeof(T) == 2, GAPS = false;
  static constexpr int LOADS = Move::STEPS;
  RowTiles<T, D, BN, NG> tk, tv;
  Move sk, sv;
  __device__ __forceinline__ RowStage(const AttnIO& io, const Span& sp, int hk, int first, int wave, int lane)
      : tk(io.k, sp.k0 + first * BN, io.ldk, hk, sp.Lk - first * BN), tv(io.v, sp.k0 + first * BN, io.ldv, hk, sp.Lk - first * BN),
        sk(io.ldk, wave, lane), sv(io.ldv, wave, lane) {}
  __device__ __forceinline__ void next_k() { tk.next(); }
  __device__ __forceinline__ void next_v() { tv.next(); }
  __device__ __forceinline__ void load_k(int i, char* kb) { sk.load(i, tk.rsrc, kb); }
  __device__ __forceinline__ void load_v(int i, char* vb) { sv.load(i, tv.rsrc, vb); }
  __device__ __forceinline__ void finish_k(char* kb) const { sk.finish(kb); }
  __device__ __forceinline__ void finish_v(char* vb) const { sv.finish(vb); }
  __device__ __forceinline__ void load(char* kb, char* vb) {  // the next tile of both
    next_k();
    next_v();
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      load_k(i, kb);
      load_v(i, vb);
    }
  }
};

template <typename T, int D>
__device__ __forceinline__ void load_rows(const void* x, int64_t at, int64_t ld, int h, int rows, int lane,
                                          Held<T, D> (&y)[D / 16]) {
  const brsrc_t r = rows_rsrc<T, D>(x, at, ld, h, rows);
  const uint32_t col = static_cast<uint32_t>((lane & 31) * ld * sizeof(T)) + 8 * (lane >> 5) * sizeof(T);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) y[ks].load(r, col + 16 * ks * sizeof(T));
}

// 128 rows a block: a tile of keys and values is read from L2 once for them (8x4096,
// 32 and 8 heads: 454 MB from memory where q, k and v have 403).  One prompt of 128
// tokens, 16 heads of 256, is 16 blocks: 16 us, the launch and four steps' latencies.
template <typename T, int D>
__global__ __launch_bounds__((256 * kAttnGroups<T, D>), (kAttnOcc<T, D>)) void k_attn_fwd(AttnIO io) {
#ifdef GDN_DEVICE_PASS
  constexpr int NG = kAttnGroups<T, D>;
  __shared__ int odd[D + 1];
  const int lane = threadIdx.x & 63, grp = NG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6 & 3);
  QueryTile x;
  if (!query_tile<kAttnRows>(io, wave, lane, &x)) return;
  Held<T, D> q[D / 16];
  load_rows<T, D>(io.q, x.sp.q0 + (x.rows > 0 ? x.r0 : 0), io.ldq, x.hq, x.rows, lane, q);
  RowStage<T, D, kAttnStep, kAttnWaves, NG> st(io, x.sp, x.hk, grp, wave, lane);
  AttnState<D> a;
  const int steps = x.last >= 0 ? x.last / kAttnStep + 1 : 0;
  attn_walk<T, T, D, kAttnWaves, NG>(st, grp, q, 0, steps, x.at, io.c, lane, odd, a);
  if (grp == 0 && x.row < x.sp.Lq) {
    store_row<D>(static_cast<T*>(io.o) + (x.sp.q0 + x.row) * io.ldo + static_cast<int64_t>(x.hq) * D, a.acc, inverse_sum(a.l), lane);
    if (io.lse && lane < 32) io.lse[(x.sp.q0 + x.row) * io.H_q + x.hq] = lse_of(a.m * io.c, a.l);
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
// right operands of dV^T = dO^T P and dK^T = Q^T dS as they stand.  S and dP are thus
// formed twice (seven products where five would do), which is cheaper than adding dq
// up in memory and keeps its order.
//
// 8x4096 tokens, 32 and 8 heads of 128, bf16: dq 1.97 ms (four products, 1120 TFLOP/s),
// dkv 2.5 ms (four, 880 TFLOP/s), bound by the matrix cores.
//
// What bf16 rows lose.  p goes into dv and dS into dk rounded to bf16, 2^-8 of each; in
// two parts both, dkv takes 3.3 ms.  dS goes into dq in two parts (in one, dq 1.58 ms).
// dO . o comes from an o that was rounded: of a row's dS, which sum to 0 but for that, dq
// takes the sum, and dk's dO . o is corrected by it at no cost; dq would need p K beside
// dS K, a product more.  Errors (norms; rounding the outputs alone is 1.66e-3), 8x4096
// tokens: dq 1.84e-3, dk 2.35e-3, dv 2.3e-3 (with dS in one part and o as given 2.52e-3,
// 2.44e-3); sequences of 16: 2.4e-3, 2.3e-3, 2.2e-3 (2.9e-3, 2.9e-3).  fp32 rows'
// operands are all taken in three parts.
struct GradIO {
  AttnIO a;  // o: the forward's output, read
  const void* dO;
  void* dq;
  void* dk;
  void* dv;
  float* stat;  // [H_q][T_q][2]: lse log2(e) and dO . o, for dk and dv
  float* part;  // [parts][2][T_k][H_kv][D] fp32 sums for dk and dv, where parts > 1
  float* qpart;  // [qcuts][T_q][H_q][D] fp32 sums for dq, where qcuts > 1
  float* gaps;   // [qcuts][H_q][T_q] sums of dS, likewise and of bf16 rows
  int qcuts;    // parts that the keys of a query tile are cut into
  int cuts;     // that the queries of a head are cut into
  int parts;    // that a group's heads and their queries are cut into
  int64_t lddo, lddq, lddk, lddv;
  float scale;
};

template <typename T, int D>
__global__ __launch_bounds__((256 * kAttnGroups<T, D>), (kAttnOcc<T, D>)) void k_attn_dq(GradIO g) {
#ifdef GDN_DEVICE_PASS
  constexpr int BN = 32, NW = 4, NG = kAttnGroups<T, D>, KS = D / 16, ND = D / 32;
  using P = Plane<T, D, BN>;
  constexpr bool SHORT = sizeof(T) == 2;  // o has lost bits of dO . o
  static_assert(!SHORT || NG == 1);
  constexpr bool TWO = 4 * P::TILE <= 144 * 1024;
  constexpr int SB = TWO ? P::TILE : 16;
  __shared__ __align__(1024) char kA_[NG * P::TILE], vA_[NG * P::TILE], kB_[NG * SB], vB_[NG * SB];
  const AttnIO& io = g.a;
  const int lane = threadIdx.x & 63, grp = NG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6 & 3);
  char *kA = kA_ + grp * P::TILE, *vA = vA_ + grp * P::TILE, *kB = kB_ + grp * SB, *vB = vB_ + grp * SB;
  QueryTile x;
  if (!query_tile<32 * NW>(io, wave, lane, &x)) return;
  const int64_t at = x.sp.q0 + (x.rows > 0 ? x.r0 : 0);
  Held<T, D> q[KS], dO[KS];
  load_rows<T, D>(io.q, at, io.ldq, x.hq, x.rows, lane, q);
  load_rows<T, D>(g.dO, at, g.lddo, x.hq, x.rows, lane, dO);
  float lse2, dot = 0.0f;
  {
    const brsrc_t rd = rows_rsrc<T, D>(g.dO, at, g.lddo, x.hq, x.rows);
    const brsrc_t ro = rows_rsrc<T, D>(io.o, at, io.ldo, x.hq, x.rows);
    const uint32_t col = 8 * (lane >> 5) * sizeof(T), r = lane & 31;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      dot = dot8<T>(rd, static_cast<uint32_t>(r * g.lddo * sizeof(T)) + col + 16 * ks * sizeof(T), ro,
                    static_cast<uint32_t>(r * io.ldo * sizeof(T)) + col + 16 * ks * sizeof(T), dot);
    dot += other_half(dot);
    lse2 = x.row < x.sp.Lq ? io.lse[(x.sp.q0 + x.row) * io.H_q + x.hq] * kLog2e : 0.0f;
  }
  float gap = 0.0f;  // sum of dS
  const int all = x.last >= 0 ? x.last / (NG * BN) + 1 : 0, each = (all + g.qcuts - 1) / g.qcuts;
  const int begin = blockIdx.y * each, end = begin + each < all ? begin + each : all;
  RowStage<T, D, BN, NW, NG> st(io, x.sp, x.hk, begin * NG + grp, wave, lane);
  v16f acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = zero16();
  auto step = [&](char* kb, char* vb, char* kn, char* vn, int j) {
    if constexpr (st.DIRECT) wait_loads();
    __syncthreads();
    st.load(kn, vn);
    const int j0 = (j * NG + grp) * BN;
    if (j0 <= x.at.hi) {
      v16f s = zero16(), dp = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        s = mma32(row_frag<T, D, BN>(kb, 0, ks, lane), q[ks].get(), s);
        dp = mma32(row_frag<T, D, BN>(vb, 0, ks, lane), dO[ks].get(), dp);
      }
      const bool edge = j0 + BN - 1 > x.at.lo;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[i], io.c, -lse2));
        s[i] = p * (dp[i] - dot);
        if (edge && j0 + c_row(i, lane) > x.at.lim) s[i] = 0.0f;
        if constexpr (SHORT) gap += s[i];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        std::conditional_t<SHORT, TwoParts, Frag<T>> ds;
        ds.pack(s, 8 * u);
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = mma32(col_frag<T, D, BN>(kb, 16 * u, d, lane), ds, acc[d]);
      }
    }
    if constexpr (!st.DIRECT) {
      if constexpr (!TWO) __syncthreads();
      st.finish_k(kn);
      st.finish_v(vn);
    }
  };
  auto keep = [&] {
    if constexpr (sizeof(T) == 4 || D == 256) {
#pragma unroll
      for (int d = 0; d < ND; ++d) in_agprs(acc[d]);
    }
  };
  if (begin < end) {
    st.load(kA, vA);
    if constexpr (!st.DIRECT) {
      st.finish_k(kA);
      st.finish_v(vA);
    }
  }
  if constexpr (TWO) {
    for (int j = begin; j < end; j += 2) {
      step(kA, vA, kB, vB, j);
      if (j + 1 < end) step(kB, vB, kA, vA, j + 1);
      keep();
    }
  } else {
    for (int j = begin; j < end; ++j) {
      step(kA, vA, kA, vA, j);
      keep();
    }
  }
  wait_loads();
  if constexpr (NG == 2) {  // both groups' sums, half in kA_ and half in vA_
    static_assert(NG * P::TILE >= D * NW * 64);
    constexpr int H = D / 4;
    const int at = threadIdx.x & 255;
    float *s0 = reinterpret_cast<float*>(kA_) + at, *s1 = reinterpret_cast<float*>(vA_) + at;
    __syncthreads();
    if (grp == 1) {
#pragma unroll
      for (int i = 0; i < 2 * H; ++i) (i < H ? s0 + i * 256 : s1 + (i - H) * 256)[0] = acc[i / 16][i % 16];
    }
    __syncthreads();
    if (grp == 1) return;
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) acc[i / 16][i % 16] += (i < H ? s0 + i * 256 : s1 + (i - H) * 256)[0];
  }
  if constexpr (SHORT) gap += other_half(gap);
  if (x.row < x.sp.Lq) {
    const int64_t row = x.sp.q0 + x.row;
    if (lane < 32) {
      const int64_t i = static_cast<int64_t>(x.hq) * io.T_q + row;
      if (SHORT && g.qcuts > 1) g.gaps[blockIdx.y * (io.H_q * io.T_q) + i] = gap;
      if (blockIdx.y == 0) {
        g.stat[2 * i] = lse2;
        g.stat[2 * i + 1] = SHORT && g.qcuts == 1 ? dot + gap : dot;
      }
    }
    if (g.qcuts == 1)
      store_row<D>(static_cast<T*>(g.dq) + row * g.lddq + static_cast<int64_t>(x.hq) * D, acc, g.scale, lane);
    else
      store_row<D>(g.qpart + ((blockIdx.y * io.T_q + row) * io.H_q + x.hq) * D, acc, g.scale, lane);
  }
#endif
}

// dO . o of bf16 rows from what dS of the parts of k_attn_dq sums to, in order.
__global__ __launch_bounds__(256) void k_attn_stat(float* stat, const float* gaps, int64_t rows, int parts) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= rows) return;
  float gap = 0.0f;
  for (int c = 0; c < parts; ++c) gap += gaps[c * rows + i];
  stat[2 * i + 1] += gap;
}

// The keys of a block of k_attn_dkv, 32 for each wave, and the query tiles of BQ
// rows that it goes over: those of each of its heads from the first that sees one
// of the keys on.
struct KeyTile {
  Span sp;
  int hk, h0, h1;   // key/value head, query heads
  int j0, key;      // the wave's first key, the lane's
  int off;          // query i sees keys up to i + off
  int first, per;   // first query tile, tiles a head
};

// WHAT: 3 both gradients, 1 dk, 2 dv (heads of 256, whose two sums and operands
// together pass the registers of a wave: 4x4096 tokens, 16 and 2 heads, bf16: 2.84 ms
// in two, 14.8 in one; 4x1024, heads of 128, fp32: 388 us in two, 282 in one).
//
// One wave a SIMD (two gradients' sums and two operands take 192 of its registers
// at d = 128), so a wave has to hide its own latencies: the products S and dP of
// one tile of queries run while p and dS of the tile before are formed.
template <typename T, int D, int WHAT>
__global__ __launch_bounds__(256, 1) void k_attn_dkv(GradIO g) {
#ifdef GDN_DEVICE_PASS
  constexpr int BQ = 32, NW = 4, BK = 32 * NW, KS = D / 16, ND = D / 32;
  constexpr bool DK = WHAT & 1, DV = WHAT & 2;
  using P = Plane<T, D, BQ>;
  constexpr int BUFS = sizeof(T) == 2 ? 4 : 4 * P::TILE <= 144 * 1024 ? 2 : 1;
  constexpr int SB = BUFS > 1 ? P::TILE : 16, SC = BUFS > 2 ? P::TILE : 16;
  __shared__ __align__(1024) char qA[P::TILE], oA[P::TILE], qB[SB], oB[SB], qC[SC], oC[SC], qD[SC], oD[SC];
  __shared__ __align__(1024) float sA[2 * BQ], sB[2 * BQ], sC[2 * BQ], sD[2 * BQ];
  const AttnIO& io = g.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  KeyTile x;
  x.hk = blockIdx.x % io.H_kv;
  int tile;
  const int n = tile_seq(io.cu_k, io.N, BK, blockIdx.x / io.H_kv, &tile);
  x.sp = span_of(io.cu_q, io.cu_k, io.T_q, io.T_k, n);
  if (tile < 0 || tile * BK >= x.sp.Lk) return;
  const int heads = (io.G * g.cuts + g.parts - 1) / g.parts, cut = blockIdx.y % g.cuts;
  x.h0 = blockIdx.y / g.cuts * heads;
  x.h1 = x.h0 + heads < io.G ? x.h0 + heads : io.G;
  x.j0 = tile * BK + wave * 32;
  x.key = x.j0 + (lane & 31);
  x.off = x.sp.Lk - x.sp.Lq;
  x.first = tile * BK - x.off > 0 ? (tile * BK - x.off) / BQ : 0;
  x.per = (x.sp.Lq + BQ - 1) / BQ - x.first;
  if (g.cuts > 1) {
    const int each = x.per > 0 ? (x.per + g.cuts - 1) / g.cuts : 0;
    x.first += cut * each;
    x.per = x.per - cut * each < each ? x.per - cut * each : each;
  }
  const int steps = x.per > 0 && x.h1 > x.h0 ? x.per * (x.h1 - x.h0) : 0;

  Held<T, D> k[KS], v[DK ? KS : 1];
  {
    const int rows = x.sp.Lk - x.j0 < 32 ? x.sp.Lk - x.j0 : 32;
    const int64_t at = x.sp.k0 + (rows > 0 ? x.j0 : 0);
    load_rows<T, D>(io.k, at, io.ldk, x.hk, rows, lane, k);
    if constexpr (DK) load_rows<T, D>(io.v, at, io.ldv, x.hk, rows, lane, v);
  }
  Stager<T, D, BQ, NW> sq(io.ldq, wave, lane), so(g.lddo, wave, lane);
  int fh = x.hk * io.G + x.h0, ft = x.first;  // the next tile to fetch
  auto start = [&](char* qb, char* ob, float* sb) {
    const int i0 = ft * BQ, rows = x.sp.Lq - i0 < BQ ? x.sp.Lq - i0 : BQ;
    sq.start(rows_rsrc<T, D>(io.q, x.sp.q0 + i0, io.ldq, fh, rows), qb);
    so.start(rows_rsrc<T, D>(g.dO, x.sp.q0 + i0, g.lddo, fh, rows), ob);
    if (wave == 0) {
      float* st = g.stat + 2 * (static_cast<int64_t>(fh) * io.T_q + x.sp.q0 + i0);
      const brsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(st, static_cast<short>(0), rows * 8, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GDN_LDS void*)sb, 4, lane * 4, 0, 0, 0);
    }
    if (++ft == x.first + x.per) {
      ft = x.first;
      ++fh;
    }
  };
  v16f ak[DK ? ND : 1], av[DV ? ND : 1];
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    if constexpr (DK) ak[d] = zero16();
    if constexpr (DV) av[d] = zero16();
  }
  auto products = [&](const char* qb, const char* ob, v16f& s, v16f& dp) {
    s = zero16();
    dp = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      s = mma32(row_frag<T, D, BQ>(qb, 0, ks, lane), k[ks].get(), s);
      if constexpr (DK) dp = mma32(row_frag<T, D, BQ>(ob, 0, ks, lane), v[ks].get(), dp);
    }
  };
  int ct = x.first;  // the tile of the sums
  auto weights = [&](const float* sb, v16f& s, v16f& dp) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float* st = sb + 2 * (8 * a + 4 * (lane >> 5));
      const v4f s0 = *reinterpret_cast<const v4f*>(st), s1 = *reinterpret_cast<const v4f*>(st + 4);
      const float lse2[4] = {s0[0], s0[2], s1[0], s1[2]}, dot[4] = {s0[1], s0[3], s1[1], s1[3]};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i = 4 * a + b;
        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], io.c, -lse2[b]));
        dp[i] = s[i] * (dp[i] - dot[b]);
      }
    }
  };
  auto hide = [&](int i0, v16f& s, v16f& dp) {
    if (i0 + x.off < x.j0 + 31) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i0 + c_row(i, lane) + x.off < x.key) s[i] = dp[i] = 0.0f;
    }
  };
  auto sums = [&](const char* qb, const char* ob, const Frag<T> (&p)[2], const Frag<T> (&ds)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        if constexpr (DV) av[d] = mma32(col_frag<T, D, BQ>(ob, 16 * u, d, lane), p[u], av[d]);
        if constexpr (DK) ak[d] = mma32(col_frag<T, D, BQ>(qb, 16 * u, d, lane), ds[u], ak[d]);
      }
  };
  auto packed = [&](const v16f& s, const v16f& dp, Frag<T> (&p)[2], Frag<T> (&ds)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (DV) p[u].pack(s, 8 * u);
      if constexpr (DK) ds[u].pack(dp, 8 * u);
    }
  };
  auto keep = [&] {
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      if constexpr (DK) in_agprs(ak[d]);
      if constexpr (DV) in_agprs(av[d]);
    }
  };
  v16f s, dp;
  if constexpr (BUFS == 4) {
    // Step i: first half, the products of tile i + 1 beside p and dS of tile i; then
    // tile i + 2 has arrived and i + 3 sets out; second half, the sums of tile i.
    // The halves are laid out in slots of one product each, with the LDS reads
    // some slots (of 32 cycles) ahead of the products that take them (a read takes
    // some 100).
    constexpr int AHEAD = 4, M1 = KS * (DK ? 2 : 1), NF = ND * ((DK ? 1 : 0) + (DV ? 1 : 0));
    Frag<T> rf[M1];  // the products' left operands: of q, and between them of dO
    auto row_of = [&](const char* qb, const char* ob, int m) {
      return DK && m % 2 ? row_frag<T, D, BQ>(ob, 0, m / 2, lane) : row_frag<T, D, BQ>(qb, 0, DK ? m / 2 : m, lane);
    };
    auto col_of = [&](const char* qb, const char* ob, int u, int f) {
      if constexpr (DK && DV) return col_frag<T, D, BQ>(f % 2 ? qb : ob, 16 * u, f / 2, lane);
      return col_frag<T, D, BQ>(DK ? qb : ob, 16 * u, f, lane);
    };
    auto step = [&](char* q0, char* o0, float* s0, char* q1, char* o1, char* q2, char* o2, char* q3, char* o3, float* s3, int i) {
      const int i0 = ct * BQ;
      if (++ct == x.first + x.per) ct = x.first;
      v16f sn = zero16(), dpn = zero16();
      Frag<T> f0[NF], f1[NF], p[2], ds[2];
      v4f st[2][2];
      auto stat = [&](int a) {
        const float* at = s0 + 2 * (8 * a + 4 * (lane >> 5));
        st[a % 2][0] = *reinterpret_cast<const v4f*>(at);
        st[a % 2][1] = *reinterpret_cast<const v4f*>(at + 4);
      };
      stat(0);
#pragma unroll
      for (int m = 0; m < M1; ++m) {  // behind the last tile: of what the buffer held before, and unused
        __builtin_amdgcn_sched_barrier(0);
        if (m + AHEAD < M1) rf[m + AHEAD] = row_of(q1, o1, m + AHEAD);
#pragma unroll
        for (int f = m * NF / M1; f < (m + 1) * NF / M1; ++f) f0[f] = col_of(q0, o0, 0, f);
        if (DK && m % 2)
          dpn = mma32(rf[m], v[DK ? m / 2 : 0].get(), dpn);
        else
          sn = mma32(rf[m], k[DK ? m / 2 : m].get(), sn);
#pragma unroll
        for (int e = m * 16 / M1; e < (m + 1) * 16 / M1; ++e) {
          const int a = e / 4, b = e % 4;
          if (b == 0 && a < 3) stat(a + 1);
          s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], io.c, -st[a % 2][b / 2][2 * (b % 2)]));
          if constexpr (DK) dp[e] = s[e] * (dp[e] - st[a % 2][b / 2][2 * (b % 2) + 1]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      hide(i0, s, dp);
      wait_loads();
      __syncthreads();
      if (i + 3 < steps) start(q3, o3, s3);
      if constexpr (DV) p[0].pack(s, 0);
      if constexpr (DK) ds[0].pack(dp, 0);
#pragma unroll
      for (int m = 0; m < 2 * NF; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        if (m < NF) f1[m] = col_of(q0, o0, 1, m);
        if (m >= 2 * NF - AHEAD) rf[m - 2 * NF + AHEAD] = row_of(q2, o2, m - 2 * NF + AHEAD);
        if (m == NF / 2) {
          if constexpr (DV) p[1].pack(s, 8);
          if constexpr (DK) ds[1].pack(dp, 8);
        }
        const int u = m / NF, f = m % NF;
        const Frag<T>& left = u ? f1[f] : f0[f];
        if (DK && DV) {
          if (f % 2)
            ak[f / 2] = mma32(left, ds[u], ak[f / 2]);
          else
            av[f / 2] = mma32(left, p[u], av[f / 2]);
        } else if (DK) {
          ak[f] = mma32(left, ds[u], ak[f]);
        } else {
          av[f] = mma32(left, p[u], av[f]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      s = sn;
      dp = dpn;
    };
    if (steps > 0) {
      start(qA, oA, sA);
      if (steps > 1) start(qB, oB, sB);
      if (steps > 2) start(qC, oC, sC);
      wait_loads();
      __syncthreads();
      products(qA, oA, s, dp);
#pragma unroll
      for (int m = 0; m < AHEAD; ++m) rf[m] = row_of(qB, oB, m);
    }
    for (int i = 0; i < steps; i += 4) {
      step(qA, oA, sA, qB, oB, qC, oC, qD, oD, sD, i);
      if (i + 1 < steps) step(qB, oB, sB, qC, oC, qD, oD, qA, oA, sA, i + 1);
      if (i + 2 < steps) step(qC, oC, sC, qD, oD, qA, oA, qB, oB, sB, i + 2);
      if (i + 3 < steps) step(qD, oD, sD, qA, oA, qB, oB, qC, oC, sC, i + 3);
      keep();
    }
  } else {
    if (steps > 0) {
      start(qA, oA, sA);
      if constexpr (!sq.DIRECT) {
        sq.finish(qA);
        so.finish(oA);
      }
    }
    constexpr bool TWO = BUFS == 2;
    auto step = [&](char* qb, char* ob, float* sb, char* qn, char* on, float* sn, int i) {
      wait_loads();
      __syncthreads();
      const bool more = i + 1 < steps;
      if (more) start(qn, on, sn);
      products(qb, ob, s, dp);
      weights(sb, s, dp);
      hide(ct * BQ, s, dp);
      if (++ct == x.first + x.per) ct = x.first;
      Frag<T> p[2], ds[2];
      packed(s, dp, p, ds);
      sums(qb, ob, p, ds);
      if constexpr (!sq.DIRECT) {
        if constexpr (!TWO) __syncthreads();
        if (more) {
          sq.finish(qn);
          so.finish(on);
        }
      }
    };
    if constexpr (TWO) {
      for (int i = 0; i < steps; i += 2) {
        step(qA, oA, sA, qB, oB, sB, i);
        if (i + 1 < steps) step(qB, oB, sB, qA, oA, sA, i + 1);
        keep();
      }
    } else {
      for (int i = 0; i < steps; i += 2) {
        step(qA, oA, sA, qA, oA, sB, i);
        if (i + 1 < steps) step(qA, oA, sB, qA, oA, sA, i + 1);
        keep();
      }
    }
  }
  if (x.key < x.sp.Lk) {
    const int64_t row = x.sp.k0 + x.key;
    if (g.parts == 1) {
      if constexpr (DK) store_row<D>(static_cast<T*>(g.dk) + row * g.lddk + static_cast<int64_t>(x.hk) * D, ak, g.scale, lane);
      if constexpr (DV) store_row<D>(static_cast<T*>(g.dv) + row * g.lddv + static_cast<int64_t>(x.hk) * D, av, 1.0f, lane);
    } else {
      const int64_t size = io.T_k * io.H_kv * D;
      float* part = g.part + 2 * blockIdx.y * size + (row * io.H_kv + x.hk) * D;
      if constexpr (DK) store_row<D>(part, ak, g.scale, lane);
      if constexpr (DV) store_row<D>(part + size, av, 1.0f, lane);
    }
  }
#endif
}

// Gradients from the fp32 sums of their parts, added in order.
struct SumIO {
  const float* part;  // [parts][T][width], `between` elements from one to the next
  int64_t between, T, width, ld;
  const int32_t* cu;  // [N + 1]
  int parts, N;
  void* out;
};
struct SumsIO { SumIO of[3]; };
template <typename T>
__global__ __launch_bounds__(256) void k_attn_sum(SumsIO sums) {
  const SumIO& io = sums.of[blockIdx.y];
  const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  int64_t end = io.cu[io.N];
  end = end < 0 ? 0 : end > io.T ? io.T : end;
  if (e >= end * io.width) return;
  const int64_t row = e / io.width, col = e - row * io.width;
  v4f y = *reinterpret_cast<const v4f*>(io.part + e);
  for (int i = 1; i < io.parts; ++i) y += *reinterpret_cast<const v4f*>(io.part + i * io.between + e);
  const float z[4] = {y[0], y[1], y[2], y[3]};
  store4(static_cast<T*>(io.out) + row * io.ld + col, z);
}

// ---- host side ----------------------------------------------------------------

template <typename T, int D>
void launch_dkv(const GradIO& g, unsigned blocks, hipStream_t st) {
  constexpr bool split = D >= 256;
  const dim3 grid(blocks, g.parts);
  hipLaunchKernelGGL((k_attn_dkv<T, D, split ? 1 : 3>), grid, dim3(256), 0, st, g);
  if constexpr (split) hipLaunchKernelGGL((k_attn_dkv<T, D, 2>), grid, dim3(256), 0, st, g);
}

// Parts that a group's heads are cut into for dk and dv: more where the blocks of
// 128 keys, one a CU and the first of a sequence twice as long as the average,
// would not fill the chip evenly (4x4096, 16 and 2 heads of 256: 2.84 ms in four, 3.15
// in two); where that does not fill it either, the queries of a head as well (2048
// tokens, 4 heads of 128: 35 us + 7 for their sums in four, 68 in one; 4096 tokens, 4
// heads and 1: 90 + 14 in twelve, 120 + 28 in twenty-four, 132 + 6 in four).  For dq the
// keys of a query tile (4096 tokens, 4 heads, bf16: 131 us in one, 63 and 10 more for
// their sums in four).
struct DkvParts {
  int heads, cuts;
  int all() const { return heads * cuts; }
};
DkvParts dkv_parts(const gdn_attn_shape_t* s, int64_t T_k) {
  const int G = s->H_q / s->H_kv;
  const int64_t blocks = (T_k + 127) / 128 * s->H_kv;
  int parts = 1, cuts = 1;
  while (parts < G && blocks * parts < 1024) ++parts;
  const int heads = (G + parts - 1) / parts;
  parts = (G + heads - 1) / heads;  // none without a head
  while (cuts < T_k / 512 && blocks * parts * cuts < 512) ++cuts;
  return DkvParts{parts, cuts};
}
int dq_cuts(const gdn_attn_shape_t* s, int64_t T_q) {
  const int64_t blocks = (T_q + 127) / 128 * s->H_q;
  int cuts = 1;
  while (cuts < T_q / 512 && blocks * cuts < 512) ++cuts;
  return cuts;
}
size_t stat_bytes(const gdn_attn_shape_t* s, int64_t T_q) {
  const size_t bytes = static_cast<size_t>(T_q) * s->H_q * 2 * sizeof(float);
  return (bytes + gdn::kAlign) / gdn::kAlign * gdn::kAlign;
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
  if (!gdn::aligned16({q, k, v}) || !gdn::aligned4({cu_q, cu_k})) return GDN_ERR_INVALID_ARG;
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
  if (!gdn::aligned16({o}) || !gdn::aligned4({lse}) || (T_q > 0 && !o)) return GDN_ERR_INVALID_ARG;
  rc = gdn::attn_rows({{ldo, static_cast<int64_t>(shape->H_q) * shape->d, &io.ldo}});
  if (rc != GDN_OK) return rc;
  if (T_q == 0) return GDN_OK;
  io.o = o; io.lse = lse;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return attn_dispatch(shape, [&]<typename T, int D>() {
    const int64_t blocks = tile_slots(T_q, n_seqs, kAttnRows) * io.H_q;
    constexpr int threads = 256 * kAttnGroups<T, D>;
    if (blocks * threads >= gdn::kLaunchThreads) return static_cast<int>(GDN_ERR_UNSUPPORTED);
    Timed t_("k_attn_fwd", st);
    hipLaunchKernelGGL((k_attn_fwd<T, D>), dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, st, io);
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}

size_t gdn_attn_workspace_bytes(const gdn_attn_shape_t* shape, int64_t T_q, int64_t T_k) {
  if (gdn::check_attn_shape(shape) != GDN_OK || T_q < 0 || T_k < 0 || T_q > INT32_MAX || T_k > INT32_MAX) return 0;
  const int parts = dkv_parts(shape, T_k).all(), cuts = dq_cuts(shape, T_q);
  const size_t dkv = parts > 1 ? static_cast<size_t>(parts) * 2 * T_k * shape->H_kv : 0;
  const size_t dq = cuts > 1 ? static_cast<size_t>(cuts) * T_q * shape->H_q : 0;
  return stat_bytes(shape, T_q) + (((dkv + dq) * shape->d + dq) * sizeof(float) + gdn::kAlign - 1) / gdn::kAlign * gdn::kAlign;
}

int gdn_attn_bwd(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_q, const int32_t* cu_k, int64_t T_q,
                 int64_t T_k, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                 const void* o, int64_t ldo, const float* lse, const void* dO, int64_t lddo, void* dq, int64_t lddq,
                 void* dk, int64_t lddk, void* dv, int64_t lddv, void* ws, size_t ws_bytes, void* stream) {
  GradIO g{};
  int rc = attn_common(shape, n_seqs, cu_q, cu_k, T_q, T_k, q, ldq, k, ldk, v, ldv, &g.a);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({o, dO, dq, dk, dv, ws}) || !gdn::aligned4({lse})) return GDN_ERR_INVALID_ARG;
  if ((T_q > 0 && (!o || !lse || !dO || !dq)) || (T_k > 0 && (!dk || !dv))) return GDN_ERR_INVALID_ARG;
  const int64_t wq = static_cast<int64_t>(shape->H_q) * shape->d, wk = static_cast<int64_t>(shape->H_kv) * shape->d;
  rc = gdn::attn_rows({{ldo, wq, &g.a.ldo}, {lddo, wq, &g.lddo}, {lddq, wq, &g.lddq}, {lddk, wk, &g.lddk}, {lddv, wk, &g.lddv}});
  if (rc != GDN_OK) return rc;
  if (!ws || ws_bytes < gdn_attn_workspace_bytes(shape, T_q, T_k)) return GDN_ERR_WORKSPACE;
  if (n_seqs == 0) return GDN_OK;
  g.a.o = const_cast<void*>(o); g.a.lse = const_cast<float*>(lse);
  g.dO = dO; g.dq = dq; g.dk = dk; g.dv = dv;
  g.stat = static_cast<float*>(ws);
  const DkvParts cut = dkv_parts(shape, T_k);
  g.cuts = cut.cuts;
  g.parts = cut.all();
  g.part = g.stat + stat_bytes(shape, T_q) / sizeof(float);
  g.qcuts = dq_cuts(shape, T_q);
  g.qpart = g.part + (g.parts > 1 ? g.parts * 2 * T_k * wk : 0);
  g.gaps = g.qpart + (g.qcuts > 1 ? g.qcuts * T_q * wq : 0);
  g.scale = shape->scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return attn_dispatch(shape, [&]<typename T, int D>() {
    const int64_t nq = tile_slots(T_q, n_seqs, 128) * g.a.H_q, nk = tile_slots(T_k, n_seqs, 128) * g.a.H_kv;
    constexpr int threads = 256 * kAttnGroups<T, D>;
    if (nq * threads >= gdn::kLaunchThreads / g.qcuts || nk * 256 >= gdn::kLaunchThreads / g.parts) return static_cast<int>(GDN_ERR_UNSUPPORTED);
    if (T_q > 0) {
      Timed t_("k_attn_dq", st);
      hipLaunchKernelGGL((k_attn_dq<T, D>), dim3(static_cast<unsigned>(nq), g.qcuts), dim3(threads), 0, st, g);
    }
    if (sizeof(T) == 2 && g.qcuts > 1 && T_k > 0) {
      Timed t_("k_attn_stat", st);
      const int64_t rows = T_q * g.a.H_q;
      hipLaunchKernelGGL(k_attn_stat, dim3(static_cast<unsigned>((rows + 255) / 256)), dim3(256), 0, st, g.stat, g.gaps, rows, g.qcuts);
    }
    if (T_k > 0) {
      Timed t_("k_attn_dkv", st);
      launch_dkv<T, D>(g, static_cast<unsigned>(nk), st);
    }
    SumsIO sums{};
    int n = 0;
    if (T_k > 0 && g.parts > 1) {
      const int64_t size = T_k * wk;
      sums.of[n++] = SumIO{g.part, 2 * size, T_k, wk, g.lddk, g.a.cu_k, g.parts, n_seqs, dk};
      sums.of[n++] = SumIO{g.part + size, 2 * size, T_k, wk, g.lddv, g.a.cu_k, g.parts, n_seqs, dv};
    }
    if (g.qcuts > 1) sums.of[n++] = SumIO{g.qpart, T_q * wq, T_q, wq, g.lddq, g.a.cu_q, g.qcuts, n_seqs, dq};
    if (n > 0) {
      Timed t_("k_attn_sum", st);
      int64_t size = 0;  // the largest that there is; what is cut has under 2^17 rows times heads
      for (int i = 0; i < n; ++i) size = sums.of[i].T * sums.of[i].width > size ? sums.of[i].T * sums.of[i].width : size;
      hipLaunchKernelGGL(k_attn_sum<T>, dim3(static_cast<unsigned>((size / 4 + 255) / 256), n), dim3(256), 0, st, sums);
    }
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}

}  // extern "C"
