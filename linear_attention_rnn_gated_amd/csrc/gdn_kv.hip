// The 8-bit key/value cache and attention over it (include/gdn.h): kernels and
// C ABI.
#include "gdn_kv.h"

namespace {

using namespace gdn;

struct KvIO {
  uint8_t* kc;  // [pages, H_kv, P, D]
  uint8_t* vc;
  float* ks;    // [pages, H_kv, P / 32]
  float* vs;
  Pages pages;
  const int32_t* cu;     // [N + 1], nullptr: a token a sequence
  const int32_t* start;  // [N], nullable
  void* k;               // rows to write, or to read into
  void* v;
  int64_t T, ldk, ldv;
  int N, H_kv;
};

// The cache block that a workgroup takes, and the packed rows that it holds.
struct KvItem {
  int64_t row0;    // packed row of the block's place 0 (may lie before the sequence's first)
  int64_t blk;     // index of the block among [pages, H_kv, P / 32]
  int lo, hi;      // places of the call's tokens
  bool older;      // places before lo hold tokens
};
__device__ __forceinline__ bool kv_item(const KvIO& io, int h, KvItem* it) {
  const int x = blockIdx.x;
  int n, local;
  int64_t c0, c1;
  if (io.cu) {
    // sequence n's slots begin at cu[n] / 32 + 2 n: its tokens lie in at most two
    // blocks more than they fill
    int lo = 0, hi = io.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (io.cu[mid] / kBlk + 2 * mid <= x) lo = mid; else hi = mid - 1;
    }
    n = lo;
    local = x - (io.cu[n] / kBlk + 2 * n);
    c0 = io.cu[n];
    c1 = io.cu[n + 1];
    c0 = c0 < 0 ? 0 : c0 > io.T ? io.T : c0;
    c1 = c1 < c0 ? c0 : c1 > io.T ? io.T : c1;
  } else {
    n = x;
    local = 0;
    c0 = n;
    c1 = n + 1;
  }
  const int64_t first = io.start ? (io.start[n] > 0 ? io.start[n] : 0) : 0, end = first + (c1 - c0);
  const int64_t b = first / kBlk + local;
  // a sequence without tokens has no block, be its start in the middle of one: another
  // may be writing there
  if (local < 0 || end <= first || b * kBlk >= end || b >= (int64_t{1} << 30)) return false;
  it->blk = io.pages.block(n, io.H_kv, h, static_cast<uint32_t>(b));
  if (it->blk < 0) return false;
  it->lo = static_cast<int>(first > b * kBlk ? first - b * kBlk : 0);
  it->hi = static_cast<int>(end - b * kBlk < kBlk ? end - b * kBlk : kBlk);
  it->older = it->lo > 0;
  it->row0 = c0 + b * kBlk - first;
  return true;
}

// The least power of two s with most / s <= 448 = 1.75 2^8, at least 2^-117 (below
// it the codes' smallest step is no normal number).
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t u = __float_as_uint(most);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < 10 ? 10 : e;
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}
// Four codes of x / s; what is not finite becomes NaN.  At the largest scale,
// 2^120, codes over 240 would stand for more than fp32 holds.
__device__ __forceinline__ uint32_t codes4(const float* x, float inv, float cap) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool fin = fabsf(x[i]) < INFINITY;
    y[i] = fin ? fminf(fmaxf(x[i] * inv, -cap), cap) : __uint_as_float(0x7fc00000u);
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
  return static_cast<uint32_t>(w);
}

template <int E>
__device__ __forceinline__ void load_row(const float* p, float* x) {
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    const v4f y = *reinterpret_cast<const v4f*>(p + i);
    x[i] = y[0]; x[i + 1] = y[1]; x[i + 2] = y[2]; x[i + 3] = y[3];
  }
}
template <int E>
__device__ __forceinline__ void load_row(const bf16_t* p, float* x) {
#pragma unroll
  for (int i = 0; i < E; i += 8) {
    const u32x4 y = *reinterpret_cast<const u32x4*>(p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[i + 2 * e] = __uint_as_float(y[e] << 16);
      x[i + 2 * e + 1] = __uint_as_float(y[e] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void decode4(uint32_t c, float s, float* x) {
  x[0] = __builtin_amdgcn_cvt_f32_fp8(c, 0) * s;
  x[1] = __builtin_amdgcn_cvt_f32_fp8(c, 1) * s;
  x[2] = __builtin_amdgcn_cvt_f32_fp8(c, 2) * s;
  x[3] = __builtin_amdgcn_cvt_f32_fp8(c, 3) * s;
}

// A workgroup takes one block of one head, D / 8 lanes a token with eight elements
// each, so that both the codes (8 bytes a lane) and the rows (16 or 32) of
// neighbouring lanes lie side by side.  Bound by memory: 32 prompts of 128 to 8192
// tokens, 8 heads of 128, written in 187 us (924 MB, 4.9 TB/s, a copy's rate); 16
// prompts, 2 heads of 256, read in 39 us (228 MB, 5.8 TB/s).  One token of 64
// sequences: 4.7 us, its loads' latency, which the scale's sum over the block lengthens.
template <int D>
struct KvTile {
  static constexpr int LANES = D / 8, ROWS = 256 / LANES, PASSES = kBlk / ROWS;
};

template <typename T, int D>
__global__ __launch_bounds__(256) void k_kv_write(KvIO io) {
  using Tile = KvTile<D>;
  __shared__ float most[2][4];
  const int h = blockIdx.y;
  KvItem it;
  if (!kv_item(io, h, &it)) return;
  const int r0 = threadIdx.x / Tile::LANES, e0 = threadIdx.x % Tile::LANES * 8;
  float x[2][Tile::PASSES][8];
#pragma unroll
  for (int p = 0; p < Tile::PASSES; ++p) {
    const int r = r0 + p * Tile::ROWS;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[0][p][i] = x[1][p][i] = 0.0f;
    if (r >= it.lo && r < it.hi) {
      load_row<8>(static_cast<const T*>(io.k) + (it.row0 + r) * io.ldk + static_cast<int64_t>(h) * D + e0, x[0][p]);
      load_row<8>(static_cast<const T*>(io.v) + (it.row0 + r) * io.ldv + static_cast<int64_t>(h) * D + e0, x[1][p]);
    }
  }
  const float was[2] = {io.ks[it.blk], io.vs[it.blk]};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < Tile::PASSES; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[w][p][i]);
        m = fmaxf(m, a < INFINITY ? a : 0.0f);
      }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    if ((threadIdx.x & 63) == 0) most[w][threadIdx.x >> 6] = m;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float m = fmaxf(fmaxf(most[w][0], most[w][1]), fmaxf(most[w][2], most[w][3]));
    const float need = scale_for(m), s = it.older && was[w] > need ? was[w] : need;
    const float inv = 1.0f / s, cap = s > 0x1p119f ? 240.0f : 448.0f;
#pragma unroll
    for (int p = 0; p < Tile::PASSES; ++p) {
      const int r = r0 + p * Tile::ROWS;
      u32x2* at = reinterpret_cast<u32x2*>((w ? io.vc : io.kc) + (it.blk * kBlk + r) * D + e0);
      if (r >= it.lo && r < it.hi) {
        *at = u32x2{codes4(x[w][p], inv, cap), codes4(x[w][p] + 4, inv, cap)};
      } else if (r < it.lo && s != was[w]) {  // older tokens go over to the larger scale
        const u32x2 c = *at;
        float y[8];
        decode4(c[0], was[w], y);
        decode4(c[1], was[w], y + 4);
        *at = u32x2{codes4(y, inv, cap), codes4(y + 4, inv, cap)};
      }
    }
    if (threadIdx.x == 0) (w ? io.vs : io.ks)[it.blk] = s;
  }
}

template <typename T, int D>
__global__ __launch_bounds__(256) void k_kv_read(KvIO io) {
  using Tile = KvTile<D>;
  const int h = blockIdx.y;
  KvItem it;
  if (!kv_item(io, h, &it)) return;
  const int r0 = threadIdx.x / Tile::LANES, e0 = threadIdx.x % Tile::LANES * 8;
  const float s[2] = {io.ks[it.blk], io.vs[it.blk]};
  u32x2 c[2][Tile::PASSES];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int p = 0; p < Tile::PASSES; ++p)
      c[w][p] = *reinterpret_cast<const u32x2*>((w ? io.vc : io.kc) + (it.blk * kBlk + r0 + p * Tile::ROWS) * D + e0);
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int p = 0; p < Tile::PASSES; ++p) {
      const int r = r0 + p * Tile::ROWS;
      if (r < it.lo || r >= it.hi) continue;
      float y[8];
      decode4(c[w][p][0], s[w], y);
      decode4(c[w][p][1], s[w], y + 4);
      store8(static_cast<T*>(w ? io.v : io.k) + (it.row0 + r) * (w ? io.ldv : io.ldk) + static_cast<int64_t>(h) * D + e0, y);
    }
}

// ---- attention over the cache ---------------------------------------------------
//
// Rows are the query heads of a group for one token after another; a workgroup
// takes 16 MT of them for one key/value head and one split of the cache, its four
// waves every fourth block of 32 tokens.  Codes go from memory into registers and
// become bf16 there, exactly (the scale is a power of two): S^T = K Q^T on 16 x 16
// x 32 products leaves a row in the lanes l % 16, and O^T = V^T P^T takes exp(S^T)
// as it stands; the bytes of 4 tokens x 4 elements are transposed in registers.
//
// Bound by memory and the loads in flight: 64 sequences of 128 to 8192 tokens, 8 heads
// of 128: 113 us, 536 MB at 4.7 TB/s (products fill 11% of the cycles); one of 131071,
// 2 heads of 256: 31 us, 135 MB at 4.3 TB/s.  With its sums in the accumulation
// registers (the compiler's choice where it has one) 134 instead of 117 and 37 instead
// of 28, with splits of 512 tokens.
//
// q of bf16 rows goes in as it is and exp(s - m) in two bf16 parts, 2^-16 of each weight:
// products have room (64 sequences: 112 us in one part, 113.5 in two, 114 in three; one
// long: 30.5, 31.5, 32.5), and in one part outputs are 2.0e-3 to 2.2e-3 off (norms) where
// their own rounding is 1.65e-3 to 1.7e-3.  Of fp32 rows both go in in three.
typedef float v4acc __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4acc mma16(u32x4 a, u32x4 b, v4acc c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Eight fp32 values in NP bf16 parts that sum to them (exactly, with three).
template <int NP>
__device__ __forceinline__ void parts8(const float* x, u32x4* p) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t w = pack_bf16(a, b);
      p[i][e] = w;
      if (i + 1 < NP) {
        a -= __uint_as_float(w << 16);
        b -= __uint_as_float(w & 0xffff0000u);
      }
    }
  }
}
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// x of the lanes with the same l % 16: the largest, and the sum.
__device__ __forceinline__ float max_rows(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float sum_rows(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// A block of 32 tokens as loaded.  Keys: 16 bytes at 64 c + 16 (l / 16) of tokens
// 16 t + l % 16.  Values: D / 16 bytes at (D / 16) (l % 16) of tokens 16 t + 4 (l /
// 16) + i.
template <int D>
struct KvRegs {
  static constexpr int W = D / 64;  // dwords of values a token
  u32x4 k[2][D / 64];
  uint32_t v[2][4][W];
  float ks, vs;
  bool there;
  __device__ __forceinline__ void load(const DecIO& io, int64_t blk, int lane) {
    there = blk >= 0;
    if (!there) return;
    ks = io.ks[blk];
    vs = io.vs[blk];
    const uint8_t* kp = io.kc + blk * (kBlk * D) + (lane & 15) * D + (lane >> 4) * 16;
    const uint8_t* vp = io.vc + blk * (kBlk * D) + (lane >> 4) * 4 * D + (lane & 15) * (D / 16);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) k[t][c] = *reinterpret_cast<const u32x4*>(kp + t * 16 * D + c * 64);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(vp + (16 * t + i) * D);
        if constexpr (W == 1) v[t][i][0] = src[0];
        if constexpr (W == 2) {
          const u32x2 y = *reinterpret_cast<const u32x2*>(src);
          v[t][i][0] = y[0];
          v[t][i][1] = y[1];
        }
        if constexpr (W == 4) {
          const u32x4 y = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[t][i][e] = y[e];
        }
      }
    }
  }
  // 4 tokens x 4 elements, tokens within a dword afterwards
  __device__ __forceinline__ void transpose() {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t a = v[t][0][w], b = v[t][1][w], c = v[t][2][w], d = v[t][3][w];
        const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
        const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
        v[t][0][w] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
        v[t][1][w] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
        v[t][2][w] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100u);
        v[t][3][w] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302u);
      }
  }
};

template <typename T, int D>
__global__ __launch_bounds__(256) void k_attn_decode(DecIO io) {
#ifdef GDN_DEVICE_PASS
  constexpr int NP = sizeof(T) == 2 ? 1 : 3, PP = sizeof(T) == 2 ? 2 : 3;  // parts of q and of the weights
  constexpr int KC = D / 32, ND = D / 16, W = D / 64;
  constexpr int PAD = D + 4;
  __shared__ __align__(16) float sh_o[4][16][PAD];
  __shared__ float sh_m[4][16], sh_l[4][16];
  // Values that some row must not see, where they are NaN (0 x NaN would take them
  // to it), count as 0, and odd[e] is the first token whose element e is one
  // (odd[D] the first of all): a row that sees that token gets NaN in the end.
  __shared__ int odd[D + 1];
  const int hk = blockIdx.x % io.H_kv;
  const int x = blockIdx.x / io.H_kv;
  const int per = narrow_tiles(io.cu != nullptr, io.G), n = x / per, tile = x - n * per;
  const DecSeq sq = dec_seq(io, n);
  const int64_t r0 = static_cast<int64_t>(tile) * 16;
  const int split = io.split0 + blockIdx.y;
  if (r0 >= sq.rows || split >= sq.splits || sq.rows >= kWideRows) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4;

  // queries: steps 2 c and 2 c + 1 hold elements 64 c + 16 g + j and + 8 + j
  u32x4 q[KC][NP];
  int lim;  // the last token that the row sees
  int lim_lo = INT32_MAX;
  {
    const int64_t r = r0 + (lane & 15);
    const bool in = r < sq.rows;
    const int64_t tok = in ? r / io.G : 0;
    const int head = hk * io.G + static_cast<int>(in ? r - tok * io.G : 0);
    lim = in ? sq.sees(tok) : -1;
    if (in && lim < lim_lo) lim_lo = lim;
    const T* src = static_cast<const T*>(io.q) + (sq.q0 + tok) * io.ldq + static_cast<int64_t>(head) * D + 16 * g;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      if constexpr (NP == 1) {
        q[k][0] = in ? *reinterpret_cast<const u32x4*>(src + 64 * (k / 2) + 8 * (k % 2)) : u32x4{0, 0, 0, 0};
      } else {
        float y[8];
        load_row<8>(reinterpret_cast<const float*>(src) + 64 * (k / 2) + 8 * (k % 2), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = in ? y[e] : 0.0f;
        parts8<NP>(y, q[k]);
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) lim_lo = min(lim_lo, __shfl_xor(lim_lo, m, 64));
  lim_lo = __builtin_amdgcn_readfirstlane(lim_lo);
  const int64_t lastrow = (r0 + 16 < sq.rows ? r0 + 16 : sq.rows) - 1;
  const int lim_hi = sq.sees(lastrow / io.G);

  const int64_t t0 = sq.split * split, t1 = t0 + sq.split < lim_hi + 1 ? t0 + sq.split : lim_hi + 1;
  const int b1 = static_cast<int>((t1 + kBlk - 1) / kBlk);
  v4acc acc[ND];
  float m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = v4acc{0, 0, 0, 0};
  for (int e = threadIdx.x; e < D + 1; e += 256) odd[e] = INT32_MAX;
  __syncthreads();
  KvRegs<D> cur, nxt;
  int b = static_cast<int>(t0 / kBlk) + wave;
  if (b < b1) cur.load(io, io.pages.block(n, io.H_kv, hk, b), lane);
  // the page is looked up a step before its block is loaded
  int64_t blk = b + 4 < b1 ? io.pages.block(n, io.H_kv, hk, b + 4) : -1;
  for (; b < b1; b += 4) {
    if (b + 4 < b1) nxt.load(io, blk, lane);
    if (b + 8 < b1) blk = io.pages.block(n, io.H_kv, hk, b + 8);
    if (cur.there) {
      const int j0 = b * kBlk;
      const bool edge = j0 + kBlk - 1 > lim_lo;
      v4acc s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t] = v4acc{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const u32x4 a = codes8(cur.k[t][k / 2][2 * (k % 2)], cur.k[t][k / 2][2 * (k % 2) + 1], cur.ks);
#pragma unroll
          for (int i = NP - 1; i >= 0; --i) s[t] = mma16(a, q[k][i], s[t]);
        }
      }
      u32x4 p[PP];
      {
        float y[8];
        float top = m;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = s[e / 4][e % 4] * io.c;
          if (edge && j0 + 16 * (e / 4) + 4 * g + e % 4 > lim) y[e] = -INFINITY;
          top = fmaxf(top, y[e]);
        }
        top = max_rows(top);
        if (__any(top > m)) {
          const float f = top > m ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
          m = top;
          l *= f;
#pragma unroll
          for (int d = 0; d < ND; ++d) acc[d] *= f;
        }
        const float mm = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = __builtin_amdgcn_exp2f(y[e] - mm);
          l += y[e];
        }
        parts8<PP>(y, p);
      }
      if (edge) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = j0 + 16 * t + 4 * g + i;
#pragma unroll
            for (int w = 0; w < W; ++w) {
              uint32_t y = tok < sq.Lk ? cur.v[t][i][w] : 0u;  // nothing stands behind the last token
              const uint32_t bad = nan_bytes(y);
              if (bad) {
                y &= ~((bad >> 7) * 0xffu);
#pragma unroll 1
                for (int e = 0; e < 4; ++e)
                  if (bad >> (8 * e) & 0x80u) {
                    atomicMin(&odd[(D / 16) * (lane & 15) + 4 * w + e], tok);
                    atomicMin(&odd[D], tok);
                  }
              }
              cur.v[t][i][w] = y;
            }
          }
      }
      cur.transpose();
#pragma unroll
      for (int d = 0; d < ND; ++d) {  // row l % 16 of tile d is element (D / 16) (l % 16) + d
        const u32x4 a = codes8(cur.v[0][d % 4][d / 4], cur.v[1][d % 4][d / 4], cur.vs);
#pragma unroll
        for (int i = PP - 1; i >= 0; --i) acc[d] = mma16(a, p[i], acc[d]);
      }
    }
    cur = nxt;
  }

  // the waves' results, joined in their order
  {
    const int row = lane & 15;
    const float lw = sum_rows(l);
    if (lane < 16) {
      sh_m[wave][row] = m;
      sh_l[wave][row] = lw;
    }
    // lane (row, g) holds elements (D / 16) (4 g + i) + d
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int d = 0; d < ND; d += 4) {
        const v4f y{acc[d][i], acc[d + 1][i], acc[d + 2][i], acc[d + 3][i]};
        *reinterpret_cast<v4f*>(&sh_o[wave][row][(D / 16) * (4 * g + i) + d]) = y;
      }
    __syncthreads();
    // 16 threads a row, D / 16 elements each
    const int rr = threadIdx.x >> 4, e0 = (threadIdx.x & 15) * 4;
    const int64_t r = r0 + rr;
    if (r < sq.rows) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, sh_m[w][rr]);
      float f[4], sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = sh_m[w][rr] == top && top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sh_m[w][rr] - top);
        sum += sh_l[w][rr] * f[w];
      }
      const int64_t tok = r / io.G;
      const int head = hk * io.G + static_cast<int>(r - tok * io.G);
      const bool whole = sq.splits == 1;
      const float inv = !whole ? 1.0f : sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
      const int64_t pr = (sq.q0 * io.G * io.mul + n * io.extra + r * sq.splits + split) * io.H_kv + hk;
#pragma unroll
      for (int e = e0; e < D; e += 64) {
        float y[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const v4f z = *reinterpret_cast<const v4f*>(&sh_o[w][rr][e]);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = fmaf(z[i], f[w], y[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= inv;
        if (odd[D] != INT32_MAX) {
          const int sees = sq.sees(tok);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (sees >= odd[e + i]) y[i] = NAN;
        }
        if (whole)
          store4(static_cast<T*>(io.o) + (sq.q0 + tok) * io.ldo + static_cast<int64_t>(head) * D + e, y);
        else
          store4(io.part + pr * D + e, y);
      }
      if (e0 == 0) {
        if (!whole) {
          io.stat[2 * pr] = top;
          io.stat[2 * pr + 1] = sum;
        } else if (io.lse) {
          io.lse[(sq.q0 + tok) * io.H_q + head] = sum > 0.0f ? (top + __log2f(sum)) * kLn2 : sum != sum ? sum : -INFINITY;
        }
      }
    }
  }
#endif
}

// Joins the splits of a row: sixteen sums, of the splits i, i + 16, ..., each in
// order, then those in order.  GROUPS 16: a block a row, D / 4 lanes for each of
// the sums; GROUPS 1, for up to sixteen splits: D / 4 lanes a row, which gives the
// same bits (products and sums are rounded apart).  Latency: 7.6 us for 16 rows of 128
// splits, 6.6 for 2048 rows of up to 8.
constexpr int kJoin = 16;
template <typename T, int D, int GROUPS>
__global__ __launch_bounds__(GROUPS == 1 ? 256 : D / 4 * kJoin) void k_attn_join(DecIO io) {
  constexpr int LANES = D / 4, PER = GROUPS == 1 ? 256 / LANES : 1;  // rows a block
  __shared__ __align__(16) float sh_y[GROUPS == 1 ? 1 : kJoin][D];
  __shared__ float sh_s[kJoin];
  const int e = threadIdx.x % LANES * 4, group = GROUPS == 1 ? 0 : threadIdx.x / LANES;
  const int64_t item = io.item0 + static_cast<int64_t>(blockIdx.x) * PER + (GROUPS == 1 ? threadIdx.x / LANES : 0);
  const int64_t tk = item / io.H_q;
  const int head = static_cast<int>(item - tk * io.H_q);
  if (tk >= io.T) return;
  int n = static_cast<int>(tk);
  if (io.cu) {
    if (tk >= io.cu[io.N]) return;
    n = find_seq(io.cu, io.N, tk);
  }
  const DecSeq sq = dec_seq(io, n);
  if (sq.splits <= 1 || tk < sq.q0 || tk >= sq.q0 + sq.Lq) return;
  const int hk = head / io.G;
  const int64_t r = (tk - sq.q0) * io.G + head - hk * io.G;
  const int64_t p0 = sq.q0 * io.G * io.mul + n * io.extra + r * sq.splits;
  const float* part = io.part + (p0 * io.H_kv + hk) * D + e;
  const float* stat = io.stat + 2 * (p0 * io.H_kv + hk);
  const int64_t dp = static_cast<int64_t>(io.H_kv) * D, ds = 2 * io.H_kv;
  // loads of U splits in flight; the first ones set out before the maximum is known
  constexpr int STEP = GROUPS == 1 ? 1 : kJoin, U = 4;
  v4f z[U];
  float m[U], l[U];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * STEP < sq.splits ? i0 + u * STEP : sq.splits - 1;
      z[u] = *reinterpret_cast<const v4f*>(part + i * dp);
      m[u] = stat[i * ds];
      l[u] = stat[i * ds + 1];
    }
  };
  load(group);
  float top = -INFINITY;
  for (int i = threadIdx.x % LANES; i < sq.splits; i += LANES) top = fmaxf(top, stat[i * ds]);
#pragma unroll
  for (int d = (LANES < 64 ? LANES : 64) / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  float sum = 0.0f;
  v4f y{0, 0, 0, 0};
  for (int i0 = group; i0 < sq.splits; i0 += U * STEP) {
    if (i0 != group) load(i0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * STEP >= sq.splits) break;
      const float f = m[u] == -INFINITY && top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[u] - top);
      sum += l[u] * f;
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] += z[u][x] * f;
    }
  }
  if constexpr (GROUPS > 1) {
    *reinterpret_cast<v4f*>(&sh_y[group][e]) = y;
    if (e == 0) sh_s[group] = sum;
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int g = 1; g < kJoin; ++g) {
      const v4f z = *reinterpret_cast<const v4f*>(&sh_y[g][e]);
      sum += sh_s[g];
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] += z[x];
    }
  }
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  const float out[4] = {y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv};
  store4(static_cast<T*>(io.o) + tk * io.ldo + static_cast<int64_t>(head) * D + e, out);
  if (io.lse && e == 0)
    io.lse[tk * io.H_q + head] = sum > 0.0f ? (top + __log2f(sum)) * kLn2 : sum != sum ? sum : -INFINITY;
}

// ---- host side ----------------------------------------------------------------

Pages make_pages(const gdn_kv_cache_t* c, const int32_t* table, int32_t width) {
  const uint32_t bpp = c->page_tokens / kBlk;
  return Pages{table, width, c->pages, bpp, bpp == 1 ? UINT32_MAX : static_cast<uint32_t>((uint64_t{1} << 32) / bpp)};
}

// Checks what kv_write and kv_read share and fills io.
int kv_common(const gdn_attn_shape_t* s, int32_t N, const int32_t* cu, const int32_t* start, int64_t T, const void* k,
              int64_t ldk, const void* v, int64_t ldv, const gdn_kv_cache_t* cache, const int32_t* table,
              int32_t max_pages, KvIO* io) {
  int rc = gdn::check_attn_shape(s);
  if (rc != GDN_OK) return rc;
  rc = gdn::check_kv_cache(cache);
  if (rc != GDN_OK) return rc;
  if (N < 0 || T < 0 || max_pages < 0) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16({k, v}) || !gdn::aligned4({cu, start, table})) return GDN_ERR_INVALID_ARG;
  if (cu ? N == 0 && T > 0 : T != N) return GDN_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v || (max_pages > 0 && !table))) return GDN_ERR_INVALID_ARG;
  if (T > INT32_MAX || s->H_kv > 65535) return GDN_ERR_UNSUPPORTED;
  const int64_t w = static_cast<int64_t>(s->H_kv) * s->d;
  rc = gdn::attn_rows({{ldk, w, &io->ldk}, {ldv, w, &io->ldv}});
  if (rc != GDN_OK) return rc;
  io->kc = static_cast<uint8_t*>(cache->k); io->vc = static_cast<uint8_t*>(cache->v);
  io->ks = cache->k_scale; io->vs = cache->v_scale;
  io->pages = make_pages(cache, table, max_pages);
  io->cu = cu; io->start = start;
  io->k = const_cast<void*>(k); io->v = const_cast<void*>(v);
  io->T = T; io->N = N; io->H_kv = s->H_kv;
  return GDN_OK;
}

int64_t kv_slots(const KvIO& io) { return io.cu ? io.T / kBlk + 2 * static_cast<int64_t>(io.N) : io.N; }

// Where partial results stand: for every query row as many as the longest cache has
// splits, or one, and for every sequence as many as make up for it: a sequence of r
// rows has at most 1 + (most - 1) / ceil(r / kRowsSplit) splits (of at least kSplit
// tokens), and so at most r + kRowsSplit (most - 1) partial rows.  The smaller of the
// two.
void decode_layout(int64_t N, int64_t T, int32_t G, int64_t max_len, int64_t* mul, int64_t* extra) {
  int64_t most = (max_len + kSplit - 1) / kSplit;
  most = most > 1 ? most : 1;
  const bool rows = T * G <= N * kRowsSplit;
  *mul = rows ? most : 1;
  *extra = rows ? 0 : kRowsSplit * (most - 1);
}

}  // namespace

extern "C" {

int gdn_kv_write(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens, const int32_t* start,
                 int64_t n_tokens, const void* k, int64_t ldk, const void* v, int64_t ldv, const gdn_kv_cache_t* cache,
                 const int32_t* block_table, int32_t max_pages, void* stream) {
  KvIO io{};
  const int rc = kv_common(shape, n_seqs, cu_seqlens, start, n_tokens, k, ldk, v, ldv, cache, block_table, max_pages, &io);
  if (rc != GDN_OK) return rc;
  if (n_tokens == 0 || max_pages == 0) return GDN_OK;
  if (kv_slots(io) * 256 >= gdn::kLaunchThreads / io.H_kv) return GDN_ERR_UNSUPPORTED;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return kv_dispatch(shape, [&]<typename T, int D>() {
    Timed t_("k_kv_write", st);
    hipLaunchKernelGGL((k_kv_write<T, D>), dim3(static_cast<unsigned>(kv_slots(io)), io.H_kv), dim3(256), 0, st, io);
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}

int gdn_kv_read(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens, const int32_t* start,
                int64_t n_tokens, const gdn_kv_cache_t* cache, const int32_t* block_table, int32_t max_pages, void* k,
                int64_t ldk, void* v, int64_t ldv, void* stream) {
  KvIO io{};
  const int rc = kv_common(shape, n_seqs, cu_seqlens, start, n_tokens, k, ldk, v, ldv, cache, block_table, max_pages, &io);
  if (rc != GDN_OK) return rc;
  if (n_tokens == 0 || max_pages == 0) return GDN_OK;
  if (kv_slots(io) * 256 >= gdn::kLaunchThreads / io.H_kv) return GDN_ERR_UNSUPPORTED;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return kv_dispatch(shape, [&]<typename T, int D>() {
    Timed t_("k_kv_read", st);
    hipLaunchKernelGGL((k_kv_read<T, D>), dim3(static_cast<unsigned>(kv_slots(io)), io.H_kv), dim3(256), 0, st, io);
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}

size_t gdn_attn_decode_workspace_bytes(const gdn_attn_shape_t* shape, int32_t n_seqs, int64_t n_tokens, int64_t max_len) {
  if (gdn::check_attn_shape(shape) != GDN_OK || n_seqs < 0 || n_tokens < 0 || max_len < 0) return 0;
  if (n_tokens > INT32_MAX || max_len > INT32_MAX) return 0;
  const int32_t G = shape->H_q / shape->H_kv;
  if (max_len <= kSplit) return gdn::kAlign;
  int64_t mul, extra;
  decode_layout(n_seqs, n_tokens, G, max_len, &mul, &extra);
  const int64_t rows = (n_tokens * G * mul + n_seqs * extra) * shape->H_kv;
  const size_t bytes = static_cast<size_t>(rows) * (shape->d + 2) * sizeof(float);
  return (bytes + gdn::kAlign) / gdn::kAlign * gdn::kAlign;
}

int gdn_attn_decode(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens, int64_t n_tokens,
                    const void* q, int64_t ldq, const gdn_kv_cache_t* cache, const int32_t* block_table,
                    int32_t max_pages, const int32_t* kv_len, int64_t max_len, void* o, int64_t ldo, float* lse,
                    void* ws, size_t ws_bytes, void* stream) {
  int rc = gdn::check_attn_shape(shape);
  if (rc != GDN_OK) return rc;
  rc = gdn::check_kv_cache(cache);
  if (rc != GDN_OK) return rc;
  if (n_seqs < 0 || n_tokens < 0 || max_pages < 0 || max_len < 0) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16({q, o, ws}) || !gdn::aligned4({cu_seqlens, block_table, kv_len, lse})) return GDN_ERR_INVALID_ARG;
  if (cu_seqlens ? n_seqs == 0 && n_tokens > 0 : n_tokens != n_seqs) return GDN_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!q || !o || !kv_len || (max_pages > 0 && !block_table))) return GDN_ERR_INVALID_ARG;
  if (n_tokens > INT32_MAX || max_len > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  DecIO io{};
  const int64_t w = static_cast<int64_t>(shape->H_q) * shape->d;
  rc = gdn::attn_rows({{ldq, w, &io.ldq}, {ldo, w, &io.ldo}});
  if (rc != GDN_OK) return rc;
  const int64_t holds = static_cast<int64_t>(max_pages) * cache->page_tokens;
  if (max_len > holds) max_len = holds;
  const int32_t G = shape->H_q / shape->H_kv;
  const int64_t splits = (max_len + kSplit - 1) / kSplit;
  decode_layout(n_seqs, n_tokens, G, max_len, &io.mul, &io.extra);
  io.rows = (n_tokens * G * io.mul + n_seqs * io.extra) * shape->H_kv;
  if (splits > 1 && (!ws || ws_bytes < static_cast<size_t>(io.rows) * (shape->d + 2) * sizeof(float)))
    return GDN_ERR_WORKSPACE;
  if (n_tokens == 0) return GDN_OK;
  io.kc = static_cast<const uint8_t*>(cache->k); io.vc = static_cast<const uint8_t*>(cache->v);
  io.ks = cache->k_scale; io.vs = cache->v_scale;
  io.pages = make_pages(cache, block_table, max_pages);
  io.cu = cu_seqlens; io.len = kv_len; io.q = q; io.o = o; io.lse = lse;
  io.part = static_cast<float*>(ws);
  io.stat = splits > 1 ? io.part + io.rows * shape->d : nullptr;
  io.T = n_tokens; io.N = n_seqs; io.H_q = shape->H_q; io.H_kv = shape->H_kv; io.G = G;
  io.max_len = static_cast<int>(max_len);
  io.c = shape->scale * kLog2e;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return kv_dispatch(shape, [&]<typename T, int D>() {
    // what a sequence's rows are decides who takes it; a kernel that none of them
    // can need is not launched.  Packed, a sequence may have anything from no rows to
    // all of them, one sequence too: only the device's cu_seqlens says how many.
    const int64_t all = n_tokens * G;
    const bool wide = (cu_seqlens ? all : G) >= kWideRows, narrow = G < kWideRows;
    const int64_t tn = int64_t{n_seqs} * narrow_tiles(cu_seqlens != nullptr, G);
    const int64_t tw = cu_seqlens ? all / kAttnRows + n_seqs : int64_t{n_seqs} * ((G + kAttnRows - 1) / kAttnRows);
    const int64_t y = splits > 0 ? splits : 1, few = kLongLen / kSplit;
    const int64_t yn = y <= few ? y : (y + 1) / 2 > few ? (y + 1) / 2 : few;
    if ((narrow && tn * io.H_kv * 256 >= gdn::kLaunchThreads) || (wide && tw * io.H_kv * 256 >= gdn::kLaunchThreads))
      return static_cast<int>(GDN_ERR_UNSUPPORTED);
    if (narrow) {
      Timed t_("k_attn_decode", st);
      in_launches(tn * io.H_kv, yn, 256, [&](int y0, unsigned ny) {
        DecIO at = io;
        at.split0 = y0;
        hipLaunchKernelGGL((k_attn_decode<T, D>), dim3(static_cast<unsigned>(tn * io.H_kv), ny), dim3(256), 0, st, at);
      });
    }
    if (wide) {
      const int rc = launch_decode_wide(shape, io, tw, y, st);
      if (rc != GDN_OK) return rc;
    }
    const int64_t most = wide ? y : yn;  // splits of a sequence
    if (most > 1) {
      Timed t_("k_attn_join", st);
      // rows of a head, and as many of them as a launch of 1024 threads each holds (a multiple of per)
      const int64_t items = n_tokens * io.H_q, fit = gdn::kLaunchThreads / 1024 - 16;
      const bool brief = most <= kJoin;
      for (io.item0 = 0; io.item0 < items; io.item0 += fit) {
        const int64_t now = items - io.item0 < fit ? items - io.item0 : fit, per = brief ? 1024 / D : 1;
        const dim3 grid(static_cast<unsigned>((now + per - 1) / per));
        if (brief)
          hipLaunchKernelGGL((k_attn_join<T, D, 1>), grid, dim3(256), 0, st, io);
        else
          hipLaunchKernelGGL((k_attn_join<T, D, kJoin>), grid, dim3(D / 4 * kJoin), 0, st, io);
      }
    }
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}

}  // extern "C"
