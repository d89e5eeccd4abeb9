// What the kernels of attention over the 8-bit cache share.
#pragma once

#include "gdn_attn_walk.h"

namespace gdn {

constexpr int kBlk = GDN_KV_BLOCK;  // tokens that share a scale
static_assert(kBlk == 32);


// Pages of one pool and the table that names those of each sequence.
struct Pages {
  const int32_t* table;  // [N, width]
  int width, pages;
  uint32_t bpp, magic;   // blocks a page; 2^32 / bpp
  // The page that holds block b and the block's place there.
  __device__ __forceinline__ uint32_t page(uint32_t b, uint32_t* place) const {
    uint32_t i = __umulhi(b, magic);  // or one less
    if (b - i * bpp >= bpp) ++i;
    *place = b - i * bpp;
    return i;
  }
  __device__ __forceinline__ int id(int n, uint32_t i) const {
    if (i >= static_cast<uint32_t>(width)) return -1;
    const int p = table[static_cast<int64_t>(n) * width + i];
    return p >= 0 && p < pages ? p : -1;
  }
  // The index of sequence n's block b among [pages, H_kv, P / 32], -1 for none.
  __device__ __forceinline__ int64_t block(int n, int H_kv, int h, uint32_t b) const {
    uint32_t place;
    const int p = id(n, page(b, &place));
    return at(p, place, H_kv, h);
  }
  __device__ __forceinline__ int64_t at(int p, uint32_t place, int H_kv, int h) const {
    return p < 0 ? -1 : (static_cast<int64_t>(p) * H_kv + h) * bpp + place;
  }
};

struct DecIO {
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  Pages pages;
  const int32_t* cu;
  const int32_t* len;
  const void* q;
  void* o;
  float* lse;
  float* part;  // [rows of partial results][D]
  float* stat;  // [..][2]: maximum (of s log2 e) and sum
  int64_t T, ldq, ldo, rows;
  int64_t mul, extra;  // sequence n's partial results begin at mul cu[n] G + extra n
  int64_t item0;       // the join's first row of a head
  int split0;          // the launch's first split
  int N, H_q, H_kv, G, max_len;
  float c;
};
constexpr int kSplit = 512;        // tokens a split
constexpr int kLongLen = 4096;     // cached tokens over which the narrow kernel takes twice as many
constexpr int kRowsSplit = 256;    // rows for which the wide one's are that many
// A sequence of so many rows goes to the wide kernel: 32 sequences of 4000 cached
// tokens, 8 heads of 128: 32 rows each 144 us there and 156 in the narrow one, 64 rows
// 173 (172), 124 rows 239 (300); 2 heads of 256: 32 rows 95 (96), 64 rows 102
// (144).  The rule counts rows and does not look at what they are of: one token of 32
// heads that share one key head loses by it (24 us where the narrow one takes 18), as
// three of the wide one's four waves then have no rows.
constexpr int kWideRows = 32;
// Tiles of 16 rows that the narrow one has for a sequence.
__host__ __device__ inline int narrow_tiles(bool packed, int G) { return (packed ? kWideRows : G + 15) / 16; }

// Tokens a split of a sequence with `rows` rows a head: more where there are rows
// enough to go round.  A function of the sequence alone, so that its bits do not
// depend on the batch.  One new token, 64 sequences of 128 to 8192: 116 us (all with
// 1024 tokens 112, with 512 123, with 256 134), four of 4000: 16 us with 512, 24 with
// 1024.  Eight sequences' 64 to 500 new tokens: 360 us with 512 for 256 rows, 391 for
// 512 rows, 380 with 1024 for 256, 609 with 256.
__host__ __device__ inline int64_t split_tokens(int64_t rows, int64_t len) {
  return rows < kWideRows ? (len > kLongLen ? 2 * kSplit : kSplit) : kSplit * ((rows + kRowsSplit - 1) / kRowsSplit);
}

struct DecSeq {
  int64_t q0;
  int n, Lq, Lk;  // Lk: cached tokens that are read
  int64_t pos;    // of the first query
  int64_t rows, split;
  int splits;
  // the last cached token that query token t sees, -1 for none
  __device__ __forceinline__ int sees(int64_t t) const {
    const int64_t p = pos + t < Lk - 1 ? pos + t : Lk - 1;
    return static_cast<int>(p < -1 ? -1 : p);
  }
};
__device__ __forceinline__ DecSeq dec_seq(const DecIO& io, int n) {
  DecSeq s;
  s.n = n;
  s.q0 = n;
  s.Lq = 1;
  if (io.cu) {
    int64_t c0 = io.cu[n], c1 = io.cu[n + 1];
    c0 = c0 < 0 ? 0 : c0 > io.T ? io.T : c0;
    c1 = c1 < c0 ? c0 : c1 > io.T ? io.T : c1;
    s.q0 = c0;
    s.Lq = static_cast<int>(c1 - c0);
  }
  int64_t len = io.len[n];
  s.pos = len - s.Lq;
  len = len < 0 ? 0 : len > io.max_len ? io.max_len : len;
  s.Lk = static_cast<int>(len);
  s.rows = static_cast<int64_t>(s.Lq) * io.G;
  s.split = split_tokens(s.rows > 0 ? s.rows : 1, len);
  s.splits = static_cast<int>((s.Lk + s.split - 1) / s.split);
  if (s.splits < 1) s.splits = 1;
  return s;
}

// Eight codes as bf16, times the power of two s.
__device__ __forceinline__ u32x4 codes8(uint32_t lo, uint32_t hi, float s) {
  u32x4 y;
  y[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false));
  y[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true));
  y[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false));
  y[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true));
  return y;
}
template <typename F>
int kv_dispatch(const gdn_attn_shape_t* s, F&& f) {
  if (s->in_dtype == GDN_BF16) {
    if (s->d == 64) return f.template operator()<bf16_t, 64>();
    if (s->d == 128) return f.template operator()<bf16_t, 128>();
    return f.template operator()<bf16_t, 256>();
  }
  if (s->d == 64) return f.template operator()<float, 64>();
  if (s->d == 128) return f.template operator()<float, 128>();
  return f.template operator()<float, 256>();
}

// Launches go(y0, y) over `y` of splits and x blocks of `threads` for each, in as
// many launches as keep each within what one may hold.
template <typename F>
void in_launches(int64_t x, int64_t y, int threads, F&& go) {
  const int64_t fit = (kLaunchThreads - 1) / (x * threads), most = fit < 65535 ? fit : 65535;
  for (int64_t y0 = 0; y0 < y; y0 += most) go(static_cast<int>(y0), static_cast<unsigned>(y - y0 < most ? y - y0 : most));
}

// Launches k_attn_decode_wide over `tiles` tiles of kAttnRows rows and `splits`
// splits a head (gdn_kv_wide.hip).
int launch_decode_wide(const gdn_attn_shape_t* shape, const DecIO& io, int64_t tiles, int64_t splits, hipStream_t st)
    __attribute__((visibility("hidden")));

}  // namespace gdn
