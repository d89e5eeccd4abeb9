// Attention over the 8-bit cache for sequences of many query rows (include/gdn.h).
// Apart from gdn_kv.hip, as its sums stay in the accumulation registers.
#include "gdn_kv.h"

namespace {

using namespace gdn;

// The sequence and the tile of `rows` rows within it that slot x takes: sequence n's
// slots begin at cu[n] G / rows + n.
__device__ __forceinline__ int row_tile(const DecIO& io, int rows, int x, int* tile) {
  if (!io.cu) {
    const int per = (io.G + rows - 1) / rows;
    *tile = x % per;
    return x / per;
  }
  int lo = 0, hi = io.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(io.cu[mid]) * io.G / rows + mid <= x) lo = mid; else hi = mid - 1;
  }
  *tile = static_cast<int>(x - (static_cast<int64_t>(io.cu[lo]) * io.G / rows + lo));
  return lo;
}

// Sequences of kWideRows rows and more: 128 rows a workgroup and the walk that
// attention over prompts takes, with codes that become bf16 on their way into LDS,
// once for all of the rows.  Eight sequences with 64 to 500 new tokens and 500 to 8192
// cached ones, 32 and 8 heads of 128: 307 us, 640 TFLOP/s (and 27 to join); bound by
// the walk's steps, in which vector instructions take 51% of the cycles (codes to bf16
// once for 128 rows) and products 30%, and by 830 blocks of uneven length on 512 places.

// Tiles of the cache, one block of it each: 16 codes a thread and step.
template <int D>
struct CacheStage {
  static constexpr bool DIRECT = false, GAPS = true;
  using P = Plane<bf16_t, D, kBlk>;
  static_assert(kAttnStep == kBlk);
  static constexpr int CPR = D / 16, PIECES = kBlk * CPR, STEPS = (PIECES + 255) / 256, LOADS = STEPS;
  const DecIO& io;
  const DecSeq& sq;
  int hk;
  u32x4 k[STEPS], v[STEPS];
  float ks, vs;
  // Blocks of the keys' tile that is held (b0) and of the one before it, without a
  // page -1; the values' tile is the one or the other.  gap: those of the keys' last
  // three tiles, the step's first.
  int64_t b0 = -1, b1 = -1, bv = -1;
  bool there[3] = {};
  bool begun = false;
  int left, rows = 0;    // tokens from the values' next tile on, of the one held
  uint32_t next, place;  // page and place of the keys' next tile
  int page;              // looked up a step ahead
  __device__ __forceinline__ CacheStage(const DecIO& io, const DecSeq& sq, int hk, int first)
      : io(io), sq(sq), hk(hk), left(sq.Lk - first * kBlk) {
    next = io.pages.page(first, &place);
    page = io.pages.id(sq.n, next);
  }
  __device__ __forceinline__ bool gap() const { return !there[0]; }
  // Without a page: block 0 is read, and not used.  Its scores are masked whatever they
  // are; its values' scale may be NaN, where nothing was written yet, and zeros for
  // codes times that would be, so finish_v takes 1.
  __device__ __forceinline__ void next_k() {
    b1 = b0;
    b0 = io.pages.at(page, place, io.H_kv, hk);
    there[0] = there[1];
    there[1] = there[2];
    there[2] = b0 >= 0;
    ks = io.ks[b0 < 0 ? 0 : b0];
    const bool wrap = ++place == io.pages.bpp;
    place = wrap ? 0 : place;
    next += wrap ? 1 : 0;
    page = io.pages.id(sq.n, next);
  }
  __device__ __forceinline__ void next_v() {  // the keys are two tiles ahead, but at first
    bv = begun ? b1 : b0;
    begun = true;
    vs = io.vs[bv < 0 ? 0 : bv];
    rows = bv < 0 ? 0 : left;  // nothing stands behind the last token
    left -= kBlk;
  }
  __device__ __forceinline__ void load_k(int i, char*) { load(io.kc, b0, i, k); }
  __device__ __forceinline__ void load_v(int i, char*) { load(io.vc, bv, i, v); }
  static __device__ __forceinline__ void load(const uint8_t* codes, int64_t blk, int i, u32x4* x) {
    if (PIECES >= 256 || threadIdx.x < PIECES)
      x[i] = *reinterpret_cast<const u32x4*>(codes + (blk < 0 ? 0 : blk) * (kBlk * D) + (i * 256 + threadIdx.x) * 16);
  }
  __device__ __forceinline__ void finish_k(char* kb) const { store(kb, k, ks, INT32_MAX); }
  __device__ __forceinline__ void finish_v(char* vb) const { store(vb, v, rows > 0 ? vs : 1.0f, rows); }
  static __device__ __forceinline__ void store(char* lds, const u32x4* x, float scale, int rows) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (PIECES < 256 && threadIdx.x >= PIECES) break;
      const int c = s * 256 + threadIdx.x, r = c / CPR, piece = c % CPR * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t lo = r < rows ? x[s][2 * e] : 0u, hi = r < rows ? x[s][2 * e + 1] : 0u;
        *reinterpret_cast<u32x4*>(lds + r * P::RB + (((piece + e) ^ swizzle<P::RB>(r)) << 4)) = codes8(lo, hi, scale);
      }
    }
  }
};

template <typename T, int D>
__global__ __launch_bounds__(256, (kAttnOcc<T, D>)) void k_attn_decode_wide(DecIO io) {
#ifdef GDN_DEVICE_PASS
  constexpr int BM = kAttnRows, BN = kAttnStep;
  __shared__ int odd[D + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = blockIdx.x % io.H_kv, x = blockIdx.x / io.H_kv, split = io.split0 + blockIdx.y;
  int tile;
  const int n = row_tile(io, BM, x, &tile);
  const DecSeq sq = dec_seq(io, n);
  const int64_t b0 = static_cast<int64_t>(tile) * BM, r0 = b0 + 32 * wave, r = r0 + (lane & 31);
  if (tile < 0 || b0 >= sq.rows || split >= sq.splits || sq.rows < kWideRows) return;
  const int64_t b1 = (b0 + BM < sq.rows ? b0 + BM : sq.rows) - 1, r1 = (r0 + 32 < sq.rows ? r0 + 32 : sq.rows) - 1;
  const bool in = r < sq.rows;
  const int64_t tok = in ? r / io.G : 0;
  const int head = hk * io.G + static_cast<int>(in ? r - tok * io.G : 0);
  AttnRows at;
  at.lim = in ? sq.sees(tok) : -1;
  at.lo = sq.sees(r0 / io.G);
  at.block_lo = sq.sees(b0 / io.G);
  Held<T, D> q[D / 16];
  {
    const int64_t t0 = r0 < sq.rows ? r0 / io.G : 0;
    const char* base = static_cast<const char*>(io.q) + (sq.q0 + t0) * io.ldq * sizeof(T);
    const int bytes = r0 < sq.rows ? static_cast<int>(((r1 / io.G - t0) * io.ldq + static_cast<int64_t>(io.H_q) * D) * sizeof(T)) : 0;
    const brsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), static_cast<short>(0), bytes, 0x00020000);
    const uint32_t from = in ? static_cast<uint32_t>(((tok - t0) * io.ldq + head * D + 8 * (lane >> 5)) * sizeof(T)) : 0x7fff0000u;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) q[ks].load(rq, from + 16 * ks * sizeof(T));
  }
  const int64_t t0 = sq.split * split;
  int64_t t1 = sq.sees(b1 / io.G) + 1;
  t1 = t0 + sq.split < t1 ? t0 + sq.split : t1;
  CacheStage<D> st(io, sq, hk, static_cast<int>(t0 / BN));
  AttnState<D> a;
  attn_walk<T, bf16_t, D, kAttnWaves, 1>(st, 0, q, static_cast<int>(t0 / BN), static_cast<int>((t1 + BN - 1) / BN), at, io.c, lane, odd, a);
  if (!in) return;
  if (sq.splits == 1) {
    store_row<D>(static_cast<T*>(io.o) + (sq.q0 + tok) * io.ldo + static_cast<int64_t>(head) * D, a.acc, inverse_sum(a.l), lane);
    if (io.lse && lane < 32) io.lse[(sq.q0 + tok) * io.H_q + head] = lse_of(a.m * io.c, a.l);
  } else {
    const int64_t pr = (sq.q0 * io.G * io.mul + n * io.extra + r * sq.splits + split) * io.H_kv + hk;
    store_row<D>(io.part + pr * D, a.acc, 1.0f, lane);
    if (lane < 32) {
      io.stat[2 * pr] = a.m * io.c;
      io.stat[2 * pr + 1] = a.l;
    }
  }
#endif
}

}  // namespace

int gdn::launch_decode_wide(const gdn_attn_shape_t* shape, const DecIO& io, int64_t tiles, int64_t splits, hipStream_t st) {
  return kv_dispatch(shape, [&]<typename T, int D>() {
    Timed t_("k_attn_decode_wide", st);
    in_launches(tiles * io.H_kv, splits, 256, [&](int y0, unsigned y) {
      DecIO at = io;
      at.split0 = y0;
      hipLaunchKernelGGL((k_attn_decode_wide<T, D>), dim3(static_cast<unsigned>(tiles * io.H_kv), y), dim3(256), 0, st, at);
    });
    return static_cast<int>(hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP);
  });
}
