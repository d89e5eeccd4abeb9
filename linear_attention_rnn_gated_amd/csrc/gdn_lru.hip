// Gated linear recurrence (include/gdn.h): kernels and C ABI.  Part of
// gdn_library.hip.
//
// Per channel, h_t = alpha_t h_{t-1} + u_t with u = b x.  A chunk of 32 tokens
// is the map h -> A h + B; its running composition (A_p, B_p) needs no state,
// so every chunk of a sequence is composed at once, the states at the chunks'
// starts follow one another with one fma per chunk, and h_p = fma(A_p, S, B_p).
// The same operations in the same order run in decode, one token at a time.
//
// Going back, a chunk maps the gradient K of the state behind its last token to
// that in front of its first one, K -> A K + Q with Q = sum_p A_p dO_p, which
// needs no state either.
//
// Two schedules give these operations, and the same bits:
//   one pass     k_lru_fwd: a block takes a channel tile of one sequence, or of
//                several short ones, and goes over their chunks in rounds, a
//                few lanes to a chunk; inputs are read once.  Prefill with
//                enough sequences and channels to fill the chip.  k_lru_train
//                is the trainer's, of sequences that fit one round.
//   three steps  k_lru_fold (every chunk's A, B and Q), k_lru_chain (the states
//                and gradients at the chunks' edges), k_lru_apply or k_lru_grad
//                (outputs): every step runs over all chunks at once, and the
//                inputs are read twice.  Prefill of long sequences of few
//                channels, and the trainer's longer sequences.
// Measured (bf16 x, norm gate, one MI355X): one pass, 4 x 2048 tokens x 4096
// channels, fp32 g 59 us = 4.6 TB/s; 32 x 128..8192 x 2048, bf16 g, complement
// gate 433 us = 4.2 TB/s; trainer, 8 x 4096 x 4096, fp32 g 600 us: fold 214 (5.0
// TB/s), chain 26, grad 360 (6.0 TB/s), 24 bytes an element where one reading
// would be 16.  Running the trainer a sequence at a time, so that the second
// reading could come out of the last-level cache, took 750 us.
//
// Bound: HBM.  An element takes 6 (bf16) or 12 (fp32) bytes in a prefill, 12 to 24
// in the trainer's one pass and 18 to 36 in its three steps, and 20 to 40 vector
// instructions.

namespace {

constexpr int kLruC = GDN_LRU_CHUNK;
constexpr int kLruPack = gdn::kLruPack;
constexpr int kLruThreads = gdn::kLruThreads;
constexpr int kLruTrain = gdn::kLruTrain;

struct LruIO {
  const void* x;
  const void* g;
  void* o;
  const float* h0;
  float* hT;
  gdn_lru_cache_t cache;  // S nullptr: none
  int resume;             // start from the cache
  const int32_t* cu;
  int N, D, gate;
  int64_t T, ldx, ldg, ldo;
  // one pass
  gdn::LruPlan plan;
  int tiles;  // channel tiles
  // three steps
  int cw;        // lanes of a block over channels; 256 / cw chunks a block
  int64_t slots; // chunk slots
  float* wA;     // [slots][D] chunk products
  float* wB;     // [slots][D] chunk states from zero, then the states at the starts
  float* wQ;     // [slots][D] the gradient's, then the gradients behind the ends
  float* keep;   // [N][2][D] the cache's A and B before the call
  // trainer
  const void* dO;
  const float* dhT;
  void* dx;
  void* dg;
  float* dh0;
  int64_t lddo, lddx, lddg;
};

__device__ __forceinline__ void stout(float* p, float x) { *p = x; }
__device__ __forceinline__ void stout(bf16_t* p, float x) {
  *p = static_cast<bf16_t>(pack_bf16(x, 0.0f));  // round to nearest even
}

// exp(g) and 1 - exp(g) of one g, both to fp32's last place, from one
// reduction g = n ln 2 + f: with p = e^f - 1 = f + f^2 q(f) (|f| <= ln 2 / 2, q
// of degree 4, p within a relative 2^-25.8),
//     exp(g) = 2^n (1 + p),   1 - exp(g) = -2 (2^(n-1) p + (2^(n-1) - 1/2)),
// the latter without cancellation near g = 0, where n = 0 leaves -p.  Limits:
// below -104 the result is 0 (2^-150), above 89 infinite; NaN stays NaN.
// By the roundings within 2 and 3 times 2^-24; measured over four
// million values 1.41 and 1.46 (and 2.5 for the norm gate's root).
struct LruExp {
  float a, m;  // exp(g), 1 - exp(g)
};
__device__ __forceinline__ LruExp lru_exp(float g) {
  float c = __builtin_amdgcn_fmed3f(g, -104.0f, 89.0f);
  c = g != g ? g : c;
  const float n = rintf(c * 1.44269504f);
  float f = fmaf(n, -0.693145751953125f, c);  // 15 bits of ln 2: the product is exact
  f = fmaf(n, -1.42860677e-06f, f);
  float q = 0.0013882518978789449f;
  q = fmaf(q, f, 0.008366530761122704f);
  q = fmaf(q, f, 0.04166720062494278f);
  q = fmaf(q, f, 0.1666654348373413f);
  q = fmaf(q, f, 0.4999999701976776f);
  const float p = fmaf(f * f, q, f);
  const int e = static_cast<int>(n);
  LruExp r;
  r.a = __builtin_amdgcn_ldexpf(1.0f + p, e);
  const float h = __builtin_amdgcn_ldexpf(0.5f, e);
  r.m = -2.0f * fmaf(h, p, h - 0.5f);
  return r;
}

// alpha and the input's weight b of one element.  In the norm gate 1 - alpha^2
// = m (1 + alpha), and the root is the hardware's (1 ulp): the correctly
// rounded one takes about ten instructions more per element for a bit that
// the products after it lose again.
template <int GATE>
__device__ __forceinline__ float lru_weight(float g, float& a) {
  const LruExp r = lru_exp(g);
  a = r.a;
  if constexpr (GATE == GDN_LRU_GATE_NONE) return 1.0f;
  if constexpr (GATE == GDN_LRU_GATE_COMPLEMENT) return r.m;
  // the maximum that keeps a NaN, and one instruction as fmaxf, which does not
  return __builtin_amdgcn_sqrtf(__builtin_elementwise_maximum(r.m * (1.0f + r.a), 0.0f));
}
// u = b x; without a gate x itself.
template <int GATE>
__device__ __forceinline__ float lru_input(float g, float x, float& a) {
  const float b = lru_weight<GATE>(g, a);
  return GATE == GDN_LRU_GATE_NONE ? x : b * x;
}

// Sequence n's rows, kept inside [0, T) whatever the device copy holds.
__device__ __forceinline__ void lru_rows(const LruIO& io, int n, int64_t& t0, int64_t& L) {
  int64_t a = io.cu[n], b = io.cu[n + 1];
  a = a < 0 ? 0 : (a > io.T ? io.T : a);
  b = b < a ? a : (b > io.T ? io.T : b);
  t0 = a;
  L = b - a;
}

// Position in the current chunk that the cache gives, inside [0, 32).
__device__ __forceinline__ int lru_pos(const LruIO& io, int n, int c) {
  const int groups = (io.D + gdn::kLruGroup - 1) / gdn::kLruGroup;
  const int p = io.cache.pos[static_cast<int64_t>(n) * groups + c / gdn::kLruGroup];
  return p < 0 ? 0 : (p >= kLruC ? kLruC - 1 : p);
}

// Block -> (unit, channel tile).  Runs of four items (neighbouring tiles of a
// unit, mostly) go to one XCD (blocks are dealt to the eight XCDs in turn), where
// tiles narrower than a cache line share it in that XCD's L2.  No item is left
// out inside a run: an XCD deals its blocks to its four shader engines in turn, so
// runs with idle places would leave whole engines idle (80 x 3000 tokens x 64
// channels, two tiles: 73 us with runs padded to four, 41 without).
__device__ __forceinline__ bool lru_item(const LruIO& io, int& unit, int& tile) {
  const int64_t b = blockIdx.x;
  const int64_t xcd = b & 7, j = b >> 3;
  const int64_t item = ((j >> 2) * 8 + xcd) * 4 + (j & 3);
  const int64_t u = item / io.tiles;
  tile = static_cast<int>(item - u * io.tiles);
  unit = static_cast<int>(u);
  return u < io.plan.units;
}
int64_t lru_blocks(int64_t units, int tiles) { return (units * tiles + 31) / 32 * 32; }

// What an empty sequence's channel e = n D + c ends with: where it began.
__device__ __forceinline__ void lru_empty(const LruIO& io, int64_t e) {
  if (io.resume) {
    if (io.hT) io.hT[e] = fmaf(io.cache.A[e], io.cache.S[e], io.cache.B[e]);
    return;
  }
  const float S = io.h0 ? io.h0[e] : 0.0f;
  if (io.hT) io.hT[e] = S;
  if (io.cache.S) {
    io.cache.S[e] = S;
    io.cache.A[e] = 1.0f;
    io.cache.B[e] = 0.0f;
  }
}

// Marks a map (mark, S) that gives S whatever was before it: a sequence's first
// chunk, whose lanes know their start.  A product that is a NaN goes into the
// chain as the plain one, so that no input's NaN can look like the mark.
constexpr uint32_t kLruMark = 0xffc0deadu, kPlainNaN = 0x7fc00000u;

// The chain S -> a S + b over m maps in LDS, W entries apart, for one channel;
// put(s, S) takes the state in front of map s (none in front of a marked one).
// U maps at a time, the next U read before the U fma's, so that a step costs its
// fma and not a round trip to LDS.
template <bool MARKS, int U, typename Put>
__device__ __forceinline__ float lru_chain(const float2* agg, int W, int maps, float S, Put&& put) {
  const int m = __builtin_amdgcn_readfirstlane(maps);  // the same for the whole block: scalar branches
  float2 ab[U], next[U];
#pragma unroll
  for (int j = 0; j < U; ++j) ab[j] = agg[(j < m ? j : m - 1) * W];
  int s0 = 0;
  for (; s0 + U <= m; s0 += U) {
#pragma unroll
    for (int j = 0; j < U; ++j) next[j] = agg[(s0 + U + j < m ? s0 + U + j : m - 1) * W];
    float before[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      before[j] = S;
      const float to = fmaf(ab[j].x, S, ab[j].y);
      S = MARKS && __float_as_uint(ab[j].x) == kLruMark ? ab[j].y : to;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (!(MARKS && __float_as_uint(ab[j].x) == kLruMark)) put(s0 + j, before[j]);
      ab[j] = next[j];
    }
  }
#pragma unroll
  for (int j = 0; j < U - 1; ++j) {
    if (s0 + j < m) {
      const bool mark = MARKS && __float_as_uint(ab[j].x) == kLruMark;
      if (!mark) put(s0 + j, S);
      S = mark ? ab[j].y : fmaf(ab[j].x, S, ab[j].y);
    }
  }
  return S;
}

// The sequences of a unit; chunk0[i] counts the chunks before its i-th.
struct LruUnit {
  int i0, count;
  __device__ __forceinline__ int sequence(const LruIO& io, int i) const {
    return io.plan.per ? i0 + i : static_cast<int>(io.plan.seq[i0 + i]);
  }
  // the last sequence that begins at or before a chunk
  __device__ __forceinline__ int find(const int64_t* chunk0, int64_t chunk) const {
    int i = 0;
    for (int d = kLruPack / 2; d >= 1; d >>= 1)
      if (i + d < count && chunk0[i + d] <= chunk) i += d;
    return i;
  }
};
__device__ __forceinline__ LruUnit lru_open(const LruIO& io, int unit, int64_t* chunk0) {
  const int per = io.plan.per;
  LruUnit of;
  of.i0 = per ? unit * per : io.plan.first[unit];
  of.count = per ? (io.N - of.i0 < per ? io.N - of.i0 : per) : io.plan.first[unit + 1] - of.i0;
  if (threadIdx.x < 64) {
    int64_t t0, L = 0, chunks = 0;
    if (static_cast<int>(threadIdx.x) < of.count) {
      const int n = of.sequence(io, threadIdx.x);
      lru_rows(io, n, t0, L);
      if (L > 0) chunks = ((io.resume ? lru_pos(io, n, 0) : 0) + L + kLruC - 1) / kLruC;
    }
    int64_t before = chunks;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t up = __shfl_up(before, m, 64);
      if (static_cast<int>(threadIdx.x) >= m) before += up;
    }
    chunk0[threadIdx.x + 1] = before;
    if (threadIdx.x == 0) chunk0[0] = 0;
  }
  __syncthreads();
  return of;
}

template <typename TX, typename TG, int GATE>
__global__ __launch_bounds__(kLruThreads) void k_lru_fwd(LruIO io) {
  __shared__ float2 agg[kLruThreads];  // [slot][channel of the tile]
  __shared__ float start[kLruThreads];
  __shared__ int64_t chunk0[kLruPack + 1];  // chunks of the unit before each of its sequences
  int unit, tile;
  if (!lru_item(io, unit, tile)) return;
  const int W = io.plan.lps;
  const int slots = blockDim.x / W;
  const int slot = threadIdx.x / W;
  const int c = tile * W + static_cast<int>(threadIdx.x) - slot * W;
  const bool live = c < io.D;
  const int cc = live ? c : io.D - 1;
  const bool folds = slot == 0 && live;  // these threads hold the chain of one channel each
  const LruUnit of = lru_open(io, unit, chunk0);
  if (folds) {
    for (int i = 0; i < of.count; ++i)
      if (chunk0[i + 1] == chunk0[i]) lru_empty(io, static_cast<int64_t>(of.sequence(io, i)) * io.D + c);
  }
  const int64_t nch = chunk0[of.count];
  float S = 0.0f;
  for (int64_t cb = 0; cb < nch; cb += slots) {
    const bool has = cb + slot < nch;
    int lo = 0, hi = 0;
    bool last = false;
    int64_t row = 0, sn = 0;  // row of the chunk's place 0, the sequence's states
    float A[kLruC], B[kLruC], ae = 1.0f, be = 0.0f;  // the chunk's composition at every place, and whole
    if (has) {
      const int i = of.find(chunk0, cb + slot);
      const int n = of.sequence(io, i);
      int64_t t0, L;
      lru_rows(io, n, t0, L);
      sn = static_cast<int64_t>(n) * io.D;
      const int64_t ch = cb + slot - chunk0[i];
      const int64_t tb = ch * kLruC - (io.resume ? lru_pos(io, n, 0) : 0);
      row = t0 + tb;
      lo = tb < 0 ? static_cast<int>(-tb) : 0;
      hi = L - tb < kLruC ? static_cast<int>(L - tb) : kLruC;
      last = cb + slot + 1 == chunk0[i + 1];
      const TX* x = static_cast<const TX*>(io.x) + cc;
      const TG* g = static_cast<const TG*>(io.g) + cc;
      float a = 1.0f, b = 0.0f;
      // sixteen rows' loads at a time: all of them at once spilled registers, and
      // four waves a SIMD keep enough in flight (32 ragged x 2048: 454 -> 436 us)
      if (__all(lo == 0 && hi == kLruC)) {  // one way for all chunks of a wave
#pragma unroll
        for (int half = 0; half < kLruC; half += kLruC / 2) {
#pragma unroll
          for (int j = half; j < half + kLruC / 2; ++j) {
            A[j] = ldin(g + (row + j) * io.ldg);
            B[j] = ldin(x + (row + j) * io.ldx);
          }
#pragma unroll
          for (int j = half; j < half + kLruC / 2; ++j) {
            float al;
            const float u = lru_input<GATE>(A[j], B[j], al);
            A[j] = a = al * a;
            B[j] = b = fmaf(al, b, u);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        if (lo > 0) {
          a = io.cache.A[sn + cc];
          b = io.cache.B[sn + cc];
        }
        // eight rows at a time, those that no lane of the wave has left out
#pragma unroll
        for (int j0 = 0; j0 < kLruC; j0 += 8) {
          if (__any(j0 < hi && j0 + 8 > lo)) {
#pragma unroll
            for (int j = j0; j < j0 + 8; ++j) {
              const int64_t t = row + (j < lo ? lo : (j >= hi ? hi - 1 : j));  // a row of this chunk
              A[j] = ldin(g + t * io.ldg);
              B[j] = ldin(x + t * io.ldx);
            }
#pragma unroll
            for (int j = j0; j < j0 + 8; ++j) {
              float al;
              float u = lru_input<GATE>(A[j], B[j], al);
              // places outside the rows change nothing: 1 a = a, fma(1, b, -0) = b
              const bool in = j >= lo && j < hi;
              al = in ? al : 1.0f;
              u = in ? u : -0.0f;
              A[j] = a = al * a;
              B[j] = b = fmaf(al, b, u);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      ae = a;
      be = b;
      if (ch == 0) {
        const float S0 = io.resume ? io.cache.S[sn + cc] : (io.h0 ? io.h0[sn + cc] : 0.0f);
        start[threadIdx.x] = S0;
        agg[threadIdx.x] = float2{__uint_as_float(kLruMark), fmaf(a, S0, b)};
      } else {
        agg[threadIdx.x] = float2{a != a ? __uint_as_float(kPlainNaN) : a, b};
      }
    }
    __syncthreads();
    if (folds)
      S = lru_chain<true, 4>(agg + threadIdx.x, W, static_cast<int>(nch - cb < slots ? nch - cb : slots), S,
                             [&](int s, float v) { start[s * W + threadIdx.x] = v; });
    __syncthreads();
    if (has && live) {
      const float st = start[threadIdx.x];
      TX* o = static_cast<TX*>(io.o) + c;
      if (__all(lo == 0 && hi == kLruC)) {
#pragma unroll
        for (int j = 0; j < kLruC; ++j) stout(o + (row + j) * io.ldo, fmaf(A[j], st, B[j]));
      } else {
#pragma unroll
        for (int j = 0; j < kLruC; ++j)
          if (j >= lo && j < hi) stout(o + (row + j) * io.ldo, fmaf(A[j], st, B[j]));
      }
      if (last) {
        const float h = fmaf(ae, st, be);
        if (io.hT) io.hT[sn + c] = h;
        if (io.cache.S) {
          const bool full = hi == kLruC;
          io.cache.S[sn + c] = full ? h : st;
          io.cache.A[sn + c] = full ? 1.0f : ae;
          io.cache.B[sn + c] = full ? 0.0f : be;
        }
      }
    }
  }
}

// Outputs and gradients of one chunk of one channel from alpha, x, dO and, in w,
// the input's weight: forward for h and
//     e_i = alpha_i h_{i-1} + b'_i x_i      (dg_i = delta_i e_i)
// in the place of x, then backward for delta.  S is the state in front of the
// chunk, K the gradient of the one behind it; places from hi on are not written
// (WHOLE: there are none).
template <int GATE, bool WHOLE, typename TX, typename TG>
__device__ __forceinline__ void lru_outputs(const float* al, float* x, const float* dy, const float* w, float S, float K,
                                            int hi, int64_t row, TX* o, int64_t ldo, TX* dx, int64_t lddx, TG* dg,
                                            int64_t lddg) {
  float a = 1.0f, b = 0.0f, hp = S;
  TX* po = o ? o + row * ldo : nullptr;
#pragma unroll
  for (int i = 0; i < kLruC; ++i) {
    const float xi = x[i];
    const float u = GATE == GDN_LRU_GATE_NONE ? xi : w[i] * xi;
    a = al[i] * a;
    b = fmaf(al[i], b, u);
    const float h = fmaf(a, S, b);
    if (o && (WHOLE || i < hi)) stout(po, h);
    po += ldo;
    float e = al[i] * hp;
    if constexpr (GATE == GDN_LRU_GATE_COMPLEMENT) e = fmaf(-al[i], xi, e);
    // b' = -alpha^2 / b, the reciprocal the hardware's (1 ulp)
    if constexpr (GATE == GDN_LRU_GATE_NORM)
      e = fmaf(w[i] > 0.0f ? -(al[i] * al[i]) * __builtin_amdgcn_rcpf(w[i]) : 0.0f, xi, e);
    x[i] = e;
    hp = h;
  }
  dx += (row + kLruC - 1) * lddx;
  dg += (row + kLruC - 1) * lddg;
#pragma unroll
  for (int i = kLruC - 1; i >= 0; --i) {
    if (WHOLE || i < hi) {
      const float d = dy[i] + K;
      K = al[i] * d;
      stout(dx, GATE == GDN_LRU_GATE_NONE ? d : w[i] * d);
      stout(dg, d * x[i]);
    }
    dx -= lddx;
    dg -= lddg;
  }
}

// The trainer of units that fit one round: a chunk's inputs stay in its lanes'
// registers from the composition to the gradients, so they are read once.  Bound
// by HBM where large: 64 x 256 tokens x 4096 channels, norm gate, bf16 and fp32 g 254
// us = 4.2 TB/s, all fp32 318 us = 5.1 TB/s (three steps: 310 and 458).  171
// registers, two waves a SIMD; held to 168 for three it spilled and took 273 us.
template <typename TX, typename TG, int GATE>
__global__ __launch_bounds__(kLruTrain) void k_lru_train(LruIO io) {
  __shared__ float2 up[kLruTrain], down[kLruTrain];  // [slot][channel of the tile]: (A, B) and (A, Q)
  __shared__ float start[kLruTrain], behind[kLruTrain];
  __shared__ int64_t chunk0[kLruPack + 1];
  int unit, tile;
  if (!lru_item(io, unit, tile)) return;
  const int W = io.plan.lps;
  const int slots = blockDim.x / W;
  const int slot = threadIdx.x / W;
  const int col = static_cast<int>(threadIdx.x) - slot * W;
  const int c = tile * W + col;
  const bool live = c < io.D;
  const int cc = live ? c : io.D - 1;
  const LruUnit of = lru_open(io, unit, chunk0);
  if (slot == 0 && live) {
    for (int i = 0; i < of.count; ++i)
      if (chunk0[i + 1] == chunk0[i]) {
        const int64_t e = static_cast<int64_t>(of.sequence(io, i)) * io.D + c;
        lru_empty(io, e);
        io.dh0[e] = io.dhT ? io.dhT[e] : 0.0f;
      }
  }
  // a device copy of cu_seqlens that disagrees with the host's may need more than a round: left out
  const int nch = static_cast<int>(chunk0[of.count] < slots ? chunk0[of.count] : slots);
  if (nch == 0) return;
  const bool has = slot < nch;
  int hi = 0;
  bool first = false, last = false;
  int64_t row = 0, e = 0;
  float al[kLruC], x[kLruC], dy[kLruC], w[GATE == GDN_LRU_GATE_NONE ? 1 : kLruC];
  float a = 1.0f, b = 0.0f, q = 0.0f;
  if (has) {
    const int i = of.find(chunk0, slot);
    const int n = of.sequence(io, i);
    int64_t t0, L;
    lru_rows(io, n, t0, L);
    const int64_t ch = slot - chunk0[i], tb = ch * kLruC;
    row = t0 + tb;
    hi = L - tb < kLruC ? static_cast<int>(L - tb) : kLruC;
    first = ch == 0;
    last = slot + 1 == chunk0[i + 1];
    e = static_cast<int64_t>(n) * io.D + c;
    const TX* px = static_cast<const TX*>(io.x) + cc;
    const TG* pg = static_cast<const TG*>(io.g) + cc;
    const TX* py = static_cast<const TX*>(io.dO) + cc;
    // all rows' loads first; eight rows that no lane of the wave has are left out.
    // Places behind the last token change nothing: 1 a = a, fma(1, b, -0) = b
    if (__all(hi == kLruC)) {  // one way for all chunks of a wave
#pragma unroll
      for (int j = 0; j < kLruC; ++j) {
        al[j] = ldin(pg + (row + j) * io.ldg);
        x[j] = ldin(px + (row + j) * io.ldx);
        dy[j] = ldin(py + (row + j) * io.lddo);
      }
#pragma unroll
      for (int j = 0; j < kLruC; ++j) {
        const float wj = lru_weight<GATE>(al[j], al[j]);
        if constexpr (GATE != GDN_LRU_GATE_NONE) w[j] = wj;
      }
    } else {
#pragma unroll
      for (int j0 = 0; j0 < kLruC; j0 += 8) {
        if (__any(j0 < hi)) {
#pragma unroll
          for (int j = j0; j < j0 + 8; ++j) {
            const int64_t t = row + (j < hi ? j : hi - 1);
            al[j] = ldin(pg + t * io.ldg);
            x[j] = ldin(px + t * io.ldx);
            dy[j] = ldin(py + t * io.lddo);
          }
        } else {
#pragma unroll
          for (int j = j0; j < j0 + 8; ++j) al[j] = x[j] = dy[j] = 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < kLruC; ++j) {
        const float wj = lru_weight<GATE>(al[j], al[j]);
        const bool in = j < hi;
        al[j] = in ? al[j] : 1.0f;
        x[j] = in ? x[j] : -0.0f;
        dy[j] = in ? dy[j] : -0.0f;
        if constexpr (GATE != GDN_LRU_GATE_NONE) w[j] = in ? wj : 1.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < kLruC; ++j) {
      a = al[j] * a;
      b = fmaf(al[j], b, GATE == GDN_LRU_GATE_NONE ? x[j] : w[j] * x[j]);
      q = fmaf(a, dy[j], q);
    }
    const float am = a != a ? __uint_as_float(kPlainNaN) : a, mark = __uint_as_float(kLruMark);
    const float S0 = first && io.h0 && live ? io.h0[e] : 0.0f, K0 = last && io.dhT && live ? io.dhT[e] : 0.0f;
    start[threadIdx.x] = S0;
    behind[threadIdx.x] = K0;
    up[threadIdx.x] = first ? float2{mark, fmaf(a, S0, b)} : float2{am, b};
    down[threadIdx.x] = last ? float2{mark, fmaf(a, K0, q)} : float2{am, q};
  }
  __syncthreads();
  // the chains: up by the first slot's threads, down by the last slot's
  if (slot == 0)
    lru_chain<true, 4>(up + col, W, nch, 0.0f, [&](int s, float v) { start[s * W + col] = v; });
  if (slot == slots - 1)
    lru_chain<true, 4>(down + (nch - 1) * W + col, -W, nch, 0.0f,
                       [&](int s, float v) { behind[(nch - 1 - s) * W + col] = v; });
  __syncthreads();
  if (!has || !live) return;
  if constexpr (GATE != GDN_LRU_GATE_NONE) {
    // products w x are formed again rather than held over the chains in 32 registers more
#pragma unroll
    for (int j = 0; j < kLruC; ++j) asm volatile("" : "+v"(w[j]));
  }
  const float S = start[threadIdx.x];
  float K = behind[threadIdx.x];
  if (last && io.hT) io.hT[e] = fmaf(a, S, b);
  if (first) io.dh0[e] = fmaf(a, K, q);
  TX* o = io.o ? static_cast<TX*>(io.o) + c : nullptr;
  TX* dx = static_cast<TX*>(io.dx) + c;
  TG* dg = static_cast<TG*>(io.dg) + c;
  lru_outputs<GATE, false>(al, x, dy, w, S, K, hi, row, o, io.ldo, dx, io.lddx, dg, io.lddg);
}

// The cache's positions after a prefill (from 0) or a continuation: a launch
// of its own, since every block of the continuation reads them.
__global__ void k_lru_pos(LruIO io) {
  const int groups = (io.D + gdn::kLruGroup - 1) / gdn::kLruGroup;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (e >= static_cast<int64_t>(io.N) * groups) return;
  const int n = static_cast<int>(e / groups);
  int64_t t0, L;
  lru_rows(io, n, t0, L);
  const int p = io.resume ? lru_pos(io, n, static_cast<int>(e % groups) * gdn::kLruGroup) : 0;
  io.cache.pos[e] = static_cast<int32_t>((p + L) % kLruC);
}

__global__ void k_lru_cache_init(LruIO io) {
  const int64_t groups = (io.D + gdn::kLruGroup - 1) / gdn::kLruGroup;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < static_cast<int64_t>(io.N) * io.D;
       e += stride) {
    if (e < io.N * groups) io.cache.pos[e] = 0;
    io.cache.S[e] = io.h0 ? io.h0[e] : 0.0f;
    io.cache.A[e] = 1.0f;
    io.cache.B[e] = 0.0f;
  }
}

// One token of one sequence, 256 channels a block of one wave, which alone
// reads and advances their position counter.  Bound by HBM where large (1024
// sequences x 4096 channels, fp32 g: 18.5 us for 117 MB, 6.3 TB/s), by the launch
// where small (64 x 4096: 3.8 us).
template <typename TX, typename TG, int GATE>
__global__ __launch_bounds__(64) void k_lru_decode(LruIO io) {
  const int n = blockIdx.y;
  const int c0 = blockIdx.x * gdn::kLruGroup;
  const int p = lru_pos(io, n, c0);
  const bool full = p == kLruC - 1;
  const int64_t sn = static_cast<int64_t>(n) * io.D;
#pragma unroll
  for (int v = 0; v < gdn::kLruGroup / 64; ++v) {
    const int c = c0 + v * 64 + static_cast<int>(threadIdx.x);
    if (c < io.D) {
      const float g = ldin(static_cast<const TG*>(io.g) + n * io.ldg + c);
      const float x = ldin(static_cast<const TX*>(io.x) + n * io.ldx + c);
      float al;
      const float u = lru_input<GATE>(g, x, al);
      const float S = io.cache.S[sn + c];
      const float A = al * io.cache.A[sn + c];
      const float B = fmaf(al, io.cache.B[sn + c], u);
      const float h = fmaf(A, S, B);
      stout(static_cast<TX*>(io.o) + n * io.ldo + c, h);
      if (full) io.cache.S[sn + c] = h;
      io.cache.A[sn + c] = full ? 1.0f : A;
      io.cache.B[sn + c] = full ? 0.0f : B;
    }
  }
  if (threadIdx.x == 0) io.cache.pos[static_cast<int64_t>(n) * gridDim.x + blockIdx.x] = full ? 0 : p + 1;
}

// ---- three steps ---------------------------------------------------------------

// Sequence n's chunks have the slots from cu[n] / 32 + 2 n on: floor(b / 32) -
// floor(a / 32) + 2 >= ceil((31 + b - a) / 32), so they end before the next
// sequence's also where the first chunk was begun by the cache.
__device__ __forceinline__ int64_t lru_slot0(const LruIO& io, int n) {
  int64_t a = io.cu[n];
  a = a < 0 ? 0 : (a > io.T ? io.T : a);
  return a / kLruC + 2 * static_cast<int64_t>(n);
}

// The chunk of a slot: its sequence, the row of its place 0 and the places
// [lo, hi) that hold tokens.  False for a slot that no chunk uses.
struct LruChunk {
  int n, lo, hi;
  int64_t row;
};
__device__ __forceinline__ bool lru_chunk(const LruIO& io, int64_t slot, LruChunk& k) {
  // the last sequence that starts at or before the slot, by a whole wave: a place
  // for each lane, so that 64 sequences take one trip to memory and 4096 two
  const int lane = threadIdx.x & 63;
  int lo = 0;
  for (int n = io.N; n > 1;) {
    const int step = (n + 63) >> 6, at = lane * step;
    const int starts = __popcll(__ballot(at < n && lru_slot0(io, lo + at) <= slot));
    const int skip = starts > 1 ? (starts - 1) * step : 0;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  k.n = lo;
  int64_t t0, L;
  lru_rows(io, lo, t0, L);
  const int p0 = io.resume ? lru_pos(io, lo, 0) : 0;
  const int64_t tb = (slot - lru_slot0(io, lo)) * kLruC - p0;
  // An empty sequence may stand inside a chunk (tb < 0); a slot in front of its sequence's first (tb < -p0) comes from
  // a device copy of cu_seqlens that is not the host's: one that starts behind row 0 or steps back.
  if (L == 0 || tb < -p0 || tb >= L) return false;
  k.row = t0 + tb;
  k.lo = tb < 0 ? static_cast<int>(-tb) : 0;
  k.hi = L - tb < kLruC ? static_cast<int>(L - tb) : kLruC;
  return true;
}
// Row of place i, or the nearest that holds a token.
template <bool WHOLE>
__device__ __forceinline__ int64_t lru_row(const LruChunk& k, int i) {
  return k.row + (WHOLE ? i : (i < k.lo ? k.lo : (i >= k.hi ? k.hi - 1 : i)));
}

// The wave's slot and the lane's channel; false past the slots.
__device__ __forceinline__ bool lru_unit(const LruIO& io, int64_t& slot, int& c) {
  const int per = 256 / io.cw;
  const int groups = (io.D + io.cw - 1) / io.cw;
  const int64_t b = blockIdx.x;
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x) / io.cw;  // io.cw is 64 at least
  slot = b / groups * per + sub;
  c = static_cast<int>(b % groups) * io.cw + static_cast<int>(threadIdx.x) - sub * io.cw;
  return slot < io.slots;
}

template <typename TX, typename TG, int GATE, bool GRAD, bool WHOLE>
__device__ __forceinline__ void lru_fold(const LruIO& io, const LruChunk& k, int64_t slot, int c) {
  const TX* x = static_cast<const TX*>(io.x) + c;
  const TG* g = static_cast<const TG*>(io.g) + c;
  const TX* dO = static_cast<const TX*>(io.dO) + c;
  float G[kLruC], X[kLruC], Y[GRAD ? kLruC : 1];
#pragma unroll
  for (int i = 0; i < kLruC; ++i) {
    const int64_t t = lru_row<WHOLE>(k, i);
    G[i] = ldin(g + t * io.ldg);
    X[i] = ldin(x + t * io.ldx);
    if constexpr (GRAD) Y[i] = ldin(dO + t * io.lddo);
  }
  float a = 1.0f, b = 0.0f, q = 0.0f;
  if (!WHOLE && k.lo > 0) {
    // the cache's composition, kept for k_lru_apply: k_lru_chain moves the cache on
    a = io.cache.A[static_cast<int64_t>(k.n) * io.D + c];
    b = io.cache.B[static_cast<int64_t>(k.n) * io.D + c];
    io.keep[2 * static_cast<int64_t>(k.n) * io.D + c] = a;
    io.keep[(2 * static_cast<int64_t>(k.n) + 1) * io.D + c] = b;
  }
#pragma unroll
  for (int i = 0; i < kLruC; ++i) {
    float al;
    float u = lru_input<GATE>(G[i], X[i], al);
    if constexpr (!WHOLE) {
      // places outside the rows change nothing: 1 a = a, fma(1, b, -0) = b
      const bool in = i >= k.lo && i < k.hi;
      al = in ? al : 1.0f;
      u = in ? u : -0.0f;
      if constexpr (GRAD) Y[i] = in ? Y[i] : -0.0f;
    }
    a = al * a;
    b = fmaf(al, b, u);
    if constexpr (GRAD) q = fmaf(a, Y[i], q);
  }
  const int64_t at = slot * io.D + c;
  io.wA[at] = a;
  io.wB[at] = b;
  if constexpr (GRAD) io.wQ[at] = q;
}
template <typename TX, typename TG, int GATE, bool GRAD>
__global__ __launch_bounds__(256) void k_lru_fold(LruIO io) {
  int64_t slot;
  int c;
  LruChunk k;
  if (!lru_unit(io, slot, c) || !lru_chunk(io, slot, k) || c >= io.D) return;
  if (k.lo == 0 && k.hi == kLruC)
    lru_fold<TX, TG, GATE, GRAD, true>(io, k, slot, c);
  else
    lru_fold<TX, TG, GATE, GRAD, false>(io, k, slot, c);
}

// The chains over a sequence's chunks, up to ROWS chunks of W channels a block at
// a time through LDS: forward S -> A S + B (wB then holds the states at the
// chunks' starts), backward (grid.y = 1) K -> A K + Q (wQ then holds the gradients
// of the states behind the chunks' ends).  Also what a sequence ends with: hT,
// the cache, dh0.  Bound by latency: a round is a trip to memory and back, and
// ROWS dependent fma's.
template <int W, int ROWS>
__global__ __launch_bounds__(256) void k_lru_chain(LruIO io) {
  __shared__ float2 agg[ROWS * W];
  const int tiles = (io.D + W - 1) / W;
  const int n = blockIdx.x / tiles;
  const int c0 = (blockIdx.x % tiles) * W;
  int64_t t0, L;
  lru_rows(io, n, t0, L);
  const int64_t sn = static_cast<int64_t>(n) * io.D;
  const bool up = blockIdx.y == 0;
  const int p0 = io.resume ? lru_pos(io, n, 0) : 0;
  const int64_t nch = L > 0 ? (p0 + L + kLruC - 1) / kLruC : 0;
  const int col = threadIdx.x & (W - 1), row = threadIdx.x / W;
  const int c = c0 + col;
  const bool live = c < io.D;
  const int64_t base = lru_slot0(io, n) * io.D + c;
  float* w = up ? io.wB : io.wQ;
  float S = 0.0f;
  const bool folds = row == 0 && live;
  if (folds) S = up ? (io.resume ? io.cache.S[sn + c] : (io.h0 ? io.h0[sn + c] : 0.0f)) : (io.dhT ? io.dhT[sn + c] : 0.0f);
  float before = S;  // the state at the start of the last chunk
  constexpr int kRowsStep = 256 / W, kPer = ROWS / kRowsStep;
  float2 in[kPer];
  // rows in the chain's order: from the first chunk up, or from the last down
  auto load = [&](int64_t r0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = r0 + row + i * kRowsStep;
      if (live && r < nch) {
        const int64_t at = base + (up ? r : nch - 1 - r) * io.D;
        in[i] = float2{io.wA[at], w[at]};
      }
    }
  };
  load(0);
  for (int64_t r0 = 0; r0 < nch; r0 += ROWS) {
    const int m = static_cast<int>(nch - r0 < ROWS ? nch - r0 : ROWS);
#pragma unroll
    for (int i = 0; i < kPer; ++i) agg[(row + i * kRowsStep) * W + col] = in[i];
    if (up && live && r0 + m == nch && io.cache.S) {
      // the last chunk as the cache keeps it
      const bool full = (p0 + L) % kLruC == 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (row + i * kRowsStep == m - 1) {
          io.cache.A[sn + c] = full ? 1.0f : in[i].x;
          io.cache.B[sn + c] = full ? 0.0f : in[i].y;
        }
      }
    }
    __syncthreads();
    load(r0 + ROWS);  // in flight beside the chain
    if (folds)
      S = lru_chain<false, 8>(agg + col, W, m, S, [&](int s, float v) {
        agg[s * W + col].x = v;
        before = v;
      });
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = r0 + row + i * kRowsStep;
      if (live && r < nch) w[base + (up ? r : nch - 1 - r) * io.D] = agg[(row + i * kRowsStep) * W + col].x;
    }
    __syncthreads();
  }
  if (!folds) return;
  if (!up) {
    io.dh0[sn + c] = S;
    return;
  }
  if (L == 0) {
    lru_empty(io, sn + c);
    return;
  }
  if (io.hT) io.hT[sn + c] = S;
  if (io.cache.S) io.cache.S[sn + c] = (p0 + L) % kLruC == 0 ? S : before;
}

template <typename TX, typename TG, int GATE, bool WHOLE>
__device__ __forceinline__ void lru_apply(const LruIO& io, const LruChunk& k, int64_t slot, int c) {
  const TX* x = static_cast<const TX*>(io.x) + c;
  const TG* g = static_cast<const TG*>(io.g) + c;
  TX* o = static_cast<TX*>(io.o) + c;
  float G[kLruC], X[kLruC];
  const float S = io.wB[slot * io.D + c];
#pragma unroll
  for (int i = 0; i < kLruC; ++i) {
    const int64_t t = lru_row<WHOLE>(k, i);
    G[i] = ldin(g + t * io.ldg);
    X[i] = ldin(x + t * io.ldx);
  }
  float a = 1.0f, b = 0.0f;
  if (!WHOLE && k.lo > 0) {
    a = io.keep[2 * static_cast<int64_t>(k.n) * io.D + c];
    b = io.keep[(2 * static_cast<int64_t>(k.n) + 1) * io.D + c];
  }
#pragma unroll
  for (int i = 0; i < kLruC; ++i) {
    if (WHOLE || (i >= k.lo && i < k.hi)) {
      float al;
      const float u = lru_input<GATE>(G[i], X[i], al);
      a = al * a;
      b = fmaf(al, b, u);
      stout(o + (k.row + i) * io.ldo, fmaf(a, S, b));
    }
  }
}
template <typename TX, typename TG, int GATE>
__global__ __launch_bounds__(256) void k_lru_apply(LruIO io) {
  int64_t slot;
  int c;
  LruChunk k;
  if (!lru_unit(io, slot, c) || !lru_chunk(io, slot, k) || c >= io.D) return;
  if (k.lo == 0 && k.hi == kLruC)
    lru_apply<TX, TG, GATE, true>(io, k, slot, c);
  else
    lru_apply<TX, TG, GATE, false>(io, k, slot, c);
}

template <typename TX, typename TG, int GATE, bool WHOLE>
__device__ __forceinline__ void lru_grad(const LruIO& io, const LruChunk& k, int64_t slot, int c) {
  const TX* x = static_cast<const TX*>(io.x) + c;
  const TG* g = static_cast<const TG*>(io.g) + c;
  const TX* dO = static_cast<const TX*>(io.dO) + c;
  TX* o = io.o ? static_cast<TX*>(io.o) + c : nullptr;
  TX* dx = static_cast<TX*>(io.dx) + c;
  TG* dg = static_cast<TG*>(io.dg) + c;
  const float S = io.wB[slot * io.D + c];
  const float K = io.wQ[slot * io.D + c];
  float al[kLruC], e[kLruC], dy[kLruC], w[GATE == GDN_LRU_GATE_NONE ? 1 : kLruC];
#pragma unroll
  for (int i = 0; i < kLruC; ++i) {
    const int64_t t = lru_row<WHOLE>(k, i);
    al[i] = ldin(g + t * io.ldg);
    e[i] = ldin(x + t * io.ldx);
    dy[i] = ldin(dO + t * io.lddo);
  }
#pragma unroll
  for (int i = 0; i < kLruC; ++i) {
    const float wi = lru_weight<GATE>(al[i], al[i]);
    if constexpr (GATE != GDN_LRU_GATE_NONE) w[i] = wi;
  }
  lru_outputs<GATE, WHOLE>(al, e, dy, w, S, K, k.hi, k.row, o, io.ldo, dx, io.lddx, dg, io.lddg);
}
template <typename TX, typename TG, int GATE>
__global__ __launch_bounds__(256) void k_lru_grad(LruIO io) {
  int64_t slot;
  int c;
  LruChunk k;
  if (!lru_unit(io, slot, c) || !lru_chunk(io, slot, k) || c >= io.D) return;
  if (k.hi == kLruC)
    lru_grad<TX, TG, GATE, true>(io, k, slot, c);
  else
    lru_grad<TX, TG, GATE, false>(io, k, slot, c);
}

// ---- host side ----------------------------------------------------------------

// Calls f.template operator()<TX, TG, GATE>() for the shape's types and gate.
template <typename TX, typename TG, typename F>
int lru_dispatch_gate(const gdn_lru_shape_t* s, F&& f) {
  if (s->gate == GDN_LRU_GATE_NONE) return f.template operator()<TX, TG, GDN_LRU_GATE_NONE>();
  if (s->gate == GDN_LRU_GATE_COMPLEMENT) return f.template operator()<TX, TG, GDN_LRU_GATE_COMPLEMENT>();
  return f.template operator()<TX, TG, GDN_LRU_GATE_NORM>();
}
template <typename F>
int lru_dispatch(const gdn_lru_shape_t* s, F&& f) {
  if (s->in_dtype == GDN_BF16)
    return s->g_dtype == GDN_BF16 ? lru_dispatch_gate<bf16_t, bf16_t>(s, f) : lru_dispatch_gate<bf16_t, float>(s, f);
  return s->g_dtype == GDN_BF16 ? lru_dispatch_gate<float, bf16_t>(s, f) : lru_dispatch_gate<float, float>(s, f);
}

// Checks and resolves what the packed calls share.
int lru_common(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_dev, const int32_t** cu_host,
               std::vector<int32_t>& buf, hipStream_t st, LruIO* io, int64_t* longest, int64_t* chunks) {
  int rc = gdn::check_lru_shape(shape);
  if (rc != GDN_OK) return rc;
  if (n_seqs < 0 || !cu_dev) return GDN_ERR_INVALID_ARG;
  try {
    rc = host_cu(cu_dev, *cu_host, n_seqs, st, buf, cu_host);
  } catch (const std::bad_alloc&) {
    rc = GDN_ERR_INVALID_ARG;  // an n_seqs whose prefix the host cannot hold
  }
  if (rc != GDN_OK) return rc;
  gdn::Counts cnt;
  if ((rc = gdn::count_chunks(*cu_host, n_seqs, kLruC, &cnt)) != GDN_OK) return rc;
  int64_t most = 0;
  for (int32_t n = 0; n < n_seqs; ++n) {
    const int64_t len = static_cast<int64_t>((*cu_host)[n + 1]) - (*cu_host)[n];
    most = len > most ? len : most;
  }
  *longest = most;
  *chunks = cnt.chunks;
  io->cu = cu_dev;
  io->N = n_seqs;
  io->D = shape->D;
  io->gate = shape->gate;
  io->T = cnt.T;
  return GDN_OK;
}

// Workspace of the three steps: A, B, for the trainer Q, and a cache's A and B.
size_t lru_ws_bytes(int64_t D, int64_t N, int64_t T, bool grad) {
  const int64_t floats = gdn::lru_slots(T, N) * D * (grad ? 3 : 2) + (grad ? 0 : 2 * N * D);
  return (static_cast<size_t>(floats) * sizeof(float) / gdn::kAlign + 4) * gdn::kAlign;
}
void lru_ws(LruIO* io, void* ws, bool grad) {
  io->slots = gdn::lru_slots(io->T, io->N);
  const int64_t step = (io->slots * io->D + 63) / 64 * 64;  // floats, 256 bytes
  io->wA = static_cast<float*>(ws);
  io->wB = io->wA + step;
  io->wQ = grad ? io->wB + step : nullptr;
  io->keep = grad ? nullptr : io->wB + step;
}
// Lanes over channels and blocks of the steps over all chunks.
int64_t lru_units(LruIO* io) {
  io->cw = 64;
  while (io->cw < 256 && io->cw < io->D) io->cw *= 2;
  const int64_t per = 256 / io->cw, groups = (io->D + io->cw - 1) / io->cw;
  return (io->slots + per - 1) / per * groups;
}
// The chain's launch, of the width that gdn::lru_chain_width gives.
void lru_launch_chain(const LruIO& io, int width, int directions, hipStream_t st) {
  Timed t_("k_lru_chain", st);
  const dim3 grid(static_cast<unsigned>(gdn::lru_chain_blocks(io.N, io.D, width)), directions);
  if (width == 16)
    hipLaunchKernelGGL((k_lru_chain<16, 512>), grid, dim3(256), 0, st, io);
  else if (width == 256)
    hipLaunchKernelGGL((k_lru_chain<256, 8>), grid, dim3(256), 0, st, io);
  else
    hipLaunchKernelGGL((k_lru_chain<32, 128>), grid, dim3(256), 0, st, io);
}
bool lru_fits(int64_t threads) { return threads < gdn::kLaunchThreads; }

int lru_prefill_entry(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_dev, const int32_t* cu_host,
                      const void* x, int64_t ldx, const void* g, int64_t ldg, const float* h0, void* o, int64_t ldo,
                      float* hT, gdn_lru_cache_t* cache, bool resume, void* ws, size_t ws_bytes, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  LruIO io{};
  std::vector<int32_t> buf;
  int64_t longest = 0, chunks = 0;
  int rc = gdn::check_lru_shape(shape);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({x, g, h0, o, hT, ws})) return GDN_ERR_INVALID_ARG;
  if ((cache || resume) && (rc = gdn::check_lru_cache(cache)) != GDN_OK) return rc;
  io.ldx = gdn::row_stride(ldx, shape->D);
  io.ldg = gdn::row_stride(ldg, shape->D);
  io.ldo = gdn::row_stride(ldo, shape->D);
  if (io.ldx < 0 || io.ldg < 0 || io.ldo < 0) return GDN_ERR_INVALID_ARG;
  if ((rc = lru_common(shape, n_seqs, cu_dev, &cu_host, buf, st, &io, &longest, &chunks)) != GDN_OK) return rc;
  if (io.T > 0 && (!x || !g || !o)) return GDN_ERR_INVALID_ARG;
  if (io.T > GDN_LRU_SMALL && (!ws || ws_bytes < lru_ws_bytes(shape->D, n_seqs, io.T, false))) return GDN_ERR_WORKSPACE;
  if (n_seqs == 0) return GDN_OK;
  io.x = x; io.g = g; io.h0 = h0; io.o = o; io.hT = hT; io.resume = resume;
  if (cache) io.cache = *cache;
  const bool three = gdn::lru_plan(cu_host, n_seqs, chunks, io.D, longest, resume, &io.plan);
  int threads = 256, width = 0;
  int64_t blocks;
  if (three) {
    lru_ws(&io, ws, false);
    blocks = lru_units(&io);
    width = gdn::lru_chain_width(n_seqs, io.D, longest, 1);
  } else {
    threads = io.plan.threads;
    io.tiles = (io.D + io.plan.lps - 1) / io.plan.lps;
    blocks = lru_blocks(io.plan.units, io.tiles);
  }
  if (!lru_fits(blocks * threads) || (three && !width)) return GDN_ERR_UNSUPPORTED;
  lru_dispatch(shape, [&]<typename TX, typename TG, int GATE>() {
    const dim3 grid(static_cast<unsigned>(blocks)), block(threads);
    if (!three) {
      Timed t_("k_lru_fwd", st);
      hipLaunchKernelGGL((k_lru_fwd<TX, TG, GATE>), grid, block, 0, st, io);
      return GDN_OK;
    }
    {
      Timed t_("k_lru_fold", st);
      hipLaunchKernelGGL((k_lru_fold<TX, TG, GATE, false>), grid, block, 0, st, io);
    }
    lru_launch_chain(io, width, 1, st);
    Timed t_("k_lru_apply", st);
    hipLaunchKernelGGL((k_lru_apply<TX, TG, GATE>), grid, block, 0, st, io);
    return GDN_OK;
  });
  if (cache) {
    const int64_t e = static_cast<int64_t>(n_seqs) * ((io.D + gdn::kLruGroup - 1) / gdn::kLruGroup);
    Timed t_("k_lru_pos", st);
    hipLaunchKernelGGL(k_lru_pos, dim3(static_cast<unsigned>((e + 255) / 256)), dim3(256), 0, st, io);
  }
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // namespace

extern "C" {

int gdn_lru_cache_init(const gdn_lru_shape_t* shape, int32_t n_seqs, const float* h0, gdn_lru_cache_t* cache,
                       void* stream) {
  int rc = gdn::check_lru_shape(shape);
  if (rc != GDN_OK) return rc;
  if (n_seqs < 0 || !gdn::aligned16({h0})) return GDN_ERR_INVALID_ARG;
  if ((rc = gdn::check_lru_cache(cache)) != GDN_OK) return rc;
  if (n_seqs == 0) return GDN_OK;
  LruIO io{};
  io.N = n_seqs; io.D = shape->D; io.h0 = h0; io.cache = *cache;
  const int64_t want = (static_cast<int64_t>(n_seqs) * shape->D + 255) / 256, blocks = want < 65536 ? want : 65536;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Timed t_("k_lru_cache_init", st);
  hipLaunchKernelGGL(k_lru_cache_init, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, io);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_lru_prefill(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                    const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g, int64_t ldg,
                    const float* h0, void* o, int64_t ldo, float* hT, gdn_lru_cache_t* cache, void* ws, size_t ws_bytes,
                    void* stream) {
  return lru_prefill_entry(shape, n_seqs, cu_seqlens_dev, cu_seqlens_host, x, ldx, g, ldg, h0, o, ldo, hT, cache, false,
                           ws, ws_bytes, stream);
}

int gdn_lru_prefill_continue(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                             const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g, int64_t ldg,
                             gdn_lru_cache_t* cache, void* o, int64_t ldo, float* hT, void* ws, size_t ws_bytes,
                             void* stream) {
  return lru_prefill_entry(shape, n_seqs, cu_seqlens_dev, cu_seqlens_host, x, ldx, g, ldg, nullptr, o, ldo, hT, cache,
                           true, ws, ws_bytes, stream);
}

int gdn_lru_decode_step(const gdn_lru_shape_t* shape, int32_t n_seqs, const void* x, int64_t ldx, const void* g,
                        int64_t ldg, gdn_lru_cache_t* cache, void* o, int64_t ldo, void* stream) {
  int rc = gdn::check_lru_shape(shape);
  if (rc != GDN_OK) return rc;
  if (n_seqs < 0 || !gdn::aligned16({x, g, o})) return GDN_ERR_INVALID_ARG;
  if ((rc = gdn::check_lru_cache(cache)) != GDN_OK) return rc;
  if (n_seqs > 0 && (!x || !g || !o)) return GDN_ERR_INVALID_ARG;
  LruIO io{};
  io.ldx = gdn::row_stride(ldx, shape->D);
  io.ldg = gdn::row_stride(ldg, shape->D);
  io.ldo = gdn::row_stride(ldo, shape->D);
  if (io.ldx < 0 || io.ldg < 0 || io.ldo < 0) return GDN_ERR_INVALID_ARG;
  if (n_seqs > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y
  if (n_seqs == 0) return GDN_OK;
  io.x = x; io.g = g; io.o = o; io.cache = *cache;
  io.N = n_seqs; io.D = shape->D; io.gate = shape->gate;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return lru_dispatch(shape, [&]<typename TX, typename TG, int GATE>() {
    Timed t_("k_lru_decode", st);
    const dim3 grid((io.D + gdn::kLruGroup - 1) / gdn::kLruGroup, n_seqs);
    hipLaunchKernelGGL((k_lru_decode<TX, TG, GATE>), grid, dim3(64), 0, st, io);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  });
}

size_t gdn_lru_workspace_bytes(const gdn_lru_shape_t* shape, int32_t n_seqs, int64_t total_tokens, int32_t op) {
  if (gdn::check_lru_shape(shape) != GDN_OK || n_seqs < 0 || total_tokens < 0 || total_tokens > INT32_MAX) return 0;
  if (op != GDN_OP_PREFILL && op != GDN_OP_PREFILL_CONTINUE && op != GDN_OP_FWD_BWD) return 0;
  return lru_ws_bytes(shape->D, n_seqs, total_tokens, op == GDN_OP_FWD_BWD);
}

int gdn_lru_fwd_bwd(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                    const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g, int64_t ldg,
                    const float* h0, const void* dO, int64_t lddo, const float* dhT, void* o, int64_t ldo, float* hT,
                    void* dx, int64_t lddx, void* dg, int64_t lddg, float* dh0, void* ws, size_t ws_bytes,
                    void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  LruIO io{};
  std::vector<int32_t> buf;
  int64_t longest = 0, chunks = 0;
  int rc = gdn::check_lru_shape(shape);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({x, g, h0, dO, dhT, o, hT, dx, dg, dh0, ws})) return GDN_ERR_INVALID_ARG;
  if (n_seqs > 0 && !dh0) return GDN_ERR_INVALID_ARG;
  io.ldx = gdn::row_stride(ldx, shape->D);
  io.ldg = gdn::row_stride(ldg, shape->D);
  io.ldo = gdn::row_stride(ldo, shape->D);
  io.lddo = gdn::row_stride(lddo, shape->D);
  io.lddx = gdn::row_stride(lddx, shape->D);
  io.lddg = gdn::row_stride(lddg, shape->D);
  if (io.ldx < 0 || io.ldg < 0 || io.ldo < 0 || io.lddo < 0 || io.lddx < 0 || io.lddg < 0) return GDN_ERR_INVALID_ARG;
  if ((rc = lru_common(shape, n_seqs, cu_seqlens_dev, &cu_seqlens_host, buf, st, &io, &longest, &chunks)) != GDN_OK) return rc;
  if (io.T > 0 && (!x || !g || !dO || !dx || !dg)) return GDN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < lru_ws_bytes(shape->D, n_seqs, io.T, true)) return GDN_ERR_WORKSPACE;
  if (n_seqs == 0) return GDN_OK;
  io.x = x; io.g = g; io.h0 = h0; io.dO = dO; io.dhT = dhT; io.o = o; io.hT = hT; io.dx = dx; io.dg = dg; io.dh0 = dh0;
  if (gdn::lru_train_plan(cu_seqlens_host, n_seqs, chunks, io.D, longest, &io.plan)) {
    io.tiles = (io.D + io.plan.lps - 1) / io.plan.lps;
    const int64_t items = lru_blocks(io.plan.units, io.tiles);
    if (!lru_fits(items * io.plan.threads)) return GDN_ERR_UNSUPPORTED;
    return lru_dispatch(shape, [&]<typename TX, typename TG, int GATE>() {
      Timed t_("k_lru_train", st);
      hipLaunchKernelGGL((k_lru_train<TX, TG, GATE>), dim3(static_cast<unsigned>(items)), dim3(io.plan.threads), 0, st, io);
      return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    });
  }
  lru_ws(&io, ws, true);
  const int64_t blocks = lru_units(&io);
  const int width = gdn::lru_chain_width(n_seqs, io.D, longest, 2);
  if (!lru_fits(blocks * 256) || !width) return GDN_ERR_UNSUPPORTED;
  return lru_dispatch(shape, [&]<typename TX, typename TG, int GATE>() {
    const dim3 grid(static_cast<unsigned>(blocks)), block(256);
    {
      Timed t_("k_lru_fold", st);
      hipLaunchKernelGGL((k_lru_fold<TX, TG, GATE, true>), grid, block, 0, st, io);
    }
    lru_launch_chain(io, width, 2, st);
    Timed t_("k_lru_grad", st);
    hipLaunchKernelGGL((k_lru_grad<TX, TG, GATE>), grid, block, 0, st, io);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  });
}

}  // extern "C"
