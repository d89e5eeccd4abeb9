// Gated linear recurrence (include/gdn.h): kernels and C ABI.  Part of
// gdn_library.hip.
//
// Per channel, h_t = alpha_t h_{t-1} + u_t with u = b x.  A chunk of 32 tokens
// is the map h -> A h + B; its running composition (A_p, B_p) needs no state,
// so every chunk of a sequence is composed at once, the states at the chunks'
// starts follow one another with one fma per chunk, and h_p = fma(A_p, S, B_p).
// The same operations in the same order run in decode, one token at a time.
//
// Bound: HBM.  An element takes 6 to 12 bytes and about 20 vector
// instructions.

namespace {

constexpr int kLruC = GDN_LRU_CHUNK;
constexpr int kLruThreads = 512;  // most threads of a scan block

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
  int lps;    // lanes per chunk: a block's channel tile is lps times a lane's channels
  int tiles;  // channel tiles
  // trainer
  const void* dO;
  const float* dhT;
  void* dx;
  void* dg;
  float* dh0;
  float* states;  // [T / 32 + N][D] chunk-start states
  int64_t lddo, lddx, lddg;
};

__device__ __forceinline__ void stout(float* p, float x) { *p = x; }
__device__ __forceinline__ void stout(bf16_t* p, float x) {
  *p = static_cast<bf16_t>(pack_bf16(x, 0.0f));  // round to nearest even
}

// alpha and u = b x of one element.
__device__ __forceinline__ void lru_gate(int gate, float g, float x, float& a, float& u) {
  a = expf(g);
  if (gate == GDN_LRU_GATE_NONE) {
    u = x;
  } else if (gate == GDN_LRU_GATE_COMPLEMENT) {
    u = -expm1f(g) * x;
  } else {
    u = sqrtf(fmaxf(-expm1f(2.0f * g), 0.0f)) * x;
  }
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

// Block -> (sequence, channel tile).  Groups of four neighbouring tiles of a
// sequence go to one XCD (blocks are dealt to the eight XCDs in turn), where
// tiles narrower than a cache line share it in that XCD's L2.
__device__ __forceinline__ bool lru_item(const LruIO& io, int& n, int& tile) {
  const int64_t b = blockIdx.x;
  const int64_t xcd = b & 7, j = b >> 3;
  const int64_t group = (j >> 2) * 8 + xcd;
  const int gps = (io.tiles + 3) >> 2;  // groups per sequence
  const int64_t seq = group / gps;
  tile = static_cast<int>(group - seq * gps) * 4 + static_cast<int>(j & 3);
  n = static_cast<int>(seq);
  return seq < io.N && tile < io.tiles;
}
int64_t lru_blocks(int64_t N, int tiles) {
  const int64_t groups = N * ((tiles + 3) / 4);
  return (groups + 7) / 8 * 8 * 4;
}

// Two channels per lane where rows are evenly aligned, else one at a time.
template <typename TX, typename TG, int V>
__global__ __launch_bounds__(kLruThreads) void k_lru_fwd(LruIO io) {
  __shared__ float2 agg[kLruThreads * V];  // [slot][channel of the tile]
  __shared__ float start[kLruThreads * V];
  int n, tile;
  if (!lru_item(io, n, tile)) return;
  int64_t t0, L;
  lru_rows(io, n, t0, L);
  const int W = io.lps * V;
  const int slots = blockDim.x / io.lps;
  const int slot = threadIdx.x / io.lps;
  const int lc = (threadIdx.x - slot * io.lps) * V;  // channel inside the tile
  const int c = tile * W + lc;
  const bool live = c < io.D;  // (D is even where V = 2)
  const int cc = live ? c : io.D - V;
  const TX* x = static_cast<const TX*>(io.x) + t0 * io.ldx + cc;
  const TG* g = static_cast<const TG*>(io.g) + t0 * io.ldg + cc;
  TX* o = io.o ? static_cast<TX*>(io.o) + t0 * io.ldo + cc : nullptr;
  const int64_t sn = static_cast<int64_t>(n) * io.D;
  const int p0 = io.resume ? lru_pos(io, n, tile * W < io.D ? tile * W : 0) : 0;
  const int64_t nch = (p0 + L + kLruC - 1) / kLruC;
  // the chain over chunks, one thread per channel of the tile
  const int fc = tile * W + static_cast<int>(threadIdx.x);
  const bool folds = static_cast<int>(threadIdx.x) < W && fc < io.D;
  float S = 0.0f;
  if (folds) S = io.resume ? io.cache.S[sn + fc] : (io.h0 ? io.h0[sn + fc] : 0.0f);
  if (L == 0) {
    if (folds) {
      if (io.resume) {
        if (io.hT) io.hT[sn + fc] = fmaf(io.cache.A[sn + fc], S, io.cache.B[sn + fc]);
      } else {
        if (io.hT) io.hT[sn + fc] = S;
        if (io.cache.S) {
          io.cache.S[sn + fc] = S;
          io.cache.A[sn + fc] = 1.0f;
          io.cache.B[sn + fc] = 0.0f;
        }
      }
    }
    return;
  }
  for (int64_t cb = 0; cb < nch; cb += slots) {
    const int64_t ch = cb + slot;
    const bool has = ch < nch;
    const int64_t tb = ch * kLruC - p0;  // row of the chunk's place 0
    const int lo = has && tb < 0 ? static_cast<int>(-tb) : 0;
    const int64_t left = L - tb;
    const int hi = has ? (left < kLruC ? static_cast<int>(left) : kLruC) : 0;
    float A[kLruC][V], B[kLruC][V];
    if (has) {
#pragma unroll
      for (int i = 0; i < kLruC; ++i) {
        const int ii = i < lo ? lo : (i >= hi ? hi - 1 : i);  // a row of this chunk
        const int64_t t = tb + ii;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          A[i][v] = ldin(g + t * io.ldg + v);
          B[i][v] = ldin(x + t * io.ldx + v);
        }
      }
      float a[V], b[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        a[v] = 1.0f;
        b[v] = 0.0f;
        if (lo > 0) {
          a[v] = io.cache.A[sn + cc + v];
          b[v] = io.cache.B[sn + cc + v];
        }
      }
#pragma unroll
      for (int i = 0; i < kLruC; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float al, u;
          lru_gate(io.gate, A[i][v], B[i][v], al, u);
          // places outside the rows change nothing: a 1 = a, fma(1, b, -0) = b
          const bool in = i >= lo && i < hi;
          al = in ? al : 1.0f;
          u = in ? u : -0.0f;
          a[v] = al * a[v];
          b[v] = fmaf(al, b[v], u);
          A[i][v] = a[v];
          B[i][v] = b[v];
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) agg[slot * W + lc + v] = float2{A[kLruC - 1][v], B[kLruC - 1][v]};
    }
    __syncthreads();
    if (folds) {
      const int m = static_cast<int>(nch - cb < slots ? nch - cb : slots);
      for (int s = 0; s < m; ++s) {
        const float2 ab = agg[s * W + threadIdx.x];
        start[s * W + threadIdx.x] = S;
        S = fmaf(ab.x, S, ab.y);
      }
    }
    __syncthreads();
    if (has && live) {
      float st[V];
#pragma unroll
      for (int v = 0; v < V; ++v) st[v] = start[slot * W + lc + v];
      if (o) {
#pragma unroll
        for (int i = 0; i < kLruC; ++i) {
          if (i >= lo && i < hi) {
#pragma unroll
            for (int v = 0; v < V; ++v) stout(o + (tb + i) * io.ldo + v, fmaf(A[i][v], st[v], B[i][v]));
          }
        }
      }
      if (ch == nch - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float h = fmaf(A[kLruC - 1][v], st[v], B[kLruC - 1][v]);
          if (io.hT) io.hT[sn + c + v] = h;
          if (io.cache.S) {
            const bool full = hi == kLruC;
            io.cache.S[sn + c + v] = full ? h : st[v];
            io.cache.A[sn + c + v] = full ? 1.0f : A[kLruC - 1][v];
            io.cache.B[sn + c + v] = full ? 0.0f : B[kLruC - 1][v];
          }
        }
      }
    }
  }
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
  const int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t groups = (io.D + gdn::kLruGroup - 1) / gdn::kLruGroup;
  if (e < io.N * groups) io.cache.pos[e] = 0;
  if (e >= static_cast<int64_t>(io.N) * io.D) return;
  io.cache.S[e] = io.h0 ? io.h0[e] : 0.0f;
  io.cache.A[e] = 1.0f;
  io.cache.B[e] = 0.0f;
}

// One token of one sequence, 256 channels a block of one wave, which alone
// reads and advances their position counter.
template <typename TX, typename TG>
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
      float al, u;
      lru_gate(io.gate, g, x, al, u);
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

// Trainer: a sweep forward over the rounds of chunks (as k_lru_fwd, keeping
// the chunk-start states), then one backward.  Going back, a chunk maps the
// gradient K of the state behind its last token to that in front of its first
// token, K -> P K + Q, so the same three steps run in reverse.
template <typename TX, typename TG>
__global__ __launch_bounds__(kLruThreads) void k_lru_bwd(LruIO io) {
  __shared__ float2 agg[kLruThreads];
  __shared__ float start[kLruThreads];
  int n, tile;
  if (!lru_item(io, n, tile)) return;
  int64_t t0, L;
  lru_rows(io, n, t0, L);
  const int W = io.lps;
  const int slots = blockDim.x / W;
  const int slot = threadIdx.x / W;
  const int lc = threadIdx.x - slot * W;
  const int c = tile * W + lc;
  const bool live = c < io.D;
  const int cc = live ? c : io.D - 1;
  const TX* x = static_cast<const TX*>(io.x) + t0 * io.ldx + cc;
  const TG* g = static_cast<const TG*>(io.g) + t0 * io.ldg + cc;
  const TX* dO = static_cast<const TX*>(io.dO) + t0 * io.lddo + cc;
  TX* o = io.o ? static_cast<TX*>(io.o) + t0 * io.ldo + cc : nullptr;
  TX* dx = static_cast<TX*>(io.dx) + t0 * io.lddx + cc;
  TG* dg = static_cast<TG*>(io.dg) + t0 * io.lddg + cc;
  const int64_t sn = static_cast<int64_t>(n) * io.D;
  const int64_t nch = (L + kLruC - 1) / kLruC;
  const int fc = tile * W + static_cast<int>(threadIdx.x);
  const bool folds = static_cast<int>(threadIdx.x) < W && fc < io.D;
  float S = 0.0f, K = 0.0f;
  if (folds) {
    S = io.h0 ? io.h0[sn + fc] : 0.0f;
    K = io.dhT ? io.dhT[sn + fc] : 0.0f;
  }
  // chunk ch of sequence n keeps its state in slot cu[n] / 32 + n + ch: at most
  // L / 32 + 1 chunks, and floor(b / 32) - floor(a / 32) + 1 >= ceil((b - a) / 32)
  float* states = io.states + (t0 / kLruC + n) * static_cast<int64_t>(io.D) + cc;
  const int64_t rounds = (nch + slots - 1) / slots;
  for (int64_t r = 0; r < rounds; ++r) {
    const int64_t ch = r * slots + slot;
    const bool has = ch < nch;
    const int64_t tb = ch * kLruC;
    const int hi = has ? static_cast<int>(L - tb < kLruC ? L - tb : kLruC) : 0;
    float A[kLruC], B[kLruC];
    if (has) {
#pragma unroll
      for (int i = 0; i < kLruC; ++i) {
        const int64_t t = tb + (i < hi ? i : hi - 1);
        A[i] = ldin(g + t * io.ldg);
        B[i] = ldin(x + t * io.ldx);
      }
      float a = 1.0f, b = 0.0f;
#pragma unroll
      for (int i = 0; i < kLruC; ++i) {
        float al, u;
        lru_gate(io.gate, A[i], B[i], al, u);
        al = i < hi ? al : 1.0f;
        u = i < hi ? u : -0.0f;
        a = al * a;
        b = fmaf(al, b, u);
        A[i] = a;
        B[i] = b;
      }
      agg[threadIdx.x] = float2{a, b};
    }
    __syncthreads();
    if (folds) {
      const int m = static_cast<int>(nch - r * slots < slots ? nch - r * slots : slots);
      for (int s = 0; s < m; ++s) {
        const float2 ab = agg[s * W + threadIdx.x];
        start[s * W + threadIdx.x] = S;
        S = fmaf(ab.x, S, ab.y);
      }
    }
    __syncthreads();
    if (has && live) {
      const float st = start[threadIdx.x];
      states[ch * io.D] = st;
      if (o) {
#pragma unroll
        for (int i = 0; i < kLruC; ++i)
          if (i < hi) stout(o + (tb + i) * io.ldo, fmaf(A[i], st, B[i]));
      }
    }
  }
  if (folds && io.hT) io.hT[sn + fc] = S;
  for (int64_t r = rounds - 1; r >= 0; --r) {
    const int64_t ch = r * slots + slot;
    const bool has = ch < nch;
    const int64_t tb = ch * kLruC;
    const int hi = has ? static_cast<int>(L - tb < kLruC ? L - tb : kLruC) : 0;
    float al[kLruC], hp[kLruC], dy[kLruC], xx[kLruC], b[kLruC];
    if (has) {
#pragma unroll
      for (int i = 0; i < kLruC; ++i) {
        const int64_t t = tb + (i < hi ? i : hi - 1);
        b[i] = ldin(g + t * io.ldg);
        xx[i] = ldin(x + t * io.ldx);
        dy[i] = ldin(dO + t * io.lddo);
      }
      float h = live ? states[ch * io.D] : 0.0f;
#pragma unroll
      for (int i = 0; i < kLruC; ++i) {
        hp[i] = h;
        const float gi = b[i];
        al[i] = expf(gi);
        b[i] = io.gate == GDN_LRU_GATE_NONE         ? 1.0f
               : io.gate == GDN_LRU_GATE_COMPLEMENT ? -expm1f(gi)
                                                    : sqrtf(fmaxf(-expm1f(2.0f * gi), 0.0f));
        al[i] = i < hi ? al[i] : 1.0f;
        dy[i] = i < hi ? dy[i] : 0.0f;
        h = fmaf(al[i], h, b[i] * xx[i]);
      }
      float p = 1.0f, q = 0.0f;
#pragma unroll
      for (int i = kLruC - 1; i >= 0; --i) {
        q = al[i] * (q + dy[i]);
        p = al[i] * p;
      }
      agg[threadIdx.x] = float2{p, q};
    }
    __syncthreads();
    if (folds) {
      const int m = static_cast<int>(nch - r * slots < slots ? nch - r * slots : slots);
      for (int s = m - 1; s >= 0; --s) {
        const float2 pq = agg[s * W + threadIdx.x];
        start[s * W + threadIdx.x] = K;
        K = fmaf(pq.x, K, pq.y);
      }
    }
    __syncthreads();
    if (has && live) {
      float k = start[threadIdx.x];
#pragma unroll
      for (int i = kLruC - 1; i >= 0; --i) {
        const float d = dy[i] + k;
        k = al[i] * d;
        if (i < hi) {
          stout(dx + (tb + i) * io.lddx, b[i] * d);
          float e = al[i] * hp[i];
          if (io.gate == GDN_LRU_GATE_COMPLEMENT) e = fmaf(-al[i], xx[i], e);
          if (io.gate == GDN_LRU_GATE_NORM) e = fmaf(b[i] > 0.0f ? -(al[i] * al[i]) / b[i] : 0.0f, xx[i], e);
          stout(dg + (tb + i) * io.lddg, d * e);
        }
      }
    }
  }
  if (folds) io.dh0[sn + fc] = K;
}

// ---- host side ----------------------------------------------------------------

// Calls f.template operator()<TX, TG>() for the shape's types.
template <typename F>
int lru_dispatch(const gdn_lru_shape_t* s, F&& f) {
  if (s->in_dtype == GDN_BF16)
    return s->g_dtype == GDN_BF16 ? f.template operator()<bf16_t, bf16_t>() : f.template operator()<bf16_t, float>();
  return s->g_dtype == GDN_BF16 ? f.template operator()<float, bf16_t>() : f.template operator()<float, float>();
}

// Lanes per chunk and threads per block.
void lru_tiling(const LruIO& io, int V, int64_t longest, int* lps, int* threads) {
  int l = 64;
  while (l > 8 && io.T * io.D < static_cast<int64_t>(l) * V * 512 * longest) l >>= 1;
  const int64_t chunks = longest / kLruC + 2;
  int64_t t = (chunks * l + 63) / 64 * 64;
  if (t < l) t = l;
  if (t < l * V) t = l * V;  // one thread per channel of the tile folds
  *lps = l;
  *threads = static_cast<int>(t < kLruThreads ? t : kLruThreads);
}

// Checks and resolves what the packed calls share.
int lru_common(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_dev, const int32_t** cu_host,
               std::vector<int32_t>& buf, hipStream_t st, LruIO* io, int64_t* longest) {
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
  io->cu = cu_dev;
  io->N = n_seqs;
  io->D = shape->D;
  io->gate = shape->gate;
  io->T = cnt.T;
  return GDN_OK;
}

int lru_prefill_entry(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_dev, const int32_t* cu_host,
                      const void* x, int64_t ldx, const void* g, int64_t ldg, const float* h0, void* o, int64_t ldo,
                      float* hT, gdn_lru_cache_t* cache, bool resume, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  LruIO io{};
  std::vector<int32_t> buf;
  int64_t longest = 0;
  int rc = gdn::check_lru_shape(shape);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({x, g, h0, o, hT})) return GDN_ERR_INVALID_ARG;
  if ((cache || resume) && (rc = gdn::check_lru_cache(cache)) != GDN_OK) return rc;
  io.ldx = gdn::row_stride(ldx, shape->D);
  io.ldg = gdn::row_stride(ldg, shape->D);
  io.ldo = gdn::row_stride(ldo, shape->D);
  if (io.ldx < 0 || io.ldg < 0 || io.ldo < 0) return GDN_ERR_INVALID_ARG;
  if ((rc = lru_common(shape, n_seqs, cu_dev, &cu_host, buf, st, &io, &longest)) != GDN_OK) return rc;
  if (io.T > 0 && (!x || !g || !o)) return GDN_ERR_INVALID_ARG;
  if (n_seqs == 0) return GDN_OK;
  io.x = x; io.g = g; io.h0 = h0; io.o = o; io.hT = hT; io.resume = resume;
  if (cache) io.cache = *cache;
  const bool f32 = shape->in_dtype == GDN_F32 && shape->g_dtype == GDN_F32;
  const bool even = shape->D % 2 == 0 && io.ldx % 2 == 0 && io.ldg % 2 == 0 && io.ldo % 2 == 0;
  const int V = !f32 && even ? 2 : 1;
  int threads;
  lru_tiling(io, V, longest, &io.lps, &threads);
  io.tiles = (io.D + io.lps * V - 1) / (io.lps * V);
  const int64_t blocks = lru_blocks(n_seqs, io.tiles);
  if (blocks > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  lru_dispatch(shape, [&]<typename TX, typename TG>() {
    Timed t_("k_lru_fwd", st);
    const dim3 grid(static_cast<unsigned>(blocks)), block(threads);
    if (V == 2)
      hipLaunchKernelGGL((k_lru_fwd<TX, TG, 2>), grid, block, 0, st, io);
    else
      hipLaunchKernelGGL((k_lru_fwd<TX, TG, 1>), grid, block, 0, st, io);
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
  const int64_t blocks = (static_cast<int64_t>(n_seqs) * shape->D + 255) / 256;
  if (blocks > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Timed t_("k_lru_cache_init", st);
  hipLaunchKernelGGL(k_lru_cache_init, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, io);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_lru_prefill(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                    const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g, int64_t ldg,
                    const float* h0, void* o, int64_t ldo, float* hT, gdn_lru_cache_t* cache, void* stream) {
  return lru_prefill_entry(shape, n_seqs, cu_seqlens_dev, cu_seqlens_host, x, ldx, g, ldg, h0, o, ldo, hT, cache, false,
                           stream);
}

int gdn_lru_prefill_continue(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                             const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g, int64_t ldg,
                             gdn_lru_cache_t* cache, void* o, int64_t ldo, float* hT, void* stream) {
  return lru_prefill_entry(shape, n_seqs, cu_seqlens_dev, cu_seqlens_host, x, ldx, g, ldg, nullptr, o, ldo, hT, cache,
                           true, stream);
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
  return lru_dispatch(shape, [&]<typename TX, typename TG>() {
    Timed t_("k_lru_decode", st);
    const dim3 grid((io.D + gdn::kLruGroup - 1) / gdn::kLruGroup, n_seqs);
    hipLaunchKernelGGL((k_lru_decode<TX, TG>), grid, dim3(64), 0, st, io);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  });
}

size_t gdn_lru_workspace_bytes(const gdn_lru_shape_t* shape, int32_t n_seqs, int64_t total_tokens) {
  if (gdn::check_lru_shape(shape) != GDN_OK || n_seqs < 0 || total_tokens < 0 || total_tokens > INT32_MAX) return 0;
  return (static_cast<size_t>(gdn::lru_slots(total_tokens, n_seqs)) * shape->D * sizeof(float) + gdn::kAlign) /
         gdn::kAlign * gdn::kAlign;
}

int gdn_lru_fwd_bwd(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                    const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g, int64_t ldg,
                    const float* h0, const void* dO, int64_t lddo, const float* dhT, void* o, int64_t ldo, float* hT,
                    void* dx, int64_t lddx, void* dg, int64_t lddg, float* dh0, void* ws, size_t ws_bytes,
                    void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  LruIO io{};
  std::vector<int32_t> buf;
  int64_t longest = 0;
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
  if ((rc = lru_common(shape, n_seqs, cu_seqlens_dev, &cu_seqlens_host, buf, st, &io, &longest)) != GDN_OK) return rc;
  if (io.T > 0 && (!x || !g || !dO || !dx || !dg)) return GDN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < gdn_lru_workspace_bytes(shape, n_seqs, io.T)) return GDN_ERR_WORKSPACE;
  if (n_seqs == 0) return GDN_OK;
  io.x = x; io.g = g; io.h0 = h0; io.dO = dO; io.dhT = dhT; io.o = o; io.hT = hT; io.dx = dx; io.dg = dg; io.dh0 = dh0;
  io.states = static_cast<float*>(ws);
  int threads;
  lru_tiling(io, 1, longest, &io.lps, &threads);
  io.tiles = (io.D + io.lps - 1) / io.lps;
  const int64_t blocks = lru_blocks(n_seqs, io.tiles);
  if (blocks > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  return lru_dispatch(shape, [&]<typename TX, typename TG>() {
    Timed t_("k_lru_bwd", st);
    hipLaunchKernelGGL((k_lru_bwd<TX, TG>), dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, st, io);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  });
}

}  // extern "C"
