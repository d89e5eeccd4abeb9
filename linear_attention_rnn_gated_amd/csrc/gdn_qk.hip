// Norms of q and k per head with rotary positions (include/gdn.h): kernels and
// C ABI.  Part of gdn_library.hip.
//
// A head's d elements are spread over a group of lanes, eight elements each in
// two quads chosen so that both elements of a rotated pair lie in one lane:
// with the half layout quads 4u and r/2 + 4u, with neighbouring pairs (and in
// the part that is not rotated) the eight elements from 8u.  A wave holds 64 /
// group heads at once and goes over all heads of a token, so a pair's angle,
// sine and cosine are formed once per token and lane.
//
// Bound: HBM (4 to 12 bytes and about 12 vector instructions per element).
// Measured (bf16, one MI355X): L2 norm and full rotation of 8192 tokens x 32 heads
// of 128 29 us = 4.6 TB/s (rotation alone 26, neither 25); rotation of 148175
// tokens x 40 heads 552 us = 5.5 TB/s; gradient of the RMS norm and rotation,
// 32768 tokens x 32 heads, 160 us = 5.0 TB/s, and 5 us to add the weights' sums.

namespace {

constexpr double kInvTwoPi = 0.15915494309189533576888376337251;

struct QkIO {
  const void* q;
  const void* k;
  void* qo;
  void* ko;
  const void* dqo;
  const void* dko;
  const int32_t* pos;
  const int32_t* cu;
  const int32_t* start;
  const float* inv_freq;
  const float* w_q;
  const float* w_k;
  float* part;  // [blocks][2][d] sums for dw_q, dw_k; nullptr: not wanted
  int64_t T, ldq, ldk, ldqo, ldko, lddqo, lddko;
  int N, H_q, H_k, d, r, norm;
  int lg;     // log2 of the lanes per head
  int split;  // parts that a token's heads are cut into
  float eps, scale, rope_scale, offset, inv_d;
};

// A lane's two quads as loaded: eight fp32 or packed bf16 values.
template <typename T>
struct QkRaw;
template <>
struct QkRaw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* x, int oa, int ob) {
    a = *reinterpret_cast<const float4*>(x + oa);
    b = *reinterpret_cast<const float4*>(x + ob);
  }
  __device__ __forceinline__ void clear() { a = b = float4{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct QkRaw<bf16_t> {
  uint2 a, b;
  __device__ __forceinline__ void load(const bf16_t* x, int oa, int ob) {
    a = *reinterpret_cast<const uint2*>(x + oa);
    b = *reinterpret_cast<const uint2*>(x + ob);
  }
  __device__ __forceinline__ void clear() { a = b = uint2{0u, 0u}; }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void st_quad(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = float4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void st_quad(bf16_t* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// Where a lane's two quads start in a head, and whether they are rotated.
struct QkLane {
  int u, head, heads;  // lane in its group, the group's head, heads per wave
  int oa, ob;
  bool active, rot;
  double rev[4];  // turns per position of the lane's four pairs
};
template <bool HALF>
__device__ __forceinline__ QkLane qk_lane(const QkIO& io) {
  QkLane l;
  const int lane = threadIdx.x & 63;
  l.u = lane & ((1 << io.lg) - 1);
  l.head = lane >> io.lg;
  l.heads = 64 >> io.lg;
  l.active = 8 * l.u < io.d;
  l.rot = 8 * l.u < io.r;
  // without a rotation the whole head is read in halves: at d = 128 the sum
  // of squares is then the prep kernel's, bit for bit
  const int half = io.r ? io.r : io.d;
  const bool h = HALF && 8 * l.u < half;
  l.oa = h ? 4 * l.u : 8 * l.u;
  l.ob = h ? half / 2 + 4 * l.u : 8 * l.u + 4;
#pragma unroll
  for (int e = 0; e < 4; ++e) l.rev[e] = l.rot ? io.inv_freq[4 * l.u + e] * kInvTwoPi : 0.0;
  return l;
}

// Token t's position; false for a row behind the last sequence.
__device__ __forceinline__ bool qk_position(const QkIO& io, int64_t t, int64_t& p) {
  if (io.pos) {
    p = io.pos[t];
    return true;
  }
  if (t >= io.cu[io.N]) return false;
  const int n = find_seq(io.cu, io.N, t);
  p = t - io.cu[n] + (io.start ? io.start[n] : 0);
  return true;
}

// cos and sin of the lane's pairs, times rope_scale.  The angle in turns is an
// fp64 product (2^-53 of at most 2^31 turns), its whole part dropped there.
__device__ __forceinline__ void qk_angles(const QkIO& io, const QkLane& l, int64_t p, float* c, float* s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double turn = static_cast<double>(p) * l.rev[e];
    float sn, cs;
    sincospif(2.0f * static_cast<float>(turn - rint(turn)), &sn, &cs);
    c[e] = cs * io.rope_scale;
    s[e] = sn * io.rope_scale;
  }
}

// Turns the lane's pairs by (c, s); a[] and b[] are its quads.
template <bool HALF>
__device__ __forceinline__ void qk_turn(float* a, float* b, const float* c, const float* s) {
  if constexpr (HALF) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = a[e], y = b[e];
      a[e] = fmaf(x, c[e], -(y * s[e]));
      b[e] = fmaf(y, c[e], x * s[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float* z = e < 2 ? a + 2 * e : b + 2 * (e - 2);
      const float x = z[0], y = z[1];
      z[0] = fmaf(x, c[e], -(y * s[e]));
      z[1] = fmaf(y, c[e], x * s[e]);
    }
  }
}

// x of the lane that `ctrl` names within its row of 16 lanes.
template <int ctrl>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), ctrl, 0xf, 0xf, true));
}
constexpr int kRowRor = 0x120, kHalfMirror = 0x141, kSwapPairs = 0x4e, kSwapOnes = 0xb1;

// Sum over the head of e[0..3] of every lane of the group: a butterfly over the
// group's lanes, in the row by data-parallel moves (lane l takes l + 8, l + 4,
// l + 2, l + 1 modulo 16, which after the steps before hold what l ^ 8, ^ 4, ^ 2,
// ^ 1 hold), above it by shuffles.  Smaller groups pair l with 7 - l first.
__device__ __forceinline__ float qk_sum(const QkIO& io, float* e) {
  for (int m = (1 << io.lg) >> 1; m >= 16; m >>= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] += __shfl_xor(e[i], m, 64);
  }
  if (io.lg >= 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] += dpp<kRowRor + 8>(e[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] += dpp<kRowRor + 4>(e[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] += dpp<kRowRor + 2>(e[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] += dpp<kRowRor + 1>(e[i]);
  } else {
    if (io.lg >= 3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] += dpp<kHalfMirror>(e[i]);
    }
    if (io.lg >= 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] += dpp<kSwapPairs>(e[i]);
    }
    if (io.lg >= 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] += dpp<kSwapOnes>(e[i]);
    }
  }
  return (e[0] + e[2]) + (e[1] + e[3]);
}
// The L2 norm is the prep kernel's, bit for bit; the RMS norm takes the
// hardware's reciprocal root (1 ulp), which takes what is below the normal
// numbers (eps = 0, elements of 1e-19) for 0.  LOW: that is scaled first; not in
// the gradient, whose n^2 is past fp32 there, and which a register more takes from
// four waves a SIMD to three (162 -> 218 us).
template <bool LOW>
__device__ __forceinline__ float qk_inverse_norm(const QkIO& io, const float* v) {
  float e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = fmaf(v[4 + i], v[4 + i], v[i] * v[i]);
  const float ss = qk_sum(io, e);
  if (io.norm == GDN_NORM_L2) return 1.0f / sqrtf(ss + io.eps);
  const float m = fmaf(ss, io.inv_d, io.eps);
  if constexpr (!LOW) return __builtin_amdgcn_rsqf(m);
  const bool low = m < 0x1p-126f;
  return __builtin_amdgcn_rsqf(low ? m * 0x1p64f : m) * (low ? 0x1p32f : 1.0f);
}

// The RMS weights of q and k, offset included, in LDS.
constexpr int kQkMaxD = 512;
__device__ __forceinline__ void qk_weights(const QkIO& io, float (*w)[kQkMaxD]) {
  if (io.norm == GDN_NORM_RMS) {
    for (int e = threadIdx.x; e < io.d; e += 256) {
      w[0][e] = io.offset + (io.w_q ? io.w_q[e] : 0.0f);
      w[1][e] = io.offset + (io.w_k ? io.w_k[e] : 0.0f);
    }
    __syncthreads();
  }
}
// The lane's eight of them.
__device__ __forceinline__ void qk_weight(const QkLane& l, const float* w, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(w + l.oa), b = *reinterpret_cast<const float4*>(w + l.ob);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Head h of token t, of q or k.
template <typename T, typename P>
__device__ __forceinline__ T* qk_head(const QkIO& io, P* q, int64_t ldq, P* k, int64_t ldk, int64_t t, int h) {
  return h < io.H_q ? static_cast<T*>(q) + t * ldq + h * io.d : static_cast<T*>(k) + t * ldk + (h - io.H_q) * io.d;
}

constexpr int kQkUnroll = 4, kQkGradUnroll = 2;  // head groups whose loads are in flight at once

template <typename TIn, typename TOut, bool HALF>
__global__ __launch_bounds__(256) void k_qk_fwd(QkIO io) {
  __shared__ __align__(16) float w[2][kQkMaxD];
  const QkLane l = qk_lane<HALF>(io);
  qk_weights(io, w);
  const int H = io.H_q + io.H_k;
  const int steps = (H + l.heads - 1) / l.heads;
  const int per = (steps + io.split - 1) / io.split;
  const int64_t items = io.T * io.split;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 4 + wave; it < items; it += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t t = it / io.split;
    const int part = static_cast<int>(it - t * io.split);
    const int s1 = (part + 1) * per < steps ? (part + 1) * per : steps;
    QkRaw<TIn> raw[kQkUnroll], next[kQkUnroll];
    auto load = [&](QkRaw<TIn>* r, int s0) {
#pragma unroll
      for (int j = 0; j < kQkUnroll; ++j) {
        const int h = (s0 + j) * l.heads + l.head;
        if (l.active && s0 + j < s1 && h < H)
          r[j].load(qk_head<const TIn>(io, io.q, io.ldq, io.k, io.ldk, t, h), l.oa, l.ob);
        else
          r[j].clear();
      }
    };
    int64_t p;
    if (!qk_position(io, t, p)) continue;
    load(raw, part * per);  // in flight while the angles are formed
    float c[4], s[4];
    if (l.rot) qk_angles(io, l, p, c, s);
    for (int s0 = part * per; s0 < s1; s0 += kQkUnroll) {
      if (s0 + kQkUnroll < s1) load(next, s0 + kQkUnroll);
#pragma unroll
      for (int j = 0; j < kQkUnroll; ++j) {
        if (s0 + j >= s1) break;
        const int h = (s0 + j) * l.heads + l.head;
        const bool is_q = h < io.H_q;
        float v[8];
        raw[j].get(v);
        if (io.norm != GDN_NORM_NONE) {
          const float n = qk_inverse_norm<true>(io, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= n;
          if (io.norm == GDN_NORM_RMS && l.active) {
            float m[8];
            qk_weight(l, w[is_q ? 0 : 1], m);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= m[e];
          }
        }
        if (l.rot) qk_turn<HALF>(v, v + 4, c, s);
        const float scale = is_q ? io.scale : 1.0f;  // (times 1 changes nothing)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
        if (l.active && h < H) {
          TOut* y = qk_head<TOut>(io, io.qo, io.ldqo, io.ko, io.ldko, t, h);
          st_quad(y + l.oa, v);
          st_quad(y + l.ob, v + 4);
        }
      }
#pragma unroll
      for (int j = 0; j < kQkUnroll; ++j) raw[j] = next[j];
    }
  }
}

// The gradient: the same walk over q, k and the gradients of the outputs; the
// weights' gradients are summed per lane over all tokens that its wave takes,
// then over the block, and k_qk_dw adds the blocks.
template <typename TIn, typename TOut, bool HALF>
__global__ __launch_bounds__(256) void k_qk_bwd(QkIO io) {
  __shared__ __align__(16) float w[2][kQkMaxD];
  const QkLane l = qk_lane<HALF>(io);
  qk_weights(io, w);
  float gq[8], gk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) gq[e] = gk[e] = 0.0f;
  const int H = io.H_q + io.H_k;
  const int steps = (H + l.heads - 1) / l.heads;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < io.T; t += static_cast<int64_t>(gridDim.x) * 4) {
    QkRaw<TIn> x0[kQkGradUnroll], x1[kQkGradUnroll];
    QkRaw<TOut> y0[kQkGradUnroll], y1[kQkGradUnroll];
    auto load = [&](QkRaw<TIn>* x, QkRaw<TOut>* y, int s0) {
#pragma unroll
      for (int j = 0; j < kQkGradUnroll; ++j) {
        const int h = (s0 + j) * l.heads + l.head;
        x[j].clear();
        y[j].clear();
        if (l.active && s0 + j < steps && h < H) {
          y[j].load(qk_head<const TOut>(io, io.dqo, io.lddqo, io.dko, io.lddko, t, h), l.oa, l.ob);
          if (io.norm != GDN_NORM_NONE)
            x[j].load(qk_head<const TIn>(io, io.q, io.ldq, io.k, io.ldk, t, h), l.oa, l.ob);
        }
      }
    };
    int64_t p;
    if (!qk_position(io, t, p)) continue;
    load(x0, y0, 0);  // in flight while the angles are formed
    float c[4], s[4];
    if (l.rot) {
      qk_angles(io, l, p, c, s);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = -s[e];
    }
    for (int s0 = 0; s0 < steps; s0 += kQkGradUnroll) {
      if (s0 + kQkGradUnroll < steps) load(x1, y1, s0 + kQkGradUnroll);
#pragma unroll
      for (int j = 0; j < kQkGradUnroll; ++j) {
        if (s0 + j >= steps) break;
        const int h = (s0 + j) * l.heads + l.head;
        const bool is_q = h < io.H_q;
        float x[8], y[8];
        x0[j].get(x);
        y0[j].get(y);
        const float scale = is_q ? io.scale : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= scale;
        if (l.rot) qk_turn<HALF>(y, y + 4, c, s);
        if (io.norm != GDN_NORM_NONE) {
          const float n = qk_inverse_norm<false>(io, x);
          if (io.norm == GDN_NORM_RMS) {
            float m[8];
            if (l.active) qk_weight(l, w[is_q ? 0 : 1], m);
            // branches, not factors of zero: 0 x NaN would take a q head's NaN into k's sum
            if (is_q) {
#pragma unroll
              for (int e = 0; e < 8; ++e) gq[e] = fmaf(y[e] * x[e], n, gq[e]);
            } else if (h < H) {
#pragma unroll
              for (int e = 0; e < 8; ++e) gk[e] = fmaf(y[e] * x[e], n, gk[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = l.active ? y[e] * m[e] : 0.0f;
          }
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4[e] = fmaf(x[4 + e], y[4 + e], x[e] * y[e]);
          const float dot = qk_sum(io, e4) * (n * n * (io.norm == GDN_NORM_RMS ? io.inv_d : 1.0f));
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = n * fmaf(-x[e], dot, y[e]);
        }
        if (l.active && h < H) {
          TIn* z = qk_head<TIn>(io, io.qo, io.ldqo, io.ko, io.ldko, t, h);
          st_quad(z + l.oa, y);
          st_quad(z + l.ob, y + 4);
        }
      }
#pragma unroll
      for (int j = 0; j < kQkGradUnroll; ++j) {
        x0[j] = x1[j];
        y0[j] = y1[j];
      }
    }
  }
  if (!io.part) return;
  __shared__ float acc[256][17];  // a column more than 16: no bank holds a whole column
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    acc[threadIdx.x][e] = gq[e];
    acc[threadIdx.x][8 + e] = gk[e];
  }
  __syncthreads();
  const int group = 1 << io.lg;
  for (int e = threadIdx.x; e < 2 * io.d; e += 256) {
    const int u = e >> 4, j = e & 15;  // lane of the group, its element
    float sum = 0.0f;
    for (int i = u; i < 256; i += group) sum += acc[i][j];
    const int half = io.r ? io.r : io.d;
    const bool hf = HALF && 8 * u < half;
    const int je = j & 7;
    const int at = je < 4 ? (hf ? 4 * u : 8 * u) + je : (hf ? half / 2 + 4 * u : 8 * u + 4) + je - 4;
    io.part[(static_cast<int64_t>(blockIdx.x) * 2 + (j >> 3)) * io.d + at] = sum;
  }
}

// dw = sum of the blocks' sums: 16 columns a block, 64 threads a column, each
// over every 64th row (four loads in flight), joined in order.
__global__ __launch_bounds__(1024) void k_qk_dw(const float* __restrict__ part, int64_t rows, int d,
                                                float* __restrict__ dw_q, float* __restrict__ dw_k) {
  __shared__ float acc[64][17];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + col;  // 2 d columns, d a multiple of 8
  float sum = 0.0f;
#pragma unroll 4
  for (int64_t r = row; r < rows; r += 64) sum += part[r * 2 * d + e];
  acc[row][col] = sum;
  __syncthreads();
  if (row < 4) {  // four runs of sixteen, then their sum
    sum = acc[16 * row][col];
    for (int i = 1; i < 16; ++i) sum += acc[16 * row + i][col];
  }
  __syncthreads();
  if (row < 4) acc[row][col] = sum;
  __syncthreads();
  if (row == 0) {
    sum = (acc[0][col] + acc[1][col]) + (acc[2][col] + acc[3][col]);
    float* out = e < d ? dw_q : dw_k;
    if (out) out[e < d ? e : e - d] = sum;
  }
}

// ---- host side ----------------------------------------------------------------

template <typename F>
int qk_dispatch(const gdn_qk_shape_t* s, F&& f) {
  const bool half = s->layout == GDN_ROPE_HALF;
  const bool ib = s->in_dtype == GDN_BF16, ob = s->out_dtype == GDN_BF16;
  if (ib && ob) return half ? f.template operator()<bf16_t, bf16_t, true>() : f.template operator()<bf16_t, bf16_t, false>();
  if (ib) return half ? f.template operator()<bf16_t, float, true>() : f.template operator()<bf16_t, float, false>();
  if (ob) return half ? f.template operator()<float, bf16_t, true>() : f.template operator()<float, bf16_t, false>();
  return half ? f.template operator()<float, float, true>() : f.template operator()<float, float, false>();
}

// Checks what the two calls share and fills io.
int qk_common(const gdn_qk_shape_t* s, int64_t T, const int32_t* pos, int32_t N, const int32_t* cu,
              const int32_t* start, const float* inv_freq, const float* w_q, const float* w_k, const void* q,
              int64_t ldq, const void* k, int64_t ldk, QkIO* io) {
  int rc = gdn::check_qk_shape(s);
  if (rc != GDN_OK) return rc;
  if (T < 0 || N < 0) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16({pos, cu, start, inv_freq, w_q, w_k, q, k})) return GDN_ERR_INVALID_ARG;
  if (!pos && (!cu || N == 0) && T > 0) return GDN_ERR_INVALID_ARG;
  if (s->r > 0 && !inv_freq) return GDN_ERR_INVALID_ARG;
  if (s->norm != GDN_NORM_RMS && (w_q || w_k)) return GDN_ERR_INVALID_ARG;
  if (T > 0 && (!q || (s->H_k > 0 && !k))) return GDN_ERR_INVALID_ARG;
  if (T > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  io->ldq = gdn::row_stride(ldq, static_cast<int64_t>(s->H_q) * s->d);
  io->ldk = gdn::row_stride(ldk, static_cast<int64_t>(s->H_k) * s->d);
  if (io->ldq < 0 || io->ldk < 0 || io->ldq % 8 || io->ldk % 8) return GDN_ERR_INVALID_ARG;
  io->q = q; io->k = k; io->pos = pos; io->cu = cu; io->start = start; io->inv_freq = inv_freq;
  io->w_q = w_q; io->w_k = w_k;
  io->T = T; io->N = N; io->H_q = s->H_q; io->H_k = s->H_k; io->d = s->d; io->r = s->r; io->norm = s->norm;
  io->eps = s->eps; io->scale = s->scale; io->rope_scale = s->rope_scale; io->offset = s->weight_offset;
  io->inv_d = 1.0f / static_cast<float>(s->d);
  io->lg = 0;
  while ((8 << io->lg) < s->d) ++io->lg;
  io->split = 1;
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_qk_rotary(const gdn_qk_shape_t* shape, int64_t n_tokens, const int32_t* pos, int32_t n_seqs,
                  const int32_t* cu_seqlens, const int32_t* start, const float* inv_freq, const float* w_q,
                  const float* w_k, const void* q, int64_t ldq, const void* k, int64_t ldk, void* qo, int64_t ldqo,
                  void* ko, int64_t ldko, void* stream) {
  QkIO io{};
  int rc = qk_common(shape, n_tokens, pos, n_seqs, cu_seqlens, start, inv_freq, w_q, w_k, q, ldq, k, ldk, &io);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({qo, ko})) return GDN_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!qo || (shape->H_k > 0 && !ko))) return GDN_ERR_INVALID_ARG;
  io.ldqo = gdn::row_stride(ldqo, static_cast<int64_t>(shape->H_q) * shape->d);
  io.ldko = gdn::row_stride(ldko, static_cast<int64_t>(shape->H_k) * shape->d);
  if (io.ldqo < 0 || io.ldko < 0 || io.ldqo % 8 || io.ldko % 8) return GDN_ERR_INVALID_ARG;
  if (n_tokens == 0) return GDN_OK;
  io.qo = qo; io.ko = ko;
  const int heads = 64 >> io.lg;
  const int steps = (io.H_q + io.H_k + heads - 1) / heads;
  // few tokens: cut each token's heads into parts until the chip has work
  while (io.split < steps && n_tokens * io.split < 2048) io.split *= 2;
  if (io.split > steps) io.split = steps;
  const int64_t want = (n_tokens * io.split + 3) / 4;
  // a wave an item: waves that take several one after another leave fewer loads
  // in flight (32 ragged x 40 heads: 557 us, in 2048 blocks 613)
  const unsigned blocks = static_cast<unsigned>(want < (1 << 22) ? want : 1 << 22);
  hipStream_t st = static_cast<hipStream_t>(stream);
  return qk_dispatch(shape, [&]<typename TIn, typename TOut, bool HALF>() {
    Timed t_("k_qk_fwd", st);
    hipLaunchKernelGGL((k_qk_fwd<TIn, TOut, HALF>), dim3(blocks), dim3(256), 0, st, io);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  });
}

size_t gdn_qk_workspace_bytes(const gdn_qk_shape_t* shape, int64_t n_tokens) {
  if (gdn::check_qk_shape(shape) != GDN_OK || n_tokens < 0 || n_tokens > INT32_MAX) return 0;
  const size_t bytes = static_cast<size_t>(gdn::qk_bwd_blocks(shape, n_tokens)) * 2 * shape->d * sizeof(float);
  return (bytes + gdn::kAlign) / gdn::kAlign * gdn::kAlign;
}

int gdn_qk_rotary_bwd(const gdn_qk_shape_t* shape, int64_t n_tokens, const int32_t* pos, int32_t n_seqs,
                      const int32_t* cu_seqlens, const int32_t* start, const float* inv_freq, const float* w_q,
                      const float* w_k, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* dqo,
                      int64_t lddqo, const void* dko, int64_t lddko, void* dq, int64_t lddq, void* dk, int64_t lddk,
                      float* dw_q, float* dw_k, void* ws, size_t ws_bytes, void* stream) {
  QkIO io{};
  int rc = qk_common(shape, n_tokens, pos, n_seqs, cu_seqlens, start, inv_freq, w_q, w_k, q, ldq, k, ldk, &io);
  if (rc != GDN_OK) return rc;
  if (!gdn::aligned16({dqo, dko, dq, dk, dw_q, dw_k, ws})) return GDN_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!dqo || !dq || (shape->H_k > 0 && (!dko || !dk)))) return GDN_ERR_INVALID_ARG;
  if (shape->norm != GDN_NORM_RMS && (dw_q || dw_k)) return GDN_ERR_INVALID_ARG;
  const int64_t rq = static_cast<int64_t>(shape->H_q) * shape->d, rk = static_cast<int64_t>(shape->H_k) * shape->d;
  io.lddqo = gdn::row_stride(lddqo, rq);
  io.lddko = gdn::row_stride(lddko, rk);
  io.ldqo = gdn::row_stride(lddq, rq);
  io.ldko = gdn::row_stride(lddk, rk);
  if (io.lddqo < 0 || io.lddko < 0 || io.ldqo < 0 || io.ldko < 0) return GDN_ERR_INVALID_ARG;
  if (io.lddqo % 8 || io.lddko % 8 || io.ldqo % 8 || io.ldko % 8) return GDN_ERR_INVALID_ARG;
  const bool sums = dw_q || dw_k;
  if (sums && (!ws || ws_bytes < gdn_qk_workspace_bytes(shape, n_tokens))) return GDN_ERR_WORKSPACE;
  io.dqo = dqo; io.dko = dko; io.qo = dq; io.ko = dk;
  io.part = sums ? static_cast<float*>(ws) : nullptr;
  const int64_t blocks = gdn::qk_bwd_blocks(shape, n_tokens);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (blocks > 0) {
    rc = qk_dispatch(shape, [&]<typename TIn, typename TOut, bool HALF>() {
      Timed t_("k_qk_bwd", st);
      hipLaunchKernelGGL((k_qk_bwd<TIn, TOut, HALF>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, io);
      return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    });
    if (rc != GDN_OK) return rc;
  }
  if (sums) {
    Timed t_("k_qk_dw", st);
    hipLaunchKernelGGL(k_qk_dw, dim3(shape->d / 8), dim3(1024), 0, st, io.part, blocks, shape->d, dw_q, dw_k);
  }
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
