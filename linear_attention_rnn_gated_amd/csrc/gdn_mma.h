// Matrix-core operands for the attention kernels: fragments of 32 x 16 values in
// registers, tiles of rows in LDS.
//
// One product step is C[32 x 32] += A[32 x 16] B[16 x 32].  Lane l holds A[l %
// 32][8 (l / 32) + j] and B[8 (l / 32) + j][l % 32], j = 0..7, and C's rows 8 (i /
// 4) + 4 (l / 32) + i % 4, i = 0..15, of column l % 32: v_mfma_f32_32x32x16_bf16,
// which sums in fp32.  fp32 operands are three bf16 parts each and take six of them,
// 192 cycles where v_mfma_f32_32x32x2_f32 would take 512 (forward and gradient of 3830
// tokens, 6 heads of 64: 1238 us with those, 431 in parts, both as first built).
//
// A tile in LDS is rows of RB bytes in 16-byte pieces; piece c of row r stands at
// c ^ swizzle(r), so that neither the reads along rows (32 rows, one piece each)
// nor those down columns (8 rows, four pieces each) meet in a bank.
#pragma once

#include "gdn_common.h"

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
using brsrc_t = __amdgpu_buffer_rsrc_t;
#define GDN_LDS __attribute__((address_space(3)))
// The host pass takes the large kernels' declarations alone: with their bodies it
// leaves some of their launch stubs undefined.
#ifdef __HIP_DEVICE_COMPILE__
#define GDN_DEVICE_PASS
#endif

__device__ __forceinline__ v16f zero16() {
  v16f z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}
__device__ __forceinline__ int c_row(int i, int lane) { return 8 * (i / 4) + 4 * (lane >> 5) + i % 4; }

// x of lane ^ 32.
__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Says that x stands in the accumulation registers here.
__device__ __forceinline__ void in_agprs(v16f& x) { asm volatile("" : "+a"(x)); }

// All loads of this wave but the last N, those into LDS among them, have arrived.
template <int N = 0>
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

template <typename T>
struct Frag;
template <>
struct Frag<bf16_t> {
  u32x4 x;
  // c[i0 .. i0 + 7], rounded to nearest even
  __device__ __forceinline__ void pack(const v16f& c, int i0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack_bf16(c[i0 + 2 * e], c[i0 + 2 * e + 1]);
  }
};
template <>
struct Frag<float> {
  u32x4 p[3];
  // x in three bf16 parts, which hold its 24 bits
  __device__ __forceinline__ void split(const float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t w = pack_bf16(a, b);
        p[i][e] = w;
        if (i < 2) {
          a -= __uint_as_float(w << 16);
          b -= __uint_as_float(w & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void pack(const v16f& c, int i0) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c[i0 + e];
    split(x);
  }
};

// Right operands in two bf16 parts, which hold 16 bits of them.
struct TwoParts {
  u32x4 p[2];
  __device__ __forceinline__ void pack(const v16f& c, int i0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = c[i0 + 2 * e], b = c[i0 + 2 * e + 1];
      const uint32_t w = pack_bf16(a, b);
      p[0][e] = w;
      p[1][e] = pack_bf16(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xffff0000u));
    }
  }
};

// An operand that a wave holds throughout: as loaded where its parts would take
// too many registers (fp32 at d = 256), else ready for the products.
template <typename T, int D>
struct Held {
  Frag<T> f;
  __device__ __forceinline__ void load(brsrc_t r, uint32_t at) {
    if constexpr (sizeof(T) == 2) {
      f.x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    } else {
      float x[8];
      load8(r, at, x);
      f.split(x);
    }
  }
  static __device__ __forceinline__ void load8(brsrc_t r, uint32_t at, float* x) {
    const v4f a = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    const v4f b = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 0));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = a[e];
      x[4 + e] = b[e];
    }
  }
  __device__ __forceinline__ const Frag<T>& get() const { return f; }
};
template <>
struct Held<float, 256> {
  float x[8];
  __device__ __forceinline__ void load(brsrc_t r, uint32_t at) { Held<float, 64>::load8(r, at, x); }
  __device__ __forceinline__ Frag<float> get() const {
    Frag<float> f;
    f.split(x);
    return f;
  }
};

// sum += a . b of eight elements read from two buffers.
template <typename T>
__device__ __forceinline__ float dot8(brsrc_t ra, uint32_t at_a, brsrc_t rb, uint32_t at_b, float sum) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, at_a, 0, 0));
    const u32x4 b = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, at_b, 0, 0));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), sum);
      sum = fmaf(__uint_as_float(a[e] & 0xffff0000u), __uint_as_float(b[e] & 0xffff0000u), sum);
    }
  } else {
    float a[8], b[8];
    Held<float, 64>::load8(ra, at_a, a);
    Held<float, 64>::load8(rb, at_b, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(a[e], b[e], sum);
  }
  return sum;
}

__device__ __forceinline__ v16f mma32(u32x4 a, u32x4 b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ v16f mma32(const Frag<bf16_t>& a, const Frag<bf16_t>& b, v16f c) { return mma32(a.x, b.x, c); }
// The products of parts down to 2^-16 of the largest, small ones first; those left
// out are 2^-24 of it.
__device__ __forceinline__ v16f mma32(const Frag<float>& a, const Frag<float>& b, v16f c) {
  c = mma32(a.p[0], b.p[2], c);
  c = mma32(a.p[2], b.p[0], c);
  c = mma32(a.p[1], b.p[1], c);
  c = mma32(a.p[0], b.p[1], c);
  c = mma32(a.p[1], b.p[0], c);
  return mma32(a.p[0], b.p[0], c);
}

// A left operand that is exact in one part.
__device__ __forceinline__ v16f mma32(const Frag<bf16_t>& a, const Frag<float>& b, v16f c) {
  c = mma32(a.x, b.p[2], c);
  c = mma32(a.x, b.p[1], c);
  return mma32(a.x, b.p[0], c);
}

__device__ __forceinline__ v16f mma32(const Frag<bf16_t>& a, const TwoParts& b, v16f c) {
  c = mma32(a.x, b.p[1], c);
  return mma32(a.x, b.p[0], c);
}

// A tile of ROWS rows in LDS: one plane of bf16, or three of an fp32 tile's parts.
template <typename T, int D, int ROWS>
struct Plane {
  static constexpr int N = sizeof(T) == 2 ? 1 : 3, RB = 2 * D, BYTES = ROWS * RB, TILE = N * BYTES;
};

template <int RB>
__device__ __forceinline__ int swizzle(int r) {
  return RB >= 256 ? (r & 3) << 2 | (r >> 2 & 3) : (r >> 1 & 1) << 2 | (r >> 2 & 3);
}

// Row operand: element j is X[r0 + l % 32][16 ks + 8 (l / 32) + j].  r0 a multiple of 32.
template <int RB>
__device__ __forceinline__ u32x4 row_plane(const char* lds, int r0, int ks, int lane) {
  const int r = lane & 31;
  return *reinterpret_cast<const u32x4*>(lds + r0 * RB + r * RB + (((2 * ks + (lane >> 5)) ^ swizzle<RB>(r)) << 4));
}
// Column operand: element j is X[r0 + c_row(j)][32 dt + l % 32], the rows in the
// order in which C holds them.  r0 a multiple of 16.  A transposing read takes 4
// rows x 16 columns for each 16 lanes: lane 4 r + c gives the address of row r's
// columns 4 c, and lane i gets column i.
template <int RB>
__device__ __forceinline__ u32x4 col_plane(const char* lds, int r0, int dt, int lane) {
  const int i = lane & 15, h = lane >> 5, g = lane >> 4 & 1;
  u32x4 a;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 8 * e + 4 * h + (i >> 2);
    const int piece = (4 * dt + 2 * g + (i >> 1 & 1)) ^ swizzle<RB>(r);
    const char* at = lds + r0 * RB + r * RB + (piece << 4) + ((i & 1) << 3);
    const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((GDN_LDS s16x4*)(at)));
    a[2 * e] = w[0];
    a[2 * e + 1] = w[1];
  }
  return a;
}
template <typename T, int D, int ROWS>
__device__ __forceinline__ Frag<T> row_frag(const char* lds, int r0, int ks, int lane) {
  using P = Plane<T, D, ROWS>;
  Frag<T> a;
  if constexpr (P::N == 1) {
    a.x = row_plane<P::RB>(lds, r0, ks, lane);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) a.p[i] = row_plane<P::RB>(lds + i * P::BYTES, r0, ks, lane);
  }
  return a;
}
template <typename T, int D, int ROWS>
__device__ __forceinline__ Frag<T> col_frag(const char* lds, int r0, int dt, int lane) {
  using P = Plane<T, D, ROWS>;
  Frag<T> a;
  if constexpr (P::N == 1) {
    a.x = col_plane<P::RB>(lds, r0, dt, lane);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) a.p[i] = col_plane<P::RB>(lds + i * P::BYTES, r0, dt, lane);
  }
  return a;
}

// A buffer over `rows` rows (0 or fewer: none) of head h, row 0 at row `at` of x:
// reads past them are 0.
template <typename T, int D>
__device__ __forceinline__ brsrc_t rows_rsrc(const void* x, int64_t at, int64_t ld, int h, int rows) {
  const char* base = static_cast<const char*>(x) + (at * ld + static_cast<int64_t>(h) * D) * sizeof(T);
  const int bytes = rows > 0 ? static_cast<int>(((rows - 1) * ld + D) * sizeof(T)) : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), static_cast<short>(0), bytes, 0x00020000);
}

// Rows of one head, ROWS at a time, of every NG-th such tile: a buffer over the
// tile's rows that there are.
template <typename T, int D, int ROWS, int NG = 1>
struct RowTiles {
  const char* at;
  int64_t step;     // bytes to the next tile
  int ld, left;     // bytes of a row, rows from the tile on
  brsrc_t rsrc;
  __device__ __forceinline__ RowTiles(const void* x, int64_t row, int64_t ld, int h, int rows)
      : at(static_cast<const char*>(x) + (row * ld + static_cast<int64_t>(h) * D) * sizeof(T)),
        step(NG * ROWS * ld * sizeof(T)), ld(static_cast<int>(ld * sizeof(T))), left(rows) {}
  __device__ __forceinline__ void next() {
    const int rows = left < ROWS ? left : ROWS;
    const int bytes = rows > 0 ? (rows - 1) * ld + static_cast<int>(D * sizeof(T)) : 0;
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), static_cast<short>(0), bytes, 0x00020000);
    at += step;
    left -= NG * ROWS;
  }
};

// Moves a tile of ROWS rows into LDS.  bf16 rows go there straight from memory
// (start), 64 pieces of 16 bytes a wave and step; fp32 rows through registers
// (start), and their parts from there (finish).
template <typename T, int D, int ROWS, int NW>
struct Stager {
  using P = Plane<T, D, ROWS>;
  static constexpr bool DIRECT = sizeof(T) == 2;
  static constexpr int CPR = P::RB / 16, STEPS = ROWS * CPR / (64 * NW);
  static_assert(ROWS * CPR % (64 * NW) == 0);
  uint32_t at[STEPS];
  u32x4 held[DIRECT ? 1 : 2 * STEPS];
  int wave, lane;
  __device__ __forceinline__ Stager(int64_t ld, int w, int l) : wave(w), lane(l) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = (s * NW + w) * 64 + l, r = c / CPR;
      at[s] = static_cast<uint32_t>(r * ld * sizeof(T)) + (((c % CPR) ^ swizzle<P::RB>(r)) * 8 * sizeof(T));
    }
  }
  __device__ __forceinline__ void start(brsrc_t rsrc, char* lds) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) load(s, rsrc, lds);
  }
  __device__ __forceinline__ void load(int s, brsrc_t rsrc, char* lds) {
    if constexpr (DIRECT) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (GDN_LDS void*)(lds + (s * NW + wave) * 1024), 16, at[s], 0, 0, 0);
    } else {
      held[2 * s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at[s], 0, 0));
      held[2 * s + 1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at[s] + 16, 0, 0));
    }
  }
  __device__ __forceinline__ void finish(char* lds) const {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(held[2 * s + e / 4][e % 4]);
        Frag<float> f;
        f.split(x);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          *reinterpret_cast<u32x4*>(lds + i * P::BYTES + ((s * NW + wave) * 64 + lane) * 16) = f.p[i];
      }
    }
  }
};

__device__ __forceinline__ void store4(float* p, const float* x) { *reinterpret_cast<v4f*>(p) = v4f{x[0], x[1], x[2], x[3]}; }
__device__ __forceinline__ void store4(bf16_t* p, const float* x) {
  *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
}

__device__ __forceinline__ void store8(float* p, const float* x) {
  store4(p, x);
  store4(p + 4, x + 4);
}
__device__ __forceinline__ void store8(bf16_t* p, const float* x) {
  *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
}

}  // namespace
