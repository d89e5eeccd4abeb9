// Matrix-core operands for the attention kernels: fragments of 32 x 16 values in
// registers, tiles of rows in LDS.
//
// One product step is C[32 x 32] += A[32 x 16] B[16 x 32].  Lane l holds A[l %
// 32][8 (l / 32) + j] and B[8 (l / 32) + j][l % 32], j = 0..7, and C's rows 8 (i /
// 4) + 4 (l / 32) + i % 4, i = 0..15, of column l % 32.  bf16: one
// v_mfma_f32_32x32x16_bf16; fp32: eight v_mfma_f32_32x32x2_f32, the j-th over k = j
// and 8 + j.  Either sums in fp32.
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

// All loads of this wave, those into LDS among them, have arrived.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <typename T>
struct Frag;
template <>
struct Frag<bf16_t> {
  u32x4 x;
  __device__ __forceinline__ void load(brsrc_t r, uint32_t at) { x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0)); }
  // c[i0 .. i0 + 7], rounded to nearest even
  __device__ __forceinline__ void pack(const v16f& c, int i0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack_bf16(c[i0 + 2 * e], c[i0 + 2 * e + 1]);
  }
  __device__ __forceinline__ float dot(const Frag& y) const {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y.x[e] << 16), s);
      s = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y.x[e] & 0xffff0000u), s);
    }
    return s;
  }
};
template <>
struct Frag<float> {
  float x[8];
  __device__ __forceinline__ void load(brsrc_t r, uint32_t at) {
    const v4f a = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    const v4f b = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 0));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = a[e];
      x[4 + e] = b[e];
    }
  }
  __device__ __forceinline__ void pack(const v16f& c, int i0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c[i0 + e];
  }
  __device__ __forceinline__ float dot(const Frag& y) const {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], y.x[e], s);
    return s;
  }
};

__device__ __forceinline__ v16f mma32(const Frag<bf16_t>& a, const Frag<bf16_t>& b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.x), __builtin_bit_cast(bf16x8, b.x), c, 0, 0, 0);
}
__device__ __forceinline__ v16f mma32(const Frag<float>& a, const Frag<float>& b, v16f c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.x[j], b.x[j], c, 0, 0, 0);
  return c;
}

template <int RB>
__device__ __forceinline__ int swizzle(int r) {
  return RB >= 256 ? (r & 3) << 2 | (r >> 2 & 3) : (r >> 1 & 1) << 2 | (r >> 2 & 3);
}

// Row operand: element j is X[r0 + l % 32][16 ks + 8 (l / 32) + j].  r0 a multiple of 32.
template <typename T, int RB>
__device__ __forceinline__ Frag<T> row_frag(const char* lds, int r0, int ks, int lane) {
  const int r = lane & 31, f = swizzle<RB>(r);
  const char* at = lds + r0 * RB + r * RB;
  Frag<T> a;
  if constexpr (sizeof(T) == 2) {
    a.x = *reinterpret_cast<const u32x4*>(at + (((2 * ks + (lane >> 5)) ^ f) << 4));
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const v4f y = *reinterpret_cast<const v4f*>(at + (((4 * ks + 2 * (lane >> 5) + e) ^ f) << 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) a.x[4 * e + i] = y[i];
    }
  }
  return a;
}

// Column operand: element j is X[r0 + c_row(j)][32 dt + l % 32], the rows in the
// order in which C holds them.  r0 a multiple of 16.
template <typename T, int RB>
__device__ __forceinline__ Frag<T> col_frag(const char* lds, int r0, int dt, int lane) {
  Frag<T> a;
  if constexpr (sizeof(T) == 2) {
    // a transposing read takes 4 rows x 16 columns for each 16 lanes: lane 4 r + c
    // gives the address of row r's columns 4 c, and lane i gets column i
    const int i = lane & 15, h = lane >> 5, g = lane >> 4 & 1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * e + 4 * h + (i >> 2);
      const int piece = (4 * dt + 2 * g + (i >> 1 & 1)) ^ swizzle<RB>(r);
      const char* at = lds + r0 * RB + r * RB + (piece << 4) + ((i & 1) << 3);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GDN_LDS s16x4*)(at));
      const u32x2 w = __builtin_bit_cast(u32x2, y);
      a.x[2 * e] = w[0];
      a.x[2 * e + 1] = w[1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = c_row(j, lane);
      const int piece = (8 * dt + ((lane & 31) >> 2)) ^ swizzle<RB>(r);
      a.x[j] = *reinterpret_cast<const float*>(lds + r0 * RB + r * RB + (piece << 4) + ((lane & 3) << 2));
    }
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

// Loads of a tile of ROWS rows straight into LDS, 64 pieces a wave and step.
template <typename T, int D, int ROWS, int NW>
struct Stager {
  static constexpr int RB = D * sizeof(T), CPR = RB / 16, STEPS = ROWS * CPR / (64 * NW);
  static_assert(ROWS * CPR % (64 * NW) == 0);
  uint32_t at[STEPS];
  int wave;
  __device__ __forceinline__ Stager(int64_t ld, int w, int lane) : wave(w) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = (s * NW + w) * 64 + lane, r = c / CPR;
      at[s] = static_cast<uint32_t>(r * ld * sizeof(T)) + (((c % CPR) ^ swizzle<RB>(r)) << 4);
    }
  }
  __device__ __forceinline__ void start(brsrc_t rsrc, char* lds) const {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (GDN_LDS void*)(lds + (s * NW + wave) * 1024), 16, at[s], 0, 0, 0);
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
