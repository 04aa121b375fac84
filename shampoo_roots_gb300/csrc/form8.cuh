// The 8-bit form of a matrix (sm_103a): e4m3 values, rows a multiple of 16
// bytes apart, and one power-of-two scale 2^e for every row and block of 128
// columns.  e is the least integer with (largest finite magnitude) <= 448 2^e,
// so that the scaled block fills e4m3's range without saturating, and scaling
// by it is exact: the only rounding is the one to e4m3.  (A scale amax / 448
// would use the last half binade too, but rounds twice, and its product with a
// transposed copy's scale is no longer a shift.)
//
// A scale is one byte, e + 127 (the e8m0 encoding).  Bytes are stored in the
// order in which tensor memory takes them, so that the product copies them
// from global to shared to tensor memory without touching them: groups of 4
// blocks (512 columns) outermost, then blocks of 128 rows, and in each such
// 512-byte piece row r, block k at (r % 32) * 16 + (r / 32) * 4 + k.  Rows and
// blocks past the matrix's end hold 127 (scale 1).
#pragma once

#include "common.cuh"

namespace precond {

constexpr int Q8_BLK = 128;       // columns that share a scale
constexpr int Q8_GROUP = 512;     // columns of a scale group
constexpr unsigned Q8_ONE = 127;  // the scale 1

__host__ __device__ __forceinline__ int64_t q8_row_blocks(int64_t rows) { return (rows + 127) / 128; }
__host__ __device__ __forceinline__ int q8_groups(int64_t cols) { return (int)((cols + Q8_GROUP - 1) / Q8_GROUP); }
__host__ __device__ __forceinline__ size_t q8_scale_at(int64_t row, int kb, int64_t row_blocks) {
  return ((size_t)(kb >> 2) * row_blocks + (row >> 7)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (kb & 3);
}

// Biased exponent of a block whose largest magnitude has these fp32 bits
// (finite): the least b with amax <= 448 2^(b - 127), 448 = 1.75 2^8; 127 for
// an empty block.
__device__ __forceinline__ unsigned q8_exponent(unsigned amax_bits) {
  if (amax_bits == 0) return Q8_ONE;
  const int b = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (unsigned)max(b, 0);
}
// 2^-(b - 127): b is at most 247 for a finite fp32 block, so this is a normal number.
__device__ __forceinline__ float q8_inverse(unsigned b) { return __uint_as_float((254u - b) << 23); }
__device__ __forceinline__ float q8_value(unsigned b) { return b ? __uint_as_float(b << 23) : __uint_as_float(0x400000u); }

// Four values to e4m3 bytes (nearest, ties to even; magnitudes up to 448; NaN stays NaN).
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Two e4m3 bytes to fp32 (through fp16, which holds every e4m3 value).
__device__ __forceinline__ void q8_unpack2(uint16_t v, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  const __half2 x = *reinterpret_cast<const __half2*>(&h);
  a = __low2float(x);
  b = __high2float(x);
}

__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr unsigned INF_BITS = 0x7F800000u;
// A block's non-finite values must not vanish in saturation: they become NaN,
// and the block's scale is that of its finite values.
__device__ __forceinline__ float finite_or_nan(float x) {
  return abs_bits(x) < INF_BITS ? x : __uint_as_float(0x7FFFFFFFu);
}
__device__ __forceinline__ unsigned finite_bits(float x) {
  const unsigned b = abs_bits(x);
  return b < INF_BITS ? b : 0u;
}

// ------------------------------------------------------------- 8 consecutive elements
// Raw loads keep a prefetched vector at its storage size.  L1 is bypassed for
// data that a kernel reads once.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 v; };
template <> struct Raw8<float> { uint4 v, w; };

__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// Elements c .. c + 7 of a row of `cols`; what lies past the row's end is zero.
// VEC: the row is 16-byte aligned and cols % 8 == 0.
template <bool VEC>
__device__ __forceinline__ void load8(Raw8<__nv_bfloat16>& o, const __nv_bfloat16* row, int64_t c, int64_t cols) {
  o.v = make_uint4(0, 0, 0, 0);
  if (VEC) {
    if (c < cols) o.v = ld_once(row + c);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    uint32_t* w = &o.v.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) w[i >> 1] |= (uint32_t)p[c + i] << (16 * (i & 1));
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(Raw8<float>& o, const float* row, int64_t c, int64_t cols) {
  o.v = o.w = make_uint4(0, 0, 0, 0);
  if (VEC) {
    if (c < cols) {
      o.v = ld_once(row + c);
      o.w = ld_once(row + c + 4);
    }
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + i < cols) (&o.v.x)[i] = p[c + i];
      if (c + 4 + i < cols) (&o.w.x)[i] = p[c + 4 + i];
    }
  }
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& o, float (&f)[8]) {
  const uint32_t* w = &o.v.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& o, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = __uint_as_float((&o.v.x)[i]);
    f[4 + i] = __uint_as_float((&o.w.x)[i]);
  }
}
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void pack8(Raw8<__nv_bfloat16>& o, const float (&f)[8]) {
  o.v = make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]), bf16x2_bits(f[6], f[7]));
}
__device__ __forceinline__ void pack8(Raw8<float>& o, const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    (&o.v.x)[i] = __float_as_uint(f[i]);
    (&o.w.x)[i] = __float_as_uint(f[4 + i]);
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int64_t c, int64_t cols, const Raw8<__nv_bfloat16>& o) {
  if (VEC) {
    if (c < cols) *reinterpret_cast<uint4*>(row + c) = o.v;
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(row);
    const uint32_t* w = &o.v.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) p[c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* row, int64_t c, int64_t cols, const Raw8<float>& o) {
  if (VEC) {
    if (c < cols) {
      *reinterpret_cast<uint4*>(row + c) = o.v;
      *reinterpret_cast<uint4*>(row + c + 4) = o.w;
    }
  } else {
    uint32_t* p = reinterpret_cast<uint32_t*>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + i < cols) p[c + i] = (&o.v.x)[i];
      if (c + 4 + i < cols) p[c + 4 + i] = (&o.w.x)[i];
    }
  }
}
// 8 e4m3 bytes at columns c .. c + 7 of a row (16-byte aligned, c % 8 == 0).
__device__ __forceinline__ void store_q8(uint8_t* row, int64_t c, int64_t cols, uint2 b) {
  if (c + 8 <= cols) {
    *reinterpret_cast<uint2*>(row + c) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = (uint8_t)((i < 4 ? b.x : b.y) >> (8 * (i & 3)));
  }
}

// Exponent byte of the 128-column block that a half-warp holds (8 values a
// lane); every lane of the half-warp gets it.  All 32 lanes call it.  Values
// that are not finite turn into NaN.
__device__ __forceinline__ unsigned q8_block_exponent(float (&f)[8]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (__any_sync(0xffffffffu, m >= INF_BITS)) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = max(m, finite_bits(f[i]));
      f[i] = finite_or_nan(f[i]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  return q8_exponent(m);
}

}  // namespace precond
