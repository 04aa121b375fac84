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

// ------------------------------------------------------------- 16 consecutive elements
// A thread's vector is 16 elements: 32 bytes of bf16 (one sector, one load), so
// that 8 lanes hold a scale block.  Arithmetic goes in fp32 pairs (add, mul and
// fma .f32x2 round each half as the scalar instruction does), half the
// instructions of the scalar form.
typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_of(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_get(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f2 v) {
  const float2 x = f2_get(v);
  return x.x + x.y;
}

struct F16 { f2 p[8]; };                               // 16 values
template <typename T> struct Raw16;                    // 16 elements as stored
template <> struct Raw16<__nv_bfloat16> { alignas(16) uint32_t w[8]; };
template <> struct Raw16<float> { alignas(16) uint32_t w[16]; };

__device__ __forceinline__ void ld_sector(uint32_t* w, const void* p) {   // 32 bytes, 32-byte aligned
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p) : "memory");
}
__device__ __forceinline__ void st_sector(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// Elements c .. c + 15 of a row of `cols`; what lies past the row's end is zero.
// VEC: rows begin at multiples of 32 bytes, and a thread takes whole sectors.
// Otherwise the warp takes its 512 elements in stripes (lane l elements l, l +
// 32, ...), which are consecutive in memory whatever the row's alignment (2 B a
// lane at a stride of 32 B costs 16 times the L1 work), and settle() exchanges
// them through the warp's scratch of 512 elements.  All lanes of a warp call
// these together, with consecutive c.
template <typename T> __device__ __forceinline__ uint32_t element_bits(const T* p);
template <> __device__ __forceinline__ uint32_t element_bits(const __nv_bfloat16* p) { return *reinterpret_cast<const uint16_t*>(p); }
template <> __device__ __forceinline__ uint32_t element_bits(const float* p) { return *reinterpret_cast<const uint32_t*>(p); }
template <typename T> struct Storage;
template <> struct Storage<__nv_bfloat16> { typedef uint16_t type; };
template <> struct Storage<float> { typedef uint32_t type; };

template <bool VEC, typename T>
__device__ __forceinline__ void load16(Raw16<T>& o, const T* row, int c, int cols) {
  constexpr int E = 4 / sizeof(T);                       // elements a word
#pragma unroll
  for (int h = 0; h < 16 / E; h += 8) {                  // a sector: 8 words
    if (VEC) {
      const int at = c + h * E;
      if (at + 8 * E <= cols) {
        ld_sector(o.w + h, row + at);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o.w[h + i] = 0;
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (at + i * E + e < cols) o.w[h + i] |= element_bits(row + at + i * E + e) << (16 * e);
        }
      }
    } else {
      const int lane = threadIdx.x & 31, at = c - 15 * lane;   // the warp's first element, + lane
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o.w[h + i] = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int k = at + 32 * ((h + i) * E + e);
          if (k < cols) o.w[h + i] |= element_bits(row + k) << (16 * e);
        }
      }
    }
  }
}
// From stripes to 16 consecutive elements a lane, and back.
template <typename T>
__device__ __forceinline__ void to_stripes(const Raw16<T>& o, typename Storage<T>::type* xs) {
  constexpr int E = 4 / sizeof(T);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 16 / E; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) xs[32 * (i * E + e) + lane] = (typename Storage<T>::type)(o.w[i] >> (16 * e));
}
template <bool VEC, typename T>
__device__ __forceinline__ void settle(Raw16<T>& o, void* scratch) {
  if (VEC) return;
  typename Storage<T>::type* xs = reinterpret_cast<typename Storage<T>::type*>(scratch);
  to_stripes(o, xs);
  __syncwarp();
  const uint4* p = reinterpret_cast<const uint4*>(xs + 16 * (threadIdx.x & 31));
#pragma unroll
  for (int i = 0; i < (int)sizeof(o.w) / 16; ++i) *reinterpret_cast<uint4*>(o.w + 4 * i) = p[i];
  __syncwarp();
}
template <bool VEC, typename T>
__device__ __forceinline__ void store16(T* row, int c, int cols, const Raw16<T>& o, void* scratch) {
  constexpr int E = 4 / sizeof(T);
  typedef typename Storage<T>::type S;
  S* p = reinterpret_cast<S*>(row);
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 16 / E; h += 8) {
      const int at = c + h * E;
      if (at + 8 * E <= cols) {
        st_sector(row + at, o.w + h);
      } else {
#pragma unroll
        for (int i = 0; i < 8 * E; ++i)
          if (at + i < cols) p[at + i] = (S)(o.w[h + i / E] >> (16 * (i % E)));
      }
    }
    return;
  }
  S* xs = reinterpret_cast<S*>(scratch);
  const int lane = threadIdx.x & 31, at = c - 15 * lane;
  uint4* q = reinterpret_cast<uint4*>(xs + 16 * lane);
#pragma unroll
  for (int i = 0; i < (int)sizeof(o.w) / 16; ++i) q[i] = *reinterpret_cast<const uint4*>(o.w + 4 * i);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (at + 32 * i < cols) p[at + 32 * i] = xs[32 * i + lane];
  __syncwarp();
}
__device__ __forceinline__ F16 unpack(const Raw16<__nv_bfloat16>& o) {
  F16 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.p[i] = f2_of(__uint_as_float(o.w[i] << 16), __uint_as_float(o.w[i] & 0xFFFF0000u));
  return f;
}
__device__ __forceinline__ F16 unpack(const Raw16<float>& o) {
  F16 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.p[i] = f2_of(__uint_as_float(o.w[2 * i]), __uint_as_float(o.w[2 * i + 1]));
  return f;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void pack(Raw16<__nv_bfloat16>& o, const F16& f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = f2_get(f.p[i]);
    o.w[i] = bf16x2_bits(x.x, x.y);
  }
}
__device__ __forceinline__ void pack(Raw16<float>& o, const F16& f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = f2_get(f.p[i]);
    o.w[2 * i] = __float_as_uint(x.x);
    o.w[2 * i + 1] = __float_as_uint(x.y);
  }
}
// 16 e4m3 bytes at columns c .. c + 15 of a row (16-byte aligned, c % 16 == 0).
__device__ __forceinline__ void store_q16(uint8_t* row, int c, int cols, uint4 b) {
  if (c + 16 <= cols) {
    *reinterpret_cast<uint4*>(row + c) = b;
  } else if (c < cols) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < cols) row[c + i] = (uint8_t)((&b.x)[i >> 2] >> (8 * (i & 3)));
  }
}
// Maxima that keep a NaN: of two values, and of a value and two magnitudes.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Exponent byte of the 128-column block that 8 lanes hold (16 values a lane);
// each of them gets it.  All 32 lanes call it.  Values that are not finite turn
// into NaN.
__device__ __forceinline__ unsigned q8_block_exponent(F16& f) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = f2_get(f.p[i]);
    m = max3_abs(m, x.x, x.y);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  unsigned b = abs_bits(m);
  if (__any_sync(0xffffffffu, b >= INF_BITS)) {
    b = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = f2_get(f.p[i]);
      b = max(b, max(finite_bits(x.x), finite_bits(x.y)));
      f.p[i] = f2_of(finite_or_nan(x.x), finite_or_nan(x.y));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  return q8_exponent(b);
}
__device__ __forceinline__ uint4 q8_pack16(const F16& f, float inv) {
  const f2 s = f2_of(inv, inv);
  uint4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f2_get(mul2(f.p[2 * i], s)), b = f2_get(mul2(f.p[2 * i + 1], s));
    (&o.x)[i] = q8_pack4(a.x, a.y, b.x, b.y);
  }
  return o;
}

}  // namespace precond
