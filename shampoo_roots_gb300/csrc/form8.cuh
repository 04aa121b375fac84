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
// The byte 255, e8m0's NaN, gives infinity: no e4m3 value times it is finite.
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
template <typename T> struct Raw16;                    // 16 elements as stored; the last two: unaligned rows (load16)
template <> struct Raw16<__nv_bfloat16> { alignas(16) uint32_t w[8]; uint32_t edge; int place; };
template <> struct Raw16<float> { alignas(16) uint32_t w[16]; uint32_t edge; int place; };

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
// Otherwise the warp's 512 elements are taken as the aligned granules of 16
// bytes that lie inside them (lane l granules l, l + 32, ...: consecutive in
// memory) and the elements before and after those, one a lane.  Registers wait
// for no load before settle(), which brings them into order through the warp's
// scratch: granules as they are, then 16 consecutive elements a lane out of
// three or five granules, shifted by the row's offset.  Nothing outside the row
// is read or written.  All lanes of a warp call these together, with
// consecutive c.  (Element loads at a stride of 32, their halves joined at once,
// took 122 us where this takes 59, for the norm of 20244 x 1213 bf16.)
template <typename T> __device__ __forceinline__ uint32_t element_bits(const T* p);
template <> __device__ __forceinline__ uint32_t element_bits(const __nv_bfloat16* p) { return *reinterpret_cast<const uint16_t*>(p); }
template <> __device__ __forceinline__ uint32_t element_bits(const float* p) { return *reinterpret_cast<const uint32_t*>(p); }
template <typename T> struct Storage;
template <> struct Storage<__nv_bfloat16> { typedef uint16_t type; };
template <> struct Storage<float> { typedef uint32_t type; };

// A warp's scratch: granules of 16 bytes, in an order in which lanes that read every second or fourth meet no bank twice.
template <typename T> struct Scratch {
  static constexpr int G = 16 / sizeof(T);             // elements of a granule
  static constexpr int PER_LANE = 16 / G;              // granules a lane
  static constexpr int BYTES = 512 * sizeof(T) + 128;  // one granule more, rounded up
  static __device__ __forceinline__ int slot(int g) { return g ^ ((g >> 3) & 7); }
  static __device__ __forceinline__ int element(int e) { return slot(e / G) * G + e % G; }
};
// An unaligned segment of up to 512 elements: `head` (1 .. G) elements, whole granules up to `tail`, the rest.
template <typename T>
struct Segment {
  static constexpr int G = Scratch<T>::G;
  int shift, head, len, tail, edge;                    // edge: this lane's single element, or -1
  __device__ __forceinline__ Segment(const T* row, int c, int cols) {
    const int lane = threadIdx.x & 31;
    shift = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (G - 1);
    head = G - shift;
    len = min(cols - (c - 16 * lane), 512);
    tail = head + max(len - head, 0) / G * G;
    edge = lane < G ? (lane < head && lane < len ? lane : -1) : lane < 2 * G && tail + lane - G < len ? tail + lane - G : -1;
  }
};

template <bool VEC, typename T>
__device__ __forceinline__ void load16(Raw16<T>& o, const T* row, int c, int cols) {
  constexpr int E = 4 / sizeof(T);                       // elements a word
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 16 / E; h += 8) {                // a sector: 8 words
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
    }
    return;
  }
  constexpr int G = Scratch<T>::G;
  const Segment<T> s(row, c, cols);
  const int lane = threadIdx.x & 31;
  const T* p = row + (c - 16 * lane);
#pragma unroll
  for (int i = 0; i < Scratch<T>::PER_LANE; ++i) {
    const int e = s.head + (lane + 32 * i) * G;
    uint32_t* w = o.w + 4 * i;
    w[0] = w[1] = w[2] = w[3] = 0;
    if (e + G <= s.len)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p + e) : "memory");
  }
  o.edge = 0;
  if (s.edge >= 0) o.edge = element_bits(p + s.edge);
  // its element in the scratch (a head's past the row's end: zero), and the shift
  const int at = s.edge >= 0 ? s.edge : lane < s.head ? lane : -1;
  o.place = (at < 0 ? 0xFFF : Scratch<T>::element(at + s.shift)) | (s.shift << 12);
}
// n words of t from word (or, for the lowest bit of bf16, half word) `shift` on.
template <int N, typename T>
__device__ __forceinline__ void shift_words(uint32_t* t, uint32_t* out, int n, int shift) {
  constexpr int E = 4 / sizeof(T);
#pragma unroll
  for (int k = 4; k > 0; k >>= 1) {
    const bool on = shift & (k * E);
#pragma unroll
    for (int i = 0; i + k < N; ++i) t[i] = on ? t[i + k] : t[i];
  }
#pragma unroll
  for (int i = 0; i < n; ++i) out[i] = E == 1 ? t[i] : __funnelshift_r(t[i], t[i + 1 < N ? i + 1 : i], (shift & 1) * 16);
}
template <bool VEC, typename T>
__device__ __forceinline__ void settle(Raw16<T>& o, void* scratch) {
  if (VEC) return;
  constexpr int P = Scratch<T>::PER_LANE;
  uint4* xs = reinterpret_cast<uint4*>(scratch);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < P; ++i)
    xs[Scratch<T>::slot(lane + 32 * i + 1)] = make_uint4(o.w[4 * i], o.w[4 * i + 1], o.w[4 * i + 2], o.w[4 * i + 3]);
  __syncwarp();
  const int at = o.place & 0xFFF;
  if (at != 0xFFF) reinterpret_cast<typename Storage<T>::type*>(scratch)[at] = (typename Storage<T>::type)o.edge;
  __syncwarp();
  uint32_t t[4 * P + 4];
#pragma unroll
  for (int i = 0; i <= P; ++i) {
    const uint4 g = xs[Scratch<T>::slot(P * lane + i)];
    t[4 * i] = g.x; t[4 * i + 1] = g.y; t[4 * i + 2] = g.z; t[4 * i + 3] = g.w;
  }
  shift_words<4 * P + 4, T>(t, o.w, 4 * P, o.place >> 12);
  __syncwarp();
}
template <bool VEC, typename T>
__device__ __forceinline__ void store16(T* row, int c, int cols, const Raw16<T>& o, void* scratch) {
  constexpr int E = 4 / sizeof(T);
  typedef typename Storage<T>::type S;
  if (VEC) {
    S* p = reinterpret_cast<S*>(row);
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
  constexpr int G = Scratch<T>::G, P = Scratch<T>::PER_LANE;
  const Segment<T> s(row, c, cols);
  const int lane = threadIdx.x & 31;
  S* p = reinterpret_cast<S*>(row) + (c - 16 * lane);
  uint4* xs = reinterpret_cast<uint4*>(scratch);
#pragma unroll
  for (int i = 0; i < P; ++i)
    xs[Scratch<T>::slot(P * lane + i)] = make_uint4(o.w[4 * i], o.w[4 * i + 1], o.w[4 * i + 2], o.w[4 * i + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int k = lane + 32 * i, e = s.head + k * G;
    if (e + G <= s.len) {                                // then k + 1 is a granule of the segment
      const uint4 a = xs[Scratch<T>::slot(k)], b = xs[Scratch<T>::slot(k + 1)];
      uint32_t t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, v[4];
      shift_words<8, T>(t, v, 4, s.head);
      *reinterpret_cast<uint4*>(p + e) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  if (s.edge >= 0) p[s.edge] = reinterpret_cast<const S*>(scratch)[Scratch<T>::element(s.edge)];
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
