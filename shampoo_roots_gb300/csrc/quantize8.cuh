// A matrix to its 8-bit form (form8.cuh), along its rows (q, blocks of 1 x 128)
// and along its columns (qt, the transposed matrix with blocks of 128 rows of
// one column), or with one scale for each 128 x 128 block, which then serves
// both orientations.
//
// Bound by memory: 2 B read and 1 B written per orientation and element (bf16).
// One block of 256 threads takes one 128 x 128 tile in one read: thread (tx,
// ty) holds rows 8 ty .. + 7 and columns 8 tx .. + 7, so that a row's maximum is
// a half-warp shuffle, a column's maximum needs one pass through shared memory,
// and the transposed bytes of a column are 8 consecutive ones of the output.
// They cross through 16 KB of shared memory, 8-byte pieces at position ty XOR tx
// of their column (no bank conflicts either way), and leave as 128-byte rows.
// The tile stays in registers as it is stored (32 registers of bf16) and is
// unpacked where it is used, which leaves room for four blocks on an SM; bf16
// maxima are taken on packed pairs.
//
// Measured (10007 x 6144 bf16): both ways 46.6 us, 79 % of the copy bandwidth,
// by rows 33.3 us, 82 %; fp32 both ways 72.5 us, 75 %.  What is left is issue
// slots: 16 conversions, shuffles and maxima for every 16 bytes moved.  A matrix
// in 8-bit form has half the bytes and more conversions: 82.5 us both ways,
// 8192 x 6144 by columns 54.5 us, 27 %.
#pragma once

#include "form8.cuh"

namespace precond {

enum { QIN_F32 = PRECOND_F32, QIN_BF16 = PRECOND_BF16, QIN_E4M3 = PRECOND_E4M3 };

struct Quant8Args {
  const void* x; int64_t ldx;
  const uint8_t* x_scale;            // 8-bit input: its scales
  int rows, cols;
  int tile;                          // 1: one scale per 128 x 128 block
  uint8_t* q; int64_t ldq; uint8_t* s;
  uint8_t* qt; int64_t ldqt; uint8_t* st;
};

// A thread's 8 x 8 elements as stored; get() gives one as fp32.
template <int IN> struct QuantTile;
template <> struct QuantTile<QIN_F32> {
  typedef float Element;
  uint32_t w[8][8];
  __device__ __forceinline__ float get(int i, int j) const { return __uint_as_float(w[i][j]); }
  __device__ __forceinline__ void set_nan(int i, int j) { w[i][j] = 0x7FFFFFFFu; }
  __device__ __forceinline__ void load(const Quant8Args& a, int i, int64_t row, int c) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(a.x) + row * a.ldx + c;
    if (c + 8 <= a.cols) {
      ld_sector(w[i], p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = c + j < a.cols ? p[j] : 0;
    }
  }
};
template <> struct QuantTile<QIN_BF16> {
  typedef __nv_bfloat16 Element;
  uint32_t w[8][4];
  __device__ __forceinline__ float get(int i, int j) const {
    return __uint_as_float(j & 1 ? w[i][j >> 1] & 0xFFFF0000u : w[i][j >> 1] << 16);
  }
  __device__ __forceinline__ void set_nan(int i, int j) { w[i][j >> 1] |= j & 1 ? 0x7FFF0000u : 0x7FFFu; }
  __device__ __forceinline__ void load(const Quant8Args& a, int i, int64_t row, int c) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.x) + row * a.ldx + c;
    if (c + 8 <= a.cols) {
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3]) : "l"(p) : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = c + 2 * j < a.cols ? p[2 * j] : 0, hi = c + 2 * j + 1 < a.cols ? p[2 * j + 1] : 0;
        w[i][j] = lo | hi << 16;
      }
    }
  }
};
template <> struct QuantTile<QIN_E4M3> {
  typedef void Element;              // its rows are aligned
  uint32_t w[8][2];
  float scale[8];                    // of the rows: a tile's columns are one block
  __device__ __forceinline__ float get(int i, int j) const {
    float lo, hi;
    q8_unpack2((uint16_t)(w[i][j >> 2] >> (16 * ((j >> 1) & 1))), lo, hi);
    return (j & 1 ? hi : lo) * scale[i];
  }
  __device__ __forceinline__ void set_nan(int i, int j) {}          // settle() has done it
  // Values that are not finite in fp32 though their bytes are numbers: beyond fp32's range, which begins at 256 2^120,
  // and all under the byte 255 (q8_value).  Their bytes become NaN here, before anything is unpacked: done where such a
  // tile is found, with unpacked values in registers on both sides, 8192 x 6144 by columns took 67 us, not 55.
  __device__ __forceinline__ void settle() {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, scale[i]);
    if (most < 0x1p120f) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (abs_bits(get(i, j)) >= INF_BITS) w[i][j >> 2] |= 0x7Fu << (8 * (j & 3));
  }
  __device__ __forceinline__ void load(const Quant8Args& a, int i, int64_t row, int c) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(a.x) + row * a.ldx + c;   // 16-byte aligned rows, c % 8 == 0
    w[i][0] = w[i][1] = 0;
    if (c + 8 <= a.cols) {
      const uint2 b = *reinterpret_cast<const uint2*>(p);
      w[i][0] = b.x;
      w[i][1] = b.y;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < a.cols) w[i][j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    }
    scale[i] = c < a.cols ? q8_value(a.x_scale[q8_scale_at(row, (int)(c >> 7), q8_row_blocks(a.rows))]) : 0.f;
  }
};

// A row of a tile that is not aligned, taken by a half-warp as the aligned
// granules of 16 bytes that lie inside it (lane tx granules tx, tx + 16) and the
// elements before and after those, one a lane (form8.cuh does the same for 512
// elements of a warp; 8000 x 7001 bf16 by rows: 46 us, in stripes 60).
template <typename T>
struct TileRow {
  static constexpr int G = 16 / sizeof(T), PER_LANE = 8 / G;
  const T* p;
  int shift, head, len, edge;         // edge: this lane's single element, or -1
  __device__ __forceinline__ TileRow(const Quant8Args& a, int64_t row, int c0, int tx) {
    p = reinterpret_cast<const T*>(a.x) + row * a.ldx + c0;
    shift = (int)(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (G - 1);
    head = G - shift;
    len = min(a.cols - c0, 128);
    const int tail = head + max(len - head, 0) / G * G;
    edge = tx < G ? (tx < head && tx < len ? tx : -1) : tx < 2 * G && tail + tx - G < len ? tail + tx - G : -1;
  }
  __device__ __forceinline__ void load(uint32_t* w, uint32_t& single, int tx) const {
#pragma unroll
    for (int k = 0; k < PER_LANE; ++k) {
      const int e = head + (tx + 16 * k) * G;
      w[4 * k] = w[4 * k + 1] = w[4 * k + 2] = w[4 * k + 3] = 0;
      if (e + G <= len)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[4 * k]), "=r"(w[4 * k + 1]), "=r"(w[4 * k + 2]), "=r"(w[4 * k + 3]) : "l"(p + e) : "memory");
    }
    single = 0;
    if (edge >= 0) single = element_bits(p + edge);
  }
  // into order, through the half-warp's scratch of 34 granules
  __device__ __forceinline__ void settle(uint32_t* w, uint32_t single, int tx, uint8_t* xs) const {
    uint4* g = reinterpret_cast<uint4*>(xs);
#pragma unroll
    for (int k = 0; k < PER_LANE; ++k) g[tx + 16 * k + 1] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    __syncwarp();
    const int at = edge >= 0 ? edge : tx < head ? tx : -1;       // a head's past the row's end: zero
    if (at >= 0) reinterpret_cast<typename Storage<T>::type*>(xs)[at + shift] = (typename Storage<T>::type)single;
    __syncwarp();
    uint32_t t[4 * PER_LANE + 4];
#pragma unroll
    for (int k = 0; k <= PER_LANE; ++k) {
      const uint4 x = g[PER_LANE * tx + k];
      t[4 * k] = x.x; t[4 * k + 1] = x.y; t[4 * k + 2] = x.z; t[4 * k + 3] = x.w;
    }
    shift_words<4 * PER_LANE + 4, T>(t, w, 4 * PER_LANE, shift);
    __syncwarp();
  }
};
// fp32: in stripes, lane tx elements tx, tx + 16, ... (8000 x 7001 by tiles, both ways: 79 us, in
// granules 94).
template <>
struct TileRow<float> {
  const uint32_t* p;
  int len;
  __device__ __forceinline__ TileRow(const Quant8Args& a, int64_t row, int c0, int)
      : p(reinterpret_cast<const uint32_t*>(a.x) + row * a.ldx + c0), len(a.cols - c0) {}
  __device__ __forceinline__ void load(uint32_t* w, uint32_t&, int tx) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (16 * j + tx < len) w[j] = p[16 * j + tx];
  }
  __device__ __forceinline__ void settle(uint32_t* w, uint32_t, int tx, uint8_t* xs) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) reinterpret_cast<uint32_t*>(xs)[16 * j + tx] = w[j];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 x = reinterpret_cast<const uint4*>(xs)[2 * tx + k];
      w[4 * k] = x.x; w[4 * k + 1] = x.y; w[4 * k + 2] = x.z; w[4 * k + 3] = x.w;
    }
    __syncwarp();
  }
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {   // keeps a NaN
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Magnitude bits (fp32) of the 8 rows' largest values over the half-warp's 128 columns, and of the thread's 8
// columns over its 8 rows; the return value is at least INF_BITS where one of the thread's values is not finite.
template <int IN>
__device__ __forceinline__ unsigned quant_maxima(const QuantTile<IN>& v, unsigned (&rm)[8], unsigned (&cm)[8], bool finite) {
  unsigned most = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rm[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned b = finite ? finite_bits(v.get(i, j)) : abs_bits(v.get(i, j));
      rm[i] = max(rm[i], b);
      cm[j] = max(cm[j], b);
    }
    most = max(most, rm[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) rm[i] = max(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], o));
  return most;
}
// bf16: on packed pairs, of columns and then of rows.
__device__ __forceinline__ unsigned quant_maxima_bf16(const QuantTile<QIN_BF16>& v, unsigned (&rm)[8], unsigned (&cm)[8]) {
  uint32_t c[4], most = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint32_t r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b[j] = v.w[i + k][j] & 0x7FFF7FFFu;
        c[j] = i + k == 0 ? b[j] : max_bf16x2(c[j], b[j]);
      }
      r[k] = max_bf16x2(max_bf16x2(b[0], b[1]), max_bf16x2(b[2], b[3]));
    }
    uint32_t m = max_bf16x2(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[0], r[1], 0x7632));   // rows i, i + 1
    most = i == 0 ? m : max_bf16x2(most, m);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    rm[i] = m << 16;
    rm[i + 1] = m & 0xFFFF0000u;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = j & 1 ? c[j >> 1] & 0xFFFF0000u : c[j >> 1] << 16;
  return max(most << 16, most & 0xFFFF0000u);
}

template <int IN, bool VEC>
__global__ void __launch_bounds__(256, IN == QIN_F32 ? 2 : IN == QIN_BF16 ? (VEC ? 4 : 3) : 3) quantize8_kernel(Quant8Args a) {
  __shared__ __align__(16) uint8_t tr[128 * 128];
  __shared__ unsigned cmax[8][128];
  __shared__ unsigned char cexp[128];
  __shared__ unsigned tmax[4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const unsigned col_tiles = (unsigned)(a.cols + 127) >> 7, row_tiles = (unsigned)(a.rows + 127) >> 7;
  const int ti = (int)(blockIdx.x / col_tiles), tj = (int)(blockIdx.x - ti * col_tiles);
  const int r0 = ti * 128 + 8 * ty, c0 = tj * 128 + 8 * tx;
  const bool whole = ti * 128 + 128 <= a.rows && tj * 128 + 128 <= a.cols;
  wait_for_previous();
  let_next_start();

  QuantTile<IN> v;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i < a.rows) {
        v.load(a, i, r0 + i, c0);
      } else {
#pragma unroll
        for (auto& x : v.w[i]) x = 0;
        if constexpr (IN == QIN_E4M3) v.scale[i] = 0.f;
      }
    }
    if constexpr (IN == QIN_E4M3) v.settle();
  } else {
    typedef TileRow<typename QuantTile<IN>::Element> Row;
    uint32_t single[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      single[i] = 0;
#pragma unroll
      for (auto& x : v.w[i]) x = 0;
      if (r0 + i < a.rows) Row(a, r0 + i, tj * 128, tx).load(v.w[i], single[i], tx);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) Row(a, r0 + i, tj * 128, tx).settle(v.w[i], single[i], tx, tr + ty * 1024);
  }
  unsigned rexp[8], cm[8], most;
  if constexpr (IN == QIN_BF16) most = quant_maxima_bf16(v, rexp, cm);
  else most = quant_maxima<IN>(v, rexp, cm, false);
  if (__syncthreads_or(most >= INF_BITS)) {
    // somewhere in the tile a value is not finite: it becomes NaN and counts for no maximum
    quant_maxima<IN>(v, rexp, cm, true);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (abs_bits(v.get(i, j)) >= INF_BITS) v.set_nan(i, j);
  }
  if (a.tile || a.qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cm[j] = max(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
      if ((threadIdx.x & 16) == 0) cmax[warp][8 * tx + j] = cm[j];
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      unsigned m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, cmax[k][threadIdx.x]);
      if (a.tile) {
        m = __reduce_max_sync(0xffffffffu, m);
        if ((threadIdx.x & 31) == 0) tmax[warp] = m;
      } else {
        cexp[threadIdx.x] = (unsigned char)q8_exponent(m);
      }
    }
    __syncthreads();
  }
  if (a.tile) {
    const unsigned b = q8_exponent(max(max(tmax[0], tmax[1]), max(tmax[2], tmax[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i) rexp[i] = b;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rexp[i] = q8_exponent(rexp[i]);
  }
  if (a.q) {
    uint8_t* p = a.q + (int64_t)r0 * a.ldq + c0;
    uint8_t* sp = a.s + q8_scale_at(r0, (int)tj, row_tiles);          // 8 rows: 16 bytes apart
#pragma unroll
    for (int i = 0; i < 8; ++i, p += a.ldq) {
      const float inv = q8_inverse(rexp[i]);
      const f2 s2 = f2_of(inv, inv);
      uint32_t b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 x = f2_get(mul2(f2_of(v.get(i, 4 * h), v.get(i, 4 * h + 1)), s2));
        const float2 y = f2_get(mul2(f2_of(v.get(i, 4 * h + 2), v.get(i, 4 * h + 3)), s2));
        b[h] = q8_pack4(x.x, x.y, y.x, y.y);
      }
      if (whole || (r0 + i < a.rows && c0 + 8 <= a.cols)) {
        *reinterpret_cast<uint2*>(p) = make_uint2(b[0], b[1]);
      } else if (r0 + i < a.rows) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < a.cols) p[j] = (uint8_t)(b[j >> 2] >> (8 * (j & 3)));
      }
      if (tx == 0) sp[16 * i] = (uint8_t)(r0 + i < a.rows ? rexp[i] : Q8_ONE);
    }
    // the blocks of the last group past the end
    if (tj == (int)col_tiles - 1 && threadIdx.x < 128)
      for (int kb = col_tiles; kb < 4 * q8_groups(a.cols); ++kb)
        a.s[q8_scale_at(ti * 128 + threadIdx.x, kb, row_tiles)] = (uint8_t)Q8_ONE;
  }
  if (a.qt) {
    uint8_t* sp = a.st + q8_scale_at(c0, (int)ti, col_tiles);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned b = a.tile ? rexp[0] : cexp[8 * tx + j];
      const float inv = q8_inverse(b);
      const f2 s2 = f2_of(inv, inv);
      uint32_t o[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 x = f2_get(mul2(f2_of(v.get(4 * h, j), v.get(4 * h + 1, j)), s2));
        const float2 y = f2_get(mul2(f2_of(v.get(4 * h + 2, j), v.get(4 * h + 3, j)), s2));
        o[h] = q8_pack4(x.x, x.y, y.x, y.y);
      }
      *reinterpret_cast<uint2*>(tr + (8 * tx + j) * 128 + ((ty ^ tx) << 3)) = make_uint2(o[0], o[1]);
      if (ty == 0) sp[16 * j] = (uint8_t)(c0 + j < a.cols ? b : Q8_ONE);
    }
    if (ti == (int)row_tiles - 1 && threadIdx.x < 128)
      for (int kb = row_tiles; kb < 4 * q8_groups(a.rows); ++kb)
        a.st[q8_scale_at(tj * 128 + threadIdx.x, kb, col_tiles)] = (uint8_t)Q8_ONE;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int piece = threadIdx.x + 256 * k;
      const int c = piece >> 3, p = piece & 7;       // column of the tile, 16-byte piece (rows 16 p ..)
      const int x = c >> 3;
      uint4 b = *reinterpret_cast<const uint4*>(tr + c * 128 + (((2 * p) ^ x) >> 1) * 16);
      if (x & 1) b = make_uint4(b.z, b.w, b.x, b.y);
      const int oc = ti * 128 + 16 * p, orow = tj * 128 + c;
      if (whole || (orow < a.cols && oc < a.rows)) {
        uint8_t* dst = a.qt + (int64_t)orow * a.ldqt + oc;
        if (whole || oc + 16 <= a.rows) {
          *reinterpret_cast<uint4*>(dst) = b;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (oc + i < a.rows) dst[i] = (uint8_t)((&b.x)[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
  }
}

}  // namespace precond
