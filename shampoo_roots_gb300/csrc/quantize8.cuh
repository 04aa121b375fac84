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
// maxima are taken on packed pairs of magnitude bits.
#pragma once

#include "form8.cuh"

namespace precond {

enum { QIN_F32 = PRECOND_F32, QIN_BF16 = PRECOND_BF16, QIN_E4M3 = PRECOND_E4M3 };

struct Quant8Args {
  const void* x; int64_t ldx;
  const uint8_t* x_scale;            // 8-bit input: its scales
  int64_t rows, cols;
  int tile;                          // 1: one scale per 128 x 128 block
  uint8_t* q; int64_t ldq; uint8_t* s;
  uint8_t* qt; int64_t ldqt; uint8_t* st;
};

// A thread's 8 x 8 elements as stored; get() gives one as fp32.
template <int IN> struct QuantTile;
template <> struct QuantTile<QIN_F32> {
  uint32_t w[8][8];
  __device__ __forceinline__ float get(int i, int j) const { return __uint_as_float(w[i][j]); }
  __device__ __forceinline__ void set_nan(int i, int j) { w[i][j] = 0x7FFFFFFFu; }
  __device__ __forceinline__ void load(const Quant8Args& a, bool vec, int i, int64_t row, int64_t c) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(a.x) + row * a.ldx + c;
    if (vec && c < a.cols) {
      ld_sector(w[i], p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = c + j < a.cols ? p[j] : 0;
    }
  }
};
template <> struct QuantTile<QIN_BF16> {
  uint32_t w[8][4];
  __device__ __forceinline__ float get(int i, int j) const {
    return __uint_as_float(j & 1 ? w[i][j >> 1] & 0xFFFF0000u : w[i][j >> 1] << 16);
  }
  __device__ __forceinline__ void set_nan(int i, int j) { w[i][j >> 1] |= j & 1 ? 0x7FFF0000u : 0x7FFFu; }
  __device__ __forceinline__ void load(const Quant8Args& a, bool vec, int i, int64_t row, int64_t c) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.x) + row * a.ldx + c;
    if (vec && c < a.cols) {
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
  uint32_t w[8][2];
  float scale[8];                    // of the rows: a tile's columns are one block
  __device__ __forceinline__ float get(int i, int j) const {
    float lo, hi;
    q8_unpack2((uint16_t)(w[i][j >> 2] >> (16 * ((j >> 1) & 1))), lo, hi);
    return (j & 1 ? hi : lo) * scale[i];
  }
  __device__ __forceinline__ void set_nan(int i, int j) {}          // e4m3's only non-finite value is NaN already
  __device__ __forceinline__ void load(const Quant8Args& a, bool, int i, int64_t row, int64_t c) {
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

// Magnitude bits (fp32) of the 8 rows' and 8 columns' largest values in the thread's tile.
template <int IN>
__device__ __forceinline__ void quant_maxima(const QuantTile<IN>& v, unsigned (&rm)[8], unsigned (&cm)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rm[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned b = abs_bits(v.get(i, j));
      rm[i] = max(rm[i], b);
      cm[j] = max(cm[j], b);
    }
  }
}
template <>
__device__ __forceinline__ void quant_maxima<QIN_BF16>(const QuantTile<QIN_BF16>& v, unsigned (&rm)[8], unsigned (&cm)[8]) {
  uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = v.w[i][j] & 0x7FFF7FFFu;
      r = __vmaxu2(r, b);
      c[j] = __vmaxu2(c[j], b);
    }
    rm[i] = max(r << 16, r & 0xFFFF0000u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = j & 1 ? c[j >> 1] & 0xFFFF0000u : c[j >> 1] << 16;
}

template <int IN>
__global__ void __launch_bounds__(256, IN == QIN_F32 ? 2 : IN == QIN_BF16 ? 4 : 3) quantize8_kernel(Quant8Args a, int vec) {
  __shared__ __align__(16) uint8_t tr[128 * 128];
  __shared__ unsigned cmax[8][128];
  __shared__ unsigned char cexp[128];
  __shared__ unsigned tmax[4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t col_tiles = (a.cols + 127) >> 7, row_tiles = (a.rows + 127) >> 7;
  const int64_t tj = blockIdx.x % col_tiles, ti = blockIdx.x / col_tiles;
  const int64_t r0 = ti * 128 + 8 * ty, c0 = tj * 128 + 8 * tx;

  QuantTile<IN> v;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + i < a.rows) {
      v.load(a, vec, i, r0 + i, c0);
    } else {
#pragma unroll
      for (auto& x : v.w[i]) x = 0;
      if constexpr (IN == QIN_E4M3) v.scale[i] = 0.f;
    }
  }
  // row maxima (a half-warp holds a row) and column maxima (over the block)
  unsigned rexp[8], cm[8];
  quant_maxima<IN>(v, rexp, cm);
  unsigned most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, rexp[i]);
  if (__syncthreads_or(most >= INF_BITS)) {
    // somewhere in the tile a value is not finite: it becomes NaN and counts for no maximum
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      rexp[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned b = finite_bits(v.get(i, j));
        if (abs_bits(v.get(i, j)) >= INF_BITS) v.set_nan(i, j);
        rexp[i] = max(rexp[i], b);
        cm[j] = max(cm[j], b);
      }
    }
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
  } else if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) rexp[i] = max(rexp[i], __shfl_xor_sync(0xffffffffu, rexp[i], o));
      rexp[i] = q8_exponent(rexp[i]);
    }
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float inv = q8_inverse(rexp[i]);
      const uint2 b = make_uint2(q8_pack4(v.get(i, 0) * inv, v.get(i, 1) * inv, v.get(i, 2) * inv, v.get(i, 3) * inv),
                                 q8_pack4(v.get(i, 4) * inv, v.get(i, 5) * inv, v.get(i, 6) * inv, v.get(i, 7) * inv));
      if (r0 + i < a.rows) {
        uint8_t* p = a.q + (r0 + i) * a.ldq + c0;
        if (c0 + 8 <= a.cols) {
          *reinterpret_cast<uint2*>(p) = b;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c0 + j < a.cols) p[j] = (uint8_t)((j < 4 ? b.x : b.y) >> (8 * (j & 3)));
        }
      }
      if (tx == 0) a.s[q8_scale_at(r0 + i, (int)tj, row_tiles)] = (uint8_t)(r0 + i < a.rows ? rexp[i] : Q8_ONE);
    }
    // the blocks of the last group past the end
    if (tj == col_tiles - 1 && threadIdx.x < 128)
      for (int64_t kb = col_tiles; kb < 4 * (int64_t)q8_groups(a.cols); ++kb)
        a.s[q8_scale_at(ti * 128 + threadIdx.x, (int)kb, row_tiles)] = (uint8_t)Q8_ONE;
  }
  if (a.qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned b = a.tile ? rexp[0] : cexp[8 * tx + j];
      const float inv = q8_inverse(b);
      *reinterpret_cast<uint2*>(tr + (8 * tx + j) * 128 + ((ty ^ tx) << 3)) =
          make_uint2(q8_pack4(v.get(0, j) * inv, v.get(1, j) * inv, v.get(2, j) * inv, v.get(3, j) * inv),
                     q8_pack4(v.get(4, j) * inv, v.get(5, j) * inv, v.get(6, j) * inv, v.get(7, j) * inv));
      if (ty == 0) a.st[q8_scale_at(c0 + j, (int)ti, col_tiles)] = (uint8_t)(c0 + j < a.cols ? b : Q8_ONE);
    }
    if (ti == row_tiles - 1 && threadIdx.x < 128)
      for (int64_t kb = row_tiles; kb < 4 * (int64_t)q8_groups(a.rows); ++kb)
        a.st[q8_scale_at(tj * 128 + threadIdx.x, (int)kb, col_tiles)] = (uint8_t)Q8_ONE;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int piece = threadIdx.x + 256 * k;
      const int c = piece >> 3, p = piece & 7;       // column of the tile, 16-byte piece (rows 16 p ..)
      const int x = c >> 3;
      uint4 b = *reinterpret_cast<const uint4*>(tr + c * 128 + (((2 * p) ^ x) >> 1) * 16);
      if (x & 1) b = make_uint4(b.z, b.w, b.x, b.y);
      const int64_t oc = ti * 128 + 16 * p, orow = tj * 128 + c;
      if (orow < a.cols && oc < a.rows) {
        uint8_t* dst = a.qt + orow * a.ldqt + oc;
        if (oc + 16 <= a.rows) {
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
