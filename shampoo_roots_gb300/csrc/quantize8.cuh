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

// Columns c .. c + 7 of row `row` as fp32; zero outside the matrix.
template <int IN, bool VEC>
__device__ __forceinline__ void quant_load(const Quant8Args& a, int64_t row, int64_t c, float (&f)[8]) {
  if (IN == QIN_F32) {
    Raw8<float> o;
    load8<VEC>(o, reinterpret_cast<const float*>(a.x) + row * a.ldx, c, a.cols);
    unpack8(o, f);
  } else if (IN == QIN_BF16) {
    Raw8<__nv_bfloat16> o;
    load8<VEC>(o, reinterpret_cast<const __nv_bfloat16*>(a.x) + row * a.ldx, c, a.cols);
    unpack8(o, f);
  } else {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(a.x) + row * a.ldx + c;   // 16-byte aligned rows, c % 8 == 0
    uint2 b = make_uint2(0, 0);
    if (c + 8 <= a.cols) {
      b = *reinterpret_cast<const uint2*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < a.cols) (i < 4 ? b.x : b.y) |= (uint32_t)p[i] << (8 * (i & 3));
    }
    const float v = c < a.cols ? q8_value(a.x_scale[q8_scale_at(row, (int)(c >> 7), q8_row_blocks(a.rows))]) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? b.x : b.y;
      q8_unpack2((uint16_t)(w >> (16 * (i & 1))), f[2 * i], f[2 * i + 1]);
      f[2 * i] *= v;
      f[2 * i + 1] *= v;
    }
  }
}

template <int IN, bool VEC>
__global__ void __launch_bounds__(256) quantize8_kernel(Quant8Args a) {
  __shared__ __align__(16) uint8_t tr[128 * 128];
  __shared__ unsigned cmax[8][128];
  __shared__ unsigned char cexp[128];
  __shared__ unsigned tmax[4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t col_tiles = (a.cols + 127) >> 7, row_tiles = (a.rows + 127) >> 7;
  const int64_t tj = blockIdx.x % col_tiles, ti = blockIdx.x / col_tiles;
  const int64_t r0 = ti * 128 + 8 * ty, c0 = tj * 128 + 8 * tx;

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + i < a.rows) {
      quant_load<IN, VEC>(a, r0 + i, c0, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  unsigned any = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) any = max(any, abs_bits(v[i][j]));
  if (any >= INF_BITS) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = finite_or_nan(v[i][j]);
  }
  // row maxima (a half-warp holds a row) and column maxima (over the block); a NaN counts as nothing
  unsigned rexp[8], cm[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned b = any >= INF_BITS ? finite_bits(v[i][j]) : abs_bits(v[i][j]);
      m = max(m, b);
      cm[j] = max(cm[j], b);
    }
    rexp[i] = m;
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
      if (r0 + i < a.rows)
        store_q8(a.q + (r0 + i) * a.ldq, c0, a.cols,
                 make_uint2(q8_pack4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv),
                            q8_pack4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv)));
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
          make_uint2(q8_pack4(v[0][j] * inv, v[1][j] * inv, v[2][j] * inv, v[3][j] * inv),
                     q8_pack4(v[4][j] * inv, v[5][j] * inv, v[6][j] * inv, v[7][j] * inv));
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
