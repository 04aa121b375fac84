// RMS norm of the residual stream with an 8-bit output, and its gradients.
//
//   h = x + r (kept in x's type),  rstd = 1 / sqrt(mean_c h^2 + eps),
//   y = h rstd w,  (q, scale) = the 8-bit form of y (form8.cuh)
//
//   n = h rstd,  g = dy w,  dx = dr + rstd (g - n mean_c(g n)),  dw = sum_rows dy n
//
// Both are bound by memory: 7 B an element forward (bf16 x, r, h and e4m3 q),
// 8 B backward (dy, h, dr, dx).  A row stays in the registers of `blockDim.x`
// threads, 8 consecutive columns a vector, so that a 128-column scale block is
// a half-warp and the row is read once; the block keeps its columns of w (and
// of the dw sum) for all of its rows, and loads the next row before it works
// on the present one.  Rows are joined by one barrier of the row's threads.
#pragma once

#include "form8.cuh"

namespace precond {

struct RmsNormArgs {
  const void* x; const void* r; const void* w; void* h; void* y;
  uint8_t* q; uint8_t* scale; float* rstd;
  int64_t rows, cols, ldx, ldr, ldh, ldy, ldq;
  float eps;
  int w_bf16;
};

struct RmsGradArgs {
  const void* dy; const void* x; const void* dr; const void* w; const float* rstd;
  void* dx; float* partial;           // partial: [gridDim.x * blockDim.y][cols]
  int64_t rows, cols, lddy, ldx, lddr, lddx;
  int w_bf16;
};

__device__ __forceinline__ float load_w(const void* w, int bf16, int64_t c) {
  return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c]) : reinterpret_cast<const float*>(w)[c];
}

// Sum over the blockDim.x threads of one row (blockDim.x a multiple of 32), the
// same value in each.  `red` has room for 2 x blockDim.y x 32; calls alternate
// between its halves, so that one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int half) {
  v = warp_sum(v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float* mine = red + (half * blockDim.y + threadIdx.y) * 32;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"((int)blockDim.x) : "memory");
  float s = 0.f;
  for (int i = 0; i < nw; ++i) s += mine[i];
  return s;
}

// One vector's 8-bit form, scale byte and plain output.
template <typename T, bool VEC>
__device__ __forceinline__ void norm_write(const RmsNormArgs& a, int64_t row, int64_t c, float (&y)[8], int64_t rblocks) {
  if (a.y) {
    Raw8<T> o;
    pack8(o, y);
    store8<VEC>(reinterpret_cast<T*>(a.y) + row * a.ldy, c, a.cols, o);
  }
  if (a.q) {
    const unsigned b = q8_block_exponent(y);
    const float inv = q8_inverse(b);
    store_q8(a.q + row * a.ldq, c, a.cols,
             make_uint2(q8_pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                        q8_pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv)));
    if ((threadIdx.x & 15) == 0 && c < a.cols) a.scale[q8_scale_at(row, (int)(c >> 7), rblocks)] = (uint8_t)b;
  }
}

// The scale bytes past the matrix's end: a row's trailing blocks, or a whole row of padding.
__device__ __forceinline__ void norm_pad(const RmsNormArgs& a, int64_t row, int64_t rblocks) {
  const int nkb = row < a.rows ? (int)((a.cols + 127) >> 7) : 0;
  for (int kb = nkb + threadIdx.x; kb < 4 * q8_groups(a.cols); kb += blockDim.x)
    a.scale[q8_scale_at(row, kb, rblocks)] = (uint8_t)Q8_ONE;
}

// NV vectors of 8 columns a thread.
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(512) rms_norm_kernel(RmsNormArgs a) {
  __shared__ float red[2 * 8 * 32];
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* r = reinterpret_cast<const T*>(a.r);
  T* h = reinterpret_cast<T*>(a.h);
  const int64_t rblocks = q8_row_blocks(a.rows);
  const int64_t last = a.q ? rblocks * 128 : a.rows;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t c[NV];
  float w[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = ((int64_t)j * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[j][i] = c[j] + i < a.cols ? load_w(a.w, a.w_bf16, c[j] + i) : 0.f;
  }
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  Raw8<T> nx[NV], nr[NV];
  if (row < a.rows) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load8<VEC>(nx[j], x + row * a.ldx, c[j], a.cols);
      if (r) load8<VEC>(nr[j], r + row * a.ldr, c[j], a.cols);
    }
  }
  for (int half = 0; row < last; row += step, half ^= 1) {
    if (a.q) norm_pad(a, row, rblocks);
    if (row >= a.rows) continue;
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack8(nx[j], v[j]);
      if (r) {
        float f[8];
        unpack8(nr[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += f[i];
        Raw8<T> o;
        pack8(o, v[j]);
        store8<VEC>(h + row * a.ldh, c[j], a.cols, o);
        unpack8(o, v[j]);                 // the norm is that of the stream as it is kept
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    }
    const int64_t next = row + step;
    if (next < a.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        load8<VEC>(nx[j], x + next * a.ldx, c[j], a.cols);
        if (r) load8<VEC>(nr[j], r + next * a.ldr, c[j], a.cols);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum(ss, red, half) / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (a.q || a.y) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] * rstd) * w[j][i];
        norm_write<T, VEC>(a, row, c[j], v[j], rblocks);
      }
    }
  }
}

// Rows too long for registers: one block a row, which is read again (from L2) after its norm is known.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(RmsNormArgs a) {
  __shared__ float red[2 * 32];
  const int64_t rblocks = q8_row_blocks(a.rows);
  const int64_t last = a.q ? rblocks * 128 : a.rows;
  const int64_t span = (a.cols + 8 * 1024 - 1) / (8 * 1024) * (8 * 1024);   // every lane takes part in the block maxima
  for (int64_t row = blockIdx.x, half = 0; row < last; row += gridDim.x, half ^= 1) {
    if (a.q) norm_pad(a, row, rblocks);
    if (row >= a.rows) continue;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* r = reinterpret_cast<const T*>(a.r) + row * a.ldr;
    T* h = reinterpret_cast<T*>(a.h) + row * a.ldh;
    float ss = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < span; c += 8 * 1024) {
      Raw8<T> o;
      float v[8];
      load8<VEC>(o, x, c, a.cols);
      unpack8(o, v);
      if (a.r) {
        float f[8];
        load8<VEC>(o, r, c, a.cols);
        unpack8(o, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
        pack8(o, v);
        store8<VEC>(h, c, a.cols, o);
        unpack8(o, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    }
    const float rstd = 1.0f / sqrtf(row_sum(ss, red, (int)half) / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (!a.q && !a.y) continue;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < span; c += 8 * 1024) {
      Raw8<T> o;
      float v[8];
      load8<VEC>(o, a.r ? h : x, c, a.cols);       // h: this thread's own stores
      unpack8(o, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < a.cols ? (v[i] * rstd) * load_w(a.w, a.w_bf16, c + i) : 0.f;
      norm_write<T, VEC>(a, row, c, v, rblocks);
    }
  }
}

// ------------------------------------------------------------- gradients
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(512) rms_grad_kernel(RmsGradArgs a) {
  __shared__ float red[2 * 8 * 32];
  const T* dy = reinterpret_cast<const T*>(a.dy);
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* dr = reinterpret_cast<const T*>(a.dr);
  T* dx = reinterpret_cast<T*>(a.dx);
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const float inv_cols = 1.0f / (float)a.cols;
  int64_t c[NV];
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = ((int64_t)j * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[j][i] = c[j] + i < a.cols ? load_w(a.w, a.w_bf16, c[j] + i) : 0.f;
      dw[j][i] = 0.f;
    }
  }
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  Raw8<T> ny[NV], nx[NV], nr[NV];
  float nrstd = 0.f;
  auto fetch = [&](int64_t k) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load8<VEC>(ny[j], dy + k * a.lddy, c[j], a.cols);
      load8<VEC>(nx[j], x + k * a.ldx, c[j], a.cols);
      if (dr) load8<VEC>(nr[j], dr + k * a.lddr, c[j], a.cols);
    }
    nrstd = a.rstd[k];
  };
  if (row < a.rows) fetch(row);
  for (int half = 0; row < a.rows; row += step, half ^= 1) {
    const float rstd = nrstd;
    float g[NV][8], n[NV][8];
    Raw8<T> res[NV];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack8(ny[j], g[j]);
      unpack8(nx[j], n[j]);
      if (dr) res[j] = nr[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[j][i] *= rstd;
        dw[j][i] = fmaf(g[j][i], n[j][i], dw[j][i]);
        g[j][i] *= w[j][i];
        dot = fmaf(g[j][i], n[j][i], dot);
      }
    }
    if (row + step < a.rows) fetch(row + step);
    const float mean = row_sum(dot, red, half) * inv_cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
      if (dr) unpack8(res[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = rstd * (g[j][i] - n[j][i] * mean);
        g[j][i] = dr ? d + f[i] : d;
      }
      Raw8<T> o;
      pack8(o, g[j]);
      store8<VEC>(dx + row * a.lddx, c[j], a.cols, o);
    }
  }
  float* out = a.partial + ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * a.cols;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c[j] + i < a.cols) out[c[j] + i] = dw[j][i];
}

// Rows too long for registers: the block's dw sums live in its row of `partial`
// (each thread adds to its own columns).
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) rms_grad_long_kernel(RmsGradArgs a) {
  __shared__ float red[2 * 32];
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  const float inv_cols = 1.0f / (float)a.cols;
  bool first = true;
  for (int64_t row = blockIdx.x, half = 0; row < a.rows; row += gridDim.x, half ^= 1) {
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.lddy;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* dr = reinterpret_cast<const T*>(a.dr) + row * a.lddr;
    T* dx = reinterpret_cast<T*>(a.dx) + row * a.lddx;
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += 8 * 1024) {
      Raw8<T> o;
      float g[8], n[8];
      load8<VEC>(o, dy, c, a.cols);
      unpack8(o, g);
      load8<VEC>(o, x, c, a.cols);
      unpack8(o, n);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < a.cols) {
          n[i] *= rstd;
          out[c + i] = first ? g[i] * n[i] : fmaf(g[i], n[i], out[c + i]);
          dot = fmaf(g[i] * load_w(a.w, a.w_bf16, c + i), n[i], dot);
        }
    }
    first = false;
    const float mean = row_sum(dot, red, (int)half) * inv_cols;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += 8 * 1024) {
      Raw8<T> o;
      float g[8], n[8], f[8];
      load8<VEC>(o, dy, c, a.cols);
      unpack8(o, g);
      load8<VEC>(o, x, c, a.cols);
      unpack8(o, n);
      if (a.dr) {
        load8<VEC>(o, dr, c, a.cols);
        unpack8(o, f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = c + i < a.cols ? load_w(a.w, a.w_bf16, c + i) : 0.f;
        const float d = rstd * (g[i] * w - (n[i] * rstd) * mean);
        g[i] = a.dr ? d + f[i] : d;
      }
      pack8(o, g);
      store8<VEC>(dx, c, a.cols, o);
    }
  }
}

// dw: the blocks' sums, added in their order (32 columns a block; 32 threads a
// column take every 32nd sum, then their results are added in order).
__global__ void __launch_bounds__(1024) rms_dw_kernel(const float* partial, int parts, int64_t cols, float* dw) {
  __shared__ float s[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < cols)
    for (int p = threadIdx.y; p < parts; p += 32) v += partial[(int64_t)p * cols + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int64_t o = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && o < cols) dw[o] = v;
}

}  // namespace precond
