// RMS norm of the residual stream with an 8-bit output, and its gradients.
//
//   h = x + r (kept in x's type),  rstd = 1 / sqrt(mean_c h^2 + eps),
//   y = h rstd w,  (q, scale) = the 8-bit form of y (form8.cuh)
//
//   n = h rstd,  g = dy w,  dx = dr + rstd (g - n mean_c(g n)),  dw = sum_rows dy n
//
// Both are bound by memory: 7 B an element forward (bf16 x, r, h and e4m3 q),
// 8 B backward (dy, h, dr, dx).  A row stays in the registers of `blockDim.x`
// threads, 16 consecutive columns a vector, so that the row is read once; the
// block keeps its columns of w (and of the dw sum) for all of its rows, and
// loads the next row before it works on the present one.  The threads of a row
// meet at one barrier a row; those of a long row, in several blocks of a
// cluster, at words of their shared memory.
//
// Measured (bf16 with residual, as a fraction of the copy bandwidth): norm of
// 8192 x 6144 55.5 us, 94 %, of 3000 x 16384 58 us, 87 %; gradients of 16384 x
// 4096 88.3 us, 90 %, of 3000 x 16384 74 us, 78 % (the join of each row); in fp32
// norm of 8192 x 6144 100 us, 97 %, of 3000 x 16384 113 us, 83 %, gradients 188
// us, 84 %, and 159 us, 73 %.  Rows that do not begin at sectors cost the exchange
// of their elements through shared memory, and at 126 registers a thread an SM
// holds too few warps to cover it (issue 56 % of the time): 7000 x 2001 27 us,
// 53 %, gradients 39 us, 42 %.  dw leaves in fp32 sums of a block's rows, at most
// 4 an SM, which a second kernel adds in their order (16384 x 4096: 304 sums, 5
// MB, 6 us).
#pragma once

#include "rows.cuh"

namespace precond {

struct RmsNormArgs {
  const void* x; const void* r; const void* w; void* h; void* y;
  uint8_t* q; uint8_t* scale; float* rstd;
  int64_t ldx, ldr, ldh, ldy, ldq;
  int rows, cols;
  float eps;
  int w_bf16;
};

struct RmsGradArgs {
  const void* dy; const void* x; const void* dr; const void* w; const float* rstd;
  void* dx; float* partial;           // partial: [blocks, or clusters][cols]
  int64_t lddy, ldx, lddr, lddx;
  int rows, cols;
  int w_bf16;
};

// NV vectors of 16 columns a thread (NV 2: whole blocks, aligned rows).  Rows of
// up to 256 columns share a warp (ROW_PART, blockDim.x 8 or 16): its lanes stay
// together, and rows past the last count as rows of no columns.
template <typename T, int NV, bool VEC, int ROWS>
__global__ void __launch_bounds__(NV == 2 || (sizeof(T) == 2 && !VEC) ? 512 : 384, NV == 1 && sizeof(T) == 2 && VEC ? 2 : 1)
    rms_norm_kernel(RmsNormArgs a) {
  constexpr bool CLUSTER = ROWS == ROW_CLUSTER, PART = ROWS == ROW_PART;
  __shared__ __align__(16) float red[2 * 8 * 32];      // of a cluster: its 2 x 8 x 16 words
  zero_red(red, 2 * 8 * 32);
  if (CLUSTER) cg::this_cluster().sync();
  wait_for_previous();
  let_next_start();
  void* xs = warp_scratch<T, VEC>();
  const int64_t rblocks = q8_row_blocks(a.rows);
  const int parts = CLUSTER ? (int)cg::this_cluster().num_blocks() : 1, rank = CLUSTER ? (int)cg::this_cluster().block_rank() : 0;
  const int step = gridDim.x / parts * blockDim.y;
  int row = blockIdx.x / parts * blockDim.y + threadIdx.y;
  const int below = PART ? (threadIdx.x + threadIdx.y * blockDim.x) % 32 / blockDim.x : 0;   // rows below it in its warp
  int cols = !PART || row < a.rows ? a.cols : 0;
  // rows' addresses are formed anew: pointers kept from row to row cost registers that the vectors need
  auto x = [&](int64_t k) { return reinterpret_cast<const T*>(a.x) + k * a.ldx; };
  auto r = [&](int64_t k) { return reinterpret_cast<const T*>(a.r) + k * a.ldr; };
  const float inv_cols = 1.0f / (float)a.cols;
  F16 w[NV];
  int c[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = ((j + rank) * (int)blockDim.x + threadIdx.x) * 16;        // one of j and rank is 0
    w[j] = load_w16(a.w, a.w_bf16, c[j], a.cols);
  }
  Raw16<T> nx[NV], nr[NV];
  bool lost = false;
  if (row - below < a.rows) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load16<VEC>(nx[j], x(row), c[j], cols);
      if (a.r) load16<VEC>(nr[j], r(row), c[j], cols);
    }
  }
  for (unsigned call = 1; row - below < a.rows; row += step, ++call) {
    F16 v[NV];
    f2 ss = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      settle<VEC>(nx[j], xs);
      if (a.r) {
        settle<VEC>(nr[j], xs);
        add_stream(nx[j], nr[j]);
        store16<VEC>(reinterpret_cast<T*>(a.h) + row * a.ldh, c[j], cols, nx[j], xs);
      }
      v[j] = unpack(nx[j]);
      ss = squares(v[j], ss);
    }
    const int next = !PART || row + step < a.rows ? a.cols : 0;
    if (row + step - below < a.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        load16<VEC>(nx[j], x(row + step), c[j], next);
        if (a.r) load16<VEC>(nr[j], r(row + step), c[j], next);
      }
    }
    const float sum = CLUSTER ? cluster_row_sum(sum2(ss), reinterpret_cast<unsigned long long*>(red), call, lost)
                              : row_sum<PART>(sum2(ss), red, call & 1);
    const float rstd = rstd_of(sum, inv_cols, a.eps);
    if (a.rstd && threadIdx.x == 0 && rank == 0 && cols) a.rstd[row] = rstd;
    if (a.q || a.y) {
      const f2 rs = f2_of(rstd, rstd);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j].p[i] = mul2(mul2(v[j].p[i], rs), w[j].p[i]);
        norm_write<T, VEC>(a, row, c[j], cols, v[j], q8_scale_at(row, c[j] >> 7, rblocks), xs);
      }
      if (a.q && (a.cols & 511) && rank == 0 && row < rblocks * 128) norm_pad(a, row, rblocks);
    }
    cols = next;
  }
  if (a.q && rank == 0)
    for (; row < rblocks * 128; row += step) norm_pad(a, row, rblocks);
  if (CLUSTER) cluster_leave();
}

// Rows too long for registers: one block a row, which is read again (from L2) after its norm is known.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512, 2) rms_norm_long_kernel(RmsNormArgs a) {
  __shared__ __align__(16) float red[2 * 32];
  zero_red(red, 2 * 32);
  wait_for_previous();
  let_next_start();
  void* xs = warp_scratch<T, VEC>();
  const int64_t rblocks = q8_row_blocks(a.rows);
  const int64_t last = a.q ? rblocks * 128 : a.rows;
  const int64_t stride = 16 * blockDim.x, span = (a.cols + stride - 1) / stride * stride;   // whole warps
  const float inv_cols = 1.0f / (float)a.cols;
  int half = 0;
  for (int64_t row = blockIdx.x; row < last; row += gridDim.x, half ^= 1) {
    if (a.q) norm_pad(a, row, rblocks);
    if (row >= a.rows) continue;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* r = reinterpret_cast<const T*>(a.r) + row * a.ldr;
    T* h = reinterpret_cast<T*>(a.h) + row * a.ldh;
    f2 ss = 0;
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o, p;
      load16<VEC>(o, x, (int)c, a.cols);
      settle<VEC>(o, xs);
      if (a.r) {
        load16<VEC>(p, r, (int)c, a.cols);
        settle<VEC>(p, xs);
        add_stream(o, p);
        store16<VEC>(h, (int)c, a.cols, o, xs);
      }
      ss = squares(unpack(o), ss);
    }
    const float rstd = rstd_of(row_sum<false>(sum2(ss), red, half), inv_cols, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (!a.q && !a.y) continue;
    const f2 rs = f2_of(rstd, rstd);
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o;
      load16<VEC>(o, a.r ? h : x, (int)c, a.cols);       // h: this warp's own stores
      settle<VEC>(o, xs);
      F16 v = unpack(o);
      const F16 w = load_w16(a.w, a.w_bf16, (int)c, a.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) v.p[i] = mul2(mul2(v.p[i], rs), w.p[i]);
      const int kb = (int)(c >> 7);
      norm_write<T, VEC>(a, row, (int)c, a.cols, v, q8_scale_at(row, kb, rblocks), xs);
    }
  }
}

// ------------------------------------------------------------- gradients
// One vector: g = dy w, n = x rstd; adds to dw and to the row's g n.
__device__ __forceinline__ f2 grad_terms(F16& g, F16& n, const F16& w, F16& dw, f2 rs, f2 dot) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    n.p[i] = mul2(n.p[i], rs);
    dw.p[i] = fma2(g.p[i], n.p[i], dw.p[i]);
    g.p[i] = mul2(g.p[i], w.p[i]);
    dot = fma2(g.p[i], n.p[i], dot);
  }
  return dot;
}
// dx = rstd (g - n mean) (+ dr)
template <typename T>
__device__ __forceinline__ void grad_out(Raw16<T>& o, const F16& g, const F16& n, f2 rs, f2 minus_mean, bool add, const Raw16<T>& dr) {
  F16 d;
#pragma unroll
  for (int i = 0; i < 8; ++i) d.p[i] = mul2(rs, fma2(n.p[i], minus_mean, g.p[i]));
  if (add) {
    const F16 f = unpack(dr);
#pragma unroll
    for (int i = 0; i < 8; ++i) d.p[i] = add2(d.p[i], f.p[i]);
  }
  pack(o, d);
}

// fp32 takes 168 registers a thread: with 128 the vectors in flight do not fit.
template <typename T, bool VEC, int ROWS>
__global__ void __launch_bounds__(sizeof(T) == 4 ? 384 : 512, 1) rms_grad_kernel(RmsGradArgs a) {
  __shared__ __align__(16) float red[2 * 8 * 32];      // of a cluster: its 2 x 8 x 16 words
  zero_red(red, 2 * 8 * 32);
  constexpr bool CLUSTER = ROWS == ROW_CLUSTER, PART = ROWS == ROW_PART;
  constexpr bool EARLY = sizeof(T) == 2 && VEC;        // dr with the row's other vectors (else there is no room for it)
  if (CLUSTER) cg::this_cluster().sync();
  wait_for_previous();
  let_next_start();
  void* xs = warp_scratch<T, VEC>();
  const int parts = CLUSTER ? (int)cg::this_cluster().num_blocks() : 1;
  const int group = CLUSTER ? blockIdx.x / parts : blockIdx.x;          // of blocks that share rows
  const int step = (CLUSTER ? gridDim.x / parts : gridDim.x) * blockDim.y;
  int row = group * blockDim.y + threadIdx.y;
  const int below = PART ? (threadIdx.x + threadIdx.y * blockDim.x) % 32 / blockDim.x : 0;   // as in the norm
  int cols = !PART || row < a.rows ? a.cols : 0;
  // addresses formed anew, as in the norm
  auto dy = [&](int64_t k) { return reinterpret_cast<const T*>(a.dy) + k * a.lddy; };
  auto x = [&](int64_t k) { return reinterpret_cast<const T*>(a.x) + k * a.ldx; };
  auto dr = [&](int64_t k) { return reinterpret_cast<const T*>(a.dr) + k * a.lddr; };
  const float inv_cols = 1.0f / (float)a.cols;
  const int c = ((CLUSTER ? (int)cg::this_cluster().block_rank() * (int)blockDim.x : 0) + threadIdx.x) * 16;
  const F16 w = load_w16(a.w, a.w_bf16, c, a.cols);
  F16 dw;
#pragma unroll
  for (int i = 0; i < 8; ++i) dw.p[i] = 0;
  Raw16<T> ny, nx, nr;
  float nrstd = 0.f;
  bool lost = false;
  if (row - below < a.rows) {
    load16<VEC>(ny, dy(row), c, cols);
    load16<VEC>(nx, x(row), c, cols);
    if (a.dr) load16<VEC>(nr, dr(row), c, cols);
    if (cols) nrstd = a.rstd[row];
  }
  for (unsigned call = 1; row - below < a.rows; row += step, ++call) {
    const f2 rs = f2_of(nrstd, nrstd);
    const bool more = row + step - below < a.rows;
    const int next = !PART || row + step < a.rows ? a.cols : 0;
    Raw16<T> res = nr;
    settle<VEC>(ny, xs);
    settle<VEC>(nx, xs);
    F16 g = unpack(ny), n = unpack(nx);
    const f2 dot = grad_terms(g, n, w, dw, rs, 0);
    if (more) {
      load16<VEC>(ny, dy(row + step), c, next);
      load16<VEC>(nx, x(row + step), c, next);
      if (EARLY && a.dr) load16<VEC>(nr, dr(row + step), c, next);
      if (next) nrstd = a.rstd[row + step];
    }
    const float sum = CLUSTER ? cluster_row_sum(sum2(dot), reinterpret_cast<unsigned long long*>(red), call, lost)
                              : row_sum<PART>(sum2(dot), red, call & 1);
    const float mean = -sum * inv_cols;
    Raw16<T> o;
    if (a.dr) settle<VEC>(res, xs);
    grad_out(o, g, n, rs, f2_of(mean, mean), a.dr != nullptr, res);
    if (!EARLY && more && a.dr) load16<VEC>(nr, dr(row + step), c, next);    // used after the next row's join
    store16<VEC>(reinterpret_cast<T*>(a.dx) + row * a.lddx, c, cols, o, xs);
    cols = next;
  }
  if (CLUSTER) cluster_leave();
  if (blockDim.y > 1) {                  // the block's rows side by side: in their order, through shared memory
    extern __shared__ __align__(16) uint8_t row_scratch[];
    F16* side = reinterpret_cast<F16*>(row_scratch);
    __syncthreads();                     // the exchange buffers lie there too
    side[threadIdx.y * blockDim.x + threadIdx.x] = dw;
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (int y = 1; y < blockDim.y; ++y)
#pragma unroll
      for (int i = 0; i < 8; ++i) dw.p[i] = add2(dw.p[i], side[y * blockDim.x + threadIdx.x].p[i]);
  }
  float* out = a.partial + (int64_t)group * a.cols;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 d = f2_get(dw.p[i]);
    if (c + 2 * i < a.cols) out[c + 2 * i] = d.x;
    if (c + 2 * i + 1 < a.cols) out[c + 2 * i + 1] = d.y;
  }
}

// Rows too long for registers: the block's dw sums live in its row of `partial`
// (each thread adds to its own columns).
template <typename T, bool VEC>
__global__ void __launch_bounds__(512, 1) rms_grad_long_kernel(RmsGradArgs a) {
  __shared__ __align__(16) float red[2 * 32];
  zero_red(red, 2 * 32);
  wait_for_previous();
  let_next_start();
  void* xs = warp_scratch<T, VEC>();
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  const float inv_cols = 1.0f / (float)a.cols;
  const int64_t stride = 16 * blockDim.x, span = (a.cols + stride - 1) / stride * stride;   // whole warps
  bool first = true;
  int half = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, half ^= 1) {
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.lddy;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* dr = reinterpret_cast<const T*>(a.dr) + row * a.lddr;
    T* dx = reinterpret_cast<T*>(a.dx) + row * a.lddx;
    const f2 rs = f2_of(a.rstd[row], a.rstd[row]);
    f2 dot = 0;
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o;
      load16<VEC>(o, dy, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 g = unpack(o);
      load16<VEC>(o, x, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 n = unpack(o), dw;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dw.p[i] = f2_of(first || c + 2 * i >= a.cols ? 0.f : out[c + 2 * i], first || c + 2 * i + 1 >= a.cols ? 0.f : out[c + 2 * i + 1]);
      dot = grad_terms(g, n, load_w16(a.w, a.w_bf16, (int)c, a.cols), dw, rs, dot);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 d = f2_get(dw.p[i]);
        if (c + 2 * i < a.cols) out[c + 2 * i] = d.x;
        if (c + 2 * i + 1 < a.cols) out[c + 2 * i + 1] = d.y;
      }
    }
    first = false;
    const float mean = -row_sum<false>(sum2(dot), red, half) * inv_cols;
    const f2 mm = f2_of(mean, mean);
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o, res;
      load16<VEC>(o, dy, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 g = unpack(o);
      load16<VEC>(o, x, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 n = unpack(o);
      const F16 w = load_w16(a.w, a.w_bf16, (int)c, a.cols);
      if (a.dr) {
        load16<VEC>(res, dr, (int)c, a.cols);
        settle<VEC>(res, xs);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n.p[i] = mul2(n.p[i], rs);
        g.p[i] = mul2(g.p[i], w.p[i]);
      }
      grad_out(o, g, n, rs, mm, a.dr != nullptr, res);
      store16<VEC>(dx, (int)c, a.cols, o, xs);
    }
  }
}

// dw: the blocks' sums, added in their order (32 columns a block; 32 threads a
// column take every 32nd sum, then their results are added in order).
__global__ void __launch_bounds__(1024) rms_dw_kernel(const float* partial, int parts, int64_t cols, float* dw) {
  __shared__ float s[32][33];
  wait_for_previous();
  let_next_start();
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += 32) v += partial[(int64_t)p * cols + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int64_t o = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && o < cols) dw[o] = v;
}

}  // namespace precond
