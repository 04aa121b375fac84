// Layer norm of the residual stream, kept or in 8 bits, and its gradients.
//
//   h = x + r (kept in x's type),  mean = sum_c h / C,  rstd = 1 / sqrt(sum_c (h - mean)^2 / C + eps),
//   y = (h - mean) rstd w + b,  (q, scale) = the 8-bit form of y (form8.cuh)
//
//   n = (h - mean) rstd,  g = dy w,  dx = dr + rstd (g - mean_c(g) - n mean_c(g n)),
//   dw = sum_rows dy n,  db = sum_rows dy
//
// Rows lie on threads as for the RMS norm (rows.cuh): read once, 16 columns a
// thread.  Where there are many, they come through a ring in shared memory (below);
// otherwise the next row's loads are under way, in registers, while the present one
// is worked on.
//
// The squares are those of h - mean, never a difference of sums.  So that a row
// meets once and not twice, each warp takes the mean and the squared deviations
// of its own columns (n_i, m_i, S_i), and the row's threads join them as Chan,
// Golub and LeVeque do:  mean = sum n_i m_i / C,  S = sum S_i + n_i (m_i - mean)^2.
// Gradients join their two sums at once.
//
// w and b lie in shared memory, where a thread's four columns are one load and a
// warp's loads meet no bank twice: in registers beside the vectors in flight they
// would leave room for half the warps.
//
// Measured (bf16 with residual): norm of 8192 x 6144 to 8 bits 56 us, 93 % of the
// copy bandwidth; gradients of 16384 x 4096 85 us, 93 %; in fp32 norm of 8192 x 6144
// 106 us, gradients of 8000 x 6144 121 us, 96 %.  What bounds them below that is
// issue slots (64 % busy at 24 warps an SM) and the latency of a row's sums: 18
// shuffles one after another, which is why lanes join means and deviations in one
// butterfly.  Rows that do not begin at sectors pass through the exchange of
// form8.cuh: gradients of 7000 x 2001 40 us, 41 %.
#pragma once

#include <type_traits>

#include "ptx.cuh"
#include "rows.cuh"

namespace precond {

struct LayerNormArgs {
  const void* x; const void* r; const void* w; const void* b; void* h; void* y;
  uint8_t* q; uint8_t* scale; float* mean; float* rstd;
  int64_t ldx, ldr, ldh, ldy, ldq;
  int rows, cols;
  float eps;
  int w_bf16;
};

struct LayerGradArgs {
  const void* dy; const void* x; const void* dr; const void* w; const float* mean; const float* rstd;
  void* dx; float* partial;           // partial: [blocks, or clusters][dw, db][columns, padded to 16]
  float* dw; float* db;               // few rows: the sums themselves, of one block or of one cluster's; else null
  int64_t lddy, ldx, lddr, lddx;
  int rows, cols;
  int w_bf16;
};

// Columns of the 32 threads that begin at `thread`, of a row whose threads have 16 each.
__device__ __forceinline__ int warp_columns(int cols, int thread) { return min(max(cols - thread * 16, 0), 512); }

// 16 columns of w (or b) in the table that a block keeps: [vector][4 columns][thread].
__device__ __forceinline__ void table_set(float4* t, int stride, const F16& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f2_get(f.p[2 * i]), b = f2_get(f.p[2 * i + 1]);
    t[i * stride] = make_float4(a.x, a.y, b.x, b.y);
  }
}
__device__ __forceinline__ F16 table_get(const float4* t, int stride) {
  F16 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = t[i * stride];
    f.p[2 * i] = f2_of(v.x, v.y);
    f.p[2 * i + 1] = f2_of(v.z, v.w);
  }
  return f;
}
__device__ __forceinline__ F16 zero16() {
  F16 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.p[i] = 0;
  return f;
}

__device__ __forceinline__ f2 total16(const F16& v, f2 s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s = add2(s, v.p[i]);
  return s;
}
// Squared deviations from m of the first `valid` of 16 columns.
__device__ __forceinline__ f2 deviations(const F16& v, float m, int valid, f2 s) {
  const f2 mm = f2_of(-m, -m);
  if (valid >= 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f2 d = add2(v.p[i], mm);
      s = fma2(d, d, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 d = f2_get(add2(v.p[i], mm));
      const f2 e = f2_of(2 * i < valid ? d.x : 0.f, 2 * i + 1 < valid ? d.y : 0.f);
      s = fma2(e, e, s);
    }
  }
  return s;
}

// Two sums over the lanes of a row that shares a warp.
__device__ __forceinline__ void part_sums(float& a, float& b) {
#pragma unroll 1
  for (int o = blockDim.x >> 1; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
}

// What a row's warps leave for one another: two values a warp, for two rows in
// turn; and the number of columns of each warp, and its inverse.
struct RowWords {
  float2 value[2][8][16];              // [row in turn][threadIdx.y][warp]
  float2 columns[16];
};
// Of a cluster: the same as words that also hold the number of the row (cluster_row_sum).
struct ClusterWords {
  unsigned long long value[2][2][128]; // [row in turn][which][block * 16 + warp]
};
__device__ __forceinline__ float2* row_exchange(RowWords& w, float a, float b, int half) {
  float2* mine = w.value[half][threadIdx.y];
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"((int)blockDim.x) : "memory");
  return mine;
}
// This warp's two values to every block of the cluster, and the values of all of
// its warps, up to 4 a lane (lane + 32 k = block * 16 + warp).  Bounds and order
// are those of cluster_row_sum; a wait that runs out makes the values NaN.
__device__ __forceinline__ void cluster_exchange(ClusterWords& w, float a, float b, unsigned call, bool& lost, float2 (&got)[4]) {
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  unsigned long long* mine = w.value[call & 1][0];
  if (lane < 2 * parts) {                              // lanes 0, 2, ... the first value to block lane / 2, the others the second
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(mine + (lane & 1) * 128 + cluster.block_rank() * 16 + (threadIdx.x >> 5))), "r"(lane >> 1));
    asm volatile("st.relaxed.cluster.shared::cluster.u64 [%0], %1;"
                 ::"r"(to), "l"((unsigned long long)call << 32 | __float_as_uint(lane & 1 ? b : a)) : "memory");
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) got[k] = make_float2(0.f, 0.f);
  for (int spin = 0; !lost; ++spin) {
    bool here = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane + 32 * k;
      if (32 * k < 16 * parts && i < 16 * parts && (i & 15) < nw) {
        unsigned long long one, two;
        asm volatile("ld.relaxed.cluster.shared::cta.u64 %0, [%1];"
                     : "=l"(one) : "r"((uint32_t)__cvta_generic_to_shared(mine + i)) : "memory");
        asm volatile("ld.relaxed.cluster.shared::cta.u64 %0, [%1];"
                     : "=l"(two) : "r"((uint32_t)__cvta_generic_to_shared(mine + 128 + i)) : "memory");
        here = here && (unsigned)(one >> 32) == call && (unsigned)(two >> 32) == call;
        got[k] = make_float2(__uint_as_float((unsigned)one), __uint_as_float((unsigned)two));
      }
    }
    if (__all_sync(0xffffffffu, here)) break;
    lost = spin > 10000000;                            // seconds: every lane counts the same
  }
  if (lost) got[0] = make_float2(__uint_as_float(0x7FFFFFFFu), __uint_as_float(0x7FFFFFFFu));
}

// Sum over the warps' values, a warp a lane: the warps that are there come first, the others are zero.
__device__ __forceinline__ float sum_warps(float v) {
  if (blockDim.x > 512) v += __shfl_xor_sync(0xffffffffu, v, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int warp_lane() { return threadIdx.x & (blockDim.x > 512 ? 31 : 15); }
// mean and squared deviations of a row from its warps' (sum, squared deviations).
__device__ __forceinline__ float2 row_moments(const float2* mine, const float2* columns, float inv_cols) {
  const float2 v = mine[warp_lane()], n = columns[warp_lane()];
  const float mean = sum_warps(v.x) * inv_cols;
  const float d = fmaf(v.x, n.y, -mean);
  return make_float2(mean, sum_warps(fmaf(n.x * d, d, v.y)));
}
__device__ __forceinline__ float2 cluster_moments(const float2 (&got)[4], int cols, float inv_cols) {
  const int lane = threadIdx.x & 31;
  const float mean = warp_sum((got[0].x + got[1].x) + (got[2].x + got[3].x)) * inv_cols;
  float dev = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k, n = (i & 15) * 32 < blockDim.x ? warp_columns(cols, (i >> 4) * blockDim.x + (i & 15) * 32) : 0;
    const float d = n == 512 ? fmaf(got[k].x, 1.f / 512, -mean) : n ? got[k].x / (float)n - mean : 0.f;
    dev += fmaf((float)n * d, d, got[k].y);
  }
  return make_float2(mean, warp_sum(dev));
}

// NV vectors of 16 columns a thread, as in the RMS norm.
template <typename T, int NV, bool VEC, int ROWS>
__global__ void __launch_bounds__(NV == 2 || (sizeof(T) == 2 && !VEC) ? 512 : 384, NV == 1 && sizeof(T) == 2 && VEC ? 2 : 1)
    layer_norm_kernel(LayerNormArgs a) {
  constexpr bool CLUSTER = ROWS == ROW_CLUSTER, PART = ROWS == ROW_PART;
  __shared__ __align__(16) typename std::conditional<CLUSTER, ClusterWords, RowWords>::type words;
  extern __shared__ __align__(16) uint8_t row_scratch[];
  zero_red(reinterpret_cast<float*>(&words), sizeof(words) / 4);
  if (CLUSTER) cg::this_cluster().sync();
  wait_for_previous();
  let_next_start();
  const int bx = blockDim.x, tx = threadIdx.x;
  float4* table = reinterpret_cast<float4*>(row_scratch) + tx;
  void* xs = VEC ? nullptr : row_scratch + bx * NV * 128 + ((threadIdx.y * bx + tx) >> 5) * Scratch<T>::BYTES;
  const int64_t rblocks = q8_row_blocks(a.rows);
  const int parts = CLUSTER ? (int)cg::this_cluster().num_blocks() : 1, rank = CLUSTER ? (int)cg::this_cluster().block_rank() : 0;
  const int step = gridDim.x / parts * blockDim.y;
  int row = blockIdx.x / parts * blockDim.y + threadIdx.y;
  const int below = PART ? (tx + threadIdx.y * bx) % 32 / bx : 0;      // rows below it in its warp
  int cols = !PART || row < a.rows ? a.cols : 0;
  auto x = [&](int64_t k) { return reinterpret_cast<const T*>(a.x) + k * a.ldx; };
  auto r = [&](int64_t k) { return reinterpret_cast<const T*>(a.r) + k * a.ldr; };
  const float inv_cols = 1.0f / (float)a.cols;
  int c[NV], mine = 0;                                                 // mine: columns of this warp
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = ((j + rank) * bx + tx) * 16;                                // one of j and rank is 0
    mine += warp_columns(a.cols, (j + rank) * bx + (tx & ~31));
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
  if (threadIdx.y == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      table_set(table + j * 8 * bx, bx, load_w16_wide(a.w, a.w_bf16, c[j], a.cols));
      table_set(table + (j * 8 + 4) * bx, bx, a.b ? load_w16_wide(a.b, a.w_bf16, c[j], a.cols) : zero16());
    }
    if constexpr (!CLUSTER)
      if (!PART && (tx & 31) == 0) words.columns[tx >> 5] = make_float2((float)mine, mine ? 1.f / (float)mine : 0.f);
  }
  __syncthreads();
  const float inv_mine = mine ? 1.f / (float)mine : 0.f;
  for (unsigned call = 1; row - below < a.rows; row += step, ++call) {
    Raw16<T> h[NV];                      // as stored: unpacked where it is used, which costs less than the registers
    f2 s = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      settle<VEC>(nx[j], xs);
      if (a.r) {
        settle<VEC>(nr[j], xs);
        add_stream(nx[j], nr[j]);
        store16<VEC>(reinterpret_cast<T*>(a.h) + row * a.ldh, c[j], cols, nx[j], xs);
      }
      h[j] = nx[j];
      s = total16(unpack(h[j]), s);
    }
    const int next = !PART || row + step < a.rows ? a.cols : 0;
    if (row + step - below < a.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        load16<VEC>(nx[j], x(row + step), c[j], next);
        if (a.r) load16<VEC>(nr[j], r(row + step), c[j], next);
      }
    }
    float sum = sum2(s), none = 0.f;
    if (PART) part_sums(sum, none);
    else sum = warp_sum(sum);
    float2 m = make_float2(sum * (PART ? inv_cols : inv_mine), 0.f);
    f2 d2 = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) d2 = deviations(unpack(h[j]), m.x, cols - c[j], d2);
    m.y = sum2(d2);
    if (PART) {
      part_sums(m.y, none);
    } else {
      m.y = warp_sum(m.y);
      if constexpr (CLUSTER) {
        float2 got[4];
        cluster_exchange(words, sum, m.y, call, lost, got);
        m = cluster_moments(got, a.cols, inv_cols);
      } else if (bx > 32) {
        m = row_moments(row_exchange(words, sum, m.y, call & 1), words.columns, inv_cols);
      }
    }
    const float rstd = rstd_of(m.y, inv_cols, a.eps);
    if (tx == 0 && rank == 0 && cols) {
      if (a.mean) a.mean[row] = m.x;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (a.q || a.y) {
      const f2 rs = f2_of(rstd, rstd), mm = f2_of(-m.x, -m.x);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        F16 v = unpack(h[j]);
        const F16 w = table_get(table + j * 8 * bx, bx), b = table_get(table + (j * 8 + 4) * bx, bx);
#pragma unroll
        for (int i = 0; i < 8; ++i) v.p[i] = fma2(mul2(add2(v.p[i], mm), rs), w.p[i], b.p[i]);
        norm_write<T, VEC>(a, row, c[j], cols, v, q8_scale_at(row, c[j] >> 7, rblocks), xs);
      }
      if (a.q && (a.cols & 511) && rank == 0 && row < rblocks * 128) norm_pad(a, row, rblocks);
    }
    cols = next;
  }
  if (a.q && rank == 0)
    for (; row < rblocks * 128; row += step) norm_pad(a, row, rblocks);
  if (CLUSTER) cluster_leave();
}

// Rows too long for registers: one block a row, which is read again (from L2) for its deviations and for y.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512, 2) layer_norm_long_kernel(LayerNormArgs a) {
  __shared__ __align__(16) float red[2 * 32];
  zero_red(red, 2 * 32);
  wait_for_previous();
  let_next_start();
  void* xs = warp_scratch<T, VEC>();
  const int64_t rblocks = q8_row_blocks(a.rows);
  const int64_t last = a.q ? rblocks * 128 : a.rows;
  const int64_t stride = 16 * blockDim.x, span = (a.cols + stride - 1) / stride * stride;   // whole warps
  const float inv_cols = 1.0f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < last; row += gridDim.x) {
    if (a.q) norm_pad(a, row, rblocks);
    if (row >= a.rows) continue;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* r = reinterpret_cast<const T*>(a.r) + row * a.ldr;
    T* h = reinterpret_cast<T*>(a.h) + row * a.ldh;
    f2 s = 0;
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
      s = total16(unpack(o), s);
    }
    const float mean = row_sum<false>(sum2(s), red, 0) * inv_cols;
    f2 d2 = 0;
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o;
      load16<VEC>(o, a.r ? h : x, (int)c, a.cols);       // h: this warp's own stores
      settle<VEC>(o, xs);
      d2 = deviations(unpack(o), mean, a.cols - (int)c, d2);
    }
    const float rstd = rstd_of(row_sum<false>(sum2(d2), red, 1), inv_cols, a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (!a.q && !a.y) continue;
    const f2 rs = f2_of(rstd, rstd), mm = f2_of(-mean, -mean);
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o;
      load16<VEC>(o, a.r ? h : x, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 v = unpack(o);
      const F16 w = load_w16_wide(a.w, a.w_bf16, (int)c, a.cols), b = a.b ? load_w16_wide(a.b, a.w_bf16, (int)c, a.cols) : zero16();
#pragma unroll
      for (int i = 0; i < 8; ++i) v.p[i] = fma2(mul2(add2(v.p[i], mm), rs), w.p[i], b.p[i]);
      norm_write<T, VEC>(a, row, (int)c, a.cols, v, q8_scale_at(row, (int)(c >> 7), rblocks), xs);
    }
  }
}

// ------------------------------------------------------------- gradients
// dw and db of the rows that a block has side by side, added in their order by the threads of the first; through shared
// memory, 4 columns at a time and thread by thread, so that no bank is met twice.
__device__ __forceinline__ void join_rows(float4* side, F16& dw, F16& db) {
  const int bx = blockDim.x, stride = bx * blockDim.y;
  float4* at = side + threadIdx.x;
  __syncthreads();                       // what lay there has been read
  if (threadIdx.y > 0) {
    table_set(at + threadIdx.y * bx, stride, dw);
    table_set(at + threadIdx.y * bx + 4 * stride, stride, db);
  }
  __syncthreads();
  if (threadIdx.y == 0)
    for (int y = 1; y < blockDim.y; ++y) {
      const F16 w2 = table_get(at + y * bx, stride), b2 = table_get(at + y * bx + 4 * stride, stride);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw.p[i] = add2(dw.p[i], w2.p[i]);
        db.p[i] = add2(db.p[i], b2.p[i]);
      }
    }
}
// The same over the blocks of a cluster: each thread's columns by one of them (`mine`).
__device__ __forceinline__ void join_blocks(float4* side, F16& dw, F16& db, bool mine) {
  cg::cluster_group cluster = cg::this_cluster();
  const int bx = blockDim.x, n = (int)cluster.num_blocks();
  float4* at = side + threadIdx.x;
  __syncthreads();
  if (threadIdx.y == 0) {
    table_set(at, bx, dw);
    table_set(at + 4 * bx, bx, db);
  }
  cluster.sync();
  if (mine) {
    dw = db = zero16();
    for (int k = 0; k < n; ++k) {
      const float4* other = cluster.map_shared_rank(at, k);
      const F16 w2 = table_get(other, bx), b2 = table_get(other + 4 * bx, bx);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw.p[i] = add2(dw.p[i], w2.p[i]);
        db.p[i] = add2(db.p[i], b2.p[i]);
      }
    }
  }
  cluster.sync();                        // no block leaves while another may read from it
}
struct GradSums { f2 g, gn; };
// One vector: n = (x - mean) rstd, g = dy w; adds to dw, db and to the row's sums of g and g n.
__device__ __forceinline__ void layer_terms(F16& g, F16& n, const F16& w, F16& dw, F16& db, f2 minus_mean, f2 rs, GradSums& s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    n.p[i] = mul2(add2(n.p[i], minus_mean), rs);
    dw.p[i] = fma2(g.p[i], n.p[i], dw.p[i]);
    db.p[i] = add2(db.p[i], g.p[i]);
    g.p[i] = mul2(g.p[i], w.p[i]);
    s.g = add2(s.g, g.p[i]);
    s.gn = fma2(g.p[i], n.p[i], s.gn);
  }
}
// dx = rstd (g - mean g - n mean gn) (+ dr)
template <typename T>
__device__ __forceinline__ void layer_out(Raw16<T>& o, const F16& g, const F16& n, f2 rs, float2 means, bool add, const Raw16<T>& dr) {
  F16 d;
  const f2 mg = f2_of(-means.x, -means.x), mgn = f2_of(-means.y, -means.y);
#pragma unroll
  for (int i = 0; i < 8; ++i) d.p[i] = mul2(rs, fma2(n.p[i], mgn, add2(g.p[i], mg)));
  if (add) {
    const F16 f = unpack(dr);
#pragma unroll
    for (int i = 0; i < 8; ++i) d.p[i] = add2(d.p[i], f.p[i]);
  }
  pack(o, d);
}
__device__ __forceinline__ void store_sums(float* out, int c, int cols, const F16& f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 d = f2_get(f.p[i]);
    if (c + 2 * i < cols) out[c + 2 * i] = d.x;
    if (c + 2 * i + 1 < cols) out[c + 2 * i + 1] = d.y;
  }
}
// A block's sums for layer_dw_kernel: whole vectors, 16 bytes at a time.
__host__ __device__ __forceinline__ int64_t partial_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }
__device__ __forceinline__ void store_partial(const LayerGradArgs& a, int64_t group, int c, const F16& dw, const F16& db) {
  if (c >= a.cols) return;
  const int64_t pitch = partial_pitch(a.cols);
  float4* out = reinterpret_cast<float4*>(a.partial + group * 2 * pitch + c);
  table_set(out, 1, dw);
  table_set(out + pitch / 4, 1, db);
}

template <typename T, bool VEC, int ROWS>
__global__ void __launch_bounds__(sizeof(T) == 4 ? 384 : 512, 1) layer_grad_kernel(LayerGradArgs a) {
  constexpr bool CLUSTER = ROWS == ROW_CLUSTER, PART = ROWS == ROW_PART;
  constexpr bool EARLY = sizeof(T) == 2 && VEC;        // dr with the row's other vectors (else there is no room for it)
  __shared__ __align__(16) typename std::conditional<CLUSTER, ClusterWords, RowWords>::type words;
  extern __shared__ __align__(16) uint8_t row_scratch[];
  zero_red(reinterpret_cast<float*>(&words), sizeof(words) / 4);
  if (CLUSTER) cg::this_cluster().sync();
  wait_for_previous();
  let_next_start();
  const int bx = blockDim.x, tx = threadIdx.x;
  float4* table = reinterpret_cast<float4*>(row_scratch) + tx;
  void* xs = VEC ? nullptr : row_scratch + bx * 64 + ((threadIdx.y * bx + tx) >> 5) * Scratch<T>::BYTES;
  const int parts = CLUSTER ? (int)cg::this_cluster().num_blocks() : 1;
  const int group = CLUSTER ? blockIdx.x / parts : blockIdx.x;         // of blocks that share rows
  const int step = (CLUSTER ? gridDim.x / parts : gridDim.x) * blockDim.y;
  int row = group * blockDim.y + threadIdx.y;
  const int below = PART ? (tx + threadIdx.y * bx) % 32 / bx : 0;      // rows below it in its warp
  int cols = !PART || row < a.rows ? a.cols : 0;
  auto dy = [&](int64_t k) { return reinterpret_cast<const T*>(a.dy) + k * a.lddy; };
  auto x = [&](int64_t k) { return reinterpret_cast<const T*>(a.x) + k * a.ldx; };
  auto dr = [&](int64_t k) { return reinterpret_cast<const T*>(a.dr) + k * a.lddr; };
  const float inv_cols = 1.0f / (float)a.cols;
  const int c = ((CLUSTER ? (int)cg::this_cluster().block_rank() * bx : 0) + tx) * 16;
  F16 dw = zero16(), db = zero16();
  Raw16<T> ny, nx, nr;
  float nmean = 0.f, nrstd = 0.f;
  bool lost = false;
  if (row - below < a.rows) {
    load16<VEC>(ny, dy(row), c, cols);
    load16<VEC>(nx, x(row), c, cols);
    if (a.dr) load16<VEC>(nr, dr(row), c, cols);
    if (cols) {
      nmean = a.mean[row];
      nrstd = a.rstd[row];
    }
  }
  if (threadIdx.y == 0) table_set(table, bx, load_w16_wide(a.w, a.w_bf16, c, a.cols));
  __syncthreads();
  for (unsigned call = 1; row - below < a.rows; row += step, ++call) {
    const f2 rs = f2_of(nrstd, nrstd);
    const bool more = row + step - below < a.rows;
    const int next = !PART || row + step < a.rows ? a.cols : 0;
    Raw16<T> res = nr;
    settle<VEC>(ny, xs);
    settle<VEC>(nx, xs);
    F16 g = unpack(ny), n = unpack(nx);
    GradSums s = {0, 0};
    layer_terms(g, n, table_get(table, bx), dw, db, f2_of(-nmean, -nmean), rs, s);
    if (more) {
      load16<VEC>(ny, dy(row + step), c, next);
      load16<VEC>(nx, x(row + step), c, next);
      if (EARLY && a.dr) load16<VEC>(nr, dr(row + step), c, next);
      if (next) {
        nmean = a.mean[row + step];
        nrstd = a.rstd[row + step];
      }
    }
    float2 t = make_float2(sum2(s.g), sum2(s.gn));
    if (PART) {
      part_sums(t.x, t.y);
    } else {
      t.x = warp_sum(t.x);
      t.y = warp_sum(t.y);
      if constexpr (CLUSTER) {
        float2 got[4];
        cluster_exchange(words, t.x, t.y, call, lost, got);
        t.x = warp_sum((got[0].x + got[1].x) + (got[2].x + got[3].x));
        t.y = warp_sum((got[0].y + got[1].y) + (got[2].y + got[3].y));
      } else if (bx > 32) {
        const float2* mine = row_exchange(words, t.x, t.y, call & 1);
        t = mine[0];
        for (int i = 1; i < bx >> 5; ++i) {
          t.x += mine[i].x;
          t.y += mine[i].y;
        }
      }
    }
    Raw16<T> o;
    if (a.dr) settle<VEC>(res, xs);
    layer_out(o, g, n, rs, make_float2(t.x * inv_cols, t.y * inv_cols), a.dr != nullptr, res);
    if (!EARLY && more && a.dr) load16<VEC>(nr, dr(row + step), c, next);    // used after the next row's join
    store16<VEC>(reinterpret_cast<T*>(a.dx) + row * a.lddx, c, cols, o, xs);
    cols = next;
  }
  if (CLUSTER) cluster_leave();
  float4* side = reinterpret_cast<float4*>(row_scratch);
  if (blockDim.y > 1) join_rows(side, dw, db);
  if (!CLUSTER && a.dw) {                // few rows
    const int n = (int)cg::this_cluster().num_blocks();
    const bool mine = threadIdx.y == 0 && (tx >> 2) % n == (int)cg::this_cluster().block_rank();   // 64 columns each
    if (n > 1) join_blocks(side, dw, db, mine);
    if (mine) {
      store_sums(a.dw, c, a.cols, dw);
      if (a.db) store_sums(a.db, c, a.cols, db);
    }
    return;
  }
  if (threadIdx.y > 0) return;
  store_partial(a, group, c, dw, db);
}

// Rows too long for registers: the block's dw and db sums live in its rows of `partial` (each thread adds to its own columns).
template <typename T, bool VEC>
__global__ void __launch_bounds__(512, 1) layer_grad_long_kernel(LayerGradArgs a) {
  __shared__ __align__(16) float red[2 * 32];
  zero_red(red, 2 * 32);
  wait_for_previous();
  let_next_start();
  void* xs = warp_scratch<T, VEC>();
  const int64_t pitch = partial_pitch(a.cols);
  const float* out = a.partial + (int64_t)blockIdx.x * 2 * pitch;
  const float inv_cols = 1.0f / (float)a.cols;
  const int64_t stride = 16 * blockDim.x, span = (a.cols + stride - 1) / stride * stride;   // whole warps
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.lddy;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* dr = reinterpret_cast<const T*>(a.dr) + row * a.lddr;
    T* dx = reinterpret_cast<T*>(a.dx) + row * a.lddx;
    const f2 rs = f2_of(a.rstd[row], a.rstd[row]), mm = f2_of(-a.mean[row], -a.mean[row]);
    GradSums s = {0, 0};
    auto kept = [&](const float* p, int c) {
      F16 f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f.p[i] = first || c >= a.cols ? 0 : f2_of(p[c + 2 * i], p[c + 2 * i + 1]);
      return f;
    };
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o;
      load16<VEC>(o, dy, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 g = unpack(o);
      load16<VEC>(o, x, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 n = unpack(o), dw = kept(out, (int)c), db = kept(out + pitch, (int)c);
      layer_terms(g, n, load_w16_wide(a.w, a.w_bf16, (int)c, a.cols), dw, db, mm, rs, s);
      store_partial(a, blockIdx.x, (int)c, dw, db);
    }
    first = false;
    const float mg = row_sum<false>(sum2(s.g), red, 0) * inv_cols, mgn = row_sum<false>(sum2(s.gn), red, 1) * inv_cols;
    for (int64_t c = threadIdx.x * 16; c < span; c += stride) {
      Raw16<T> o, res;
      load16<VEC>(o, dy, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 g = unpack(o);
      load16<VEC>(o, x, (int)c, a.cols);
      settle<VEC>(o, xs);
      F16 n = unpack(o);
      const F16 w = load_w16_wide(a.w, a.w_bf16, (int)c, a.cols);
      if (a.dr) {
        load16<VEC>(res, dr, (int)c, a.cols);
        settle<VEC>(res, xs);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n.p[i] = mul2(add2(n.p[i], mm), rs);
        g.p[i] = mul2(g.p[i], w.p[i]);
      }
      layer_out(o, g, n, rs, make_float2(mg, mgn), a.dr != nullptr, res);
      store16<VEC>(dx, (int)c, a.cols, o, xs);
    }
  }
}

// ------------------------------------------------------------- rows streamed through shared memory
// Where a group of threads has several rows, whole 16-byte vectors each, one of
// its threads copies them into a ring of rows in shared memory (bulk copies that
// an mbarrier counts), `stages` rows ahead, and the registers hold the present row
// alone.  A block's groups share the table of w and b; an SM has one block.
//
// A stage's row has been read by all of the group's threads when they have met for
// its sums, and is filled again by then.

// The group's part of the block's shared memory.
struct RowRing {
  uint8_t* rows;                       // [stage][input][bytes of a row]
  unsigned long long* full;            // [stage]
  float2* words;                       // [row in turn][warp]
  int stages, inputs, bytes;
  static __host__ __device__ size_t size(int stages, int inputs, int bytes) {
    return (size_t)stages * inputs * bytes + (stages + 1) / 2 * 16 + 2 * 32 * sizeof(float2);
  }
  __device__ __forceinline__ RowRing(uint8_t* base, int group, int stages_, int inputs_, int bytes_)
      : stages(stages_), inputs(inputs_), bytes(bytes_) {
    rows = base + group * size(stages, inputs, bytes);
    words = reinterpret_cast<float2*>(rows + (size_t)stages * inputs * bytes);
    full = reinterpret_cast<unsigned long long*>(words + 2 * 32);
  }
  __device__ __forceinline__ void start() const {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(full + i), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __device__ __forceinline__ void fill(int stage, const void* const (&from)[3]) const {
    const uint32_t bar = smem_u32(full + stage);
    mbar_expect_tx(bar, inputs * bytes);
    for (int i = 0; i < inputs; ++i)
      asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                   ::"r"(smem_u32(rows + ((size_t)stage * inputs + i) * bytes)), "l"(from[i]), "r"(bytes), "r"(bar) : "memory");
  }
  __device__ __forceinline__ const uint8_t* row(int stage, int input) const { return rows + ((size_t)stage * inputs + input) * bytes; }
};

// 16 columns from a row in shared memory; what lies past its end is zero.  Lanes begin with different 16-byte pieces, so
// that no bank is met twice, and put them in order.
__device__ __forceinline__ void ring_load(Raw16<__nv_bfloat16>& o, const uint8_t* row, int c, int cols) {
  const int turn = (threadIdx.x >> 2) & 1;
  uint4 v[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int at = c + 8 * (k ^ turn);
    v[k] = at < cols ? *reinterpret_cast<const uint4*>(row + at * 2) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o.w[i] = turn ? (&v[1].x)[i] : (&v[0].x)[i];
    o.w[4 + i] = turn ? (&v[0].x)[i] : (&v[1].x)[i];
  }
}
__device__ __forceinline__ void ring_load(Raw16<float>& o, const uint8_t* row, int c, int cols) {
  const int turn = (threadIdx.x >> 1) & 3;
  uint4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = c + 4 * (k ^ turn);
    v[k] = at < cols ? *reinterpret_cast<const uint4*>(row + at * 4) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)            // by the turn's low bit, then by its high bit
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[4 * k + i] = turn & 1 ? (&v[k ^ 1].x)[i] : (&v[k].x)[i];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = o.w[4 * k + i], hi = o.w[4 * (k + 2) + i];
      o.w[4 * k + i] = turn & 2 ? hi : lo;
      o.w[4 * (k + 2) + i] = turn & 2 ? lo : hi;
    }
}
// Two values of every warp of the group, after which all of its threads are done with the stage's row.
__device__ __forceinline__ const float2* ring_exchange(const RowRing& ring, float a, float b, int half) {
  float2* mine = ring.words + half * 32;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = make_float2(a, b);
  if (blockDim.x > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"((int)blockDim.x) : "memory");
  else __syncwarp();
  return mine;
}

constexpr int STREAM_THREADS[5] = {0, 768, 640, 0, 512};       // most of a norm's block, by vectors a thread: what the registers allow

// (sum, squared deviations) of a warp's columns, `mine` of them, NV vectors a lane.  Where the warp is full its lanes join
// in pairs, both values at once: of two halves of n columns, m = (m1 + m2) / 2 and S = S1 + S2 + n (m1 - m2)^2 / 2.
template <int NV>
__device__ __forceinline__ float2 warp_moments(const F16 (&v)[NV], const int (&c)[NV], int cols, int mine, float inv_mine) {
  f2 s = 0, d2 = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) s = total16(v[j], s);
  if (mine == 512 * NV) {
    float m = sum2(s) * (1.f / (16 * NV));
#pragma unroll
    for (int j = 0; j < NV; ++j) d2 = deviations(v[j], m, 16, d2);
    float dev = sum2(d2);
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, 1 << k), dev2 = __shfl_xor_sync(0xffffffffu, dev, 1 << k), d = m2 - m;
      dev = fmaf(d * (float)(8 * NV << k), d, dev + dev2);
      m = 0.5f * (m + m2);
    }
    return make_float2(m * (512 * NV), dev);
  }
  const float sum = warp_sum(sum2(s)), m = sum * inv_mine;
#pragma unroll
  for (int j = 0; j < NV; ++j) d2 = deviations(v[j], m, cols - c[j], d2);
  return make_float2(sum, warp_sum(sum2(d2)));
}

template <typename T, int NV>
__global__ void __launch_bounds__(STREAM_THREADS[NV], 1) layer_norm_stream_kernel(LayerNormArgs a, int stages) {
  __shared__ float2 columns[32];
  extern __shared__ __align__(16) uint8_t row_scratch[];
  const int bx = blockDim.x, tx = threadIdx.x, step = gridDim.x * blockDim.y;
  float4* table = reinterpret_cast<float4*>(row_scratch) + tx;
  const RowRing ring(row_scratch + bx * NV * 128, threadIdx.y, stages, a.r ? 2 : 1, a.cols * (int)sizeof(T));
  int row = blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t rblocks = q8_row_blocks(a.rows);
  const float inv_cols = 1.0f / (float)a.cols;
  if (tx == 0) ring.start();
  for (int i = tx; i < 64; i += bx) ring.words[i] = make_float2(0.f, 0.f);
  int c[NV], mine = 0;                                                 // mine: columns of this warp
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = (j * bx + tx) * 16;
    mine += warp_columns(a.cols, j * bx + (tx & ~31));
  }
  const float inv_mine = mine ? 1.f / (float)mine : 0.f;
  if (threadIdx.y == 0 && tx < 32) columns[tx] = make_float2(0.f, 0.f);
  __syncthreads();
  wait_for_previous();
  let_next_start();
  auto fill = [&](int stage, int64_t k) {
    const void* const from[3] = {reinterpret_cast<const T*>(a.x) + k * a.ldx, reinterpret_cast<const T*>(a.r) + k * a.ldr, nullptr};
    ring.fill(stage, from);
  };
  if (tx == 0)
    for (int i = 0; i < stages && (int64_t)row + (int64_t)i * step < a.rows; ++i) fill(i, (int64_t)row + (int64_t)i * step);
  if (threadIdx.y == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      table_set(table + j * 8 * bx, bx, load_w16_wide(a.w, a.w_bf16, c[j], a.cols));
      table_set(table + (j * 8 + 4) * bx, bx, a.b ? load_w16_wide(a.b, a.w_bf16, c[j], a.cols) : zero16());
    }
    if ((tx & 31) == 0) columns[tx >> 5] = make_float2((float)mine, inv_mine);
  }
  __syncthreads();
  int stage = 0, phase = 0, half = 0;
  for (; row < a.rows; row += step, half ^= 1) {
    const bool lost = !mbar_wait_own(smem_u32(ring.full + stage), phase, nullptr);
    F16 v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Raw16<T> h;
      ring_load(h, ring.row(stage, 0), c[j], a.cols);
      if (a.r) {
        Raw16<T> r;
        ring_load(r, ring.row(stage, 1), c[j], a.cols);
        add_stream(h, r);
        store16<true>(reinterpret_cast<T*>(a.h) + row * a.ldh, c[j], a.cols, h, nullptr);
      }
      v[j] = unpack(h);
    }
    const float2 w = warp_moments<NV>(v, c, a.cols, mine, inv_mine);
    float2 t = row_moments(ring_exchange(ring, w.x, w.y, half), columns, inv_cols);
    if (tx == 0 && (int64_t)row + (int64_t)stages * step < a.rows) fill(stage, (int64_t)row + (int64_t)stages * step);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
    if (lost) t = make_float2(__uint_as_float(0x7FFFFFFFu), 0.f);
    const float rstd = rstd_of(t.y, inv_cols, a.eps);
    if (tx == 0) {
      if (a.mean) a.mean[row] = t.x;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (!a.q && !a.y) continue;
    const f2 rs = f2_of(rstd, rstd), mm = f2_of(-t.x, -t.x);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const F16 w = table_get(table + j * 8 * bx, bx), b = table_get(table + (j * 8 + 4) * bx, bx);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j].p[i] = fma2(mul2(add2(v[j].p[i], mm), rs), w.p[i], b.p[i]);
      norm_write<T, true>(a, row, c[j], a.cols, v[j], q8_scale_at(row, c[j] >> 7, rblocks), nullptr);
    }
    if (a.q && (a.cols & 511)) norm_pad(a, row, rblocks);
  }
  if (a.q)
    for (; row < rblocks * 128; row += step) norm_pad(a, row, rblocks);
}

template <typename T>
__global__ void __launch_bounds__(512, 1) layer_grad_stream_kernel(LayerGradArgs a, int stages) {
  extern __shared__ __align__(16) uint8_t row_scratch[];
  const int bx = blockDim.x, tx = threadIdx.x, step = gridDim.x * blockDim.y;
  float4* table = reinterpret_cast<float4*>(row_scratch) + tx;
  const RowRing ring(row_scratch + bx * 64, threadIdx.y, stages, a.dr ? 3 : 2, a.cols * (int)sizeof(T));
  int row = blockIdx.x * blockDim.y + threadIdx.y;
  const float inv_cols = 1.0f / (float)a.cols;
  const int c = tx * 16;
  if (tx == 0) ring.start();
  for (int i = tx; i < 64; i += bx) ring.words[i] = make_float2(0.f, 0.f);
  __syncthreads();
  wait_for_previous();
  let_next_start();
  auto fill = [&](int stage, int64_t k) {
    const void* const from[3] = {reinterpret_cast<const T*>(a.dy) + k * a.lddy, reinterpret_cast<const T*>(a.x) + k * a.ldx,
                                 reinterpret_cast<const T*>(a.dr) + k * a.lddr};
    ring.fill(stage, from);
  };
  if (tx == 0)
    for (int i = 0; i < stages && (int64_t)row + (int64_t)i * step < a.rows; ++i) fill(i, (int64_t)row + (int64_t)i * step);
  float nmean = 0.f, nrstd = 0.f;
  if (row < a.rows) {
    nmean = a.mean[row];
    nrstd = a.rstd[row];
  }
  if (threadIdx.y == 0) table_set(table, bx, load_w16_wide(a.w, a.w_bf16, c, a.cols));
  __syncthreads();
  F16 dw = zero16(), db = zero16();
  int stage = 0, phase = 0, half = 0;
  for (; row < a.rows; row += step, half ^= 1) {
    const float mean = nmean;
    const f2 rs = f2_of(nrstd, nrstd);
    if (row + step < a.rows) {
      nmean = a.mean[row + step];
      nrstd = a.rstd[row + step];
    }
    const bool lost = !mbar_wait_own(smem_u32(ring.full + stage), phase, nullptr);
    Raw16<T> o, res;
    ring_load(o, ring.row(stage, 0), c, a.cols);
    F16 g = unpack(o);
    ring_load(o, ring.row(stage, 1), c, a.cols);
    F16 n = unpack(o);
    if (a.dr) ring_load(res, ring.row(stage, 2), c, a.cols);
    GradSums s = {0, 0};
    layer_terms(g, n, table_get(table, bx), dw, db, f2_of(-mean, -mean), rs, s);
    const float2* all = ring_exchange(ring, warp_sum(sum2(s.g)), warp_sum(sum2(s.gn)), half);
    if (tx == 0 && (int64_t)row + (int64_t)stages * step < a.rows) fill(stage, (int64_t)row + (int64_t)stages * step);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
    const float2 v = all[warp_lane()];
    float2 t = make_float2(sum_warps(v.x), sum_warps(v.y));
    if (lost) t.x = __uint_as_float(0x7FFFFFFFu);
    layer_out(o, g, n, rs, make_float2(t.x * inv_cols, t.y * inv_cols), a.dr != nullptr, res);
    store16<true>(reinterpret_cast<T*>(a.dx) + row * a.lddx, c, a.cols, o, nullptr);
  }
  if (blockDim.y > 1) {                  // every row that was copied has been read
    join_rows(reinterpret_cast<float4*>(row_scratch + bx * 64), dw, db);
    if (threadIdx.y > 0) return;
  }
  store_partial(a, blockIdx.x, c, dw, db);
}

// dw and db: the blocks' sums, added in their order (32 columns a block; blockDim.y threads a column take every
// blockDim.y-th sum, then their results are added in order).
template <int = 0>
__global__ void __launch_bounds__(1024) layer_dw_kernel(const float* partial, int parts, int64_t cols, float* dw, float* db) {
  __shared__ float s[32][33];
  wait_for_previous();
  let_next_start();
  const int64_t pitch = partial_pitch(cols), c = (int64_t)blockIdx.x * 32 + threadIdx.x;      // dw's columns, then db's
  float v = 0.f;
  if (c < 2 * pitch) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += blockDim.y) v += partial[(int64_t)p * 2 * pitch + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y > 0) return;
  for (int y = 1; y < blockDim.y; ++y) v += s[y][threadIdx.x];
  if (c < cols) dw[c] = v;
  else if (db && c >= pitch && c < pitch + cols) db[c - pitch] = v;
}

}  // namespace precond
