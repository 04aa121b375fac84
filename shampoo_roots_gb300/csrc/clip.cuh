// The norm of a list of tensors, and the tensors scaled by one factor.
//
//   norm = sqrt(sum_t sum_i g_ti^2),   g <- g min(1, max_norm / norm)
//
// Bound by memory: the norm reads every element once; the factor is known only
// then, so clipping reads them again and writes them.  The second pass goes
// through each block's tensors from the end, so that what the first one read last
// is still in L2 (129 MB).  Where the norm needs no clipping nothing more is read.
//
// The list comes as a kernel parameter (no upload, so that a captured call holds
// its own copy).  Tensors are cut into pieces of 16 KB; a block takes consecutive
// pieces, and writes one fp64 sum of its squares, in the workspace; every block of
// the second kernel adds these in the same order.
//
// A thread squares up to four sectors (128 B) in fp32 and adds their sum to its
// fp64 sum.  Where that fp32 sum lies outside 2^-70 .. 2^120, so that squares may
// have overflowed or been lost, the same registers are squared in fp64.
#pragma once

#include "form8.cuh"

namespace precond {

constexpr int CLIP_THREADS = 512, CLIP_PIECE = 512;   // a piece: sectors of 32 bytes
constexpr int CLIP_U = 4;                             // sectors a thread has under way

struct ClipTensor {
  void* p;
  int64_t n;                                          // elements; bf16: negative
};
template <int MAX>
struct ClipTable {
  ClipTensor tensor[MAX];
  uint32_t first[MAX + 1];                            // pieces before each tensor; first[count]: all
  int count;
};

// A tensor's elements as whole sectors, and up to 15 single ones before and after.
struct ClipView {
  char* body;
  int64_t sectors;
  int size, head, tail;                               // bytes an element; single elements
  __host__ __device__ __forceinline__ ClipView(const ClipTensor& t) {
    size = t.n < 0 ? 2 : 4;
    const int64_t n = t.n < 0 ? -t.n : t.n;
    const int64_t before = (int64_t)((32 - (reinterpret_cast<uintptr_t>(t.p) & 31)) & 31) / size;
    head = (int)(before < n ? before : n);
    body = reinterpret_cast<char*>(t.p) + head * size;
    sectors = (n - head) * size / 32;
    tail = (int)(n - head - sectors * (32 / size));
  }
  __host__ __device__ __forceinline__ int64_t pieces() const {
    return sectors ? (sectors + CLIP_PIECE - 1) / CLIP_PIECE : head + tail > 0;
  }
};

__device__ __forceinline__ void clip_load(uint32_t (&w)[8], const char* p) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p) : "memory");
}

// Calls f(tensor, its sectors s0 .. s1 - 1, whether they begin it) for each tensor that a block has pieces of; `back`:
// from the last one.  A tensor's single elements go with its first piece.
template <int MAX, typename F>
__device__ __forceinline__ void clip_walk(const ClipTable<MAX>& t, bool back, F f) {
  const int64_t all = t.first[t.count];
  const int64_t lo = all * blockIdx.x / gridDim.x, hi = all * (blockIdx.x + 1) / gridDim.x;
  if (lo >= hi) return;
  const int64_t at = back ? hi - 1 : lo;
  int a = 0, b = t.count - 1;                         // the last tensor that begins at or before this piece
  while (a < b) {
    const int m = (a + b + 1) / 2;
    if ((int64_t)t.first[m] <= at) a = m;
    else b = m - 1;
  }
  for (; a >= 0 && a < t.count; a += back ? -1 : 1) {
    const int64_t p0 = max(lo, (int64_t)t.first[a]), p1 = min(hi, (int64_t)t.first[a + 1]);
    if (back ? (int64_t)t.first[a + 1] <= lo : (int64_t)t.first[a] >= hi) break;
    if (p0 >= p1) continue;                           // an empty tensor
    const ClipView v(t.tensor[a]);
    const int64_t s0 = (p0 - t.first[a]) * CLIP_PIECE, s1 = min(v.sectors, (p1 - t.first[a]) * CLIP_PIECE);
    f(v, s0, s1, p0 == (int64_t)t.first[a]);
  }
}

// ------------------------------------------------------------- the norm
__device__ __forceinline__ f2 clip_square(const uint32_t (&w)[8], bool bf16, f2 s) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    if (bf16) {
#pragma unroll
      for (int k = i; k < i + 2; ++k) {
        const f2 x = f2_of(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
        s = fma2(x, x, s);
      }
    } else {
      const f2 x = f2_of(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
      s = fma2(x, x, s);
    }
  }
  return s;
}
__device__ __noinline__ double clip_square_wide(const uint32_t* w, int n, bool bf16) {
  double s = 0;
  for (int i = 0; i < n; ++i) {
    const double lo = __uint_as_float(bf16 ? w[i] << 16 : w[i]), hi = bf16 ? __uint_as_float(w[i] & 0xFFFF0000u) : 0.0;
    s += lo * lo + hi * hi;
  }
  return s;
}
// The block's sum in thread 0: lanes and warps in a fixed order.
__device__ __forceinline__ double clip_block_sum(double v) {
  __shared__ double red[CLIP_THREADS / 32];
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) v = warp_sum((int)threadIdx.x < (int)(blockDim.x >> 5) ? red[threadIdx.x] : 0.0);
  return v;
}

template <int MAX>
__global__ void __launch_bounds__(CLIP_THREADS, 2) clip_norm_kernel(const __grid_constant__ ClipTable<MAX> t, double* partial) {
  wait_for_previous();
  let_next_start();
  double sum = 0;
  clip_walk(t, false, [&](const ClipView& v, int64_t s0, int64_t s1, bool begins) {
    const bool bf16 = v.size == 2;
    for (int64_t s = s0 + threadIdx.x; s < s1; s += CLIP_U * CLIP_THREADS) {
      uint32_t w[CLIP_U][8];
#pragma unroll
      for (int u = 0; u < CLIP_U; ++u) {
        if (s + u * CLIP_THREADS < s1) {
          clip_load(w[u], v.body + (s + u * CLIP_THREADS) * 32);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[u][i] = 0;
        }
      }
      f2 e = 0;
#pragma unroll
      for (int u = 0; u < CLIP_U; ++u) e = clip_square(w[u], bf16, e);
      const float q = sum2(e);
      if (q >= 0x1p-70f && q <= 0x1p120f) {
        sum += (double)q;
      } else {                                        // nothing but zeros needs no second look
        uint32_t any = 0;
#pragma unroll
        for (int u = 0; u < CLIP_U; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) any |= w[u][i];
        if (any & (bf16 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) {
          for (int u = 0; u < CLIP_U; ++u)
            if (s + u * CLIP_THREADS < s1) sum += clip_square_wide(reinterpret_cast<const uint32_t*>(v.body + (s + u * CLIP_THREADS) * 32), 8, bf16);
        }
      }
    }
    if (begins && (int)threadIdx.x < v.head + v.tail) {
      const int64_t bytes = (int)threadIdx.x < v.head ? ((int)threadIdx.x - v.head) * v.size : v.sectors * 32 + ((int)threadIdx.x - v.head) * v.size;
      const uint32_t w = bf16 ? (uint32_t) * reinterpret_cast<const uint16_t*>(v.body + bytes) : *reinterpret_cast<const uint32_t*>(v.body + bytes);
      sum += clip_square_wide(&w, 1, bf16);
    }
  });
  sum = clip_block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm of all sums, in every thread.
__device__ __forceinline__ float clip_total(const double* partial, int n) {
  __shared__ float norm;
  double v = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) v += partial[i];
  v = clip_block_sum(v);
  if (threadIdx.x == 0) norm = (float)sqrt(v);
  __syncthreads();
  return norm;
}
template <int = 0>
__global__ void __launch_bounds__(CLIP_THREADS) clip_total_kernel(const double* partial, int n, float* norm) {
  wait_for_previous();
  let_next_start();
  const float v = clip_total(partial, n);
  if (threadIdx.x == 0) *norm = v;
}

// ------------------------------------------------------------- scaling
__device__ __forceinline__ void clip_scale(uint32_t (&w)[8], bool bf16, float c) {
  const f2 cc = f2_of(c, c);
  if (bf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = f2_get(mul2(f2_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), cc));
      w[i] = bf16x2_bits(x.x, x.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 x = f2_get(mul2(f2_of(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), cc));
      w[i] = __float_as_uint(x.x);
      w[i + 1] = __float_as_uint(x.y);
    }
  }
}

// sums: how many of `partial` make the norm, which block 0 then leaves in `norm`; 0: it is there already.
template <int MAX>
__global__ void __launch_bounds__(CLIP_THREADS, 2) clip_scale_kernel(const __grid_constant__ ClipTable<MAX> t, const double* partial, int sums,
                                                                     float max_norm, float* norm) {
  wait_for_previous();
  let_next_start();
  const float total = sums ? clip_total(partial, sums) : *norm;
  if (sums && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  if (!(total > max_norm) || !(total < INFINITY)) return;       // also where the norm is not a number
  const float c = max_norm / total;
  clip_walk(t, true, [&](const ClipView& v, int64_t s0, int64_t s1, bool begins) {
    const bool bf16 = v.size == 2;
    if (begins && (int)threadIdx.x < v.head + v.tail) {
      const int64_t bytes = (int)threadIdx.x < v.head ? ((int)threadIdx.x - v.head) * v.size : v.sectors * 32 + ((int)threadIdx.x - v.head) * v.size;
      if (bf16) {
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(v.body + bytes);
        *p = __float2bfloat16_rn(__bfloat162float(*p) * c);
      } else {
        *reinterpret_cast<float*>(v.body + bytes) *= c;
      }
    }
    const int64_t steps = (s1 - s0 + CLIP_U * CLIP_THREADS - 1) / (CLIP_U * CLIP_THREADS);
    for (int64_t k = steps - 1; k >= 0; --k) {
      const int64_t s = s0 + k * (CLIP_U * CLIP_THREADS) + threadIdx.x;
      uint32_t w[CLIP_U][8];
#pragma unroll
      for (int u = 0; u < CLIP_U; ++u)
        if (s + u * CLIP_THREADS < s1) clip_load(w[u], v.body + (s + u * CLIP_THREADS) * 32);
#pragma unroll
      for (int u = 0; u < CLIP_U; ++u)
        if (s + u * CLIP_THREADS < s1) {
          clip_scale(w[u], bf16, c);
          st_sector(v.body + (s + u * CLIP_THREADS) * 32, w[u]);
        }
    }
  });
}

}  // namespace precond
