// The norm of a list of tensors, and the tensors scaled by one factor.
//
//   norm = sqrt(sum_t sum_i g_ti^2),   g <- g min(1, max_norm / norm)
//
// Bound by memory: the norm reads every element once; the factor is known only
// then, so clipping reads them again and writes them.  The second pass goes
// through each block's tensors from the end, so that what the first one read last
// is still in L2 (129 MB); what it read before that is asked to leave L2 first.
// Where the norm needs no clipping nothing more is read.
//
// Measured: norm of 604 MB 88 us (the copy bandwidth); clipping of 604 MB of bf16
// 261 to 283 us, where three passes over it take 267 and two 179: of the 60 MB that are
// asked to stay in L2 some 20 are found there.  97 weights of 333 KB with three
// vectors each, clipped, 15 us.
//
// A short list takes one launch: a cluster of 8 blocks, which read it a second time
// when they have joined their sums through distributed shared memory (one layer of
// 256 x 128, clipped: 4.0 us, with two kernels 6.7).
//
// The list comes as a kernel parameter (no upload, so that a captured call holds
// its own copy).  Tensors are cut into pieces of 4 KB, four sectors a lane; a
// block's pieces are consecutive and its warps take them in turn, so that many
// small tensors are under way at once and a block reads 64 KB in a row (pieces of
// 16 KB, a block each: the 97 weights took 25 us; consecutive pieces to each warp:
// norm of 604 MB 92 us).
// A block writes the sum of its squares, in the workspace; every block of the
// second kernel adds these in the same order.
//
// A lane squares up to four sectors (128 B) in fp32; above that sums are pairs of
// fp32 numbers, joined by TwoSum (Knuth), so that no length of list costs digits.
// (fp64 additions, two a clock and SM, took a block's join a microsecond.)  Where
// the squares of a lane's sectors add up to less than 2^-70 or more than 2^80, so
// that some may have been lost or the pair's range may not do, the same registers
// are squared again times a power of two, into a pair of their own (Blue's method).
#pragma once

#include <cooperative_groups.h>

#include "form8.cuh"

namespace precond {

constexpr int CLIP_THREADS = 512, CLIP_WARPS = CLIP_THREADS / 32;
constexpr int CLIP_U = 4;                             // sectors a lane has under way
constexpr int CLIP_PIECE = 32 * CLIP_U;               // a piece: sectors of 32 bytes
constexpr int CLIP_KEPT = (60 << 20) / 32 / CLIP_PIECE; // pieces that L2 is asked to keep between the passes

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
  // a lane's single element (there are up to 30), or null
  __device__ __forceinline__ char* single(int lane) const {
    return lane >= head + tail ? nullptr : body + (lane < head ? (int64_t)(lane - head) * size : sectors * 32 + (lane - head) * size);
  }
  __host__ __device__ __forceinline__ int64_t pieces() const {
    return sectors ? (sectors + CLIP_PIECE - 1) / CLIP_PIECE : head + tail > 0;
  }
};

// A sector that stays in L2, or that leaves it before others do.
__device__ __forceinline__ void clip_load(uint32_t (&w)[8], const char* p, bool stays) {
  if (stays)
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p) : "memory");
  else
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p) : "memory");
}
__device__ __forceinline__ void clip_store(char* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// A warp's pieces of a list: a block's are consecutive, its warps take every 16th of them.  The place in the table is
// found before the kernel waits for its predecessor.
struct ClipWalk {
  int64_t lo, hi, keep, at;                           // the block's pieces; those that L2 may keep; the warp's first
  int tensor;
  template <int MAX>
  __device__ __forceinline__ ClipWalk(const ClipTable<MAX>& t, bool back) {
    const int64_t all = t.first[t.count];
    lo = all * blockIdx.x / gridDim.x;
    hi = all * (blockIdx.x + 1) / gridDim.x;
    keep = hi - (hi - lo) * min(all, (int64_t)CLIP_KEPT) / all;          // the last of every block's
    at = back ? hi - 1 - (threadIdx.x >> 5) : lo + (threadIdx.x >> 5);
    // the last tensor that begins at or before this piece
    int a = 0, b = t.count - 1;
    while (a < b) {
      const int m = (a + b + 1) / 2;
      if ((int64_t)t.first[m] <= at) a = m;
      else b = m - 1;
    }
    tensor = a;
  }
  // Calls f(tensor, first sector of the piece, whether the piece begins it, whether it stays in L2); `back`: from the last
  // one.  A tensor's single elements go with its first piece.
  template <int MAX, typename F>
  __device__ __forceinline__ void each(const ClipTable<MAX>& t, bool back, F f) const {
    int64_t i = at;
    int a = tensor;
    if (i < lo || i >= hi) return;
    while (true) {
      const ClipView v(t.tensor[a]);
      const int64_t p0 = t.first[a], p1 = t.first[a + 1];
      for (; i >= max(lo, p0) && i < min(hi, p1); i += back ? -CLIP_WARPS : CLIP_WARPS)
        f(v, (i - p0) * CLIP_PIECE + (threadIdx.x & 31), i == p0, i >= keep);
      if (i < lo || i >= hi) return;
      if (back)
        while ((int64_t)t.first[a] > i) --a;
      else
        while ((int64_t)t.first[a + 1] <= i) ++a;
    }
  }
};

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
__device__ __forceinline__ f2 clip_square_scaled(const uint32_t (&w)[8], bool bf16, float by, f2 s) {
  const f2 k = f2_of(by, by);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    if (bf16) {
#pragma unroll
      for (int j = i; j < i + 2; ++j) {
        const f2 x = mul2(f2_of(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), k);
        s = fma2(x, x, s);
      }
    } else {
      const f2 x = mul2(f2_of(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), k);
      s = fma2(x, x, s);
    }
  }
  return s;
}
// A sum hi + lo.  An infinite hi, or one that is not a number, stays, whatever lo says.
struct ClipPair {
  float hi, lo;
  __device__ __forceinline__ void add(float h, float l) {
    const float s = hi + h, b = s - hi;
    lo += ((hi - (s - b)) + (h - b)) + l;
    hi = s;
  }
  __device__ __forceinline__ void join(int o) {
    const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
    add(h, l);
  }
  __device__ __forceinline__ float value() const { return hi < INFINITY ? hi + lo : hi; }
};
// A sum of squares: of ordinary size; of elements times 2^80; of elements times 2^-80.
constexpr float CLIP_LEAST = 0x1p-70f, CLIP_MOST = 0x1p80f, CLIP_UP = 0x1p80f, CLIP_DOWN = 0x1p-80f;
struct ClipSum {
  ClipPair mid, low, high;
  __device__ __forceinline__ void add(const ClipSum& o) {
    mid.add(o.mid.hi, o.mid.lo);
    if (o.low.hi != 0.f) low.add(o.low.hi, o.low.lo);
    if (o.high.hi != 0.f) high.add(o.high.hi, o.high.lo);
  }
  // over the lanes, the same in each
  __device__ __forceinline__ void join() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mid.join(o);
    if (__any_sync(0xffffffffu, low.hi != 0.f || high.hi != 0.f)) {
      for (int o = 16; o > 0; o >>= 1) {
        low.join(o);
        high.join(o);
      }
    }
  }
  // the square root of the whole
  __device__ __forceinline__ float root() const {
    const float m = mid.value(), l = low.value(), h = high.value();
    if (h != 0.f) return sqrtf(fmaf(m * CLIP_DOWN, CLIP_DOWN, h)) * CLIP_UP;           // also where h is not finite
    return m != 0.f ? sqrtf(fmaf(l * CLIP_DOWN, CLIP_DOWN, m)) : sqrtf(l) * CLIP_DOWN;
  }
};
constexpr ClipSum CLIP_NOTHING = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
// The block's sum in the first warp: lanes and warps in a fixed order.
__device__ __forceinline__ ClipSum clip_block_sum(ClipSum v) {
  __shared__ ClipSum red[CLIP_WARPS];
  v.join();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < CLIP_WARPS ? red[threadIdx.x] : CLIP_NOTHING;
    v.join();
  }
  return v;
}

// The sum of the squares of a block's pieces, in thread 0.
template <int MAX>
__device__ __forceinline__ ClipSum clip_squares(const ClipTable<MAX>& t, const ClipWalk& walk) {
  ClipSum sum = CLIP_NOTHING;
  walk.each(t, false, [&](const ClipView& v, int64_t s, bool begins, bool stays) {
    const bool bf16 = v.size == 2;
    uint32_t w[CLIP_U][8];
    const char* single = begins ? v.single(threadIdx.x & 31) : nullptr;
    float x = 0.f;
    if (single) x = bf16 ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(single)) : *reinterpret_cast<const float*>(single);
#pragma unroll
    for (int u = 0; u < CLIP_U; ++u) {
      if (s + u * 32 < v.sectors) {
        clip_load(w[u], v.body + (s + u * 32) * 32, stays);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[u][i] = 0;
      }
    }
    f2 e = f2_of(x * x, 0.f);
#pragma unroll
    for (int u = 0; u < CLIP_U; ++u) e = clip_square(w[u], bf16, e);
    const float q = sum2(e);
    if (q >= CLIP_LEAST && q <= CLIP_MOST) {
      sum.mid.add(q, 0.f);
    } else {
      const float by = q < CLIP_LEAST ? CLIP_UP : CLIP_DOWN, y = x * by;
      e = f2_of(y * y, 0.f);
#pragma unroll
      for (int u = 0; u < CLIP_U; ++u) e = clip_square_scaled(w[u], bf16, by, e);
      if (q < CLIP_LEAST) sum.low.add(sum2(e), 0.f);
      else sum.high.add(sum2(e), 0.f);
    }
  });
  return clip_block_sum(sum);
}
template <int MAX>
__global__ void __launch_bounds__(CLIP_THREADS, 2) clip_norm_kernel(const __grid_constant__ ClipTable<MAX> t, ClipSum* partial) {
  const ClipWalk walk(t, false);
  wait_for_previous();
  let_next_start();
  const ClipSum sum = clip_squares(t, walk);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm of all sums, in every thread.
__device__ __forceinline__ float clip_total(const ClipSum* partial, int n) {
  __shared__ float norm;
  ClipSum v = CLIP_NOTHING;
  for (int i = threadIdx.x; i < n; i += blockDim.x) v.add(partial[i]);
  v = clip_block_sum(v);
  if (threadIdx.x == 0) norm = v.root();
  __syncthreads();
  return norm;
}
template <int = 0>
__global__ void __launch_bounds__(CLIP_THREADS) clip_total_kernel(const ClipSum* partial, int n, float* norm) {
  wait_for_previous();
  let_next_start();
  const float v = clip_total(partial, n);
  if (threadIdx.x == 0) *norm = v;
}

// ------------------------------------------------------------- scaling
// max_norm / norm; below fp32's normal numbers in two steps, so that large elements keep their digits: 2^-126, which is exact
// for what does not end below the normal numbers, and 2^126 max_norm / norm (no overflow: max_norm < 4 then).
struct ClipFactor {
  float first, c;
  __device__ __forceinline__ ClipFactor(float max_norm, float norm) : first(1.f), c(max_norm / norm) {
    if (c < 0x1p-126f) {
      first = 0x1p-126f;
      c = max_norm * 0x1p126f / norm;
    }
  }
  __device__ __forceinline__ float operator()(float x) const { return x * first * c; }
  __device__ __forceinline__ f2 operator()(f2 x) const {
    if (first != 1.f) x = mul2(x, f2_of(first, first));
    return mul2(x, f2_of(c, c));
  }
};
__device__ __forceinline__ void clip_scale(uint32_t (&w)[8], bool bf16, const ClipFactor& factor) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = f2_get(factor(f2_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))));
      w[i] = bf16x2_bits(x.x, x.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 x = f2_get(factor(f2_of(__uint_as_float(w[i]), __uint_as_float(w[i + 1]))));
      w[i] = __float_as_uint(x.x);
      w[i + 1] = __float_as_uint(x.y);
    }
  }
}

template <int MAX>
__device__ __forceinline__ void clip_scale_all(const ClipTable<MAX>& t, const ClipWalk& walk, bool back, const ClipFactor& factor) {
  walk.each(t, back, [&](const ClipView& v, int64_t s, bool begins, bool stays) {
    const bool bf16 = v.size == 2;
    uint32_t w[CLIP_U][8];
#pragma unroll
    for (int u = 0; u < CLIP_U; ++u)
      if (s + u * 32 < v.sectors) clip_load(w[u], v.body + (s + u * 32) * 32, stays);
    if (char* single = begins ? v.single(threadIdx.x & 31) : nullptr) {
      if (bf16) {
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(single);
        *p = __float2bfloat16_rn(factor(__bfloat162float(*p)));
      } else {
        float* p = reinterpret_cast<float*>(single);
        *p = factor(*p);
      }
    }
#pragma unroll
    for (int u = 0; u < CLIP_U; ++u)
      if (s + u * 32 < v.sectors) {
        clip_scale(w[u], bf16, factor);
        clip_store(v.body + (s + u * 32) * 32, w[u]);
      }
  });
}
// Whether a norm is clipped: not where it is infinite or not a number.
__device__ __forceinline__ bool clips(float norm, float max_norm) { return norm > max_norm && norm < INFINITY; }

// sums: how many of `partial` make the norm, which block 0 then leaves in `norm`; 0: it is there already.
template <int MAX>
__global__ void __launch_bounds__(CLIP_THREADS, 2) clip_scale_kernel(const __grid_constant__ ClipTable<MAX> t, const ClipSum* partial, int sums,
                                                                     float max_norm, float* norm) {
  const ClipWalk walk(t, true);
  wait_for_previous();
  let_next_start();
  const float total = sums ? clip_total(partial, sums) : *norm;
  if (sums && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  if (clips(total, max_norm)) clip_scale_all(t, walk, true, ClipFactor(max_norm, total));
}

// A short list: one cluster.  max_norm infinite: the norm alone.
constexpr int CLIP_CLUSTER = 8;
template <int MAX>
__global__ void __launch_bounds__(CLIP_THREADS, 2) clip_short_kernel(const __grid_constant__ ClipTable<MAX> t, float max_norm, float* norm) {
  namespace cg = cooperative_groups;
  __shared__ ClipSum sums[CLIP_CLUSTER];
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");      // the blocks have begun
  const ClipWalk walk(t, false);
  wait_for_previous();
  let_next_start();
  const ClipSum sum = clip_squares(t, walk);
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x == 0)
    for (int i = 0; i < CLIP_CLUSTER; ++i) *cluster.map_shared_rank(&sums[blockIdx.x], i) = sum;
  cluster.sync();
  ClipSum v = sums[0];
#pragma unroll
  for (int i = 1; i < CLIP_CLUSTER; ++i) v.add(sums[i]);
  const float total = v.root();
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  if (clips(total, max_norm)) clip_scale_all(t, walk, false, ClipFactor(max_norm, total));
}

}  // namespace precond
