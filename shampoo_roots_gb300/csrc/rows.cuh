// Rows on threads, shared by the norms: 16 consecutive columns a thread, a row on
// a block, on the blocks of a cluster or on part of a warp; sums over its threads.
#pragma once

#include <cooperative_groups.h>

#include "form8.cuh"

namespace precond {

namespace cg = cooperative_groups;

// How a row lies on threads: whole warps of a block, those of a cluster's blocks, part of a warp.
enum { ROW_BLOCK, ROW_CLUSTER, ROW_PART };

__device__ __forceinline__ float load_w(const void* w, int bf16, int c) {
  return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c]) : reinterpret_cast<const float*>(w)[c];
}
__device__ __forceinline__ F16 load_w16(const void* w, int bf16, int c, int cols) {
  F16 f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f.p[i] = f2_of(c + 2 * i < cols ? load_w(w, bf16, c + 2 * i) : 0.f, c + 2 * i + 1 < cols ? load_w(w, bf16, c + 2 * i + 1) : 0.f);
  return f;
}
// The same where whole vectors are aligned: 4 or 2 loads in place of 16.
__device__ __forceinline__ F16 load_w16_wide(const void* w, int bf16, int c, int cols) {
  if (c + 16 > cols || (reinterpret_cast<uintptr_t>(w) & 15)) return load_w16(w, bf16, c, cols);
  F16 f;
  if (bf16) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(w) + c);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 v = p[k];
#pragma unroll
      for (int i = 0; i < 4; ++i) f.p[4 * k + i] = f2_of(__uint_as_float((&v.x)[i] << 16), __uint_as_float((&v.x)[i] & 0xFFFF0000u));
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(w) + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = p[k];
      f.p[2 * k] = f2_of(v.x, v.y);
      f.p[2 * k + 1] = f2_of(v.z, v.w);
    }
  }
  return f;
}
__device__ __forceinline__ f2 squares(const F16& v, f2 s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fma2(v.p[i], v.p[i], s);
  return s;
}

// Sum over the blockDim.x threads of one row (a multiple of 32; PART: 8 or 16),
// the same value in each.  `red` has room for 2 x blockDim.y x 32, zeroed; calls
// alternate between its halves, so that one barrier a call is enough.
template <bool PART>
__device__ __forceinline__ float row_sum(float v, float* red, int half) {
  const int nw = blockDim.x >> 5;
  if (PART) {
#pragma unroll 1
    for (int o = blockDim.x >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  v = warp_sum(v);
  if (nw == 1) return v;
  float* mine = red + (half * blockDim.y + threadIdx.y) * 32;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"((int)blockDim.x) : "memory");
  float4 s = *reinterpret_cast<const float4*>(mine);
  for (int i = 4; i < nw; i += 4) {
    const float4 t = *reinterpret_cast<const float4*>(mine + i);
    s = make_float4(s.x + t.x, s.y + t.y, s.z + t.z, s.w + t.w);
  }
  return (s.x + s.y) + (s.z + s.w);
}
// The same over the blocks of a cluster (blockDim.y is 1, at most 16 warps a
// block).  Every warp leaves its sum with each block, as a word that also holds
// the number of the call, and every warp polls its own block's words: the join
// waits for these sums alone.  (A cluster barrier, or any release, also waits
// for the previous row's dx to reach L2: 110 us where this took 88, for the
// gradient of 3000 x 16384 bf16.)  Calls alternate between the halves of
// `slots` (2 x 8 x 16, zeroed in every block): a warp writes for call n + 2 when
// it has seen call n + 1 from every warp, so that all of them have read call n.
// The blocks of a cluster are resident together; a wait that runs out all the
// same gives NaN, for this row and the block's later ones.
__device__ __forceinline__ float cluster_row_sum(float v, unsigned long long* slots, unsigned call, bool& lost) {
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), lane = threadIdx.x & 31;
  v = warp_sum(v);
  unsigned long long* mine = slots + (call & 1) * 128;
  if (lane < parts) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(mine + cluster.block_rank() * 16 + (threadIdx.x >> 5))), "r"(lane));
    asm volatile("st.relaxed.cluster.shared::cluster.u64 [%0], %1;"
                 ::"r"(to), "l"((unsigned long long)call << 32 | __float_as_uint(v)) : "memory");
  }
  const int nw = blockDim.x >> 5;
  float s = 0.f;
  // All lanes poll together, up to 4 words each: lanes that left the loop one by one took 3 us more a row.
  for (int spin = 0; !lost; ++spin) {
    bool here = true;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane + 32 * k;
      if (32 * k < 16 * parts && i < 16 * parts && (i & 15) < nw) {
        unsigned long long got;
        asm volatile("ld.relaxed.cluster.shared::cta.u64 %0, [%1];"
                     : "=l"(got) : "r"((uint32_t)__cvta_generic_to_shared(mine + i)) : "memory");
        here = here && (unsigned)(got >> 32) == call;
        s += __uint_as_float((unsigned)got);
      }
    }
    if (__all_sync(0xffffffffu, here)) break;
    lost = spin > 10000000;                              // seconds: every lane counts the same
  }
  if (lost) s = __uint_as_float(0x7FFFFFFFu);
  return warp_sum(s);
}
// No block leaves while another may still write to it: every one has the last row's words by then, unless a wait ran out.
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void zero_red(float* red, int n) {
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < n; i += blockDim.x * blockDim.y) red[i] = 0.f;
  __syncthreads();
}

// h = x + r, rounded to the stream's type.  The bf16 addition rounds the exact
// sum once; the fp32 sum rounded to bf16 is the same (where fp32 drops bits of
// the sum, the smaller term lies below 2^-16 of the larger and cannot reach a tie).
__device__ __forceinline__ void add_stream(Raw16<__nv_bfloat16>& x, const Raw16<__nv_bfloat16>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(x.w[i]) : "r"(r.w[i]));
}
__device__ __forceinline__ void add_stream(Raw16<float>& x, const Raw16<float>& r) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x.w[i] = __float_as_uint(__uint_as_float(x.w[i]) + __uint_as_float(r.w[i]));
}

// A warp's exchange buffer where rows are not aligned (form8.cuh), in dynamic shared memory.
template <typename T, bool VEC>
__device__ __forceinline__ void* warp_scratch() {
  extern __shared__ __align__(16) uint8_t row_scratch[];
  return VEC ? nullptr : row_scratch + ((threadIdx.y * blockDim.x + threadIdx.x) >> 5) * Scratch<T>::BYTES;
}

// 1 / sqrt(mean + eps): the hardware's estimate and one Newton step, y (3 - x y^2) / 2.  (Every thread of a row
// computes it; a division and a correctly rounded root cost 40 instructions of the 390 a vector took.)
__device__ __forceinline__ float rstd_of(float sum, float inv_cols, float eps) {
  const float x = fmaf(sum, inv_cols, eps);
  const float y = rsqrtf(x);
  const float z = y * fmaf(-0.5f * x * y, y, 1.5f);
  return x < 1e30f ? z : y;            // x y y may overflow only where x does
}

// One vector's outputs; `at` is its scale byte's place.
template <typename T, bool VEC, typename A>
__device__ __forceinline__ void norm_write(const A& a, int64_t row, int c, int cols, F16& y, size_t at, void* xs) {
  if (a.y) {
    Raw16<T> o;
    pack(o, y);
    store16<VEC>(reinterpret_cast<T*>(a.y) + row * a.ldy, c, cols, o, xs);
  }
  if (a.q) {
    const unsigned b = q8_block_exponent(y);
    store_q16(a.q + row * a.ldq, c, cols, q8_pack16(y, q8_inverse(b)));
    if ((threadIdx.x & 7) == 0 && c < cols) a.scale[at] = (uint8_t)b;
  }
}
// The scale bytes past the matrix's end: a row's trailing blocks, or a whole row of padding.
template <typename A>
__device__ __forceinline__ void norm_pad(const A& a, int64_t row, int64_t rblocks) {
  const int nkb = row < a.rows ? (a.cols + 127) >> 7 : 0;
  for (int kb = nkb + threadIdx.x; kb < 4 * q8_groups(a.cols); kb += blockDim.x)
    a.scale[q8_scale_at(row, kb, rblocks)] = (uint8_t)Q8_ONE;
}

}  // namespace precond
