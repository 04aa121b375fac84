// C = A B^T of two matrices in 8-bit form (form8.cuh), M x K and N x K:
//
//   C_ij = sum_kb 2^(ea[i,kb] + eb[j,kb]) sum_{k in block kb} qa_ik qb_jk   (+ C_ij)
//
// on tcgen05.mma kind::mxf8f6f4 with block scales.  The instruction takes one
// e8m0 scale for every row and 32 columns; a block of 128 uses the same scale
// byte for its four instructions (the descriptor's scale id picks one of the
// four bytes, so one 32-bit tensor-memory column holds a row's scales of 512
// columns).  Scaling happens inside the tensor core, so the sums need not leave
// tensor memory at every block.
//
// The tensor core's fp32 sums truncate, which biases a long chain: for fp32
// results (PROMOTE) the sum of every G8_SEGMENT blocks is added to fp32
// registers (round to nearest) while the next segment runs in the other
// tensor-memory buffer.  A bf16 result's own rounding is far above the bias, so
// its sums stay in tensor memory over the whole of K.
//
// Pipeline: TMA (128-byte swizzle, one block of 128 columns a stage) into a
// ring of shared memory; the stage of a group's first block also carries the
// group's scales, 512 bytes for 128 rows, which the MMA thread copies to tensor
// memory (tcgen05.cp) in front of its MMAs.  Warp 0 loads, warp 1 issues, warps
// 2..9 drain (two a tensor-memory lane quadrant, half of the columns each).
//
// Every mbarrier wait is bounded; on a time-out the kernel sets the error word,
// every role leaves, and the kernel returns.
//
// Bound by the tensor cores where there are many tokens, by the weight's bytes
// where there are few.  Measured: 16384 x 6144 x 6144 to bf16 395 us, 3140
// TFLOP/s at the power limit (a single call 3500); 4096 x 1024 x 8191
// accumulated in fp32 32.0 us, 2150 TFLOP/s; 1 x 6144 x 6144 10.0 us, of which
// the bytes take 5.6; 16 x 4096 x 4096 6.2 us.
#pragma once

#include <cooperative_groups.h>
#include <cuda.h>

#include <type_traits>

#include "form8.cuh"
#include "ptx.cuh"

namespace precond {

constexpr int G8_BM = 128;             // rows of A a CTA takes (the MMA's M)
constexpr int G8_BK = 128;             // one scale block, one swizzled row
constexpr int G8_SEGMENT = 4;          // blocks between promotions (512 columns: one scale group)
constexpr int G8_PAIR_SEGMENT = 8;     // the same, for pairs of CTAs
constexpr int G8_EPI_WARPS = 8;
constexpr int G8_XS = 32 * 32;         // a drain warp's scratch: 32 x 32 results
constexpr int G8_THREADS = 64 + 32 * G8_EPI_WARPS;
constexpr int G8_PAIR_THREADS = 128 + 32 * G8_EPI_WARPS;   // a warpgroup that loads and issues, two that drain

struct Gemm8Args {
  int64_t M, N, K;                     // of the MMA's view: M rows of its A operand
  const uint8_t* sa; int64_t sa_rb;    // scales and their blocks of 128 rows
  const uint8_t* sb; int64_t sb_rb;
  void* c; int64_t ldc;
  int c_bf16, accumulate;
  int sectors, quads;                  // C's rows begin at multiples of 32 bytes, of 4 elements
  int swap;                            // 1: C is N x M (the operands were exchanged)
  unsigned int* err;
};

template <int BN>
struct Gemm8Smem {
  static constexpr int A_BYTES = G8_BM * G8_BK;
  static constexpr int B_BYTES = BN * G8_BK;
  static constexpr int SF_BYTES = 1024;                 // 128 rows of A and of B
  static constexpr int CTAS = BN <= 32 ? 2 : 1;         // on an SM: few tokens need all SMs' loads, not wide tiles
  static constexpr int STAGES = BN == 128 ? 5 : BN == 64 ? 7 : BN == 32 ? 4 : 5;
  static constexpr int DRAIN_WARPS = BN >= 64 ? G8_EPI_WARPS : 4;      // that have columns of their own
  static constexpr int OFF_SF = STAGES * (A_BYTES + B_BYTES);
  static constexpr int OFF_XS = OFF_SF + STAGES * SF_BYTES;                 // a scratch of each drain warp
  static constexpr int OFF_BAR = OFF_XS + DRAIN_WARPS * G8_XS * 4;
  // a stretch's sums, over the ring, along C's rows: [128][BN], transposed [BN][128], 4 floats apart modulo 32
  static constexpr int PART_LD = BN + 4, PART_LDT = G8_BM + 4;
  static_assert(G8_BM * PART_LD * 4 <= OFF_SF && BN * PART_LDT * 4 <= OFF_SF, "the sums fit into the ring");
  static constexpr int BYTES = 1024 + OFF_BAR + 256;
  static_assert(CTAS * (BYTES + 1024) <= 228 * 1024, "shared memory of an SM");
  // tensor memory: two sum buffers, then two scale buffers
  static constexpr int ACC_COLS = BN < 32 ? 32 : BN;
  static constexpr int SF_COL = 2 * ACC_COLS;
  static constexpr int SF_COLS = 8;
  static constexpr int TMEM_COLS = 2 * ACC_COLS + 2 * SF_COLS <= 128 ? 128 : 2 * ACC_COLS + 2 * SF_COLS <= 256 ? 256 : 512;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// K-major operand, 128-byte swizzle: 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Scales: 32 rows of 16 bytes, no swizzle (8-row groups 128 B apart).
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// 512 bytes of scales into 4 tensor-memory columns, repeated for the four lane quadrants.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// Instruction descriptor of kind::mxf8f6f4: e4m3 A and B (K-major), e8m0 scales; `id` picks the scale byte.
template <int BN>
__device__ __forceinline__ uint32_t mx_idesc(uint32_t id) {
  return id << 4 | (uint32_t)(BN >> 3) << 17 | 1u << 23 | (uint32_t)(G8_BM >> 4) << 24 | id << 29;
}
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc));
}
// N consecutive fp32 columns of this warp's 32 lanes, without waiting for them.
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// One element of the result.  Accumulating, the addition is the memory's: each element gets one a call, so its place
// in time changes nothing, and nobody waits for the old value (loads of 8 rows before their stores kept 8 KB an SM in
// flight: 4085 x 2834 x 768 took 80 us).  It flushes subnormal sums to zero.
template <bool F32>
__device__ __forceinline__ void g8_put(const Gemm8Args& g, int64_t o, float v) {
  if (!F32) reinterpret_cast<__nv_bfloat16*>(g.c)[o] = __float2bfloat16_rn(v);
  else if (g.accumulate) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(reinterpret_cast<float*>(g.c) + o), "f"(v) : "memory");
  else reinterpret_cast<float*>(g.c)[o] = v;
}

// Place of a result in the scratch: the groups of 4 of a row in an order of their own, so that neither rows nor
// columns meet a bank twice.
__device__ __forceinline__ int g8_at(int r, int c) { return r * 32 + (((c >> 2) ^ (r & 7)) << 2) + (c & 3); }

// Four elements of a row of C from a multiple of 4 on, of which `left` exist.
template <bool F32>
__device__ __forceinline__ void g8_put4(const Gemm8Args& g, int64_t o, float4 v, int64_t left) {
  if (left >= 4) {
    if (!F32)
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(g.c) + o) = make_uint2(bf16x2_bits(v.x, v.y), bf16x2_bits(v.z, v.w));
    else if (g.accumulate)
      asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};"
                   ::"l"(reinterpret_cast<float*>(g.c) + o), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(g.c) + o) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) g8_put<F32>(g, o + i, (&v.x)[i]);
}

// Columns n .. n + 31 of the warp's 32 MMA rows m0 .. (one a lane).  Where C's rows are whole sectors a lane
// stores its row's; otherwise, and when accumulating, the rows pass through the warp's scratch and leave 32 columns
// at a time, 4 a lane where C's rows allow it (12000 x 3000 x 250 to bf16: 35 us, one a lane 48).  The loops over rows
// are short on purpose: unrolled to the end, their addresses spilled registers and that took 66.
template <bool F32>
__device__ __forceinline__ void g8_store32(const Gemm8Args& g, float* xs, int64_t m0, int64_t n, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  if (m0 >= g.M || n >= g.N) return;
  const int64_t m = m0 + lane;
  if (g.swap) {                         // lanes hold consecutive elements of a row of C
    if (m >= g.M) return;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (n + i < g.N) g8_put<F32>(g, (n + i) * g.ldc + m, v[i]);
    return;
  }
  if (g.sectors && !g.accumulate && n + 32 <= g.N) {
    if (m >= g.M) return;
    char* p = reinterpret_cast<char*>(g.c) + (m * g.ldc + n) * (F32 ? 4 : 2);
    uint32_t w[8];
    if (!F32) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = bf16x2_bits(v[16 * j + 2 * i], v[16 * j + 2 * i + 1]);
        st_sector(p + 32 * j, w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * j + i]);
        st_sector(p + 32 * j, w);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(xs + g8_at(lane, i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  __syncwarp();
  const int rows = (int)min((int64_t)32, g.M - m0);
  if (g.quads) {                        // 8 lanes a row
    const int r0 = lane >> 3, c = 4 * (lane & 7);
    const int64_t o = (m0 + r0) * g.ldc + n + c, left = g.N - n - c;
#pragma unroll 2
    for (int i = 0; i < 32; i += 4)
      if (r0 + i < rows) g8_put4<F32>(g, o + i * g.ldc, *reinterpret_cast<const float4*>(xs + g8_at(r0 + i, c)), left);
    __syncwarp();
    return;
  }
  if (n + lane < g.N) {
    const int64_t o = m0 * g.ldc + n + lane;
#pragma unroll 8
    for (int i = 0; i < rows; ++i) g8_put<F32>(g, o + i * g.ldc, xs[g8_at(i, lane)]);
  }
  __syncwarp();
}

// One lane of the warp; what it issues keeps its operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

constexpr int G8_RASTER = 8;           // tile rows that run side by side, so that their panels stay in L2

__device__ __forceinline__ void g8_tile(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t& ti, int64_t& tj) {
  const int64_t per = G8_RASTER * tiles_n, first = t / per * G8_RASTER;
  const int64_t rows = min(tiles_m - first, (int64_t)G8_RASTER), loc = t % per;
  ti = first + loc % rows;
  tj = loc / rows;
}

// A cluster's stretches: every CTA adds 1 / P of the tile's elements, the
// stretches in their order, lanes along C's rows, 4 elements at a time where C's
// rows allow it.  8 loads of 16 bytes from the others' shared memory are in
// flight (61 x 448 x 2560 fp32: 7.0 us; single elements,
// 4 in flight, 15.5).
template <int BN, int P, bool F32>
__device__ __forceinline__ void g8_join(const Gemm8Args& g, float* sums, int64_t m0, int64_t n0, int part) {
  using SM = Gemm8Smem<BN>;
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const float* from[P];
#pragma unroll
  for (int k = 0; k < P; ++k) from[k] = cluster.map_shared_rank(sums, k);
  constexpr int LOG = BN == 16 ? 4 : BN == 32 ? 5 : BN == 64 ? 6 : 7;
  const int log = g.swap ? 7 : LOG, mask = (1 << log) - 1, ld = g.swap ? SM::PART_LDT : SM::PART_LD;       // C's rows in the tile
  const int64_t row0 = g.swap ? n0 : m0, col0 = g.swap ? m0 : n0, rows = g.swap ? g.N : g.M, cols = g.swap ? g.M : g.N;
  constexpr int SHARE = G8_BM * BN / P;
  if (g.quads) {
    constexpr int U = 8 / P;
    for (int u0 = threadIdx.x; u0 < SHARE / 4; u0 += U * G8_THREADS) {
      float4 w[U][P];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = part * SHARE + 4 * (u0 + u * G8_THREADS);
#pragma unroll
        for (int k = 0; k < P; ++k)
          if (u0 + u * G8_THREADS < SHARE / 4) w[u][k] = *reinterpret_cast<const float4*>(from[k] + (e >> log) * ld + (e & mask));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = part * SHARE + 4 * (u0 + u * G8_THREADS);
        const int64_t row = row0 + (e >> log), col = col0 + (e & mask);
        if (u0 + u * G8_THREADS >= SHARE / 4 || row >= rows || col >= cols) continue;
        float4 v = w[u][0];
#pragma unroll
        for (int k = 1; k < P; ++k) v = make_float4(v.x + w[u][k].x, v.y + w[u][k].y, v.z + w[u][k].z, v.w + w[u][k].w);
        g8_put4<F32>(g, row * g.ldc + col, v, cols - col);
      }
    }
    return;
  }
  constexpr int U = 32 / P;
  for (int e0 = threadIdx.x; e0 < SHARE; e0 += U * G8_THREADS) {
    float w[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = part * SHARE + e0 + u * G8_THREADS;
#pragma unroll
      for (int k = 0; k < P; ++k)
        if (e0 + u * G8_THREADS < SHARE) w[u][k] = from[k][(e >> log) * ld + (e & mask)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = part * SHARE + e0 + u * G8_THREADS;
      const int64_t row = row0 + (e >> log), col = col0 + (e & mask);
      if (e0 + u * G8_THREADS >= SHARE || row >= rows || col >= cols) continue;
      float v = w[u][0];
#pragma unroll
      for (int k = 1; k < P; ++k) v += w[u][k];
      g8_put<F32>(g, row * g.ldc + col, v);
    }
  }
}

// A persistent CTA takes tiles blockIdx.x, + gridDim.x, ...; a cluster (few
// tiles) shares one tile, each CTA a stretch of K, and every CTA adds and
// writes its share of the columns, in the order of the stretches.
template <int BN, bool PROMOTE>
__global__ void __launch_bounds__(G8_THREADS, Gemm8Smem<BN>::CTAS)
gemm8_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, Gemm8Args g) {
  using SM = Gemm8Smem<BN>;
  namespace cg = cooperative_groups;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  uint8_t* tail = gbase + SM::OFF_BAR;
  const uint32_t bars = smem_u32(tail);
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (SM::STAGES + s); };
  auto acc_full = [&](uint32_t b) { return bars + 8u * (2 * SM::STAGES + b); };
  auto acc_empty = [&](uint32_t b) { return bars + 8u * (2 * SM::STAGES + 2 + b); };
  const uint32_t final_bar = bars + 8u * (2 * SM::STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 8 * (2 * SM::STAGES + 5));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();

  if (threadIdx.x == 0) {
    if (g.K > 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    }
    for (int s = 0; s < SM::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), G8_EPI_WARPS);
    }
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(tmem_slot)), "r"((uint32_t)SM::TMEM_COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_previous();
  let_next_start();

  const int64_t tiles_m = (g.M + G8_BM - 1) / G8_BM, tiles_n = (g.N + BN - 1) / BN;
  const int64_t tiles = tiles_m * tiles_n;
  const int64_t first_tile = blockIdx.x / parts, tile_step = gridDim.x / parts;
  // this CTA's stretch of K in blocks (whole scale groups)
  const int nkb = (int)((g.K + G8_BK - 1) / G8_BK);
  const int groups = (nkb + 3) / 4;
  const int kb0 = 4 * (int)((int64_t)groups * part / parts), kb1 = min(nkb, 4 * (int)((int64_t)groups * (part + 1) / parts));

  if (warp == 0) {
    // ------------------------------------------------ loads
    uint32_t q = 0;
    bool ok = true;
    for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
      int64_t ti, tj;
      g8_tile(t, tiles_m, tiles_n, ti, tj);
      const int64_t rb_b = tj * BN / 128;              // first 128-row block of B's scales
      for (int kb = kb0; kb < kb1; ++kb, ++q) {
        const uint32_t s = q % SM::STAGES, round = q / SM::STAGES;
        if (round > 0 && !mbar_wait(empty_bar(s), (round - 1) & 1, g.err, abort_flag)) {
          ok = false;
          break;
        }
        const bool head = (kb & 3) == 0;
        const uint32_t st = base + s * (SM::A_BYTES + SM::B_BYTES);
        if (elect_one()) {
          mbar_expect_tx(full_bar(s), SM::A_BYTES + SM::B_BYTES + (head ? 1024u : 0u));
          tma_load_2d(st, &map_a, full_bar(s), kb * G8_BK, (int)(ti * G8_BM));
          tma_load_2d(st + SM::A_BYTES, &map_b, full_bar(s), kb * G8_BK, (int)(tj * BN));
          if (head) {
            const uint32_t sf = base + SM::OFF_SF + s * SM::SF_BYTES;
            bulk_load(sf, g.sa + ((int64_t)(kb >> 2) * g.sa_rb + ti) * 512, 512u, full_bar(s));
            bulk_load(sf + 512, g.sb + ((int64_t)(kb >> 2) * g.sb_rb + rb_b) * 512, 512u, full_bar(s));
          }
        }
        __syncwarp();
      }
    }
    // every copy issued has landed before the CTA may exit
    for (uint32_t i = (q > (uint32_t)SM::STAGES ? q - SM::STAGES : 0u); i < q; ++i)
      mbar_wait_own(full_bar(i % SM::STAGES), (i / SM::STAGES) & 1, g.err);
  } else if (warp == 1) {
    // ------------------------------------------------ MMAs
    // The warp runs the loop together and one elected lane issues: descriptors then stay in uniform
    // registers (a loop of lane 0 alone took 0.39 us a block of a pair's tile, not 0.26).
    uint32_t q = 0, seg = 0, grp = 0;
    bool ok = true;
    for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
      for (int kb = kb0; kb < kb1; ++kb, ++q) {
        const bool first = PROMOTE ? ((kb - kb0) % G8_SEGMENT == 0) : kb == kb0;
        const bool last = kb == kb1 - 1 || (PROMOTE && (kb - kb0) % G8_SEGMENT == G8_SEGMENT - 1);
        const uint32_t buf = seg & 1, s = q % SM::STAGES;
        if ((first && seg >= 2 && !mbar_wait(acc_empty(buf), ((seg >> 1) - 1) & 1, g.err, abort_flag)) ||
            !mbar_wait(full_bar(s), (q / SM::STAGES) & 1, g.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = base + s * (SM::A_BYTES + SM::B_BYTES);
        const bool head = (kb & 3) == 0;
        grp += head;
        const uint32_t tsf = tmem + SM::SF_COL + (grp & 1) * SM::SF_COLS;
        const uint32_t idesc = mx_idesc<BN>(kb & 3);
        const uint64_t da = sw128_desc(st), db = sw128_desc(st + SM::A_BYTES);
        const uint32_t d = tmem + buf * SM::ACC_COLS;
        if (elect_one()) {
          if (head) {
            const uint64_t sf = scale_desc(base + SM::OFF_SF + s * SM::SF_BYTES);
            copy_scales(tsf, sf);
            copy_scales(tsf + 4, sf + 32);
          }
#pragma unroll
          for (int k = 0; k < G8_BK / 32; ++k)
            mx_mma(d, da + 2 * k, db + 2 * k, idesc, tsf, tsf + 4, first && k == 0 ? 0u : 1u);
          tc_commit(empty_bar(s));
          if (last) tc_commit(acc_full(buf));
        }
        __syncwarp();
        seg += last;
      }
    }
    // every MMA issued has completed before tensor memory is released
    if (elect_one()) tc_commit(final_bar);
    __syncwarp();
    mbar_wait_own(final_bar, 0, g.err);
  } else {
    // ------------------------------------------------ sums and results
    constexpr int HALF = BN >= 64 ? BN / 2 : BN;       // columns of a warp (BN <= 32: the first four warps take all)
    constexpr int STEP = HALF < 32 ? HALF : 32;
    const int qd = warp & 3, own = (warp - 2) >> 2;
    const bool works = BN >= 64 || own == 0;
    const uint32_t tlane = tmem + ((uint32_t)(qd * 32) << 16) + (uint32_t)(own * HALF);
    float* xs = reinterpret_cast<float*>(gbase + SM::OFF_XS) + (warp - 2) * G8_XS;
    const int segs = kb1 <= kb0 ? 0 : PROMOTE ? (kb1 - kb0 + G8_SEGMENT - 1) / G8_SEGMENT : 1;
    uint32_t seg = 0;
    for (int64_t t = first_tile; t < tiles; t += tile_step) {
      int64_t ti, tj;
      g8_tile(t, tiles_m, tiles_n, ti, tj);
      float sum[HALF];
#pragma unroll
      for (int j = 0; j < HALF; ++j) sum[j] = 0.f;
      bool ok = true;
      for (int i = 0; i < segs; ++i, ++seg) {
        const uint32_t buf = seg & 1;
        if (!mbar_wait(acc_full(buf), (seg >> 1) & 1, g.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (works) {
#pragma unroll
          for (int j = 0; j < HALF; j += STEP) {
            uint32_t v[STEP];
#pragma unroll
            for (int k = 0; k < STEP; k += 16) tmem_ld16_nowait(tlane + buf * SM::ACC_COLS + j + k, v + k);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < STEP; ++k) sum[j + k] += __uint_as_float(v[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buf));
      }
      if (!ok) break;
      if (!works) continue;
      if (parts == 1) {
#pragma unroll
        for (int j = 0; j < HALF; j += STEP) {
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = k < STEP ? sum[j + k] : 0.f;
          g8_store32<PROMOTE>(g, xs, ti * G8_BM + qd * 32, tj * BN + own * HALF + j, v);
        }
      } else {
        // to this CTA's own shared memory (the ring is idle: its last MMA has completed), for the cluster
        float* mine = reinterpret_cast<float*>(gbase);
        const int r = qd * 32 + lane;
        if (g.swap) {
#pragma unroll
          for (int j = 0; j < HALF; ++j) mine[(own * HALF + j) * SM::PART_LDT + r] = sum[j];
        } else {
#pragma unroll
          for (int j = 0; j < HALF; j += 4)
            *reinterpret_cast<float4*>(mine + r * SM::PART_LD + own * HALF + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
        }
      }
    }
  }

  if (parts > 1) {
    __syncwarp();
    cluster.sync();
    int64_t ti, tj;
    g8_tile(first_tile, tiles_m, tiles_n, ti, tj);
    if (parts == 2) g8_join<BN, 2, PROMOTE>(g, reinterpret_cast<float*>(gbase), ti * G8_BM, tj * BN, part);
    else if (parts == 4) g8_join<BN, 4, PROMOTE>(g, reinterpret_cast<float*>(gbase), ti * G8_BM, tj * BN, part);
    else g8_join<BN, 8, PROMOTE>(g, reinterpret_cast<float*>(gbase), ti * G8_BM, tj * BN, part);
    // the others have read this CTA's sums (nothing else is ordered: its results need not have reached memory)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 ::"r"(tmem), "r"((uint32_t)SM::TMEM_COLS) : "memory");
  }
}

// ------------------------------------------------------------------ pairs of CTAs
// Larger products: the two SMs of a CTA pair share one tcgen05.mma of M = N = 256
// (cta_group::2).  Each CTA holds 128 rows of A and 128 of B, so that a block of
// 128 columns costs it 32 KB of loads and 512 cycles of MMA: half the loads and
// shared-memory reads of a 128 x 128 tile at the same rate.
//
// The even CTA (the leader) issues the MMAs and the scale copies for both.
// Both CTAs' loads complete on the leader's barriers; commits go to both CTAs;
// "drained" comes back to the leader from both.
//
// Tensor memory holds two sum buffers and two of scales.  Two buffers of 256
// columns do not fit beside the scales: they share 32 columns (0..255 and
// 224..479), which the drain reads first; the next tile's MMAs wait for those,
// and for the rest of the tile before it.
struct PairSmem {
  static constexpr int BN = 256;
  static constexpr int A_BYTES = 128 * G8_BK;
  static constexpr int B_BYTES = BN / 2 * G8_BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SF_BYTES = 512 * 3;                             // own rows of A, all of B
  static constexpr int STAGES = 5;
  static constexpr int OFF_SF = STAGES * STAGE_BYTES;
  static constexpr int OFF_XS = OFF_SF + STAGES * SF_BYTES;            // a scratch of each drain warp
  static constexpr int OFF_BAR = OFF_XS + G8_EPI_WARPS * G8_XS * 4;
  static constexpr int BYTES = 1024 + OFF_BAR + 256;
  static constexpr int ACC1 = 224;                                     // second buffer's first column
  static constexpr int SF_COL = ACC1 + BN, SF_COLS = 12;
  static_assert(SF_COL + 2 * SF_COLS <= 512, "tensor memory");
  static_assert(BYTES <= 232448, "shared memory");
};

struct PairMaps {
  CUtensorMap a, b, sa, sb;
};

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void mx_mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                            uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc));
}
// Arrives on the barrier of both CTAs once the MMAs and copies issued so far have completed.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(bar), "h"((uint16_t)3) : "memory");
}
// On a barrier of another CTA of the cluster.  Relaxed: it tells that tensor memory has been read
// (tcgen05.wait::ld has returned), and no memory is handed over; a release waited for everything this
// thread had in flight, 0.8 us of every segment (4096 x 1024 x 8192 to fp32: 43.0 us, 36.9 us relaxed).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <bool PROMOTE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(G8_PAIR_THREADS, 1)
gemm8_pair_kernel(const __grid_constant__ PairMaps maps, Gemm8Args g) {
  using SM = PairSmem;
  constexpr int BN = SM::BN;
  namespace cg = cooperative_groups;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* tail = smem_raw + (base - raw) + SM::OFF_BAR;
  const uint32_t bars = smem_u32(tail);
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (SM::STAGES + s); };
  auto acc_full = [&](uint32_t b) { return bars + 8u * (2 * SM::STAGES + b); };
  auto acc_empty = [&](uint32_t b) { return bars + 8u * (2 * SM::STAGES + 2 + b); };
  const uint32_t shared_empty = bars + 8u * (2 * SM::STAGES + 4);
  const uint32_t final_bar = bars + 8u * (2 * SM::STAGES + 5);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 8 * (2 * SM::STAGES + 6));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    const CUtensorMap* all[4] = {&maps.a, &maps.b, &maps.sa, &maps.sb};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(all[i])) : "memory");
    for (int s = 0; s < SM::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 2 * G8_EPI_WARPS);
    }
    mbar_init(shared_empty, G8_EPI_WARPS);          // four warps of each CTA
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster.sync();                                    // the peer's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_previous();
  let_next_start();
  uint32_t to_leader;                                // from a barrier to the leader's
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to_leader) : "r"(bars));
  to_leader -= bars;

  const int64_t tiles_m = (g.M + 255) / 256, tiles_n = (g.N + BN - 1) / BN;
  const int64_t tiles = tiles_m * tiles_n;
  const int64_t first_tile = blockIdx.x / 2, tile_step = gridDim.x / 2;
  const int nkb = (int)((g.K + G8_BK - 1) / G8_BK);

  // registers: 384 x 168 at launch; 128 x 80 + 256 x 208 = 63488 now
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  if (warp == 0) {
    // ------------------------------------------------ loads of this CTA's halves
    uint32_t q = 0;
    bool ok = true;
    for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
      int64_t ti, tj;
      g8_tile(t, tiles_m, tiles_n, ti, tj);
      const int ra = (int)(2 * ti + rank), rb = (int)(tj * BN / 128);   // (first) blocks of 128 rows
      for (int kb = 0; kb < nkb; ++kb, ++q) {
        const uint32_t s = q % SM::STAGES, round = q / SM::STAGES;
        if (round > 0 && !mbar_wait(empty_bar(s), (round - 1) & 1, g.err, abort_flag)) {
          ok = false;
          break;
        }
        const bool head = (kb & 3) == 0;
        const uint32_t st = base + s * SM::STAGE_BYTES, bar = full_bar(s) + to_leader;
        if (elect_one()) {
          if (leader) mbar_expect_tx(full_bar(s), 2 * (SM::STAGE_BYTES + (head ? SM::SF_BYTES : 0)));
          tma_load_2d_pair(st, &maps.a, bar, kb * G8_BK, ra * 128);
          tma_load_2d_pair(st + SM::A_BYTES, &maps.b, bar, kb * G8_BK, (int)(tj * BN) + (int)rank * (BN / 2));
          if (head) {
            const uint32_t sf = base + SM::OFF_SF + s * SM::SF_BYTES;
            tma_load_2d_pair(sf, &maps.sa, bar, 0, (kb >> 2) * (int)g.sa_rb + ra);
            tma_load_2d_pair(sf + 512, &maps.sb, bar, 0, (kb >> 2) * (int)g.sb_rb + rb);
          }
        }
        __syncwarp();
      }
    }
    // the leader sees every copy of both CTAs land before either may exit
    if (leader)
      for (uint32_t i = (q > (uint32_t)SM::STAGES ? q - SM::STAGES : 0u); i < q; ++i)
        mbar_wait_own(full_bar(i % SM::STAGES), (i / SM::STAGES) & 1, g.err);
  } else if (warp == 1) {
    // ------------------------------------------------ MMAs (leader)
    // The warp runs the loop together and one elected lane issues: descriptors then stay in uniform registers.
    if (leader) {
      uint32_t q = 0, seg = 0, grp = 0;
      bool ok = true;
      for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
        for (int kb = 0; kb < nkb; ++kb, ++q) {
          const bool first = PROMOTE ? kb % G8_PAIR_SEGMENT == 0 : kb == 0;
          const bool last = kb == nkb - 1 || (PROMOTE && kb % G8_PAIR_SEGMENT == G8_PAIR_SEGMENT - 1);
          const uint32_t buf = seg & 1;
          if (first) {
            if ((seg >= 1 && !mbar_wait(shared_empty, (seg - 1) & 1, g.err, abort_flag)) ||
                (seg >= 2 && !mbar_wait(acc_empty(buf), ((seg >> 1) - 1) & 1, g.err, abort_flag))) {
              ok = false;
              break;
            }
          }
          const uint32_t s = q % SM::STAGES;
          if (!mbar_wait(full_bar(s), (q / SM::STAGES) & 1, g.err, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = base + s * SM::STAGE_BYTES;
          const bool head = (kb & 3) == 0;
          grp += head;
          const uint32_t tsf = tmem + SM::SF_COL + (grp & 1) * SM::SF_COLS;
          const uint32_t id = kb & 3;
          const uint32_t idesc = id << 4 | (uint32_t)(BN >> 3) << 17 | 1u << 23 | (256u >> 4) << 24 | id << 29;
          const uint64_t da = sw128_desc(st), db = sw128_desc(st + SM::A_BYTES);
          const uint32_t d = tmem + buf * SM::ACC1;
          if (elect_one()) {
            if (head) {
              const uint64_t sf = scale_desc(base + SM::OFF_SF + s * SM::SF_BYTES);
#pragma unroll
              for (int b = 0; b < 3; ++b) copy_scales_pair(tsf + 4 * b, sf + 32 * b);
            }
#pragma unroll
            for (int k = 0; k < G8_BK / 32; ++k)
              mx_mma_pair(d, da + 2 * k, db + 2 * k, idesc, tsf, tsf + 4, first && k == 0 ? 0u : 1u);
            tc_commit_pair(empty_bar(s));
            if (last) tc_commit_pair(acc_full(buf));
          }
          __syncwarp();
          seg += last;
        }
      }
      if (elect_one()) tc_commit_pair(final_bar);
      __syncwarp();
      mbar_wait_own(final_bar, 0, g.err);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------ sums and results
    constexpr int HALF = BN / 2, STEP = 32;            // columns of a warp, and of one read
    const int qd = warp & 3, own = (warp >> 2) - 1;   // tensor-memory lane quadrant, column half
    const uint32_t tlane = tmem + ((uint32_t)(qd * 32) << 16) + own * HALF;
    float* xs = reinterpret_cast<float*>(smem_raw + (base - raw) + SM::OFF_XS) + (warp - 4) * G8_XS;
    const int segs = PROMOTE ? (nkb + G8_PAIR_SEGMENT - 1) / G8_PAIR_SEGMENT : 1;
    uint32_t seg = 0;
    for (int64_t t = first_tile; t < tiles; t += tile_step) {
      int64_t ti, tj;
      g8_tile(t, tiles_m, tiles_n, ti, tj);
      float sum[HALF];
      bool ok = true;
      for (int i = 0; i < segs; ++i, ++seg) {
        const uint32_t buf = seg & 1;
        if (!mbar_wait(acc_full(buf), (seg >> 1) & 1, g.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // where the buffers share columns (224..255 of the first, 0..31 of the second), the upper
        // half's warps go downwards, so that both begin with those
#pragma unroll
        for (int j = 0; j < HALF; j += STEP) {
          uint32_t v[STEP];
          const uint32_t at = tlane + buf * SM::ACC1 + (own ? HALF - STEP - j : j);
#pragma unroll
          for (int k = 0; k < STEP; k += 16) tmem_ld16_nowait(at + k, v + k);
          tmem_ld_wait();
          if (j == 0 && own != (int)buf) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(shared_empty + to_leader);
          }
#pragma unroll
          for (int k = 0; k < STEP; ++k) sum[j + k] = (PROMOTE && i > 0 ? sum[j + k] : 0.f) + __uint_as_float(v[k]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty(buf) + to_leader);
      }
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < HALF; j += STEP) {
        float v[STEP];
#pragma unroll
        for (int k = 0; k < STEP; ++k) v[k] = sum[j + k];
g8_store32<PROMOTE>(g, xs, ti * 256 + rank * 128 + qd * 32, tj * BN + own * HALF + (own ? HALF - STEP - j : j), v);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster.sync();                                    // both CTAs are done with each other's barriers and tensor memory
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace precond
