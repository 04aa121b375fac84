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
#pragma once

#include <cooperative_groups.h>
#include <cuda.h>

#include "form8.cuh"
#include "ptx.cuh"

namespace precond {

constexpr int G8_BM = 128;             // rows of A a CTA takes (the MMA's M)
constexpr int G8_BK = 128;             // one scale block, one swizzled row
constexpr int G8_SEGMENT = 4;          // blocks between promotions (512 columns: one scale group)
constexpr int G8_EPI_WARPS = 8;
constexpr int G8_THREADS = 64 + 32 * G8_EPI_WARPS;

struct Gemm8Args {
  int64_t M, N, K;                     // of the MMA's view: M rows of its A operand
  const uint8_t* sa; int64_t sa_rb;    // scales and their blocks of 128 rows
  const uint8_t* sb; int64_t sb_rb;
  void* c; int64_t ldc;
  int c_bf16, accumulate;
  int swap;                            // 1: C is N x M (the operands were exchanged)
  unsigned int* err;
};

template <int BN>
struct Gemm8Smem {
  static constexpr int A_BYTES = G8_BM * G8_BK;
  static constexpr int B_BYTES = BN * G8_BK;
  static constexpr int SFB_ATOMS = (BN + 127) / 128;
  static constexpr int SF_BYTES = 512 * (1 + SFB_ATOMS);
  static constexpr int STAGES = BN >= 128 ? 6 : 8;
  static constexpr int OFF_SF = STAGES * (A_BYTES + B_BYTES);
  static constexpr int OFF_BAR = OFF_SF + STAGES * SF_BYTES;
  static constexpr int BYTES = 1024 + OFF_BAR + 256;
  // tensor memory: two sum buffers, then two scale buffers
  static constexpr int ACC_COLS = BN < 32 ? 32 : BN;
  static constexpr int SF_COL = 2 * ACC_COLS;
  static constexpr int SF_COLS = 4 * (1 + SFB_ATOMS);
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

// One element of the result.
__device__ __forceinline__ void g8_store(const Gemm8Args& g, int64_t o, float v) {
  if (g.c_bf16) {
    reinterpret_cast<__nv_bfloat16*>(g.c)[o] = __float2bfloat16_rn(v);
  } else {
    float* p = reinterpret_cast<float*>(g.c) + o;
    *p = g.accumulate ? *p + v : v;
  }
}

// 16 consecutive columns n .. of MMA row m.
__device__ __forceinline__ void g8_store16(const Gemm8Args& g, int64_t m, int64_t n, const float (&v)[16]) {
  if (m >= g.M) return;
  if (g.swap) {                         // lanes hold consecutive elements of a row of C
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n + i < g.N) g8_store(g, (n + i) * g.ldc + m, v[i]);
    return;
  }
  const int64_t o = m * g.ldc + n;
  const int size = g.c_bf16 ? 2 : 4;
  char* p = reinterpret_cast<char*>(g.c) + o * size;
  if (n + 16 <= g.N && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    if (g.c_bf16) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = bf16x2_bits(v[2 * i], v[2 * i + 1]);
      reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4* q = reinterpret_cast<float4*>(p) + i;
        float4 x = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (g.accumulate) {
          const float4 y = *q;
          x = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
        }
        *q = x;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (n + i < g.N) g8_store(g, o + i, v[i]);
}

constexpr int G8_RASTER = 8;           // tile rows that run side by side, so that their panels stay in L2

__device__ __forceinline__ void g8_tile(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t& ti, int64_t& tj) {
  const int64_t per = G8_RASTER * tiles_n, first = t / per * G8_RASTER;
  const int64_t rows = min(tiles_m - first, (int64_t)G8_RASTER), loc = t % per;
  ti = first + loc % rows;
  tj = loc / rows;
}

// A persistent CTA takes tiles blockIdx.x, + gridDim.x, ...; a cluster (few
// tiles) shares one tile, each CTA a stretch of K, and every CTA adds and
// writes its share of the columns, in the order of the stretches.
template <int BN, bool PROMOTE>
__global__ void __launch_bounds__(G8_THREADS, 1)
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

  const int64_t tiles_m = (g.M + G8_BM - 1) / G8_BM, tiles_n = (g.N + BN - 1) / BN;
  const int64_t tiles = tiles_m * tiles_n;
  const int64_t first_tile = blockIdx.x / parts, tile_step = gridDim.x / parts;
  // this CTA's stretch of K in blocks (whole scale groups)
  const int nkb = (int)((g.K + G8_BK - 1) / G8_BK);
  const int groups = (nkb + 3) / 4;
  const int kb0 = 4 * (int)((int64_t)groups * part / parts), kb1 = min(nkb, 4 * (int)((int64_t)groups * (part + 1) / parts));

  if (warp == 0) {
    // ------------------------------------------------ loads
    if (lane == 0) {
      uint32_t q = 0;
      bool ok = true;
      for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
        int64_t ti, tj;
        g8_tile(t, tiles_m, tiles_n, ti, tj);
        const int64_t rb_b = tj * BN / 128;              // first 128-row block of B's scales
        const uint32_t sfb_bytes = 512u * (uint32_t)min((int64_t)SM::SFB_ATOMS, g.sb_rb - rb_b);
        for (int kb = kb0; kb < kb1; ++kb, ++q) {
          const uint32_t s = q % SM::STAGES, round = q / SM::STAGES;
          if (round > 0 && !mbar_wait(empty_bar(s), (round - 1) & 1, g.err, abort_flag)) {
            ok = false;
            break;
          }
          const bool head = (kb & 3) == 0;
          const uint32_t st = base + s * (SM::A_BYTES + SM::B_BYTES);
          mbar_expect_tx(full_bar(s), SM::A_BYTES + SM::B_BYTES + (head ? 512u + sfb_bytes : 0u));
          tma_load_2d(st, &map_a, full_bar(s), kb * G8_BK, (int)(ti * G8_BM));
          tma_load_2d(st + SM::A_BYTES, &map_b, full_bar(s), kb * G8_BK, (int)(tj * BN));
          if (head) {
            const uint32_t sf = base + SM::OFF_SF + s * SM::SF_BYTES;
            bulk_load(sf, g.sa + ((int64_t)(kb >> 2) * g.sa_rb + ti) * 512, 512u, full_bar(s));
            bulk_load(sf + 512, g.sb + ((int64_t)(kb >> 2) * g.sb_rb + rb_b) * 512, sfb_bytes, full_bar(s));
          }
        }
      }
      // every copy issued has landed before the CTA may exit
      for (uint32_t i = (q > (uint32_t)SM::STAGES ? q - SM::STAGES : 0u); i < q; ++i)
        mbar_wait_own(full_bar(i % SM::STAGES), (i / SM::STAGES) & 1, g.err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMAs
    if (lane == 0) {
      uint32_t q = 0, seg = 0, grp = 0;
      bool ok = true;
      for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
        for (int kb = kb0; kb < kb1; ++kb, ++q) {
          const bool first = PROMOTE ? ((kb - kb0) % G8_SEGMENT == 0) : kb == kb0;
          const uint32_t buf = seg & 1;
          if (first) {
            if (seg >= 2 && !mbar_wait(acc_empty(buf), ((seg >> 1) - 1) & 1, g.err, abort_flag)) {
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
          const uint32_t st = base + s * (SM::A_BYTES + SM::B_BYTES);
          if ((kb & 3) == 0) {
            ++grp;
            const uint32_t sf = base + SM::OFF_SF + s * SM::SF_BYTES;
            const uint32_t tsf = tmem + SM::SF_COL + (grp & 1) * SM::SF_COLS;
            copy_scales(tsf, scale_desc(sf));
#pragma unroll
            for (int b = 0; b < SM::SFB_ATOMS; ++b) copy_scales(tsf + 4 + 4 * b, scale_desc(sf + 512 + 512 * b));
          }
          const uint32_t tsf = tmem + SM::SF_COL + (grp & 1) * SM::SF_COLS;
          const uint32_t idesc = mx_idesc<BN>(kb & 3);
#pragma unroll
          for (int k = 0; k < G8_BK / 32; ++k)
            mx_mma(tmem + buf * SM::ACC_COLS, sw128_desc(st + 32 * k), sw128_desc(st + SM::A_BYTES + 32 * k), idesc, tsf,
                   tsf + 4, first && k == 0 ? 0u : 1u);
          tc_commit(empty_bar(s));
          if (kb == kb1 - 1 || (PROMOTE && (kb - kb0) % G8_SEGMENT == G8_SEGMENT - 1)) {
            tc_commit(acc_full(buf));
            ++seg;
          }
        }
      }
      // every MMA issued has completed before tensor memory is released
      tc_commit(final_bar);
      mbar_wait_own(final_bar, 0, g.err);
    }
  } else {
    // ------------------------------------------------ sums and results
    constexpr int HALF = BN >= 32 ? BN / 2 : BN;       // columns of this warp (BN = 16: the first four warps take all)
    const int qd = warp & 3, own = (warp - 2) >> 2;
    const bool works = BN >= 32 || own == 0;
    const int r = qd * 32 + lane;
    const uint32_t tlane = tmem + ((uint32_t)(qd * 32) << 16) + (uint32_t)(own * HALF);
    const int segs = kb1 <= kb0 ? 0 : PROMOTE ? (kb1 - kb0 + G8_SEGMENT - 1) / G8_SEGMENT : 1;
    uint32_t seg = 0;
    for (int64_t t = first_tile; t < tiles; t += tile_step) {
      int64_t ti, tj;
      g8_tile(t, tiles_m, tiles_n, ti, tj);
      const int64_t m = ti * G8_BM + r, n0 = tj * BN + own * HALF;
      float acc[HALF];
#pragma unroll
      for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
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
          for (int j = 0; j < HALF; j += 16) {
            uint32_t v[16];
            tmem_ld16_nowait(tlane + buf * SM::ACC_COLS + j, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[j + k] += __uint_as_float(v[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buf));
      }
      if (!ok) break;
      if (parts == 1) {
        if (works) {
#pragma unroll
          for (int j = 0; j < HALF; j += 16) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = acc[j + k];
            g8_store16(g, m, n0 + j, v);
          }
        }
      } else if (works) {
        // this CTA's sums to its own shared memory (the ring is idle: its last MMA has completed),
        // columns outermost, for the cluster to read
        float* mine = reinterpret_cast<float*>(gbase);
#pragma unroll
        for (int j = 0; j < HALF; ++j) mine[(own * HALF + j) * G8_BM + r] = acc[j];
      }
    }
  }

  if (parts > 1) {
    __syncwarp();
    cluster.sync();
    // column c of the tile belongs to CTA c % parts; 128 threads a column
    int64_t ti, tj;
    g8_tile(first_tile, tiles_m, tiles_n, ti, tj);
    if (threadIdx.x < 256) {
      const int r = threadIdx.x & 127;
      const int64_t m = ti * G8_BM + r;
      for (int c = part + parts * (threadIdx.x >> 7); c < BN; c += 2 * parts) {
        float v = 0.f;
        for (int k = 0; k < parts; ++k)
          v += cluster.map_shared_rank(reinterpret_cast<float*>(gbase), k)[c * G8_BM + r];
        const int64_t n = tj * BN + c;
        if (m < g.M && n < g.N) g8_store(g, g.swap ? n * g.ldc + m : m * g.ldc + n, v);
      }
    }
    cluster.sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 ::"r"(tmem), "r"((uint32_t)SM::TMEM_COLS) : "memory");
  }
}

}  // namespace precond
