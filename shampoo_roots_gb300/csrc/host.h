// Host side of the operators, shared by their translation units: argument
// checks, launches, and the rules by which rows are laid on threads.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "form8.cuh"
#include "handle.h"

namespace precond {

constexpr int64_t MAX_SIDE = (int64_t)1 << 30;     // rows, columns: kernels index a side with 32 bits
constexpr int PLAN_SMS = 152;                       // a GB300's: sizes the dw workspace without a device
constexpr int PLAN_CLUSTERS[9] = {0, 152, 76, 0, 38, 0, 0, 0, 19};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t size_of(int dtype) { return dtype == PRECOND_F32 ? 4 : dtype == PRECOND_BF16 ? 2 : 1; }
inline bool float_type(int d) { return d == PRECOND_F32 || d == PRECOND_BF16; }
inline bool side(int64_t n) { return n >= 0 && n <= MAX_SIDE; }
// A matrix of `rows` x `cols` elements with rows `ld` apart; a matrix without elements needs neither pointer nor pitch.
inline bool matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype) {
  if (rows == 0 || cols == 0) return true;
  return ld >= cols && ld <= MAX_SIDE && p && aligned(p, size_of(dtype));
}
// An 8-bit matrix: 16-byte aligned rows, scales on 16 bytes.
inline bool matrix8(const void* q, int64_t ld, const uint8_t* s, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return true;
  return ld >= cols && ld % 16 == 0 && ld <= MAX_SIDE && q && s && aligned(q, 16) && aligned(s, 16);
}
// Rows that begin at multiples of 32 bytes.
inline bool sector_rows(const void* p, int64_t ld, int dtype) {
  return !p || (aligned(p, 32) && ld * (int64_t)size_of(dtype) % 32 == 0);
}
struct Range { const char* lo; const char* hi; int64_t pitch, width; };      // rows of `width` bytes, `pitch` apart
constexpr Range NOWHERE = {nullptr, nullptr, 0, 0};
inline Range range(const void* p, int64_t rows, int64_t ld, int64_t cols, size_t size) {
  const char* b = reinterpret_cast<const char*>(p);
  if (!p || rows <= 0 || cols <= 0) return NOWHERE;
  return {b, b + ((rows - 1) * ld + cols) * (int64_t)size, ld * (int64_t)size, cols * (int64_t)size};
}
// Where rows are equally far apart (column slices of one buffer), those of one may lie between the other's.
inline bool overlap(const Range& a, const Range& b) {
  if (!a.lo || !b.lo || a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.pitch != b.pitch || a.pitch <= 0) return true;
  const int64_t d = ((b.lo - a.lo) % a.pitch + a.pitch) % a.pitch;            // b's rows begin d bytes after a's
  return d < a.width || d + b.width > a.pitch;
}
inline Range scale_range(const uint8_t* s, int64_t rows, int64_t cols) {
  return range(s, 1, 0, (int64_t)q8_groups(cols) * q8_row_blocks(rows) * 512, 1);
}

inline int cuda_error(const char* what, cudaError_t e) {
  fprintf(stderr, "libprecond: %s: %s\n", what, cudaGetErrorString(e));
  return PRECOND_ECUDA;
}
#define OP_CK(call)                                              \
  do {                                                           \
    const cudaError_t e_ = (call);                               \
    if (e_ != cudaSuccess) return cuda_error(#call, e_);         \
  } while (0)

// The handle's device current, and (once) the kernels' attributes set: those of training.cu by training_attributes.
int prepare(Handle* h);
cudaError_t training_attributes();

// The attributes of a launch: programmatic (common.cuh, wait_for_previous), and a cluster of blocks; returns how many.
inline int launch_attributes(cudaLaunchAttribute (&at)[2], int cluster) {
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  return cluster > 1 ? 2 : 1;
}
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*k)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  cfg.numAttrs = launch_attributes(at, cluster);
  cfg.attrs = at;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// ------------------------------------------------------------------------- rows on threads
// Threads of a row, rows of a block and blocks of a row.  16 columns a thread, up
// to 384 threads (a bf16 gradient: 512); then a norm of aligned rows has 32 up
// to 512 threads (3000 x 16384 bf16: 58 us, in clusters of 4 61; without a
// residual 38 and 52; fp32, which spills in this form, 113 and 122, without a
// residual 68 and 87), and what is still longer a cluster of 2, 4 or 8 blocks.
// Longer rows (parts 0) take the kernels that read a row twice.  Blocks of short
// rows hold several, to have warps on each of the SM's four parts (norm of 20244
// x 1213 bf16: 4 rows of 3 warps 59 us, one row 84); up to 256 columns, where
// rows begin at sectors, a warp does.
struct RowShape { int threads, rows, vectors, parts; };
inline RowShape row_shape(int64_t cols, int dtype, bool grad, bool vec) {
  const int64_t one = grad && dtype == PRECOND_BF16 ? 512 : 384, n = (cols + 15) / 16;
  if (!grad && vec && n > one && n <= 1024) return {(int)((n + 63) / 64 * 32), 1, 2, 1};
  int parts = 1;
  while (parts < 8 && n > parts * one) parts *= 2;
  if (n > parts * one) return {512, 1, 0, 0};
  const int64_t mine = (n + parts - 1) / parts;
  const int threads = vec && n <= 16 ? (n <= 8 ? 8 : 16) : (int)std::max<int64_t>(32, (mine + 31) / 32 * 32);
  int rows = 1;
  while (parts == 1 && threads * rows % 128 && threads * (rows + 1) <= 384) ++rows;
  return {threads, rows, 1, parts};
}

// Blocks (or clusters) of a persistent grid: what the registers let an SM hold
// (norm of aligned bf16 rows, 16 columns a thread: 80 registers; other bf16:
// 128; fp32: 168).  Fewer clusters fit than SMs would hold, as each lies within
// a part of the chip; `clusters` of them with one block on an SM.
inline int64_t row_blocks_of(const RowShape& s, int64_t rows, int sm_threads, int sms, const int* clusters) {
  const int64_t resident = std::max(1, sm_threads / (s.threads * s.rows));
  const int64_t most = resident * (s.parts > 1 ? clusters[s.parts] : sms);
  return std::max<int64_t>(1, std::min((rows + s.rows - 1) / s.rows, most));
}
// ------------------------------------------------------------------------- gradients of the layer norm
// Rows of a gradient's block: as many as an SM's registers hold, for each block leaves sums of dw and db (777 x 1000 fp32).
inline RowShape layer_grad_shape(int64_t cols, int dtype, bool vec) {
  RowShape s = row_shape(cols, dtype, true, vec);
  if (s.parts == 1 && s.threads >= 32) s.rows = std::min(8, std::max(1, (dtype == PRECOND_F32 ? 384 : 512) / s.threads));
  return s;
}
inline int64_t layer_grad_blocks(const RowShape& s, int64_t rows, int dtype, int sms, const int* clusters) {
  return row_blocks_of(s, rows, dtype == PRECOND_F32 ? 384 : 512, sms, clusters);
}
// Few rows: a block, or a cluster of them, leaves dw and db itself, without a second kernel or a workspace: its blocks
// (0: not this way).  (14 x 192 fp32: 5.0 us, with two kernels 7.5; with a second turn, 100 x 1000 bf16, 10.3 and 8.3.)
inline int layer_grad_whole(const RowShape& s, int64_t rows) {
  const int64_t blocks = (rows + s.rows - 1) / s.rows;
  return s.parts != 1 || blocks > 8 ? 0 : blocks > 4 ? 8 : blocks > 2 ? 4 : (int)blocks;
}

}  // namespace precond
