// Host side of the training-step operators of include/precond.h: RMS norm and
// its gradients, the 8-bit form, the product of two 8-bit matrices and the
// distillation loss.  Arguments are checked here, before anything is enqueued;
// kernels go to the caller's stream and use no memory but the caller's.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>

#include "distill.cuh"
#include "gemm8.cuh"
#include "handle.h"
#include "quantize8.cuh"
#include "rms_norm.cuh"

using namespace precond;

namespace {

constexpr int64_t MAX_SIDE = (int64_t)1 << 30;     // rows, columns: kernels index a side with 32 bits
constexpr int GRAD_IN_PLACE = 8192;                 // columns up to which a gradient may be written over its inputs
constexpr int PLAN_SMS = 152;                       // a GB300's: sizes the dw workspace without a device
constexpr int PLAN_CLUSTERS[9] = {0, 152, 76, 0, 38, 0, 0, 0, 19};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t size_of(int dtype) { return dtype == PRECOND_F32 ? 4 : dtype == PRECOND_BF16 ? 2 : 1; }
bool float_type(int d) { return d == PRECOND_F32 || d == PRECOND_BF16; }
bool side(int64_t n) { return n >= 0 && n <= MAX_SIDE; }
// A matrix of `rows` x `cols` elements with rows `ld` apart; a matrix without elements needs neither pointer nor pitch.
bool matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype) {
  if (rows == 0 || cols == 0) return true;
  return ld >= cols && ld <= MAX_SIDE && p && aligned(p, size_of(dtype));
}
// An 8-bit matrix: 16-byte aligned rows, scales on 16 bytes.
bool matrix8(const void* q, int64_t ld, const uint8_t* s, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return true;
  return ld >= cols && ld % 16 == 0 && ld <= MAX_SIDE && q && s && aligned(q, 16) && aligned(s, 16);
}
// Rows that begin at multiples of 32 bytes.
bool sector_rows(const void* p, int64_t ld, int dtype) {
  return !p || (aligned(p, 32) && ld * (int64_t)size_of(dtype) % 32 == 0);
}
struct Range { const char* lo; const char* hi; int64_t pitch, width; };      // rows of `width` bytes, `pitch` apart
constexpr Range NOWHERE = {nullptr, nullptr, 0, 0};
Range range(const void* p, int64_t rows, int64_t ld, int64_t cols, size_t size) {
  const char* b = reinterpret_cast<const char*>(p);
  if (!p || rows <= 0 || cols <= 0) return NOWHERE;
  return {b, b + ((rows - 1) * ld + cols) * (int64_t)size, ld * (int64_t)size, cols * (int64_t)size};
}
// Where rows are equally far apart (column slices of one buffer), those of one may lie between the other's.
bool overlap(const Range& a, const Range& b) {
  if (!a.lo || !b.lo || a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.pitch != b.pitch || a.pitch <= 0) return true;
  const int64_t d = ((b.lo - a.lo) % a.pitch + a.pitch) % a.pitch;            // b's rows begin d bytes after a's
  return d < a.width || d + b.width > a.pitch;
}
Range scale_range(const uint8_t* s, int64_t rows, int64_t cols) {
  return range(s, 1, 0, (int64_t)q8_groups(cols) * q8_row_blocks(rows) * 512, 1);
}

int cuda_error(const char* what, cudaError_t e) {
  fprintf(stderr, "libprecond: %s: %s\n", what, cudaGetErrorString(e));
  return PRECOND_ECUDA;
}
#define OP_CK(call)                                              \
  do {                                                           \
    const cudaError_t e_ = (call);                               \
    if (e_ != cudaSuccess) return cuda_error(#call, e_);         \
  } while (0)

typedef void (*DistillKernel)(DistillArgs);
const DistillKernel distill_fused_kernels[2][5] = {
    {distill_kernel<float, 0, true>, distill_kernel<float, 1, true>, distill_kernel<float, 2, true>, distill_kernel<float, 4, true>,
     distill_kernel<float, 8, true>},
    {distill_kernel<__nv_bfloat16, 0, true>, distill_kernel<__nv_bfloat16, 1, true>, distill_kernel<__nv_bfloat16, 2, true>,
     distill_kernel<__nv_bfloat16, 4, true>, distill_kernel<__nv_bfloat16, 8, true>}};
const DistillKernel distill_split_kernels[2][5] = {
    {distill_kernel<float, 0, false>, distill_kernel<float, 1, false>, distill_kernel<float, 2, false>,
     distill_kernel<float, 4, false>, distill_kernel<float, 8, false>},
    {distill_kernel<__nv_bfloat16, 0, false>, distill_kernel<__nv_bfloat16, 1, false>, distill_kernel<__nv_bfloat16, 2, false>,
     distill_kernel<__nv_bfloat16, 4, false>, distill_kernel<__nv_bfloat16, 8, false>}};
const DistillKernel distill_candidates_kernels[2][3] = {
    {distill_candidates_kernel<float, FewCandidates<4>>, distill_candidates_kernel<float, FewCandidates<8>>,
     distill_candidates_kernel<float, ManyCandidates>},
    {distill_candidates_kernel<__nv_bfloat16, FewCandidates<4>>, distill_candidates_kernel<__nv_bfloat16, FewCandidates<8>>,
     distill_candidates_kernel<__nv_bfloat16, ManyCandidates>}};

// The device current and the kernels' attributes set.
template <int BN>
cudaError_t gemm8_attributes() {
  cudaError_t e = cudaFuncSetAttribute(gemm8_kernel<BN, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Gemm8Smem<BN>::BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(gemm8_kernel<BN, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Gemm8Smem<BN>::BYTES);
  return e;
}
int prepare(Handle* h) {
  int now = -1;
  OP_CK(cudaGetDevice(&now));
  if (now != h->device) OP_CK(cudaSetDevice(h->device));
  if (!h->op_ready) {
    OP_CK(gemm8_attributes<16>());
    OP_CK(gemm8_attributes<32>());
    OP_CK(gemm8_attributes<64>());
    OP_CK(gemm8_attributes<128>());
    OP_CK(cudaFuncSetAttribute(gemm8_pair_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, PairSmem::BYTES));
    OP_CK(cudaFuncSetAttribute(gemm8_pair_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, PairSmem::BYTES));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(h->num_sms / 2 * 2);
    cfg.blockDim = dim3(G8_PAIR_THREADS);
    cfg.dynamicSmemBytes = PairSmem::BYTES;
    OP_CK(cudaOccupancyMaxActiveClusters(&h->pairs, gemm8_pair_kernel<false>, &cfg));
    if (h->pairs < 1) return PRECOND_ECUDA;
    for (int n = 2; n <= 8; n *= 2) {
      cudaLaunchAttribute size = {};
      size.id = cudaLaunchAttributeClusterDimension;
      size.val.clusterDim.x = n;
      size.val.clusterDim.y = size.val.clusterDim.z = 1;
      cfg.gridDim = dim3(n * PLAN_CLUSTERS[n]);
      cfg.blockDim = dim3(512);
      cfg.dynamicSmemBytes = 0;
      cfg.attrs = &size;
      cfg.numAttrs = 1;
      OP_CK(cudaOccupancyMaxActiveClusters(&h->clusters[n], rms_grad_kernel<__nv_bfloat16, true, ROW_CLUSTER>, &cfg));
      h->clusters[n] = std::min(h->clusters[n], PLAN_CLUSTERS[n]);
      if (h->clusters[n] < 1) return PRECOND_ECUDA;
    }
    OP_CK(cudaMalloc(&h->op_err, sizeof(unsigned int)));
    OP_CK(cudaMemset(h->op_err, 0, sizeof(unsigned int)));
    OP_CK(cudaDeviceSynchronize());
    h->op_ready = true;
  }
  return PRECOND_OK;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*k)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;     // common.cuh, wait_for_previous
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// ------------------------------------------------------------------------- norm
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
RowShape row_shape(int64_t cols, int dtype, bool grad, bool vec) {
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
int64_t row_blocks_of(const RowShape& s, int64_t rows, int sm_threads, int sms, const int* clusters) {
  const int64_t resident = std::max(1, sm_threads / (s.threads * s.rows));
  const int64_t most = resident * (s.parts > 1 ? clusters[s.parts] : sms);
  return std::max<int64_t>(1, std::min((rows + s.rows - 1) / s.rows, most));
}
int64_t norm_blocks(const RowShape& s, int64_t rows, int dtype, bool vec, int sms, const int* clusters) {
  return row_blocks_of(s, rows, s.vectors == 2 ? 512 : dtype == PRECOND_F32 ? 384 : vec ? 768 : 512, sms, clusters);
}
int64_t grad_blocks(const RowShape& s, int64_t rows, int dtype, int sms, const int* clusters) {
  return row_blocks_of(s, rows, dtype == PRECOND_F32 ? 384 : 512, sms, clusters);
}

template <typename T, bool VEC>
cudaError_t launch_norm(const RmsNormArgs& a, const RowShape& s, unsigned grid, cudaStream_t st) {
  const dim3 block(s.threads, s.rows);
  const size_t smem = VEC ? 0 : (size_t)s.threads * s.rows / 32 * Scratch<T>::BYTES;    // the warps' exchange buffers
  if (s.parts == 0) return launch(rms_norm_long_kernel<T, VEC>, dim3(grid), block, smem, st, 1, a);
  if (s.parts > 1) return launch(rms_norm_kernel<T, 1, VEC, ROW_CLUSTER>, dim3(grid * s.parts), block, smem, st, s.parts, a);
  if (s.vectors == 2) return launch(rms_norm_kernel<T, 2, true, ROW_BLOCK>, dim3(grid), block, smem, st, 1, a);
  if (s.threads < 32) return launch(rms_norm_kernel<T, 1, true, ROW_PART>, dim3(grid), block, smem, st, 1, a);
  return launch(rms_norm_kernel<T, 1, VEC, ROW_BLOCK>, dim3(grid), block, smem, st, 1, a);
}
template <typename T, bool VEC>
cudaError_t launch_grad(const RmsGradArgs& a, const RowShape& s, unsigned grid, cudaStream_t st) {
  const dim3 block(s.threads, s.rows);
  // the warps' exchange buffers, and then the dw sums of the rows side by side
  const size_t smem = std::max<size_t>(VEC ? 0 : (size_t)s.threads * s.rows / 32 * Scratch<T>::BYTES, s.rows > 1 ? (size_t)s.threads * s.rows * 64 : 0);
  if (s.parts == 0) return launch(rms_grad_long_kernel<T, VEC>, dim3(grid), block, smem, st, 1, a);
  if (s.parts > 1) return launch(rms_grad_kernel<T, VEC, ROW_CLUSTER>, dim3(grid * s.parts), block, smem, st, s.parts, a);
  if (s.threads < 32) return launch(rms_grad_kernel<T, true, ROW_PART>, dim3(grid), block, smem, st, 1, a);
  return launch(rms_grad_kernel<T, VEC, ROW_BLOCK>, dim3(grid), block, smem, st, 1, a);
}

// ------------------------------------------------------------------------- distillation
// Blocks of a row: as many as hold it in registers, and more where rows are few, each with at least 8192 logits.
int distill_parts(int64_t rows, int64_t vocab, int dtype) {
  const int64_t sz = (int64_t)size_of(dtype), capacity = 8 * DISTILL_THREADS * 16 / sz;
  int parts = 1;
  while (parts < 8 && (((vocab + parts - 1) / parts + 63) / 64 * 64 > capacity ||
                       (rows * parts < 2 * PLAN_SMS && vocab / (parts * 2) >= 8192)))
    parts *= 2;
  return parts;
}
// Whether the candidates have a kernel of their own: with many rows or blocks, one more launch costs less than warps
// that wait for them.  (2000 x 131072 bf16 with 128 of them, 8000 blocks: 191 us, together 248; 1900 x 32000 fp32 with
// 64, 86 and 89; 1000 x 32000 fp32, 2000 blocks: 51.8 and 51.3, bf16 32.6 and 27.9; 500 x 32000 fp32 32.0 and 28.3.  Many
// candidates over a large vocabulary would part earlier: 800 x 131072, 3200 blocks: 87 and 103.)
bool distill_split(int64_t rows, int64_t vocab, int dtype) {
  return rows >= 12 * PLAN_SMS || rows * distill_parts(rows, vocab, dtype) >= 24 * PLAN_SMS;
}
// ------------------------------------------------------------------------- product
int encode8(Handle* h, CUtensorMap* map, const void* q, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {(cuuint32_t)G8_BK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = h->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fprintf(stderr, "libprecond: cuTensorMapEncodeTiled failed (%d)\n", (int)r);
    return PRECOND_ECUDA;
  }
  return PRECOND_OK;
}

// The scales of `blocks` x 128 rows a group as rows of 512 bytes; boxes of `box` of them.
int encode_scales(Handle* h, CUtensorMap* map, const uint8_t* s, int64_t blocks, int groups, int box_rows) {
  cuuint64_t dims[2] = {128, (cuuint64_t)(blocks * groups)};
  cuuint64_t strides[1] = {512};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = h->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(s), dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fprintf(stderr, "libprecond: cuTensorMapEncodeTiled failed (%d)\n", (int)r);
    return PRECOND_ECUDA;
  }
  return PRECOND_OK;
}

int launch_pair(Handle* h, const void* A, int64_t lda, const void* B, int64_t ldb, const Gemm8Args& g, cudaStream_t st) {
  PairMaps maps;
  const int groups = q8_groups(g.K);
  int rc;
  if ((rc = encode8(h, &maps.a, A, g.M, g.K, lda, 128)) || (rc = encode8(h, &maps.b, B, g.N, g.K, ldb, 128)) ||
      (rc = encode_scales(h, &maps.sa, g.sa, g.sa_rb, groups, 1)) || (rc = encode_scales(h, &maps.sb, g.sb, g.sb_rb, groups, 2)))
    return rc;
  const int64_t tiles = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(tiles, h->pairs);
  auto k = g.c_bf16 ? gemm8_pair_kernel<false> : gemm8_pair_kernel<true>;
  OP_CK(launch(k, dim3(grid), dim3(G8_PAIR_THREADS), PairSmem::BYTES, st, 1, maps, g));
  return PRECOND_OK;
}

template <int BN>
cudaError_t launch_gemm8(const CUtensorMap& ma, const CUtensorMap& mb, const Gemm8Args& g, int64_t tiles, int parts, int sms,
                         cudaStream_t st) {
  const unsigned grid = parts > 1 ? (unsigned)(tiles * parts) : (unsigned)std::min<int64_t>(tiles, sms * Gemm8Smem<BN>::CTAS);
  auto k = g.c_bf16 ? gemm8_kernel<BN, false> : gemm8_kernel<BN, true>;
  return launch(k, dim3(grid), dim3(G8_THREADS), Gemm8Smem<BN>::BYTES, st, parts, ma, mb, g);
}

}  // namespace

extern "C" {

int precond_rms_norm(precond_t ph, const void* x, const void* residual, const void* weight, int dtype, int weight_dtype,
                     int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, float eps, void* total, int64_t ldt, void* y,
                     int64_t ldy, void* q, int64_t ldq, uint8_t* scale, float* rstd, void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !float_type(dtype) || !float_type(weight_dtype) || !side(rows) || !side(cols) || !(eps > 0.f)) return PRECOND_EINVAL;
  const size_t sz = size_of(dtype);
  if (!matrix(x, rows, cols, ldx, dtype) || !matrix(weight, 1, cols, cols, weight_dtype) || !aligned(rstd, 4)) return PRECOND_EINVAL;
  if ((residual != nullptr) != (total != nullptr)) return PRECOND_EINVAL;
  if (residual && (!matrix(residual, rows, cols, ldr, dtype) || !matrix(total, rows, cols, ldt, dtype))) return PRECOND_EINVAL;
  if (y && !matrix(y, rows, cols, ldy, dtype)) return PRECOND_EINVAL;
  if ((q != nullptr) != (scale != nullptr) || (q && !matrix8(q, ldq, scale, rows, cols))) return PRECOND_EINVAL;
  if (rows && cols && !total && !y && !q && !rstd) return PRECOND_EINVAL;
  // outputs may not overlap anything, but for `total` over x or residual, element for element
  const Range in[3] = {range(x, rows, ldx, cols, sz), range(residual, rows, ldr, cols, sz),
                       range(weight, 1, 0, cols, size_of(weight_dtype))};
  const Range out[5] = {range(total, rows, ldt, cols, sz), range(y, rows, ldy, cols, sz), range(q, rows, ldq, cols, 1),
                        q ? scale_range(scale, rows, cols) : NOWHERE, range(rstd, 1, 0, rows, 4)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 3; ++j) {
      const bool same = i == 0 && ((j == 0 && total == x && ldt == ldx) || (j == 1 && total == residual && ldt == ldr));
      if (!same && overlap(out[i], in[j])) return PRECOND_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return PRECOND_EINVAL;
  }
  if (h->device < 0) return PRECOND_ENODEV;
  if (rows == 0 || cols == 0) return PRECOND_OK;
  int rc = prepare(h);
  if (rc) return rc;
  RmsNormArgs a = {x, residual, weight, total, y, (uint8_t*)q, scale, rstd, ldx, ldr, ldt, ldy, ldq, (int)rows, (int)cols, eps,
                   weight_dtype == PRECOND_BF16};
  const bool vec = sector_rows(x, ldx, dtype) && sector_rows(residual, ldr, dtype) && sector_rows(total, ldt, dtype) &&
                   sector_rows(y, ldy, dtype);
  const RowShape s = row_shape(cols, dtype, false, vec);
  const unsigned grid = (unsigned)norm_blocks(s, q ? q8_row_blocks(rows) * 128 : rows, dtype, vec, h->num_sms, h->clusters);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PRECOND_BF16)
    OP_CK((vec ? launch_norm<__nv_bfloat16, true>(a, s, grid, st) : launch_norm<__nv_bfloat16, false>(a, s, grid, st)));
  else
    OP_CK((vec ? launch_norm<float, true>(a, s, grid, st) : launch_norm<float, false>(a, s, grid, st)));
  ++h->launches;
  return PRECOND_OK;
}

int64_t precond_rms_norm_grad_workspace(int64_t rows, int64_t cols) {
  if (!side(rows) || !side(cols)) return -1;
  if (rows == 0 || cols == 0) return 0;
  // of either type; rows in parts of a warp, and clusters that do not fit, only make fewer
  int64_t blocks = 0;
  for (const int dtype : {PRECOND_BF16, PRECOND_F32})
    blocks = std::max(blocks, grad_blocks(row_shape(cols, dtype, true, false), rows, dtype, PLAN_SMS, PLAN_CLUSTERS));
  return blocks * cols * 4;
}

int precond_rms_norm_grad(precond_t ph, const void* dy, const void* x, const void* weight, const float* rstd,
                          const void* dresidual, int dtype, int weight_dtype, int64_t rows, int64_t cols, int64_t lddy,
                          int64_t ldx, int64_t lddr, void* dx, int64_t lddx, float* dw, void* workspace,
                          int64_t workspace_bytes, void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !float_type(dtype) || !float_type(weight_dtype) || !side(rows) || !side(cols)) return PRECOND_EINVAL;
  const size_t sz = size_of(dtype);
  if (!matrix(dy, rows, cols, lddy, dtype) || !matrix(x, rows, cols, ldx, dtype) || !matrix(dx, rows, cols, lddx, dtype) ||
      !matrix(weight, 1, cols, cols, weight_dtype) || !matrix(rstd, 1, rows, rows, PRECOND_F32) ||
      !matrix(dw, 1, cols, cols, PRECOND_F32) || (dresidual && !matrix(dresidual, rows, cols, lddr, dtype)))
    return PRECOND_EINVAL;
  const int64_t need = precond_rms_norm_grad_workspace(rows, cols);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return PRECOND_EINVAL;
  const Range in[5] = {range(dy, rows, lddy, cols, sz), range(dresidual, rows, lddr, cols, sz), range(x, rows, ldx, cols, sz),
                       range(weight, 1, 0, cols, size_of(weight_dtype)), range(rstd, 1, 0, rows, 4)};
  const Range out[3] = {range(dx, rows, lddx, cols, sz), range(dw, 1, 0, cols, 4), range(workspace, 1, 0, need, 1)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j) {
      // dx may lie over dy, dresidual or x, element for element, where a row is surely read once
      const bool same = i == 0 && cols <= GRAD_IN_PLACE &&
                        ((j == 0 && dx == dy && lddx == lddy) || (j == 1 && dx == dresidual && lddx == lddr) ||
                         (j == 2 && dx == x && lddx == ldx));
      if (!same && overlap(out[i], in[j])) return PRECOND_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return PRECOND_EINVAL;
  }
  if (h->device < 0) return PRECOND_ENODEV;
  if (cols == 0) return PRECOND_OK;
  int rc = prepare(h);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {
    OP_CK(cudaMemsetAsync(dw, 0, cols * 4, st));
    return PRECOND_OK;
  }
  RmsGradArgs a = {dy, x, dresidual, weight, rstd, dx, (float*)workspace, lddy, ldx, lddr, lddx, (int)rows, (int)cols,
                   weight_dtype == PRECOND_BF16};
  const bool vec = sector_rows(dy, lddy, dtype) && sector_rows(x, ldx, dtype) && sector_rows(dresidual, lddr, dtype) &&
                   sector_rows(dx, lddx, dtype);
  const RowShape s = row_shape(cols, dtype, true, vec);
  const unsigned grid = (unsigned)grad_blocks(s, rows, dtype, std::min(h->num_sms, PLAN_SMS), h->clusters);
  if (dtype == PRECOND_BF16)
    OP_CK((vec ? launch_grad<__nv_bfloat16, true>(a, s, grid, st) : launch_grad<__nv_bfloat16, false>(a, s, grid, st)));
  else
    OP_CK((vec ? launch_grad<float, true>(a, s, grid, st) : launch_grad<float, false>(a, s, grid, st)));
  OP_CK(launch(rms_dw_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(32, 32), 0, st, 1, (const float*)workspace,
               (int)grid, cols, dw));
  h->launches += 2;
  return PRECOND_OK;
}

int precond_quantize8(precond_t ph, const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const uint8_t* x_scale,
                      int block, void* q, int64_t ldq, uint8_t* scale, void* qt, int64_t ldqt, uint8_t* scale_t, void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !side(rows) || !side(cols) || (block != PRECOND_BLOCK_ROW && block != PRECOND_BLOCK_TILE)) return PRECOND_EINVAL;
  if (dtype == PRECOND_E4M3) {
    if (!matrix8(x, ldx, x_scale, rows, cols)) return PRECOND_EINVAL;
  } else if (!float_type(dtype) || x_scale || !matrix(x, rows, cols, ldx, dtype)) {
    return PRECOND_EINVAL;
  }
  if ((q != nullptr) != (scale != nullptr) || (qt != nullptr) != (scale_t != nullptr) || (rows && cols && !q && !qt)) return PRECOND_EINVAL;
  if ((q && !matrix8(q, ldq, scale, rows, cols)) || (qt && !matrix8(qt, ldqt, scale_t, cols, rows))) return PRECOND_EINVAL;
  const Range in[2] = {range(x, rows, ldx, cols, size_of(dtype)),
                       x_scale ? scale_range(x_scale, rows, cols) : NOWHERE};
  const Range out[4] = {range(q, rows, ldq, cols, 1), q ? scale_range(scale, rows, cols) : NOWHERE,
                        range(qt, cols, ldqt, rows, 1), qt ? scale_range(scale_t, cols, rows) : NOWHERE};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 2; ++j)
      if (overlap(out[i], in[j])) return PRECOND_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return PRECOND_EINVAL;
  }
  const int64_t tiles = q8_row_blocks(rows) * q8_row_blocks(cols);
  if (tiles > INT32_MAX) return PRECOND_EINVAL;
  if (h->device < 0) return PRECOND_ENODEV;
  if (rows == 0 || cols == 0) return PRECOND_OK;
  int rc = prepare(h);
  if (rc) return rc;
  Quant8Args a = {x, ldx, x_scale, (int)rows, (int)cols, block == PRECOND_BLOCK_TILE, (uint8_t*)q, ldq, scale, (uint8_t*)qt, ldqt, scale_t};
  // 8 columns in one load: 16 bytes of bf16, 32 of fp32
  const int64_t step = 8 * (int64_t)size_of(dtype);
  const bool vec = aligned(x, step) && ldx * (int64_t)size_of(dtype) % step == 0;
  auto k = dtype == PRECOND_E4M3   ? quantize8_kernel<QIN_E4M3, true>
           : dtype == PRECOND_BF16 ? (vec ? quantize8_kernel<QIN_BF16, true> : quantize8_kernel<QIN_BF16, false>)
                                   : (vec ? quantize8_kernel<QIN_F32, true> : quantize8_kernel<QIN_F32, false>);
  OP_CK(launch(k, dim3((unsigned)tiles), dim3(256), 0, (cudaStream_t)stream, 1, a));
  ++h->launches;
  return PRECOND_OK;
}

int precond_gemm8(precond_t ph, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const uint8_t* scale_a,
                  const void* B, int64_t ldb, const uint8_t* scale_b, void* C, int64_t ldc, int c_dtype, int accumulate,
                  void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !side(M) || !side(N) || !side(K) || !float_type(c_dtype)) return PRECOND_EINVAL;
  if (accumulate && c_dtype != PRECOND_F32) return PRECOND_EINVAL;
  if (!matrix8(A, lda, scale_a, M, K) || !matrix8(B, ldb, scale_b, N, K) || !matrix(C, M, N, ldc, c_dtype)) return PRECOND_EINVAL;
  const Range in[4] = {range(A, M, lda, K, 1), range(B, N, ldb, K, 1),
                       M && K ? scale_range(scale_a, M, K) : NOWHERE,
                       N && K ? scale_range(scale_b, N, K) : NOWHERE};
  const Range out = range(C, M, ldc, N, size_of(c_dtype));
  for (const Range& r : in)
    if (overlap(out, r)) return PRECOND_EINVAL;
  if (h->device < 0) return PRECOND_ENODEV;
  if (M == 0 || N == 0) return PRECOND_OK;
  int rc = prepare(h);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;

  // The MMA's rows are always 128 a tile, its columns 16 to 128.  A side of at most 64
  // goes to the columns (a few tokens against a weight: the weight's rows fill the tile
  // and its bytes, which bound the call, are read once).
  const bool swap = M <= 64 && M < N;
  Gemm8Args g = {swap ? N : M, swap ? M : N, K, scale_a, q8_row_blocks(M), scale_b, q8_row_blocks(N), C, ldc,
                 c_dtype == PRECOND_BF16, accumulate, aligned(C, 32) && ldc * (int64_t)size_of(c_dtype) % 32 == 0,
                 aligned(C, 4 * size_of(c_dtype)) && ldc % 4 == 0, swap, h->op_err};
  if (swap) {
    std::swap(A, B);
    std::swap(lda, ldb);
    std::swap(g.sa, g.sb);
    std::swap(g.sa_rb, g.sb_rb);
  }
  const int bn = g.N <= 16 ? 16 : g.N <= 32 ? 32 : g.N <= 64 ? 64 : 128;
  const int64_t tiles = ((g.M + G8_BM - 1) / G8_BM) * ((g.N + bn - 1) / bn);
  if (tiles > INT32_MAX) return PRECOND_EINVAL;
  // Few tiles: a cluster of up to 8 CTAs shares each, a stretch of whole scale groups of K each.
  const int blocks = (int)((K + G8_BK - 1) / G8_BK), groups = q8_groups(K);
  int parts = 1;
  const int places = h->num_sms * (bn <= 32 ? 2 : 1);
  while (parts < 8 && tiles * parts * 2 <= places && parts * 2 <= groups) parts *= 2;
  // Pairs of CTAs where they are expected to end first: a 256 x 256 tile's block of K takes a pair 0.30 us, a 128 x 128
  // tile's a CTA 0.25 us; results leave beside the next tile's products, in the times below (as g8_store32 writes
  // them: rows of whole sectors, 4 elements at a time, single ones; bf16, fp32); joining stretches takes 1.5 us more.
  // (Measured: 6734 x 832 x 468 accumulated 17.3 us in pairs, 11.6 alone; 2048^3 to bf16 11.1 and 14.1.)
  static const double results_us[2][3][2] = {{{1.1, 1.3}, {2.0, 2.4}, {3.0, 4.0}}, {{2.5, 3.5}, {4.0, 6.0}, {4.5, 8.0}}};
  const int how = g.sectors && !accumulate ? 0 : g.quads ? 1 : 2;
  auto expected = [&](int pair, double products, int64_t waves) {
    const double results = results_us[pair][how][!g.c_bf16];
    return products + (double)(waves - 1) * std::max(products, results) + results;
  };
  const int64_t pair_tiles = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  const double pair_us = expected(1, 0.30 * blocks, (pair_tiles + h->pairs - 1) / h->pairs);
  const double lone_us = expected(0, 0.25 * ((groups + parts - 1) / parts * 4), (tiles * parts + h->num_sms - 1) / h->num_sms) + (parts > 1 ? 1.5 : 0.0);
  if (bn == 128 && K > 0 && pair_us <= lone_us) {
    if ((rc = launch_pair(h, A, lda, B, ldb, g, st))) return rc;
    ++h->launches;
    return PRECOND_OK;
  }
  CUtensorMap ma, mb;
  memset(&ma, 0, sizeof(ma));
  memset(&mb, 0, sizeof(mb));
  if (K > 0 && ((rc = encode8(h, &ma, A, g.M, K, lda, G8_BM)) || (rc = encode8(h, &mb, B, g.N, K, ldb, bn)))) return rc;
  cudaError_t e = cudaSuccess;
  switch (bn) {
    case 16: e = launch_gemm8<16>(ma, mb, g, tiles, parts, h->num_sms, st); break;
    case 32: e = launch_gemm8<32>(ma, mb, g, tiles, parts, h->num_sms, st); break;
    case 64: e = launch_gemm8<64>(ma, mb, g, tiles, parts, h->num_sms, st); break;
    default: e = launch_gemm8<128>(ma, mb, g, tiles, parts, h->num_sms, st); break;
  }
  OP_CK(e);
  ++h->launches;
  return PRECOND_OK;
}

int precond_gemm8_status(precond_t ph, void* stream) {
  Handle* h = as_handle(ph);
  if (!h) return PRECOND_EINVAL;
  if (h->device < 0) return PRECOND_ENODEV;
  int rc = prepare(h);
  if (rc) return rc;
  unsigned int word = 0;
  cudaStream_t st = (cudaStream_t)stream;
  OP_CK(cudaMemcpyAsync(&word, h->op_err, sizeof(word), cudaMemcpyDeviceToHost, st));
  OP_CK(cudaMemsetAsync(h->op_err, 0, sizeof(word), st));
  OP_CK(cudaStreamSynchronize(st));
  return word ? PRECOND_ECUDA : PRECOND_OK;
}

int64_t precond_distill_workspace(int64_t rows, int64_t vocab, int top, int dtype, int in_place) {
  if (!side(rows) || !side(vocab) || vocab < 1 || top < 1 || top > DISTILL_MAX_TOP || !float_type(dtype)) return -1;
  if (!distill_split(rows, vocab, dtype)) return 0;
  return rows * 8 + (in_place ? rows * top * 4 : 0);
}

int precond_distill(precond_t ph, const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ldz, const void* ids,
                    int id_bits, int64_t ldi, const void* teacher, int teacher_dtype, int64_t ldt, int top,
                    const float* weight, float temperature, float* loss, void* dlogits, int64_t lddz, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !float_type(dtype) || !float_type(teacher_dtype) || !side(rows) || !side(vocab) || vocab < 1) return PRECOND_EINVAL;
  if ((id_bits != 32 && id_bits != 64) || top < 1 || top > DISTILL_MAX_TOP || !(temperature >= 1e-18f && temperature <= 1e18f))
    return PRECOND_EINVAL;               // temperature^2 and log2(e) / temperature are fp32 numbers
  const size_t sz = size_of(dtype);
  if (!matrix(logits, rows, vocab, ldz, dtype) || !matrix(teacher, rows, top, ldt, teacher_dtype) ||
      !matrix(loss, 1, rows, rows, PRECOND_F32) || (dlogits && !matrix(dlogits, rows, vocab, lddz, dtype)) ||
      (weight && !aligned(weight, 4)) || ldi < top || ldi > MAX_SIDE || (rows && (!ids || !aligned(ids, id_bits / 8))))
    return PRECOND_EINVAL;
  const int64_t need = precond_distill_workspace(rows, vocab, top, dtype, dlogits == logits);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return PRECOND_EINVAL;
  const Range in[4] = {range(logits, rows, ldz, vocab, sz), range(ids, rows, ldi, top, id_bits / 8),
                       range(teacher, rows, ldt, top, size_of(teacher_dtype)), range(weight, 1, 0, rows, 4)};
  const Range out[3] = {range(dlogits, rows, lddz, vocab, sz), range(loss, 1, 0, rows, 4), range(workspace, 1, 0, need, 1)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 4; ++j) {
      const bool same = i == 0 && j == 0 && dlogits == logits && lddz == ldz;
      if (!same && overlap(out[i], in[j])) return PRECOND_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return PRECOND_EINVAL;
  }
  if (rows > (int64_t)INT32_MAX / 8 || rows * top / 256 > INT32_MAX) return PRECOND_EINVAL;
  if (h->device < 0) return PRECOND_ENODEV;
  if (rows == 0) return PRECOND_OK;
  int rc = prepare(h);
  if (rc) return rc;
  const bool bf16 = dtype == PRECOND_BF16, split = distill_split(rows, vocab, dtype);
  cudaStream_t st = (cudaStream_t)stream;
  DistillArgs a = {logits, ldz, ids, ldi, id_bits == 64, teacher, ldt, teacher_dtype == PRECOND_BF16, weight, loss, dlogits, lddz,
                   rows, vocab, top, temperature, (float2*)workspace, nullptr};
  const int parts = distill_parts(rows, vocab, dtype);
  const int64_t vecs = ((vocab + parts - 1) / parts + 63) / 64 * 64 * (int64_t)sz / 16;
  // Vectors a thread: one block after another on an SM hides nothing, so a block has as few threads as hold its part, 64
  // at least (8192 x 8000 bf16: 53 us, with 512 threads of 2 vectors 77).
  int i = 0;
  if (vecs <= 8 * DISTILL_THREADS)
    for (i = 1; i < 4 && vecs >= 128 << (i - 1);) ++i;
  const int nv = i ? 1 << (i - 1) : 0;
  const int threads = nv == 0 ? DISTILL_THREADS : (int)std::max<int64_t>(64, ((vecs + nv - 1) / nv + 31) / 32 * 32);
  if (split && dlogits == logits) {
    a.kept = (float*)((char*)workspace + rows * 8);
    OP_CK(launch(bf16 ? distill_keep_kernel<__nv_bfloat16> : distill_keep_kernel<float>, dim3((unsigned)((rows * top + 255) / 256)),
                 dim3(256), 0, st, 1, a));
    ++h->launches;
  }
  const int sums = parts * threads / 32;
  OP_CK(launch((split ? distill_split_kernels : distill_fused_kernels)[bf16][i], dim3((unsigned)(rows * parts)),
               dim3(threads + (split ? 0 : 32)), split ? sums * 8 : DistillShared::bytes(top, sums), st, parts, a));
  ++h->launches;
  if (split) {
    // a warp a row, eight to a block where their candidates fit
    const int each = DistillShared::bytes(top, 0), warps = std::max(1, std::min(8, (48 << 10) / each));
    const int in = top <= 128 ? 0 : top <= DISTILL_FEW ? 1 : 2;  // registers of 4 or 8 a lane, shared memory
    auto k = distill_candidates_kernels[bf16][in];
    OP_CK(launch(k, dim3((unsigned)((rows + warps - 1) / warps)), dim3(32 * warps), (size_t)each * warps, st, 1, a));
    ++h->launches;
  }
  return PRECOND_OK;
}

}  // extern "C"
