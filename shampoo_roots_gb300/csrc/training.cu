// Host side of the operators that train a policy (include/precond.h): layer norm
// and its gradients, the clipped policy loss, the norm of a list of gradients and
// their clipping.  Arguments are checked here, before anything is enqueued;
// kernels go to the caller's stream and use no memory but the caller's.

#include <cmath>
#include <cstring>

#include <vector>

#include "clip.cuh"
#include "host.h"
#include "layer_norm.cuh"
#include "policy.cuh"

using namespace precond;

namespace {

constexpr int64_t LAYER_IN_PLACE = 32768;           // columns up to which every shape of row is read once

// ------------------------------------------------------------------------- layer norm
template <typename T, bool VEC>
struct LayerKernels {
  typedef void (*Norm)(LayerNormArgs);
  typedef void (*Grad)(LayerGradArgs);
  static Norm norm(const RowShape& s) {
    if (s.parts == 0) return layer_norm_long_kernel<T, VEC>;
    if (s.parts > 1) return layer_norm_kernel<T, 1, VEC, ROW_CLUSTER>;
    if (VEC && s.vectors == 2) return layer_norm_kernel<T, 2, true, ROW_BLOCK>;
    if (VEC && s.threads < 32) return layer_norm_kernel<T, 1, true, ROW_PART>;
    return layer_norm_kernel<T, 1, VEC, ROW_BLOCK>;
  }
  static Grad grad(const RowShape& s) {
    if (s.parts == 0) return layer_grad_long_kernel<T, VEC>;
    if (s.parts > 1) return layer_grad_kernel<T, VEC, ROW_CLUSTER>;
    if (VEC && s.threads < 32) return layer_grad_kernel<T, true, ROW_PART>;
    return layer_grad_kernel<T, VEC, ROW_BLOCK>;
  }
  static size_t scratch(const RowShape& s) { return VEC ? 0 : (size_t)s.threads * s.rows / 32 * Scratch<T>::BYTES; }
  // the table of w and b, the warps' exchange buffers
  static size_t norm_bytes(const RowShape& s) { return (s.parts ? (size_t)s.threads * s.vectors * 128 : 0) + scratch(s); }
  // the table of w, the warps' exchange buffers; then the dw and db sums of the rows side by side
  static size_t grad_bytes(const RowShape& s) {
    return std::max((s.parts ? (size_t)s.threads * 64 : 0) + scratch(s), s.parts == 1 ? (size_t)s.threads * s.rows * 128 : 0);
  }
  static cudaError_t attributes() {
    // one of each kernel; the shapes decide how much they ask for
    const RowShape one[] = {{384, 1, 1, 1}, {512, 1, 2, 1}, {16, 8, 1, 1}, {384, 1, 1, 2}};
    for (const RowShape& s : one) {
      cudaError_t e = cudaFuncSetAttribute(norm(s), cudaFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(grad(s), cudaFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
};
int64_t layer_norm_blocks(const RowShape& s, int64_t rows, int dtype, bool vec, int sms, const int* clusters) {
  return row_blocks_of(s, rows, s.vectors == 2 ? 512 : dtype == PRECOND_F32 ? 384 : vec ? 768 : 512, sms, clusters);
}
template <typename T, bool VEC>
cudaError_t launch_layer_norm(const LayerNormArgs& a, const RowShape& s, unsigned grid, cudaStream_t st) {
  typedef LayerKernels<T, VEC> K;
  return launch(K::norm(s), dim3(grid * std::max(1, s.parts)), dim3(s.threads, s.rows), K::norm_bytes(s), st, std::max(1, s.parts), a);
}
template <typename T, bool VEC>
cudaError_t launch_layer_grad(const LayerGradArgs& a, const RowShape& s, unsigned grid, cudaStream_t st) {
  typedef LayerKernels<T, VEC> K;
  const int cluster = a.dw ? (int)grid : std::max(1, s.parts);
  return launch(K::grad(s), dim3(a.dw ? grid : grid * cluster), dim3(s.threads, s.rows), K::grad_bytes(s), st, cluster, a);
}

// Rows through shared memory: threads of a row, rows of a block, rows of each in the ring (0: not this way).  For rows of
// more than 256 columns, whole 16-byte vectors, enough of them that a group has its second one.  (Norm of 8192 x 6144
// bf16 56 us, with the next row in registers 63; of 20000 x 1024 27 and 38; gradients of 16384 x 4096 92 and 97.)
// Vectors a thread, of a norm: one where rows are short, and, with a residual, where whole warps of them fill the block's 768
// threads (bf16 to 8 bits, one and two: 8192 x 6144 56 and 63 us, 8192 x 4096 39 and 43, 4000 x 12288 58 and 61; y kept 72 and
// 70, 48 and 49, 68 and 70; without a residual, which leaves room for more stages, 52 and 49, 36 and 34, 53 and 55; a last warp
// half empty, 8548 x 5888, 65 and 60).  Else two, or four for wide rows, whose groups are more (one, two and four: 6000 x 8192
// 65, 59 and 57, 4000 x 12288 without a residual 53, 55 and 50).  fp32: one up to 768 threads (10000 x 4096 without a residual,
// y kept, one and two 53 and 60, to 8 bits 46 and 43).
constexpr int STREAM_BYTES = 225 << 10;
typedef void (*StreamNorm)(LayerNormArgs, int);
typedef void (*StreamGrad)(LayerGradArgs, int);
const StreamNorm stream_norm_kernels[2][3] = {                   // 1, 2, 4 vectors a thread
    {layer_norm_stream_kernel<float, 1>, layer_norm_stream_kernel<float, 2>, nullptr},
    {layer_norm_stream_kernel<__nv_bfloat16, 1>, layer_norm_stream_kernel<__nv_bfloat16, 2>, layer_norm_stream_kernel<__nv_bfloat16, 4>}};
const StreamGrad stream_grad_kernels[2] = {layer_grad_stream_kernel<float>, layer_grad_stream_kernel<__nv_bfloat16>};
struct StreamShape { int threads, rows, vectors, stages; size_t bytes; };
StreamShape stream_shape(int64_t cols, int dtype, int inputs, bool grad, int64_t rows, int sms) {
  StreamShape s = {0, 0, 1, 0, 0};
  const int64_t n = (cols + 15) / 16, row = cols * (int64_t)size_of(dtype);
  if (n <= 16 || row % 16 || n > (grad ? 512 : 1024)) return s;
  if (!grad && dtype == PRECOND_F32 && n > 768) s.vectors = 2;
  const bool fills = inputs == 2 && n % 32 == 0 && STREAM_THREADS[1] % n == 0;
  if (!grad && dtype == PRECOND_BF16 && n > 200 && !fills) s.vectors = n > 512 ? 4 : 2;
  const int most = grad ? 512 : STREAM_THREADS[s.vectors];
  s.threads = (int)((n + 32 * s.vectors - 1) / (32 * s.vectors) * 32);
  s.rows = std::max(1, std::min(most / s.threads, s.threads > 32 ? 15 : 16));
  if (rows <= (int64_t)s.rows * sms) return s;
  const size_t table = (size_t)s.threads * (grad ? 64 : s.vectors * 128);
  while (s.stages < 8 && table + s.rows * RowRing::size(s.stages + 1, inputs, (int)row) <= STREAM_BYTES) ++s.stages;
  if (s.stages < 2) s.stages = 0;
  s.bytes = table + std::max(s.rows * RowRing::size(s.stages, inputs, (int)row), grad && s.rows > 1 ? (size_t)s.threads * s.rows * 128 : 0);
  return s;
}

// ------------------------------------------------------------------------- policy loss
typedef void (*PolicyKernel)(PolicyArgs);
const PolicyKernel policy_kernels[2][2] = {{policy_kernel<float, false>, policy_kernel<float, true>},
                                           {policy_kernel<__nv_bfloat16, false>, policy_kernel<__nv_bfloat16, true>}};
// Bytes of a row that a warp takes in registers: 1, 2, 4 or 8 vectors a lane (8192 x 1000 bf16 9.9 us, by blocks 18.3; of rows
// of 8 KB, with 16 vectors, an SM holds half the warps: 8192 x 4000 33 us, by blocks 31).  From 2 KB on shared memory is
// quicker with a gradient and slower without (8192 x 1500 bf16 15.6 and 12.6 us, scoring 9.0 and 9.2; 30000 x 1500 41 and 35,
// scoring 26 and 31); the rule does not ask which, so that a token's log probability is the same in both.
constexpr int64_t POLICY_WARP = 4096;
const PolicyKernel policy_warp_kernels[2][4] = {
    {policy_warp_kernel<float, 1>, policy_warp_kernel<float, 2>, policy_warp_kernel<float, 4>, policy_warp_kernel<float, 8>},
    {policy_warp_kernel<__nv_bfloat16, 1>, policy_warp_kernel<__nv_bfloat16, 2>, policy_warp_kernel<__nv_bfloat16, 4>,
     policy_warp_kernel<__nv_bfloat16, 8>}};
// Bytes of a row that a warp takes in shared memory, where there are more rows than SMs: half as many for fewer rows than 4
// to an SM, whose warps are too few to hide each other's waits (by a block of several warps: 8192 x 2500 bf16 26.2 us, by a
// warp 16.0; 8192 x 4000 31.4 and 23.4; 8192 x 10000 53.7 and 51.4, scoring 35.5 and 30.4; 8192 x 16000 78.6 and 82.6; 500 x
// 4000 6.8 and 5.2, 500 x 8000 7.1 and 7.5; four warps to a block, or warps that go from row to row: 8192 x 8000 46 and 49
// us, by one 42).
constexpr int64_t POLICY_ROW = 24 << 10;
const PolicyKernel policy_row_kernels[2] = {policy_row_kernel<float>, policy_row_kernel<__nv_bfloat16>};
const PolicyKernel policy_few_kernels[2][4] = {
    {policy_few_kernel<float, 1>, policy_few_kernel<float, 2>, policy_few_kernel<float, 4>, policy_few_kernel<float, 8>},
    {policy_few_kernel<__nv_bfloat16, 1>, policy_few_kernel<__nv_bfloat16, 2>, policy_few_kernel<__nv_bfloat16, 4>,
     policy_few_kernel<__nv_bfloat16, 8>}};
// Blocks of a row, threads of a block, bytes of a part in shared memory.  A part takes at most what lets an SM hold three
// blocks (8192 x 131072 bf16 by parts of 64 KB 671 us, of 32 KB 707, of 128 KB 893; 1900 x 151936 by 74 KB 188, by 37 KB
// 199); a few rows take more blocks, each with at least 8192 logits.  Threads have 192 bytes each, up to 256 of them (8192 x
// 8000 bf16, 16 KB: 96 threads 45 us, 128 47, 256 62, 512 99; 2999 x 50001: 256 threads 98 us, 512 118).  Blocks alone on
// their SMs keep up to 64 KB in registers (24 x 50001 bf16 scored: 3.2 us on the device, by shared memory 4.2); where there
// are more blocks than SMs it goes either way (300 x 10000 fp32 7.4 and 8.8 us, 100 x 30000 11.5 and 9.7).
struct PolicyShape { PolicyKernel kernel; int parts, threads, bytes; };
PolicyShape policy_shape(int64_t rows, int64_t vocab, int dtype) {
  const int64_t sz = (int64_t)size_of(dtype), third = 76288;
  const bool bf16 = dtype == PRECOND_BF16;
  int parts = 1;
  auto bytes = [&]() { return ((vocab + parts - 1) / parts + 63) / 64 * 64 * sz; };
  while (parts < 8 && (bytes() > third || (rows * parts < 2 * PLAN_SMS && vocab / (parts * 2) >= 8192))) parts *= 2;
  const int64_t each = bytes(), vectors = each / 16;
  if (rows * parts <= PLAN_SMS && vectors <= 8 * POLICY_THREADS) {
    int i = 0;
    while (vectors > POLICY_THREADS << i) ++i;
    return {policy_few_kernels[bf16][i], parts, (int)std::max<int64_t>(64, ((vectors + (1 << i) - 1) / (1 << i) + 31) / 32 * 32), 0};
  }
  const int threads = (int)std::min<int64_t>(256, (each / 192 + 31) / 32 * 32);
  return each <= POLICY_PART ? PolicyShape{policy_kernels[bf16][1], parts, threads, (int)each}
                             : PolicyShape{policy_kernels[bf16][0], parts, threads, 0};
}

// ------------------------------------------------------------------------- lists of tensors
// Tensors of a launch: tables of 0.6, 2.5, 10 and 28 KB of parameters.
constexpr int CLIP_SIZES[4] = {32, 128, 512, 1400};
constexpr int CLIP_BLOCKS = 2 * PLAN_SMS;

// A short list has at most CLIP_SHORT tensors: the larger tables need no kernel for it.
constexpr int CLIP_SHORT = 128;                      // pieces of a list that one cluster takes (512 KB: two launches 6.7 us, one 5.2; 128 KB 6.7 and 3.8)
struct ClipKernels { const void *norm, *scale, *one; };
template <int MAX>
ClipKernels clip_kernels() {
  ClipKernels k = {(const void*)clip_norm_kernel<MAX>, (const void*)clip_scale_kernel<MAX>, nullptr};
  if constexpr (MAX <= CLIP_SHORT) k.one = (const void*)clip_short_kernel<MAX>;
  return k;
}
const ClipKernels clip_of[4] = {clip_kernels<32>(), clip_kernels<128>(), clip_kernels<512>(), clip_kernels<1400>()};

// Tensors and the tables of their launches.
struct List {
  std::vector<ClipTensor> tensors;                   // without the empty ones
  std::vector<Range> ranges;                         // of those, by address
  int size = 0;                                      // which of CLIP_SIZES
  std::vector<std::vector<char>> tables;
  std::vector<int64_t> pieces;                       // of each
  int64_t bytes() const { return is_short() ? 0 : (int64_t)tables.size() * CLIP_BLOCKS * (int64_t)sizeof(ClipSum); }
  bool meets(const Range& r) const {
    if (!r.lo) return false;
    auto at = std::lower_bound(ranges.begin(), ranges.end(), r, [](const Range& a, const Range& b) { return a.hi <= b.lo; });
    return at != ranges.end() && at->lo < r.hi;
  }
  template <int MAX>
  void fill() {
    for (size_t from = 0; from < tensors.size(); from += MAX) {
      tables.emplace_back(sizeof(ClipTable<MAX>));
      ClipTable<MAX>& t = *reinterpret_cast<ClipTable<MAX>*>(tables.back().data());
      t.count = (int)std::min<size_t>(MAX, tensors.size() - from);
      uint32_t n = 0;
      for (int i = 0; i < t.count; ++i) {
        t.tensor[i] = tensors[from + i];
        t.first[i] = n;
        n += (uint32_t)ClipView(t.tensor[i]).pieces();
      }
      t.first[t.count] = n;
      pieces.push_back(n);
    }
  }
  void make_tables() {
    while (size < 3 && tensors.size() > (size_t)CLIP_SIZES[size]) ++size;
    if (size == 0) fill<CLIP_SIZES[0]>();
    else if (size == 1) fill<CLIP_SIZES[1]>();
    else if (size == 2) fill<CLIP_SIZES[2]>();
    else fill<CLIP_SIZES[3]>();
  }
  bool is_short() const { return tables.empty() || (tables.size() == 1 && pieces[0] <= CLIP_SHORT); }   // needs no workspace
};

int launch_list(Handle* h, const void* kernel, int grid, int cluster, void** args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(CLIP_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  cfg.numAttrs = launch_attributes(at, cluster);
  cfg.attrs = at;
  OP_CK(cudaLaunchKernelExC(&cfg, kernel, args));       // the table is copied once, from the list
  ++h->launches;
  return PRECOND_OK;
}
int clip_grid(const Handle* h, int64_t pieces) { return (int)std::min<int64_t>((pieces + 3) / 4, std::min(CLIP_BLOCKS, 2 * h->num_sms)); }
// The sums of squares of a list; *sums: how many.
int squares(Handle* h, const List& l, ClipSum* partial, int* sums, cudaStream_t st) {
  *sums = 0;
  for (size_t i = 0; i < l.tables.size(); ++i) {
    ClipSum* at = partial + *sums;
    void* args[] = {(void*)l.tables[i].data(), &at};
    const int grid = clip_grid(h, l.pieces[i]), rc = launch_list(h, clip_of[l.size].norm, grid, 1, args, st);
    if (rc) return rc;
    *sums += grid;
  }
  return PRECOND_OK;
}
int scale(Handle* h, const List& l, const ClipSum* partial, int sums, float max_norm, float* norm, cudaStream_t st) {
  for (size_t i = 0; i < l.tables.size(); ++i) {
    int mine = i ? 0 : sums;                            // the first launch leaves the norm, the others (and a caller's norm) find it
    void* args[] = {(void*)l.tables[i].data(), &partial, &mine, &max_norm, &norm};
    const int rc = launch_list(h, clip_of[l.size].scale, clip_grid(h, l.pieces[i]), 1, args, st);
    if (rc) return rc;
  }
  return PRECOND_OK;
}
int short_list(Handle* h, const List& l, float max_norm, float* norm, cudaStream_t st) {
  if (l.tables.empty()) {
    OP_CK(cudaMemsetAsync(norm, 0, 4, st));
    return PRECOND_OK;
  }
  void* args[] = {(void*)l.tables[0].data(), &max_norm, &norm};
  return launch_list(h, clip_of[l.size].one, CLIP_CLUSTER, CLIP_CLUSTER, args, st);
}
int total(Handle* h, const ClipSum* partial, int sums, float* norm, cudaStream_t st) {
  OP_CK(launch(clip_total_kernel<0>, dim3(1), dim3(CLIP_THREADS), 0, st, 1, partial, sums, norm));
  ++h->launches;
  return PRECOND_OK;
}
const List* as_list(precond_list_t l) { return reinterpret_cast<const List*>(l); }

// What both calls on a list ask of their arguments.
bool list_arguments(const Handle* h, const List* l, const float* norm, const void* workspace, int64_t workspace_bytes, int64_t need) {
  if (!h || !l || !norm || !aligned(norm, 4)) return false;
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return false;
  const Range n = range(norm, 1, 0, 1, 4), w = need > 0 ? range(workspace, 1, 0, need, 1) : NOWHERE;
  return !l->meets(n) && !l->meets(w) && !overlap(n, w);
}

}  // namespace

cudaError_t precond::training_attributes() {
  cudaError_t e = LayerKernels<float, true>::attributes();
  if (e == cudaSuccess) e = LayerKernels<float, false>::attributes();
  if (e == cudaSuccess) e = LayerKernels<__nv_bfloat16, true>::attributes();
  if (e == cudaSuccess) e = LayerKernels<__nv_bfloat16, false>::attributes();
  for (int i = 0; i < 2; ++i) {
    for (const StreamNorm k : stream_norm_kernels[i])
      if (k && e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, STREAM_BYTES);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(stream_grad_kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, STREAM_BYTES);
  }
  for (int i = 0; i < 2 && e == cudaSuccess; ++i)
    e = cudaFuncSetAttribute(policy_kernels[i][1], cudaFuncAttributeMaxDynamicSharedMemorySize, POLICY_PART);
  return e;
}

extern "C" {

int precond_layer_norm(precond_t ph, const void* x, const void* residual, const void* weight, const void* bias, int dtype,
                       int weight_dtype, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, float eps, void* total, int64_t ldt,
                       void* y, int64_t ldy, void* q, int64_t ldq, uint8_t* scale, float* mean, float* rstd, void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !float_type(dtype) || !float_type(weight_dtype) || !side(rows) || !side(cols) || !(eps > 0.f)) return PRECOND_EINVAL;
  const size_t sz = size_of(dtype), wz = size_of(weight_dtype);
  if (!matrix(x, rows, cols, ldx, dtype) || !matrix(weight, 1, cols, cols, weight_dtype) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      (bias && !aligned(bias, wz)))
    return PRECOND_EINVAL;
  if ((residual != nullptr) != (total != nullptr)) return PRECOND_EINVAL;
  if (residual && (!matrix(residual, rows, cols, ldr, dtype) || !matrix(total, rows, cols, ldt, dtype))) return PRECOND_EINVAL;
  if (y && !matrix(y, rows, cols, ldy, dtype)) return PRECOND_EINVAL;
  if ((q != nullptr) != (scale != nullptr) || (q && !matrix8(q, ldq, scale, rows, cols))) return PRECOND_EINVAL;
  if (rows && cols && !total && !y && !q && !mean && !rstd) return PRECOND_EINVAL;
  // outputs may not overlap anything, but for `total` over x or residual, element for element
  const Range in[4] = {range(x, rows, ldx, cols, sz), range(residual, rows, ldr, cols, sz), range(weight, 1, 0, cols, wz),
                       range(bias, 1, 0, cols, wz)};
  const Range out[6] = {range(total, rows, ldt, cols, sz), range(y, rows, ldy, cols, sz), range(q, rows, ldq, cols, 1),
                        q ? scale_range(scale, rows, cols) : NOWHERE, range(mean, 1, 0, rows, 4), range(rstd, 1, 0, rows, 4)};
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 4; ++j) {
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
  LayerNormArgs a = {x, residual, weight, bias, total, y, (uint8_t*)q, scale, mean, rstd, ldx, ldr, ldt, ldy, ldq, (int)rows, (int)cols,
                     eps, weight_dtype == PRECOND_BF16};
  const bool vec = sector_rows(x, ldx, dtype) && sector_rows(residual, ldr, dtype) && sector_rows(total, ldt, dtype) &&
                   sector_rows(y, ldy, dtype);
  const StreamShape f = vec ? stream_shape(cols, dtype, residual ? 2 : 1, false, rows, h->num_sms) : StreamShape{};
  if (f.stages) {
    OP_CK(launch(stream_norm_kernels[dtype == PRECOND_BF16][f.vectors / 2], dim3((unsigned)h->num_sms), dim3(f.threads, f.rows), f.bytes, (cudaStream_t)stream, 1, a, f.stages));
    ++h->launches;
    return PRECOND_OK;
  }
  const RowShape s = row_shape(cols, dtype, false, vec);
  const unsigned grid = (unsigned)layer_norm_blocks(s, q ? q8_row_blocks(rows) * 128 : rows, dtype, vec, h->num_sms, h->clusters);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PRECOND_BF16)
    OP_CK((vec ? launch_layer_norm<__nv_bfloat16, true>(a, s, grid, st) : launch_layer_norm<__nv_bfloat16, false>(a, s, grid, st)));
  else
    OP_CK((vec ? launch_layer_norm<float, true>(a, s, grid, st) : launch_layer_norm<float, false>(a, s, grid, st)));
  ++h->launches;
  return PRECOND_OK;
}

int64_t precond_layer_norm_grad_workspace(int64_t rows, int64_t cols) {
  if (!side(rows) || !side(cols)) return -1;
  if (rows == 0 || cols == 0) return 0;
  // Rows of either type, at sectors or not: the most blocks of any form (up to 256 columns those at sectors have smaller
  // blocks, and more of them).  Fewer clusters that fit only make fewer.
  bool whole = true;
  int64_t blocks = std::min<int64_t>(rows, PLAN_SMS);    // rows through shared memory: a block an SM
  for (const int dtype : {PRECOND_BF16, PRECOND_F32})
    for (const bool vec : {false, true}) {
      const RowShape s = layer_grad_shape(cols, dtype, vec);
      whole = whole && layer_grad_whole(s, rows);
      blocks = std::max(blocks, layer_grad_blocks(s, rows, dtype, PLAN_SMS, PLAN_CLUSTERS));
    }
  if (whole) return 0;
  return blocks * partial_pitch(cols) * 8;
}

int precond_layer_norm_grad(precond_t ph, const void* dy, const void* x, const void* weight, const float* mean, const float* rstd,
                            const void* dresidual, int dtype, int weight_dtype, int64_t rows, int64_t cols, int64_t lddy, int64_t ldx,
                            int64_t lddr, void* dx, int64_t lddx, float* dw, float* db, void* workspace, int64_t workspace_bytes,
                            void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !float_type(dtype) || !float_type(weight_dtype) || !side(rows) || !side(cols)) return PRECOND_EINVAL;
  const size_t sz = size_of(dtype);
  if (!matrix(dy, rows, cols, lddy, dtype) || !matrix(x, rows, cols, ldx, dtype) || !matrix(dx, rows, cols, lddx, dtype) ||
      !matrix(weight, 1, cols, cols, weight_dtype) || !matrix(mean, 1, rows, rows, PRECOND_F32) ||
      !matrix(rstd, 1, rows, rows, PRECOND_F32) || !matrix(dw, 1, cols, cols, PRECOND_F32) || !aligned(db, 4) ||
      (dresidual && !matrix(dresidual, rows, cols, lddr, dtype)))
    return PRECOND_EINVAL;
  const int64_t need = precond_layer_norm_grad_workspace(rows, cols);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return PRECOND_EINVAL;
  const Range in[6] = {range(dy, rows, lddy, cols, sz), range(dresidual, rows, lddr, cols, sz), range(x, rows, ldx, cols, sz),
                       range(weight, 1, 0, cols, size_of(weight_dtype)), range(mean, 1, 0, rows, 4), range(rstd, 1, 0, rows, 4)};
  const Range out[4] = {range(dx, rows, lddx, cols, sz), range(dw, 1, 0, cols, 4), range(db, 1, 0, cols, 4), range(workspace, 1, 0, need, 1)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 6; ++j) {
      // dx may lie over dy, dresidual or x, element for element, where a row is surely read once
      const bool same = i == 0 && cols <= LAYER_IN_PLACE &&
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
    if (db) OP_CK(cudaMemsetAsync(db, 0, cols * 4, st));
    return PRECOND_OK;
  }
  LayerGradArgs a = {dy, x, dresidual, weight, mean, rstd, dx, (float*)workspace, nullptr, nullptr, lddy, ldx, lddr, lddx, (int)rows, (int)cols,
                     weight_dtype == PRECOND_BF16};
  const bool vec = sector_rows(dy, lddy, dtype) && sector_rows(x, ldx, dtype) && sector_rows(dresidual, lddr, dtype) &&
                   sector_rows(dx, lddx, dtype);
  const RowShape s = layer_grad_shape(cols, dtype, vec);
  const int sms = std::min(h->num_sms, PLAN_SMS);
  unsigned grid = (unsigned)layer_grad_blocks(s, rows, dtype, sms, h->clusters);
  const int whole = need ? 0 : layer_grad_whole(s, rows);
  if (whole) {
    grid = (unsigned)whole;
    a.dw = dw;
    a.db = db;
  }
  const StreamShape f = vec && !whole ? stream_shape(cols, dtype, dresidual ? 3 : 2, true, rows, sms) : StreamShape{};
  if (f.stages) {
    grid = (unsigned)sms;                // the rows' shapes have at least as many groups
    OP_CK(launch(stream_grad_kernels[dtype == PRECOND_BF16], dim3(grid), dim3(f.threads, f.rows), f.bytes, st, 1, a, f.stages));
  } else if (dtype == PRECOND_BF16)
    OP_CK((vec ? launch_layer_grad<__nv_bfloat16, true>(a, s, grid, st) : launch_layer_grad<__nv_bfloat16, false>(a, s, grid, st)));
  else
    OP_CK((vec ? launch_layer_grad<float, true>(a, s, grid, st) : launch_layer_grad<float, false>(a, s, grid, st)));
  ++h->launches;
  if (whole) return PRECOND_OK;
  OP_CK(launch(layer_dw_kernel<0>, dim3((unsigned)((2 * partial_pitch(cols) + 31) / 32)), dim3(32, grid > 64 ? 32 : 8), 0, st, 1,
               (const float*)workspace, (int)grid, cols, dw, db));
  ++h->launches;
  return PRECOND_OK;
}

int precond_policy(precond_t ph, const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ldz, const void* ids, int id_bits,
                   const float* advantage, const float* old_logp, const float* ref_logp, const float* weight, float temperature,
                   float clip_low, float clip_high, float kl, float* loss, float* logp, void* dlogits, int64_t lddz, void* stream) {
  Handle* h = as_handle(ph);
  if (!h || !float_type(dtype) || !side(rows) || !side(vocab) || vocab < 1 || rows > (int64_t)INT32_MAX / 8) return PRECOND_EINVAL;
  if ((id_bits != 32 && id_bits != 64) || !(temperature >= 1e-18f && temperature <= 1e18f)) return PRECOND_EINVAL;
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !(kl >= 0.f && kl < INFINITY)) return PRECOND_EINVAL;
  const size_t sz = size_of(dtype);
  if (!matrix(logits, rows, vocab, ldz, dtype) || (dlogits && !matrix(dlogits, rows, vocab, lddz, dtype)) ||
      (rows && (!ids || !aligned(ids, id_bits / 8))))
    return PRECOND_EINVAL;
  for (const void* p : {(const void*)advantage, (const void*)old_logp, (const void*)ref_logp, (const void*)weight, (const void*)loss,
                        (const void*)logp})
    if (!aligned(p, 4)) return PRECOND_EINVAL;
  // without an advantage there is no loss, only the log probabilities
  if (rows && ((advantage ? !loss && !dlogits : loss || dlogits || old_logp || ref_logp || !logp) || (kl != 0.f && !ref_logp && advantage)))
    return PRECOND_EINVAL;
  const Range in[6] = {range(logits, rows, ldz, vocab, sz), range(ids, 1, 0, rows, id_bits / 8), range(advantage, 1, 0, rows, 4),
                       range(old_logp, 1, 0, rows, 4), range(ref_logp, 1, 0, rows, 4), range(weight, 1, 0, rows, 4)};
  const Range out[3] = {range(dlogits, rows, lddz, vocab, sz), range(loss, 1, 0, rows, 4), range(logp, 1, 0, rows, 4)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 6; ++j) {
      const bool same = i == 0 && j == 0 && dlogits == logits && lddz == ldz;
      if (!same && overlap(out[i], in[j])) return PRECOND_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return PRECOND_EINVAL;
  }
  if (h->device < 0) return PRECOND_ENODEV;
  if (rows == 0) return PRECOND_OK;
  int rc = prepare(h);
  if (rc) return rc;
  const PolicyArgs a = {logits, ldz, ids, id_bits == 64, advantage, old_logp, kl != 0.f ? ref_logp : nullptr, weight, loss, logp, dlogits,
                        lddz, rows, vocab, temperature, clip_low, clip_high, kl};
  const int64_t bytes = vocab * (int64_t)sz;
  if (bytes <= POLICY_WARP) {
    int i = 0;
    while (bytes > (int64_t)512 << i) ++i;
    OP_CK(launch(policy_warp_kernels[dtype == PRECOND_BF16][i], dim3((unsigned)std::min<int64_t>((rows + 7) / 8, 4 * h->num_sms)), dim3(256), 0,
                 (cudaStream_t)stream, 1, a));
    ++h->launches;
    return PRECOND_OK;
  }
  if (rows > PLAN_SMS && bytes <= (rows > 4 * PLAN_SMS ? POLICY_ROW : POLICY_ROW / 2)) {
    OP_CK(launch(policy_row_kernels[dtype == PRECOND_BF16], dim3((unsigned)rows), dim3(32), (size_t)bytes, (cudaStream_t)stream, 1, a));
    ++h->launches;
    return PRECOND_OK;
  }
  const PolicyShape s = policy_shape(rows, vocab, dtype);
  OP_CK(launch(s.kernel, dim3((unsigned)(rows * s.parts)), dim3(s.threads), (size_t)s.bytes, (cudaStream_t)stream, s.parts, a));
  ++h->launches;
  return PRECOND_OK;
}

int precond_list_create(precond_list_t* out, int count, void* const tensors[], const int dtypes[], const int64_t sizes[]) {
  if (!out || count < 0 || (count && (!tensors || !dtypes || !sizes))) return PRECOND_EINVAL;
  *out = nullptr;
  try {
    List l;
    l.tensors.reserve(count);
    l.ranges.reserve(count);
    int64_t pieces = 0;
    for (int i = 0; i < count; ++i) {
      if (!float_type(dtypes[i]) || sizes[i] < 0 || sizes[i] > (int64_t)1 << 44) return PRECOND_EINVAL;
      if (sizes[i] == 0) continue;
      const size_t sz = size_of(dtypes[i]);
      if (!tensors[i] || !aligned(tensors[i], sz)) return PRECOND_EINVAL;
      l.tensors.push_back({tensors[i], dtypes[i] == PRECOND_BF16 ? -sizes[i] : sizes[i]});
      l.ranges.push_back(range(tensors[i], 1, 0, sizes[i], sz));
      pieces += ClipView(l.tensors.back()).pieces();
    }
    if (pieces > INT32_MAX) return PRECOND_EINVAL;
    std::sort(l.ranges.begin(), l.ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    for (size_t i = 1; i < l.ranges.size(); ++i)
      if (l.ranges[i].lo < l.ranges[i - 1].hi) return PRECOND_EINVAL;     // one tensor over another would be scaled twice
    l.make_tables();
    *out = reinterpret_cast<precond_list_t>(new List(std::move(l)));
  } catch (...) {                                      // of a vector: memory
    return PRECOND_ENOMEM;
  }
  return PRECOND_OK;
}

int precond_list_destroy(precond_list_t l) {
  delete reinterpret_cast<List*>(l);
  return PRECOND_OK;
}

int64_t precond_list_workspace(precond_list_t list) {
  const List* l = as_list(list);
  return l ? l->bytes() : -1;
}

int precond_grad_norm(precond_t ph, precond_list_t list, float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
  Handle* h = as_handle(ph);
  const List* l = as_list(list);
  if (!list_arguments(h, l, norm, workspace, workspace_bytes, l ? l->bytes() : 0)) return PRECOND_EINVAL;
  if (h->device < 0) return PRECOND_ENODEV;
  int rc = prepare(h), sums = 0;
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  ClipSum* partial = reinterpret_cast<ClipSum*>(workspace);
  if (l->is_short()) return short_list(h, *l, INFINITY, norm, st);
  if ((rc = squares(h, *l, partial, &sums, st))) return rc;
  return ::total(h, partial, sums, norm, st);
}

int precond_clip_grads(precond_t ph, precond_list_t list, float max_norm, float* norm, int given, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  Handle* h = as_handle(ph);
  const List* l = as_list(list);
  if (!(max_norm >= 0.f) || !list_arguments(h, l, norm, workspace, workspace_bytes, l && !given ? l->bytes() : 0)) return PRECOND_EINVAL;
  if (h->device < 0) return PRECOND_ENODEV;
  int rc = prepare(h), sums = 0;
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  ClipSum* partial = reinterpret_cast<ClipSum*>(workspace);
  if (!given && l->is_short()) return short_list(h, *l, max_norm, norm, st);
  if (!given && (rc = squares(h, *l, partial, &sums, st))) return rc;
  return scale(h, *l, partial, sums, max_norm, norm, st);
}

}  // extern "C"
