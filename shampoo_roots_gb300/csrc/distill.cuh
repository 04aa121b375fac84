// Distillation loss against a teacher's top logits, and its gradient.
//
//   p = softmax(t / tau) over the row's candidates,  q = softmax(z / tau) over the vocabulary,
//   loss = weight tau^2 sum_j p_j (log p_j - log q_{id_j}),   dz_v = weight tau (q_v - sum_{j: id_j = v} p_j)
//
// (tau^2 keeps the gradient's size when tau changes.)  Bound by memory: the
// logits are read once and the gradient is written once.  A row belongs to a
// cluster of 1 to 8 blocks, whose threads keep its logits in registers as they
// are stored (up to 64 KB a block): a thread takes the maximum and the sum of its
// own part, the blocks join theirs through distributed shared memory in their
// order, and the gradient is formed from the registers.  (Reading the row again
// from L2 cost DRAM 3.6 GB for 1.9 GB of logits at 8192 x 131072: the rows in
// flight do not fit beside the gradients.  967 us.)  Rows beyond 8 blocks'
// registers take the kernel that reads them twice.
//
// With c = log2(e) / tau and m = max(z), q_v = 2^(z_v c - k) / S, S = sum 2^(z_v
// c - k), k = m c: the exponent is one fma, and the rounding of k cancels.  Where
// m c is so large that its rounding would move the exponent (beyond 10^6: a row
// that is masked with the type's lowest value throughout) it is (z_v - m) c
// instead; both are (z_v - b) c - k.
//
// The candidates are the work of a warp of their own, beside those that stream
// the logits (one of these doing both held the others up: 1200 us, 830 without
// candidates).  Their logits are read before anything is written, so that dz may
// be z itself, and their gradients are written last, those of one id added in
// the candidates' order.
#pragma once

#include <cooperative_groups.h>

#include "form8.cuh"

namespace precond {

constexpr int DISTILL_THREADS = 512;                 // most that stream a block's part; 32 more for the candidates
constexpr int DISTILL_MAX_TOP = 1024;

struct DistillArgs {
  const void* z; int64_t ldz;
  const void* ids; int64_t ldi; int ids64;
  const void* t; int64_t ldt; int t_bf16;
  const float* weight;            // null: 1
  float* loss;
  void* dz; int64_t lddz;
  int64_t rows, vocab;
  int top;
  float tau;
};

// 2^x; and with results below 2^-126 flushed to 0, one instruction instead of four.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_flush(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Shift {
  float b, k;
  __device__ __forceinline__ Shift(float m, float c) {
    const bool far = !(fabsf(m) * c <= 1e6f);
    b = far ? m : 0.f;
    k = far ? 0.f : m * c;
  }
  __device__ __forceinline__ float operator()(float z, float c) const { return fmaf(z - b, c, -k); }
};
// Running (maximum m, sum S of 2^(z c - m c)): joins (m2, s2) to (m, s).  Equal maxima (-inf among them) need no factor.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float c) {
  const float M = max_nan(m, m2);
  const Shift sh(M, c);
  const float a = m == M ? s : s * ex2(sh(m, c));
  const float b = m2 == M ? s2 : s2 * ex2(sh(m2, c));
  m = M;
  s = a + b;
}

template <typename T> struct LogitVec;                    // one 16-byte vector of logits
template <> struct LogitVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float((&w.x)[i] << 16);
      f[2 * i + 1] = __uint_as_float((&w.x)[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]), bf16x2_bits(f[6], f[7]));
  }
};
template <> struct LogitVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void set_float(float* p, float x) { *p = x; }
__device__ __forceinline__ void set_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

struct DistillShared {
  float p[DISTILL_MAX_TOP], logp[DISTILL_MAX_TOP], z[DISTILL_MAX_TOP];
  int id[DISTILL_MAX_TOP];          // -1: no candidate
  float m[8][DISTILL_THREADS / 32], s[8][DISTILL_THREADS / 32];   // of the streaming warps of the cluster's blocks
  float most;                       // the teacher's largest logit
  // ids already seen: open addressing, each slot an id and the first candidate that has it
  int key[2 * DISTILL_MAX_TOP], first[2 * DISTILL_MAX_TOP];
};

// A block's part of a row: elements [lo, hi), 16-byte vectors from `body` on, single ones before and after.
struct Slice {
  int lo, hi, body, nvec, tail;
  template <typename T>
  __device__ __forceinline__ Slice(const T* z, int vocab, int parts, int part) {
    const int per = (((vocab + parts - 1) / parts) + 63) / 64 * 64;
    lo = min(vocab, part * per);
    hi = min(vocab, lo + per);
    const int head = (int)(((16 - (reinterpret_cast<uintptr_t>(z + lo) & 15)) & 15) / sizeof(T));
    body = lo + min(hi - lo, head);
    nvec = (hi - body) / LogitVec<T>::N;
    tail = body + nvec * LogitVec<T>::N;
  }
  // the single element of thread `tid` (there are fewer than 2 x 8), or -1
  __device__ __forceinline__ int single(int tid) const {
    if (tid < body - lo) return lo + tid;
    tid -= body - lo;
    return tid < hi - tail ? tail + tid : -1;
  }
};

// The candidates' ids, the teacher's and the student's logits, log p and p, by one warp.  (Of the student's logits a
// block needs those of its part, and the first block all of them, for the loss.)
template <typename T>
__device__ __forceinline__ void distill_candidates(const DistillArgs& a, DistillShared& sh, int64_t row, const T* z,
                                                   const Slice& sl, bool all) {
  const int lane = threadIdx.x & 31;
  float most = -INFINITY;
  for (int j = lane; j < a.top; j += 32) {
    const int64_t id = a.ids64 ? reinterpret_cast<const int64_t*>(a.ids)[row * a.ldi + j]
                               : (int64_t) reinterpret_cast<const int32_t*>(a.ids)[row * a.ldi + j];
    const bool ok = id >= 0 && id < a.vocab;
    const float t = !ok ? -INFINITY : (a.t_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.t)[row * a.ldt + j])
                                                : reinterpret_cast<const float*>(a.t)[row * a.ldt + j]);
    sh.id[j] = ok ? (int)id : -1;
    sh.logp[j] = t;
    sh.z[j] = ok && (all || (id >= sl.lo && id < sl.hi)) ? as_float(z[id]) : 0.f;
    most = max_nan(most, t);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) sh.most = most;         // -inf: no candidate
  float st = 0.f;
  for (int j = lane; j < a.top; j += 32) {
    const float d = (sh.logp[j] - most) / a.tau;
    sh.logp[j] = d;
    st += expf(d);
  }
  const float ls = logf(warp_sum(st));
  for (int j = lane; j < a.top; j += 32) {
    sh.logp[j] -= ls;
    sh.p[j] = expf(sh.logp[j]);
  }
  __syncwarp();
}

// Makes p[j] the sum over all candidates of id[j] in this block's part, for the first of them; the ids of the others,
// and of candidates elsewhere, become -1.  By one warp, after the loss (which takes each p by itself).
__device__ __forceinline__ void distill_unite(const DistillArgs& a, DistillShared& sh, const Slice& sl) {
  const int lane = threadIdx.x & 31;
  int size = 64;
  while (size < 2 * a.top) size *= 2;
  for (int i = lane; i < size; i += 32) {
    sh.key[i] = -1;
    sh.first[i] = DISTILL_MAX_TOP;
  }
  __syncwarp();
  auto find = [&](int id) {              // the slot of an id, taken if it is new; at most half of them are taken
    int h = (int)((unsigned)id * 2654435761u >> 16) & (size - 1);
    for (int tries = 0; tries < size; ++tries, h = (h + 1) & (size - 1)) {
      const int k = atomicCAS(&sh.key[h], -1, id);
      if (k == -1 || k == id) break;
    }
    return h;
  };
  bool again = false;
  for (int j = lane; j < a.top; j += 32) {
    const int id = sh.id[j];
    if (id >= sl.lo && id < sl.hi) atomicMin(&sh.first[find(id)], j);
  }
  __syncwarp();
  for (int j = lane; j < a.top; j += 32) {
    const int id = sh.id[j];
    if (id >= sl.lo && id < sl.hi) again |= sh.first[find(id)] != j;
  }
  if (__any_sync(0xffffffffu, again)) {  // an id more than once: add in order
    for (int j = lane; j < a.top; j += 32) {
      const int id = sh.id[j];
      if (id < sl.lo || id >= sl.hi || sh.first[find(id)] != j) continue;
      float p = 0.f;
      for (int i = j; i < a.top; ++i)
        if (sh.id[i] == id) p += sh.p[i];
      sh.logp[j] = p;                    // the loss is done with log p
    }
    __syncwarp();
    for (int j = lane; j < a.top; j += 32) {
      const int id = sh.id[j];
      if (id < sl.lo || id >= sl.hi) continue;
      sh.p[j] = sh.first[find(id)] == j ? sh.logp[j] : -1.f;   // -1 marks the others: ids are still being compared
    }
    __syncwarp();
    for (int j = lane; j < a.top; j += 32)
      if (sh.p[j] == -1.f) sh.id[j] = -1;
  }
  __syncwarp();
}

// (maximum, sum) over the cluster; every thread gets it.  Each streaming warp gives its own to every block, and after
// one barrier each warp joins them all, in the order of blocks and warps.  `use` is uniform over the cluster.
__device__ __forceinline__ void distill_join(DistillShared& sh, cooperative_groups::cluster_group& cluster, float& m, float& s,
                                             float c, bool use, int streaming) {
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (use && warp < streaming) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      join(m, s, m2, s2, c);
    }
    if (lane < parts) {
      *cluster.map_shared_rank(&sh.m[part][warp], lane) = m;
      *cluster.map_shared_rank(&sh.s[part][warp], lane) = s;
    }
  }
  if (parts > 1) cluster.sync();
  else __syncthreads();
  if (use) {
    m = -INFINITY;
    s = 0.f;
    for (int i = lane; i < parts * streaming; i += 32) join(m, s, sh.m[i / streaming][i % streaming], sh.s[i / streaming][i % streaming], c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      join(m, s, m2, s2, c);
    }
  }
}

// The row's loss, by one warp: log q = ln 2 (z c - k) - ln S.
__device__ __forceinline__ void distill_loss(const DistillArgs& a, const DistillShared& sh, int64_t row, float weight, float c,
                                             const Shift& at, float s, bool teaches) {
  const int lane = threadIdx.x & 31;
  float l = 0.f;
  if (teaches) {
    const float ls = logf(s);
    for (int j = lane; j < a.top; j += 32)
      if (sh.p[j] != 0.0f) l += sh.p[j] * (sh.logp[j] - fmaf(at(sh.z[j], c), LN2, -ls));
    l = warp_sum(l);
  }
  if (lane == 0) a.loss[row] = teaches ? weight * (a.tau * a.tau) * l : 0.0f;
}

// The candidates' gradients, over the dense ones: scale (q - p), by the warp that united them.
template <typename T>
__device__ __forceinline__ void distill_patch(const DistillArgs& a, const DistillShared& sh, const Slice& sl, T* dz, float scale,
                                              float c, const Shift& at, float s) {
  for (int j = threadIdx.x & 31; j < a.top; j += 32) {
    const int id = sh.id[j];
    if (id >= sl.lo && id < sl.hi) set_float(dz + id, scale * (ex2(at(sh.z[j], c)) / s - sh.p[j]));
  }
}

// The candidates' gradients come after the streaming warps' stores: one barrier of the whole block, in both roles.
__device__ __forceinline__ void dense_done() { asm volatile("bar.sync 1, %0;" ::"r"((int)blockDim.x) : "memory"); }

// One logit into a thread's running (maximum, sum).
__device__ __forceinline__ void distill_take(float& m, float& s, float v, float c) {
  const float M = max_nan(m, v);
  const Shift at(M, c);
  if (M != m) {
    s *= ex2(at(m, c));                 // 0 at the first finite value; NaN stays
    m = M;
  }
  if (m != -INFINITY) s += ex2(at(v, c));
}
// 2^(z c - k) of a vector, in pairs.  A sum flushes what lies 2^-126 below its largest term; a gradient (which a
// large weight may scale up) takes the slower form for a vector that has such a value.
template <int N, bool KEEP>
__device__ __forceinline__ void distill_powers(float (&f)[N], const Shift& at, float c) {
  const f2 b = f2_of(-at.b, -at.b), c2 = f2_of(c, c), k = f2_of(-at.k, -at.k);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = f2_get(fma2(add2(f2_of(f[i], f[i + 1]), b), c2, k));
    f[i] = x.x;
    f[i + 1] = x.y;
  }
  bool low = false;
  if (KEEP) {
    float least = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) least = fminf(least, f[i]);
    low = least < -126.f;
  }
  if (low) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = ex2(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = ex2_flush(f[i]);
  }
}
template <typename T>
__device__ __forceinline__ void distill_take(float& m, float& s, float (&f)[LogitVec<T>::N], float c) {
  constexpr int N = LogitVec<T>::N;
  float M = max3_nan(m, f[0], f[1]);
#pragma unroll
  for (int i = 2; i < N; i += 2) M = max3_nan(M, f[i], f[i + 1]);
  const Shift at(M, c);
  if (M != m) {
    s *= ex2(at(m, c));
    m = M;
  }
  if (m != -INFINITY) {
    distill_powers<N, false>(f, at, c);
    f2 e = f2_of(f[0], f[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) e = add2(e, f2_of(f[i], f[i + 1]));
    s += sum2(e);
  }
}
// scale 2^(z c - k) of a vector.
template <typename T>
__device__ __forceinline__ void distill_dense(float (&f)[LogitVec<T>::N], const Shift& at, float c, float g) {
  constexpr int N = LogitVec<T>::N;
  distill_powers<N, true>(f, at, c);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = f2_get(mul2(f2_of(f[i], f[i + 1]), f2_of(g, g)));
    f[i] = x.x;
    f[i + 1] = x.y;
  }
}

// ------------------------------------------------------------- rows in registers: NV vectors a thread
template <typename T, int NV>
__global__ void __launch_bounds__(DISTILL_THREADS + 32, 2) distill_kernel(DistillArgs a) {
  namespace cg = cooperative_groups;
  using V = LogitVec<T>;
  __shared__ DistillShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / parts;
  const int tid = threadIdx.x, threads = blockDim.x - 32;      // the last warp: candidates
  const bool streams = tid < threads;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const float c = LOG2E / a.tau;
  const Slice sl(z, (int)a.vocab, parts, part);
  const bool reads = weight != 0.0f;

  // what lies past the part's end counts as -infinity
  uint4 w[NV];
  constexpr uint32_t NONE = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  float one = -INFINITY;
  const int at = streams ? sl.single(tid) : -1;
  if (reads && streams) {
    const uint4* zv = reinterpret_cast<const uint4*>(z + sl.body);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      w[u] = make_uint4(NONE, NONE, NONE, NONE);
      if (tid + u * threads < sl.nvec) w[u] = zv[tid + u * threads];
    }
    if (at >= 0) one = as_float(z[at]);
  }
  if (reads && !streams) distill_candidates(a, sh, row, z, sl, part == 0);
  float m = one, s = 0.f;
  if (reads && streams) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float f[V::N];
      V::unpack(w[u], f);
#pragma unroll
      for (int e = 0; e < V::N; e += 2) m = max3_nan(m, f[e], f[e + 1]);
    }
    if (m != -INFINITY) {
      const Shift mine(m, c);
      f2 e2 = f2_of(ex2(mine(one, c)), 0.f);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float f[V::N];
        V::unpack(w[u], f);
        distill_powers<V::N, false>(f, mine, c);
#pragma unroll
        for (int e = 0; e < V::N; e += 2) e2 = add2(e2, f2_of(f[e], f[e + 1]));
      }
      s = sum2(e2);
    }
  }
  distill_join(sh, cluster, m, s, c, reads, threads >> 5);
  const Shift shift(m, c);
  const bool teaches = reads && sh.most != -INFINITY;
  if (!streams) {
    if (part == 0) distill_loss(a, sh, row, weight, c, shift, s, teaches);
    if (!a.dz) return;
    if (teaches) distill_unite(a, sh, sl);
    dense_done();
    if (teaches) distill_patch(a, sh, sl, reinterpret_cast<T*>(a.dz) + row * a.lddz, weight * a.tau, c, shift, s);
    return;
  }
  if (!a.dz) return;

  const float scale = weight * a.tau;
  const float g = teaches ? scale / s : 0.f;
  if (at >= 0) set_float(dz + at, teaches ? g * ex2(shift(one, c)) : 0.f);
  const bool aligned = (reinterpret_cast<uintptr_t>(dz + sl.body) & 15) == 0;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = tid + u * threads;
    if (i >= sl.nvec) break;
    float f[V::N];
    if (teaches) {
      V::unpack(w[u], f);
      distill_dense<T>(f, shift, c, g);
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e) f[e] = 0.f;
    }
    if (aligned) {
      reinterpret_cast<uint4*>(dz + sl.body)[i] = V::pack(f);
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e) set_float(dz + sl.body + i * V::N + e, f[e]);
    }
  }
  dense_done();
}

// ------------------------------------------------------------- longer rows, read twice
template <typename T>
__global__ void __launch_bounds__(DISTILL_THREADS + 32) distill_long_kernel(DistillArgs a) {
  namespace cg = cooperative_groups;
  using V = LogitVec<T>;
  constexpr int U = 4;              // vectors in flight a thread
  __shared__ DistillShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / parts;
  const int tid = threadIdx.x, threads = blockDim.x - 32;      // the last warp: candidates
  const bool streams = tid < threads;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const float c = LOG2E / a.tau;
  const Slice sl(z, (int)a.vocab, parts, part);
  const bool reads = weight != 0.0f;
  const uint4* zv = reinterpret_cast<const uint4*>(z + sl.body);
  const int at = streams ? sl.single(tid) : -1;

  if (reads && !streams) distill_candidates(a, sh, row, z, sl, part == 0);
  float m = -INFINITY, s = 0.f;
  if (reads && streams) {
    if (at >= 0) distill_take(m, s, as_float(z[at]), c);
    for (int i0 = tid; i0 < sl.nvec; i0 += U * threads) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * threads < sl.nvec) w[u] = zv[i0 + u * threads];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * threads < sl.nvec) {
          float f[V::N];
          V::unpack(w[u], f);
          distill_take<T>(m, s, f, c);
        }
      }
    }
  }
  distill_join(sh, cluster, m, s, c, reads, threads >> 5);
  const Shift shift(m, c);
  const bool teaches = reads && sh.most != -INFINITY;
  if (!streams) {
    if (part == 0) distill_loss(a, sh, row, weight, c, shift, s, teaches);
    if (!a.dz) return;
    if (teaches) distill_unite(a, sh, sl);
    dense_done();
    if (teaches) distill_patch(a, sh, sl, reinterpret_cast<T*>(a.dz) + row * a.lddz, weight * a.tau, c, shift, s);
    return;
  }
  if (!a.dz) return;

  const float scale = weight * a.tau;
  const float g = teaches ? scale / s : 0.f;
  if (at >= 0) set_float(dz + at, teaches ? g * ex2(shift(as_float(z[at]), c)) : 0.f);
  const bool aligned = (reinterpret_cast<uintptr_t>(dz + sl.body) & 15) == 0;
  for (int i0 = tid; i0 < sl.nvec; i0 += U * threads) {
    uint4 w[U];
    if (teaches) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * threads < sl.nvec) w[u] = zv[i0 + u * threads];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * threads;
      if (i >= sl.nvec) break;
      float f[V::N];
#pragma unroll
      for (int e = 0; e < V::N; ++e) f[e] = 0.f;
      if (teaches) {
        V::unpack(w[u], f);
        distill_dense<T>(f, shift, c, g);
      }
      if (aligned) {
        reinterpret_cast<uint4*>(dz + sl.body)[i] = V::pack(f);
      } else {
#pragma unroll
        for (int e = 0; e < V::N; ++e) set_float(dz + sl.body + i * V::N + e, f[e]);
      }
    }
  }
  dense_done();
}

}  // namespace precond
