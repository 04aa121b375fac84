// Distillation loss against a teacher's top logits, and its gradient.
//
//   p = softmax(t / tau) over the row's candidates,  q = softmax(z / tau) over the vocabulary,
//   loss = weight tau^2 sum_j p_j (log p_j - log q_{id_j}),   dz_v = weight tau (q_v - sum_{j: id_j = v} p_j)
//
// (tau^2 keeps the gradient's size when tau changes.)  Bound by memory: the
// logits are read once and the gradient is written once.  A row belongs to a
// cluster of 1 to 8 blocks, whose threads keep its logits in registers as they
// are stored (up to 64 KB a block): a thread takes the maximum and the sum of its
// own part, the blocks join theirs through distributed shared memory in a fixed
// order, and the gradient is formed from the registers.  (Reading the row again
// from L2 cost DRAM 3.6 GB for 1.9 GB of logits at 8192 x 131072: the rows in
// flight do not fit beside the gradients.  967 us.)  Rows beyond 8 blocks'
// registers are read twice.
//
// The candidates take one warp some microseconds of latency: two dependent loads,
// a softmax, a table that unites equal ids.  That warp is part of the row's
// block, beside those that stream the logits.  Many rows leave the candidates to
// a second kernel with a warp a row, which finds the (m, S) of the rows in a
// workspace: as a part of each block that warp kept it on the SM longer than the
// logits did (8192 x 131072: 904 us, without candidates 713).  A call in place
// gathers the candidates' logits first.
//
// Measured: 8192 x 131072 bf16, 128 candidates, 744 us, 80 % of the copy
// bandwidth (in place 756); 1000 x 32000 fp32, 64 candidates, 51 us, 70 %; 24 x
// 50001 without a gradient 4.2 us.  Rows read twice, 1000 x 151936 fp32: 273 us,
// 62 %.
//
// With c = log2(e) / tau and m = max(z), q_v = 2^(z_v c - k) / S, S = sum 2^(z_v
// c - k), k = m c: the exponent is one fma, and the rounding of k cancels, as
// sums over parts of a row, each with the k of its own maximum, are joined by
// their difference in k as it was rounded.  (By m c instead, S was off by 4e-4
// for logits around 10^5.)  Where m c is so large that its rounding would move
// the exponent (beyond 10^6: a row that is masked with the type's lowest value
// throughout) it is (z_v - m) c instead; both are (z_v - b) c - k.
//
// The candidates' logits are read before anything is written, so that dz may be
// z itself, and their gradients are written last, those of one id added in the
// candidates' order.
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
  float2* stats;                  // many rows: (m, S) of each
  float* kept;                    // many rows in place: the candidates' logits, rows x top
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
    k = far ? 0.f : __fmul_rn(m, c);    // rounded for good: contracted into an fma, it would differ from use to use
  }
  __device__ __forceinline__ float operator()(float z, float c) const { return fmaf(z - b, c, -k); }
  // the exponent of the factor that takes a sum from the shift `o` to this one: -inf from -infinity, where the sum is 0
  __device__ __forceinline__ float from(const Shift& o, float c) const { return fmaf(o.b - b, c, o.k - k); }
};
// (maximum m, sum S of 2^(z c - m c)) of the lanes, joined over the warp: the common maximum first, then one factor
// a lane.  (A butterfly that joins pairs takes two factors and a shift at each of its five steps.)
__device__ __forceinline__ void join_warp(float& m, float& s, float c) {
  float M = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
  s = warp_sum(m == M ? s : s * ex2(Shift(M, c).from(Shift(m, c), c)));   // equal maxima (-inf among them) need no factor
  m = M;
}

template <typename T> struct LogitVec;                    // one 16-byte vector of logits
template <> struct LogitVec<__nv_bfloat16> {
  static constexpr int N = 8;
  // the largest of NV vectors; a NaN stays
  template <int NV>
  static __device__ __forceinline__ float largest(const uint4 (&w)[NV]) {
    uint32_t m = w[0].x;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"((&w[u].x)[i]));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
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
  template <int NV>
  static __device__ __forceinline__ float largest(const uint4 (&w)[NV]) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      m = max3_nan(m, __uint_as_float(w[u].x), __uint_as_float(w[u].y));
      m = max3_nan(m, __uint_as_float(w[u].z), __uint_as_float(w[u].w));
    }
    return m;
  }
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

// A row's shared memory, as large as its candidates need.  Up to DISTILL_FEW of them only their ids lie here, and p over
// the table when it has served: the streaming kernel, which may start while the candidates' still runs, has as much L1
// as that leaves it (with all of the SM's memory shared it took 870 us for 8192 x 131072, not 717).
constexpr int DISTILL_FEW = 256;
struct DistillShared {
  float2* sums;                     // (maximum, sum) of the streaming warps of the cluster's blocks
  float* p; float* logp; float* z; int* id;      // candidates; id -1: none
  uint16_t* key;                    // a table to find equal ids
  float* most;                      // the teacher's largest logit
  int slots;
  static __host__ __device__ int slots_for(int top) {
    int n = 64;
    while (n < 4 * top) n *= 2;
    return n;
  }
  static __host__ __device__ int bytes(int top, int sums) {
    return (sums + 1) / 2 * 16 + (top <= DISTILL_FEW ? 4 : 16) * ((top + 3) / 4 * 4) + 2 * slots_for(top) + 16;
  }
  __device__ __forceinline__ DistillShared(uint8_t* base, int top, int nsums) {
    const int n = (top + 3) / 4 * 4;
    sums = reinterpret_cast<float2*>(base);
    id = reinterpret_cast<int*>(sums + (nsums + 1) / 2 * 2);
    slots = slots_for(top);
    key = reinterpret_cast<uint16_t*>(id + n);
    most = reinterpret_cast<float*>(key + slots);
    p = top <= DISTILL_FEW ? reinterpret_cast<float*>(key) : most + 4;
    logp = p + n;
    z = logp + n;
  }
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

// The candidates of a row, the work of one warp, in its steps: gather (ids, the teacher's and the student's logits;
// of these a block needs those of its part, and the first block all, for the loss), teach (log p and p), loss, unite
// (p of the first candidate of an id becomes the sum over all of that id; the others, and those outside the block's
// part, drop out) and patch (their gradients).  `most` is the teacher's largest logit, -inf where there is no
// candidate.
template <typename T>
__device__ __forceinline__ void candidate(const DistillArgs& a, int64_t row, int j, int& id, float& t) {
  const int64_t i = a.ids64 ? reinterpret_cast<const int64_t*>(a.ids)[row * a.ldi + j]
                            : (int64_t) reinterpret_cast<const int32_t*>(a.ids)[row * a.ldi + j];
  t = a.t_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.t)[row * a.ldt + j])
               : reinterpret_cast<const float*>(a.t)[row * a.ldt + j];
  id = i >= 0 && i < a.vocab ? (int)i : -1;
  if (id < 0) t = -INFINITY;
}
template <typename T>
__device__ __forceinline__ float candidate_logit(const DistillArgs& a, int64_t row, int j, int id, const T* z, const Slice& sl, bool all) {
  if (id < 0) return 0.f;
  if (a.kept) return a.kept[row * a.top + j];
  return all || (id >= sl.lo && id < sl.hi) ? as_float(z[id]) : 0.f;
}
__device__ __forceinline__ float warp_max_nan(float m) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Second occurrences among the ids >= 0 of sh.id (j = lane, lane + 32, ...; -1 elsewhere): the lane's, a bit each; of
// equal ids all but one.  Each id writes its index to a place of the table that its hash and the round give, and reads
// it back: an index of the same id there is another occurrence, one of another id a collision, which the next round
// tells apart.  Equal ids always have the same place, so they are all done in the round in which one of them is read
// back.
__device__ __forceinline__ unsigned repeated_ids(const DistillShared& sh, int top) {
  const int lane = threadIdx.x & 31, mask = sh.slots - 1;
  unsigned open = 0, twice = 0;          // candidates that have not been read back; second occurrences
  for (int q = 0; lane + 32 * q < top; ++q) open |= sh.id[lane + 32 * q] >= 0 ? 1u << q : 0;
  for (unsigned round = 1; __any_sync(0xffffffffu, open != 0); round += 2) {
    auto place = [&](int id) { return (int)(((unsigned)id * 2654435761u * round) >> 15) & mask; };
    for (unsigned m = open; m; m &= m - 1) {
      const int j = lane + 32 * (__ffs(m) - 1);
      sh.key[place(sh.id[j])] = (uint16_t)j;
    }
    __syncwarp();
    for (unsigned m = open; m; m &= m - 1) {
      const int q = __ffs(m) - 1, j = lane + 32 * q, id = sh.id[j], k = sh.key[place(id)];
      if (k == j || sh.id[k] == id) open &= ~(1u << q);
      if (k != j && sh.id[k] == id) twice |= 1u << q;
    }
    __syncwarp();
  }
  return twice;
}
// Then, one id after another: p of its first place becomes the sum over all of them in order, the others' ids -1 (the
// loss is done with p).
__device__ __forceinline__ void unite_ids(const DistillShared& sh, int top, unsigned twice) {
  const int lane = threadIdx.x & 31;
  for (unsigned any; (any = __ballot_sync(0xffffffffu, twice != 0)) != 0;) {
    const int from = __ffs(any) - 1;
    const int id = sh.id[from + 32 * (__shfl_sync(0xffffffffu, __ffs(twice), from) - 1)];
    __syncwarp();
    float sum = 0.f;
    int first = -1;
    for (int q = 0; 32 * q < top; ++q) {
      const int j = lane + 32 * q;
      const bool same = j < top && sh.id[j] == id;
      for (unsigned m = __ballot_sync(0xffffffffu, same); m; m &= m - 1) {
        const int k = __ffs(m) - 1 + 32 * q;
        if (first < 0) first = k;
        sum += sh.p[k];
      }
      if (same) {
        twice &= ~(1u << q);
        if (j != first) sh.id[j] = -1;
      }
    }
    __syncwarp();
    if (lane == 0) sh.p[first] = sum;
    __syncwarp();
  }
}

// Up to 128 or 256: Q a lane, in registers.
template <int Q>
struct FewCandidates {
  int id[Q];
  float logp[Q], z[Q], p[Q], most;
  template <typename T>
  __device__ __forceinline__ void gather(const DistillArgs& a, const DistillShared&, int64_t row, const T* z_, const Slice& sl, bool all) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      id[q] = -1;
      logp[q] = -INFINITY;
      if (lane + 32 * q < a.top) candidate<T>(a, row, lane + 32 * q, id[q], logp[q]);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) z[q] = candidate_logit(a, row, lane + 32 * q, id[q], z_, sl, all);
    most = logp[0];
#pragma unroll
    for (int q = 1; q < Q; ++q) most = max_nan(most, logp[q]);
    most = warp_max_nan(most);
  }
  __device__ __forceinline__ void teach(const DistillArgs& a, const DistillShared&) {
    float st = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      logp[q] = (logp[q] - most) / a.tau;
      st += expf(logp[q]);               // 0 for what is no candidate
    }
    const float ls = logf(warp_sum(st));
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      logp[q] -= ls;
      p[q] = id[q] >= 0 ? expf(logp[q]) : 0.f;
    }
  }
  __device__ __forceinline__ float divergence(const DistillArgs&, const DistillShared&, float c, const Shift& at, float ls) const {
    float l = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (p[q] != 0.0f) l += p[q] * (logp[q] - fmaf(at(z[q], c), LN2, -ls));
    return l;
  }
  __device__ __forceinline__ void unite(const DistillArgs& a, const DistillShared& sh, const Slice& sl) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (id[q] < sl.lo || id[q] >= sl.hi) id[q] = -1;
      if (lane + 32 * q < a.top) sh.id[lane + 32 * q] = id[q];
    }
    __syncwarp();
    const unsigned twice = repeated_ids(sh, a.top);
    if (!__any_sync(0xffffffffu, twice != 0)) return;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (lane + 32 * q < a.top) sh.p[lane + 32 * q] = p[q];
    __syncwarp();
    unite_ids(sh, a.top, twice);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (lane + 32 * q < a.top) {
        id[q] = sh.id[lane + 32 * q];
        p[q] = sh.p[lane + 32 * q];
      }
  }
  template <typename T>
  __device__ __forceinline__ void patch(const DistillArgs&, const DistillShared&, T* dz, float scale, float c, const Shift& at, float s) const {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (id[q] >= 0) set_float(dz + id[q], scale * (ex2(at(z[q], c)) / s - p[q]));
  }
};

// More: in shared memory.
struct ManyCandidates {
  float most;
  template <typename T>
  __device__ __forceinline__ void gather(const DistillArgs& a, const DistillShared& sh, int64_t row, const T* z, const Slice& sl, bool all) {
    const int lane = threadIdx.x & 31;
    most = -INFINITY;
    for (int j = lane; j < a.top; j += 32) {
      candidate<T>(a, row, j, sh.id[j], sh.logp[j]);
      sh.z[j] = candidate_logit(a, row, j, sh.id[j], z, sl, all);
      most = max_nan(most, sh.logp[j]);
    }
    most = warp_max_nan(most);
    __syncwarp();
  }
  __device__ __forceinline__ void teach(const DistillArgs& a, const DistillShared& sh) {
    const int lane = threadIdx.x & 31;
    float st = 0.f;
    for (int j = lane; j < a.top; j += 32) {
      const float d = (sh.logp[j] - most) / a.tau;
      sh.logp[j] = d;
      st += expf(d);
    }
    const float ls = logf(warp_sum(st));
    for (int j = lane; j < a.top; j += 32) {
      sh.logp[j] -= ls;
      sh.p[j] = sh.id[j] >= 0 ? expf(sh.logp[j]) : 0.f;
    }
    __syncwarp();
  }
  __device__ __forceinline__ float divergence(const DistillArgs& a, const DistillShared& sh, float c, const Shift& at, float ls) const {
    float l = 0.f;
    for (int j = threadIdx.x & 31; j < a.top; j += 32)
      if (sh.p[j] != 0.0f) l += sh.p[j] * (sh.logp[j] - fmaf(at(sh.z[j], c), LN2, -ls));
    return l;
  }
  __device__ __forceinline__ void unite(const DistillArgs& a, const DistillShared& sh, const Slice& sl) {
    for (int j = threadIdx.x & 31; j < a.top; j += 32)
      if (sh.id[j] < sl.lo || sh.id[j] >= sl.hi) sh.id[j] = -1;
    __syncwarp();
    unite_ids(sh, a.top, repeated_ids(sh, a.top));
  }
  template <typename T>
  __device__ __forceinline__ void patch(const DistillArgs& a, const DistillShared& sh, T* dz, float scale, float c, const Shift& at, float s) const {
    for (int j = threadIdx.x & 31; j < a.top; j += 32)
      if (sh.id[j] >= 0) set_float(dz + sh.id[j], scale * (ex2(at(sh.z[j], c)) / s - sh.p[j]));
  }
};

// The row's loss: log q = ln 2 (z c - k) - ln S.
template <typename C>
__device__ __forceinline__ void distill_loss(const DistillArgs& a, const DistillShared& sh, const C& cand, int64_t row, float weight,
                                             float c, const Shift& at, float s, bool teaches) {
  const float l = teaches ? warp_sum(cand.divergence(a, sh, c, at, logf(s))) : 0.f;
  if ((threadIdx.x & 31) == 0) a.loss[row] = teaches ? weight * (a.tau * a.tau) * l : 0.0f;
}

// A block may be written to by the others of its cluster once it has begun.  It says so first of all, and waits for the
// others where it writes to them (or, writing nothing, before its next cluster barrier), with its loads in between.
__device__ __forceinline__ void begun_arrive(int parts) {
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void begun_wait(int parts) {
  __syncwarp();
  if (parts > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The barrier of a row, in two halves: the streaming warps' sums are there and the candidates' logits have been read.
// Without a cluster it is two named barriers of the block: the streaming warps wait for the candidates' warp at one,
// it for them at the other, after its work in between.
__device__ __forceinline__ void row_arrive(int parts, bool streams) {
  __syncwarp();
  if (parts > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  else asm volatile("bar.arrive %0, %1;" ::"r"(streams ? 2 : 3), "r"((int)blockDim.x) : "memory");
}
__device__ __forceinline__ void row_wait(int parts, bool streams) {
  __syncwarp();
  if (parts > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else asm volatile("bar.sync %0, %1;" ::"r"(streams ? 3 : 2), "r"((int)blockDim.x) : "memory");
}
// All warps' sums (up to 128: four a lane), joined in a fixed order; every thread gets them.
__device__ __forceinline__ void join_sums(const DistillShared& sh, int n, float& m, float& s, float c) {
  const int lane = threadIdx.x & 31;
  float2 x[4];
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lane + 32 * i < n ? sh.sums[lane + 32 * i] : make_float2(-INFINITY, 0.f);
    m = max_nan(m, x[i].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const Shift at(m, c);
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (32 * i < n) s += x[i].x == m ? x[i].y : x[i].y * ex2(at.from(Shift(x[i].x, c), c));
  s = warp_sum(s);
}

// One logit into a thread's running (maximum, sum).
__device__ __forceinline__ void distill_take(float& m, float& s, float v, float c) {
  const float M = max_nan(m, v);
  const Shift at(M, c);
  if (M != m) {
    s *= ex2(at.from(Shift(m, c), c));  // 0 at the first finite value; NaN stays
    m = M;
  }
  if (m != -INFINITY) s += ex2(at(v, c));
}
// 2^(z c - k) of a vector, in pairs; FAR and KEEP are the rare forms (Shift, ex2).
template <int N, bool FAR, bool KEEP>
__device__ __forceinline__ void distill_powers(float (&f)[N], const Shift& at, float c) {
  const f2 b = f2_of(-at.b, -at.b), c2 = f2_of(c, c), k = f2_of(-at.k, -at.k);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    f2 z = f2_of(f[i], f[i + 1]);
    if (FAR) z = add2(z, b);
    const float2 x = f2_get(fma2(z, c2, k));
    f[i] = KEEP ? ex2(x.x) : ex2_flush(x.x);
    f[i + 1] = KEEP ? ex2(x.y) : ex2_flush(x.y);
  }
}
template <int N>
__device__ __forceinline__ f2 distill_sum(f2 e, float (&f)[N], const Shift& at, float c) {
  if (at.b != 0.f) distill_powers<N, true, false>(f, at, c);
  else distill_powers<N, false, false>(f, at, c);
#pragma unroll
  for (int i = 0; i < N; i += 2) e = add2(e, f2_of(f[i], f[i + 1]));
  return e;
}
template <typename T>
__device__ __forceinline__ void distill_take(float& m, float& s, float (&f)[LogitVec<T>::N], float c) {
  constexpr int N = LogitVec<T>::N;
  float M = max3_nan(m, f[0], f[1]);
#pragma unroll
  for (int i = 2; i < N; i += 2) M = max3_nan(M, f[i], f[i + 1]);
  const Shift at(M, c);
  if (M != m) {
    s *= ex2(at.from(Shift(m, c), c));
    m = M;
  }
  if (m != -INFINITY) s += sum2(distill_sum<N>(0, f, at, c));
}
// g 2^(z c - k) of a vector.  A power below 2^-126 is flushed, unless a large factor might bring it back (`rare`: or
// the shift is of the other form).
template <typename T>
__device__ __forceinline__ void distill_dense(float (&f)[LogitVec<T>::N], const Shift& at, float c, float g, bool rare) {
  constexpr int N = LogitVec<T>::N;
  if (rare) distill_powers<N, true, true>(f, at, c);
  else distill_powers<N, false, false>(f, at, c);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = f2_get(mul2(f2_of(f[i], f[i + 1]), f2_of(g, g)));
    f[i] = x.x;
    f[i + 1] = x.y;
  }
}
// The streaming warps' logits of a row's part: NV vectors a thread in registers, or (NV = 0, longer rows) read twice.
template <typename T, int NV>
struct Part {
  uint4 w[NV > 0 ? NV : 1];
  float one;                            // the thread's single element
  int at;
  using V = LogitVec<T>;
  static constexpr int U = 4;           // NV = 0: vectors in flight
  // what lies past the part's end counts as -infinity
  __device__ __forceinline__ void load(const T* z, const Slice& sl, int tid, int threads) {
    constexpr uint32_t NONE = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    const uint4* zv = reinterpret_cast<const uint4*>(z + sl.body);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      w[u] = make_uint4(NONE, NONE, NONE, NONE);
      if (tid + u * threads < sl.nvec) w[u] = zv[tid + u * threads];
    }
    one = at >= 0 ? as_float(z[at]) : -INFINITY;
  }
  __device__ __forceinline__ void sums(const T* z, const Slice& sl, int tid, int threads, float c, float& m, float& s) {
    m = -INFINITY;
    s = 0.f;
    if constexpr (NV > 0) {
      m = max_nan(one, V::template largest<NV>(w));
      if (m != -INFINITY) {
        const Shift mine(m, c);
        f2 e2 = f2_of(ex2(mine(one, c)), 0.f);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          float f[V::N];
          V::unpack(w[u], f);
          e2 = distill_sum<V::N>(e2, f, mine, c);
        }
        s = sum2(e2);
      }
    } else {
      distill_take(m, s, one, c);       // +infinity and NaN make the sum NaN
      const uint4* zv = reinterpret_cast<const uint4*>(z + sl.body);
      for (int i0 = tid; i0 < sl.nvec; i0 += U * threads) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i0 + u * threads < sl.nvec) x[u] = zv[i0 + u * threads];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i0 + u * threads < sl.nvec) {
            float f[V::N];
            V::unpack(x[u], f);
            distill_take<T>(m, s, f, c);
          }
        }
      }
    }
  }
  // the gradient of the part, or zeros (`g` 0 and nothing read)
  __device__ __forceinline__ void store(const T* z, T* dz, const Slice& sl, int tid, int threads, bool teaches, const Shift& shift,
                                        float c, float g) {
    const bool rare = shift.b != 0.f || fabsf(g) > 1e6f;
    const bool aligned = (reinterpret_cast<uintptr_t>(dz + sl.body) & 15) == 0;
    if (at >= 0) set_float(dz + at, teaches ? g * ex2(shift(one, c)) : 0.f);
    auto vec = [&](int i, const uint4& x) {
      float f[V::N];
      if (teaches) {
        V::unpack(x, f);
        distill_dense<T>(f, shift, c, g, rare);
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
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (tid + u * threads < sl.nvec) vec(tid + u * threads, w[u]);
    } else {
      const uint4* zv = reinterpret_cast<const uint4*>(z + sl.body);
      for (int i0 = tid; i0 < sl.nvec; i0 += U * threads) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (teaches && i0 + u * threads < sl.nvec) x[u] = zv[i0 + u * threads];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i0 + u * threads < sl.nvec) vec(i0 + u * threads, x[u]);
      }
    }
  }
};

// A cluster takes a row.  FUSED: the block's last warp does the candidates; otherwise every warp streams, and (m, S)
// goes to the workspace.
template <typename T, int NV, bool FUSED>
__global__ void __launch_bounds__(DISTILL_THREADS + (FUSED ? 32 : 0), 2) distill_kernel(DistillArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t distill_smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int tid = threadIdx.x, threads = FUSED ? blockDim.x - 32 : blockDim.x, streaming = threads >> 5;
  const int warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / parts;
  const DistillShared sh(distill_smem, a.top, parts * streaming);
  const float c = LOG2E / a.tau;
  begun_arrive(parts);
  wait_for_previous();
  let_next_start();
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const bool reads = weight != 0.0f;    // uniform over the cluster
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const Slice sl(z, (int)a.vocab, parts, part);
  float m, s;

  if (!FUSED || tid < threads) {
    // ------------------------------------------------ logits
    Part<T, NV> x;
    x.at = sl.single(tid);
    Shift shift(0.f, c);
    bool teaches = false;
    if (reads) {
      x.load(z, sl, tid, threads);
      x.sums(z, sl, tid, threads, c, m, s);
      join_warp(m, s, c);
      begun_wait(parts);
      if (lane < parts) *cluster.map_shared_rank(&sh.sums[part * streaming + warp], lane) = make_float2(m, s);
      if (FUSED || parts > 1) {
        row_arrive(parts, true);
        row_wait(parts, true);
      } else {
        __syncthreads();
      }
      join_sums(sh, parts * streaming, m, s, c);
      shift = Shift(m, c);
      teaches = !FUSED || *sh.most != -INFINITY;
      if (!FUSED && part == 0 && tid == 0) a.stats[row] = make_float2(m, s);
    } else {
      begun_wait(parts);
    }
    if (a.dz) {
      x.store(z, dz, sl, tid, threads, teaches, shift, c, teaches ? weight * a.tau / s : 0.f);
      if (FUSED && reads) {
        __syncwarp();
        asm volatile("bar.arrive 1, %0;" ::"r"((int)blockDim.x) : "memory");   // the candidates' gradients come after these
      }
    }
  } else if (reads) {
    // ------------------------------------------------ candidates
    auto work = [&](auto cand) {
      cand.gather(a, sh, row, z, sl, part == 0);
      if (lane == 0) *sh.most = cand.most;
      begun_wait(parts);
      row_arrive(parts, false);
      cand.teach(a, sh);
      const bool teaches = cand.most != -INFINITY;
      row_wait(parts, false);
      join_sums(sh, parts * streaming, m, s, c);
      const Shift shift(m, c);
      if (part == 0) distill_loss(a, sh, cand, row, weight, c, shift, s, teaches);
      if (a.dz) {
        if (teaches) cand.unite(a, sh, sl);
        __syncwarp();
        asm volatile("bar.sync 1, %0;" ::"r"((int)blockDim.x) : "memory");
        if (teaches) cand.patch(a, sh, dz, weight * a.tau, c, shift, s);
      }
    };
    if (a.top <= 128) work(FewCandidates<4>());
    else if (a.top <= DISTILL_FEW) work(FewCandidates<8>());
    else work(ManyCandidates());
  } else {
    begun_wait(parts);
    if (part == 0 && lane == 0) a.loss[row] = 0.0f;
  }
}

// Many rows in place: the candidates' logits, before they are overwritten.
template <typename T>
__global__ void __launch_bounds__(256) distill_keep_kernel(DistillArgs a) {
  wait_for_previous();
  let_next_start();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.rows * a.top) return;
  const int64_t row = i / a.top, j = i % a.top;
  const int64_t id = a.ids64 ? reinterpret_cast<const int64_t*>(a.ids)[row * a.ldi + j]
                             : (int64_t) reinterpret_cast<const int32_t*>(a.ids)[row * a.ldi + j];
  a.kept[i] = id >= 0 && id < a.vocab ? as_float((reinterpret_cast<const T*>(a.z) + row * a.ldz)[id]) : 0.f;
}

// Many rows: a warp does the loss and the candidates' gradients of a row, after distill_kernel; 47 us at 8192 x 128
// candidates, with 40 registers (six blocks an SM) 60.
template <typename T, typename C>
__global__ void __launch_bounds__(256, 4) distill_candidates_kernel(DistillArgs a) {
  extern __shared__ __align__(16) uint8_t distill_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  wait_for_previous();
  let_next_start();
  if (row >= a.rows) return;
  const DistillShared sh(distill_smem + warp * DistillShared::bytes(a.top, 0), a.top, 0);
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const Slice whole(z, (int)a.vocab, 1, 0);
  const float c = LOG2E / a.tau;
  const float weight = a.weight ? a.weight[row] : 1.0f;
  if (weight == 0.0f) {
    if (lane == 0) a.loss[row] = 0.0f;
    return;
  }
  const float2 st = a.stats[row];
  C cand;
  cand.gather(a, sh, row, z, whole, true);
  cand.teach(a, sh);
  const bool teaches = cand.most != -INFINITY;
  const Shift shift(st.x, c);
  distill_loss(a, sh, cand, row, weight, c, shift, st.y, teaches);
  if (!a.dz) return;
  if (teaches) {
    cand.unite(a, sh, whole);
    cand.patch(a, sh, dz, weight * a.tau, c, shift, st.y);
  } else {                              // nothing is taught: the gradient of the softmax alone is taken back
    for (int64_t i = lane; i < a.vocab; i += 32) set_float(dz + i, 0.f);
  }
}

}  // namespace precond
