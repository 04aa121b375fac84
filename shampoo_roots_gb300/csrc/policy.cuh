// Clipped policy loss of the taken tokens, with a KL term against a reference
// policy, and its gradient; or the tokens' log probabilities alone.
//
//   q = softmax(z / tau),  s = log q_id,  ratio = exp(s - old),  d = ref - s,
//   loss = weight (-min(ratio A, clip(ratio, 1 - low, 1 + high) A) + kl (exp(d) - 1 - d))
//   slope = dloss / ds = weight (-ratio A [not clipped] + kl (1 - exp(d))),
//   dz_v = slope / tau ([v = id] - q_v)
//
// Bound by memory: the logits are read once and the gradient is written once.  A
// row belongs to a cluster of 1 to 8 blocks.  Each copies its part into shared
// memory with one bulk copy, three blocks to an SM, so that one's loads run beside
// another's powers and a third's stores, and goes over it three times: maxima, the
// sum, the gradient.  (In registers, as the distillation loss keeps its rows, an SM
// holds two blocks: 817 us where this takes 671, for 8192 x 131072.)  Rows too long
// for 8 blocks' shared memory, 1.7 MB, are read twice.
//
// What a row takes beside its elements, the join of its sums and the loss, is the
// work of one warp of each block; the others find the shift and the factor in
// shared memory.  (Done by every thread, that was as many instructions as the
// elements: 824 us.)
//
// Rows of up to 4 KB are a warp's, in registers, and a warp goes from row to row
// (4013 x 1774 bf16 8.3 us, with a block a row 15.2); rows of up to 24 KB are a warp's
// in shared memory, if there are many (8192 x 4000 bf16 23.4 us, with several warps to a
// row 31.4).  Few rows, a block or less to
// an SM, stay in registers too: less to begin with.
//
// Measured: 8192 x 131072 bf16 671 us, 89 % of the copy bandwidth; 2999 x 50001
// bf16 98 us, 85 %; 1000 x 32000 fp32 45 us, 79 % (four waves of blocks and the
// first one's latency); scoring 24 x 50001 3.2 us on the device, 3.7 in a row (the host's
// call takes 3.1).
//
// The taken token is left out of the streamed sum: with R the sum of the others,
// s = -log(1 + R / e_id) and 1 - q_id = R / (R + e_id) keep their digits where the
// policy is sure of it (q_id near 1, where 1 - q_id would be all rounding).
#pragma once

#include <type_traits>

#include "distill.cuh"
#include "ptx.cuh"

namespace precond {

struct PolicyArgs {
  const void* z; int64_t ldz;
  const void* ids; int ids64;
  const float* advantage;         // null: log probabilities alone
  const float* old;               // null: ratio 1
  const float* ref;               // null: no KL term
  const float* weight;            // null: 1
  float* loss; float* logp;       // either may be null
  void* dz; int64_t lddz;         // null: no gradient
  int64_t rows, vocab;
  float tau, low, high, kl;
};

// The taken token's element of a vector of logits: -infinity.
__device__ __forceinline__ void hide_element(uint4& w, int e, const __nv_bfloat16*) {
  const uint32_t keep = e & 1 ? 0x0000FFFFu : 0xFFFF0000u, none = e & 1 ? 0xFF800000u : 0x0000FF80u;
  const int i = e >> 1;
  w = make_uint4(i == 0 ? (w.x & keep) | none : w.x, i == 1 ? (w.y & keep) | none : w.y, i == 2 ? (w.z & keep) | none : w.z,
                 i == 3 ? (w.w & keep) | none : w.w);
}
__device__ __forceinline__ void hide_element(uint4& w, int e, const float*) {
  constexpr uint32_t NONE = 0xFF800000u;
  w = make_uint4(e == 0 ? NONE : w.x, e == 1 ? NONE : w.y, e == 2 ? NONE : w.z, e == 3 ? NONE : w.w);
}

constexpr int POLICY_THREADS = 512;                  // most of a block
constexpr int POLICY_PART = 220 << 10;               // bytes of a row that fit into a block's shared memory
constexpr int POLICY_U = 4;                          // vectors a thread has under way

// f(i, vectors i, i + threads, ...) over a thread's vectors of n, U of them at a time, then one by one; `load(i)`.
template <int U, typename L, typename F>
__device__ __forceinline__ void policy_each(int n, int tid, int threads, L load, F f) {
  int i = tid;
  for (; i + (U - 1) * threads < n; i += U * threads) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = load(i + u * threads);
#pragma unroll
    for (int u = 0; u < U; ++u) f(i + u * threads, w[u]);
  }
  for (; i < n; i += threads) f(i, load(i));
}
__device__ __forceinline__ float warp_max_fast(float m) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
  return r;
}
__device__ __forceinline__ float largest_of(uint4 w, float m, const __nv_bfloat16*) {
  uint32_t x = w.x;
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(w.y));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(w.z));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(w.w));
  return max3_nan(m, __uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
__device__ __forceinline__ float largest_of(uint4 w, float m, const float*) {
  m = max3_nan(m, __uint_as_float(w.x), __uint_as_float(w.y));
  return max3_nan(m, __uint_as_float(w.z), __uint_as_float(w.w));
}

// What a row's threads need of its sums and of its loss, from one warp of each block.
struct PolicyRow {
  float b, k, g;                                     // the shift, and the factor of 2^(z c - k) in dz
  float taken;                                       // dz of the taken token
};

__device__ __forceinline__ int policy_id(const PolicyArgs& a, int64_t row) {
  const int64_t id = a.ids64 ? reinterpret_cast<const int64_t*>(a.ids)[row] : (int64_t) reinterpret_cast<const int32_t*>(a.ids)[row];
  return id >= 0 && id < a.vocab ? (int)id : -1;
}
// From the others' (maximum, sum) and the taken token's logit.
__device__ __forceinline__ PolicyRow policy_result(const PolicyArgs& a, float c, float weight, float advantage, float old, float ref,
                                                   float taken, float m, float s, float& loss, float& logp) {
  const float M = max_nan(m, taken);
  const Shift shift(M, c);
  const float rest = m == M ? s : s * ex2(shift.from(Shift(m, c), c)), mine = ex2(shift(taken, c)), total = rest + mine;
  // x, log2 of the taken power, may pass fp32's range where the log probability, 0.69 times as large, does not (a token masked with
  // the type's lowest value); halves, as the difference may pass it too
  const float x = shift(taken, c);
  logp = taken >= m       ? -log1pf(rest / mine)
         : x > -INFINITY ? fmaf(x, LN2, -logf(total))
                          : 2.f * ((0.5f * taken - 0.5f * M) / a.tau) - logf(total);
  loss = 0.f;
  float slope = 0.f;
  if (a.advantage) {
    const float ratio = a.old ? expf(logp - old) : logp != logp ? logp : 1.0f;   // what is not a number shows
    const float free = ratio * advantage, held = fminf(fmaxf(ratio, 1.0f - a.low), 1.0f + a.high) * advantage;
    loss = free > held ? -held : -free;
    slope = free > held ? 0.f : -free;
    if (a.ref) {
      const float d = ref - logp, e = expm1f(d);
      loss = fmaf(a.kl, e < INFINITY ? e - d : e, loss);             // d may be infinite with e
      slope = fmaf(-a.kl, e, slope);
    }
    loss *= weight;
    slope *= weight / a.tau;
  }
  return {shift.b, shift.k, -slope / total, slope * (rest / total)};
}

// (maximum, sum of 2^(z c - k)) of a warp's share of n vectors and its single elements, from shared memory in two passes:
// the maximum, which is one shift for the warp, then the sum.
template <typename T>
__device__ __forceinline__ void policy_sums(const uint4* kept, int n, int tid, int threads, float open, float c, float& m, float& s) {
  using V = LogitVec<T>;
  auto load = [&](int i) { return kept[i]; };
  m = open;
  policy_each<POLICY_U>(n, tid, threads, load, [&](int, uint4 w) { m = largest_of(w, m, (const T*)nullptr); });
  m = warp_max_fast(m);
  s = 0.f;
  if (m == -INFINITY) return;
  const Shift mine(m, c);
  f2 e = f2_of(ex2(mine(open, c)), 0.f);
  auto add = [&](auto far) {
    policy_each<POLICY_U>(n, tid, threads, load, [&](int, uint4 w) {
      float f[V::N];
      V::unpack(w, f);
      distill_powers<V::N, decltype(far)::value, false>(f, mine, c);
#pragma unroll
      for (int i = 0; i < V::N; i += 2) e = add2(e, f2_of(f[i], f[i + 1]));
    });
  };
  if (mine.b != 0.f) add(std::true_type());
  else add(std::false_type());
  s = warp_sum(sum2(e));
}
// Vector i of a row's gradient, at `body`, which may lie at any element.
template <typename T>
__device__ __forceinline__ void policy_put(T* body, bool aligned, int i, uint4 w) {
  if (aligned) {
    reinterpret_cast<uint4*>(body)[i] = w;
  } else {
    float f[LogitVec<T>::N];
    LogitVec<T>::unpack(w, f);
#pragma unroll
    for (int e = 0; e < LogitVec<T>::N; ++e) set_float(body + i * LogitVec<T>::N + e, f[e]);
  }
}
// The gradient of n vectors that `load` gives.
template <typename T, typename L>
__device__ __forceinline__ void policy_store(T* body, bool aligned, int n, int tid, int threads, L load, const PolicyRow& r, const Shift& shift,
                                             float c) {
  auto write = [&](auto rare) {
    policy_each<POLICY_U>(n, tid, threads, load, [&](int i, uint4 w) {
      float f[LogitVec<T>::N];
      LogitVec<T>::unpack(w, f);
      distill_dense<T>(f, shift, c, r.g, decltype(rare)::value);
      policy_put(body, aligned, i, LogitVec<T>::pack(f));
    });
  };
  if (shift.b != 0.f || fabsf(r.g) > 1e6f) write(std::true_type());
  else write(std::false_type());
}

// Short rows, up to 32 NV vectors: a warp has each in its registers, and goes on to another.
template <typename T, int NV>
__global__ void __launch_bounds__(256, 4) policy_warp_kernel(PolicyArgs a) {
  const int lane = threadIdx.x & 31;
  const float c = LOG2E / a.tau;
  wait_for_previous();
  let_next_start();
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.rows; row += (int64_t)gridDim.x * 8) {
    const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
    T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
    const Slice sl(z, (int)a.vocab, 1, 0);
    const float weight = a.weight ? a.weight[row] : 1.0f;
    const int id = policy_id(a, row);
    Part<T, NV> x;
    x.at = sl.single(lane);
    Shift shift(0.f, c);
    if (weight == 0.0f || id < 0) {
      if (lane == 0) {
        if (a.loss) a.loss[row] = 0.f;
        if (a.logp) a.logp[row] = 0.f;
      }
      if (a.dz) x.store(z, dz, sl, lane, 32, false, shift, c, 0.f);
      continue;
    }
    x.load(z, sl, lane, 32);
    const float taken = as_float(z[id]), advantage = a.advantage ? a.advantage[row] : 0.f, old = a.old ? a.old[row] : 0.f,
                ref = a.ref ? a.ref[row] : 0.f;
    const int vec = id >= sl.body && id < sl.tail ? (id - sl.body) / LogitVec<T>::N : -1, element = (id - sl.body) % LogitVec<T>::N;
    if (x.at == id) x.one = -INFINITY;
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (lane + 32 * u == vec) hide_element(x.w[u], element, z);
    float m, s, loss, logp;
    x.sums(z, sl, lane, 32, c, m, s);
    join_warp(m, s, c);
    const PolicyRow r = policy_result(a, c, weight, advantage, old, ref, taken, m, s, loss, logp);
    if (lane == 0) {
      if (a.loss) a.loss[row] = loss;
      if (a.logp) a.logp[row] = logp;
    }
    if (!a.dz) continue;
    __syncwarp();                                      // every lane has read the taken token: dz may be z
    shift.b = r.b;
    shift.k = r.k;
    x.store(z, dz, sl, lane, 32, true, shift, c, r.g);
    if (vec >= 0 ? (vec & 31) == lane : x.at == id) set_float(dz + id, r.taken);
  }
}

// Rows of middle length: a warp has a block to itself and copies its row to shared memory, so that nothing waits for
// another warp; one row a block, as the next begins when any other ends.  All that the row needs beside its logits is
// loaded before the copy begins (after it, one load waits for another: 8192 x 4000 bf16 24.6 us, where this takes 23.4).
template <typename T>
__global__ void __launch_bounds__(32, 32) policy_row_kernel(PolicyArgs a) {
  using V = LogitVec<T>;
  extern __shared__ __align__(16) uint8_t policy_smem[];
  __shared__ __align__(8) unsigned long long arrived;
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float c = LOG2E / a.tau;
  const uint32_t bar = smem_u32(&arrived);
  if (lane == 0) {
    mbar_init(bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  wait_for_previous();
  let_next_start();
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const int id = policy_id(a, row);
  const float advantage = a.advantage ? a.advantage[row] : 0.f, old = a.old ? a.old[row] : 0.f, ref = a.ref ? a.ref[row] : 0.f;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const Slice sl(z, (int)a.vocab, 1, 0);
  const int single = sl.single(lane), n = sl.nvec;
  const bool aligned = (reinterpret_cast<uintptr_t>(dz + sl.body) & 15) == 0;
  if (weight == 0.0f || id < 0) {
    if (lane == 0) {
      if (a.loss) a.loss[row] = 0.f;
      if (a.logp) a.logp[row] = 0.f;
    }
    if (a.dz) {
      for (int i = lane; i < n; i += 32) policy_put(dz + sl.body, aligned, i, make_uint4(0, 0, 0, 0));
      if (single >= 0) set_float(dz + single, 0.f);
    }
    return;
  }
  if (n && lane == 0) {
    mbar_expect_tx(bar, n * 16);
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(policy_smem)), "l"(z + sl.body), "r"(n * 16), "r"(bar) : "memory");
  }
  const int vec = id >= sl.body && id < sl.tail ? (id - sl.body) / V::N : -1;
  const float one = single >= 0 ? as_float(z[single]) : -INFINITY, open = single == id ? -INFINITY : one;
  const float taken = as_float(z[id]);
  uint4* kept = reinterpret_cast<uint4*>(policy_smem);
  const bool lost = n && !mbar_wait_own(bar, 0, nullptr) && !mbar_wait_own(bar, 0, nullptr);
  if (vec >= 0 && (vec & 31) == lane) {                  // a vector that this lane alone reads
    uint4 v = kept[vec];
    hide_element(v, (id - sl.body) % V::N, z);
    kept[vec] = v;
  }
  float m, s, loss, logp;
  policy_sums<T>(kept, n, lane, 32, open, c, m, s);
  if (lost) m = s = __builtin_nanf("");
  const PolicyRow r = policy_result(a, c, weight, advantage, old, ref, taken, m, s, loss, logp);
  if (lane == 0) {
    if (a.loss) a.loss[row] = loss;
    if (a.logp) a.logp[row] = logp;
  }
  if (!a.dz) return;
  Shift shift(0.f, c);
  shift.b = r.b;
  shift.k = r.k;
  __syncwarp();                                          // every lane has read the taken token: dz may be z
  policy_store<T>(dz + sl.body, aligned, n, lane, 32, [&](int i) { return kept[i]; }, r, shift, c);
  if (single >= 0) set_float(dz + single, r.g * ex2(shift(one, c)));
  if (vec >= 0 ? (vec & 31) == lane : single == id) set_float(dz + id, r.taken);
}

// Few rows: a block alone on its SM has its part of a row, up to NV vectors a thread, in registers, which is quicker to
// begin with than a copy to shared memory; every thread joins the sums and computes the loss, rather than wait for one.
template <typename T, int NV>
__global__ void __launch_bounds__(POLICY_THREADS, 1) policy_few_kernel(PolicyArgs a) {
  namespace cg = cooperative_groups;
  __shared__ float2 sums[8 * POLICY_THREADS / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / parts;
  const float c = LOG2E / a.tau;
  begun_arrive(parts);
  wait_for_previous();
  let_next_start();
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const Slice sl(z, (int)a.vocab, parts, part);
  const float weight = a.weight ? a.weight[row] : 1.0f;
  Part<T, NV> x;
  x.at = sl.single(tid);
  if (weight != 0.0f) x.load(z, sl, tid, threads);
  const int id = policy_id(a, row);
  const float advantage = a.advantage ? a.advantage[row] : 0.f, old = a.old ? a.old[row] : 0.f, ref = a.ref ? a.ref[row] : 0.f;
  Shift shift(0.f, c);
  if (weight == 0.0f || id < 0) {                        // uniform over the cluster
    begun_wait(parts);
    if (part == 0 && tid == 0) {
      if (a.loss) a.loss[row] = 0.f;
      if (a.logp) a.logp[row] = 0.f;
    }
    if (a.dz) x.store(z, dz, sl, tid, threads, false, shift, c, 0.f);
    return;
  }
  const float taken = as_float(z[id]);                   // before anything is written: dz may be z
  const int vec = id >= sl.body && id < sl.tail ? (id - sl.body) / LogitVec<T>::N : -1, element = (id - sl.body) % LogitVec<T>::N;
  if (x.at == id) x.one = -INFINITY;
#pragma unroll
  for (int u = 0; u < NV; ++u)
    if (tid + u * threads == vec) hide_element(x.w[u], element, z);
  float m, s, loss, logp;
  x.sums(z, sl, tid, threads, c, m, s);
  join_warp(m, s, c);
  begun_wait(parts);
  if (lane < parts) *cluster.map_shared_rank(&sums[part * warps + warp], lane) = make_float2(m, s);
  if (parts > 1) {
    row_arrive(parts, true);
    row_wait(parts, true);
  } else {
    __syncthreads();
  }
  join_sums(sums, parts * warps, m, s, c);
  const PolicyRow r = policy_result(a, c, weight, advantage, old, ref, taken, m, s, loss, logp);
  if (part == 0 && tid == 0) {
    if (a.loss) a.loss[row] = loss;
    if (a.logp) a.logp[row] = logp;
  }
  if (!a.dz) return;
  shift.b = r.b;
  shift.k = r.k;
  x.store(z, dz, sl, tid, threads, true, shift, c, r.g);
  // the taken token's, after the vector that it lies in, by the same thread
  if (vec >= 0 ? vec % threads == tid : x.at == id) set_float(dz + id, r.taken);
}

// Longer rows.  KEPT: a block's part of the row lies in its shared memory; otherwise the row is read twice.
template <typename T, bool KEPT>
__global__ void __launch_bounds__(POLICY_THREADS, 3) policy_kernel(PolicyArgs a) {
  namespace cg = cooperative_groups;
  using V = LogitVec<T>;
  constexpr float NOT_A_NUMBER = __builtin_nanf("");
  extern __shared__ __align__(16) uint8_t policy_smem[];
  __shared__ float2 own[POLICY_THREADS / 32], sums[8];   // (maximum, sum) of the block's warps, of the cluster's blocks
  __shared__ PolicyRow result;
  __shared__ __align__(8) unsigned long long arrived;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / parts;
  const float c = LOG2E / a.tau;
  begun_arrive(parts);
  if (KEPT) {
    if (tid == 0) {
      mbar_init(smem_u32(&arrived), 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
  }
  wait_for_previous();
  let_next_start();
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const Slice sl(z, (int)a.vocab, parts, part);
  const int single = sl.single(tid), n = sl.nvec;
  const bool copies = KEPT && n && weight != 0.0f;       // before the taken token is known
  if (copies && tid == 0) {
    mbar_expect_tx(smem_u32(&arrived), n * 16);
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(policy_smem)), "l"(z + sl.body), "r"(n * 16), "r"(smem_u32(&arrived)) : "memory");
  }
  const int id = policy_id(a, row);
  const bool reads = weight != 0.0f && id >= 0;          // uniform over the cluster
  const bool aligned = (reinterpret_cast<uintptr_t>(dz + sl.body) & 15) == 0;
  auto arrive = [&]() { return mbar_wait_own(smem_u32(&arrived), 0, nullptr) || mbar_wait_own(smem_u32(&arrived), 0, nullptr); };
  if (!reads) {
    begun_wait(parts);
    if (copies) arrive();                                // no block leaves while its copy is under way
    if (part == 0 && tid == 0) {
      if (a.loss) a.loss[row] = 0.f;
      if (a.logp) a.logp[row] = 0.f;
    }
    if (a.dz) {
      for (int i = tid; i < n; i += threads) policy_put(dz + sl.body, aligned, i, make_uint4(0, 0, 0, 0));
      if (single >= 0) set_float(dz + single, 0.f);
    }
    return;
  }
  const int vec = id >= sl.body && id < sl.tail ? (id - sl.body) / V::N : -1, element = (id - sl.body) % V::N;
  bool lost = false;
  float one = single >= 0 ? as_float(z[single]) : -INFINITY;
  const float open = single == id ? -INFINITY : one;     // without the taken token
  float taken = 0.f, advantage = 0.f, old = 0.f, ref = 0.f;
  if (warp == 0) {                                       // before anything is written: dz may be z
    taken = as_float(z[id]);
    if (a.advantage) advantage = a.advantage[row];
    if (a.old) old = a.old[row];
    if (a.ref) ref = a.ref[row];
  }
  float m, s;
  if (KEPT) {
    if (n) lost = !arrive();
    uint4* kept = reinterpret_cast<uint4*>(policy_smem);
    if (vec >= 0 && vec % threads == tid) {              // a vector that this thread alone reads
      uint4 v = kept[vec];
      hide_element(v, element, z);
      kept[vec] = v;
    }
    policy_sums<T>(kept, n, tid, threads, open, c, m, s);
    if (lost) m = s = NOT_A_NUMBER;
  } else {
    const uint4* v = reinterpret_cast<const uint4*>(z + sl.body);
    m = -INFINITY;
    s = 0.f;
    distill_take(m, s, open, c);
    policy_each<POLICY_U>(n, tid, threads, [&](int i) { return v[i]; }, [&](int i, uint4 w) {
      if (i == vec) hide_element(w, element, z);
      float f[V::N];
      V::unpack(w, f);
      distill_take<T>(m, s, f, c);
    });
    join_warp(m, s, c);
  }
  if (lane == 0) own[warp] = make_float2(m, s);
  __syncthreads();
  begun_wait(parts);
  if (warp == 0) {
    join_sums(own, warps, m, s, c);
    if (lane < parts) *cluster.map_shared_rank(&sums[part], lane) = make_float2(m, s);
  }
  if (parts > 1) {
    row_arrive(parts, true);
    row_wait(parts, true);
  }
  if (warp == 0) {
    __syncwarp();
    join_sums(sums, parts, m, s, c);
    float loss, logp;
    const PolicyRow r = policy_result(a, c, weight, advantage, old, ref, taken, m, s, loss, logp);
    if (lane == 0) {
      if (part == 0 && a.loss) a.loss[row] = loss;
      if (part == 0 && a.logp) a.logp[row] = logp;
      result = r;
    }
  }
  if (!a.dz) return;
  __syncthreads();
  const PolicyRow r = result;
  Shift shift(0.f, c);
  shift.b = r.b;
  shift.k = r.k;
  const uint4* from = KEPT ? reinterpret_cast<const uint4*>(policy_smem) : reinterpret_cast<const uint4*>(z + sl.body);
  policy_store<T>(dz + sl.body, aligned, n, tid, threads, [&](int i) { return from[i]; }, r, shift, c);
  if (single >= 0) set_float(dz + single, r.g * ex2(shift(one, c)));
  // the taken token's, after the vector that it lies in, by the same thread
  if (vec >= 0 ? vec % threads == tid : single == id) set_float(dz + id, r.taken);
}

}  // namespace precond
