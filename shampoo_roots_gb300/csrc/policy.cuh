// Clipped policy loss of the taken tokens, with a KL term against a reference
// policy, and its gradient; or the tokens' log probabilities alone.
//
//   q = softmax(z / tau),  s = log q_id,  ratio = exp(s - old),  d = ref - s,
//   loss = weight (-min(ratio A, clip(ratio, 1 - low, 1 + high) A) + kl (exp(d) - 1 - d))
//   slope = dloss / ds = weight (-ratio A [not clipped] + kl (1 - exp(d))),
//   dz_v = slope / tau ([v = id] - q_v)
//
// Bound by memory: the logits are read once and the gradient is written once.  A
// row lies in the registers of a cluster's blocks as in the distillation loss
// (distill.cuh: Part, Shift, the joins), which this shares; but one token needs no
// warp of its own, and no second kernel.
//
// The taken token is left out of the streamed sum: with R the sum of the others,
// s = -log(1 + R / e_id) and 1 - q_id = R / (R + e_id) keep their digits where the
// policy is sure of it (q_id near 1, where 1 - q_id would be all rounding).
#pragma once

#include "distill.cuh"

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

template <typename T, int NV>
__global__ void __launch_bounds__(DISTILL_THREADS, 2) policy_kernel(PolicyArgs a) {
  namespace cg = cooperative_groups;
  __shared__ float2 sums[8 * DISTILL_THREADS / 32];
  constexpr int N = LogitVec<T>::N;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / parts;
  const float c = LOG2E / a.tau;
  begun_arrive(parts);
  wait_for_previous();
  let_next_start();
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const int64_t wide = a.ids64 ? reinterpret_cast<const int64_t*>(a.ids)[row] : (int64_t) reinterpret_cast<const int32_t*>(a.ids)[row];
  const int id = wide >= 0 && wide < a.vocab ? (int)wide : -1;
  const float advantage = a.advantage ? a.advantage[row] : 0.f, old = a.old ? a.old[row] : 0.f, ref = a.ref ? a.ref[row] : 0.f;
  const bool reads = weight != 0.0f && id >= 0;          // uniform over the cluster
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const Slice sl(z, (int)a.vocab, parts, part);
  // the vector that holds the taken token, where this block's part has it, and the thread that has that vector
  const int vec = id >= sl.body && id < sl.tail ? (id - sl.body) / N : -1, element = (id - sl.body) % N;

  Part<T, NV> x;
  x.at = sl.single(tid);
  Shift shift(0.f, c);
  float slope = 0.f, logp = 0.f, loss = 0.f, total = 1.f, rest = 0.f;
  if (reads) {
    x.load(z, sl, tid, threads);
    const float taken = as_float(z[id]);                 // before anything is written: dz may be z
    if (x.at == id) x.one = -INFINITY;
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (tid + u * threads == vec) hide_element(x.w[u], element, z);
    float m, s;
    x.sums(z, sl, tid, threads, c, m, s, [&](int i, uint4& w) {
      if (i == vec) hide_element(w, element, z);
    });
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
    const float M = max_nan(m, taken);
    shift = Shift(M, c);
    rest = m == M ? s : s * ex2(shift.from(Shift(m, c), c));
    const float mine = ex2(shift(taken, c));
    total = rest + mine;
    logp = taken >= m ? -log1pf(rest / mine) : fmaf(shift(taken, c), LN2, -logf(total));
    rest /= total;
    if (a.advantage) {
      const float ratio = a.old ? expf(logp - old) : logp != logp ? logp : 1.0f;   // what is not a number shows
      const float free = ratio * advantage, held = fminf(fmaxf(ratio, 1.0f - a.low), 1.0f + a.high) * advantage;
      loss = free > held ? -held : -free;
      slope = free > held ? 0.f : -free;
      if (a.ref) {
        const float d = ref - logp, e = expm1f(d);
        loss = fmaf(a.kl, e - d, loss);
        slope = fmaf(-a.kl, e, slope);
      }
      loss *= weight;
      slope *= weight / a.tau;
    }
  } else {
    begun_wait(parts);
  }
  if (part == 0 && tid == 0) {
    if (a.loss) a.loss[row] = loss;
    if (a.logp) a.logp[row] = logp;
  }
  if (!a.dz) return;
  x.store(z, dz, sl, tid, threads, reads, shift, c, -slope / total);
  // its own store after the vector's, by the same thread
  if (reads && (vec >= 0 ? vec % threads == tid : x.at == id)) set_float(dz + id, slope * rest);
}

}  // namespace precond
