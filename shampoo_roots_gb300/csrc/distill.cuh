// Distillation loss against a teacher's top logits, and its gradient.
//
//   p = softmax(t / tau) over the row's candidates,  q = softmax(z / tau) over the vocabulary,
//   loss = weight tau^2 sum_j p_j (log p_j - log q_{id_j}),   dz_v = weight tau (q_v - sum_{j: id_j = v} p_j)
//
// (tau^2 keeps the gradient's size when tau changes.)  Bound by memory: the
// logits are read once for the running maximum and sum, and the gradient is
// written once.  A row belongs to a cluster of 1 to 8 blocks (more where there
// are few rows), which join their (maximum, sum) through distributed shared
// memory in the blocks' order; the gradient's pass reads the row's slice again,
// from L2, where it still is (a row is at most some hundred KB, and the rows in
// flight stay below the 129 MB).  The candidates' logits are read before
// anything is written, so that dz may be z itself, and their gradients are
// written last, the candidates of one id added in their order.
#pragma once

#include <cooperative_groups.h>

#include "form8.cuh"

namespace precond {

constexpr int DISTILL_THREADS = 512;
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

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float LOG2E = 1.4426950408889634f;

// Running (maximum, sum of exp((z - max) / tau)): joins (m2, s2) to (m, s).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float c) {
  const float M = max_nan(m, m2);
  const float a = m == M ? s : s * ex2((m - M) * c);     // equal maxima (-inf among them): no factor
  const float b = m2 == M ? s2 : s2 * ex2((m2 - M) * c);
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
  float wm[DISTILL_THREADS / 32], ws[DISTILL_THREADS / 32];
  float cm[8], cs[8];               // the cluster's blocks
  int live;
};

template <typename T>
__global__ void __launch_bounds__(DISTILL_THREADS) distill_kernel(DistillArgs a) {
  namespace cg = cooperative_groups;
  using V = LogitVec<T>;
  constexpr int U = 4;              // vectors in flight a thread
  __shared__ DistillShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / parts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.ldz;
  T* dz = reinterpret_cast<T*>(a.dz) + row * a.lddz;
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const float c = LOG2E / a.tau;
  const int V64 = (int)a.vocab;

  // this block's slice of the row: [lo, hi), with 16-byte aligned vectors from `body` on
  const int per = (((V64 + parts - 1) / parts) + 63) / 64 * 64;
  const int lo = min(V64, part * per), hi = min(V64, lo + per);
  const int head = min(hi - lo, (int)(((16 - (reinterpret_cast<uintptr_t>(z + lo) & 15)) & 15) / sizeof(T)));
  const int body = lo + head;
  const int nvec = (hi - body) / V::N;
  const int tail = body + nvec * V::N;

  // ---- the candidates (warp 0 of each block, while the others begin with the logits)
  if (warp == 0) {
    float mt = -INFINITY;
    for (int j = lane; j < a.top; j += 32) {
      const int64_t id = a.ids64 ? reinterpret_cast<const int64_t*>(a.ids)[row * a.ldi + j]
                                 : (int64_t) reinterpret_cast<const int32_t*>(a.ids)[row * a.ldi + j];
      const bool ok = id >= 0 && id < a.vocab;
      const float t = !ok ? -INFINITY : (a.t_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.t)[row * a.ldt + j])
                                                  : reinterpret_cast<const float*>(a.t)[row * a.ldt + j]);
      sh.id[j] = ok ? (int)id : -1;
      sh.logp[j] = t;
      sh.z[j] = ok ? as_float(z[id]) : 0.f;
      mt = max_nan(mt, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mt = max_nan(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    const bool live = mt != -INFINITY;
    float st = 0.f;
    for (int j = lane; j < a.top; j += 32) {
      const float d = live ? (sh.logp[j] - mt) / a.tau : -INFINITY;
      sh.logp[j] = d;
      st += expf(d);
    }
    st = warp_sum(st);
    const float ls = logf(st);
    for (int j = lane; j < a.top; j += 32) {
      sh.logp[j] = sh.logp[j] - ls;
      sh.p[j] = live ? expf(sh.logp[j]) : 0.f;
    }
    if (lane == 0) sh.live = live;
  }
  bool teaches = weight != 0.0f;

  // ---- running maximum and sum of this block's slice
  float m = -INFINITY, s = 0.f;
  if (teaches) {
    auto take = [&](float v) {
      const float M = max_nan(m, v);
      if (M != m) {
        s *= ex2((m - M) * c);            // 0 at the first finite value; NaN stays
        m = M;
      }
      if (m != -INFINITY) s += ex2((v - m) * c);
    };
    for (int i = tid; i < head; i += DISTILL_THREADS) take(as_float(z[lo + i]));
    for (int i = tail + tid; i < hi; i += DISTILL_THREADS) take(as_float(z[i]));
    const uint4* zv = reinterpret_cast<const uint4*>(z + body);
    for (int i0 = tid; i0 < nvec; i0 += U * DISTILL_THREADS) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * DISTILL_THREADS;
        w[u] = zv[i < nvec ? i : i0];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * DISTILL_THREADS < nvec) {
          float f[V::N];
          V::unpack(w[u], f);
          float M = m;
#pragma unroll
          for (int k = 0; k < V::N; ++k) M = max_nan(M, f[k]);
          if (M != m) {
            s *= ex2((m - M) * c);
            m = M;
          }
          if (m != -INFINITY) {
            float e = 0.f;
#pragma unroll
            for (int k = 0; k < V::N; ++k) e += ex2((f[k] - m) * c);
            s += e;
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      join(m, s, m2, s2, c);
    }
    if (lane == 0) {
      sh.wm[warp] = m;
      sh.ws[warp] = s;
    }
  }
  __syncthreads();
  teaches = teaches && sh.live;
  if (weight != 0.0f) {
    if (warp == 0) {
      m = lane < DISTILL_THREADS / 32 ? sh.wm[lane] : -INFINITY;
      s = lane < DISTILL_THREADS / 32 ? sh.ws[lane] : 0.f;
#pragma unroll
      for (int o = DISTILL_THREADS / 64; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        join(m, s, m2, s2, c);
      }
      if (lane < parts) {               // to every block of the cluster
        *cluster.map_shared_rank(&sh.cm[part], lane) = m;
        *cluster.map_shared_rank(&sh.cs[part], lane) = s;
      }
    }
  }
  cluster.sync();
  if (weight != 0.0f) {
    m = sh.cm[0];
    s = sh.cs[0];
    for (int k = 1; k < parts; ++k) join(m, s, sh.cm[k], sh.cs[k], c);
  }

  // ---- the loss (block 0, warp 0)
  if (part == 0 && warp == 0) {
    float l = 0.f;
    if (teaches) {
      const float ls = logf(s), it = 1.0f / a.tau;
      for (int j = lane; j < a.top; j += 32)
        if (sh.p[j] != 0.0f) l += sh.p[j] * (sh.logp[j] - ((sh.z[j] - m) * it - ls));
      l = warp_sum(l);
    }
    if (lane == 0) a.loss[row] = teaches ? weight * (a.tau * a.tau) * l : 0.0f;
  }
  if (!a.dz) return;

  // ---- the gradient of this block's slice
  const float scale = weight * a.tau;
  const float f = teaches ? scale / s : 0.f;
  for (int i = tid; i < head; i += DISTILL_THREADS) set_float(dz + lo + i, teaches ? f * ex2((as_float(z[lo + i]) - m) * c) : 0.f);
  for (int i = tail + tid; i < hi; i += DISTILL_THREADS) set_float(dz + i, teaches ? f * ex2((as_float(z[i]) - m) * c) : 0.f);
  const uint4* zv = reinterpret_cast<const uint4*>(z + body);
  const bool aligned = (reinterpret_cast<uintptr_t>(dz + body) & 15) == 0;
  for (int i0 = tid; i0 < nvec; i0 += U * DISTILL_THREADS) {
    uint4 w[U];
    if (teaches) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * DISTILL_THREADS;
        w[u] = zv[i < nvec ? i : i0];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * DISTILL_THREADS;
      if (i >= nvec) break;
      float g[V::N];
#pragma unroll
      for (int k = 0; k < V::N; ++k) g[k] = 0.f;
      if (teaches) {
        V::unpack(w[u], g);
#pragma unroll
        for (int k = 0; k < V::N; ++k) g[k] = f * ex2((g[k] - m) * c);
      }
      if (aligned) {
        reinterpret_cast<uint4*>(dz + body)[i] = V::pack(g);
      } else {
#pragma unroll
        for (int k = 0; k < V::N; ++k) set_float(dz + body + i * V::N + k, g[k]);
      }
    }
  }
  if (!teaches) return;
  __syncthreads();
  for (int j = tid; j < a.top; j += DISTILL_THREADS) {
    const int id = sh.id[j];
    if (id < lo || id >= hi) continue;
    bool first = true;
    float p = 0.f;
    for (int k = 0; k < a.top; ++k) {
      if (sh.id[k] == id) {
        if (k < j) first = false;
        p += sh.p[k];
      }
    }
    if (first) set_float(dz + id, scale * (ex2((sh.z[j] - m) * c) / s - p));
  }
}

}  // namespace precond
