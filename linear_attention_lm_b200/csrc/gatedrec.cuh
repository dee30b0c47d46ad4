// gatedrec.cuh -- gated linear recurrence over [B, L, D], channel by channel
// (the "based/train" README's decay: a state that forgets at a learned rate):
//   a_t = sigmoid(g_t),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  y_t = round_dt(h_t)
// and its gradient, with l_t = dL/dh_t in all:
//   l_t = dy_t + a_{t+1} l_{t+1},  dx_t = (1 - a_t) l_t,
//   dg_t = l_t (h_{t-1} - x_t) a_t (1 - a_t),  dh0 = a_0 l_0.
// Gates are logits: a bf16 gate could not hold a decay between 0.996 and 1.
#pragma once

#include "common.cuh"
#include "umma.cuh"
#include "vec.cuh"

namespace based {

constexpr int kGrChunk = 64;  // tokens between two saved states

// a = sigmoid(g) and n = 1 - a.  The smaller of the two is formed with its full
// relative precision, t = e / (1 + e) with e = exp(-|g|), and the other is its
// complement to 1, so that a slow decay (1 - a << 1) keeps its rate.
struct Gate {
  float a, n;
};
__device__ __forceinline__ Gate gate_of(float g) {
  const float e = ex2_approx(-1.4426950408889634f * fabsf(g));
  const float t = __fdividef(e, 1.0f + e);
  const float u = 1.0f - t;
  return g >= 0.0f ? Gate{u, t} : Gate{t, u};
}

struct GrFwdParams {
  const void *x, *g;
  void* y;
  const float* h0;
  float *h_last, *h_chunks;
  const long long* lengths;
  int B, L, D;
};

// Length of sequence b; -1 (and a recorded error) if the array's entry is not in [0, L].
__device__ __forceinline__ int gr_length(const long long* lengths, int b, int L) {
  if (!lengths) return L;
  const long long n = lengths[b];
  if (n < 0 || n > L) {
    record_device_error(BASED_ERR_INVALID_ARG);
    return -1;
  }
  return (int)n;
}

template <typename T>
__global__ void __launch_bounds__(128) gatedrec_fwd_kernel(const GrFwdParams p) {
  umma::grid_dep_wait();
  const int cb = (p.D + 127) / 128;
  const int b = blockIdx.x / cb, c = (blockIdx.x % cb) * 128 + threadIdx.x;
  const int len = gr_length(p.lengths, b, p.L);
  if (c >= p.D || len < 0) return;
  const size_t base = (size_t)b * p.L * p.D + c;
  const int n_chunks = (p.L + kGrChunk - 1) / kGrChunk;
  float h = p.h0 ? p.h0[(size_t)b * p.D + c] : 0.0f;
  for (int t = 0; t < p.L; ++t) {
    if (p.h_chunks && t % kGrChunk == 0)
      p.h_chunks[((size_t)b * n_chunks + t / kGrChunk) * p.D + c] = t < len ? h : 0.0f;
    const size_t i = base + (size_t)t * p.D;
    if (t < len) {
      const Gate gt = gate_of(to_f32<T>(static_cast<const T*>(p.g)[i]));
      h = gt.a * h + gt.n * to_f32<T>(static_cast<const T*>(p.x)[i]);
    }
    static_cast<T*>(p.y)[i] = from_f32<T>(t < len ? h : 0.0f);
  }
  if (p.h_last) p.h_last[(size_t)b * p.D + c] = h;
}

struct GrBwdParams {
  const void *x, *g, *dy;
  const float *h_chunks, *dh_last;
  float *dx, *dg, *dh0;
  const long long* lengths;
  int B, L, D;
};

template <typename T>
__global__ void __launch_bounds__(64) gatedrec_bwd_kernel(const GrBwdParams p) {
  __shared__ float hs[kGrChunk][64];
  umma::grid_dep_wait();
  const int cb = (p.D + 63) / 64;
  const int b = blockIdx.x / cb, c = (blockIdx.x % cb) * 64 + threadIdx.x;
  const int len = gr_length(p.lengths, b, p.L);
  if (c >= p.D || len < 0) return;
  const size_t base = (size_t)b * p.L * p.D + c;
  const int n_chunks = (p.L + kGrChunk - 1) / kGrChunk;
  float l = p.dh_last ? p.dh_last[(size_t)b * p.D + c] : 0.0f;
  for (int k = n_chunks - 1; k >= 0; --k) {
    const int t0 = k * kGrChunk, t1 = min(t0 + kGrChunk, len);
    float h = t0 < t1 ? p.h_chunks[((size_t)b * n_chunks + k) * p.D + c] : 0.0f;
    for (int t = t0; t < t1; ++t) {  // the states that enter each token
      const size_t i = base + (size_t)t * p.D;
      hs[t - t0][threadIdx.x] = h;
      const Gate gt = gate_of(to_f32<T>(static_cast<const T*>(p.g)[i]));
      h = gt.a * h + gt.n * to_f32<T>(static_cast<const T*>(p.x)[i]);
    }
    for (int t = min(t0 + kGrChunk, p.L) - 1; t >= t0; --t) {
      const size_t i = base + (size_t)t * p.D;
      float dx = 0.0f, dg = 0.0f;
      if (t < len) {
        const Gate gt = gate_of(to_f32<T>(static_cast<const T*>(p.g)[i]));
        l += to_f32<T>(static_cast<const T*>(p.dy)[i]);
        dx = gt.n * l;
        dg = l * (hs[t - t0][threadIdx.x] - to_f32<T>(static_cast<const T*>(p.x)[i])) * gt.a * gt.n;
        l *= gt.a;
      }
      p.dx[i] = dx;
      p.dg[i] = dg;
    }
  }
  if (p.dh0) p.dh0[(size_t)b * p.D + c] = l;
}

// One token: h = a h + (1 - a) x in place, y = round_dt(h).
template <typename T, int V>
__global__ void __launch_bounds__(128) gatedrec_step_kernel(const T* __restrict__ x,
                                                            const T* __restrict__ g,
                                                            float* __restrict__ h,
                                                            T* __restrict__ y, long long n) {
  umma::grid_dep_wait();
  const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) * V;
  if (i >= n) return;
  Pack<T, V> xv, gv;
  float hv[V];
  xv.load(x + i);
  gv.load(g + i);
  load_f32<V>(h + i, hv);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const Gate gt = gate_of(gv.get(e));
    hv[e] = gt.a * hv[e] + gt.n * xv.get(e);
    xv.set(e, hv[e]);
  }
  store_f32<V>(h + i, hv);
  xv.store(y + i);
}

}  // namespace based
