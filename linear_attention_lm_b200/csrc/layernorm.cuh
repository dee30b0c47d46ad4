// layernorm.cuh -- layer norm over the last axis with the residual add, and its
// gradient (the "based/train" README builds its layers with a fused layer norm).
//
//   r = round_dt(x + residual)        (r = x without a residual)
//   m = mean(r),  s = 1 / sqrt(mean((r - m)^2) + eps),  y = (r - m) s w + b
//   gradient, with xh = (r - m) s and t = w dy:
//     dx = s (t - mean(t) - xh mean(t xh)) + dresid
//     dw = sum_rows dy xh,  db = sum_rows dy
//
// Both are bound by HBM bandwidth: a row is read once, stays in registers for
// its sums (the variance is summed over the centred values, so a large mean
// costs no precision) and its outputs are written once.  All sums are fp32.
#pragma once

#include "common.cuh"
#include "umma.cuh"
#include "vec.cuh"

namespace based {

constexpr int kLnThreads = 256;   // threads of a CTA (more only for rows of over 8192 values)
constexpr int kLnMaxD = 16384;

// Sums of N values over the threads of a row: row_warps warps of the CTA, warp
// index in the row wr.  Every thread of the CTA calls it; `red` holds
// N floats per warp and is free again after the caller's next barrier.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int warp, int wr,
                                        int row_warps) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = warp_sum(v[n]);
  if (row_warps == 1) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) red[warp * N + n] = v[n];
  }
  __syncthreads();
  const float* r = red + (warp - wr) * N;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float t = 0.0f;
    for (int i = 0; i < row_warps; ++i) t += r[i * N + n];
    v[n] = t;
  }
}

struct LnFwdParams {
  const void *x, *residual;
  const float *w, *b;
  void *y, *resid_out;
  float *mean, *rstd;
  long long rows;
  int D, row_warps;
  float eps;
};

// One row per row_warps warps, E values per thread in vectors of V.
template <typename T, int V, int E>
__global__ void __launch_bounds__(512) layernorm_fwd_kernel(const LnFwdParams p) {
  constexpr int NV = E / V;
  __shared__ float red[2][16];
  const int warp = threadIdx.x >> 5, wr = warp % p.row_warps;
  const int lane = threadIdx.x - (warp - wr) * 32;  // thread index in the row
  const int tpr = p.row_warps * 32;
  const long long row =
      (long long)blockIdx.x * (blockDim.x / tpr) + warp / p.row_warps;
  const bool live = row < p.rows;
  const size_t off = live ? (size_t)row * p.D : 0;
  umma::grid_dep_wait();

  float f[NV][V];
  Pack<T, V> a[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * V;
    a[i].zero();
    if (live && c < p.D) a[i].load(static_cast<const T*>(p.x) + off + c);
  }
  if (p.residual) {
    Pack<T, V> b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      b[i].zero();
      if (live && c < p.D) b[i].load(static_cast<const T*>(p.residual) + off + c);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) a[i].set(e, a[i].get(e) + b[i].get(e));
      if (live && c < p.D) a[i].store(static_cast<T*>(p.resid_out) + off + c);
    }
  }
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      f[i][e] = a[i].get(e);
      sum[0] += f[i][e];
    }
  row_sum<1>(sum, red[0], warp, wr, p.row_warps);
  const float mean = sum[0] / p.D;
  float sq[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = (i * tpr + lane) * V < p.D;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      f[i][e] = in ? f[i][e] - mean : 0.0f;
      sq[0] += f[i][e] * f[i][e];
    }
  }
  row_sum<1>(sq, red[1], warp, wr, p.row_warps);
  const float rstd = 1.0f / sqrtf(sq[0] / p.D + p.eps);
  if (!live) return;
  if (lane == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * V;
    if (c < p.D) {
      float w[V], b[V];
      load_f32<V>(p.w + c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) b[e] = 0.0f;
      if (p.b) load_f32<V>(p.b + c, b);
#pragma unroll
      for (int e = 0; e < V; ++e) a[i].set(e, fmaf(f[i][e] * rstd, w[e], b[e]));
      a[i].store(static_cast<T*>(p.y) + off + c);
    }
  }
}

struct LnBwdParams {
  const void *dy, *x;
  const float *w, *mean, *rstd, *dresid;
  float *dx, *parts;
  long long rows;
  int D, row_warps;
};

// CTA i takes rows i*rpb, i*rpb + gridDim*rpb, ...; a thread owns its columns
// for all of them and sums dweight and dbias in registers; the row groups of the
// CTA meet in shared memory, and the CTA writes one part [2][D] (fp32).
template <typename T, int V, int E>
__global__ void __launch_bounds__(1024) layernorm_bwd_kernel(const LnBwdParams p) {
  constexpr int NV = E / V;
  extern __shared__ float smem[];
  __shared__ float red[2][64];
  const int warp = threadIdx.x >> 5, wr = warp % p.row_warps;
  const int lane = threadIdx.x - (warp - wr) * 32;
  const int tpr = p.row_warps * 32, rpb = blockDim.x / tpr;
  umma::grid_dep_wait();

  float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.0f;
    if (c < p.D) load_f32<V>(p.w + c, w[i]);
  }
  const float inv_d = 1.0f / p.D;
  int buf = 0;
  for (long long r0 = (long long)blockIdx.x * rpb; r0 < p.rows; r0 += (long long)gridDim.x * rpb) {
    const long long row = r0 + warp / p.row_warps;
    const bool live = row < p.rows;
    const size_t off = live ? (size_t)row * p.D : 0;
    const float mean = live ? p.mean[row] : 0.0f, rstd = live ? p.rstd[row] : 0.0f;
    Pack<T, V> x[NV], g[NV];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      x[i].zero();
      g[i].zero();
      if (live && c < p.D) {
        x[i].load(static_cast<const T*>(p.x) + off + c);
        g[i].load(static_cast<const T*>(p.dy) + off + c);
      }
    }
    float xh[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float gv = g[i].get(e);
        xh[i][e] = (x[i].get(e) - mean) * rstd;
        const float t = gv * w[i][e];
        s[0] += t;
        s[1] += t * xh[i][e];
        dw[i][e] += gv * xh[i][e];
        db[i][e] += gv;
      }
    row_sum<2>(s, red[buf], warp, wr, p.row_warps);
    buf ^= 1;
    const float c0 = s[0] * inv_d, c1 = s[1] * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      if (live && c < p.D) {
        float o[V], d[V];
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = 0.0f;
        if (p.dresid) load_f32<V>(p.dresid + off + c, d);
#pragma unroll
        for (int e = 0; e < V; ++e)
          o[e] = fmaf(rstd, g[i].get(e) * w[i][e] - c0 - xh[i][e] * c1, d[e]);
        store_f32<V>(p.dx + off + c, o);
      }
    }
  }
  // rows of the CTA together: group 0 adds the others' sums in order
  float* part = p.parts + (size_t)blockIdx.x * 2 * p.D;
  for (int grp = rpb - 1; grp > 0; --grp) {
    __syncthreads();
    if (warp / p.row_warps == grp) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + lane) * V;
        if (c < p.D)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            smem[c + e] = dw[i][e];
            smem[p.D + c + e] = db[i][e];
          }
      }
    }
    __syncthreads();
    if (warp / p.row_warps == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + lane) * V;
        if (c < p.D)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            dw[i][e] += smem[c + e];
            db[i][e] += smem[p.D + c + e];
          }
      }
    }
  }
  if (warp / p.row_warps == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      if (c < p.D) {
        store_f32<V>(part + c, dw[i]);
        store_f32<V>(part + p.D + c, db[i]);
      }
    }
  }
}

// Sum of the parts, column by column, in a fixed order: 32 columns per CTA,
// thread row y takes parts y, y + 32, ...
__global__ void __launch_bounds__(1024) layernorm_parts_kernel(const float* __restrict__ parts,
                                                               int n_parts, int D, float* dw,
                                                               float* db) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;  // of [2][D]
  umma::grid_dep_wait();
  float t = 0.0f;
  if (c < 2 * D)
    for (int i = threadIdx.y; i < n_parts; i += 32) t += parts[(size_t)i * 2 * D + c];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  t = warp_sum(s[threadIdx.x][threadIdx.y]);  // column blockIdx.x * 32 + threadIdx.y
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < 2 * D) {
    if (col < D) dw[col] = t;
    else if (db) db[col - D] = t;
  }
}

}  // namespace based
