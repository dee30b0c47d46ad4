// layernorm.cuh -- layer norm over the last axis with the residual add, and its
// gradient (the "based/train" README builds its layers with a fused layer norm).
//
//   r = round_dt(x + residual)        (r = x without a residual)
//   m = mean(r),  s = 1 / sqrt(mean((r - m)^2) + eps),  y = (r - m) s w + b
//   gradient, with xh = (r - m) s and t = w dy:
//     dx = s (t - mean(t) - xh mean(t xh)) + dresid
//     dw = sum_rows dy xh,  db = sum_rows dy
//
// A row is read once, stays in registers for its sums (the variance is summed over the
// centred values, so a large mean costs no precision) and its outputs are written
// once.  All sums are fp32.  Rows of whole vectors are bound by HBM bandwidth; rows that
// no vector divides by single-value accesses (74 and 78 instructions per value); the
// gradient of rows of more than 8192 by its loads, see there.
//
// Measured on B200 (a plain device copy of as many bytes in brackets): forward
// with residual, 16384 x 1024 bf16, 134 MB: 24.0 us, 5.6 TB/s (24.6 us); gradient
// with dresid, 16384 x 2048 bf16, 403 MB: 66 us, 6.1 TB/s.  Loading one row per
// short-lived warp, with nothing ahead, took 30.0 and 146 us.  Forward fp32, 16384 x
// 1024 with residual, 268 MB: 47.4 us (44.2 us).  16384 x 999 bf16 with residual and
// dresid: forward 60.5, gradient 58.5 us.
#pragma once

#include "common.cuh"
#include "umma.cuh"
#include "vec.cuh"

namespace based {

constexpr int kLnThreads = 256;   // threads of a CTA (more only for the longest rows)
constexpr int kLnMaxD = 16384;

// Barrier of the threads of a row.  Rows of several warps have a named barrier of
// their own, so the rows of a CTA run at their own pace.
__device__ __forceinline__ void row_barrier(int warp, int row_warps) {
  if (row_warps == 1) __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / row_warps), "r"(row_warps * 32) : "memory");
}

// Sums of N values over the threads of a row: row_warps warps of the CTA, this
// one the wr-th, or (kSub) tpr lanes of a warp, a power of two.  `red` holds N
// floats per warp and is free again after the row's next barrier.
template <int N, bool kSub>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int warp, int wr, int row_warps,
                                        int tpr) {
  if constexpr (kSub) {
    for (int o = tpr / 2; o > 0; o /= 2)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    return;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = warp_sum(v[n]);
  if (row_warps == 1) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) red[warp * N + n] = v[n];
  }
  row_barrier(warp, row_warps);
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
  int D, row_warps, lanes;
  float eps;
};

// Rows of up to 256 values (E = 8) take 4 to 32 lanes of a warp, so that a warp
// works on up to eight rows (524288 x 32 bf16 with residual: 163 us with a warp per
// row, 25 here); longer ones one warp or several.
__host__ __device__ constexpr bool ln_sub(int E) { return E == 8; }

// E values per thread in vectors of V; a group of threads takes every (number of
// groups)-th row and loads the next one before it works on this one.
template <typename T, int V, int E, bool kResidual, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads > 256 ? 1 : E == 8 ? 4 : 2)
    layernorm_fwd_kernel(const LnFwdParams p) {
  constexpr int NV = E / V;
  __shared__ float red[2][32];
  constexpr bool kSub = ln_sub(E);
  const int tpr = kSub ? p.lanes : p.row_warps * 32, rpb = kThreads / tpr;
  const int warp = threadIdx.x >> 5, wr = warp % p.row_warps;
  const int group = kSub ? threadIdx.x / tpr : warp / p.row_warps;
  const int lane = kSub ? threadIdx.x - group * tpr : threadIdx.x - (warp - wr) * 32;  // in the row
  const float inv_d = 1.0f / p.D;
  umma::grid_dep_wait();

  Pack<T, V> x[NV], r[NV];
  auto fetch = [&](long long row) {
    const size_t off = (size_t)row * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      if (c < p.D) {
        x[i].load(static_cast<const T*>(p.x) + off + c);
        if (kResidual) r[i].load(static_cast<const T*>(p.residual) + off + c);
      }
    }
  };
  long long row = (long long)blockIdx.x * rpb + group;
  const long long step = (long long)gridDim.x * rpb;
  // the rows of a warp stay together: its first one decides
  const int after = kSub ? group % (32 / tpr) : 0;
  if (row < p.rows) fetch(row);
  for (; row < p.rows + after; row += step) {
    const bool live = !kSub || row < p.rows;
    const size_t off = (size_t)row * p.D;
    float f[NV][V];
    // a thread's sum as a tree (vectors, then four parts): 5 to 11 roundings in a row
    // instead of 32, which a mean near zero shows
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      const bool in = live && c < p.D;
      if (kResidual) {
#pragma unroll
        for (int e = 0; e < V; ++e) x[i].set(e, x[i].get(e) + r[i].get(e));
        if (in) x[i].store(static_cast<T*>(p.resid_out) + off + c);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) f[i][e] = in ? x[i].get(e) : 0.0f;
      float t[V];
#pragma unroll
      for (int e = 0; e < V; ++e) t[e] = f[i][e];
#pragma unroll
      for (int d = V / 2; d > 0; d /= 2)
#pragma unroll
        for (int e = 0; e < d; ++e) t[e] += t[e + d];
      part[i % 4] += t[0];
    }
    float sum[1] = {(part[0] + part[1]) + (part[2] + part[3])};
    if (row + step < p.rows) fetch(row + step);
    row_sum<1, kSub>(sum, red[0], warp, wr, p.row_warps, tpr);
    const float mean = sum[0] * inv_d;
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = live && (i * tpr + lane) * V < p.D;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[i][e] = in ? f[i][e] - mean : 0.0f;
        sq[0] += f[i][e] * f[i][e];
      }
    }
    row_sum<1, kSub>(sq, red[1], warp, wr, p.row_warps, tpr);
    const float rstd = 1.0f / sqrtf(sq[0] * inv_d + p.eps);
    if (live && lane == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      if (live && c < p.D) {
        float w[V], b[V];
        load_f32<V>(p.w + c, w);
#pragma unroll
        for (int e = 0; e < V; ++e) b[e] = 0.0f;
        if (p.b) load_f32<V>(p.b + c, b);
        Pack<T, V> y;
#pragma unroll
        for (int e = 0; e < V; ++e) y.set(e, fmaf(f[i][e] * rstd, w[e], b[e]));
        y.store(static_cast<T*>(p.y) + off + c);
      }
    }
  }
}

struct LnBwdParams {
  const void *dy, *x;
  const float *w, *mean, *rstd, *dresid;
  float *dx, *parts;
  long long rows;
  int D, row_warps, lanes;
};

// A thread owns its columns for all the rows of its group and sums dweight and
// dbias in registers; the groups of the CTA meet in shared memory at the end, and
// the CTA writes one part [2][D] (fp32).  Vectors are four values at most: 16
// bytes of the fp32 arrays, which are most of the traffic.  The rows to come are
// copied ahead by cp.async.  Where rows are whole vectors of four, each thread
// copies what it will read itself and no barrier is between a row's arrival and its
// use; other rows are copied as the 16-byte pieces that hold them, by the whole
// group (3001 x 999 fp32: 19.8 us with 4-byte copies, 15.8 with pieces; 16384 x 999
// bf16, where two-byte copies have no asynchronous form: 148 and 59 us).
//
// Rows of more than 8192 values take 1024 threads, which may have 64 registers each: the
// five arrays of 16 values do not fit (488 to 792 bytes of spill stores per thread,
// 368 to 816 of loads) and nothing is copied ahead, so every row waits for its loads.
// 2048 rows bf16 with dresid: width 8192 40.9 us, 12288 169, 16384 190, 16383 282.
template <typename T, int V, int E, int kThreads>
struct LnBwdShape {
  static constexpr int NV = E / V;
  static constexpr bool kAhead = kThreads <= 512;  // the longest rows leave no room
  static constexpr bool kOwn = kAhead && V == 4, kShare = kAhead && V < 4;
  static constexpr int kStages = sizeof(T) == 2 ? 3 : 2;  // two CTAs of 256 threads fit an SM
  static constexpr int kX = V * (int)sizeof(T), kR = V * 4;  // bytes of a vector
  static constexpr int kThread = NV * (2 * kX + kR);         // bytes of a thread's row
  // a row of n bytes starts anywhere in its first 16-byte piece
  __host__ __device__ static constexpr int pieces(int n) { return (n + 15 + 15) / 16 * 16; }
  __host__ __device__ static constexpr int shared_row(int D) {
    return 2 * pieces(D * (int)sizeof(T)) + pieces(D * 4);
  }
  static constexpr size_t smem(int tpr, int D) {
    const size_t ring = kOwn     ? (size_t)kStages * kThread * kThreads
                        : kShare ? (size_t)kStages * shared_row(D) * (kThreads / tpr)
                                 : 0;
    const size_t join = tpr < kThreads ? (size_t)D * 8 * (kThreads / tpr) : 0;
    return join > ring ? join : ring;
  }
  // that of the widest rows (a thread has E values) of any number of threads
  static constexpr size_t most_smem() {
    size_t most = 0;
    for (int tpr = ln_sub(E) ? 4 : 32; tpr <= kThreads; tpr *= 2)
      if (smem(tpr, tpr * E) > most) most = smem(tpr, tpr * E);
    return most;
  }
};

// Whether the 16-byte pieces that hold row `row` of an array of `rows` rows of n bytes
// lie in the array: a row's last piece holds up to 15 bytes of the rows behind it, which
// are the next one (rows of 15 bytes or more) or some more.  kShort: n may be under 15.
template <bool kShort>
__host__ __device__ constexpr bool pieces_inside(long long row, int n, long long rows) {
  return row + (kShort && n < 15 ? 15 : 1) < rows;
}
// Row `row` of D values, as those pieces, into `to`, by the tpr threads of a group.  Of a
// piece that may reach past the array only the row's own bytes are read.
template <bool kShort, typename T>
__device__ __forceinline__ void copy_row_pieces(unsigned char* to, const T* from, long long row,
                                                int D, long long rows, int lane, int tpr) {
  const long long begin = row * D * (long long)sizeof(T);
  const int shift = (int)(begin & 15), len = shift + D * (int)sizeof(T);
  const unsigned char* src = reinterpret_cast<const unsigned char*>(from) + (begin - shift) + lane * 16;
  to += lane * 16;
  if (pieces_inside<kShort>(row, D * (int)sizeof(T), rows)) {
    for (int o = lane * 16; o < len; o += tpr * 16, src += tpr * 16, to += tpr * 16)
      umma::cp_async16(to, src, true);
  } else {
    for (int o = lane * 16; o < len; o += tpr * 16, src += tpr * 16, to += tpr * 16)
      umma::cp_async16_part(to, src, min(16, len - o));
  }
}
// Where the row's first value lies in its pieces.
template <typename T>
__device__ __forceinline__ int row_shift(long long row, int D) {
  return (int)((unsigned)row * (unsigned)D * (unsigned)sizeof(T) & 15u);  // low bits only
}

template <int Bytes>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  if constexpr (Bytes == 16) umma::cp_async16(to, from, true);
  else umma::cp_async_small<Bytes>(to, from, true);
}

// A thread's NV vectors of V elements as pairs.  at(i): where vector i lies (aligned
// to all its elements); in(i): whether it does (zeros if not).
template <typename T, int V, int NV, typename At, typename In>
__device__ __forceinline__ void load_pairs(F2* v, At at, In in) {
  if constexpr (V == 1) {
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
      const float lo = in(i) ? to_f32<T>(*at(i)) : 0.0f;
      const float hi = in(i + 1) ? to_f32<T>(*at(i + 1)) : 0.0f;
      v[i / 2] = f2(lo, hi);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Pack<T, V> r;
      r.zero();
      if (in(i)) r.load(at(i));
#pragma unroll
      for (int e = 0; e < V; e += 2) v[(i * V + e) / 2] = load_pair(&r.e[e]);
    }
  }
}
template <int V, int NV, typename At, typename In>
__device__ __forceinline__ void store_pairs(const F2* v, At at, In in) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 f = f2_get(v[(i * V + e) / 2]);
      o[e] = (i * V + e) % 2 ? f.y : f.x;
    }
    if (in(i)) store_f32<V>(at(i), o);
  }
}

// kRowWarps: warps of a row; 0: p.row_warps (rows that are not whole vectors of four).
template <typename T, int V, int E, int kThreads, int kRowWarps>
__global__ void __launch_bounds__(kThreads, kThreads > 256 ? 1 : E == 8 && V == 4 ? 3 : 2)
    layernorm_bwd_kernel(const LnBwdParams p) {
  using Shape = LnBwdShape<T, V, E, kThreads>;
  constexpr int NV = Shape::NV, kStages = Shape::kStages;
  extern __shared__ __align__(16) unsigned char ln_smem[];
  __shared__ float red[2][64];
  constexpr bool kSub = ln_sub(E);
  const int row_warps = kRowWarps ? kRowWarps : p.row_warps;
  const int tpr = kSub ? p.lanes : row_warps * 32, rpb = kThreads / tpr;
  const int warp = threadIdx.x >> 5, wr = warp % row_warps;
  const int group = kSub ? threadIdx.x / tpr : warp / row_warps;
  const int lane = kSub ? threadIdx.x - group * tpr : threadIdx.x - (warp - wr) * 32;
  umma::grid_dep_wait();

  // this thread's E columns: vector i starts at column col(i)
  auto col = [&](int i) { return (i * tpr + lane) * V; };
  auto in = [&](int i) { return col(i) < p.D; };
  const F2 zero = f2(0.0f, 0.0f);
  F2 w[E / 2], dw[E / 2], db[E / 2];
#pragma unroll
  for (int j = 0; j < E / 2; ++j) dw[j] = db[j] = zero;
  load_pairs<float, V, NV>(w, [&](int i) { return p.w + col(i); }, in);
  // vector i of an array (0: x, 1: dy, 2: dresid) of this thread's row in a stage
  const int row_bytes = Shape::kShare ? Shape::shared_row(p.D) : 0,
            array_bytes = Shape::pieces(p.D * (int)sizeof(T));
  auto slot = [&](int stage, int array, int i, long long row) -> unsigned char* {
    const int size = array == 2 ? Shape::kR : Shape::kX;
    int at;
    if constexpr (Shape::kOwn)
      at = (stage * Shape::kThread + array * NV * Shape::kX + i * size) * kThreads +
           (int)threadIdx.x * size;
    else
      at = (stage * rpb + group) * row_bytes + array * array_bytes +
           (array == 2 ? row_shift<float>(row, p.D) : row_shift<T>(row, p.D)) +
           (i * tpr + lane) * size;
    return ln_smem + at;
  };
  const T *x = static_cast<const T*>(p.x), *dy = static_cast<const T*>(p.dy);
  auto fetch = [&](long long row, int stage) {
    if (row < p.rows) {
      if constexpr (Shape::kOwn) {
        const size_t off = (size_t)row * p.D + lane * V;
        const T *fx = x + off, *fg = dy + off;
        const float* fr = p.dresid + off;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (in(i)) {
            copy_async<Shape::kX>(slot(stage, 0, i, row), fx + i * tpr * V);
            copy_async<Shape::kX>(slot(stage, 1, i, row), fg + i * tpr * V);
            if (p.dresid) copy_async<Shape::kR>(slot(stage, 2, i, row), fr + i * tpr * V);
          }
        }
      } else {
        unsigned char* s = ln_smem + (stage * rpb + group) * row_bytes;
        copy_row_pieces<kSub>(s, x, row, p.D, p.rows, lane, tpr);
        copy_row_pieces<kSub>(s + array_bytes, dy, row, p.D, p.rows, lane, tpr);
        if (p.dresid)
          copy_row_pieces<kSub>(s + 2 * array_bytes, p.dresid, row, p.D, p.rows, lane, tpr);
      }
    }
    umma::cp_async_commit();
  };
  const float inv_d = 1.0f / p.D;
  const long long step = (long long)gridDim.x * rpb;
  long long row = (long long)blockIdx.x * rpb + group;
  if constexpr (Shape::kAhead) {
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(row + k * step, k);
  }
  float mean = 0.0f, rstd = 0.0f;
  if (row < p.rows) mean = p.mean[row], rstd = p.rstd[row];
  int buf = 0, stage = 0;
  const int after = kSub ? group % (32 / tpr) : 0;
  for (; row < p.rows + after; row += step) {
    const bool live = !kSub || row < p.rows;
    auto inside = [&](int i) { return live && in(i); };
    const size_t off = (size_t)row * p.D;
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (row + step < p.rows) next_mean = p.mean[row + step], next_rstd = p.rstd[row + step];
    F2 xh[E / 2], g[E / 2];
    if constexpr (Shape::kAhead) umma::cp_async_wait<kStages - 2>();
    if constexpr (Shape::kShare) row_barrier(warp, row_warps);  // and the row before is done with
    auto input = [&](const T* from, int array) {
      return [=](int i) {
        if constexpr (Shape::kAhead) return reinterpret_cast<const T*>(slot(stage, array, i, row));
        else return from + off + col(i);
      };
    };
    load_pairs<T, V, NV>(xh, input(x, 0), inside);
    load_pairs<T, V, NV>(g, input(dy, 1), inside);
    // into the slot of the row before
    if constexpr (Shape::kAhead)
      fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
    F2 s0 = zero, s1 = zero;
    const F2 nm = f2(-mean, -mean), r2 = f2(rstd, rstd);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const F2 t = g[j] * w[j];
      xh[j] = (xh[j] + nm) * r2;
      s0 = s0 + t;
      s1 = f2_fma(t, xh[j], s1);
      dw[j] = f2_fma(g[j], xh[j], dw[j]);
      db[j] = db[j] + g[j];
    }
    float s[2] = {f2_get(s0).x + f2_get(s0).y, f2_get(s1).x + f2_get(s1).y};
    row_sum<2, kSub>(s, red[buf], warp, wr, row_warps, tpr);
    buf ^= 1;
    const F2 c0 = f2(-s[0] * inv_d, -s[0] * inv_d), c1 = f2(-s[1] * inv_d, -s[1] * inv_d);
#pragma unroll
    for (int j = 0; j < E / 2; ++j)  // t - mean(t) - xh mean(t xh), times s below
      g[j] = f2_fma(xh[j], c1, f2_fma(g[j], w[j], c0));
    if (p.dresid) {
      load_pairs<float, V, NV>(
          xh,
          [&](int i) {
            if constexpr (Shape::kAhead) return reinterpret_cast<const float*>(slot(stage, 2, i, row));
            else return p.dresid + off + col(i);
          },
          inside);
#pragma unroll
      for (int j = 0; j < E / 2; ++j) g[j] = f2_fma(g[j], r2, xh[j]);
    } else {
#pragma unroll
      for (int j = 0; j < E / 2; ++j) g[j] = g[j] * r2;
    }
    float* dx = p.dx + off + lane * V;
    store_pairs<V, NV>(g, [&](int i) { return dx + i * tpr * V; }, inside);
    mean = next_mean;
    rstd = next_rstd;
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  if constexpr (Shape::kAhead) umma::cp_async_wait<0>();
  // the groups of the CTA together, in order
  float* part = p.parts + (size_t)blockIdx.x * 2 * p.D;
  if (rpb == 1) {
    store_pairs<V, NV>(dw, [&](int i) { return part + col(i); }, in);
    store_pairs<V, NV>(db, [&](int i) { return part + p.D + col(i); }, in);
    return;
  }
  float* join = reinterpret_cast<float*>(ln_smem);  // [group][2][D]
  float* own = join + group * 2 * p.D;
  __syncthreads();
  store_pairs<V, NV>(dw, [&](int i) { return own + col(i); }, in);
  store_pairs<V, NV>(db, [&](int i) { return own + p.D + col(i); }, in);
  __syncthreads();
#pragma unroll 4
  for (int c = threadIdx.x * V; c < 2 * p.D; c += kThreads * V) {
    float s[V], o[V];
    load_f32<V>(join + c, s);
    for (int k = 1; k < rpb; ++k) {
      load_f32<V>(join + k * 2 * p.D + c, o);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += o[e];
    }
    store_f32<V>(part + c, s);
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
