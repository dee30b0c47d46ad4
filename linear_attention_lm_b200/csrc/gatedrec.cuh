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

// How the sequence is cut: lanes own V neighbouring channels, a warp S tokens, a
// CTA kGrWarps warps, one after another (a tile of T = 8 S tokens), and a cluster
// of N CTAs walks the sequence N tiles at a time.  A tile is read once, into
// registers.  Each warp forms its tokens' map h -> A h + H (A the product of its
// gates, H its end state from zero), the maps of the CTA's warps meet in shared
// memory and those of the cluster's CTAs in every CTA's shared memory (one
// cluster barrier per N tiles); then every warp knows the state that enters its
// tokens and runs them again from its registers.  The next tile's loads are
// issued before the barriers, so memory stays busy across them.
constexpr int kGrWarps = 8;
constexpr int kGrThreads = 32 * kGrWarps;
constexpr int kGrMaxCluster = 16;

template <typename T, int V>
struct GrShape {
  // about 128 bytes of x and g in flight per thread; T a multiple of kGrChunk
  static constexpr int S = V * sizeof(T) >= 8 ? 8 : 16;
  static constexpr int kTile = S * kGrWarps;
};

// V channels' maps as one shared-memory vector per lane
template <int V>
struct GrMap {
  float A[V], H[V];
};
template <int V>
__device__ __forceinline__ void map_store(float* p, const GrMap<V>& m) {
  if constexpr (V == 1) {
    *reinterpret_cast<float2*>(p) = make_float2(m.A[0], m.H[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      *reinterpret_cast<float4*>(p + 2 * i) = make_float4(m.A[i], m.H[i], m.A[i + 1], m.H[i + 1]);
  }
}
template <int V>
__device__ __forceinline__ GrMap<V> map_load(const float* p) {
  GrMap<V> m;
  if constexpr (V == 1) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    m.A[0] = v.x; m.H[0] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float4 v = *reinterpret_cast<const float4*>(p + 2 * i);
      m.A[i] = v.x; m.H[i] = v.y; m.A[i + 1] = v.z; m.H[i + 1] = v.w;
    }
  }
  return m;
}
// into CTA `rank` of the cluster, at the place that p has in this CTA
template <int V>
__device__ __forceinline__ void map_store_peer(float* p, uint32_t rank, const GrMap<V>& m) {
  const uint32_t at = umma::cluster_addr(p, rank);
#pragma unroll
  for (int i = 0; i < V; ++i)
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at + 8 * i), "f"(m.A[i]),
                 "f"(m.H[i])
                 : "memory");
}
// m, then next
template <int V>
__device__ __forceinline__ void map_then(GrMap<V>& m, const GrMap<V>& next) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    m.H[v] = fmaf(next.A[v], m.H[v], next.H[v]);
    m.A[v] *= next.A[v];
  }
}
template <int V>
__device__ __forceinline__ void map_apply(float (&h)[V], const GrMap<V>& m) {
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = fmaf(m.A[v], h[v], m.H[v]);
}

// Maps of a CTA's warps and of a cluster's CTAs, two sets in turn.  A set is
// written again two rounds later, behind a barrier that every reader of the
// first round has passed.
template <int V>
struct GrShared {
  float warp[2][kGrWarps][32 * 2 * V];
  float cta[2][kGrMaxCluster][32 * 2 * V];
};

// One round: every warp of the cluster gives its map `mine`, in the order of the
// scan (order index of this warp w, of this CTA r: position in the scan, not
// rank).  h: the state that enters the round; on return the state that leaves
// it, and `enter` the one that enters this warp's tokens.  `to(r)` is the rank
// of the CTA at position r.
template <int V, typename Rank>
__device__ __forceinline__ void gr_round(GrShared<V>& sh, int buf, int w, int r, int N, int lane,
                                         const GrMap<V>& mine, float (&h)[V], float (&enter)[V],
                                         Rank to) {
  map_store<V>(&sh.warp[buf][w][lane * 2 * V], mine);
  __syncthreads();
  GrMap<V> before, all;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    all.A[v] = before.A[v] = 1.0f;
    all.H[v] = before.H[v] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kGrWarps; ++i) {
    if (i == w) before = all;
    map_then<V>(all, map_load<V>(&sh.warp[buf][i][lane * 2 * V]));
  }
  if (N > 1) {
    for (int k = w; k < N; k += kGrWarps)
      map_store_peer<V>(&sh.cta[buf][r][lane * 2 * V], (uint32_t)to(k), all);
    umma::cluster_sync();
    for (int k = 0; k < N; ++k) {
      if (k == r) {
#pragma unroll
        for (int v = 0; v < V; ++v) enter[v] = h[v];
      }
      map_apply<V>(h, map_load<V>(&sh.cta[buf][k][lane * 2 * V]));
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) enter[v] = h[v];
    map_apply<V>(h, all);
  }
  map_apply<V>(enter, before);
}

struct GrFwdParams {
  const void *x, *g;
  void* y;
  const float* h0;
  float *h_last, *h_chunks;
  const long long* lengths;
  int L, D, n_blk, N;  // n_blk: channel blocks of a sequence; N: CTAs per cluster
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

// The number of rounds goes by L alone, never by what memory holds: every thread
// of a cluster reaches the same barriers.
template <typename T, int V>
__global__ void __launch_bounds__(kGrThreads, 2) gatedrec_fwd_kernel(const GrFwdParams p) {
  constexpr int S = GrShape<T, V>::S, kTile = GrShape<T, V>::kTile;
  __shared__ __align__(16) GrShared<V> sh;
  if (p.N > 1) umma::cluster_sync();  // every CTA has started before its shared memory is written
  umma::grid_dep_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.N, cid = blockIdx.x / p.N;
  const int b = cid / p.n_blk, c = (cid % p.n_blk * 32 + lane) * V;
  const int len = gr_length(p.lengths, b, p.L);
  const bool live = c < p.D && len >= 0;
  const int end = live ? len : 0;  // tokens this lane reads
  const size_t base = (size_t)b * p.L * p.D + c;
  const int n_chunks = (p.L + kGrChunk - 1) / kGrChunk;

  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.0f;
  if (live && p.h0) load_f32<V>(p.h0 + (size_t)b * p.D + c, h);

  Pack<T, V> xr[S], gr[S];
  auto fetch = [&](int t0) {
    const T* x = static_cast<const T*>(p.x) + base + (size_t)t0 * p.D;
    const T* g = static_cast<const T*>(p.g) + base + (size_t)t0 * p.D;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (t0 + s < end) {
        xr[s].load(x + (size_t)s * p.D);
        gr[s].load(g + (size_t)s * p.D);
      }
    }
  };
  int t0 = rank * kTile + w * S;
  fetch(t0);
  const int rounds = (p.L + p.N * kTile - 1) / (p.N * kTile);
  for (int k = 0; k < rounds; ++k, t0 += p.N * kTile) {
    float a[S][V], u[S][V];  // h -> a h + u; the identity past the end
    GrMap<V> m;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m.A[v] = 1.0f;
      m.H[v] = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool in = t0 + s < end;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gate gt = gate_of(gr[s].get(v));
        a[s][v] = in ? gt.a : 1.0f;
        u[s][v] = in ? gt.n * xr[s].get(v) : 0.0f;
        m.H[v] = fmaf(a[s][v], m.H[v], u[s][v]);
        m.A[v] *= a[s][v];
      }
    }
    if (k + 1 < rounds) fetch(t0 + p.N * kTile);
    float e[V];
    gr_round<V>(sh, k & 1, w, rank, p.N, lane, m, h, e, [](int r) { return r; });
    if (live && p.h_chunks && t0 % kGrChunk == 0 && t0 < p.L) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = t0 < end ? e[v] : 0.0f;
      store_f32<V>(p.h_chunks + ((size_t)b * n_chunks + t0 / kGrChunk) * p.D + c, o);
    }
    T* y = static_cast<T*>(p.y) + base + (size_t)t0 * p.D;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      Pack<T, V> o;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        e[v] = fmaf(a[s][v], e[v], u[s][v]);
        o.set(v, t0 + s < end ? e[v] : 0.0f);
      }
      if (live && t0 + s < p.L) o.store(y + (size_t)s * p.D);
    }
  }
  if (p.h_last) {
    __syncthreads();  // h_last may be h0: every warp has read it (other CTAs: the rounds' barriers)
    if (live && rank == 0 && w == 0) store_f32<V>(p.h_last + (size_t)b * p.D + c, h);
  }
}

struct GrBwdParams {
  const void *x, *g, *dy;
  const float *h_chunks, *dh_last;
  float *dx, *dg, *dh0;
  const long long* lengths;
  int L, D, n_blk, N;
};

template <typename T, int V>
struct GrBwdShape {
  // tiles of one chunk: the forward states of a tile start from its saved state
  static constexpr int S = kGrChunk / kGrWarps;
};

// The same cut, walked from the end.  The state that enters a tile is the saved
// one, so the forward maps only have to meet inside the CTA; the gradient's maps
// l -> A l + Q go through the cluster.
template <typename T, int V>
__global__ void __launch_bounds__(kGrThreads, 2) gatedrec_bwd_kernel(const GrBwdParams p) {
  constexpr int S = GrBwdShape<T, V>::S, kTile = S * kGrWarps;
  static_assert(kTile == kGrChunk, "one saved state per tile");
  __shared__ __align__(16) GrShared<V> sh;
  __shared__ __align__(16) float fwd[2][kGrWarps][32 * 2 * V];
  if (p.N > 1) umma::cluster_sync();
  umma::grid_dep_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.N, cid = blockIdx.x / p.N;
  const int b = cid / p.n_blk, c = (cid % p.n_blk * 32 + lane) * V;
  const int len = gr_length(p.lengths, b, p.L);
  const bool live = c < p.D && len >= 0;
  const int end = live ? len : 0;
  const size_t base = (size_t)b * p.L * p.D + c;
  const int n_chunks = (p.L + kGrChunk - 1) / kGrChunk;

  float l[V];  // a_{t+1} l_{t+1} at the end of the round
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = 0.0f;
  if (live && p.dh_last) load_f32<V>(p.dh_last + (size_t)b * p.D + c, l);

  Pack<T, V> xr[S], gr[S], dr[S];
  float hc[V];
  auto fetch = [&](int t0) {
    const size_t at = base + (size_t)t0 * p.D;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (t0 + s < end) {
        xr[s].load(static_cast<const T*>(p.x) + at + (size_t)s * p.D);
        gr[s].load(static_cast<const T*>(p.g) + at + (size_t)s * p.D);
        dr[s].load(static_cast<const T*>(p.dy) + at + (size_t)s * p.D);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) hc[v] = 0.0f;
    if (t0 < end)
      load_f32<V>(p.h_chunks + ((size_t)b * n_chunks + t0 / kGrChunk) * p.D + c, hc);
  };
  const int rounds = (p.L + p.N * kTile - 1) / (p.N * kTile);
  int t0 = (rounds - 1) * p.N * kTile + rank * kTile + w * S;
  if (rounds > 0) fetch(t0);
  for (int k = 0; k < rounds; ++k, t0 -= p.N * kTile) {
    float a[S][V], n[S][V], x[S][V], d[S][V];
    GrMap<V> f, q;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f.A[v] = 1.0f;
      f.H[v] = q.H[v] = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool in = t0 + s < end;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gate gt = gate_of(gr[s].get(v));
        a[s][v] = in ? gt.a : 1.0f;
        n[s][v] = in ? gt.n : 0.0f;
        x[s][v] = in ? xr[s].get(v) : 0.0f;
        d[s][v] = in ? dr[s].get(v) : 0.0f;
        f.H[v] = fmaf(a[s][v], f.H[v], n[s][v] * x[s][v]);
        f.A[v] *= a[s][v];
      }
    }
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = hc[v];
      q.A[v] = f.A[v];
    }
#pragma unroll
    for (int s = S - 1; s >= 0; --s)
#pragma unroll
      for (int v = 0; v < V; ++v) q.H[v] = a[s][v] * (q.H[v] + d[s][v]);
    if (k + 1 < rounds) fetch(t0 - p.N * kTile);
    map_store<V>(&fwd[k & 1][w][lane * 2 * V], f);
    // the scan runs from the last token: positions count from the end
    float e[V];
    gr_round<V>(sh, k & 1, kGrWarps - 1 - w, p.N - 1 - rank, p.N, lane, q, l, e,
                [&](int r) { return p.N - 1 - r; });
    for (int i = 0; i < w; ++i) map_apply<V>(h, map_load<V>(&fwd[k & 1][i][lane * 2 * V]));
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float u = n[s][v] * x[s][v];
        x[s][v] = h[v] - x[s][v];
        h[v] = fmaf(a[s][v], h[v], u);
      }
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
      float dx[V], dg[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float lt = e[v] + d[s][v];
        dx[v] = n[s][v] * lt;  // past the end n is 0
        e[v] = a[s][v] * lt;
        dg[v] = dx[v] * x[s][v] * a[s][v];
      }
      if (live && t0 + s < p.L) {
        const size_t at = base + (size_t)(t0 + s) * p.D;
        store_f32<V>(p.dx + at, dx);
        store_f32<V>(p.dg + at, dg);
      }
    }
  }
  if (p.dh0) {
    __syncthreads();  // dh0 may be dh_last, as above
    if (live && rank == 0 && w == 0) store_f32<V>(p.dh0 + (size_t)b * p.D + c, l);
  }
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
