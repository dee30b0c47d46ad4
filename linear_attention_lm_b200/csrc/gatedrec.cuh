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

// a = sigmoid(g) and n = 1 - a.  The smaller of the two is t = e / (1 + e) with
// e = exp(-|g|), the other is its complement to 1.  t is off by about 2^-21 + |g| 2^-23
// of itself: the hardware's 2^x and reciprocal (2^-22 and 2^-23), the rounding of the
// exponent, which grows with |g|, and that of the product; beyond |g| = 87 it is 0.
//
// Just below 1 fp32 has steps of 2^-24, so a alone would hold a slow decay's rate n only
// to 2^-25 (0.07% at a logit of 10, up to a quarter at 16), the same way at every token of a
// constant gate.  What decays a state takes the rate from n instead: the map of a lane's
// tokens by map_kept, the walk token by token by gate_rest.  What stays is the rounding
// of the fp32 state itself, at each update.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
struct Gate {
  float a, n;
};
__device__ __forceinline__ Gate gate_of(float g) {
  const float e = ex2_approx(-1.4426950408889634f * fabsf(g));
  const float t = e * rcp_approx(1.0f + e);
  const float u = __fsub_rn(1.0f, t);  // of the rounded t, not contracted with its product
  return g >= 0.0f ? Gate{u, t} : Gate{t, u};
}
struct Gate2 {
  F2 a, n;
};
__device__ __forceinline__ Gate2 gate_of(F2 g2) {
  const float2 g = f2_get(g2);
  const float ex = ex2_approx(-1.4426950408889634f * fabsf(g.x));
  const float ey = ex2_approx(-1.4426950408889634f * fabsf(g.y));
  const F2 e = f2(ex, ey), one = f2(1.0f, 1.0f);
  const float2 d = f2_get(e + one);
  const F2 t2 = e * f2(rcp_approx(d.x), rcp_approx(d.y));
  const float2 t = f2_get(t2), u = f2_get(f2_fma(t2, f2(-1.0f, -1.0f), one));
  const bool px = g.x >= 0.0f, py = g.y >= 0.0f;
  return Gate2{f2(px ? u.x : t.x, py ? u.y : t.y), f2(px ? t.x : u.x, py ? t.y : u.y)};
}
// What the rounded a leaves out: 1 - n = a + gate_rest, exactly (0 where a is the smaller
// of the two).
__device__ __forceinline__ float gate_rest(const Gate& g) {
  return __fsub_rn(__fsub_rn(1.0f, g.a), g.n);
}
__device__ __forceinline__ F2 gate_rest(const Gate2& g) {
  const F2 one = f2(1.0f, 1.0f), minus = f2(-1.0f, -1.0f);
  return f2_fma(g.n, minus, f2_fma(g.a, minus, one));
}

// How the sequence is cut: a lane takes S tokens of two channels; a warp G groups of
// lanes, each with the next S tokens of the same 64 / G channels; a CTA kGrWarps
// warps, one after another (a tile of kGrWarps G S tokens), and a cluster of N CTAs
// walks the sequence N tiles at a time.  Each lane forms its tokens' map
// h -> A h + H (A the product of its gates, H its end state from zero); the maps
// meet in a warp by shuffles, in a CTA in its shared memory and in a cluster in
// every CTA's shared memory; then every lane knows the state that enters its
// tokens and runs them again from its registers.  Inputs are read once: each warp
// copies its own tokens of the next tiles into a ring of kGrStages slots
// (cp.async), so loads run ahead of the barriers and hold no registers.
//
// What bounds it: the latency of a round.  About 26 instructions per value forward and
// 46 in the gradient (the gate alone has two special-function and ten other
// instructions) fill 56 and 50% of the issue slots, with 13 warps per SM between the
// barriers of a round, on 86% of the SMs (256 CTAs of 296).  8 x 2048 x 1024 bf16, 101
// MB: 24.2 us (4.2 TB/s; a copy of as many bytes 19 us); its gradient, 235 MB, 48.8 us
// (4.8 TB/s); 4 x 2048 x 1024 fp32 22.0 and 38.1 us.  One thread per channel took 1221
// and (padded batch) 2194 us; loads into registers one tile ahead 39.0 and 64.8 us.
// 1 x 16384 x 1024 (N = 8): 32.0 us, of which the exchanges between CTAs, about 0.9 us
// per round, are 7.  Odd bf16 widths, whose copies are not asynchronous, take 69 and
// 107 instructions per value and wait for them: 8 x 2048 x 999 76 and 106 us.
constexpr int kGrWarps = 8;
constexpr int kGrThreads = 32 * kGrWarps;
constexpr int kGrStages = 3;
constexpr int kGrMaxCluster = 8;
constexpr int kGrMaxD = 1 << 20;  // 32-bit offsets inside a tile of at most 512 tokens

// A map of two channels per lane in shared memory: A, H of the one, of the other
struct GrMap {
  F2 A, H;
};
__device__ __forceinline__ GrMap map_one() { return GrMap{f2(1.0f, 1.0f), f2(0.0f, 0.0f)}; }
__device__ __forceinline__ void map_store(ulonglong2* p, const GrMap& m) {
  *p = make_ulonglong2(m.A.v, m.H.v);
}
__device__ __forceinline__ GrMap map_load(const ulonglong2* p) {
  const ulonglong2 v = *p;
  return GrMap{F2{v.x}, F2{v.y}};
}
__device__ __forceinline__ void map_then(GrMap& m, const GrMap& next) {
  m.H = f2_fma(next.A, m.H, next.H);
  m.A = m.A * next.A;
}
// after prev
__device__ __forceinline__ void map_after(GrMap& m, const GrMap& prev) {
  m.H = f2_fma(m.A, prev.H, m.H);
  m.A = m.A * prev.A;
}
__device__ __forceinline__ F2 f2_shfl(F2 a, int src) {
  const float2 v = f2_get(a);
  return f2(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src));
}
// The maps of a warp's G groups of lanes in the order of the scan (o: this
// lane's position; kBack: from the last group): `m` becomes that of the groups up
// to this one, the result is that of the groups before.
template <int G, bool kBack>
__device__ __forceinline__ GrMap map_scan_groups(GrMap& m, int o, int lane) {
  constexpr int W = 32 / G;
  GrMap before = map_one();
#pragma unroll
  for (int d = 1; d < G; d *= 2) {
    const int src = (kBack ? lane + d * W : lane - d * W) & 31;
    const GrMap prev{f2_shfl(m.A, src), f2_shfl(m.H, src)};
    if (o >= d) {
      if (d == 1) before = prev;
      else map_after(before, prev);
      map_after(m, prev);
    }
  }
  return before;
}
__device__ __forceinline__ void map_apply(F2& h, const GrMap& m) { h = f2_fma(m.A, h, m.H); }
// What a product of gates leaves out of 1, with one more gate 1 - n.
__device__ __forceinline__ F2 map_lost(F2 lost, F2 n) {
  return f2_fma(n, f2_fma(lost, f2(-1.0f, -1.0f), f2(1.0f, 1.0f)), lost);
}
// The product A of a lane's gates, from what it leaves out where that is under a half:
// one rounding for all the lane's tokens, not one for each (8 x 2048 x 1024 bf16: 24.2
// us, 24.1 without; 25.3 with what is left out summed from n times A).
__device__ __forceinline__ F2 map_kept(F2 A, F2 lost) {
  const float2 p = f2_get(A), l = f2_get(lost);
  return f2(l.x < 0.5f ? 1.0f - l.x : p.x, l.y < 0.5f ? 1.0f - l.y : p.y);
}

// Maps of a CTA's warps and of a cluster's CTAs, two sets in turn.  The CTAs send
// each other their maps with stores that complete on the receiver's barrier of
// the set (a cluster barrier would also wait for the outputs' stores to global
// memory: 29.1 against 27.0 us at N = 2, 8 x 2048 x 1024 bf16).  A set is written again two rounds later: a CTA
// sends in round k + 2 when it has received round k + 1 of every CTA, and each
// sent that when all its warps had read the set of round k.
struct GrShared {
  ulonglong2 warp[2][kGrWarps][32];
  ulonglong2 cta[2][kGrMaxCluster][32];
  uint64_t bar[2];
  int len;
  int pad[11];
};
template <int G>
__device__ __forceinline__ uint32_t gr_round_bytes(int N) {
  return (uint32_t)N * (32 / G) * 16;
}

// Before the first round; also: every CTA of the cluster has started.
template <int G>
__device__ __forceinline__ void gr_cluster_begin(GrShared& sh, int N) {
  if (N == 1) return;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) umma::mbar_init(&sh.bar[i], 1);
    umma::fence_mbar_init();
#pragma unroll
    for (int i = 0; i < 2; ++i) umma::mbar_arrive_expect_tx(&sh.bar[i], gr_round_bytes<G>(N));
  }
  __syncwarp();
  umma::cluster_sync();
}

// After the last round: no CTA leaves before the others' sends to it (or their
// giving up), and every thread of the cluster has read h0.
__device__ __forceinline__ void gr_cluster_end(int N, bool ok) {
  if (!ok) record_device_error(BASED_ERR_TIMEOUT);
  __syncwarp();
  if (N > 1) umma::cluster_sync();
  else __syncthreads();
  if (!ok) {  // sends that this CTA did not wait for have long been issued: let them land
    const uint64_t t0 = umma::global_timer_ns();
    while (umma::global_timer_ns() - t0 < 100000) {
    }
  }
}

// One round k: every lane of the cluster gives its map `mine`.  w, r and o are the
// positions of the warp in its CTA, of the CTA in its cluster and of the lane's
// group in its warp in the order of the scan, to(r) the rank of the CTA at
// position r, l the lane's place in its group.  h: the state that enters the round;
// on return the state that leaves it, and `enter` the one that enters this lane's
// tokens.  False: a wait was given up (and every later one is).
template <int G, bool kBack, typename Rank>
__device__ __forceinline__ bool gr_round(GrShared& sh, int k, int w, int r, int o, int N, int lane,
                                         GrMap mine, F2& h, F2& enter, bool ok, Rank to) {
  const int buf = k & 1, l = lane % (32 / G);
  const GrMap groups = map_scan_groups<G, kBack>(mine, o, lane);
  if (G == 1 || o == G - 1) map_store(&sh.warp[buf][w][l], mine);
  __syncthreads();
  if (N > 1) {
    if (w < N) {  // the CTA's map, to the CTA at position w
      GrMap all = map_load(&sh.warp[buf][0][l]);
#pragma unroll
      for (int i = 1; i < kGrWarps; ++i) map_then(all, map_load(&sh.warp[buf][i][l]));
      if (o == 0 && !(k == 0 && w == 1 && stall_test(kStallGatedrec)))
        umma::st_async_16(umma::cluster_addr(&sh.cta[buf][r][l], (uint32_t)to(w)), all.A.v, all.H.v,
                          umma::cluster_addr(&sh.bar[buf], (uint32_t)to(w)));
    }
    if (ok) ok = umma::mbar_wait_cluster_inline(&sh.bar[buf], (k >> 1) & 1);
    if (threadIdx.x == 0) {  // for round k + 2
      if (ok) umma::mbar_arrive_expect_tx(&sh.bar[buf], gr_round_bytes<G>(N));
      else umma::mbar_expect_tx(&sh.bar[buf], gr_round_bytes<G>(N));  // no wait: bytes that still come
    }
    for (int i = 0; i < N; ++i) {
      if (i == r) enter = h;
      map_apply(h, map_load(&sh.cta[buf][i][l]));
    }
#pragma unroll
    for (int i = 0; i < kGrWarps - 1; ++i)
      if (i < w) map_apply(enter, map_load(&sh.warp[buf][i][l]));
  } else {
#pragma unroll
    for (int i = 0; i < kGrWarps; ++i) {
      if (i == w) enter = h;
      map_apply(h, map_load(&sh.warp[buf][i][l]));
    }
  }
  if (G > 1) map_apply(enter, groups);
  return ok;
}
static_assert(kGrMaxCluster <= kGrWarps, "warp i sends to the CTA at position i");

// Copies the G S tokens x 64 / G channels of a warp (row length D, from token t0 on)
// into `slot`; tokens from `end` on and channels from `cols` on become zero.  Token
// g S + s lies in row s G + g, so that the G groups of a warp read G rows side by
// side.  CW bytes at a time: the widest size that divides a row.  Rows of an odd
// number of bf16 have no asynchronous copy and are copied through registers.
template <typename T, int S, int G, int CW>
__device__ __forceinline__ void gr_fetch(T* slot, const T* src, int D, int t0, int end, int cols,
                                         int lane) {
  constexpr int kCols = 64 / G;
  constexpr int E = CW / (int)sizeof(T), RC = kCols / E;  // elements per copy, copies per row
  auto copy = [](T* to, const T* from, bool in) {
    if constexpr (CW == 16) umma::cp_async16(to, from, in);
    else if constexpr (CW >= 4) umma::cp_async_small<CW>(to, from, in);
    else *to = in ? *from : from_f32<T>(0.0f);
  };
  if constexpr (CW >= 4 && RC <= 32) {  // every token inside: a start and constant steps
    constexpr int R = 32 / RC;  // rows per copy instruction
    static_assert(RC <= 32 && (S % R == 0 || R % S == 0), "the step of a row is a constant");
    if (t0 + G * S <= end) {
      const int row = lane / RC, col = lane % RC * E;
      const bool in = col < cols;
      const T* from = src + (in ? (size_t)(t0 + row) * D + col : 0);
      T* to = slot + (row % S * G + row / S) * kCols + col;
      const size_t step = in ? (size_t)R * D : 0;
#pragma unroll
      for (int i = 0; i < S * G / R; ++i, from += step)
        copy(to + (i * R % S * G + i * R / S) * kCols, from, in);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < S * 64 / E / 32; ++i) {
    const int n = i * 32 + lane, row = n / RC, col = n % RC * E;
    const bool in = t0 + row < end && col < cols;
    copy(slot + (row % S * G + row / S) * kCols + col,
         src + (in ? (size_t)(t0 + row) * D + col : 0), in);
  }
}

// Length of sequence b; -1 (and a recorded error) if the array's entry is not in
// [0, L].  One thread reads it for the CTA, whose barriers then agree.
__device__ __forceinline__ int gr_length(GrShared& sh, const long long* lengths, int b, int L) {
  if (!lengths) return L;
  if (threadIdx.x == 0) {
    const long long n = lengths[b];
    const bool in = n >= 0 && n <= L;
    if (!in) record_device_error(BASED_ERR_INVALID_ARG);
    sh.len = in ? (int)n : -1;
  }
  __syncthreads();
  return sh.len;
}

// Two channels of an fp32 [.., D] row at p; kPair: rows start at even elements.
template <bool kPair>
__device__ __forceinline__ F2 gr_load(const float* p, bool two) {
  if constexpr (kPair) return load_pair(p);
  else return f2(p[0], two ? p[1] : 0.0f);
}
template <bool kPair, typename T>
__device__ __forceinline__ void gr_store(T* p, F2 v, bool two) {
  if constexpr (kPair) store_pair(p, v);
  else store_ends(p, v, two);
}

struct GrFwdParams {
  const void *x, *g;
  void* y;
  const float* h0;
  float *h_last, *h_chunks;
  const long long* lengths;
  int L, D, n_blk, N;  // n_blk: channel blocks of a sequence; N: CTAs per cluster
};

template <typename T, int G>
struct GrFwdShape {
  static constexpr int S = 32 / (int)sizeof(T);  // a ring slot of x and g: 4 KiB per warp
  static constexpr int kTile = S * G * kGrWarps;
  static constexpr int kSlot = 2 * S * 64;  // elements
  static constexpr size_t kSmem = sizeof(GrShared) + sizeof(T) * kGrWarps * kGrStages * kSlot;
  static_assert(kGrChunk % S == 0 && kTile % kGrChunk == 0, "chunks start with a warp's tokens");
};

// Rounds that lie past the end of a sequence are not walked: their outputs are
// zeros, written at the end.
template <typename T, int G, int CW>
__global__ void __launch_bounds__(kGrThreads, 2) gatedrec_fwd_kernel(const GrFwdParams p) {
  using Shape = GrFwdShape<T, G>;
  constexpr int S = Shape::S, kTile = Shape::kTile, kCols = 64 / G;
  constexpr bool kPair = CW > (int)sizeof(T);
  extern __shared__ __align__(16) unsigned char gr_smem[];
  GrShared& sh = *reinterpret_cast<GrShared*>(gr_smem);
  gr_cluster_begin<G>(sh, p.N);
  umma::grid_dep_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane / (32 / G), pair = lane % (32 / G) * 2;
  T* ring = reinterpret_cast<T*>(gr_smem + sizeof(GrShared)) + w * kGrStages * Shape::kSlot;
  const int rank = blockIdx.x % p.N, cid = blockIdx.x / p.N;
  const int b = cid / p.n_blk, c0 = cid % p.n_blk * kCols, c = c0 + pair;
  const int len = gr_length(sh, p.lengths, b, p.L), end = max(len, 0);
  const bool live = c < p.D && len >= 0, two = c + 1 < p.D;
  const int cols = min(p.D - c0, kCols);
  const T* x = static_cast<const T*>(p.x) + (size_t)b * p.L * p.D + c0;
  const T* g = static_cast<const T*>(p.g) + (size_t)b * p.L * p.D + c0;
  T* y = static_cast<T*>(p.y) + (size_t)b * p.L * p.D;
  const int n_chunks = (p.L + kGrChunk - 1) / kGrChunk;

  F2 h = f2(0.0f, 0.0f);
  if (live && p.h0) h = gr_load<kPair>(p.h0 + (size_t)b * p.D + c, two);

  const int rounds = (end + p.N * kTile - 1) / (p.N * kTile);
  auto fetch = [&](int k) {
    if (k < rounds) {
      T* slot = ring + k % kGrStages * Shape::kSlot;
      const int t0 = (k * p.N + rank) * kTile + w * G * S;
      gr_fetch<T, S, G, CW>(slot, x, p.D, t0, end, cols, lane);
      gr_fetch<T, S, G, CW>(slot + S * 64, g, p.D, t0, end, cols, lane);
    }
    umma::cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kGrStages - 1; ++k) fetch(k);
  bool ok = true;
  for (int k = 0; k < rounds; ++k) {
    const int t0 = (k * p.N + rank) * kTile + (w * G + grp) * S;  // this lane's first token
    umma::cp_async_wait<kGrStages - 2>();
    __syncwarp();
    fetch(k + kGrStages - 1);  // into the slot read in the round before
    const T* xs = ring + k % kGrStages * Shape::kSlot + grp * kCols + pair;
    const T* gs = xs + S * 64;
    F2 a[S], u[S];  // h -> a h + u
    GrMap m = map_one();
    F2 lost = f2(0.0f, 0.0f);  // 1 less the product of the gates
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const Gate2 gt = gate_of(load_pair(gs + s * 64));
      a[s] = gt.a;
      u[s] = gt.n * load_pair(xs + s * 64);
      lost = map_lost(lost, gt.n);
    }
    if (t0 + S > end) {  // past the end: the identity
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (t0 + s >= end) {
          a[s] = f2(1.0f, 1.0f);
          u[s] = f2(0.0f, 0.0f);
        }
      lost = f2(1.0f, 1.0f);  // the product
    }
#pragma unroll
    for (int s = 0; s < S; ++s) map_then(m, GrMap{a[s], u[s]});
    m.A = map_kept(m.A, lost);
    F2 e;
    ok = gr_round<G, false>(sh, k, w, rank, grp, p.N, lane, m, h, e, ok, [](int r) { return r; });
    if (live) {
      if (p.h_chunks && t0 % kGrChunk == 0 && t0 < p.L)
        gr_store<kPair>(p.h_chunks + ((size_t)b * n_chunks + t0 / kGrChunk) * p.D + c,
                        t0 < end ? e : f2(0.0f, 0.0f), two);
      // the tile's outputs at 32-bit offsets from its first token
      T* out = y + (size_t)(k * p.N + rank) * kTile * p.D;
      uint32_t at = (uint32_t)((w * G + grp) * S) * p.D + c;
      if (t0 + S <= end) {
#pragma unroll
        for (int s = 0; s < S; ++s, at += p.D) {
          e = f2_fma(a[s], e, u[s]);
          gr_store<kPair>(out + at, e, two);
        }
      } else {
#pragma unroll
        for (int s = 0; s < S; ++s, at += p.D) {
          e = f2_fma(a[s], e, u[s]);
          if (t0 + s < p.L) gr_store<kPair>(out + at, t0 + s < end ? e : f2(0.0f, 0.0f), two);
        }
      }
    }
  }
  if (live) {
    for (int i = rounds * p.N * kTile + (rank * kGrWarps + w) * G + grp; i < p.L;
         i += p.N * kGrWarps * G)
      gr_store<kPair>(y + (size_t)i * p.D + c, f2(0.0f, 0.0f), two);
    if (p.h_chunks && rank == 0)
      for (int i = rounds * p.N * kTile / kGrChunk + w * G + grp; i < n_chunks; i += kGrWarps * G)
        gr_store<kPair>(p.h_chunks + ((size_t)b * n_chunks + i) * p.D + c, f2(0.0f, 0.0f), two);
  }
  gr_cluster_end(p.N, ok);
  if (p.h_last) {
    if (live && rank == 0 && w == 0 && grp == 0) gr_store<kPair>(p.h_last + (size_t)b * p.D + c, h, two);
  }
}

struct GrBwdParams {
  const void *x, *g, *dy;
  const float *h_chunks, *dh_last;
  float *dx, *dg, *dh0;
  const long long* lengths;
  int L, D, n_blk, N;
};

template <typename T, int G>
struct GrBwdShape {
  static constexpr int S = 16 / (int)sizeof(T);  // a ring slot of x, g and dy: 3 KiB per warp
  static constexpr int kTile = S * G * kGrWarps;
  static constexpr int kSlot = 3 * S * 64;
  static constexpr size_t kShared = sizeof(GrShared) + sizeof(ulonglong2) * 2 * kGrWarps * 32;
  static constexpr size_t kSmem = kShared + sizeof(T) * kGrWarps * kGrStages * kSlot;
};
template <typename T>
constexpr int kGrBwdMinG = sizeof(T) == 2 ? 1 : 2;  // whole chunks

// The same cut, walked from the end.  The state that enters a tile is the saved
// one, so the forward maps only have to meet inside the CTA; the gradient's maps
// l -> A l + Q go through the cluster.
template <typename T, int G, int CW>
__global__ void __launch_bounds__(kGrThreads, 2) gatedrec_bwd_kernel(const GrBwdParams p) {
  using Shape = GrBwdShape<T, G>;
  constexpr int S = Shape::S, kTile = Shape::kTile, kCols = 64 / G;
  static_assert(kTile % kGrChunk == 0, "the forward states of a tile start from a saved state");
  constexpr bool kPair = CW > (int)sizeof(T);
  extern __shared__ __align__(16) unsigned char gr_smem[];
  GrShared& sh = *reinterpret_cast<GrShared*>(gr_smem);
  auto fwd = reinterpret_cast<ulonglong2(*)[kGrWarps][32]>(gr_smem + sizeof(GrShared));
  gr_cluster_begin<G>(sh, p.N);
  umma::grid_dep_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane / (32 / G), pair = lane % (32 / G) * 2;
  T* ring = reinterpret_cast<T*>(gr_smem + Shape::kShared) + w * kGrStages * Shape::kSlot;
  const int rank = blockIdx.x % p.N, cid = blockIdx.x / p.N;
  const int b = cid / p.n_blk, c0 = cid % p.n_blk * kCols, c = c0 + pair;
  const int len = gr_length(sh, p.lengths, b, p.L), end = max(len, 0);
  const bool live = c < p.D && len >= 0, two = c + 1 < p.D;
  const int cols = min(p.D - c0, kCols);
  const size_t seq = (size_t)b * p.L * p.D;
  const T* x = static_cast<const T*>(p.x) + seq + c0;
  const T* g = static_cast<const T*>(p.g) + seq + c0;
  const T* dy = static_cast<const T*>(p.dy) + seq + c0;
  const int n_chunks = (p.L + kGrChunk - 1) / kGrChunk;
  const F2 zero = f2(0.0f, 0.0f), minus = f2(-1.0f, -1.0f);

  F2 l = zero;  // a_{t+1} l_{t+1} at the end of the round
  if (live && p.dh_last) l = gr_load<kPair>(p.dh_last + (size_t)b * p.D + c, two);

  const int rounds = (end + p.N * kTile - 1) / (p.N * kTile);
  auto first = [&](int k) { return ((rounds - 1 - k) * p.N + rank) * kTile; };  // the tile's token
  auto fetch = [&](int k) {
    if (k < rounds) {
      T* slot = ring + k % kGrStages * Shape::kSlot;
      const int t0 = first(k) + w * G * S;
      gr_fetch<T, S, G, CW>(slot, x, p.D, t0, end, cols, lane);
      gr_fetch<T, S, G, CW>(slot + S * 64, g, p.D, t0, end, cols, lane);
      gr_fetch<T, S, G, CW>(slot + 2 * S * 64, dy, p.D, t0, end, cols, lane);
    }
    umma::cp_async_commit();
  };
  auto saved = [&](int k) {
    if (k >= rounds || !live || first(k) >= end) return zero;
    return gr_load<kPair>(p.h_chunks + ((size_t)b * n_chunks + first(k) / kGrChunk) * p.D + c, two);
  };
#pragma unroll
  for (int k = 0; k < kGrStages - 1; ++k) fetch(k);
  bool ok = true;
  F2 next = saved(0);
  for (int k = 0; k < rounds; ++k) {
    const int t0 = first(k) + (w * G + grp) * S;  // this lane's first token
    F2 h = next;  // the state that enters the tile
    next = saved(k + 1);
    umma::cp_async_wait<kGrStages - 2>();
    __syncwarp();
    fetch(k + kGrStages - 1);
    const T* xs = ring + k % kGrStages * Shape::kSlot + grp * kCols + pair;
    F2 a[S], n[S], xv[S], d[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const Gate2 gt = gate_of(load_pair(xs + (S + s) * 64));
      a[s] = gt.a;
      n[s] = gt.n;
      xv[s] = load_pair(xs + s * 64);
      d[s] = load_pair(xs + (2 * S + s) * 64);
    }
    if (t0 + S > end) {  // past the end: the identity (x and dy were copied as zero)
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (t0 + s >= end) {
          a[s] = f2(1.0f, 1.0f);
          n[s] = zero;
        }
    }
    GrMap f = map_one(), q;
    F2 lost = zero;  // 1 less the product of the gates
#pragma unroll
    for (int s = 0; s < S; ++s) {
      lost = f2_fma(n[s], f.A, lost);
      map_then(f, GrMap{a[s], n[s] * xv[s]});
    }
    q.A = f.A = map_kept(f.A, lost);
    q.H = zero;
#pragma unroll
    for (int s = S - 1; s >= 0; --s) q.H = a[s] * (q.H + d[s]);
    const GrMap groups = map_scan_groups<G, false>(f, grp, lane);
    if (grp == G - 1) map_store(&fwd[k & 1][w][pair / 2], f);
    // the scan runs from the last token: positions count from the end
    F2 e;
    ok = gr_round<G, true>(sh, k, kGrWarps - 1 - w, p.N - 1 - rank, G - 1 - grp, p.N, lane, q, l,
                           e, ok, [&](int r) { return p.N - 1 - r; });
    if (live) {
#pragma unroll
      for (int i = 0; i < kGrWarps - 1; ++i)
        if (i < w) map_apply(h, map_load(&fwd[k & 1][i][pair / 2]));
      map_apply(h, groups);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const F2 u = n[s] * xv[s];
        xv[s] = f2_fma(xv[s], minus, h);  // h_{t-1} - x_t
        h = f2_fma(a[s], h, u);
      }
      float *dx = p.dx + seq + (size_t)first(k) * p.D, *dg = p.dg + seq + (size_t)first(k) * p.D;
      uint32_t at = (uint32_t)((w * G + grp) * S + S - 1) * p.D + c;
      if (t0 + S <= end) {
#pragma unroll
        for (int s = S - 1; s >= 0; --s, at -= p.D) {
          const F2 lt = e + d[s], dxv = n[s] * lt;
          e = a[s] * lt;
          gr_store<kPair>(dx + at, dxv, two);
          gr_store<kPair>(dg + at, dxv * xv[s] * a[s], two);
        }
      } else {
#pragma unroll
        for (int s = S - 1; s >= 0; --s, at -= p.D) {
          const bool token = t0 + s < end;
          const F2 lt = e + d[s], dxv = n[s] * lt;
          e = a[s] * lt;  // past the end a is 1
          if (t0 + s < p.L) {  // zero past the end, whatever dh_last is
            gr_store<kPair>(dx + at, token ? dxv : zero, two);
            gr_store<kPair>(dg + at, token ? dxv * xv[s] * a[s] : zero, two);
          }
        }
      }
    }
  }
  if (live) {
    for (int i = rounds * p.N * kTile + (rank * kGrWarps + w) * G + grp; i < p.L;
         i += p.N * kGrWarps * G) {
      gr_store<kPair>(p.dx + seq + (size_t)i * p.D + c, zero, two);
      gr_store<kPair>(p.dg + seq + (size_t)i * p.D + c, zero, two);
    }
  }
  gr_cluster_end(p.N, ok);
  if (p.dh0) {
    if (live && rank == 0 && w == 0 && grp == 0) gr_store<kPair>(p.dh0 + (size_t)b * p.D + c, l, two);
  }
}

// Short sequences, or very many: a thread walks one sequence's two channels from
// end to end, the next kGrBatch tokens in flight.
constexpr int kGrShortThreads = 128, kGrBatch = 8;
static_assert(kGrChunk % kGrBatch == 0, "chunks start with a batch");

template <typename T, bool kPair>
struct GrWalk {
  int b, c, len;
  bool live, two;
  size_t seq;
  __device__ __forceinline__ GrWalk(const long long* lengths, int B, int L, int D) {
    const int pairs = (D + 1) / 2;
    const long long i = (long long)blockIdx.x * kGrShortThreads + threadIdx.x;
    live = i < (long long)B * pairs;
    b = live ? (int)(i / pairs) : 0;
    c = live ? (int)(i % pairs) * 2 : 0;
    two = c + 1 < D;
    len = L;
    if (lengths && live) {
      const long long n = lengths[b];
      if (n < 0 || n > L) {
        if (c == 0) record_device_error(BASED_ERR_INVALID_ARG);
        live = false;
      } else {
        len = (int)n;
      }
    }
    seq = (size_t)b * L * D + c;
  }
  // two channels of tensor p, `at` values on, as they lie in memory
  __device__ __forceinline__ void get(Pack<T, 2>& v, const void* p, size_t at) const {
    const T* q = static_cast<const T*>(p) + seq + at;
    if constexpr (kPair) {
      v.load(q);
    } else {
      v.e[0] = q[0];
      v.e[1] = two ? q[1] : q[0];
    }
  }
};
template <typename T>
__device__ __forceinline__ F2 to_pair(const Pack<T, 2>& v) { return load_pair(&v.e[0]); }

template <typename T, bool kPair>
__global__ void __launch_bounds__(kGrShortThreads) gatedrec_short_fwd_kernel(const GrFwdParams p,
                                                                             int B) {
  umma::grid_dep_wait();
  const GrWalk<T, kPair> k(p.lengths, B, p.L, p.D);
  if (!k.live) return;
  const size_t state = (size_t)k.b * p.D + k.c;
  const F2 zero = f2(0.0f, 0.0f);
  F2 h = p.h0 ? gr_load<kPair>(p.h0 + state, k.two) : zero;
  const int n_chunks = (p.L + kGrChunk - 1) / kGrChunk;
  float* chunk = p.h_chunks ? p.h_chunks + (size_t)k.b * n_chunks * p.D + k.c : nullptr;
  T* y = static_cast<T*>(p.y) + k.seq;
  Pack<T, 2> x[kGrBatch], g[kGrBatch];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s)
      if (t0 + s < k.len) {
        k.get(x[s], p.x, (size_t)(t0 + s) * p.D);
        k.get(g[s], p.g, (size_t)(t0 + s) * p.D);
      }
  };
  fetch(0);
  for (int t0 = 0; t0 < p.L; t0 += kGrBatch) {
    if (chunk && t0 % kGrChunk == 0) {
      gr_store<kPair>(chunk, t0 < k.len ? h : zero, k.two);
      chunk += p.D;
    }
    F2 a[kGrBatch], r[kGrBatch], u[kGrBatch];
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s) {
      const Gate2 gt = gate_of(to_pair(g[s]));
      a[s] = gt.a;
      r[s] = gate_rest(gt);
      u[s] = gt.n * to_pair(x[s]);
    }
    fetch(t0 + kGrBatch);
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s)
      if (t0 + s < p.L) {
        if (t0 + s < k.len) h = f2_fma(a[s], h, f2_fma(r[s], h, u[s]));
        gr_store<kPair>(y + (size_t)(t0 + s) * p.D, t0 + s < k.len ? h : zero, k.two);
      }
  }
  if (p.h_last) gr_store<kPair>(p.h_last + state, h, k.two);
}

// Dynamic shared memory: the state that enters each token, [L][threads] pairs.
template <typename T, bool kPair>
__global__ void __launch_bounds__(kGrShortThreads) gatedrec_short_bwd_kernel(const GrBwdParams p,
                                                                             int B) {
  extern __shared__ __align__(16) unsigned char gr_smem[];
  F2* before = reinterpret_cast<F2*>(gr_smem) + threadIdx.x;
  umma::grid_dep_wait();
  const GrWalk<T, kPair> k(p.lengths, B, p.L, p.D);
  if (!k.live) return;
  const size_t state = (size_t)k.b * p.D + k.c;
  const F2 zero = f2(0.0f, 0.0f), minus = f2(-1.0f, -1.0f);
  F2 h = k.len > 0 ? gr_load<kPair>(p.h_chunks + state, k.two) : zero;
  Pack<T, 2> x[kGrBatch], g[kGrBatch], d[kGrBatch];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s)
      if (t0 + s < k.len) {
        k.get(x[s], p.x, (size_t)(t0 + s) * p.D);
        k.get(g[s], p.g, (size_t)(t0 + s) * p.D);
      }
  };
  fetch(0);
  for (int t0 = 0; t0 < k.len; t0 += kGrBatch) {
    F2 a[kGrBatch], r[kGrBatch], u[kGrBatch];
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s) {
      const Gate2 gt = gate_of(to_pair(g[s]));
      a[s] = gt.a;
      r[s] = gate_rest(gt);
      u[s] = gt.n * to_pair(x[s]);
    }
    fetch(t0 + kGrBatch);
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s)
      if (t0 + s < k.len) {
        before[(t0 + s) * kGrShortThreads] = h;
        h = f2_fma(a[s], h, f2_fma(r[s], h, u[s]));
      }
  }
  F2 l = p.dh_last ? gr_load<kPair>(p.dh_last + state, k.two) : zero;
  float *dx = p.dx + k.seq, *dg = p.dg + k.seq;
  for (int t = p.L - 1; t >= k.len; --t) {
    gr_store<kPair>(dx + (size_t)t * p.D, zero, k.two);
    gr_store<kPair>(dg + (size_t)t * p.D, zero, k.two);
  }
  auto fetch_back = [&](int t1) {  // tokens t1 - 1, t1 - 2, ...
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s)
      if (t1 - 1 - s >= 0) {
        const size_t at = (size_t)(t1 - 1 - s) * p.D;
        k.get(x[s], p.x, at);
        k.get(g[s], p.g, at);
        k.get(d[s], p.dy, at);
      }
  };
  fetch_back(k.len);
  for (int t1 = k.len; t1 > 0; t1 -= kGrBatch) {
    F2 a[kGrBatch], n[kGrBatch], dv[kGrBatch], diff[kGrBatch];
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s) {
      const Gate2 gt = gate_of(to_pair(g[s]));
      a[s] = gt.a;
      n[s] = gt.n;
      dv[s] = to_pair(d[s]);
      diff[s] = f2_fma(to_pair(x[s]), minus, before[max(t1 - 1 - s, 0) * kGrShortThreads]);
    }
    fetch_back(t1 - kGrBatch);
#pragma unroll
    for (int s = 0; s < kGrBatch; ++s)
      if (t1 - 1 - s >= 0) {
        const size_t at = (size_t)(t1 - 1 - s) * p.D;
        const F2 lt = l + dv[s], dxv = n[s] * lt;
        l = f2_fma(a[s], lt, gate_rest(Gate2{a[s], n[s]}) * lt);
        gr_store<kPair>(dx + at, dxv, k.two);
        gr_store<kPair>(dg + at, dxv * diff[s] * a[s], k.two);
      }
  }
  if (p.dh0) gr_store<kPair>(p.dh0 + state, l, k.two);
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
    hv[e] = fmaf(gt.a, hv[e], fmaf(gate_rest(gt), hv[e], gt.n * xv.get(e)));
    xv.set(e, hv[e]);
  }
  store_f32<V>(h + i, hv);
  xv.store(y + i);
}

}  // namespace based
