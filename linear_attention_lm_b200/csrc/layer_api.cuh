// layer_api.cuh -- entry points of the operators around a mixer: layer norm,
// rotary positions, gated recurrence.  Part of based_api.cu's translation unit
// (included at its end; uses its launch and checking helpers).
#pragma once

#include "gatedrec.cuh"
#include "layernorm.cuh"
#include "rotary.cuh"

namespace {

inline bool dtype_ok(based_dtype_t dt) { return dt == BASED_F32 || dt == BASED_BF16; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Runs f(T{}, integral_constant<V>) for the type and the widest vector of at
// most 16 bytes whose V divides n (row starts are then multiples of it).
template <typename F>
based_status_t for_vector(based_dtype_t dt, long long n, F f) {
  using std::integral_constant;
  if (dt == BASED_F32) {
    if (n % 4 == 0) return f(float{}, integral_constant<int, 4>{});
    if (n % 2 == 0) return f(float{}, integral_constant<int, 2>{});
    return f(float{}, integral_constant<int, 1>{});
  }
  if (n % 8 == 0) return f(__nv_bfloat16{}, integral_constant<int, 8>{});
  if (n % 4 == 0) return f(__nv_bfloat16{}, integral_constant<int, 4>{});
  if (n % 2 == 0) return f(__nv_bfloat16{}, integral_constant<int, 2>{});
  return f(__nv_bfloat16{}, integral_constant<int, 1>{});
}

// Warps of a row of D values at E values per thread: a power of two.
inline int row_warps_for(int D, int E) {
  int w = 1;
  while ((long long)w * 32 * E < D) w *= 2;
  return w;
}

// Threads of a CTA for rows of row_warps warps, and the CTAs that run at once: one per
// SM of more than 256 threads (4000 x 8192 bf16 gradient: 70 us, 79 in two waves), two
// of 256, and more where a thread has only 8 values in flight (262144 x 64 bf16,
// forward: 31.0 us with two, 24.4 with four, 29.2 with six; gradient, whole
// vectors of four, 38.9 with two, 35.8 with three).
inline int row_threads(int row_warps) {
  return row_warps * 32 > kLnThreads ? row_warps * 32 : kLnThreads;
}
inline long long row_ctas(int threads, int per_sm = 2) {
  return (threads > kLnThreads ? 1LL : per_sm) * device_sm_count();
}

// Lanes of a row of up to 256 values at 8 per lane.
inline int row_lanes_for(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

template <typename T, int V, int E>
based_status_t launch_layernorm_fwd(LnFwdParams p, cudaStream_t st) {
  p.row_warps = row_warps_for(p.D, E);
  p.lanes = row_lanes_for(p.D);
  const int threads = row_threads(p.row_warps);
  const long long want = ceil_div(p.rows, threads / (ln_sub(E) ? p.lanes : p.row_warps * 32));
  const long long most = row_ctas(threads, E == 8 ? 4 : 2);
  const dim3 grid((unsigned)(want < most ? want : most));
  auto go = [&](auto kern) -> based_status_t {
    if (!launch_dependent(kern, grid, dim3(threads), 0, st, p)) return BASED_ERR_CUDA;
    return launch_status();
  };
  auto pick = [&](auto n) {
    constexpr int kN = decltype(n)::value;
    return p.residual ? go(layernorm_fwd_kernel<T, V, E, true, kN>)
                      : go(layernorm_fwd_kernel<T, V, E, false, kN>);
  };
  using std::integral_constant;
  if constexpr (E == 32 || (E == 16 && V < 4)) {
    if (threads == 512) return pick(integral_constant<int, 512>{});
  }
  if constexpr (E == 16 && V < 4) {
    if (threads == 1024) return pick(integral_constant<int, 1024>{});
  }
  return pick(integral_constant<int, 256>{});
}

struct LnBwdPlan {
  int E, row_warps, tpr, threads, parts;
};
LnBwdPlan plan_layernorm_bwd(long long rows, int D) {
  LnBwdPlan pl;
  pl.E = D <= 256 ? 8 : 16;
  pl.row_warps = row_warps_for(D, pl.E);
  pl.tpr = ln_sub(pl.E) ? row_lanes_for(D) : pl.row_warps * 32;
  pl.threads = row_threads(pl.row_warps);
  const long long want = ceil_div(rows, pl.threads / pl.tpr);
  const long long most = row_ctas(pl.threads, pl.E == 8 && D % 4 == 0 ? 3 : 2);
  pl.parts = (int)(want < most ? want : most);
  return pl;
}

template <typename T, int V, int E>
based_status_t launch_layernorm_bwd(LnBwdParams p, const LnBwdPlan& pl, float* dw, float* db,
                                    cudaStream_t st) {
  p.row_warps = pl.row_warps;
  p.lanes = pl.tpr;
  if (pl.parts > 0) {
    auto go = [&](auto n, auto row_warps) {
      constexpr int kN = decltype(n)::value;
      auto kern = layernorm_bwd_kernel<T, V, E, kN, decltype(row_warps)::value>;
      using Shape = LnBwdShape<T, V, E, kN>;
      const size_t smem = Shape::smem(pl.tpr, p.D);
      static_assert(Shape::most_smem() <= 226 * 1024, "beside the static shared memory");
      return set_smem(kern, Shape::most_smem()) &&
             launch_dependent(kern, dim3((unsigned)pl.parts), dim3(kN), smem, st, p);
    };
    constexpr std::integral_constant<int, 256> k256{};
    constexpr std::integral_constant<int, 512> k512{};
    constexpr std::integral_constant<int, 1024> k1024{};
    constexpr std::integral_constant<int, 0> any{};
    bool ok;
    if constexpr (E == 8) {
      ok = go(k256, std::integral_constant<int, 1>{});
    } else if constexpr (V == 4) {
      switch (pl.row_warps) {
        case 1: ok = go(k256, std::integral_constant<int, 1>{}); break;
        case 2: ok = go(k256, std::integral_constant<int, 2>{}); break;
        case 4: ok = go(k256, std::integral_constant<int, 4>{}); break;
        case 8: ok = go(k256, std::integral_constant<int, 8>{}); break;
        case 16: ok = go(k512, std::integral_constant<int, 16>{}); break;
        default: ok = go(k1024, std::integral_constant<int, 32>{});
      }
    } else {
      ok = pl.threads == 256   ? go(k256, any)
           : pl.threads == 512 ? go(k512, any)
                               : go(k1024, any);
    }
    if (!ok) return BASED_ERR_CUDA;
  }
  if (!launch_dependent(layernorm_parts_kernel, dim3((unsigned)ceil_div(2LL * p.D, 32)),
                        dim3(32, 32), 0, st, (const float*)p.parts, pl.parts, p.D, dw, db))
    return BASED_ERR_CUDA;
  return launch_status();
}

based_status_t check_layernorm(long long rows, int D, based_dtype_t dt) {
  if (rows < 0 || D <= 0 || !dtype_ok(dt)) return BASED_ERR_INVALID_ARG;
  if (D > kLnMaxD || rows > (1LL << 47)) return BASED_ERR_UNSUPPORTED;
  return BASED_OK;
}

based_status_t launch_rotary(RotaryParams p, int B, bool interleaved, based_dtype_t dt,
                             cudaStream_t st) {
  // 2V values per chunk in two vectors: V has to divide the head and, where the
  // pairs are halves apart, half of the turned part
  const long long n = interleaved ? p.D : std::gcd(p.D, p.rot / 2);
  return for_vector(dt, n, [&](auto t, auto v) -> based_status_t {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    RotaryParams r = p;
    r.rot_chunks = (int)ceil_div(r.rot, 2 * V);
    r.chunks = r.rot_chunks;
    const bool in_place = (!r.H_q || r.q == r.q_out) && (!r.H_k || r.k == r.k_out);
    if (!in_place)
      r.chunks = (int)(interleaved ? ceil_div(r.D, 2 * V)
                                   : r.rot_chunks + ceil_div(r.D - r.rot, 2 * V));
    r.items = (long long)B * r.L * r.chunks;
    const long long blocks = ceil_div(r.items, kRotThreads);
    if (blocks > 0x7fffffffLL) return BASED_ERR_UNSUPPORTED;
    // a thread's sines and cosines serve 16 heads (8 x 32 heads x 2048 x 64 bf16: 25.1 us,
    // 25.8 with 8, 27.0 with 4), fewer where that leaves SMs idle (128 x 32 heads x 1 x 64:
    // 6.5 us with 16, 3.1 with 4)
    r.heads_per_cta = 16;
    while (r.heads_per_cta > 1 &&
           blocks * ceil_div(r.H_q + r.H_k, r.heads_per_cta) < 2LL * device_sm_count())
      r.heads_per_cta /= 2;
    const dim3 grid((unsigned)blocks, (unsigned)ceil_div(r.H_q + r.H_k, r.heads_per_cta));
    if (grid.y > 65535) return BASED_ERR_UNSUPPORTED;
    const bool ok = interleaved ? launch_dependent(rotary_kernel<T, V, true>, grid,
                                                   dim3(kRotThreads), 0, st, r)
                                : launch_dependent(rotary_kernel<T, V, false>, grid,
                                                   dim3(kRotThreads), 0, st, r);
    if (!ok) return BASED_ERR_CUDA;
    return launch_status();
  });
}

based_status_t rotary_impl(const void* q, const void* k, void* q_out, void* k_out,
                           const double* freqs, const long long* pos, long long pos0, int B,
                           int H_q, int H_k, int L, int D, int rot_dim,
                           based_rotary_layout_t layout, float mscale, bool inverse,
                           based_dtype_t dt, based_stream_t stream) {
  if (B < 0 || H_q < 0 || H_k < 0 || L < 0 || D <= 0 || rot_dim <= 0 || rot_dim > D ||
      rot_dim % 2 != 0 || !dtype_ok(dt) || !isfinite(mscale))
    return BASED_ERR_INVALID_ARG;
  if (layout != BASED_ROTARY_HALF && layout != BASED_ROTARY_INTERLEAVED)
    return BASED_ERR_INVALID_ARG;
  if (!pos && pos0 < 0) return BASED_ERR_INVALID_ARG;
  if (!pos && pos0 > (1LL << 31) - L) return BASED_ERR_UNSUPPORTED;
  const bool no_q = B == 0 || H_q == 0 || L == 0, no_k = B == 0 || H_k == 0 || L == 0;
  based_status_t s;
  if ((s = check_tensor(q, no_q)) != BASED_OK) return s;
  if ((s = check_tensor(q_out, no_q)) != BASED_OK) return s;
  if ((s = check_tensor(k, no_k)) != BASED_OK) return s;
  if ((s = check_tensor(k_out, no_k)) != BASED_OK) return s;
  if (no_q && no_k) return BASED_OK;
  if ((long long)B * L > (1LL << 40) || (long long)H_q + H_k > (1 << 19) || D > (1 << 16))
    return BASED_ERR_UNSUPPORTED;
  if (!freqs || (reinterpret_cast<uintptr_t>(freqs) & 7u) ||
      (reinterpret_cast<uintptr_t>(pos) & 7u))
    return BASED_ERR_INVALID_ARG;
  RotaryParams p{};
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
  p.freqs = freqs; p.pos_arr = pos; p.pos0 = pos0;
  p.L = L; p.D = D; p.rot = rot_dim; p.H_q = H_q; p.H_k = H_k;
  p.mscale = mscale; p.sign = inverse ? -1.0f : 1.0f;
  return launch_rotary(p, B, layout == BASED_ROTARY_INTERLEAVED, dt,
                       static_cast<cudaStream_t>(stream));
}

based_status_t check_gatedrec(const void* x, const void* g, const void* y, const void* lengths,
                              int B, int L, int D, based_dtype_t dt) {
  if (B < 0 || L < 0 || D <= 0 || !dtype_ok(dt)) return BASED_ERR_INVALID_ARG;
  const bool empty = (long long)B * L == 0;
  based_status_t s;
  for (const void* t : {x, g, y})
    if ((s = check_tensor(t, empty)) != BASED_OK) return s;
  if (reinterpret_cast<uintptr_t>(lengths) & 7u) return BASED_ERR_INVALID_ARG;
  if ((long long)B * ceil_div(D, 16) > 0x7fffffffLL || L > 0x7fff0000 || D > kGrMaxD)
    return BASED_ERR_UNSUPPORTED;
  return BASED_OK;
}

// Runs f(T{}, integral_constant<CW>) with the copy size: the widest of 16, 8, 4
// and 2 bytes that divides a row of D values.
template <typename F>
based_status_t for_copies(based_dtype_t dt, int D, F f) {
  return for_vector(dt, D, [&](auto t, auto v) {
    using T = decltype(t);
    return f(T{}, std::integral_constant<int, decltype(v)::value * (int)sizeof(T)>{});
  });
}

// Launches kern on B * n_blk clusters of N CTAs, as a dependent launch.
template <typename P>
bool launch_gatedrec(void (*kern)(P), const P& p, long long clusters, size_t smem,
                     cudaStream_t st) {
  if (!set_smem(kern, smem)) return false;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.N;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(clusters * p.N));
  cfg.blockDim = dim3(kGrThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = p.N > 1 ? 2 : 1;
  return succeeded(cudaLaunchKernelEx(&cfg, kern, p));
}

// The cut of a recurrence: G groups of lanes per warp (64 / G channels per CTA) and N
// CTAs per cluster, for up to two CTAs per SM.  Two groups cost less than two CTAs
// (8 x 2048 x 1024 bf16: forward 24.2 us with G = 2, N = 1, 27.3 with G = 1, N = 2 and
// 27.2 with neither; gradient 48.9, 53.7 and 55.7), but rows of 32 bytes (G = 4) lose
// to eight CTAs (1 x 16384 x 1024: forward 31.8 us with G = 2, N = 8, 34.6 with G = 4,
// N = 4), so G = 4 is for fewer channels than eight CTAs fill the GPU with.  A padded
// batch leaves SMs to its longest sequences early: twice the CTAs, and G = 4 before
// clusters (8 sequences of 0 to 2048 tokens x 1024: forward 21.5 us, gradient 37.3;
// as for full sequences 23.6 and 45.6; G = 2, N = 2: 22.2 and 41.6).
struct GrPlan {
  int G, N, n_blk;
};
inline GrPlan plan_gatedrec(int B, int L, int D, int group_tokens, bool padded, int min_g) {
  const long long slots = (padded && B > 1 ? 4LL : 2LL) * device_sm_count();
  auto cut = [&](int G) {
    GrPlan pl{G, 1, (int)ceil_div(D, 64 / G)};
    const long long clusters = (long long)B * pl.n_blk, tile = (long long)G * kGrWarps * group_tokens;
    while (pl.N < kGrMaxCluster && clusters * (pl.N + 1) <= slots && pl.N * tile < L) ++pl.N;
    return pl;
  };
  // more groups while they double the CTAs at work and each still has tokens
  auto more = [&](int G) {
    return B * ceil_div(D, 64 / G) <= slots && (long long)G / 2 * kGrWarps * group_tokens < L;
  };
  GrPlan pl = cut(min_g);
  if (pl.G == 1 && more(2)) pl = cut(2);
  if (pl.G == 2 && more(4) && (padded || (long long)B * pl.n_blk * pl.N * 2 <= slots)) pl = cut(4);
  return pl;
}

// The longest walk of the gradient, which keeps 1 KiB of shared memory per token.
constexpr int kGrShortBwdMostL = 48;

// Whether one thread per two channels walks the sequences: they are shorter than
// a round of tiles, or so many that the walk fills the GPU.  128 x L x 1024 bf16,
// forward, walked and in tiles: L = 16 4.3 and 26.1 us, 64: 14.3 and 26.4, 128: 25.9
// and 29.6 (64 x 128 x 1024: 18.0 and 16.7); gradient: L = 16 8.5 and 25.5, 48: 22.6
// and 30.9, 64: 42.1 and 34.0.  Odd rows, with single loads, lose beyond the shortest
// (128 x 128 x 999: 90 and 64 us).
inline bool gatedrec_short(int B, int L, int D, bool forward) {
  if (L <= 16) return true;
  if (D % 2 != 0) return false;
  const long long per_sm = (long long)B * D / device_sm_count();
  return per_sm >= 128 && L <= (forward ? (per_sm >= 800 ? 128 : 64) : kGrShortBwdMostL);
}
template <typename P>
based_status_t launch_gatedrec_short(void (*pair)(P, int), void (*single)(P, int), const P& p, int B,
                                     size_t smem, size_t most_smem, cudaStream_t st) {
  auto kern = p.D % 2 == 0 ? pair : single;
  const long long blocks = ceil_div((long long)B * ((p.D + 1) / 2), kGrShortThreads);
  if (blocks > 0x7fffffffLL) return BASED_ERR_UNSUPPORTED;
  if (!set_smem(kern, most_smem) ||
      !launch_dependent(kern, dim3((unsigned)blocks), dim3(kGrShortThreads), smem, st, p, B))
    return BASED_ERR_CUDA;
  return launch_status();
}

}  // namespace

extern "C" {

based_status_t based_layernorm_fwd(const void* x, const void* residual, const float* weight,
                                   const float* bias, void* y, void* resid_out, float* mean,
                                   float* rstd, long long rows, int D, based_dtype_t dt, float eps,
                                   based_stream_t stream) {
  based_status_t s = check_layernorm(rows, D, dt);
  if (s != BASED_OK) return s;
  if (!(eps > 0.0f) || !isfinite(eps)) return BASED_ERR_INVALID_ARG;
  if ((residual == nullptr) != (resid_out == nullptr) && rows > 0) return BASED_ERR_INVALID_ARG;
  for (const void* t : {x, static_cast<const void*>(y), static_cast<const void*>(weight)})
    if ((s = check_tensor(t, rows == 0)) != BASED_OK) return s;
  for (const void* t : {residual, static_cast<const void*>(bias),
                        static_cast<const void*>(resid_out), static_cast<const void*>(mean),
                        static_cast<const void*>(rstd)})
    if (!aligned16(t)) return BASED_ERR_INVALID_ARG;
  if (rows == 0) return BASED_OK;
  LnFwdParams p{};
  p.x = x; p.residual = residual; p.w = weight; p.b = bias; p.y = y; p.resid_out = resid_out;
  p.mean = mean; p.rstd = rstd; p.rows = rows; p.D = D; p.eps = eps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return for_vector(dt, D, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    return D <= 256                 ? launch_layernorm_fwd<T, V, 8>(p, st)
           : D <= 512 || V < 4      ? launch_layernorm_fwd<T, V, 16>(p, st)
                                    : launch_layernorm_fwd<T, V, (V < 4 ? 16 : 32)>(p, st);
  });
}

size_t based_layernorm_bwd_workspace_bytes(long long rows, int D) {
  if (check_layernorm(rows, D, BASED_F32) != BASED_OK) return (size_t)-1;
  return (size_t)plan_layernorm_bwd(rows, D).parts * 2 * (size_t)D * sizeof(float);
}

based_status_t based_layernorm_bwd(const void* dy, const void* x, const float* weight,
                                   const float* mean, const float* rstd, const float* dresid,
                                   float* dx, float* dweight, float* dbias, long long rows, int D,
                                   based_dtype_t dt, void* workspace, size_t workspace_bytes,
                                   based_stream_t stream) {
  based_status_t s = check_layernorm(rows, D, dt);
  if (s != BASED_OK) return s;
  for (const void* t : {dy, x, static_cast<const void*>(weight), static_cast<const void*>(mean),
                        static_cast<const void*>(rstd), static_cast<const void*>(dx)})
    if ((s = check_tensor(t, rows == 0)) != BASED_OK) return s;
  if (!dweight || !aligned16(dweight) || !aligned16(dbias) || !aligned16(dresid))
    return BASED_ERR_INVALID_ARG;
  const LnBwdPlan pl = plan_layernorm_bwd(rows, D);
  if (pl.parts > 0 &&
      (!workspace || workspace_bytes < (size_t)pl.parts * 2 * (size_t)D * sizeof(float)))
    return BASED_ERR_WORKSPACE;
  if (!aligned16(workspace)) return BASED_ERR_INVALID_ARG;
  LnBwdParams p{};
  p.dy = dy; p.x = x; p.w = weight; p.mean = mean; p.rstd = rstd; p.dresid = dresid;
  p.dx = dx; p.parts = static_cast<float*>(workspace); p.rows = rows; p.D = D;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return for_vector(dt, D, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value < 4 ? decltype(v)::value : 4;
    return pl.E == 8 ? launch_layernorm_bwd<T, V, 8>(p, pl, dweight, dbias, st)
                     : launch_layernorm_bwd<T, V, 16>(p, pl, dweight, dbias, st);
  });
}

based_status_t based_rotary_freqs(double* freqs, int rot_dim, double base,
                                  based_rotary_scaling_t scaling, double factor,
                                  long long original_len, double low_turns, double high_turns) {
  if (!freqs || rot_dim <= 0 || rot_dim % 2 != 0 || !(base > 0.0) || !isfinite(base))
    return BASED_ERR_INVALID_ARG;
  if (scaling != BASED_ROTARY_NONE && scaling != BASED_ROTARY_LINEAR &&
      scaling != BASED_ROTARY_BY_PARTS)
    return BASED_ERR_INVALID_ARG;
  if (scaling != BASED_ROTARY_NONE && (!(factor >= 1.0) || !isfinite(factor)))
    return BASED_ERR_INVALID_ARG;
  if (scaling == BASED_ROTARY_BY_PARTS &&
      (original_len < 1 || !(high_turns > low_turns) || !isfinite(high_turns) ||
       !isfinite(low_turns)))
    return BASED_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim) / (2.0 * M_PI);
    if (scaling == BASED_ROTARY_LINEAR) f /= factor;
    if (scaling == BASED_ROTARY_BY_PARTS) {
      const double turns = f * (double)original_len;
      double keep = (turns - low_turns) / (high_turns - low_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f *= keep + (1.0 - keep) / factor;
    }
    freqs[i] = f;
  }
  return BASED_OK;
}

based_status_t based_rotary_fwd(const void* q, const void* k, void* q_out, void* k_out,
                                const double* freqs, const long long* pos, long long pos0, int B,
                                int H_q, int H_k, int L, int D, int rot_dim,
                                based_rotary_layout_t layout, float mscale, based_dtype_t dt,
                                based_stream_t stream) {
  return rotary_impl(q, k, q_out, k_out, freqs, pos, pos0, B, H_q, H_k, L, D, rot_dim, layout,
                     mscale, false, dt, stream);
}

based_status_t based_rotary_bwd(const float* dq_out, const float* dk_out, float* dq, float* dk,
                                const double* freqs, const long long* pos, long long pos0, int B,
                                int H_q, int H_k, int L, int D, int rot_dim,
                                based_rotary_layout_t layout, float mscale,
                                based_stream_t stream) {
  return rotary_impl(dq_out, dk_out, dq, dk, freqs, pos, pos0, B, H_q, H_k, L, D, rot_dim, layout,
                     mscale, true, BASED_F32, stream);
}

based_status_t based_gatedrec_fwd(const void* x, const void* g, void* y, const float* h0,
                                  float* h_last, float* h_chunks, const long long* lengths, int B,
                                  int L, int D, based_dtype_t dt, based_stream_t stream) {
  based_status_t s = check_gatedrec(x, g, y, lengths, B, L, D, dt);
  if (s != BASED_OK) return s;
  if (!aligned16(h0) || !aligned16(h_last) || !aligned16(h_chunks)) return BASED_ERR_INVALID_ARG;
  if (B == 0 || (L == 0 && !h_last)) return BASED_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  GrFwdParams p{};
  p.x = x; p.g = g; p.y = y; p.h0 = h0; p.h_last = h_last; p.h_chunks = h_chunks;
  p.lengths = lengths; p.L = L; p.D = D;
  if (gatedrec_short(B, L, D, true)) {
    return dt == BASED_F32
               ? launch_gatedrec_short(gatedrec_short_fwd_kernel<float, true>,
                                       gatedrec_short_fwd_kernel<float, false>, p, B, 0, 0, st)
               : launch_gatedrec_short(gatedrec_short_fwd_kernel<__nv_bfloat16, true>,
                                       gatedrec_short_fwd_kernel<__nv_bfloat16, false>, p, B, 0, 0,
                                       st);
  }
  return for_copies(dt, D, [&](auto t, auto cw) -> based_status_t {
    using T = decltype(t);
    constexpr int CW = decltype(cw)::value;
    const GrPlan pl = plan_gatedrec(B, L, D, GrFwdShape<T, 1>::S, lengths != nullptr, 1);
    p.n_blk = pl.n_blk;
    p.N = pl.N;
    const long long clusters = (long long)B * pl.n_blk;
    const size_t smem = GrFwdShape<T, 1>::kSmem;  // the same for every G
    const bool ok = pl.G == 1   ? launch_gatedrec(gatedrec_fwd_kernel<T, 1, CW>, p, clusters, smem, st)
                    : pl.G == 2 ? launch_gatedrec(gatedrec_fwd_kernel<T, 2, CW>, p, clusters, smem, st)
                                : launch_gatedrec(gatedrec_fwd_kernel<T, 4, CW>, p, clusters, smem, st);
    if (!ok) return BASED_ERR_CUDA;
    return launch_status();
  });
}

based_status_t based_gatedrec_bwd(const void* x, const void* g, const void* dy,
                                  const float* h_chunks, const float* dh_last, float* dx, float* dg,
                                  float* dh0, const long long* lengths, int B, int L, int D,
                                  based_dtype_t dt, based_stream_t stream) {
  based_status_t s = check_gatedrec(x, g, dy, lengths, B, L, D, dt);
  if (s != BASED_OK) return s;
  const bool empty = (long long)B * L == 0;
  for (const void* t : {static_cast<const void*>(h_chunks), static_cast<const void*>(dx),
                        static_cast<const void*>(dg)})
    if ((s = check_tensor(t, empty)) != BASED_OK) return s;
  if (!aligned16(dh_last) || !aligned16(dh0)) return BASED_ERR_INVALID_ARG;
  if (B == 0 || (L == 0 && !dh0)) return BASED_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  GrBwdParams p{};
  p.x = x; p.g = g; p.dy = dy; p.h_chunks = h_chunks; p.dh_last = dh_last;
  p.dx = dx; p.dg = dg; p.dh0 = dh0; p.lengths = lengths; p.L = L; p.D = D;
  if (gatedrec_short(B, L, D, false)) {
    const size_t token = sizeof(F2) * kGrShortThreads, smem = token * L,
                 most = token * kGrShortBwdMostL;
    return dt == BASED_F32
               ? launch_gatedrec_short(gatedrec_short_bwd_kernel<float, true>,
                                       gatedrec_short_bwd_kernel<float, false>, p, B, smem, most, st)
               : launch_gatedrec_short(gatedrec_short_bwd_kernel<__nv_bfloat16, true>,
                                       gatedrec_short_bwd_kernel<__nv_bfloat16, false>, p, B, smem,
                                       most, st);
  }
  return for_copies(dt, D, [&](auto t, auto cw) -> based_status_t {
    using T = decltype(t);
    constexpr int CW = decltype(cw)::value;
    const GrPlan pl = plan_gatedrec(B, L, D, GrBwdShape<T, 1>::S, lengths != nullptr,
                                    kGrBwdMinG<T>);
    p.n_blk = pl.n_blk;
    p.N = pl.N;
    const long long clusters = (long long)B * pl.n_blk;
    const size_t smem = GrBwdShape<T, 1>::kSmem;  // the same for every G
    if constexpr (kGrBwdMinG<T> == 1) {
      if (pl.G == 1) {
        if (!launch_gatedrec(gatedrec_bwd_kernel<T, 1, CW>, p, clusters, smem, st))
          return BASED_ERR_CUDA;
        return launch_status();
      }
    }
    const bool ok = pl.G == 2 ? launch_gatedrec(gatedrec_bwd_kernel<T, 2, CW>, p, clusters, smem, st)
                              : launch_gatedrec(gatedrec_bwd_kernel<T, 4, CW>, p, clusters, smem, st);
    if (!ok) return BASED_ERR_CUDA;
    return launch_status();
  });
}

based_status_t based_gatedrec_step(const void* x, const void* g, float* h, void* y, int B, int D,
                                   based_dtype_t dt, based_stream_t stream) {
  if (B < 0 || D <= 0 || !dtype_ok(dt)) return BASED_ERR_INVALID_ARG;
  based_status_t s;
  for (const void* t : {x, g, static_cast<const void*>(h), static_cast<const void*>(y)})
    if ((s = check_tensor(t, B == 0)) != BASED_OK) return s;
  if (B == 0) return BASED_OK;
  const long long n = (long long)B * D;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return for_vector(dt, n, [&](auto t, auto v) -> based_status_t {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    const long long blocks = ceil_div(n, 128LL * V);
    if (blocks > 0x7fffffffLL) return BASED_ERR_UNSUPPORTED;
    if (!launch_dependent(gatedrec_step_kernel<T, V>, dim3((unsigned)blocks), dim3(128), 0, st,
                          static_cast<const T*>(x), static_cast<const T*>(g), h,
                          static_cast<T*>(y), n))
      return BASED_ERR_CUDA;
    return launch_status();
  });
}

}  // extern "C"
