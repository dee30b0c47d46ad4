// rotary.cuh -- rotary positions of the window attention's queries and keys
// (the "based/train" README's training stack carries a rotary kernel).
//
// Pair i of a head at position p turns by 2 pi p f_i (f_i: turns per position,
// a table in fp64): (u, v) -> m (u cos - v sin, u sin + v cos); the gradient is
// the transpose, m times the turn backwards.  Pairs are (i, i + rot/2) ("half")
// or (2i, 2i+1) ("interleaved"); values from rot on pass through.
//
// Angles: p f_i is formed in fp64 and its whole turns are taken off before it
// becomes fp32, so positions up to 2^31 keep about 2^-24 of a turn.
//
// Bound by HBM bandwidth (2 reads and writes of every value).  A thread owns V
// pairs of one position and walks the heads, queries' and then keys', so that
// its V sines and cosines are computed once for all of them.
#pragma once

#include "common.cuh"
#include "umma.cuh"
#include "vec.cuh"

namespace based {

constexpr int kRotThreads = 128;

struct RotaryParams {
  const void *q, *k;
  void *q_out, *k_out;
  const double* freqs;
  const long long* pos_arr;  // [B], or null: pos0 for all
  long long pos0;
  long long items;  // B * L * chunks
  int L, D, rot, H_q, H_k;
  int chunks;      // of 2V values of a head: turned ones, then those that pass
  int rot_chunks;  // (interleaved: the last may hold values that pass)
  int heads_per_cta;
  float mscale;   // negative sine: inverse
  float sign;
};

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p) {
  umma::grid_dep_wait();
  const long long item = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  if (item >= p.items) return;
  const int ch = (int)(item % p.chunks);
  const long long bt = item / p.chunks;
  const int t = (int)(bt % p.L);
  const long long b = bt / p.L;
  long long pos = p.pos0;
  if (p.pos_arr) {
    pos = p.pos_arr[b];
    if (pos < 0 || pos > (1LL << 31) - p.L) {
      record_device_error(BASED_ERR_INVALID_ARG);
      return;
    }
  }
  pos += t;
  const bool turned = ch < p.rot_chunks;
  // the chunk's two vectors of V values
  int c0 = 2 * ch * V, c1 = c0 + V;
  if (!kInter) {
    c0 = turned ? ch * V : p.rot + 2 * (ch - p.rot_chunks) * V;
    c1 = c0 + (turned ? p.rot / 2 : V);
  }
  const bool two = c1 < p.D;
  float cs[V], sn[V];
  if (turned) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (kInter && ch * V + i >= p.rot / 2) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
        continue;
      }
      const double turns = (double)pos * p.freqs[ch * V + i];
      const float part = (float)(turns - rint(turns));
      float s, c;
      sincospif(2.0f * part, &s, &c);
      cs[i] = c * p.mscale;
      sn[i] = s * p.mscale * p.sign;
    }
  }
  const int h_end = min(p.H_q + p.H_k, (int)(blockIdx.y + 1) * p.heads_per_cta);
  for (int h = blockIdx.y * p.heads_per_cta; h < h_end; ++h) {
    const bool is_q = h < p.H_q;
    const long long row = is_q ? b * p.H_q + h : b * p.H_k + (h - p.H_q);
    const size_t off = ((size_t)row * p.L + t) * p.D;
    const T* src = static_cast<const T*>(is_q ? p.q : p.k) + off;
    T* dst = static_cast<T*>(is_q ? p.q_out : p.k_out) + off;
    if (!turned && src == dst) continue;
    Pack<T, V> a, c;
    a.load(src + c0);
    if (two) c.load(src + c1);
    if (turned) {
      if (kInter && V > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          Pack<T, V>& z = 2 * i < V ? a : c;
          const int e = (2 * i) % V;
          const float u = z.get(e), v = z.get(e + 1);
          z.set(e, u * cs[i] - v * sn[i]);
          z.set(e + 1, u * sn[i] + v * cs[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float u = a.get(i), v = c.get(i);
          a.set(i, u * cs[i] - v * sn[i]);
          c.set(i, u * sn[i] + v * cs[i]);
        }
      }
    }
    a.store(dst + c0);
    if (two) c.store(dst + c1);
  }
}

}  // namespace based
