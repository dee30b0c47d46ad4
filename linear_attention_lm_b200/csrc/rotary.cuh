// rotary.cuh -- rotary positions of the window attention's queries and keys
// (the "based/train" README's training stack carries a rotary kernel).
//
// Pair i of a head at position p turns by 2 pi p f_i (f_i: turns per position,
// a table in fp64): (u, v) -> m (u cos - v sin, u sin + v cos); the gradient is
// the transpose, m times the turn backwards.  Pairs are (i, i + rot/2) ("half")
// or (2i, 2i+1) ("interleaved"); values from rot on pass through.
//
// Angles: p f_i is formed in fp64 and its whole turns are taken off before it
// becomes fp32, so positions up to 2^31 keep about 2^-24 of a turn.  Sine and cosine
// are fp32, and their products with an m that is not a power of two are rounded too.
//
// Bound by HBM bandwidth (every value read and written once).  A thread owns V
// pairs of one position and walks the heads, queries' and then keys', so that
// its V sines and cosines are computed once for all of them.  Vectors are up to
// 16 bytes; halves of an odd length (rot / 2) and odd heads leave single values.
//
// Measured on B200: 8 x (16 + 16) heads x 2048 x 64 bf16, 134 MB: 25.1 us, 5.3 TB/s
// (a plain device copy of as many bytes: 24.6 us); fp32 42.9 us, 6.3 TB/s; 34 of
// 64 values turned in halves (V = 1) 36.7 us.
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
  // heads whose loads a thread has in flight: with 16 sines and cosines already in
  // registers, four of them cost more warps than they are worth (31.1 against 26.0 us)
  constexpr int kBatch = V == 8 ? 1 : 4;
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
  // pairs of the chunk that turn (interleaved: the rest of the last one passes)
  const int n_turned = kInter ? min(V, p.rot / 2 - ch * V) : V;
  float cs[V], sn[V];
  if (turned) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      cs[i] = sn[i] = 0.0f;
      if (i >= n_turned) continue;
      const double turns = (double)pos * p.freqs[ch * V + i];
      const float part = (float)(turns - rint(turns));
      float s, c;
      sincospif(2.0f * part, &s, &c);
      cs[i] = c * p.mscale;
      sn[i] = s * p.mscale * p.sign;
    }
  }
  auto turn = [&](Pack<T, V>& a, Pack<T, V>& c) {
    if (kInter && V > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        Pack<T, V>& z = 2 * i < V ? a : c;
        const int e = (2 * i) % V;
        const float u = z.get(e), v = z.get(e + 1);
        if (i < n_turned) {
          z.set(e, u * cs[i] - v * sn[i]);
          z.set(e + 1, u * sn[i] + v * cs[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float u = a.get(i), v = c.get(i);
        a.set(i, u * cs[i] - v * sn[i]);
        c.set(i, u * sn[i] + v * cs[i]);
      }
    }
  };
  // the heads [h, end) of one tensor of H heads, kBatch of them in flight
  auto walk = [&](const void* in, void* out, int H, int h, int end) {
    if (h >= end || (!turned && in == out)) return;
    const size_t stride = (size_t)p.L * p.D;
    const size_t off = ((size_t)b * H + h) * stride + (size_t)t * p.D;
    const T* src = static_cast<const T*>(in) + off;
    T* dst = static_cast<T*>(out) + off;
    for (; h < end; h += kBatch, src += kBatch * stride, dst += kBatch * stride) {
      Pack<T, V> a[kBatch], c[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < end) {
          a[i].load(src + i * stride + c0);
          if (two) c[i].load(src + i * stride + c1);
        }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (h + i < end) {
          if (turned) turn(a[i], c[i]);
          a[i].store(dst + i * stride + c0);
          if (two) c[i].store(dst + i * stride + c1);
        }
    }
  };
  const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(p.H_q + p.H_k, h0 + p.heads_per_cta);
  walk(p.q, p.q_out, p.H_q, h0, min(h1, p.H_q));
  walk(p.k, p.k_out, p.H_k, max(h0 - p.H_q, 0), h1 - p.H_q);
}

}  // namespace based
