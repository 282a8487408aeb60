// fa_rope.cu -- rotary positions of q and k, forward and gradient.
//
//     (x, y) -> mscale * (x cos a - y sin a, y cos a + x sin a),  a = t * f_p
//
// The gradient is the transposed map, i.e. the same kernel with -sin a.
//
// Memory-bound: every element is read once and written once, 16 bytes at a
// time.  A thread owns V pairs of one position (two vectors of V columns) and
// takes their cos and sin once for several heads of q and k.
//
// Angles: f_p / 2 pi mod 1, formed in float64, becomes a 64-bit fraction of a
// turn (once a block, in shared memory); times the position, modulo 2^64, it is
// the fraction of the turn at t, whose upper 32 bits go to float32.  So the
// reduction costs an integer product, and a position of millions keeps its
// angle: 2^-32 of a turn beside what float64 rounds in f_p / 2 pi, times t.
//
// Measured on B200: bf16, B 4, 16 + 16 heads, N 4096, d 128 (268 MB) 44.9 us = 6.0
// TB/s, 91 % of a plain copy's rate; float32, B 2, 16 + 4 heads, N 1999, d 64 (41 MB)
// 8.4 us; one token of 32 sequences 2.5 us, which is what a launch takes.
#include "common.cuh"
#include "launch.h"

namespace fa {
namespace {

// V consecutive elements, loaded and stored as one access, held as float32.
template <class T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
};
template <>
struct Vec<__nv_bfloat16, 4> {
  using Raw = uint2;
};
template <>
struct Vec<float, 4> {
  using Raw = uint4;
};

template <class T, int V, class Raw>
__device__ __forceinline__ void unpack(const Raw &r, float (&x)[V]) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <class T, int V, class Raw>
__device__ __forceinline__ Raw pack(const float (&x)[V]) {
  Raw r;
  uint32_t *w = reinterpret_cast<uint32_t *>(&r);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  }
  return r;
}

// Thread (position, group c): c < pair_groups turns V pairs, whose vectors
// start at columns u and w (half layout: V c and V c + rot / 2; interleaved: 2
// V c and 2 V c + V); the groups behind them copy two vectors (the last perhaps
// one).  Blocks are (groups, positions); blockIdx.y: heads [y * per, y * per +
// per) of q's and then k's.
template <class T, int V, bool INTER>
__global__ void __launch_bounds__(64) rope_kernel(const RopeArgs a, int pair_groups, int per) {
  using Raw = typename Vec<T, V>::Raw;
  __shared__ unsigned long long s_turn[128];
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < a.rot / 2; i += blockDim.x * blockDim.y) {
    double r = a.freqs[i] * 0.15915494309189533577;
    r -= floor(r);   // whole turns a token do not matter
    s_turn[i] = __double2ull_rn(r * 18446744073709551616.0);   // 2^64 (1 saturates: 2^-64 off)
  }
  const int c = threadIdx.x;
  const unsigned bn = blockIdx.x * blockDim.y + threadIdx.y;   // B * N is below 2^31
  const bool live = bn < (unsigned)a.B * (unsigned)a.N;
  const unsigned b = live ? bn / (unsigned)a.N : 0, n = live ? bn - b * a.N : 0;
  const int h0 = blockIdx.y * per, h1 = live ? min(h0 + per, a.Hq + a.Hkv) : h0;
  // this position's row of head 0 of q and, Hq heads back, of k
  const long long head = (long long)a.N * a.d;
  const long long q0 = (long long)b * a.Hq * head + (long long)n * a.d;
  const long long k0 = ((long long)b * a.Hkv - a.Hq) * head + (long long)n * a.d;
  auto in = [&](int h) { return (const T *)(h < a.Hq ? a.q : a.k) + ((h < a.Hq ? q0 : k0) + h * head); };
  auto out = [&](int h) { return (T *)(h < a.Hq ? a.q_out : a.k_out) + ((h < a.Hq ? q0 : k0) + h * head); };
  const bool turns = c < pair_groups;
  int u, w;
  if (turns) {
    u = INTER ? 2 * V * c : V * c;
    w = INTER ? u + V : u + a.rot / 2;
  } else {
    u = a.rot + 2 * V * (c - pair_groups);
    w = u + V < a.d ? u + V : u;   // an odd vector at the end: copied twice
  }
  constexpr int AHEAD = 2;   // heads in flight
  Raw x[AHEAD], y[AHEAD];
  // the first heads' loads are under way while the angles are formed
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (h0 + i < h1) {
      x[i] = *reinterpret_cast<const Raw *>(in(h0 + i) + u);
      y[i] = *reinterpret_cast<const Raw *>(in(h0 + i) + w);
    }
  float cs[V], sn[V];
  const int t = !live ? 0 : a.positions[a.pos_per_batch ? bn : n];
  __syncthreads();
  if (turns) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned long long turn = s_turn[V * c + i] * (unsigned long long)(long long)t;
      // half turns in [-1, 1)
      sincospif((float)(int)(turn >> 32) * 4.656612873077392578125e-10f, &sn[i], &cs[i]);
      cs[i] *= a.mscale;
      sn[i] *= a.backward ? -a.mscale : a.mscale;
    }
  }
  for (int h = h0; h < h1; h += AHEAD) {
    if (h != h0) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (h + i < h1) {
          x[i] = *reinterpret_cast<const Raw *>(in(h + i) + u);
          y[i] = *reinterpret_cast<const Raw *>(in(h + i) + w);
        }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (h + i >= h1) continue;
      if (turns) {
        float p[V], q[V], ru[V], rw[V];
        unpack<T, V>(x[i], p);
        unpack<T, V>(y[i], q);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (INTER) {   // pair e: elements 2 e, 2 e + 1 of the two vectors
            const float p0 = 2 * e < V ? p[(2 * e) % V] : q[(2 * e) % V];
            const float p1 = 2 * e < V ? p[(2 * e + 1) % V] : q[(2 * e + 1) % V];
            const float r0 = p0 * cs[e] - p1 * sn[e], r1 = p1 * cs[e] + p0 * sn[e];
            if (2 * e < V) { ru[(2 * e) % V] = r0; ru[(2 * e + 1) % V] = r1; }
            else { rw[(2 * e) % V] = r0; rw[(2 * e + 1) % V] = r1; }
          } else {
            ru[e] = p[e] * cs[e] - q[e] * sn[e];
            rw[e] = q[e] * cs[e] + p[e] * sn[e];
          }
        }
        x[i] = pack<T, V, Raw>(ru);
        y[i] = pack<T, V, Raw>(rw);
      }
      *reinterpret_cast<Raw *>(out(h + i) + u) = x[i];
      *reinterpret_cast<Raw *>(out(h + i) + w) = y[i];
    }
  }
}

constexpr int kMaxHeads = 32;        // heads that share a thread's cos and sin, at most
constexpr long long kThreads = 148LL * 2048;   // threads that fill the GPU

template <class T, int V, bool INTER>
int run(const RopeArgs &a) {
  const int pair_groups = a.rot / (2 * V);
  // in place, the columns that do not turn are there already
  const bool in_place = a.q == a.q_out && a.k == a.k_out;
  const int groups = pair_groups + (in_place ? 0 : ((a.d - a.rot) / V + 1) / 2);
  const long long one = (long long)a.B * a.N * groups;   // threads of one head
  // positions of a block: 64 threads (B4 H16 N4096 d128 measured 45.2 us with
  // 64, 45.8 with 128, 47.8 with 256)
  const int deep = groups < 64 ? 64 / groups : 1;
  const int heads = a.Hq + a.Hkv;
  int per = heads < kMaxHeads ? heads : kMaxHeads;
  while (per > 1 && one * ((heads + per - 1) / per) < kThreads) per = (per + 1) / 2;
  const dim3 grid((unsigned)(((long long)a.B * a.N + deep - 1) / deep), (unsigned)((heads + per - 1) / per));
  rope_kernel<T, V, INTER><<<grid, dim3(groups, deep), 0, a.stream>>>(a, pair_groups, per);
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

template <class T, int V>
int run(const RopeArgs &a) {
  return a.interleaved ? run<T, V, true>(a) : run<T, V, false>(a);
}

}  // namespace

int launch_rope(const RopeArgs &a) {
  if (a.f32) return run<float, 4>(a);
  // bfloat16: 16-byte vectors where rows and halves are multiples of them
  return a.d % 8 == 0 && a.rot % 16 == 0 ? run<__nv_bfloat16, 8>(a) : run<__nv_bfloat16, 4>(a);
}

}  // namespace fa
