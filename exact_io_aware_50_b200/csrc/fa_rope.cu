// fa_rope.cu -- rotary positions of q and k, forward and gradient.
//
//     (x, y) -> mscale * (x cos a - y sin a, y cos a + x sin a),  a = t * f_p
//
// The gradient is the transposed map, i.e. the same kernel with -sin a.
//
// Memory-bound: every element is read once and written once, 16 bytes at a
// time.  A thread owns V pairs of one position (two vectors of V columns) and
// takes their cos and sin once for up to kMaxHeads heads of q and k, so the
// float64 angles and the sine cost little beside the traffic; with few
// positions (decoding) the heads are spread over more threads instead.
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
// V c and 2 V c + V); the others copy the vector from column `rot` on.
// blockIdx.y: heads [y * per, y * per + per) of q's and then k's.
template <class T, int V, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a, int groups, int pair_groups, int per) {
  using Raw = typename Vec<T, V>::Raw;
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long bn = idx / groups;
  if (bn >= (long long)a.B * a.N) return;
  const int c = (int)(idx - bn * groups);
  const int b = (int)(bn / a.N), n = (int)(bn - (long long)b * a.N);
  const int h0 = blockIdx.y * per, h1 = min(h0 + per, a.Hq + a.Hkv);
  // element (head h, position n, column 0) of q or k
  auto row = [&](int h) {
    return h < a.Hq ? (((long long)b * a.Hq + h) * a.N + n) * a.d
                    : (((long long)b * a.Hkv + h - a.Hq) * a.N + n) * a.d;
  };
  auto in = [&](int h) { return (const T *)(h < a.Hq ? a.q : a.k) + row(h); };
  auto out = [&](int h) { return (T *)(h < a.Hq ? a.q_out : a.k_out) + row(h); };
  constexpr int AHEAD = 4;   // heads in flight
  if (c >= pair_groups) {
    const int u = a.rot + (c - pair_groups) * V;
    for (int h = h0; h < h1; h += AHEAD) {
      Raw x[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (h + i < h1) x[i] = *reinterpret_cast<const Raw *>(in(h + i) + u);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (h + i < h1) *reinterpret_cast<Raw *>(out(h + i) + u) = x[i];
    }
    return;
  }
  const int u = INTER ? 2 * V * c : V * c, w = INTER ? u + V : u + a.rot / 2;
  Raw x[AHEAD], y[AHEAD];
  // the first heads' loads are under way while the angles are formed
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (h0 + i < h1) {
      x[i] = *reinterpret_cast<const Raw *>(in(h0 + i) + u);
      y[i] = *reinterpret_cast<const Raw *>(in(h0 + i) + w);
    }
  float cs[V], sn[V];
  const double t = (double)a.positions[a.pos_per_batch ? bn : n];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // turns of the circle in float64, reduced to [-1/2, 1/2] before float32:
    // the angle of any int32 position keeps 2^-25 half turns
    double r = t * (a.freqs[V * c + i] * 0.15915494309189533577);
    r -= rint(r);
    sincospif((float)(2.0 * r), &sn[i], &cs[i]);
    cs[i] *= a.mscale;
    sn[i] *= a.backward ? -a.mscale : a.mscale;
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
      *reinterpret_cast<Raw *>(out(h + i) + u) = pack<T, V, Raw>(ru);
      *reinterpret_cast<Raw *>(out(h + i) + w) = pack<T, V, Raw>(rw);
    }
  }
}

constexpr int kMaxHeads = 32;        // heads that share a thread's cos and sin, at most
constexpr long long kThreads = 148LL * 1024;   // threads that fill the GPU

template <class T, int V, bool INTER>
int run(const RopeArgs &a) {
  const int pair_groups = a.rot / (2 * V);
  // in place, the columns that do not turn are there already
  const bool in_place = a.q == a.q_out && a.k == a.k_out;
  const int groups = pair_groups + (in_place ? 0 : (a.d - a.rot) / V);
  const long long one = (long long)a.B * a.N * groups;   // threads of one head
  const int heads = a.Hq + a.Hkv;
  int per = heads < kMaxHeads ? heads : kMaxHeads;
  while (per > 1 && one * ((heads + per - 1) / per) < kThreads) per = (per + 1) / 2;
  const long long blocks = (one + 255) / 256;
  if (blocks > 2147483647LL) return 2;
  const dim3 grid((unsigned)blocks, (unsigned)((heads + per - 1) / per));
  rope_kernel<T, V, INTER><<<grid, 256, 0, a.stream>>>(a, groups, pair_groups, per);
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
