// fa_rope.cu -- rotary positions of q and k, forward and gradient.
//
//     (x, y) -> mscale * (x cos a - y sin a, y cos a + x sin a),  a = t * f_p
//
// The gradient is the transposed map, i.e. the same kernel with -sin a.
// Memory-bound: every element is read once and written once.
#include "common.cuh"
#include "launch.h"

namespace fa {
namespace {

// One thread per (batch, position, pair): cos and sin once, then every head.
template <class T>
__global__ void rope_kernel(const RopeArgs a) {
  const int pairs = a.rot / 2;
  const int cols = pairs + (a.d - a.rot);   // pairs, then one column each that is copied
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long bn = idx / cols;
  if (bn >= (long long)a.B * a.N) return;
  const int c = (int)(idx - bn * cols);
  const int b = (int)(bn / a.N), n = (int)(bn - (long long)b * a.N);
  float cs = 1.f, sn = 0.f;
  int x = a.rot + c - pairs, y = x;
  if (c < pairs) {
    const int t = a.positions[a.pos_per_batch ? bn : n];
    // turns of the circle in float64, reduced to [-1/2, 1/2] before float32
    double r = (double)t * (a.freqs[c] * 0.15915494309189533577);
    r -= rint(r);
    sincospif((float)(2.0 * r), &sn, &cs);
    cs *= a.mscale;
    sn *= a.backward ? -a.mscale : a.mscale;
    x = a.interleaved ? 2 * c : c;
    y = a.interleaved ? 2 * c + 1 : c + pairs;
  }
  for (int h = 0; h < a.Hq + a.Hkv; ++h) {
    const bool is_q = h < a.Hq;
    const long long row = is_q ? ((long long)b * a.Hq + h) * a.N + n
                               : ((long long)b * a.Hkv + h - a.Hq) * a.N + n;
    const T *in = (const T *)(is_q ? a.q : a.k) + row * a.d;
    T *out = (T *)(is_q ? a.q_out : a.k_out) + row * a.d;
    if (x == y) {
      out[x] = in[x];
    } else {
      const float u = (float)in[x], v = (float)in[y];
      out[x] = (T)(u * cs - v * sn);
      out[y] = (T)(v * cs + u * sn);
    }
  }
}

}  // namespace

int launch_rope(const RopeArgs &a) {
  const long long threads = (long long)a.B * a.N * (a.rot / 2 + a.d - a.rot);
  const long long blocks = (threads + 255) / 256;
  if (blocks > 2147483647LL) return 2;
  if (a.f32)
    rope_kernel<float><<<(unsigned)blocks, 256, 0, a.stream>>>(a);
  else
    rope_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

}  // namespace fa
