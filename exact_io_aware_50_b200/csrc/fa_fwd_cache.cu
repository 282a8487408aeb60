// fa_fwd_cache.cu -- attention over the paged E4M3 cache.
//
//     s_j = scale * sk * (q . K^_j),  m = max s,  l = sum e^{s_j - m},
//     O = sum e^{s_j - m} sv V^_j / l,  L = m + ln l
//
// with sk, sv the scales of the page that token j stands in.
#include <math.h>

#include "cache.cuh"

namespace fa {
namespace {

// One CTA per query row; each warp takes every fourth token, a lane D / 32
// columns; the four warps' (m, l, O) are merged at the end.
template <int D>
__global__ void fwd_cache_row_kernel(const CacheArgs a) {
  constexpr int PER = D / 32;
  __shared__ float s_m[4], s_l[4], s_o[4][D];
  const int i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z;
  const int h = hq / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = checked_len(a.lens, b, a.max_pages, a.page, a.err);
  const int lim = a.causal ? min(len, len - a.Nq + i + 1) : len;
  const long long row = ((long long)b * a.Hq + hq) * a.Nq + i;
  float q[PER], acc[PER];
  for (int e = 0; e < PER; ++e) {
    q[e] = __bfloat162float(((const __nv_bfloat16 *)a.q)[row * D + lane * PER + e]) * a.scale;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < lim; j += 4) {
    const int pg = checked_page(a.table, (long long)b * a.max_pages + j / a.page, a.num_pages, a.err);
    if (pg < 0) continue;
    const long long page_h = (long long)pg * a.Hkv + h;
    const long long at = (page_h * a.page + j % a.page) * D + lane * PER;
    float s = 0.f;
    for (int e = 0; e < PER; ++e) s += q[e] * e4m3x2_to_float2(a.k_cache[at + e]).x;
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.k_scale[page_h];
    const float m_new = fmaxf(m, s);
    const float alpha = m == -INFINITY ? 0.f : __expf(m - m_new), p = expf(s - m_new);
    m = m_new;
    l = l * alpha + p;
    const float pv = p * a.v_scale[page_h];
    for (int e = 0; e < PER; ++e)
      acc[e] = acc[e] * alpha + pv * e4m3x2_to_float2(a.v_cache[at + e]).x;
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
  for (int e = 0; e < PER; ++e) s_o[warp][lane * PER + e] = acc[e];
  __syncthreads();
  const float mm = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float w[4], tot = 0.f;
  for (int u = 0; u < 4; ++u) {
    w[u] = s_m[u] == -INFINITY ? 0.f : expf(s_m[u] - mm);
    tot += w[u] * s_l[u];
  }
  const float inv = tot > 0.f || tot != tot ? 1.f / tot : 0.f;
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    float o = 0.f;
    for (int u = 0; u < 4; ++u) o += w[u] * s_o[u][c];
    ((__nv_bfloat16 *)a.o)[row * D + c] = __float2bfloat16(o * inv);
  }
  if (threadIdx.x == 0) a.lse[row] = tot == 0.f ? -INFINITY : mm + logf(tot);
}

}  // namespace

size_t fwd_cache_ws_bytes(int, int, int, int, int) { return 0; }

int launch_fwd_cache(const CacheArgs &a) {
  if (a.Hq > 65535 || a.B > 65535) return 2;
  const dim3 grid((unsigned)a.Nq, (unsigned)a.Hq, (unsigned)a.B);
  switch (a.d) {
    case 64: fwd_cache_row_kernel<64><<<grid, 128, 0, a.stream>>>(a); break;
    case 128: fwd_cache_row_kernel<128><<<grid, 128, 0, a.stream>>>(a); break;
    case 256: fwd_cache_row_kernel<256><<<grid, 128, 0, a.stream>>>(a); break;
    default: return 2;
  }
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

}  // namespace fa
