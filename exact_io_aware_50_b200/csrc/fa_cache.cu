// fa_cache.cu -- the paged E4M3 key/value cache: writing new tokens with a
// scale for each page (block of tokens) and head, and reading them back.
//
// Writing: with amax the largest finite magnitude of the new values that fall
// into a page, scale = 2^k, the least with amax <= 448 * 2^k, or the page's
// older scale where that is larger; code = E4M3(x / scale).  Scales are powers
// of two, so dividing by one and growing one are exact but for codes that
// leave E4M3's normal range.  Memory-bound: es bytes read and one written an
// element (es + 1 reading back).
#include "cache.cuh"

namespace fa {
namespace {

__device__ __forceinline__ float load_f(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_f(const float *p) { return *p; }

// One CTA per (touched page of a sequence, batch and head, K or V).
template <class T>
__global__ void cache_append_kernel(const CacheArgs a) {
  __shared__ float s_red[32];
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int start = a.start[b];
  int n = a.count ? a.count[b] : a.T;
  n = max(0, min(n, a.T));
  if (n == 0) return;
  if (start < 0 || start > a.max_pages * a.page - n) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) atomicOr(a.err, kErrPage);
    if (start < 0) return;
  }
  const int pi = start / a.page + blockIdx.x;            // page of the sequence
  if (pi >= a.max_pages) return;
  const int lo = max(start, pi * a.page);                // positions [lo, hi) of it are written
  const int hi = min(start + n, (pi + 1) * a.page);
  if (lo >= hi) return;
  const int pg = checked_page(a.table, (long long)b * a.max_pages + pi, a.num_pages, a.err);
  if (pg < 0) return;
  const T *src = (const T *)(blockIdx.z ? a.v : a.k) + ((long long)bh * a.T + (lo - start)) * a.d;
  const long long page_h = (long long)pg * a.Hkv + h;
  uint8_t *dst = (blockIdx.z ? a.v_cache : a.k_cache) + page_h * a.page * a.d;
  float *scale = (blockIdx.z ? a.v_scale : a.k_scale) + page_h;

  const int slot = lo - pi * a.page, elems = (hi - lo) * a.d;
  float amax = 0.f;
  for (int i = threadIdx.x; i < elems; i += blockDim.x) {
    const float x = fabsf(load_f(src + i));
    if (x <= 3.402823466e38f) amax = fmaxf(amax, x);   // finite
  }
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = amax;
  const float old = slot ? *scale : 0.f;
  __syncthreads();
  amax = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) amax = fmaxf(amax, s_red[w]);
  const float need = e4m3_block_scale(amax);
  const float s = fmaxf(need, old);
  if (s > old && slot) {   // older codes follow the scale
    const float r = old / s;
    for (int i = threadIdx.x; i < slot * a.d / 2; i += blockDim.x) {
      const float2 f = e4m3x2_to_float2(((const unsigned short *)dst)[i]);
      ((unsigned short *)dst)[i] = (unsigned short)pack_e4m3x2(f.x * r, f.y * r);
    }
  }
  const float inv = 1.f / s;
  for (int i = threadIdx.x; i < elems / 2; i += blockDim.x)
    ((unsigned short *)(dst + slot * a.d))[i] =
        (unsigned short)pack_e4m3x2(load_f(src + 2 * i) * inv, load_f(src + 2 * i + 1) * inv);
  if (threadIdx.x == 0) *scale = s;
}

template <class T>
__global__ void cache_read_kernel(const CacheArgs a) {
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;   // one element
  const long long row = idx / a.d;
  if (row >= (long long)a.B * a.Hkv * a.T) return;
  const int c = (int)(idx - row * a.d);
  const int bh = (int)(row / a.T), j = (int)(row - (long long)bh * a.T);
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int len = checked_len(a.lens, b, a.max_pages, a.page, a.err);
  int pg = -1;
  if (j < len) pg = checked_page(a.table, (long long)b * a.max_pages + j / a.page, a.num_pages, a.err);
  float k = 0.f, v = 0.f;
  if (pg >= 0) {
    const long long page_h = (long long)pg * a.Hkv + h;
    const long long at = (page_h * a.page + j % a.page) * a.d + c;
    k = e4m3x2_to_float2(a.k_cache[at]).x * a.k_scale[page_h];
    v = e4m3x2_to_float2(a.v_cache[at]).x * a.v_scale[page_h];
  }
  ((T *)a.k_out)[idx] = (T)k;
  ((T *)a.v_out)[idx] = (T)v;
}

}  // namespace

int launch_cache_append(const CacheArgs &a) {
  const long long pages = ((long long)a.T + a.page - 2) / a.page + 1;   // touched, at most
  if ((long long)a.B * a.Hkv > 65535) return 2;
  const dim3 grid((unsigned)pages, (unsigned)(a.B * a.Hkv), 2);
  if (a.f32)
    cache_append_kernel<float><<<grid, 128, 0, a.stream>>>(a);
  else
    cache_append_kernel<__nv_bfloat16><<<grid, 128, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

int launch_cache_read(const CacheArgs &a) {
  const long long blocks = ((long long)a.B * a.Hkv * a.T * a.d + 255) / 256;
  if (blocks > 2147483647LL) return 2;
  if (a.f32)
    cache_read_kernel<float><<<(unsigned)blocks, 256, 0, a.stream>>>(a);
  else
    cache_read_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

}  // namespace fa
