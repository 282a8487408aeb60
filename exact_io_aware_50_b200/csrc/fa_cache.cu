// fa_cache.cu -- the paged E4M3 key/value cache: writing new tokens with a
// scale for each page (block of tokens) and head, and reading them back.
//
// Writing: with amax the largest finite magnitude of the new values that fall
// into a page, scale = 2^k, the least with amax <= 448 * 2^k, or the page's
// older scale where that is larger; code = E4M3(x / scale).  These scales are powers
// of two, so dividing by one and growing one are exact but for codes that
// leave E4M3's normal range.  An older scale may be any other number (a cache that
// something else filled): then quotients and products are taken in float64 and
// rounded once, in loops of their own.  Memory-bound: es bytes read and one written an
// element (es + 1 reading back); both kernels move 16 bytes of the wider side at
// a time.
//
// Measured on B200, bf16, Hkv 8, d 128, pages of 64: four prompts of 2048 to 4096 tokens
// written (82 MB) 18.3 us = 4.5 TB/s, 69 % of a plain copy's rate, four of 4096 (101 MB)
// 19.9 us = 5.1 TB/s; in float32 (168 MB) 27.7 us = 6.1 TB/s, 92 %.  In bf16 instructions
// bound it as much as DRAM: 2.6 a cycle of four, about 17 an element, with 84 bytes
// spilled (its 64 registers are those that 1024 threads may have, where a page of 64 x
// 128 has 128); and a CTA's stores wait for the maximum over its page, so that loads and
// stores overlap between CTAs only.  64 x 1 token 2.9 us, a launch; 4 x 5001 to 8192 tokens
// read back (192 MB) 33.6 us = 5.7 TB/s, 87 %.
#include "cache.cuh"

namespace fa {
namespace {

// 16 bytes of T as float32.
template <class T>
struct Chunk {
  static constexpr int N = 16 / sizeof(T);   // elements: 8 or 4
  uint4 raw;
  __device__ __forceinline__ void get(float (&x)[N]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};

// A CTA's n codes of x / s, and n codes of a page times r, in float64 (apart from the
// kernel, whose registers they would take).
template <class T>
__device__ __noinline__ void encode_any(const T *x, uint8_t *codes, int n, float s) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) codes[i] = (uint8_t)e4m3_code((double)(float)x[i] / (double)s);
}
__device__ __noinline__ void grow_any(uint8_t *codes, int n, double r) {
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    codes[i] = (uint8_t)e4m3_code((double)e4m3x2_to_float2(codes[i]).x * r);
}

// One CTA per (touched page of a sequence, batch and head, K or V).  The new
// tokens of a page lie together; each thread keeps its chunks of them in
// registers between the maximum and the conversion, so they are read once.
template <class T, int CHUNKS>
__global__ void __launch_bounds__(CHUNKS == 8 ? 1024 : 512) cache_append_kernel(const CacheArgs a) {
  constexpr int N = Chunk<T>::N;
  __shared__ float s_red[32];
  __shared__ float s_old;
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int start = a.start[b];
  const int n = a.count ? max(0, min(a.count[b], a.T)) : a.T;
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
  const T *src = (const T *)(blockIdx.z ? a.v : a.k) + ((long long)bh * a.T + (lo - start)) * a.d;
  const int chunks = (hi - lo) * a.d / N;
  Chunk<T> x[CHUNKS];
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    x[i].raw = c < chunks ? *reinterpret_cast<const uint4 *>(src + (long long)c * N) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int pg = checked_page(a.table, (long long)b * a.max_pages + pi, a.num_pages, a.err);
  if (pg < 0) return;
  const long long page_h = (long long)pg * a.Hkv + h;
  uint8_t *dst = (blockIdx.z ? a.v_cache : a.k_cache) + page_h * a.page * a.d;
  float *scale = (blockIdx.z ? a.v_scale : a.k_scale) + page_h;
  const int slot = lo - pi * a.page;

  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    float f[N];
    x[i].get(f);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float m = fabsf(f[e]);
      if (m <= 3.402823466e38f) amax = fmaxf(amax, m);   // finite
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = amax;
  if (threadIdx.x == 0) s_old = slot ? *scale : 0.f;
  __syncthreads();
  amax = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) amax = fmaxf(amax, s_red[w]);
  const float old = s_old, s = fmaxf(e4m3_block_scale(amax), old);
  if (slot && s > old && !power_of_two(old)) {   // the older tokens' codes follow the scale
    grow_any(dst, slot * a.d, (double)old / (double)s);
  } else if (slot && s > old) {
    const float r = old / s;
    for (int i = threadIdx.x; i < slot * a.d / 16; i += blockDim.x) {
      uint4 v = reinterpret_cast<const uint4 *>(dst)[i];
      uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 lo2 = e4m3x2_to_float2(w[k] & 0xFFFFu), hi2 = e4m3x2_to_float2(w[k] >> 16);
        w[k] = pack_e4m3x2(lo2.x * r, lo2.y * r) | (pack_e4m3x2(hi2.x * r, hi2.y * r) << 16);
      }
      reinterpret_cast<uint4 *>(dst)[i] = v;
    }
  }
  if (threadIdx.x == 0) *scale = s;
  if (!power_of_two(s)) {   // an older scale
    encode_any(src, dst + slot * a.d, (hi - lo) * a.d, s);
    return;
  }
  const float inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    if (c >= chunks) continue;
    float f[N];
    x[i].get(f);
    uint32_t w[N / 4];
#pragma unroll
    for (int k = 0; k < N / 4; ++k)
      w[k] = pack_e4m3x2(f[4 * k] * inv, f[4 * k + 1] * inv) |
             (pack_e4m3x2(f[4 * k + 2] * inv, f[4 * k + 3] * inv) << 16);
    uint8_t *to = dst + slot * a.d + c * N;
    if constexpr (N == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(to) = w[0];
  }
}

// A thread takes 16 bytes of each output in `kReads` rows of one (b, h).
constexpr int kReads = 4;
template <class T>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheArgs a) {
  constexpr int N = Chunk<T>::N;
  const int per_row = a.d / N, rows = blockDim.x / per_row;   // rows of a block at a time
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int len = checked_len(a.lens, b, a.max_pages, a.page, a.err);
  const int col = (threadIdx.x % per_row) * N;
  const int first = blockIdx.x * rows * kReads + threadIdx.x / per_row;
  int pg[kReads];
#pragma unroll
  for (int i = 0; i < kReads; ++i) {
    const int j = first + i * rows;
    pg[i] = j < min(len, a.T)
                ? checked_page(a.table, (long long)b * a.max_pages + j / a.page, a.num_pages, a.err)
                : -1;
  }
  uint2 codes[2][kReads];
  float sc[2][kReads];
#pragma unroll
  for (int i = 0; i < kReads; ++i) {
    const int j = first + i * rows;
    const long long page_h = (long long)max(pg[i], 0) * a.Hkv + h;
    const long long at = (page_h * a.page + j % a.page) * a.d + col;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      codes[k][i] = make_uint2(0u, 0u);
      sc[k][i] = 0.f;
      if (pg[i] < 0) continue;
      const uint8_t *src = (k ? a.v_cache : a.k_cache) + at;
      if constexpr (N == 8) codes[k][i] = *reinterpret_cast<const uint2 *>(src);
      else codes[k][i].x = *reinterpret_cast<const uint32_t *>(src);
      sc[k][i] = (k ? a.v_scale : a.k_scale)[page_h];
    }
  }
#pragma unroll
  for (int i = 0; i < kReads; ++i) {
    const int j = first + i * rows;
    if (j >= a.T) continue;
    const long long to = ((long long)bh * a.T + j) * a.d + col;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w[2] = {codes[k][i].x, codes[k][i].y};
      uint4 out;
      uint32_t *o = reinterpret_cast<uint32_t *>(&out);
#pragma unroll
      for (int e = 0; e < N / 4; ++e) {
        const float2 lo = e4m3x2_to_float2(w[e] & 0xFFFFu), hi = e4m3x2_to_float2(w[e] >> 16);
        const float s = sc[k][i];
        if constexpr (N == 8) {
          o[2 * e] = pack_bf16x2(lo.x * s, lo.y * s);
          o[2 * e + 1] = pack_bf16x2(hi.x * s, hi.y * s);
        } else {
          o[0] = __float_as_uint(lo.x * s); o[1] = __float_as_uint(lo.y * s);
          o[2] = __float_as_uint(hi.x * s); o[3] = __float_as_uint(hi.y * s);
        }
      }
      *reinterpret_cast<uint4 *>((T *)(k ? a.v_out : a.k_out) + to) = out;
    }
  }
}

template <class T>
int run_append(const CacheArgs &a) {
  const long long pages = ((long long)a.T + a.page - 2) / a.page + 1;   // touched, at most
  const dim3 grid((unsigned)pages, (unsigned)(a.B * a.Hkv), 2);
  // A page's new tokens are at most min(T, page): 8 to 8192 chunks of 16 bytes.
  // A thread holds eight of them, so that small CTAs keep many loads in flight
  // (4 x 4096 tokens, Hkv 8, d 128, page 64: 17.8 us, against 33.6 with two a
  // thread), or two where a decode step brings few (64 x 1 token: 2.6 us).
  const int chunks = (a.T < a.page ? a.T : a.page) * a.d * (int)sizeof(T) / 16;
  if (chunks <= 128) {
    const int threads = chunks <= 64 ? 32 : (chunks / 2 + 31) / 32 * 32;
    cache_append_kernel<T, 2><<<grid, threads, 0, a.stream>>>(a);
  } else {
    cache_append_kernel<T, 8><<<grid, (chunks / 8 + 31) / 32 * 32, 0, a.stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

template <class T>
int run_read(const CacheArgs &a) {
  const int rows = 256 / (a.d * (int)sizeof(T) / 16) * kReads;
  const dim3 grid((unsigned)((a.T + rows - 1) / rows), (unsigned)(a.B * a.Hkv));
  cache_read_kernel<T><<<grid, 256, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

}  // namespace

int launch_cache_append(const CacheArgs &a) {
  return a.f32 ? run_append<float>(a) : run_append<__nv_bfloat16>(a);
}

int launch_cache_read(const CacheArgs &a) {
  return a.f32 ? run_read<float>(a) : run_read<__nv_bfloat16>(a);
}

}  // namespace fa
