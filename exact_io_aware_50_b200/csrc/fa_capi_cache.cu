// fa_capi_cache.cu -- the C entry points of the serving operators declared in
// include/fa.h: rotary positions, the paged E4M3 key/value cache, attention
// over it.  Argument checks, then dispatch to the launchers.
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "common.cuh"
#include "launch.h"

namespace fa {
namespace {

// Tensors are read in 16-byte pieces; int32, float32 and float64 arrays by element.
bool aligned(const void *p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

int run_rope(RopeArgs &a) {
  const bool with_k = a.k || a.k_out;
  if (!a.q || !a.q_out || !a.positions || !a.freqs || (with_k && (!a.k || !a.k_out)))
    return FA_ERR_INVALID_ARG;
  if (!with_k) a.Hkv = 0;
  if (a.B <= 0 || a.Hq <= 0 || (with_k && a.Hkv <= 0) || a.N <= 0 || a.d <= 0 || a.rot <= 0)
    return FA_ERR_INVALID_ARG;
  if (!(a.mscale > 0.f) || !isfinite(a.mscale)) return FA_ERR_INVALID_ARG;
  if (a.d > 256 || a.d % 4 || a.rot % 8 || a.rot > a.d) return FA_ERR_UNSUPPORTED;
  // the kernel indexes B * N * (d / 4) threads and Hq + Hkv heads
  if ((double)a.B * a.N * a.d > 2.0e12 || (double)a.Hq + a.Hkv > 65535.0 ||
      (double)a.B * a.N > 2147483647.0)
    return FA_ERR_UNSUPPORTED;
  const void *ptrs[] = {a.q, a.k, a.q_out, a.k_out};
  for (const void *p : ptrs)
    if (!aligned(p, 16)) return FA_ERR_ALIGNMENT;
  if (!aligned(a.positions, 4) || !aligned(a.freqs, 8)) return FA_ERR_ALIGNMENT;
  AttnArgs dev_args;
  int dev;
  const int st = device_prologue(&dev, dev_args);
  return st ? st : launch_rope(a);
}

// Size rules of the cache calls; tokens: T, N or Nq.
int check_cache(const CacheArgs &a, int tokens) {
  if (a.B <= 0 || a.Hkv <= 0 || tokens <= 0 || a.d <= 0 || a.page <= 0 || a.num_pages <= 0 ||
      a.max_pages <= 0)
    return FA_ERR_INVALID_ARG;
  if (a.d != 64 && a.d != 128 && a.d != 256) return FA_ERR_UNSUPPORTED;
  if (a.page != 16 && a.page != 32 && a.page != 64 && a.page != 128) return FA_ERR_UNSUPPORTED;
  // index arithmetic: positions in int32, elements in int64
  if ((double)a.max_pages * a.page > (double)(1 << 28) || tokens > (1 << 28) ||
      (double)a.B * a.Hkv > (double)(1 << 28) || (double)a.num_pages * a.Hkv > 2147483647.0 ||
      (double)a.B * a.max_pages > 2147483647.0 ||
      (double)a.B * a.Hkv * tokens * a.d > 4.0e12 ||
      (double)a.num_pages * a.Hkv * a.page > 4294967294.0)   // cache rows, in uint32
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

bool cache_aligned(const CacheArgs &a) {
  return aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.k_out, 16) && aligned(a.v_out, 16) &&
         aligned(a.k_cache, 16) && aligned(a.v_cache, 16) && aligned(a.q, 16) && aligned(a.o, 16) &&
         aligned(a.k_scale, 4) && aligned(a.v_scale, 4) && aligned(a.table, 4) &&
         aligned(a.start, 4) && aligned(a.count, 4) && aligned(a.lens, 4) && aligned(a.lse, 4);
}

int prologue(CacheArgs &a) {
  AttnArgs dev_args;
  int dev;
  const int st = device_prologue(&dev, dev_args);
  a.err = dev_args.err;
  return st;
}

int run_append(CacheArgs &a) {
  const void *const ptrs[] = {a.k, a.v, a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.table, a.start};
  for (const void *p : ptrs)
    if (!p) return FA_ERR_INVALID_ARG;
  int st = check_cache(a, a.T);
  if (st) return st;
  if ((double)a.B * a.Hkv > 65535.0) return FA_ERR_UNSUPPORTED;   // a grid dimension
  if (!cache_aligned(a)) return FA_ERR_ALIGNMENT;
  if ((st = prologue(a))) return st;
  return launch_cache_append(a);
}

int run_read(CacheArgs &a) {
  const void *const ptrs[] = {a.k_cache, a.v_cache, a.k_scale, a.v_scale,
                              a.table,   a.lens,    a.k_out,   a.v_out};
  for (const void *p : ptrs)
    if (!p) return FA_ERR_INVALID_ARG;
  int st = check_cache(a, a.T);
  if (st) return st;
  if ((double)a.B * a.Hkv > 65535.0) return FA_ERR_UNSUPPORTED;   // a grid dimension
  if (!cache_aligned(a)) return FA_ERR_ALIGNMENT;
  if ((st = prologue(a))) return st;
  return launch_cache_read(a);
}

}  // namespace
}  // namespace fa

using fa::CacheArgs;
using fa::RopeArgs;

#define FA_EXPORT __attribute__((visibility("default")))

extern "C" {

#define FA_ROPE_ENTRY(name, T, is_f32, is_bwd)                                                     \
  FA_EXPORT int name(const T *q, const T *k, T *q_out, T *k_out, const int *positions,             \
                     const double *freqs, int B, int Hq, int Hkv, int N, int d, int rot_dim,       \
                     int pos_per_batch, int interleaved, float mscale, fa_stream_t stream) {       \
    RopeArgs a;                                                                                    \
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out; a.positions = positions; a.freqs = freqs;  \
    a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.N = N; a.d = d; a.rot = rot_dim;                            \
    a.pos_per_batch = pos_per_batch ? 1 : 0; a.interleaved = interleaved ? 1 : 0;                  \
    a.backward = is_bwd; a.f32 = is_f32; a.mscale = mscale; a.stream = (cudaStream_t)stream;       \
    return fa::run_rope(a);                                                                        \
  }
FA_ROPE_ENTRY(fa_rope, void, 0, 0)
FA_ROPE_ENTRY(fa_rope_f32, float, 1, 0)
FA_ROPE_ENTRY(fa_rope_bwd, void, 0, 1)
FA_ROPE_ENTRY(fa_rope_bwd_f32, float, 1, 1)

FA_EXPORT int fa_rope_freqs(double *freqs, float *mscale, int rot_dim, double theta, int kind,
                            double factor, int original_len, double beta_fast, double beta_slow) {
  if (!freqs || rot_dim <= 0 || !(theta > 0.0) || !isfinite(theta)) return FA_ERR_INVALID_ARG;
  if (kind < FA_ROPE_PLAIN || kind > FA_ROPE_YARN) return FA_ERR_INVALID_ARG;
  if (kind != FA_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return FA_ERR_INVALID_ARG;
  if (kind == FA_ROPE_YARN && (original_len <= 0 || !(beta_fast > beta_slow) ||
                               !isfinite(beta_fast) || !isfinite(beta_slow)))
    return FA_ERR_INVALID_ARG;
  if (rot_dim % 8 || rot_dim > 256) return FA_ERR_UNSUPPORTED;
  if (kind == FA_ROPE_NTK) theta *= pow(factor, (double)rot_dim / (rot_dim - 2));
  for (int p = 0; p < rot_dim / 2; ++p) {
    double f = pow(theta, -2.0 * p / rot_dim);
    if (kind == FA_ROPE_LINEAR) f /= factor;
    if (kind == FA_ROPE_YARN) {
      const double turns = original_len * f / 6.283185307179586476925286766559;
      double g = (turns - beta_slow) / (beta_fast - beta_slow);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      f = (1.0 - g) * f / factor + g * f;
    }
    freqs[p] = f;
  }
  if (mscale) *mscale = kind == FA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return FA_OK;
}

#define FA_APPEND_ENTRY(name, T_, is_f32)                                                          \
  FA_EXPORT int name(const T_ *k, const T_ *v, void *k_cache, void *v_cache, float *k_scale,       \
                     float *v_scale, const int *block_table, const int *start, const int *count,   \
                     int B, int Hkv, int T, int d, int page, int num_pages, int max_pages,         \
                     fa_stream_t stream) {                                                         \
    CacheArgs a;                                                                                   \
    a.k = k; a.v = v; a.k_cache = (uint8_t *)k_cache; a.v_cache = (uint8_t *)v_cache;              \
    a.k_scale = k_scale; a.v_scale = v_scale; a.table = block_table; a.start = start;              \
    a.count = count; a.B = B; a.Hkv = Hkv; a.T = T; a.d = d; a.page = page;                        \
    a.num_pages = num_pages; a.max_pages = max_pages; a.f32 = is_f32;                              \
    a.stream = (cudaStream_t)stream;                                                               \
    return fa::run_append(a);                                                                      \
  }
FA_APPEND_ENTRY(fa_cache_append, void, 0)
FA_APPEND_ENTRY(fa_cache_append_f32, float, 1)

#define FA_READ_ENTRY(name, T_, is_f32)                                                            \
  FA_EXPORT int name(const void *k_cache, const void *v_cache, const float *k_scale,               \
                     const float *v_scale, const int *block_table, const int *lens, T_ *k, T_ *v,  \
                     int B, int Hkv, int N, int d, int page, int num_pages, int max_pages,         \
                     fa_stream_t stream) {                                                         \
    CacheArgs a;                                                                                   \
    a.k_cache = (uint8_t *)const_cast<void *>(k_cache);                                            \
    a.v_cache = (uint8_t *)const_cast<void *>(v_cache);                                            \
    a.k_scale = const_cast<float *>(k_scale); a.v_scale = const_cast<float *>(v_scale);            \
    a.table = block_table; a.lens = lens; a.k_out = k; a.v_out = v; a.B = B; a.Hkv = Hkv;          \
    a.T = N; a.d = d; a.page = page; a.num_pages = num_pages; a.max_pages = max_pages;             \
    a.f32 = is_f32; a.stream = (cudaStream_t)stream;                                               \
    return fa::run_read(a);                                                                        \
  }
FA_READ_ENTRY(fa_cache_read, void, 0)
FA_READ_ENTRY(fa_cache_read_f32, float, 1)

FA_EXPORT size_t fa_fwd_cache_workspace_size(int B, int Hq, int Hkv, int Nq, int d, int page,
                                             int max_pages) {
  CacheArgs a;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.Nq = Nq; a.d = d; a.page = page; a.max_pages = max_pages;
  a.num_pages = 1;
  if (fa::check_cache(a, Nq) || Hq <= 0 || Hq % Hkv) return 0;
  return fa::fwd_cache_ws_bytes(a);
}

FA_EXPORT int fa_fwd_cache(const void *q, const void *k_cache, const void *v_cache,
                           const float *k_scale, const float *v_scale, const int *block_table,
                           const int *lens, void *o, float *lse, void *workspace, int B, int Hq,
                           int Hkv, int Nq, int d, int page, int num_pages, int max_pages,
                           float scale, int causal, fa_stream_t stream) {
  CacheArgs a;
  a.q = q; a.k_cache = (uint8_t *)const_cast<void *>(k_cache);
  a.v_cache = (uint8_t *)const_cast<void *>(v_cache);
  a.k_scale = const_cast<float *>(k_scale); a.v_scale = const_cast<float *>(v_scale);
  a.table = block_table; a.lens = lens; a.o = o; a.lse = lse; a.ws = workspace;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.Nq = Nq; a.T = Nq; a.d = d; a.page = page;
  a.num_pages = num_pages; a.max_pages = max_pages; a.scale = scale; a.causal = causal ? 1 : 0;
  a.stream = (cudaStream_t)stream;
  const void *const ptrs[] = {q, k_cache, v_cache, k_scale, v_scale, block_table, lens, o, lse};
  for (const void *p : ptrs)
    if (!p) return FA_ERR_INVALID_ARG;
  int st = fa::check_cache(a, Nq);
  if (st) return st;
  if (Hq <= 0 || Hq % Hkv || !(scale > 0.f) || !isfinite(scale)) return FA_ERR_INVALID_ARG;
  if ((double)B * Hq * Nq > 2147483647.0 || fa::fwd_cache_granules(a) > 2.0e9)
    return FA_ERR_UNSUPPORTED;
  const bool need_ws = fa::fwd_cache_ws_bytes(a) > 0;
  if (need_ws && !workspace) return FA_ERR_INVALID_ARG;
  if (!fa::cache_aligned(a)) return FA_ERR_ALIGNMENT;
  if (need_ws && ((uintptr_t)workspace & 255u)) return FA_ERR_ALIGNMENT;
  if ((st = fa::prologue(a))) return st;
  return fa::launch_fwd_cache(a);
}

}  // extern "C"
