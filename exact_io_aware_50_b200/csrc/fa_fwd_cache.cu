// fa_fwd_cache.cu -- attention over the paged E4M3 cache.
//
//     s_j = scale * sk * (q . K^_j),  m = max s,  l = sum 2^{s_j - m},
//     O = sum 2^{s_j - m} sv V^_j / l,  L = (m + log2 l) ln 2
//
// with s in base-2 units, sk and sv the scales of the page token j stands in.
//
// Rows: the g * Nq query rows that read one key/value head (contiguous in q)
// are cut into tiles of 16 * MT rows, so a page is read once for all of them.
// Work: a unit is (sequence, key/value head, row tile); its tokens come in
// granules of 64.  The granules of all units, in one line, are divided evenly
// among the CTAs (two per SM), so ragged lengths, few heads and long caches
// all fill the GPU: a CTA's run may start inside one unit and end inside
// another.  A unit that one CTA covers is finished there; the others leave
// their normalised partial O and log-sum-exp in the workspace, and the merge
// kernel joins them (L = log sum 2^{L_c}, O = sum 2^{L_c - L} O_c).  Nothing
// is accumulated by atomics: results do not depend on timing.
//
// A warp takes 16 tokens of each granule.  It keeps its own ring of shared
// memory, filled by 16-byte asynchronous copies, and its own (m, l, O): the
// four warps meet only at the end of a unit.  The E4M3 codes become halves,
// exactly, on their way into mma.m16n8k16; q becomes halves too, each row
// times a power of two that brings its largest entry to [2^13, 2^14), so an
// entry keeps its 8 bits unless it is 2^-28 of the largest.  The weight that
// multiplies V is 2^{s - m} sv, rounded to a half.  It has a reference M of its
// own, the running maximum of s + log2 sv: terms down to 2^-26 of the largest
// keep 11 bits whatever the pages' scales, and smaller ones err by at most
// 2^-37 of the largest weight.
#include <math.h>

#include "cache.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kSub = 16;                        // tokens of a subtile (one page's, or part of it)
constexpr int kGranule = kWarps * kSub;
constexpr int kRingBytes = 24 * 1024;           // per warp
constexpr int kMaxCtas = 2 * 148;               // two per SM
constexpr float kLag = 3.f;                     // a maximum may lag by 2^3
constexpr float kShift = 12.f;                  // weights are stored times 2^12: at most 2^15

template <int D, int MT>
struct RowCfg {
  static constexpr int ROWS = 16 * MT;
  static constexpr int CH = D / 16;             // 16-byte chunks of a token
  // Subtiles a warp takes at a time: two where the registers allow (their
  // scores beside q and O), which halves the work around them.
  static constexpr int NS = D * MT <= 128 ? 2 : 1;
  static constexpr int TILE = kSub * D;         // K or V codes of a subtile
  static constexpr int STAGE = 2 * NS * TILE;
  static constexpr int STAGES = kRingBytes / STAGE;
  static constexpr int OFF_SCALE = kWarps * kRingBytes;                  // [warp][stage][NS] (sk, sv)
  static constexpr int OFF_STAT = OFF_SCALE + kWarps * STAGES * NS * 8;  // [warp][ROWS]
  static constexpr int SMEM = OFF_STAT + kWarps * ROWS * 4;
  static_assert(ROWS * D * 4 <= kRingBytes, "a warp's O fits in its ring");
  static_assert(STAGES >= 3, "ring depth");
};

// Byte offset of 16-byte chunk c of token r in a subtile's tile: chunks are
// permuted so that eight tokens' chunk c lie in eight different bank groups.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  if constexpr (D == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return r * D + ((c ^ (r & 7)) << 4);
}
// The same for chunk 32 i + lane of the tile in token order, `first` being
// tile_at of chunk `lane`: a warp-wide copy moves 512 bytes.
template <int D>
__device__ __forceinline__ uint32_t tile_chunk(uint32_t first, int i) {
  constexpr int RPI = 512 / D;   // tokens of one copy
  return 512 * i + (D == 64 ? first : first ^ (((i * RPI) & 7) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += A B: 16 x 16 halves, 16 x 8 halves, float32 accumulator.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}

// Programmatic dependent launch: the next kernel of the stream may start; a
// dependent kernel waits here until the one before it has ended.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_primary() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct RowParams {
  const __nv_bfloat16 *q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *table, *lens;
  __nv_bfloat16 *o;
  float *lse;
  float *o_part, *l_part;   // [grid][2][prows][D], [grid][2][prows] (base 2)
  int B, Hq, Hkv, Nq, R, tiles;   // R = g * Nq rows of a key/value head, in `tiles` tiles
  int page_log2, num_pages, max_pages;
  int causal, ctas, prows;   // prows: rows of a partial, min(R, rows of a tile)
  float scale_log2;
  unsigned *err;
};

__device__ __forceinline__ int granules_of(const RowParams &p, int b) {
  const int n = p.lens[b];
  return (min(max(n, 0), p.max_pages << p.page_log2) + kGranule - 1) / kGranule;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The line of granules: sequences in order, each with Hkv * tiles units of
// granules_of(b).  Granules of all sequences, and of those before sequence b
// (of one unit each); every warp forms them for itself.
__device__ __forceinline__ void line_of(const RowParams &p, int b, long long *total, long long *before) {
  const int lane = threadIdx.x & 31;
  long long all = 0, pre = 0;
  for (int i = lane; i < p.B; i += 32) {
    const int n = granules_of(p, i);
    all += n;
    if (i < b) pre += n;
  }
  *total = warp_sum(all);
  *before = b > 0 ? warp_sum(pre) : 0;
}

// The sequence that holds granule `pos` of the line cut to one unit a
// sequence (pos < the total), and the granules before it.
__device__ __forceinline__ int sequence_at(const RowParams &p, long long pos, long long *before) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int i0 = 0;; i0 += 32) {
    const int n = i0 + lane < p.B ? granules_of(p, i0 + lane) : 0;
    long long inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    inc += base;
    const unsigned past = __ballot_sync(0xffffffffu, pos < inc);
    if (past || i0 + 32 >= p.B) {
      const int at = past ? __ffs(past) - 1 : 31;
      *before = __shfl_sync(0xffffffffu, inc - n, at);
      return min(i0 + at, p.B - 1);
    }
    base = __shfl_sync(0xffffffffu, inc, 31);
  }
}

template <int D, int MT>
__global__ void __launch_bounds__(kWarps * 32, 2) fwd_cache_rows_kernel(const RowParams p) {
  using C = RowCfg<D, MT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = warp_id_uniform(), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int units = p.Hkv * p.tiles;
  launch_dependents();   // the merge kernel's CTAs may take their places

  // This CTA's run of the line, and the sequence it starts in.
  long long total, pos, end, b_first;
  line_of(p, 0, &total, &b_first);
  total *= units;
  {
    const long long per = (total + p.ctas - 1) / p.ctas;
    pos = per * blockIdx.x;
    end = min(total, pos + per);
  }
  if (pos >= end) return;
  int b = sequence_at(p, units == 1 ? pos : pos / units, &b_first);
  b_first *= units;

  const uint32_t ring = smem_u32(smem) + warp * kRingBytes;
  float2 *scales = reinterpret_cast<float2 *>(smem + C::OFF_SCALE) + warp * C::STAGES * C::NS;
  float *stat = reinterpret_cast<float *>(smem + C::OFF_STAT);   // [warp][ROWS]
  const uint32_t copy_dst = tile_at<D>(lane / C::CH, lane % C::CH);

  while (pos < end) {
    int ng = granules_of(p, b);
    while (pos >= b_first + (long long)ng * units) {   // next sequence with tokens
      b_first += (long long)ng * units;
      ++b;
      ng = granules_of(p, b);
    }
    const int u = (int)((pos - b_first) / ng);
    const int g0 = (int)(pos - b_first - (long long)u * ng);
    const int g1 = (int)min((long long)ng, g0 + (end - pos));
    pos += g1 - g0;
    const int h = u / p.tiles, r0 = (u - h * p.tiles) * C::ROWS;
    if (threadIdx.x == 0) (void)checked_len(p.lens, b, p.max_pages, 1 << p.page_log2, p.err);
    const int len = min(max(p.lens[b], 0), p.max_pages << p.page_log2);
    const int group = p.Hq / p.Hkv;
    const long long row_base = ((long long)b * p.Hq + (long long)h * group) * p.Nq;   // row 0 of q, o, lse

    // ---- pages: lane i holds the page number of the warp's subtile 32 k + i
    const int subs = g1 - g0;                             // subtiles of this warp
    const int steps = (subs + C::NS - 1) / C::NS;
    const int *tab = p.table + (long long)b * p.max_pages;
    auto token_of = [&](int i) { return (g0 + i) * kGranule + warp * kSub; };
    auto lookup = [&](int i) {
      const int j = token_of(i);
      return i < subs && j < len ? checked_page(tab, j >> p.page_log2, p.num_pages, p.err) : -1;
    };
    int cur = lookup(lane), nxt = subs > 32 ? lookup(32 + lane) : -1;
    // Copies of step s into stage st; always one commit group a step.  What
    // is no token of the sequence becomes zeros, and its page's scales too.
    auto issue = [&](int s, int st) {
      if (s < steps) {
        const int i0 = s * C::NS;
        if (i0 && (i0 & 31) == 0) {
          cur = nxt;
          nxt = lookup(i0 + 32 + lane);
        }
        const uint32_t stage = ring + st * C::STAGE;
#pragma unroll
        for (int n = 0; n < C::NS; ++n) {
          const int pg = __shfl_sync(0xffffffffu, cur, (i0 + n) & 31);
          const int j = token_of(i0 + n);
          const int live = pg < 0 ? 0 : min(kSub, len - j) * C::CH;   // chunks
          const long long page_h = (long long)max(pg, 0) * p.Hkv + h;
          const long long at = ((page_h << p.page_log2) + (j & ((1 << p.page_log2) - 1))) * D + lane * 16;
          const uint8_t *ks = p.k_cache + at, *vs = p.v_cache + at;
          const uint32_t dst = stage + 2 * n * C::TILE;
#pragma unroll
          for (int i = 0; i < C::TILE / 512; ++i) {
            const bool in = 32 * i + lane < live;
            const int off = in ? 512 * i : 0;
            cp_async16(dst + tile_chunk<D>(copy_dst, i), in ? ks + off : p.k_cache, in);
            cp_async16(dst + C::TILE + tile_chunk<D>(copy_dst, i), in ? vs + off : p.v_cache, in);
          }
          if (lane < 2)
            cp_async4(smem_u32(scales + st * C::NS + n) + 4 * lane,
                      (lane ? p.v_scale : p.k_scale) + page_h, pg >= 0);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) issue(s, s);

    // ---- q: A fragments of halves, each row times a power of two
    uint32_t qa[MT][C::CH][4];
    float row_c[MT][2];        // scale * log2 e / that power of two
    int lim[MT][2];            // keys [0, lim) visible
    int lim_min = len;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint2 raw[2][C::CH];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + mt * 16 + g + 8 * e;
        const bool live = r < p.R;
        const __nv_bfloat16 *src = p.q + (row_base + (live ? r : 0)) * D + 4 * t;
#pragma unroll
        for (int c = 0; c < C::CH; ++c)
          raw[e][c] = live ? *reinterpret_cast<const uint2 *>(src + 16 * c) : make_uint2(0u, 0u);
        lim[mt][e] = !live ? 0 : (p.causal ? max(0, len - p.Nq + r % p.Nq + 1) : len);
        if (live) lim_min = min(lim_min, lim[mt][e]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < C::CH; ++c) {
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(raw[e][c].x << 16)),
                               fabsf(__uint_as_float(raw[e][c].x & 0xFFFF0000u))));
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(raw[e][c].y << 16)),
                               fabsf(__uint_as_float(raw[e][c].y & 0xFFFF0000u))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // mx in [2^k, 2^{k+1}); zero rows and exponents past float32's reach are cut off
        const int k = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 126);
        const float up = __uint_as_float((uint32_t)(13 - k + 127) << 23);
        row_c[mt][e] = p.scale_log2 * __uint_as_float((uint32_t)(k - 13 + 127) << 23);
#pragma unroll
        for (int c = 0; c < C::CH; ++c) {
          qa[mt][c][e] = pack_half2(__uint_as_float(raw[e][c].x << 16) * up,
                                    __uint_as_float(raw[e][c].x & 0xFFFF0000u) * up);
          qa[mt][c][2 + e] = pack_half2(__uint_as_float(raw[e][c].y << 16) * up,
                                        __uint_as_float(raw[e][c].y & 0xFFFF0000u) * up);
        }
      }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    float o[MT][D / 8][4];
    float m_s[MT][2], m_o[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_s[mt][e] = m_o[mt][e] = -INFINITY;
        l[mt][e] = 0.f;
      }
    }

    int st = 0;   // stage of step s
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();
      issue(s + C::STAGES - 1, st == 0 ? C::STAGES - 1 : st - 1);
      const uint32_t stage = ring + st * C::STAGE;

      // ---- S = q K^T: two groups of 8 tokens a subtile
      float sc[MT][2 * C::NS][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2 * C::NS; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.f;
#pragma unroll
      for (int c = 0; c < C::CH; c += 4)
#pragma unroll
        for (int n = 0; n < 2 * C::NS; ++n) {
          uint32_t kb[4];
          ldsm4(stage + (n >> 1) * 2 * C::TILE + tile_at<D>(8 * (n & 1) + (lane & 7), c + (lane >> 3)), kb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b0 = e4m3x2_to_half2(kb[i]), b1 = e4m3x2_to_half2(kb[i] >> 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma_f16(sc[mt][n], qa[mt][c + i], b0, b1);
          }
        }

      // ---- softmax
      float sk[C::NS], lsv[C::NS];
      int j0[C::NS], nv[C::NS];
      bool whole = true;
#pragma unroll
      for (int n = 0; n < C::NS; ++n) {
        const float2 x = scales[st * C::NS + n];
        j0[n] = token_of(s * C::NS + n);
        // a subtile without a page has scales 0: no token of it is visible
        nv[n] = x.y > 0.f ? min(kSub, len - j0[n]) : 0;
        sk[n] = x.x;
        lsv[n] = nv[n] > 0 ? __log2f(x.y) : 0.f;
        whole = whole && nv[n] == kSub && j0[n] + kSub <= lim_min;
      }
      bool moved = false;
      float mxs[MT][2], mxo[MT][2];   // row maxima of s and of s + log2 sv
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mxs[mt][e] = mxo[mt][e] = -INFINITY;
#pragma unroll
          for (int n = 0; n < C::NS; ++n) {
            const float cf = row_c[mt][e] * sk[n];
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x = sc[mt][2 * n + (i >> 1)][2 * e + (i & 1)] * cf;
              if (!whole && 8 * (i >> 1) + 2 * t + (i & 1) >= min(nv[n], lim[mt][e] - j0[n])) x = -INFINITY;
              sc[mt][2 * n + (i >> 1)][2 * e + (i & 1)] = x;
              mx = fmaxf(mx, x);
            }
            mxs[mt][e] = fmaxf(mxs[mt][e], mx);
            mxo[mt][e] = fmaxf(mxo[mt][e], mx + lsv[n]);
          }
          moved |= mxs[mt][e] > m_s[mt][e] + kLag || mxo[mt][e] > m_o[mt][e] + kLag;
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float vs = mxs[mt][e], vo = mxo[mt][e];
            vs = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, 1));
            vo = fmaxf(vo, __shfl_xor_sync(0xffffffffu, vo, 1));
            vs = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, 2));
            vo = fmaxf(vo, __shfl_xor_sync(0xffffffffu, vo, 2));
            const float ns = fmaxf(m_s[mt][e], vs), no = fmaxf(m_o[mt][e], vo);
            // a row that has seen no key yet has l = 0 and O = 0
            const float al = ns == m_s[mt][e] ? 1.f : fast_exp2(m_s[mt][e] - ns);
            const float ao = no == m_o[mt][e] ? 1.f : fast_exp2(m_o[mt][e] - no);
            m_s[mt][e] = ns;
            m_o[mt][e] = no;
            l[mt][e] *= al;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[mt][n][2 * e] *= ao;
              o[mt][n][2 * e + 1] *= ao;
            }
          }
      }
      uint32_t pa[MT][C::NS][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool none = m_s[mt][e] == -INFINITY;
          const float ms = none ? 0.f : m_s[mt][e];
          const float diff = none ? 0.f : m_s[mt][e] - m_o[mt][e] + kShift;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < C::NS; ++n) {
            const float gain = fast_exp2(diff + lsv[n]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p0 = fast_exp2(sc[mt][2 * n + i][2 * e] - ms);
              const float p1 = fast_exp2(sc[mt][2 * n + i][2 * e + 1] - ms);
              sum += p0 + p1;
              pa[mt][n][2 * i + e] = pack_half2(p0 * gain, p1 * gain);
            }
          }
          l[mt][e] += sum;
        }

      // ---- a token that some row does not see may hold a NaN code in V, and
      // 0 * NaN is NaN: such codes become 0, and the columns of the rows that
      // do see the token become NaN
#pragma unroll
      for (int n = 0; n < C::NS; ++n) {
        if (j0[n] + nv[n] <= lim_min) continue;
#pragma unroll 1
        for (int w = lane; w < C::TILE / 4; w += 32) {
          const int r = w / (D / 4), col = (w - r * (D / 4)) * 4;
          uint32_t *word = reinterpret_cast<uint32_t *>(
              smem + warp * kRingBytes + st * C::STAGE + (2 * n + 1) * C::TILE + tile_at<D>(r, col >> 4) +
              (col & 15));
          const uint32_t nan4 = __vcmpeq4(*word & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
          unsigned who = __ballot_sync(0xffffffffu, nan4 != 0);
          if (nan4) *word &= ~nan4;
          for (; who; who &= who - 1) {
            const int from = __ffs(who) - 1;
            const uint32_t bytes = __shfl_sync(0xffffffffu, nan4, from);
            const int rr = __shfl_sync(0xffffffffu, r, from), cc = __shfl_sync(0xffffffffu, col, from);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int k = 0; k < D / 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int at = 16 * (k >> 1) + (k & 1) + 4 * t + 2 * (e & 1) - cc;   // column within the word
                  if (at >= 0 && at < 4 && ((bytes >> (8 * at)) & 1u) && j0[n] + rr < lim[mt][e >> 1])
                    o[mt][k][e] = __uint_as_float(0x7FC00000u);
                }
          }
        }
        __syncwarp();
      }

      // ---- O += P V: ldmatrix.trans hands out pairs of columns of two
      // tokens; a byte swap makes them pairs of tokens of one column
#pragma unroll
      for (int n = 0; n < C::NS; ++n)
#pragma unroll
        for (int c = 0; c < C::CH; c += 2) {
          uint32_t vb[4];   // chunk c: tokens 0-7, 8-15; chunk c + 1: the same
          ldsm4_trans(stage + (2 * n + 1) * C::TILE + tile_at<D>((lane & 7) + (lane & 8), c + (lane >> 4)), vb);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w0 = __byte_perm(vb[2 * i], 0, 0x3120), w1 = __byte_perm(vb[2 * i + 1], 0, 0x3120);
            const uint32_t e0 = e4m3x2_to_half2(w0), e1 = e4m3x2_to_half2(w1);
            const uint32_t d0 = e4m3x2_to_half2(w0 >> 16), d1 = e4m3x2_to_half2(w1 >> 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16(o[mt][2 * (c + i)], pa[mt][n], e0, e1);       // columns 16 (c + i) + 2 k
              mma_f16(o[mt][2 * (c + i) + 1], pa[mt][n], d0, d1);   // and + 1
            }
          }
        }
      st = st + 1 == C::STAGES ? 0 : st + 1;
    }
    cp_async_wait<0>();

    // ---- the four warps' results joined: each row's log-sum-exp first
    const int rows = min(C::ROWS, p.R - r0);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[mt][e];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        l[mt][e] = v;
        if (t == 0) stat[warp * C::ROWS + mt * 16 + g + 8 * e] = v == 0.f ? -INFINITY : m_s[mt][e] + log2f(v);
      }
    __syncthreads();
    // o of columns 16 c + 4 t .. + 3 lies in two accumulators
    float *mine = reinterpret_cast<float *>(smem + warp * kRingBytes);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + g + 8 * e;
        if (r >= rows) continue;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w * C::ROWS + r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          sum += stat[w * C::ROWS + r] == -INFINITY ? 0.f : fast_exp2(stat[w * C::ROWS + r] - top);
        // O / l_warp * 2^{L_warp - L}, O being in units of 2^{M - shift - m}
        const float f = l[mt][e] == 0.f ? 0.f
                                        : fast_exp2(m_o[mt][e] - kShift - m_s[mt][e]) / l[mt][e] *
                                              (fast_exp2(stat[warp * C::ROWS + r] - top) / sum);
#pragma unroll
        for (int c = 0; c < C::CH; ++c)
          *reinterpret_cast<float4 *>(mine + r * D + 16 * c + 4 * t) =
              make_float4(o[mt][2 * c][2 * e] * f, o[mt][2 * c + 1][2 * e] * f,
                          o[mt][2 * c][2 * e + 1] * f, o[mt][2 * c + 1][2 * e + 1] * f);
      }
    __syncthreads();
    const bool final = g0 == 0 && g1 == ng;
    const long long part = ((long long)blockIdx.x * 2 + (g0 == 0 ? 1 : 0)) * p.prows;
    for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
      const int r = i / (D / 4), c4 = i - r * (D / 4);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4 *>(smem + w * kRingBytes + (r * D + 4 * c4) * 4);
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      }
      if (final)
        *reinterpret_cast<uint2 *>(p.o + (row_base + r0 + r) * D + 4 * c4) =
            make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      else
        *reinterpret_cast<float4 *>(p.o_part + (part + r) * D + 4 * c4) = a;
    }
    if ((int)threadIdx.x < rows) {
      const int r = threadIdx.x;
      float top = -INFINITY, sum = 0.f;
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w * C::ROWS + r]);
      for (int w = 0; w < kWarps; ++w)
        sum += stat[w * C::ROWS + r] == -INFINITY ? 0.f : fast_exp2(stat[w * C::ROWS + r] - top);
      const float L2 = sum == 0.f ? -INFINITY : top + log2f(sum);
      if (final) p.lse[row_base + r0 + r] = L2 * 0.69314718055994531f;
      else p.l_part[part + r] = L2;
    }
    __syncthreads();   // rings and statistics are free again
  }
}

template <int PER>
__device__ __forceinline__ void load_floats(const float *src, float (&v)[PER]) {
  if constexpr (PER == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(src);
    v[0] = x.x; v[1] = x.y;
  } else {
#pragma unroll
    for (int e = 0; e < PER; e += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(src + e);
      v[e] = x.x; v[e + 1] = x.y; v[e + 2] = x.z; v[e + 3] = x.w;
    }
  }
}

// Joins the pieces of the units that several CTAs covered, one CTA per query
// row; rows of sequences without tokens become O = 0, L = -inf.
constexpr int kMergeWarps = 8;

template <int D, int MT>
__global__ void __launch_bounds__(kMergeWarps * 32) fwd_cache_merge_kernel(const RowParams p) {
  using C = RowCfg<D, MT>;
  __shared__ float s_o[kMergeWarps][D], s_w[kMaxCtas];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x;
  const int b = row / (p.Hq * p.Nq), hr = row - b * p.Hq * p.Nq;   // row within the sequence
  const int h = hr / p.R, r = hr - h * p.R, tile = r / C::ROWS, rr = r - tile * C::ROWS;
  const int ng = granules_of(p, b);
  __nv_bfloat16 *dst = p.o + (long long)row * D;
  if (ng == 0) {
    wait_for_primary();
    if (threadIdx.x < D / 2) reinterpret_cast<uint32_t *>(dst)[threadIdx.x] = 0u;
    if (threadIdx.x == 0) {
      p.lse[row] = -INFINITY;
      if (p.lens[b] < 0) atomicOr(p.err, kErrPage);
    }
    return;
  }
  long long total, first;
  line_of(p, b, &total, &first);
  const int units = p.Hkv * p.tiles;
  const long long per = (total * units + p.ctas - 1) / p.ctas;
  first = first * units + ((long long)h * p.tiles + tile) * ng;
  const int c0 = (int)(first / per), n = (int)((first + ng - 1) / per) - c0 + 1;
  // every CTA waits, so that what follows in the stream finds o and lse whole
  wait_for_primary();
  if (n == 1) return;
  // piece i: the unit's start lies in the second slot of CTA c0, the rest in first ones
  auto at = [&](int i) { return ((long long)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * p.prows + rr; };
  constexpr int PER = D / 32, AHEAD = 8;
  const float *src = p.o_part + lane * PER;
  // warp w adds pieces w, w + 8, ...: the first loads go out before the weights are known
  float v[AHEAD][PER];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (warp + kMergeWarps * k < n) load_floats<PER>(src + at(warp + kMergeWarps * k) * D, v[k]);
  float top = -INFINITY, sum = 0.f;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, p.l_part[at(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  for (int i = lane; i < n; i += 32) {
    const float x = p.l_part[at(i)];
    const float w = x == -INFINITY ? 0.f : fast_exp2(x - top);
    sum += w;
    if (i % kMergeWarps == warp) s_w[i] = w;   // each warp keeps its own pieces' weights
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  __syncwarp();
  float acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int i0 = warp; i0 < n; i0 += AHEAD * kMergeWarps) {
    if (i0 != warp) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (i0 + kMergeWarps * k < n) load_floats<PER>(src + at(i0 + kMergeWarps * k) * D, v[k]);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (i0 + kMergeWarps * k < n) {
        const float w = s_w[i0 + kMergeWarps * k];
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
      }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < PER; ++e) s_o[warp][lane * PER + e] = acc[e] * inv;
  __syncthreads();
  if (threadIdx.x < D / 2) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      x += s_o[w][2 * threadIdx.x];
      y += s_o[w][2 * threadIdx.x + 1];
    }
    reinterpret_cast<uint32_t *>(dst)[threadIdx.x] = pack_bf16x2(x, y);
  }
  if (threadIdx.x == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

// Rows of a tile: 32 where more than 16 rows read a key/value head and O's
// registers allow it (d <= 128), else 16.
int tile_rows(double R, int d) { return R > 16 && d <= 128 ? 32 : 16; }

// What the host knows of the work: rows, tiles, CTAs (two per SM, fewer when
// the block table has room for fewer granules).
struct RowPlan {
  double R;
  int rows, prows;
  long long tiles;
  int ctas;
};
RowPlan plan_of(const CacheArgs &a) {
  RowPlan x;
  x.R = (double)(a.Hq / a.Hkv) * a.Nq;
  x.rows = tile_rows(x.R, a.d);
  x.prows = x.R < x.rows ? (int)x.R : x.rows;
  x.tiles = (long long)((x.R + x.rows - 1) / x.rows);
  const double most = (double)a.B * a.Hkv * x.tiles * (((long long)a.max_pages * a.page + kGranule - 1) / kGranule);
  x.ctas = most < kMaxCtas ? (int)most : kMaxCtas;
  return x;
}

template <int D, int MT>
int run_rows(const CacheArgs &a, const RowPlan &x) {
  using C = RowCfg<D, MT>;
  RowParams p;
  p.q = (const __nv_bfloat16 *)a.q;
  p.k_cache = a.k_cache; p.v_cache = a.v_cache; p.k_scale = a.k_scale; p.v_scale = a.v_scale;
  p.table = a.table; p.lens = a.lens;
  p.o = (__nv_bfloat16 *)a.o; p.lse = a.lse;
  p.o_part = (float *)a.ws;
  p.l_part = p.o_part + (size_t)x.ctas * 2 * x.prows * D;
  p.B = a.B; p.Hq = a.Hq; p.Hkv = a.Hkv; p.Nq = a.Nq;
  p.R = (int)x.R;
  p.tiles = (int)x.tiles;
  p.page_log2 = a.page == 16 ? 4 : a.page == 32 ? 5 : a.page == 64 ? 6 : 7;
  p.num_pages = a.num_pages; p.max_pages = a.max_pages;
  p.causal = a.causal; p.ctas = x.ctas; p.prows = x.prows;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.err = a.err;
  auto kern = fwd_cache_rows_kernel<D, MT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return 5;
  kern<<<x.ctas, kWarps * 32, C::SMEM, a.stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return 5;
  // The merge kernel is launched while the main one runs: its CTAs find their
  // pieces, then wait for the main kernel's end.
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hq * a.Nq), 1, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.stream = a.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fwd_cache_merge_kernel<D, MT>, p) != cudaSuccess) return 5;
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

}  // namespace

size_t fwd_cache_ws_bytes(const CacheArgs &a) {
  const RowPlan x = plan_of(a);
  return (size_t)x.ctas * 2 * x.prows * (a.d + 1) * 4;
}

int launch_fwd_cache(const CacheArgs &a) {
  const RowPlan x = plan_of(a);
  if (x.R > 2147483647.0 || (double)a.Hkv * x.tiles > 2147483647.0) return 2;
  const bool wide = x.rows == 32;
  switch (a.d) {
    case 64: return wide ? run_rows<64, 2>(a, x) : run_rows<64, 1>(a, x);
    case 128: return wide ? run_rows<128, 2>(a, x) : run_rows<128, 1>(a, x);
    case 256: return run_rows<256, 1>(a, x);
    default: return 2;
  }
}

}  // namespace fa
