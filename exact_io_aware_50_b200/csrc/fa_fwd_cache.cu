// fa_fwd_cache.cu -- attention over the paged E4M3 cache.
//
//     s_j = scale * sk * (q . K^_j),  m = max s,  l = sum 2^{s_j - m},
//     O = sum 2^{s_j - m} sv V^_j / l,  L = (m + log2 l) ln 2
//
// with s in base-2 units, sk and sv the scales of the page token j stands in.
//
// Rows: the g * Nq query rows that read one key/value head (contiguous in q)
// are cut into tiles of 16 rows, so a page is read once for all rows of a tile.
// Work: a unit is (sequence, key/value head, row tile); its tokens come in
// granules of 64.  The granules of all units, in one line, are divided evenly
// among the CTAs (two per SM), so ragged lengths, few heads and long caches all
// fill the GPU: a CTA's run may start inside one unit and end inside another.
// A unit that one CTA covers is finished there; the others leave their
// normalised partial O, m and l in the workspace, and the merge kernel joins them
// (m = max m_c, l = sum 2^{m_c - m} l_c, O = sum 2^{m_c - m} l_c O_c / l; not by m +
// log2 l, which large scores round by more than l matters).  Nothing is accumulated
// by atomics: results do not depend on timing.
//
// Each of a CTA's four warps takes 16 tokens of a granule, NS granules a step,
// into a ring of its own (three stages of 8 KB) by 16-byte asynchronous copies,
// with its own (m, l, O): the warps meet only at the end of a unit.  There the
// first copies of the CTA's next piece are issued before the warps' O are
// joined, in the stage that those copies leave free.
//
// The E4M3 codes become halves, exactly, on their way into mma.m16n8k16; q
// becomes halves too, each row times a power of two that brings its largest
// entry to [2^13, 2^14), so an entry keeps its 8 bits unless it is 2^-28 of the
// largest.  The weight that multiplies V is 2^{s - m} sv, rounded to a half.
// It has a reference M of its own, the running maximum of s + log2 sv: terms
// down to 2^-26 of the largest keep 11 bits whatever the pages' scales, and
// smaller ones err by at most 2^-37 of the largest weight.  M is kept as M - m, and
// scores are subtracted before anything is added to them, so this holds for scores of
// any size.
//
// Measured on B200, a call in a graph, Hq 32, Hkv 8, d 128: 32 sequences of 2047 to
// 16384 tokens (612 MB) 98 us = 6.2 TB/s, 95 % of a plain copy's rate, the bound of
// long batches (109 us = 5.6 TB/s called from Python); one of 16384 tokens 13.5 us, of
// which 7 are the latency of a call's two launches, the page look-up, the first copies
// and the merge.  d = 256 holds O in 128 registers a thread: B 8, Hq 16, Hkv 4, 16384
// tokens 51 us = 5.3 TB/s.  Many short sequences are bound by a unit's start and end,
// about 3.5 us of a CTA: 256 of 256 tokens 38 us = 3.5 TB/s.  Copying the next unit's
// first steps before this one's last did not shorten that (2 to 5 % slower), nor did
// copies by TMA (boxes of 2 to 8 KB, one CTA an SM: 130 us for the batch where this form
// then took 109).
#include <type_traits>

#include "fwd_cache.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kSub = 16;                        // tokens of a subtile (one page's, or part of it)
constexpr int kGranule = kWarps * kSub;
constexpr int kStage = 8 * 1024, kStages = 3;   // a warp's ring
constexpr int kRing = kStage * kStages;

template <int D>
struct RowCfg {
  static constexpr int ROWS = 16;
  // CTAs take whole units where the block table has room for this many tokens.
  // Measured, us a call in a graph with the line and with whole units, Hkv 8, Hq 32,
  // one set of inputs: d = 64, 512 tokens, B 1 7.3 / 5.5, B 64 18.0 / 11.9; d = 128, 256
  // tokens 7.3 / 5.1 and 14.6 / 11.1, 512 tokens 7.4 / 7.1 and 21.1 / 16.2 (and a launch
  // less, 3 us of the host's time); d = 256, 256 tokens 8.1 / 7.8 and 22.9 / 18.5, 512
  // tokens 7.8 / 11.5 and 37.4 / 30.2.  With a unit for every CTA (B 64; B 50 ragged; B
  // 38, eight units more than CTAs, the worst: a second round for the eight), d = 64,
  // 2048 tokens 37.2 / 33.5, 26.9 / 25.0 and 24.2 / 27.4; d = 128, 1024 tokens 33.0 /
  // 29.3, 20.1 / 21.2 and 22.0 / 23.0, 2048 tokens 50.8 / 49.4, 27.8 / 36.7 and 34.6 /
  // 43.1; d = 256, 512 tokens 37.5 / 30.2, 23.1 / 22.5 and 24.2 / 24.7, 1024 tokens 55.8 /
  // 50.1, 32.0 / 37.6 and 38.0 / 43.3.
  static constexpr int WHOLE = D == 256 ? 256 : 512, WHOLE_MANY = D == 128 ? 1024 : D == 64 ? 2048 : 512;
  // A unit's start counts as four granules.  Measured, us a call in a graph
  // with 0 / 2 / 4 / 6: one sequence of 16384 tokens (Hq 32, Hkv 8, d 128) 16.3 /
  // 15.2 / 14.1 / 14.1; 32 ragged ones to 16384 104.7 / 103.0 / 100.4 / 100.5;
  // d = 256, B 8, four drafted tokens 32.3 / 29.9 / 28.5 / 28.2.
  using L = Line<ROWS, kGranule, false, 4>;
  static constexpr int CH = D / 16;             // 16-byte chunks of a token
  static constexpr int NS = 256 / D;            // subtiles of a step
  static constexpr int TILE = kSub * D;         // K or V codes of a subtile
  // Steps copied ahead of the one at hand.  Those of the next piece are under way
  // when the warps' O are joined, in the stage that is left: JOIN columns at a time.
  static constexpr int AHEAD = kStages - 1, JOIN = D < 128 ? D : 128;
  static constexpr int QROW = D * 2 + 16;       // q rows are padded: no two of eight in one bank group
  static constexpr int OFF_Q = kWarps * kRing;
  // d = 256: O's 128 registers leave no room for q's 64, which wait in shared
  // memory, a lane's fragment of a chunk in 16 bytes
  static constexpr bool QS = D == 256;
  static constexpr int OFF_QF = OFF_Q + ROWS * QROW;
  static constexpr int OFF_SCALE = OFF_QF + (QS ? CH * 512 : 0);         // [warp][stage][NS] (sk, sv)
  static constexpr int OFF_STAT = OFF_SCALE + kWarps * kStages * NS * 8; // [warp][ROWS] (m, l)
  static constexpr int SMEM = OFF_STAT + kWarps * ROWS * 8;
  static_assert(2 * NS * TILE == kStage, "K and V codes of a step");
  static_assert(ROWS * JOIN * 4 <= kStage, "a warp's O fits beside the copies ahead");
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs an SM");
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

// 16 bytes from src + OFF.
template <int OFF>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1+%2], 16;" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
}
// 16 or 4 bytes, or zeros.
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4z(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four E4M3 codes -> halves: the lower two, the upper two.
__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t codes, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Four 8 x 8 matrices of 16-bit elements at [addr + OFF].
template <int OFF>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4+%5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF)
               : "memory");
}
template <int OFF>
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4+%5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF)
               : "memory");
}

// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, class F, int I = 0>
__device__ __forceinline__ void unroll(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<N, F, I + 1>(static_cast<F &&>(f));
  }
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

// HALF: eight rows a head or fewer, so that a lane's second row (g + 8) does not
// exist and gets no work (Hq 32, Hkv 8, d 128, us a call in a graph without and with:
// one sequence of 16384 tokens 14.6 / 13.1, 32 of 2047 to 16384 101 / 98, 1024 of 256
// tokens 163 / 135, the last two with the changes to a unit's end made beside it).
template <int D, bool HALF>
__global__ void __launch_bounds__(kWarps * 32, 2) fwd_cache_rows_kernel(const FwdCacheParams p) {
  using C = RowCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = warp_id_uniform(), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  launch_dependents();   // the merge kernel's CTAs may take their places
  Run<typename C::L> run;
  if (!run.start(p) || !run.template next<D>(p, warp == 0)) return;

  const uint32_t sbase = smem_u32(smem), ring = sbase + warp * kRing;
  float2 *scales = reinterpret_cast<float2 *>(smem + C::OFF_SCALE) + warp * kStages * C::NS;
  float2 *stat = reinterpret_cast<float2 *>(smem + C::OFF_STAT);   // [warp][ROWS]
  const uint32_t copy_dst = tile_at<D>(lane / C::CH, lane % C::CH);
  // this lane's row and chunk of a tile's first ldmatrix of K and of V
  const uint32_t k_off = tile_at<D>(lane & 7, lane >> 3), v_off = tile_at<D>(lane & 15, lane >> 4);

  // ---- copies.  Lane i holds the page number of the warp's subtile 32 k + i
  // of the piece, and of the 32 after them.
  int cur, nxt;
  auto token_of = [&](int i) { return (run.g0 + i) * kGranule + warp * kSub; };
  // fetched first and looked at later, so that a load is not waited for
  auto fetch = [&](int i) {
    const int j = token_of(i);
    return j >= run.stop ? 0 : p.table[(long long)run.b * p.max_pages + (j >> p.page_log2)];
  };
  auto checked = [&](int pg, int i) {
    if (token_of(i) >= run.stop) return -1;
    if ((unsigned)pg < (unsigned)p.num_pages) return pg;
    atomicOr(p.err, kErrPage);
    return -1;
  };
  auto fetch_first = [&]() {
    cur = fetch(lane);
    nxt = fetch(32 + lane);
  };
  // Step s of the piece into stage st; always one commit group a step.  What
  // is no token of the piece becomes zeros, and its page's scales too.
  auto issue = [&](int s, int st) {
    const int i0 = s * C::NS;
    if (i0 < run.g1 - run.g0) {
      if (i0 && (i0 & 31) == 0) {
        cur = checked(nxt, i0 + lane);
        nxt = fetch(i0 + 32 + lane);
      }
#pragma unroll
      for (int n = 0; n < C::NS; ++n) {
        const int pg = __shfl_sync(0xffffffffu, cur, (i0 + n) & 31);
        const int j = token_of(i0 + n);
        const long long page_h = (long long)max(pg, 0) * p.Hkv + run.h;
        const long long at = ((page_h << p.page_log2) + (j & ((1 << p.page_log2) - 1))) * D + lane * 16;
        const uint8_t *ks = p.k_cache + at, *vs = p.v_cache + at;
        const uint32_t dst = ring + st * kStage + 2 * n * C::TILE;
        if (pg >= 0 && j + kSub <= run.stop) {
          unroll<C::TILE / 512>([&](auto i) {
            cp_async16<512 * i>(dst + tile_chunk<D>(copy_dst, i), ks);
            cp_async16<512 * i>(dst + C::TILE + tile_chunk<D>(copy_dst, i), vs);
          });
        } else {
          const int live = pg < 0 ? 0 : (run.stop - j) * C::CH;   // chunks
          unroll<C::TILE / 512>([&](auto i) {
            const bool in = 32 * i + lane < live;
            cp_async16z(dst + tile_chunk<D>(copy_dst, i), in ? ks + 512 * i : p.k_cache, in);
            cp_async16z(dst + C::TILE + tile_chunk<D>(copy_dst, i), in ? vs + 512 * i : p.v_cache, in);
          });
        }
        if (lane < 2)
          cp_async4z(smem_u32(scales + st * C::NS + n) + 4 * lane, (lane ? p.v_scale : p.k_scale) + page_h,
                     pg >= 0);
      }
    }
    cp_async_commit();
  };
  // The piece's q rows and, its first pages fetched, first AHEAD steps, from stage st on.
  auto begin = [&](int st) {
    const int rows = min(C::ROWS, p.R - run.r0);
    const uint8_t *q = (const uint8_t *)(p.q + (((long long)run.b * p.Hkv + run.h) * p.R + run.r0) * D);
    for (int i = threadIdx.x; i < rows * 2 * C::CH; i += kWarps * 32)   // a head's R rows lie together
      cp_async16<0>(sbase + C::OFF_Q + i / (2 * C::CH) * C::QROW + i % (2 * C::CH) * 16, q + i * 16);
    cur = checked(cur, lane);
#pragma unroll
    for (int k = 0; k < C::AHEAD; ++k) issue(k, (st + k) % kStages);
    if (threadIdx.x == 0) (void)checked_len(p.lens, run.b, p.max_pages, 1 << p.page_log2, p.err);
  };

  int st = 0;   // stage of the step at hand
  fetch_first();
  begin(st);
  while (true) {
    // the piece at hand (`run` moves on before its merge)
    const int subs = run.g1 - run.g0, steps = (subs + C::NS - 1) / C::NS;
    const int rows = min(C::ROWS, p.R - run.r0), len = run.len, stop = run.stop;
    const int token = token_of(0);   // of this warp; its subtile i starts kGranule * i later

    // ---- q: A fragments of halves, each row times a power of two
    cp_async_wait<C::AHEAD - 1>();   // q came with the first step
    __syncthreads();
    uint32_t qa[C::CH][4];
    float row_c[2];        // scale * log2 e / that power of two
    int lim[2];            // keys [0, lim) visible
    int lim_min = len;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      const bool live = r < rows;
      row_c[e] = 0.f;
      lim[e] = 0;
      if (HALF && e) {
#pragma unroll
        for (int c = 0; c < C::CH; ++c) qa[c][1] = qa[c][3] = 0u;
        continue;
      }
      const uint8_t *src = smem + C::OFF_Q + r * C::QROW + 8 * t;
      uint2 raw[C::CH];
      float mx = 0.f;
#pragma unroll
      for (int c = 0; c < C::CH; ++c) {
        raw[c] = live ? *reinterpret_cast<const uint2 *>(src + 32 * c) : make_uint2(0u, 0u);
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(raw[c].x << 16)),
                             fabsf(__uint_as_float(raw[c].x & 0xFFFF0000u))));
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(raw[c].y << 16)),
                             fabsf(__uint_as_float(raw[c].y & 0xFFFF0000u))));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // mx in [2^k, 2^{k+1}); zero rows and exponents past float32's reach are cut off
      const int k = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 126);
      const float up = __uint_as_float((uint32_t)(13 - k + 127) << 23);
      row_c[e] = p.scale_log2 * __uint_as_float((uint32_t)(k - 13 + 127) << 23);
#pragma unroll
      for (int c = 0; c < C::CH; ++c) {
        qa[c][e] = pack_half2(__uint_as_float(raw[c].x << 16) * up,
                              __uint_as_float(raw[c].x & 0xFFFF0000u) * up);
        qa[c][2 + e] = pack_half2(__uint_as_float(raw[c].y << 16) * up,
                                  __uint_as_float(raw[c].y & 0xFFFF0000u) * up);
      }
      lim[e] = !live ? 0 : (p.causal ? max(0, len - p.Nq + (run.r0 + r) % p.Nq + 1) : len);
      if (live) lim_min = min(lim_min, lim[e]);
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    uint4 *qf = reinterpret_cast<uint4 *>(smem + C::OFF_QF) + lane;
    if constexpr (C::QS) {   // all warps hold the same fragments: each stores a quarter
#pragma unroll
      for (int c = 0; c < C::CH; ++c)
        if (c / (C::CH / kWarps) == warp) qf[32 * c] = make_uint4(qa[c][0], qa[c][1], qa[c][2], qa[c][3]);
      __syncthreads();
    }

    float o[D / 8][4];
    float m_s[2], m_d[2], l[2];   // m, M - m, sum of 2^{s - m}
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m_s[e] = -INFINITY;
      m_d[e] = l[e] = 0.f;
    }

#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      cp_async_wait<C::AHEAD - 1>();   // step s has landed
      __syncwarp();
      if (s + C::AHEAD < steps) issue(s + C::AHEAD, (st + C::AHEAD) % kStages);
      else cp_async_commit();
      const uint32_t kt = ring + st * kStage, vt = kt + C::TILE;

      // ---- S = q K^T: two groups of 8 tokens a subtile
      float sc[2 * C::NS][4];
#pragma unroll
      for (int n = 0; n < 2 * C::NS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
      // (chunk c + x of a row lies at the place of chunk x with c << 4 flipped,
      // where x is below the multiple c of a power of two)
      unroll<C::CH / 4>([&](auto ci) {
        constexpr int c = 4 * ci;
        const uint32_t at = kt + (k_off ^ (c << 4));
        uint32_t qc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (C::QS) {
            const uint4 x = qf[32 * (c + i)];
            qc[i][0] = x.x; qc[i][1] = x.y; qc[i][2] = x.z; qc[i][3] = x.w;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) qc[i][k] = qa[c + i][k];
          }
        }
        unroll<2 * C::NS>([&](auto n) {
          uint32_t kb[4];
          ldsm4<(n >> 1) * 2 * C::TILE + 8 * (n & 1) * D>(at, kb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            e4m3x4_to_half2x2(kb[i], b0, b1);
            mma_f16(sc[n], qc[i], b0, b1);
          }
        });
      });

      // ---- softmax
      float sk[C::NS], lsv[C::NS];
      int j0[C::NS], nv[C::NS];
      bool whole = true;
#pragma unroll
      for (int n = 0; n < C::NS; ++n) {
        const float2 x = scales[st * C::NS + n];
        j0[n] = token + (s * C::NS + n) * kGranule;
        nv[n] = x.y > 0.f ? min(kSub, stop - j0[n]) : 0;
        sk[n] = x.x;
        lsv[n] = nv[n] > 0 ? __log2f(x.y) : 0.f;
        whole = whole && nv[n] == kSub && j0[n] + kSub <= lim_min;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int n = 0; n < C::NS; ++n) {
          if (HALF && e) continue;
          const float cf = row_c[e] * sk[n];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float &x = sc[2 * n + (i >> 1)][2 * e + (i & 1)];
            x = __fmul_rn(x, cf);   // rounded before m is subtracted: equal scores, equal powers
          }
        }
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int n = 0; n < C::NS; ++n) {
            if (HALF && e) continue;
            const int seen = min(nv[n], lim[e] - j0[n]) - 2 * t;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (8 * (i >> 1) + (i & 1) >= seen) sc[2 * n + (i >> 1)][2 * e + (i & 1)] = -INFINITY;
          }
      }
      // Scores may be of any size, so they are compared by their differences, which
      // are exact where they are small.
      bool moved = false, over = false;   // over: some weight's factor passes 2^kOver
      float mx[2][C::NS];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (HALF && e) continue;
        float mxs = -INFINITY, mxo = -INFINITY;   // of s, of s - m + log2 sv
#pragma unroll
        for (int n = 0; n < C::NS; ++n) {
          float v = sc[2 * n][2 * e];
#pragma unroll
          for (int i = 1; i < 4; ++i) v = fmaxf(v, sc[2 * n + (i >> 1)][2 * e + (i & 1)]);
          mx[e][n] = v;
          mxs = fmaxf(mxs, v);
          mxo = fmaxf(mxo, v - m_s[e] + lsv[n]);   // infinite for a row's first keys
          moved |= lsv[n] - m_d[e] > kOver - kShift;
        }
        moved |= mxs - m_s[e] > kLag || mxo > m_d[e] + kLag;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (HALF && e) continue;
          float ns = m_s[e];
#pragma unroll
          for (int n = 0; n < C::NS; ++n) ns = fmaxf(ns, mx[e][n]);
          ns = fmaxf(ns, __shfl_xor_sync(0xffffffffu, ns, 1));
          ns = fmaxf(ns, __shfl_xor_sync(0xffffffffu, ns, 2));
          // a row that has seen no key yet has l = 0 and O = 0
          const float shift = ns == m_s[e] ? 0.f : m_s[e] - ns;
          float nd = shift + m_d[e];
#pragma unroll
          for (int n = 0; n < C::NS; ++n) nd = fmaxf(nd, mx[e][n] - ns + lsv[n]);
          nd = fmaxf(nd, __shfl_xor_sync(0xffffffffu, nd, 1));
          nd = fmaxf(nd, __shfl_xor_sync(0xffffffffu, nd, 2));
          const float al = fast_exp2(shift), ao = fast_exp2(shift + (m_d[e] - nd));   // 1 where nothing moved
          m_s[e] = ns;
          m_d[e] = nd;
          l[e] *= al;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * e] *= ao;
            o[n][2 * e + 1] *= ao;
          }
#pragma unroll
          for (int n = 0; n < C::NS; ++n) over |= lsv[n] - nd > kOver - kShift;
        }
        over = __any_sync(0xffffffffu, over);
      }
      uint32_t pa[C::NS][4];
      float ms[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (HALF && e) {
#pragma unroll
          for (int n = 0; n < C::NS; ++n) pa[n][1] = pa[n][3] = 0u;
          continue;
        }
        ms[e] = m_s[e] == -INFINITY ? 0.f : m_s[e];
      }
      // sums of a row's tokens' powers, and their weights
      auto weigh = [&](auto apart) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (HALF && e) continue;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < C::NS; ++n) {
            const float up = kShift - m_d[e] + lsv[n], gain = fast_exp2(up);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x0 = sc[2 * n + i][2 * e] - ms[e], x1 = sc[2 * n + i][2 * e + 1] - ms[e];
              const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
              sum += p0 + p1;
              pa[n][2 * i + e] = apart ? pack_half2(p0 * gain, p1 * gain)
                                       : pack_half2(fast_exp2(x0 + up), fast_exp2(x1 + up));
            }
          }
          l[e] += sum;
        }
      };
      if (over) weigh(std::false_type{});
      else weigh(std::true_type{});

      // ---- a token that some row does not see may hold a NaN code in V, and
      // 0 * NaN is NaN: such codes become 0, and the columns of the rows that
      // do see the token become NaN
      if (!whole) {
#pragma unroll 1
        for (int n = 0; n < C::NS; ++n) {
          const int j = token + (s * C::NS + n) * kGranule;
          if (min(j + kSub, stop) <= lim_min) continue;
          uint8_t *v = smem + warp * kRing + st * kStage + (2 * n + 1) * C::TILE;
          // a look at the whole tile first (four drafted tokens over 512, d = 256, B 8:
          // 15.5 us a call without it, 13.3 with): only a NaN's byte carries into bit 7
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < C::TILE / 512; ++i) {
            const uint4 x = reinterpret_cast<const uint4 *>(v)[32 * i + lane];
            top |= ((x.x & 0x7F7F7F7Fu) + 0x01010101u) | ((x.y & 0x7F7F7F7Fu) + 0x01010101u) |
                   ((x.z & 0x7F7F7F7Fu) + 0x01010101u) | ((x.w & 0x7F7F7F7Fu) + 0x01010101u);
          }
          if (!__any_sync(0xffffffffu, top & 0x80808080u)) continue;
#pragma unroll 1
          for (int w = lane; w < C::TILE / 4; w += 32) {
            const int r = w / (D / 4), col = (w - r * (D / 4)) * 4;
            uint32_t *word = reinterpret_cast<uint32_t *>(v + tile_at<D>(r, col >> 4) + (col & 15));
            const uint32_t x = *word, nan4 = __vcmpeq4(x & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            unsigned who = __ballot_sync(0xffffffffu, nan4 != 0);
            if (nan4) *word = x & ~nan4;
            for (; who; who &= who - 1) {
              const int from = __ffs(who) - 1;
              const uint32_t bytes = __shfl_sync(0xffffffffu, nan4, from);
              const int rr = __shfl_sync(0xffffffffu, r, from), cc = __shfl_sync(0xffffffffu, col, from);
#pragma unroll
              for (int k = 0; k < D / 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int at = 16 * (k >> 1) + (k & 1) + 4 * t + 2 * (e & 1) - cc;   // column within the word
                  if (at >= 0 && at < 4 && ((bytes >> (8 * at)) & 1u) && j + rr < lim[e >> 1])
                    o[k][e] = __uint_as_float(0x7FC00000u);
                }
            }
          }
        }
        __syncwarp();
      }

      // ---- O += P V: ldmatrix.trans hands out pairs of columns of two
      // tokens; a byte swap makes them pairs of tokens of one column
      unroll<C::CH / 2>([&](auto ci) {
        constexpr int c = 2 * ci;
        const uint32_t at = vt + (v_off ^ (c << 4));
        unroll<C::NS>([&](auto n) {
          uint32_t vb[4];   // chunk c: tokens 0-7, 8-15; chunk c + 1: the same
          ldsm4_trans<n * 2 * C::TILE>(at, vb);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t e0, e1, d0, d1;
            e4m3x4_to_half2x2(__byte_perm(vb[2 * i], 0, 0x3120), e0, d0);
            e4m3x4_to_half2x2(__byte_perm(vb[2 * i + 1], 0, 0x3120), e1, d1);
            mma_f16(o[2 * (c + i)], pa[n], e0, e1);       // columns 16 (c + i) + 2 k
            mma_f16(o[2 * (c + i) + 1], pa[n], d0, d1);   // and + 1
          }
        });
      });
      st = st + 1 == kStages ? 0 : st + 1;
    }

    // ---- on to the next piece: its pages are looked up, and its first copies go
    // out before the merge
    const long long row0 = ((long long)run.b * p.Hkv + run.h) * p.R + run.r0;
    const int part = run.part(p);
    const bool more = run.template next<D>(p, warp == 0);
    if (more) fetch_first();
    // each row's m and l in this warp
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (HALF && e) continue;
      float v = l[e];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      l[e] = v;
      if (t == 0) stat[warp * C::ROWS + g + 8 * e] = make_float2(m_s[e], v);
    }
    __syncthreads();   // every warp is done with q and its ring
    if (more) begin(st);

    // ---- the four warps' results joined
    // row r of a warp's O: the stage that the copies ahead leave
    auto o_at = [&](int w, int r) {
      return reinterpret_cast<float4 *>(smem + w * kRing + (st + C::AHEAD) % kStages * kStage + r * C::JOIN * 4);
    };
    // O's factor 2^{m_warp - m} 2^{M - shift - m_warp} / l as two, its power's root and
    // the rest: a page of tiny V brings the power near float32's end, a distant
    // maximum past it, where the whole product is not
    float f0[2], f1[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      if (HALF && e) continue;
      float2 ml[kWarps];
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = stat[w * C::ROWS + r];
        top = fmaxf(top, ml[w].x);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += ml[w].y == 0.f ? 0.f : fast_exp2(ml[w].x - top) * ml[w].y;
      f0[e] = l[e] == 0.f ? 0.f : fast_exp2(0.5f * (m_s[e] - top + (m_d[e] - kShift)));
      f1[e] = l[e] == 0.f ? 0.f : __fdividef(f0[e], sum);   // sum is below 2^32
      if (warp == 0 && t == 0 && r < rows) {
        if (part < 0) p.lse[row0 + r] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        else p.l_part[part + r] = make_float2(top, sum);
      }
    }
#pragma unroll
    for (int half = 0; half < D / C::JOIN; ++half) {
      if (half) __syncthreads();   // the columns before have been read
      // o of columns 16 c + 4 t .. + 3 lies in two accumulators
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e;
        if (r >= rows) continue;
        float4 *dst = o_at(warp, r) + t;
#pragma unroll
        for (int i = 0; i < C::JOIN / 16; ++i) {
          const int c = half * (C::JOIN / 16) + i;
          dst[4 * i] = make_float4(o[2 * c][2 * e] * f1[e] * f0[e], o[2 * c + 1][2 * e] * f1[e] * f0[e],
                                   o[2 * c][2 * e + 1] * f1[e] * f0[e], o[2 * c + 1][2 * e + 1] * f1[e] * f0[e]);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < rows * (C::JOIN / 4); i += kWarps * 32) {
        const int r = i / (C::JOIN / 4), c4 = i - r * (C::JOIN / 4), col = half * C::JOIN + 4 * c4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 x = o_at(w, r)[c4];
          a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        }
        if (part < 0)
          *reinterpret_cast<uint2 *>(p.o + (row0 + r) * D + col) =
              make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        else
          *reinterpret_cast<float4 *>(p.o_part + (long long)(part + r) * D + col) = a;
      }
    }
    if (!more) return;
    // (the barrier before q is read frees the ring and the statistics)
  }
}

template <int D>
int run_rows(const CacheArgs &a, const FwdCachePlan &x) {
  using C = RowCfg<D>;
  const FwdCacheParams p = fwd_cache_params(a, x);
  const bool half = p.R <= C::ROWS / 2;
  auto kern = half ? fwd_cache_rows_kernel<D, true> : fwd_cache_rows_kernel<D, false>;
  static unsigned long long allowed[2] = {0, 0};
  if (!allow_smem(kern, C::SMEM, &allowed[half])) return 5;
  kern<<<x.ctas, kWarps * 32, C::SMEM, a.stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return 5;
  return launch_fwd_cache_merge<D, typename C::L>(p, a.stream);
}

// Up to three tiles of 16 rows (five at d = 64) go to the kernel of this file,
// which reads the cache for each (a cache larger than L2 from DRAM each time: 48 rows
// over 524 MB read 1579, 20 rows 1052, counted), converts and multiplies it anew; more
// rows read it once for 128 of them on tcgen05 (fa_fwd_cache_sm100.cu).  Measured on
// B200, us a call in a graph here / there, B 32, 8000 tokens, 2 key/value heads: d = 64,
// 80 rows 78.4 / 82.7, 96 rows 92.3 / 83.0; d = 128, 48 rows 72.5 / 84.9, 64 rows 89.6 /
// 85.1; d = 256, 48 rows 124 / 119; B 1, 16000 tokens, 8 heads, 48 rows at d = 256 39.9 /
// 44.2; B 16, 400 tokens, 8 heads, 80 rows at d = 64 20.5 / 16.4, 40 rows at d = 256
// 27.0 / 21.9.
bool few_rows(const CacheArgs &a) {
  return (double)(a.Hq / a.Hkv) * a.Nq <= (a.d == 64 ? 5 : 3) * 16;
}

FwdCachePlan plan_of(const CacheArgs &a) {
  if (!few_rows(a)) return fwd_cache_tile_plan(a);
  return a.d == 64    ? fwd_cache_plan<RowCfg<64>::L>(a, kMaxCtas, RowCfg<64>::WHOLE, RowCfg<64>::WHOLE_MANY)
         : a.d == 128 ? fwd_cache_plan<RowCfg<128>::L>(a, kMaxCtas, RowCfg<128>::WHOLE, RowCfg<128>::WHOLE_MANY)
                      : fwd_cache_plan<RowCfg<256>::L>(a, kMaxCtas, RowCfg<256>::WHOLE, RowCfg<256>::WHOLE_MANY);
}

}  // namespace

size_t fwd_cache_ws_bytes(const CacheArgs &a) { return fwd_cache_plan_bytes(plan_of(a), a.d); }
double fwd_cache_granules(const CacheArgs &a) { return plan_of(a).most; }

int launch_fwd_cache(const CacheArgs &a) {
  const FwdCachePlan x = plan_of(a);
  if (!few_rows(a)) return launch_fwd_cache_tiles(a, x);
  switch (a.d) {
    case 64: return run_rows<64>(a, x);
    case 128: return run_rows<128>(a, x);
    case 256: return run_rows<256>(a, x);
    default: return 2;
  }
}

}  // namespace fa
