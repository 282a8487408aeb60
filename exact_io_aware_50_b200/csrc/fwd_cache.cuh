// fwd_cache.cuh -- what the two kernels of attention over the paged cache share:
// parameters, the division of the work among CTAs, the merge of partial results.
#pragma once

#include <math.h>

#include "cache.cuh"

namespace fa {

// Programmatic dependent launch: the next kernel of the stream may start; a
// dependent kernel waits here until the one before it has ended.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_primary() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr int kMaxCtas = 2 * 148;   // CTAs of a launch, at most
constexpr float kLag = 3.f;         // a maximum may lag by 2^3
constexpr float kShift = 12.f;      // weights are stored times 2^12: at most 2^15
// A weight 2^{s - m} * 2^up, up = m - M + kShift + log2 sv, is the product of its two
// powers where up is at most this (the second is the same for a page's tokens), and
// one power of the exponents' sum where it is more: there 2^up nears float32's end,
// and infinity times the 0 of a hidden or distant token is NaN.  Up to 2^100, a first
// power that is flushed to 0 (below 2^-126) stands for less than 2^-26, which is 0 as
// a half.  Pages of zeros make up large: their scale is 2^-112.
constexpr float kOver = 100.f;

struct FwdCacheParams {
  const __nv_bfloat16 *q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *table, *lens;
  __nv_bfloat16 *o;
  float *lse;
  float *o_part;            // [ctas][2][prows][D], normalised
  float2 *l_part;           // [ctas][2][prows] (m, l): maximum (base 2) and sum
  int B, Hq, Hkv, Nq, g, R, tiles;   // R = g * Nq rows of a key/value head, in `tiles` tiles
  int page_log2, num_pages, max_pages;
  int causal, ctas, prows;   // prows: rows of a partial, min(R, rows of a tile)
  int whole;                 // CTAs take whole units in turn: no line, no partials, no merge
  float scale_log2;
  unsigned long long g_inv;   // ceil(2^64 / g), 0 for g = 1
  unsigned *err;
};

// x / p.g, x >= 0: below 2^32 a product, which is exact (the excess of g_inv g over
// 2^64 is less than g < 2^31, so x times it stays below 2^64).
__device__ __forceinline__ long long div_g(long long x, int g, unsigned long long g_inv) {
  if (x >> 32) return x / g;
  return g_inv ? (long long)__umul64hi((unsigned long long)x, g_inv) : x;
}

// The parts of the line (below) of the tiles before `tile`, causal, for tiles of
// 128 NT rows and granules of 128 tokens: tile t but the last sees floor((NT t + c)
// / g) granules where that is positive, with c = floor(((len - Nq + 128) g + 128 NT
// - 1) / 128), so the sum has a closed form.  With t0 the first tile that sees a
// token, n = tile - t0 and NT t0 + c = base g + rest it is
//     n (base + START) + sum_{i < n} floor((NT i + rest) / g),
// whose last sum counts, for k = 1 .. K = floor((NT (n - 1) + rest) / g), the i with
// NT i + rest >= k g: K n - sum_k ceil((k g - rest) / NT).  (A tile by tile sum took
// 3.4 ms of a square causal call of 8192 queries, Hq 32, Hkv 8, d 128: all else 0.8.)
template <int NT, int START>
__device__ __forceinline__ int parts_before(int tile, int len, int Nq, int g, unsigned long long g_inv) {
  static_assert(NT == 1 || NT == 2, "the odd terms");
  long long c = ((long long)(len - Nq + 128) * g + 128 * NT - 1) >> 7, t0 = 0;
  if (c < g) {
    t0 = (g - c + NT - 1) / NT;
    c += NT * t0;
  }
  if (tile <= t0) return 0;
  const long long base = div_g(c, g, g_inv), rest = c - base * g, n = tile - t0;
  const long long K = div_g(NT * (n - 1) + rest, g, g_inv);
  long long up = g * (K * (K + 1) / 2) - K * rest;   // sum of k g - rest
  if (NT == 2) up = (up + (g & 1 ? (K + 1 - (rest & 1)) / 2 : K * (rest & 1))) / 2;   // the odd ones round up
  return (int)(n * (base + START) + K * n - up);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The work: a unit is (sequence, key/value head, tile of ROWS query rows), its
// tokens in granules of GRANULE.  The granules of all units stand in one line
// (sequences in order, each its heads, each its tiles; fewer than 2^31: the
// launcher checks), which is cut into p.ctas even runs.  A unit that begins in a
// run costs its CTA some time before and after its granules: each unit stands in
// the line with START empty granules in front, so that a CTA that ends one unit
// and begins another gets less of them.  Where the block table has room for few
// tokens only (p.whole), CTA c takes units c, c + p.ctas, ... from end to end
// instead, and there is nothing to merge.
//
// QMAJOR: row r of a head is query r / g of its group's head r % g, so a tile
// holds consecutive queries and, causal, sees no further than its last one;
// else row r is query r % Nq of head r / Nq, the order of memory, and every tile
// of a sequence has the same granules.
template <int ROWS_, int GRANULE_, bool QMAJOR_, int START_>
struct Line {
  static constexpr int ROWS = ROWS_, GRANULE = GRANULE_, START = START_;
  static constexpr bool QMAJOR = QMAJOR_;

  static __device__ __forceinline__ int len(const FwdCacheParams &p, int b) {
    return min(max(p.lens[b], 0), p.max_pages << p.page_log2);
  }
  // tokens that some row of the tile sees, as granules
  static __device__ __forceinline__ int granules(const FwdCacheParams &p, int len, int tile) {
    int seen = len;
    if (QMAJOR && p.causal) {
      const int last = (int)div_g((tile + 1 < p.tiles ? (tile + 1) * ROWS : p.R) - 1, p.g, p.g_inv);
      seen = max(0, len - p.Nq + last + 1);
    }
    return (seen + GRANULE - 1) / GRANULE;
  }
  // the unit's part of the line
  static __device__ __forceinline__ int span(const FwdCacheParams &p, int len, int tile) {
    const int n = granules(p, len, tile);
    return n ? n + START : 0;
  }
  // the parts of the tiles before `tile` of one head
  static __device__ __forceinline__ int before(const FwdCacheParams &p, int len, int tile) {
    if constexpr (QMAJOR) {
      static_assert(GRANULE == 128 && ROWS % 128 == 0, "parts_before");
      if (p.causal && tile > 0) return parts_before<ROWS / 128, START>(tile, len, p.Nq, p.g, p.g_inv);
    }
    return tile * span(p, len, 0);
  }
  // one head's: all its tiles
  static __device__ __forceinline__ int head(const FwdCacheParams &p, int len) {
    return before(p, len, p.tiles - 1) + span(p, len, p.tiles - 1);
  }
  // The tile whose part holds place `at` of a head's, at < head(len), and the
  // place within it; a warp looks together.
  static __device__ __forceinline__ int tile_at(const FwdCacheParams &p, int len, int &at) {
    int lo = 0;
    if (!QMAJOR || !p.causal) {
      lo = at / span(p, len, 0);
    } else {
      const int lane = threadIdx.x & 31;
      for (int n = p.tiles; n > 1;) {   // in [lo, lo + n)
        const int step = (n + 31) / 32;
        const bool under = lane * step < n && before(p, len, lo + lane * step) <= at;
        const int k = __popc(__ballot_sync(0xffffffffu, under)) - 1;   // lane 0 is: before(lo) <= at
        lo += k * step;
        n = min(step, n - k * step);
      }
    }
    at -= before(p, len, lo);
    return lo;
  }
  // The parts of one head of all sequences, and of those before sequence
  // b; every warp forms them for itself.
  static __device__ __forceinline__ void sums(const FwdCacheParams &p, int b, int *total, int *before) {
    int all = 0, pre = 0;
    for (int i = threadIdx.x & 31; i < p.B; i += 32) {
      const int n = head(p, len(p, i));
      all += n;
      if (i < b) pre += n;
    }
    *total = warp_sum(all);
    *before = b > 0 ? warp_sum(pre) : 0;
  }
  // The sequence that holds granule `pos` of the line cut to one head a
  // sequence (pos < the total), and the granules before it.
  static __device__ __forceinline__ int sequence_at(const FwdCacheParams &p, int pos, int *before) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int i0 = 0;; i0 += 32) {
      const int n = i0 + lane < p.B ? head(p, len(p, i0 + lane)) : 0;
      int inc = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
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
};

// A CTA's run of the line, piece by piece, or its units (p.whole).
template <class L>
struct Run {
  int pos, end;        // granules left: [pos, end); units pos, pos + p.ctas, ... below end
  int b, b_first;      // the sequence of the current piece, the line's granules before it
  // the current piece: granules [g0, g1) of ng of the unit (b, h, tile from
  // row r0 on), tokens [.., stop) of the sequence's len
  int h, r0, g0, g1, ng, len, stop;

  __device__ __forceinline__ bool start(const FwdCacheParams &p) {
    const int lane = threadIdx.x & 31;
    if (p.whole) {
      pos = blockIdx.x;
      end = p.B * p.Hkv * p.tiles;
      return pos < end;
    }
    if (p.B <= 32) {   // one look at the lengths
      const int n = lane < p.B ? L::head(p, L::len(p, lane)) : 0;
      int inc = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
      }
      if (!cut(p, __shfl_sync(0xffffffffu, inc, 31))) return false;
      const unsigned past = __ballot_sync(0xffffffffu, pos < inc * p.Hkv);   // not empty: pos < the total
      b = __ffs(past) - 1;
      b_first = __shfl_sync(0xffffffffu, inc - n, b) * p.Hkv;
      return true;
    }
    int total, unused;
    L::sums(p, 0, &total, &unused);
    if (!cut(p, total)) return false;
    b = L::sequence_at(p, pos / p.Hkv, &b_first);
    b_first *= p.Hkv;
    return true;
  }
  // [pos, end) of a line of `head` granules a head
  __device__ __forceinline__ bool cut(const FwdCacheParams &p, int head) {
    const int total = head * p.Hkv, per = (total + p.ctas - 1) / p.ctas;
    pos = per * (int)blockIdx.x;      // at most total + per
    end = min(total, pos + per);
    return pos < end;
  }
  // O = 0, L = -inf for the rows of the unit.
  template <int D>
  __device__ __forceinline__ void nothing(const FwdCacheParams &p) const {
    const int lane = threadIdx.x & 31, rows = min(L::ROWS, p.R - r0);
    const long long head = ((long long)b * p.Hkv + h) * p.R;
    for (int i = lane; i < rows * (D / 8); i += 32) {
      const int r = r0 + i / (D / 8), c = i % (D / 8);
      const long long row = head + (L::QMAJOR ? r % p.g * p.Nq + r / p.g : r);
      reinterpret_cast<uint4 *>(p.o + row * D)[c] = make_uint4(0u, 0u, 0u, 0u);
      if (c == 0) p.lse[row] = -INFINITY;
    }
    if (lane == 0 && p.lens[b] < 0) atomicOr(p.err, kErrPage);
  }
  // On to the next piece; whole units that see no token are written here, by the
  // warp that `writes`.
  template <int D>
  __device__ __forceinline__ bool next(const FwdCacheParams &p, bool writes) {
    while (p.whole && pos < end) {
      const int bh = pos / p.tiles, tile = pos - bh * p.tiles;
      pos += p.ctas;
      b = bh / p.Hkv;
      h = bh - b * p.Hkv;
      r0 = tile * L::ROWS;
      len = L::len(p, b);
      g0 = 0;
      g1 = ng = L::granules(p, len, tile);
      stop = min(len, ng * L::GRANULE);
      if (ng > 0) return true;
      if (writes) nothing<D>(p);
    }
    while (!p.whole && pos < end) {
      len = L::len(p, b);
      int n = L::head(p, len);
      while (pos - b_first >= n * p.Hkv) {   // on to the next sequence with tokens
        b_first += n * p.Hkv;
        ++b;
        len = L::len(p, b);
        n = L::head(p, len);
      }
      h = (pos - b_first) / n;
      int at = pos - b_first - h * n;   // place within the head, then the unit
      const int tile = L::tile_at(p, len, at), span = L::span(p, len, tile);
      const int to = min(span, at + (end - pos));
      pos += to - at;
      ng = span - L::START;
      g0 = max(0, at - L::START);
      g1 = to - L::START;
      r0 = tile * L::ROWS;
      stop = min(len, g1 * L::GRANULE);
      if (g0 < g1) return true;   // else the run ended before the unit's first granule
    }
    return false;
  }
  // first row of the piece's partial, -1 where the piece is the whole unit: a
  // run has at most one piece that starts inside its unit (slot 0) and one that
  // starts a unit and does not end it (slot 1)
  __device__ __forceinline__ int part(const FwdCacheParams &p) const {
    return g0 == 0 && g1 == ng ? -1 : ((int)blockIdx.x * 2 + (g0 == 0 ? 1 : 0)) * p.prows;
  }
};

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

// Joins the pieces of the units that several CTAs covered: W warps of a CTA of
// kMergeWarps take one query row.  W is kMergeWarps where a unit has many pieces, 1
// where it has few.  Rows of tiles that see no token become O = 0, L = -inf.
constexpr int kMergeWarps = 8;
constexpr int kMergeCtas = 148 * 16;   // of warps a row, at most

// Pieces in flight.  Units of 128 rows and more have two or three pieces, and rows
// enough that more warps matter more: four (512 queries over 16384 tokens, Hq 8,
// Hkv 8, d 128: 67.2 us a call with eight, 66.0 with four; a square causal call of
// 2048 queries, Hq 32: 115.7 and 112.6).
template <class L, int W>
constexpr int merge_ahead() { return W == 1 && L::QMAJOR ? 4 : 8; }

// Row `row` of O and L from its unit's n pieces (n = 0: nothing), row rr of the
// tile, the first of CTA c0; warp w of W.
template <int D, class L, int W>
__device__ __forceinline__ void merge_row(const FwdCacheParams &p, int row, int rr, int c0, int n, int warp, int lane,
                                          float (*s_o)[D], float2 *s_w) {
  // piece i: the unit's start lies in the second slot of CTA c0, the rest in first ones
  auto at = [&](int i) { return ((long long)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * p.prows + rr; };
  constexpr int PER = D / 32, AHEAD = merge_ahead<L, W>();
  const float *src = p.o_part + lane * PER;
  // warp w adds pieces w, w + W, ...: the first loads go out before the weights are known
  float v[AHEAD][PER];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (warp + W * k < n) load_floats<PER>(src + at(warp + W * k) * D, v[k]);
  // lane i looks at pieces i, i + 32, ...
  const float2 none = make_float2(-INFINITY, 0.f), mine = lane < n ? p.l_part[at(lane)] : none;
  float top = mine.x;
  for (int i = lane + 32; i < n; i += 32) top = fmaxf(top, p.l_part[at(i)].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  // a piece's weight 2^{m - top} l as two factors, the power's root and the rest: O of
  // a page of large V may lie past float32's end where the product does not
  auto weight = [&](const float2 &x) {
    const float root = x.y == 0.f ? 0.f : fast_exp2(0.5f * (x.x - top));
    return make_float2(root, x.y == 0.f ? 0.f : root * x.y);
  };
  const float2 own = weight(mine);   // of piece `lane`
  float sum = own.x * own.y;
  if (W > 1 && lane < n && lane % W == warp) s_w[lane] = own;   // each warp keeps its own pieces' weights
  for (int i = lane + 32; i < n; i += 32) {
    const float2 w = weight(p.l_part[at(i)]);
    sum += w.x * w.y;
    if (W > 1 && i % W == warp) s_w[i] = w;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  __syncwarp();
  float acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int i0 = warp; i0 < n; i0 += AHEAD * W) {
    if (i0 != warp) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (i0 + W * k < n) load_floats<PER>(src + at(i0 + W * k) * D, v[k]);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (i0 + W * k < n) {
        const int i = i0 + W * k;
        float2 w;
        if (W > 1) {
          w = s_w[i];
        } else {
          w.x = __shfl_sync(0xffffffffu, own.x, i & 31);
          w.y = __shfl_sync(0xffffffffu, own.y, i & 31);
          if (i >= 32) w = weight(p.l_part[at(i)]);   // more pieces than lanes: the weight again
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(w.y, w.x * v[k][e], acc[e]);
      }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] *= inv;
  __nv_bfloat16 *dst = p.o + (long long)row * D;
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < PER; ++e) s_o[warp][lane * PER + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D / 2) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x += s_o[w][2 * threadIdx.x];
        y += s_o[w][2 * threadIdx.x + 1];
      }
      reinterpret_cast<uint32_t *>(dst)[threadIdx.x] = pack_bf16x2(x, y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < PER; e += 2)
      reinterpret_cast<uint32_t *>(dst)[(lane * PER + e) / 2] = pack_bf16x2(acc[e], acc[e + 1]);
  }
  if (lane == 0 && warp == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

template <int D, class L, int W>
__global__ void __launch_bounds__(kMergeWarps * 32, merge_ahead<L, W>() == 8 ? 1 : D == 256 ? 3 : 4) fwd_cache_merge_kernel(const FwdCacheParams p, int each) {
  __shared__ float s_o[W > 1 ? kMergeWarps : 1][D];
  __shared__ float2 s_w[kMaxCtas];
  __shared__ int s_unit[5];
  const int warp = W > 1 ? threadIdx.x >> 5 : 0, lane = threadIdx.x & 31;
  const int rows = p.B * p.Hq * p.Nq;   // < 2^31: the launcher checks
  const long long cta0 = (long long)blockIdx.x * (W > 1 ? 1 : kMergeWarps * each);   // the CTA's first row
  const int row0 = (int)min((long long)rows, cta0 + (W > 1 ? 0 : (int)(threadIdx.x >> 5) * each));
  const int row1 = min(rows - row0, each) + row0;
  int b = 0, h = 0, tile = 0, rr = 0;   // of a row: its unit, the row of the tile
  int unit_b = -1, unit_h = 0, unit_tile = 0, c0 = 0, n = 0;   // a unit, its first CTA and pieces
  auto place = [&](int row) {
    b = row / (p.Hq * p.Nq);
    const int hr = row - b * p.Hq * p.Nq;   // row within the sequence
    h = hr / p.R;
    int r = hr - h * p.R;   // row of the head, in the order of memory
    if constexpr (L::QMAJOR) {
      const int head = r / p.Nq;
      r = (r - head * p.Nq) * p.g + head;
    }
    tile = r / L::ROWS;
    rr = r - tile * L::ROWS;
  };
  auto look = [&]() {
    unit_b = b; unit_h = h; unit_tile = tile;
    const int len = L::len(p, b), ng = L::granules(p, len, tile);
    int total, first;
    L::sums(p, b, &total, &first);
    const int per = max((total * p.Hkv + p.ctas - 1) / p.ctas, 1);
    // the unit's first granule
    first = first * p.Hkv + h * L::head(p, len) + L::before(p, len, tile) + L::START;
    c0 = first / per;
    n = ng == 0 ? 0 : (first + ng - 1) / per - c0 + 1;
  };
  // With tiles of 128 rows and more most rows of the CTA are of one unit: one warp
  // looks for it (512 queries over 16384 tokens, Hq 8, Hkv 8, d 128: 66.2 -> 63.8 us a
  // call; with 16 rows a tile it costs 1 us, for the CTA's other units).
  constexpr bool SHARE = L::QMAJOR && W == 1;
  if (SHARE ? threadIdx.x < 32 : row0 < row1) {
    place(SHARE ? (int)cta0 : row0);
    look();
    if (SHARE && lane == 0) {
      s_unit[0] = unit_b; s_unit[1] = unit_h; s_unit[2] = unit_tile; s_unit[3] = c0; s_unit[4] = n;
    }
  }
  // every CTA waits, so that what follows in the stream finds o and lse whole
  wait_for_primary();
  if (SHARE) {
    __syncthreads();
    unit_b = s_unit[0]; unit_h = s_unit[1]; unit_tile = s_unit[2]; c0 = s_unit[3]; n = s_unit[4];
  }
#pragma unroll 1
  for (int row = row0; row < row1; ++row) {
    if (SHARE || row > row0) place(row);
    if (b != unit_b || h != unit_h || tile != unit_tile) look();
    if (n == 1) continue;
    merge_row<D, L, W>(p, row, rr, c0, n, warp, lane, s_o, s_w);
    if (lane == 0 && warp == 0 && p.lens[b] < 0) atomicOr(p.err, kErrPage);
  }
}

// The same where units are more than twice the CTAs, most of them whole: CTA (x, c) takes eight rows
// of the one unit that begins in run c and does not end there.  Units that see no
// token are looked for only if a sequence has one.  Measured, a call by rows / by
// CTAs, causal, Hq 32, Hkv 8, d 128: B 1, 2048 queries (256 units) 110 / 117 us; B 8, 512
// of 1024 tokens (512 units) 178 / 164; B 32, 512 of 512 (2048 units) 398 / 305.
template <int D, class L>
__global__ void __launch_bounds__(kMergeWarps * 32, D == 256 ? 3 : 4) fwd_cache_merge_split_kernel(const FwdCacheParams p) {
  __shared__ int s_unit[5];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.y;
  if (warp == 0) {
    bool empty = false;   // a tile of some sequence sees no token
    for (int i = lane; i < p.B; i += 32) empty |= L::granules(p, L::len(p, i), 0) == 0;
    empty = __any_sync(0xffffffffu, empty);
    int total, unused, b = 0, h = 0, tile = 0, n = 0;
    L::sums(p, 0, &total, &unused);
    total *= p.Hkv;
    const int per = max((total + p.ctas - 1) / p.ctas, 1), end = min(total, per * (c + 1));
    if (per * c < end) {
      const int pos = end - 1;   // the unit that the run ends in
      int before;
      b = L::sequence_at(p, pos / p.Hkv, &before);
      const int len = L::len(p, b), head = L::head(p, len);
      h = (pos - before * p.Hkv) / head;
      int at = pos - before * p.Hkv - h * head;
      tile = L::tile_at(p, len, at);
      const int first = pos - at + L::START, last = pos - at + L::span(p, len, tile) - 1;   // its granules
      n = first / per == c ? last / per - c + 1 : 1;
    }
    if (lane == 0) {
      s_unit[0] = b * p.Hkv + h; s_unit[1] = tile; s_unit[2] = n; s_unit[3] = empty;
    }
  }
  // every CTA waits, so that what follows in the stream finds o and lse whole
  wait_for_primary();
  __syncthreads();
  const int bh = s_unit[0], rr = blockIdx.x * kMergeWarps + warp, r = s_unit[1] * L::ROWS + rr, n = s_unit[2];
  if (n > 1 && rr < L::ROWS && r < p.R)
    merge_row<D, L, 1>(p, bh * p.R + r % p.g * p.Nq + r / p.g, rr, c, n, 0, lane, nullptr, nullptr);
  if (!s_unit[3]) return;
  const long long warps = (long long)gridDim.x * gridDim.y * kMergeWarps, rows = (long long)p.B * p.Hq * p.Nq;
  for (long long row = ((long long)c * gridDim.x + blockIdx.x) * kMergeWarps + warp; row < rows; row += warps) {
    const int b = (int)(row / (p.Hq * p.Nq)), q = (int)(row % (p.Hq * p.Nq)), i = q % p.Nq, head = q / p.Nq % p.g;
    if (L::granules(p, L::len(p, b), (int)(((long long)i * p.g + head) / L::ROWS))) continue;
    for (int x = lane; x < D / 8; x += 32) reinterpret_cast<uint4 *>(p.o + row * D)[x] = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) {
      p.lse[row] = -INFINITY;
      if (p.lens[b] < 0) atomicOr(p.err, kErrPage);
    }
  }
}

// Launches the merge while the main kernel runs: its CTAs find their pieces,
// then wait for the main kernel's end.
template <int D, class L>
int launch_fwd_cache_merge(const FwdCacheParams &p, cudaStream_t stream) {
  if (p.whole) return 0;
  const long long rows = (long long)p.B * p.Hq * p.Nq, units = (long long)p.B * p.Hkv * p.tiles;
  // A warp a row: about eight pieces a unit, or fewer, or more rows than CTAs that
  // run at once.  Measured, a call: Hq 16, Hkv 4, d 256, B 8, 2304 tokens, 4 queries
  // (512 rows, 9 pieces) 20.2 us with a warp a row, 26.3 with eight; Hq 32, Hkv 8, d
  // 128, B 4, 16384 tokens (128 rows, 9 pieces) 32.7 and 31.3.
  const bool many = units * 8 >= p.ctas || rows > 2 * 148;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // a warp takes neighbouring rows, which share their unit, rather than that more CTAs start
  const long long each = many ? (rows + kMergeCtas * kMergeWarps - 1) / (kMergeCtas * kMergeWarps) : 1;
  const long long warps = (rows + each - 1) / each;
  cfg.gridDim = dim3((unsigned)(many ? (warps + kMergeWarps - 1) / kMergeWarps : rows), 1, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (L::QMAJOR) {
    if (units > 2 * p.ctas) {
      cfg.gridDim = dim3((unsigned)((p.prows + kMergeWarps - 1) / kMergeWarps), (unsigned)p.ctas, 1);
      return cudaLaunchKernelEx(&cfg, fwd_cache_merge_split_kernel<D, L>, p) == cudaSuccess &&
             cudaGetLastError() == cudaSuccess ? 0 : 5;
    }
  }
  if ((many ? cudaLaunchKernelEx(&cfg, fwd_cache_merge_kernel<D, L, 1>, p, (int)each)
            : cudaLaunchKernelEx(&cfg, fwd_cache_merge_kernel<D, L, kMergeWarps>, p, 1)) != cudaSuccess)
    return 5;
  return cudaGetLastError() == cudaSuccess ? 0 : 5;
}

// What the host knows of the work of a line: CTAs (fewer than `most_ctas` when
// the block table has room for fewer granules), rows of a partial; whether the table
// has room for so few tokens that CTAs take whole units: `whole`, or `whole_many` where
// every CTA has a unit without a cut.
struct FwdCachePlan {
  double R, most;   // most: the line's length when every sequence fills its table
  long long tiles;
  int prows, ctas;
  bool whole;
};
template <class L>
FwdCachePlan fwd_cache_plan(const CacheArgs &a, int most_ctas, int whole, int whole_many) {
  FwdCachePlan x;
  x.R = (double)(a.Hq / a.Hkv) * a.Nq;
  x.prows = x.R < L::ROWS ? (int)x.R : L::ROWS;
  x.tiles = (long long)((x.R + L::ROWS - 1) / L::ROWS);
  x.most = (double)a.B * a.Hkv * x.tiles *
           (((long long)a.max_pages * a.page + L::GRANULE - 1) / L::GRANULE + L::START);
  const double units = (double)a.B * a.Hkv * x.tiles;
  x.whole = (long long)a.max_pages * a.page <= (units < most_ctas ? whole : whole_many);
  const double parts = x.whole ? units : x.most;
  x.ctas = parts < most_ctas ? (int)parts : most_ctas;
  return x;
}
// The kernel for many query rows (fa_fwd_cache_sm100.cu).
FwdCachePlan fwd_cache_tile_plan(const CacheArgs &a);
int launch_fwd_cache_tiles(const CacheArgs &a, const FwdCachePlan &x);

inline size_t fwd_cache_plan_bytes(const FwdCachePlan &x, int d) {
  return x.whole ? 0 : (size_t)x.ctas * 2 * x.prows * (d + 2) * 4;
}
inline FwdCacheParams fwd_cache_params(const CacheArgs &a, const FwdCachePlan &x) {
  FwdCacheParams p;
  p.q = (const __nv_bfloat16 *)a.q;
  p.k_cache = a.k_cache; p.v_cache = a.v_cache;
  p.k_scale = a.k_scale; p.v_scale = a.v_scale;
  p.table = a.table; p.lens = a.lens;
  p.o = (__nv_bfloat16 *)a.o; p.lse = a.lse;
  p.o_part = (float *)a.ws;
  p.l_part = (float2 *)(p.o_part + (size_t)x.ctas * 2 * x.prows * a.d);
  p.B = a.B; p.Hq = a.Hq; p.Hkv = a.Hkv; p.Nq = a.Nq; p.g = a.Hq / a.Hkv;
  p.g_inv = p.g == 1 ? 0 : ~0ull / p.g + 1;
  p.R = (int)x.R;
  p.tiles = (int)x.tiles;
  p.page_log2 = a.page == 16 ? 4 : a.page == 32 ? 5 : a.page == 64 ? 6 : 7;
  p.num_pages = a.num_pages; p.max_pages = a.max_pages;
  p.causal = a.causal; p.ctas = x.ctas; p.prows = x.prows; p.whole = x.whole;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.err = a.err;
  return p;
}

}  // namespace fa
