// fa_fwd_cache_sm100.cu -- attention over the paged E4M3 cache for many query
// rows (chunks of a prompt, drafted tokens of grouped heads): tiles of 128 rows
// on tcgen05, TMEM accumulators.
//
// The mathematics are those of fa_fwd_cache.cu, with the same two references
// (m for the sum of 2^{s - m}, M, kept as M - m, for the weights 2^{s - m} sv) and the
// same roundings: q and the weights as halves, the codes exactly as halves.
//
// A CTA (one per SM, 16 warps) takes NT tiles of 128 rows of one key/value
// head, row r being query r / g of the group's head r % g, and blocks of 128
// tokens of its run of the line:
//   warps 0 .. 4 NT - 1  softmax and epilogue, a thread per row (TMEM lane);
//                        they convert their rows of q first
//   the others but one   converters: they read the pages' codes into registers a
//                        block ahead, and write halves into 128-byte-swizzled
//                        shared memory when the block before has left it; tokens
//                        that do not exist become zeros
//   warp 15              issues the MMAs (lane 0)
// S_t = Q_t K^T lands in TMEM; the softmax thread reads its row, which frees S
// for the next block's product, and writes the weights to shared memory; O_t +=
// P_t V accumulates in TMEM.  All MMAs are kind::f16 with halves: M 128, N 128
// (N d for O).  E4M3 operands would halve the product's cost but hold a weight
// to 4 bits (8 in two parts, which cost as much as halves), down to 2^-18 of
// the largest only.
//
// Measured on B200, a call: 512 queries over 16384 tokens, causal, Hq 8, Hkv 8, d 128,
// 63 us = 537 TFLOP/s; 8192 square, Hq 32, 717 us = 767 TFLOP/s causal, 1233 us = 892
// TFLOP/s not; d = 256, Hq 16, Hkv 4, 4096 square causal, one tile a CTA, 246 us = 559.
// A block of 128 tokens took about 5000 cycles for two tiles (clock stamps, calls then
// 3 % slower), of which the tensor pipe's work is 2050 and the exponentials' 2050: the
// softmax's 4600 set the pace, 72 % of the issue slots with the converters'
// instructions, and neither removing the maxima, the exponentials or the conversion
// alone (timing copies) shortened a call by more than 2 us.  The blocks are 35 us of the
// first call; the rest is its start (9700 cycles to the first S), the partials' stores
// (6000), the merge and the launches.  Tried and slower: the weights in TMEM instead of
// shared memory, S of a block behind P V of the one before (68 us where this form
// took 65), S read 32 columns at a time ahead of use (68), converters that sleep
// between polls (67); pairs of float32 in one instruction changed nothing (65).
#include "fwd_cache.cuh"

namespace fa {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int kMmaWarp = 15;
constexpr int kThreads = 512;
// CTAs take whole units where the block table has room for this many tokens.
// Measured, us a call in a graph with the line and with whole units, causal, d 128, Hkv
// 8: B 1, Hq 8, 128 queries of 128 tokens 15.3 / 10.5, 512 of 512 22.7 / 22.2, 64 of 512
// 15.1 / 16.3; B 1, Hq 32, 512 of 512 37.3 / 21.4; B 8, Hq 32, 128 of 128 31.6 / 14.5,
// 512 of 512 107 / 64.6.  With a unit for every CTA, B 8, 512 of 2048 232 / 188 (ragged
// 204 / 170), 512 of 4096 367 / 352 (ragged 266 / 314); B 19, 64 queries, four units more
// than CTAs, 1024 tokens 71.6 / 59.3, 2048 tokens 98.0 / 101.1.
constexpr int kWhole = 512, kWholeMany = 2048;
constexpr float kBig = 1048576.f;               // past it, s - m in one rounding is off by 2^-4 and more
constexpr float kTiny = 1.17549435e-38f;        // least factor of a score: a hidden -inf stays one

template <int D_, int NT_>
struct TileCfg {
  static constexpr int D = D_, NT = NT_;
  // A unit's start counts as five granules.  Measured, us a call in a graph with
  // 0 / 2 / 3 / 5: 512 queries over 16384 tokens, causal, Hq 8, Hkv 8, d 128:
  // 71.4 / 66.6 / 65.7 / 65.2.
  using L = Line<NT * BM, BN, true, 5>;
  static constexpr int SOFT = 4 * NT;                 // softmax warps
  static constexpr int CONV = kMmaWarp - SOFT;        // converter warps
  static constexpr int CT = CONV * 32;
  static constexpr int CHUNK = BN * 128;              // 128 rows of 64 halves
  static constexpr int DCH = D / 64;
  static constexpr int TILE = CHUNK * DCH;            // Q, K or V as halves
  static constexpr int P_TILE = CHUNK * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + NT * TILE;
  static constexpr int OFF_K = OFF_P + NT * P_TILE;
  static constexpr int OFF_V = OFF_K + TILE;
  static constexpr int OFF_SCALE = OFF_V + TILE;             // [4][8] (sk, log2 sv) of a block's 16-token groups
  static constexpr int OFF_PAGES = OFF_SCALE + 4 * 8 * 8;    // [4] Pages of a block
  static constexpr int OFF_NAN = OFF_PAGES + 4 * 8;          // [2][D] first NaN token of a column
  static constexpr int OFF_ANY = OFF_NAN + 2 * D * 4;        // [2] whether there is one
  static constexpr int OFF_PIECE = OFF_ANY + 8;              // [2] Piece
  static constexpr int OFF_BAR = OFF_PIECE + 2 * 32;
  static constexpr int NBAR = 10 + 6 * NT;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;        // TMEM base, abort flag
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr int TM_S = 0, TM_O = NT * BN;
  static_assert(NT * (BN + D) <= 512, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

// The other roles' copy of the converters' piece; no blocks: the run is over.
struct Piece {
  int b, h, r0, blocks, token, len, part, unused;
};
static_assert(sizeof(Piece) == 32, "Piece");

// What the converters say of a block's pages: whether some group has none; the
// largest log2 sv of the block, where the piece's so far differ by so much that a
// weight's factor may pass 2^kOver (up is at most kShift + their difference), else -inf.
struct Pages {
  int hole;
  float top;
};
static_assert(sizeof(Pages) == 8, "Pages");

// D[tmem] (+)= A B with halves: the format fields 0.
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}

// 16 E4M3 codes -> 16 halves, in the 16-byte units at `at` and `at ^ 16`.
__device__ __forceinline__ void store_halves(uint32_t at, const uint4 &codes) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = e4m3x2_to_half2(w[i] & 0xFFFFu);
    h[2 * i + 1] = e4m3x2_to_half2(w[i] >> 16);
  }
  st_shared_v4(at, h[0], h[1], h[2], h[3]);
  st_shared_v4(at ^ 16, h[4], h[5], h[6], h[7]);
}

// The largest of each N neighbouring lanes' values.
template <int N>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = N / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// The running maximum m of a row's scores and the largest s - m + log2 sv of a block,
// for scores so large that one rounding of s - m is off by whole units: s is rounded
// once, by which equal scores stay equal, and the differences are exact.  The best of
// s + log2 sv is kept as its two parts.
__device__ __noinline__ float2 maxima_apart(uint32_t ts, const float2 *scs, float rc, float m, int lim) {
  float best_s = -INFINITY, best_v = 0.f;
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    const float2 kv = scs[q];
    const int seen = kv.y == -INFINITY ? 0 : lim - 16 * q;
    uint32_t sq[16];
    tmem_ld16(ts + 16 * q, sq);
    tmem_wait_ld();
    float mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, e < seen ? __uint_as_float(sq[e]) : -INFINITY);
    mx = __fmul_rn(mx, fmaxf(rc * kv.x, kTiny));
    m = fmaxf(m, mx);
    if (mx - best_s + (kv.y - best_v) > 0.f) {
      best_s = mx;
      best_v = kv.y;
    }
  }
  return make_float2(m, best_s - m + best_v);
}

// The weights of a block's 128 columns where they are not formed as products, and the
// sum of the row's powers: 16 columns at a time.  Both are calls, apart from the
// kernel's code, whose loops the rare path would lengthen (8192 square, Hq 32, Hkv 8, d
// 128, causal: 748 us with them inline, 723 as calls).
template <int CHUNK>
__device__ __noinline__ float weigh_apart(uint32_t ts, uint32_t prow, const float2 *scs, float rc, float ms, float diff,
                                          int lim, int r) {
  float sum = 0.f;
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    const float2 kv = scs[q];
    const float cf = fmaxf(rc * kv.x, kTiny), up = diff + kv.y;
    const int seen = kv.y == -INFINITY ? 0 : lim - 16 * q;
    uint32_t sq[16], pk[8];
    tmem_ld16(ts + 16 * q, sq);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      // s rounded before m is subtracted: the largest gives 0, equal ones the same
      const float x0 = e < seen ? __fmul_rn(__uint_as_float(sq[e]), cf) - ms : -INFINITY;
      const float x1 = e + 1 < seen ? __fmul_rn(__uint_as_float(sq[e + 1]), cf) - ms : -INFINITY;
      sum += fast_exp2(x0) + fast_exp2(x1);
      pk[e / 2] = pack_half2(fast_exp2(x0 + up), fast_exp2(x1 + up));
    }
    const uint32_t at = prow + (q >> 2) * CHUNK + (((2 * (q & 3)) ^ (r & 7)) << 4);
    st_shared_v4(at, pk[0], pk[1], pk[2], pk[3]);
    st_shared_v4(at ^ 16, pk[4], pk[5], pk[6], pk[7]);
  }
  return sum;
}

// 32 bytes, a whole sector, in one store.
__device__ __forceinline__ void store8(void *dst, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1) fwd_cache_tile_kernel(const FwdCacheParams p) {
  constexpr int D = C::D, NT = C::NT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrConfig);
    return;
  }
  launch_dependents();   // the merge kernel's CTAs may take their places
  auto bar = [&](int i) { return sbase + C::OFF_BAR + i * 8; };
  constexpr int B_UFULL = 0, B_UEMPTY = 2, B_QFULL = 4, B_KFULL = 5, B_KEMPTY = 6, B_VFULL = 7,
                B_VEMPTY = 8, B_DRAIN = 9, B_SFULL = 10, B_SEMPTY = 10 + NT, B_PFULL = 10 + 2 * NT,
                B_PEMPTY = 10 + 3 * NT, B_OFULL = 10 + 4 * NT, B_OEMPTY = 10 + 5 * NT;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
  float2 *scales = reinterpret_cast<float2 *>(smem + C::OFF_SCALE);
  Pages *block_pages = reinterpret_cast<Pages *>(smem + C::OFF_PAGES);
  // Two lists of NaN codes, for pieces in turn.  A piece's converters clear the
  // next piece's list before they hand over their last V.
  int *nan_at = reinterpret_cast<int *>(smem + C::OFF_NAN), *nan_any = reinterpret_cast<int *>(smem + C::OFF_ANY);
  Piece *pieces = reinterpret_cast<Piece *>(smem + C::OFF_PIECE);
  const int warp = warp_id_uniform(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_UFULL + i), 1);
      mbar_init(bar(B_UEMPTY + i), NT * BM + 1);   // softmax threads, the MMA issuer
    }
    mbar_init(bar(B_QFULL), NT * BM);
    mbar_init(bar(B_KFULL), C::CT);
    mbar_init(bar(B_KEMPTY), 1);
    mbar_init(bar(B_VFULL), C::CT);
    mbar_init(bar(B_VEMPTY), 1);
    mbar_init(bar(B_DRAIN), 1);
    for (int t = 0; t < NT; ++t) {
      mbar_init(bar(B_SFULL + t), 1);
      mbar_init(bar(B_SEMPTY + t), BM);
      mbar_init(bar(B_PFULL + t), BM);
      mbar_init(bar(B_PEMPTY + t), 1);
      mbar_init(bar(B_OFULL + t), 1);
      mbar_init(bar(B_OEMPTY + t), BM);
    }
    *abort_flag = 0;
    nan_any[0] = nan_any[1] = 0;
    fence_barrier_init();
  }
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) nan_at[i] = 0x7FFFFFFF;
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{p.err, abort_flag, kWaitLimitNs};

  // Blocks of the run are counted by g, pieces by u: barrier phases.
  if (warp >= C::SOFT && warp < kMmaWarp) {
    // ---------------------------------------------------------- converters
    const int ct = threadIdx.x - C::SOFT * 32;    // 0 .. CT - 1
    const bool leader = ct == 0;
    // Four lanes take 64 columns of a token, a warp eight tokens at a time: "row"
    // i * CT / 4 + ct / 4 of the DCH * 128 rows of 64 halves that a tile has.
    // Its place mod 8, and so the swizzle, is the thread's own; eight lanes store
    // to eight bank groups.
    constexpr int RPI = C::CT / 4, ROWS = BN * C::DCH;
    constexpr int NL = (ROWS + RPI - 1) / RPI;    // chunks of 16 codes of a thread
    static_assert(RPI % 8 == 0, "the swizzle is the thread's own");
    const int ct4 = ct >> 2;
    const uint32_t my_dst = sbase + ct4 * 128 + ((((ct & 3) * 2) ^ (ct4 & 7)) << 4);
    const uint32_t my_src = (ct & 3) * 16;
    bool ok = true;
    int g = 0, u = 0;
    Run<typename C::L> run;
    bool more = run.start(p);
    for (; ok; ++u) {
      if (more) more = run.template next<D>(p, warp == C::SOFT);
      const int n = more ? run.g1 - run.g0 : 0;
      if (leader) {
        ok = bounded_wait(bar(B_UEMPTY + (u & 1)), ((u >> 1) & 1) ^ 1, wc);
        if (ok) {
          Piece x;
          x.b = run.b; x.h = run.h; x.r0 = run.r0; x.blocks = n;
          x.token = run.g0 * BN; x.len = run.len;
          x.part = more ? run.part(p) : -1;
          x.unused = 0;
          pieces[u & 1] = x;
          mbar_arrive(bar(B_UFULL + (u & 1)));
          if (more) (void)checked_len(p.lens, run.b, p.max_pages, 1 << p.page_log2, p.err);
        }
      }
      if (warp == C::SOFT) ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      if (!more || !ok) break;
      const int *tab = p.table + (long long)run.b * p.max_pages;
      // of a block's 16-token group `lane` (lanes 0 .. 7): the cache row of its
      // first token (rows of d codes), kNone: no page
      // (Page numbers are fetched a block before they are looked at, scales a
      // block before they are used, so that no load is waited for.)
      constexpr uint32_t kNone = 0xFFFFFFFFu;
      auto token_of = [&](int j) { return lane >= 8 || j >= n ? run.len : (run.g0 + j) * BN + lane * 16; };
      auto fetch = [&](int j) {
        const int tok = token_of(j);
        return tok >= run.len ? 0 : tab[tok >> p.page_log2];
      };
      auto row_of = [&](int pg, int j) {
        const int tok = token_of(j);
        if (tok >= run.len) return kNone;
        if ((unsigned)pg < (unsigned)p.num_pages)
          return (((uint32_t)pg * p.Hkv + run.h) << p.page_log2) + (tok & ((1 << p.page_log2) - 1));
        atomicOr(p.err, kErrPage);
        return kNone;
      };
      // this thread's chunks of K or V of block j, whose groups lie at `rows`
      auto load = [&](const uint8_t *cache, int j, uint32_t rows, uint4 (&x)[NL]) {
        const int left = run.len - (run.g0 + j) * BN;   // tokens there are
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int row = i * RPI + ct4, r = row & (BN - 1);
          const uint32_t at = __shfl_sync(0xffffffffu, rows, r >> 4);
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row < ROWS && at != kNone && r < left)
            x[i] = *reinterpret_cast<const uint4 *>(cache + (size_t)(at + (r & 15)) * D + (row / BN) * 64 + my_src);
        }
      };
      auto store = [&](int tile, const uint4 (&x)[NL]) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if (i * RPI + ct4 < ROWS) store_halves(my_dst + tile + i * RPI * 128, x[i]);
      };
      // (sk, sv) of a group; without a page (1, 0), whose log2 sv hides it
      auto scale_of = [&](uint32_t row) {
        if (row == kNone) return make_float2(1.f, 0.f);
        const uint32_t i = row >> p.page_log2;
        return make_float2(p.k_scale[i], p.v_scale[i]);
      };
      // ---- the first blocks' codes are on their way while q is converted
      uint32_t row0, row1;   // of blocks j and j + 1
      int pg2;               // of block j + 2
      {
        const int a0 = fetch(0), a1 = fetch(1);
        pg2 = fetch(2);
        row0 = row_of(a0, 0);
        row1 = row_of(a1, 1);
      }
      uint4 kr[NL], vr[NL];
      load(p.k_cache, 0, row0, kr);
      load(p.v_cache, 0, row0, vr);
      float2 sc = scale_of(row0);
      float lo = INFINITY, hi = -INFINITY;   // log2 sv of the piece's pages so far

      // tokens that every row of the piece sees
      const int lim_min = p.causal ? max(0, min(run.len, run.len - p.Nq + run.r0 / p.g + 1)) : run.len;

      for (int j = 0; j <= n && ok; ++j) {
        // K runs a block ahead of V
        if (j < n) {
          ok = warp_wait_all(bar(B_KEMPTY), ((g + j) & 1) ^ 1, wc);
          if (!ok) break;
          if (warp == C::SOFT) {
            const float lsv = log2f(sc.y);
            if (lane < 8) scales[((g + j) & 3) * 8 + lane] = make_float2(sc.x, lsv);
            const unsigned there = __ballot_sync(0xffffffffu, lsv != -INFINITY);   // lanes 8 and up: none
            const float top = group_max<8>(lsv);
            hi = fmaxf(hi, top);
            lo = fminf(lo, -group_max<8>(lsv != -INFINITY ? -lsv : -INFINITY));
            if (leader)
              block_pages[(g + j) & 3] = Pages{(there & 0xFFu) != 0xFFu, hi - lo > kOver - kShift ? top : -INFINITY};
          }
          store(C::OFF_K, kr);
          fence_proxy_async_smem();
          mbar_arrive(bar(B_KFULL));
          if (j + 1 < n) {
            load(p.k_cache, j + 1, row1, kr);
            sc = scale_of(row1);
          }
        }
        if (j > 0) {   // V of block j - 1
          const int jv = j - 1;
          ok = warp_wait_all(bar(B_VEMPTY), ((g + jv) & 1) ^ 1, wc);
          if (!ok) break;
          if (j == n) {
            // the epilogue of the piece before has read its list: clear it for
            // the next piece, whose V waits for this one's
            for (int t = 0; t < NT && ok && u > 0; ++t) ok = warp_wait_all(bar(B_OEMPTY + t), (u - 1) & 1, wc);
            if (!ok) break;
            for (int i = ct; i < D; i += C::CT) nan_at[((u + 1) & 1) * D + i] = 0x7FFFFFFF;
            if (leader) nan_any[(u + 1) & 1] = 0;
          }
          store(C::OFF_V, vr);
          // A token that some row does not see may hold a NaN code, and 0 * NaN
          // is NaN: such codes become 0, and the epilogue makes their columns of
          // the rows that see the first of them NaN.
          if ((run.g0 + jv + 1) * BN > lim_min) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < NL; ++i)
              any |= (__vcmpeq4(vr[i].x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(vr[i].y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                      __vcmpeq4(vr[i].z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(vr[i].w & 0x7F7F7F7Fu, 0x7F7F7F7Fu)) != 0;
            if (any) {
#pragma unroll 1
              for (int row = ct4; row < ROWS; row += RPI) {
                uint8_t *at = smem + C::OFF_V + (my_dst - sbase) + (row - ct4) * 128;
#pragma unroll 1
                for (int e = 0; e < 16; ++e) {
                  unsigned short *h = reinterpret_cast<unsigned short *>(
                      e < 8 ? at : smem + ((uint32_t)(at - smem) ^ 16u)) + (e & 7);
                  if ((*h & 0x7FFFu) <= 0x7C00u) continue;
                  *h = 0;
                  atomicMin(nan_at + (u & 1) * D + row / BN * 64 + my_src + e, (run.g0 + jv) * BN + (row & (BN - 1)));
                  nan_any[u & 1] = 1;
                }
              }
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(B_VFULL));
          if (j < n) load(p.v_cache, j, row0, vr);
        }
        row0 = row1;
        row1 = row_of(pg2, j + 2);
        pg2 = fetch(j + 3);
      }
      g += n;
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t IDESC_S = idesc_f16(BM, BN, 0), IDESC_PV = idesc_f16(BM, D, 1);
    const uint64_t dq0 = sw128_desc(sbase + C::OFF_Q, 16, 1024), dk0 = sw128_desc(sbase + C::OFF_K, 16, 1024);
    const uint64_t dv0 = sw128_desc(sbase + C::OFF_V, C::CHUNK, 1024), dp0 = sw128_desc(sbase + C::OFF_P, 16, 1024);
    auto issue_s = [&](int t) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * C::CHUNK + (k & 3) * 32;
        mma_ss(tmem + C::TM_S + t * BN, desc_add(dq0, t * C::TILE + off), desc_add(dk0, off), IDESC_S, k > 0);
      }
    };
    auto issue_pv = [&](int t, bool first) {
#pragma unroll
      for (int k = 0; k < BN / 16; ++k)
        mma_ss(tmem + C::TM_O + t * D, desc_add(dp0, t * C::P_TILE + (k >> 2) * C::CHUNK + (k & 3) * 32),
               desc_add(dv0, k * 16 * 128), IDESC_PV, !first || k > 0);
    };
    if (lane == 0) {
      bool ok = true;
      int g = 0;
      for (int u = 0; ok; ++u) {
        ok = bounded_wait(bar(B_UFULL + (u & 1)), (u >> 1) & 1, wc);
        if (!ok) break;
        const int n = pieces[u & 1].blocks;
        if (n == 0) break;
        ok = bounded_wait(bar(B_QFULL), u & 1, wc) && bounded_wait(bar(B_KFULL), g & 1, wc);
        // S of block 0 reuses columns that the softmax read in the piece before
        for (int t = 0; t < NT && ok; ++t) {
          if (g > 0) ok = bounded_wait(bar(B_SEMPTY + t), (g - 1) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          issue_s(t);
          mma_commit(bar(B_SFULL + t));
        }
        if (!ok) break;
        mma_commit(bar(B_KEMPTY));
        for (int j = 0; j < n && ok; ++j) {
          const int gj = g + j;
          if (j + 1 < n) {
            ok = bounded_wait(bar(B_KFULL), (gj + 1) & 1, wc);
            for (int t = 0; t < NT && ok; ++t) {
              ok = bounded_wait(bar(B_SEMPTY + t), gj & 1, wc);
              if (!ok) break;
              tc_fence_after();
              issue_s(t);
              mma_commit(bar(B_SFULL + t));
            }
            if (!ok) break;
            mma_commit(bar(B_KEMPTY));
          }
          ok = bounded_wait(bar(B_VFULL), gj & 1, wc);
          for (int t = 0; t < NT && ok; ++t) {
            ok = bounded_wait(bar(B_PFULL + t), gj & 1, wc);
            if (ok && j == 0 && u > 0) ok = bounded_wait(bar(B_OEMPTY + t), (u - 1) & 1, wc);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, j == 0);
            mma_commit(bar(B_PEMPTY + t));
            if (j + 1 == n) mma_commit(bar(B_OFULL + t));
          }
          if (ok) mma_commit(bar(B_VEMPTY));
        }
        g += n;
        mbar_arrive(bar(B_UEMPTY + (u & 1)));
      }
      if (!ok) {
        mma_commit(bar(B_DRAIN));   // every MMA issued so far must end before TMEM is freed
        (void)drain_wait(bar(B_DRAIN), 0, p.err, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------- softmax, epilogue
    const int t = warp >> 2, r = threadIdx.x & 127;   // tile, row = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::TM_S + t * BN, to = tmem + lane_off + C::TM_O + t * D;
    const uint32_t prow = sbase + C::OFF_P + t * C::P_TILE + r * 128;
    bool ok = true;
    int g = 0;
    for (int u = 0; ok; ++u) {
      ok = warp_wait_all(bar(B_UFULL + (u & 1)), (u >> 1) & 1, wc);
      if (!ok) break;
      const Piece x = pieces[u & 1];
      if (x.blocks == 0) break;
      const int rr = x.r0 + t * BM + r;              // row of the head
      const bool live = rr < p.R;
      const int i = (live ? rr : 0) / p.g, hq = x.h * p.g + (live ? rr : 0) - i * p.g;
      // tokens [0, lim) visible; the warp's least, for whole blocks
      const int lim = !live ? x.len : (p.causal ? max(0, min(x.len, x.len - p.Nq + i + 1)) : x.len);
      const int lim_warp = __reduce_min_sync(0xffffffffu, lim);
      const long long row = ((long long)x.b * p.Hq + hq) * p.Nq + i;   // of q, o, lse
      float m_s = -INFINITY, m_d = -INFINITY, l = 0.f;   // m, M - m, sum of 2^{s - m}
      bool big = false;   // some row's m is past kBig

      // ---- q: the warp converts its 32 rows (D / 8 lanes a row), each times a
      // power of two that brings its largest entry to [2^13, 2^14).  The tile is
      // free: this warp has seen the last S of the piece before.
      float rc = 0.f;   // this row's scale * log2 e / that power of two
      {
        constexpr int LPR = D / 8, RPW = 32 / LPR, AHEAD = 8;   // lanes of a row, rows at a time, loads in flight
        const int sub = lane / LPR, col = lane % LPR;
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += RPW * AHEAD) {
          uint4 raw[AHEAD];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            // the row's place in memory lies with the thread whose row it is
            const int lr = r0 + k * RPW + sub;
            const long long at = __shfl_sync(0xffffffffu, live ? row : -1, lr & 31);
            raw[k] = make_uint4(0u, 0u, 0u, 0u);
            if (lr < 32 && at >= 0) raw[k] = *reinterpret_cast<const uint4 *>(p.q + at * D + col * 8);
          }
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            const int lr = r0 + k * RPW + sub, tr = (warp & 3) * 32 + lr;   // row of the warp, of the tile
            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
            float mx = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 126);
            const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
            const float down = p.scale_log2 * __uint_as_float((uint32_t)(e - 13 + 127) << 23);
            // lane of row r0 + k * RPW + i takes group i's factor
            const int i = lane - (r0 + k * RPW);
            const float got = __shfl_sync(0xffffffffu, down, (i & (RPW - 1)) * LPR);
            if (i >= 0 && i < RPW) rc = got;
            if (lr >= 32) continue;
            uint32_t h[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
              h[b] = pack_half2(__uint_as_float(w[b] << 16) * up, __uint_as_float(w[b] & 0xFFFF0000u) * up);
            st_shared_v4(sbase + C::OFF_Q + t * C::TILE + (col >> 3) * C::CHUNK + tr * 128 + (((col & 7) ^ (tr & 7)) << 4),
                         h[0], h[1], h[2], h[3]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(B_QFULL));
      }

      for (int j = 0; j < x.blocks; ++j) {
        ok = warp_wait_all(bar(B_SFULL + t), (g + j) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        // S is read in halves of 64 columns, so that a thread keeps to 128
        // registers and the loops' code to the instruction cache: both for the
        // maxima, then the second from registers and the first again.
        const float2 *scs = scales + ((g + j) & 3) * 8;
        const int col0 = x.token + j * BN;
        uint32_t sr[64];
        float *s = reinterpret_cast<float *>(sr);
        const Pages pages = block_pages[(g + j) & 3];
        const bool whole = col0 + BN <= lim_warp && !pages.hole;
        auto read_half = [&](int h) {
          tmem_ld32(ts + h * 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld32(ts + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_wait_ld();
          if (!whole) {   // what the row does not see, or has no page: -inf
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int seen = scs[4 * h + q].y == -INFINITY ? 0 : lim - col0 - 64 * h - 16 * q;
#pragma unroll
              for (int e = 0; e < 16; ++e) s[16 * q + e] = e < seen ? s[16 * q + e] : -INFINITY;
            }
          }
        };
        // row maxima of s - m (base 2; of s for the first keys), by the pages' groups,
        // and of s - m + log2 sv
        const float m_0 = m_s == -INFINITY ? 0.f : m_s;
        float mxs = -INFINITY, mxo = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          read_half(h);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 kv = scs[4 * h + q];
            float mx = s[16 * q];
#pragma unroll
            for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[16 * q + e]);
            mx = fmaf(mx, fmaxf(rc * kv.x, kTiny), -m_0);
            mxs = fmaxf(mxs, mx);
            mxo = fmaxf(mxo, mx + kv.y);
          }
        }
        float al = 1.f, ao = 1.f;
        const bool rescale = __any_sync(0xffffffffu, mxs > kLag || mxo > m_d + kLag) || big;
        if (rescale) {
          float ns = m_s == -INFINITY ? mxs : m_s + fmaxf(mxs, 0.f), top = mxo - (ns - m_0);
          big = __any_sync(0xffffffffu, fabsf(m_0) > kBig || (fabsf(ns) > kBig && ns != -INFINITY));
          if (big) {
            // Scores so large that s - m above is off by whole units: once more, exactly.
            const float2 m = maxima_apart(ts, scs, rc, m_s, lim - col0);
            ns = m.x;
            top = m.y;
          }
          // a row that has seen no key yet has l = 0 and O = 0 (or nothing, block 0)
          const float shift = ns == m_s ? 0.f : m_s - ns, nd = fmaxf(shift + m_d, top);
          al = fast_exp2(shift);
          ao = nd == m_d ? al : fast_exp2(shift + (m_d - nd));
          m_s = ns;
          m_d = nd;
        }
        const bool none = m_s == -INFINITY;
        const float ms = none ? 0.f : m_s, diff = none ? 0.f : kShift - m_d;
        float sum = 0.f;
        const bool apart = __any_sync(0xffffffffu, diff + pages.top > kOver) || big;
#pragma unroll 1
        for (int h = 1; h >= 0; --h) {
          if (h == 0) {
            read_half(0);
            tc_fence_before();
            mbar_arrive(bar(B_SEMPTY + t));   // the next block's S may take the columns
          } else if (g + j > 0) {             // P V of the block before is done with P
            ok = warp_wait_all(bar(B_PEMPTY + t), (g + j - 1) & 1, wc);
            tc_fence_after();
            if (!ok) break;
          }
          if (apart) {                        // all of the block
            sum = weigh_apart<C::CHUNK>(ts, prow, scs, rc, ms, diff, lim - col0, r);
            tc_fence_before();
            mbar_arrive(bar(B_SEMPTY + t));
            break;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 kv = scs[4 * h + q];
            const float cf = fmaxf(rc * kv.x, kTiny);
            const float gain = fast_exp2(diff + kv.y);
            uint32_t pk[8];
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float p0 = fast_exp2(fmaf(s[16 * q + 2 * e], cf, -ms));
              const float p1 = fast_exp2(fmaf(s[16 * q + 2 * e + 1], cf, -ms));
              part[e & 3] += p0 + p1;
              pk[e] = pack_half2(p0 * gain, p1 * gain);
            }
            sum += (part[0] + part[1]) + (part[2] + part[3]);
            // 16 columns = 32 bytes: two 16-byte units of the row
            const uint32_t at = prow + h * C::CHUNK + (((2 * q) ^ (r & 7)) << 4);
            st_shared_v4(at, pk[0], pk[1], pk[2], pk[3]);
            st_shared_v4(at ^ 16, pk[4], pk[5], pk[6], pk[7]);
          }
        }
        l = l * al + sum;
        if (!ok) break;
        fence_proxy_async_smem();
        if (rescale && j > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(to + c * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * ao);
            tmem_st32(to + c * 32, ov);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(bar(B_PFULL + t));
      }
      if (ok) ok = warp_wait_all(bar(B_OFULL + t), u & 1, wc);
      if (!ok) break;
      // ------------------------------------------------------------ epilogue
      tc_fence_after();
      const bool seen = !(l == 0.f);
      // O's factor as two, as in the other kernel
      const float f0 = seen ? fast_exp2(0.5f * (m_d - kShift)) : 0.f, f1 = seen ? f0 / l : 0.f;
      const bool nans = nan_any[u & 1] != 0;
      const long long prt = x.part < 0 ? 0 : (long long)(x.part + t * BM + r);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(to + c * 32, ov);
        tmem_wait_ld();
        float *o = reinterpret_cast<float *>(ov);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = seen ? o[e] * f1 * f0 : 0.f;
        if (nans) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (nan_at[(u & 1) * D + c * 32 + e] < lim) o[e] = __uint_as_float(0x7FC00000u);
        }
        if (!live) continue;
        if (x.part < 0) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
          // (rows of o are 16-byte aligned only: the caller's pointer may be)
          uint4 *dst = reinterpret_cast<uint4 *>(p.o + row * D + c * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        } else {
          float *dst = p.o_part + prt * D + c * 32;
#pragma unroll
          for (int e = 0; e < 4; ++e) store8(dst + 8 * e, &ov[8 * e]);
        }
      }
      if (live) {
        if (x.part < 0) p.lse[row] = seen ? (m_s + log2f(l)) * 0.69314718055994531f : -INFINITY;
        else p.l_part[prt] = make_float2(m_s, l);
      }
      tc_fence_before();
      mbar_arrive(bar(B_OEMPTY + t));
      mbar_arrive(bar(B_UEMPTY + (u & 1)));
      g += x.blocks;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class C>
int run_tiles(const CacheArgs &a, const FwdCachePlan &x) {
  const FwdCacheParams p = fwd_cache_params(a, x);
  auto kern = fwd_cache_tile_kernel<C>;
  static unsigned long long allowed = 0;
  if (!allow_smem(kern, C::SMEM, &allowed)) return 5;
  kern<<<x.ctas, kThreads, C::SMEM, a.stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return 5;
  return launch_fwd_cache_merge<C::D, typename C::L>(p, a.stream);
}

// Two tiles where more than one is filled and TMEM holds two (d <= 128).
bool two_tiles(const CacheArgs &a) { return a.d <= 128 && (double)(a.Hq / a.Hkv) * a.Nq > BM; }

}  // namespace

FwdCachePlan fwd_cache_tile_plan(const CacheArgs &a) {
  return two_tiles(a) ? fwd_cache_plan<TileCfg<128, 2>::L>(a, 148, kWhole, kWholeMany)
                      : fwd_cache_plan<TileCfg<128, 1>::L>(a, 148, kWhole, kWholeMany);
}

int launch_fwd_cache_tiles(const CacheArgs &a, const FwdCachePlan &x) {
  switch (a.d) {
    case 64: return two_tiles(a) ? run_tiles<TileCfg<64, 2>>(a, x) : run_tiles<TileCfg<64, 1>>(a, x);
    case 128: return two_tiles(a) ? run_tiles<TileCfg<128, 2>>(a, x) : run_tiles<TileCfg<128, 1>>(a, x);
    case 256: return run_tiles<TileCfg<256, 1>>(a, x);
    default: return 2;
  }
}

}  // namespace fa
