"""Float64 CPU oracle of the serving operators: rotary positions, the paged
E4M3 key/value cache, attention over it.

TEST INFRASTRUCTURE ONLY, as the rest of this package; it shares no code with
the CUDA library.  Definitions (include/fa.h states the same):

* rope: pair p of a row at position t turns by a = t f_p,
  (x, y) -> m (x cos a - y sin a, y cos a + x sin a); its gradient is the
  transposed map.
* cache: pages of P tokens, E4M3 codes and one scale per page and head.
  Appending sets scale = the least power of two s >= 2^-112 with amax <= 448 s
  over the call's new finite values of the page (max with the older scale when
  the page holds older tokens, whose codes are then rounded again at the new
  scale), code = E4M3(x / scale), infinities saturating.
* attention: softmax(scale q K^T [bottom-right causal]) V over the first
  lens[b] tokens; rows that see no key give O = 0, L = -inf.

Parity: pinned by tests/test_oracle_serving.py.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_decode, e4m3_round

__all__ = ["rope", "rope_freqs", "block_scale", "cache_append", "cache_tokens", "cache_attention",
           "SCALE_MIN"]

SCALE_MIN = 2.0 ** -112


def rope_freqs(rot, theta=10000.0, kind="none", factor=1.0, original_len=4096, beta_fast=32.0,
               beta_slow=1.0):
    if kind == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * np.arange(rot // 2) / rot)
    m = 1.0
    if kind == "linear":
        f = f / factor
    if kind == "yarn":
        g = np.clip((original_len * f / (2 * np.pi) - beta_slow) / (beta_fast - beta_slow), 0, 1)
        f = f * (1 - g) / factor + f * g
        m = 0.1 * np.log(factor) + 1.0
    return f, m


def rope(x, positions, freqs, mscale=1.0, interleaved=False, backward=False):
    """x [B, H, N, d], positions [B, N] or [N]; float64 result."""
    x = np.asarray(x, np.float64)
    rot = 2 * len(freqs)
    pos = np.broadcast_to(np.asarray(positions, np.float64), (x.shape[0], x.shape[2]))
    a = pos[:, None, :, None] * np.asarray(freqs, np.float64)
    z = np.exp(1j * (-a if backward else a)) * mscale
    i = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    j = i + (1 if interleaved else rot // 2)
    w = (x[..., i] + 1j * x[..., j]) * z
    y = x.copy()
    y[..., i], y[..., j] = w.real, w.imag
    return y


def block_scale(amax: float) -> float:
    """Least power of two s >= 2^-112 with amax <= 448 s."""
    s = SCALE_MIN
    if amax > 448.0 * s:
        s = 2.0 ** (np.floor(np.log2(amax / 448.0)) - 1)
        while amax > 448.0 * s:
            s *= 2.0
    return s


def _encode(x):
    """E4M3 codes of float64 values: round to nearest even, saturating; NaN -> 0x7F."""
    x = np.asarray(x, np.float64)
    v = e4m3_round(np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448))
    table = e4m3_decode(np.arange(0x7F, dtype=np.uint8))
    c = np.searchsorted(table, v).astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), c).astype(np.uint8)


def cache_append(x, cache, scale, table, start, count, page):
    """Append x [B, H, T, d] to (cache uint8 [pages, H, page, d], scale
    [pages, H]) in place, by the definition above; out-of-range pages and
    positions are left out."""
    B, H, T, _ = x.shape
    for b in range(B):
        n = T if count is None else max(0, min(int(count[b]), T))
        if start[b] < 0:
            continue
        t = 0
        while t < n:
            pos = int(start[b]) + t
            slot = pos % page
            m = min(page - slot, n - t)
            pi = pos // page
            pg = int(table[b][pi]) if pi < len(table[b]) else -1
            if 0 <= pg < cache.shape[0]:
                for h in range(H):
                    new = np.asarray(x[b, h, t:t + m], np.float64)
                    fin = np.abs(new[np.isfinite(new)])
                    s = block_scale(float(fin.max()) if fin.size else 0.0)
                    if slot:
                        old = float(scale[pg, h])
                        s = max(s, old)
                        if s > old:
                            c = cache[pg, h, :slot]
                            cache[pg, h, :slot] = _encode(e4m3_decode(c) * (old / s))
                    scale[pg, h] = s
                    cache[pg, h, slot:slot + m] = _encode(new / s)
            t += m


def cache_tokens(cache, scale, table_b, n, page):
    """The first n tokens of one sequence, float64 [H, n, d]; tokens on pages
    out of range are NaN (no value)."""
    H, d = cache.shape[1], cache.shape[3]
    out = np.full((H, n, d), np.nan)
    for pi in range((n + page - 1) // page):
        pg = int(table_b[pi])
        hi = min(n, (pi + 1) * page)
        if 0 <= pg < cache.shape[0]:
            out[:, pi * page:hi] = (e4m3_decode(cache[pg]) * scale[pg].astype(np.float64)[:, None, None])[:, :hi - pi * page]
    return out


def cache_attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, page, scale, causal):
    """(O, L, W, A, U) float64; tokens on pages out of range are hidden.  For
    error bounds: W[b, h, i, c] = sum_j p_j |v_jc|, the size of the terms O is
    summed from; A[b, h, i], the largest scale * sum |q k| of a row; and
    U[b, h, i, c] = max_j (p_j sv_j) * sum_j |code_jc|, what O would be off by
    were every weight p_j sv_j off by as much as the largest."""
    q = np.asarray(q, np.float64)
    B, Hq, Nq, d = q.shape
    Hkv = k_cache.shape[1]
    o = np.zeros(q.shape)
    w = np.zeros(q.shape)
    lse = np.full((B, Hq, Nq), -np.inf)
    amp = np.zeros((B, Hq, Nq))
    unit = np.zeros(q.shape)
    for b in range(B):
        n = max(0, min(int(lens[b]), len(table[b]) * page))
        if n == 0:
            continue
        k = cache_tokens(k_cache, k_scale, table[b], n, page)
        v = cache_tokens(v_cache, v_scale, table[b], n, page)
        sv = np.stack([v_scale[int(table[b][j // page]) % v_scale.shape[0]] for j in range(n)], 1)
        there = np.array([0 <= int(table[b][j // page]) < k_cache.shape[0] for j in range(n)])
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            for i in range(Nq):
                lim = min(n, n - Nq + i + 1) if causal else n
                see = np.flatnonzero(there[:max(lim, 0)])
                if not see.size:
                    continue
                kk, vv = k[hk][see], v[hk][see]
                s = scale * (kk @ q[b, h, i])
                amp[b, h, i] = scale * (np.abs(kk) @ np.abs(q[b, h, i])).max()
                m = s.max()
                e = np.exp(s - m)
                lse[b, h, i] = m + np.log(e.sum())
                p = e / e.sum()
                o[b, h, i] = p @ vv
                w[b, h, i] = p @ np.abs(vv)
                unit[b, h, i] = (p * sv[hk][see]).max() * (np.abs(vv) / sv[hk][see][:, None]).sum(0)
    return o, lse, w, amp, unit
