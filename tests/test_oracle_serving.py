"""Pins of oracle/serving.py (CPU): closed forms and identities of the
definitions, torch's own E4M3 conversion, finite differences of the rotation."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S


def test_rope_is_a_rotation():
    rng = np.random.default_rng(1)
    f, _ = S.rope_freqs(8)
    q, k = rng.normal(size=(2, 1, 1, 5, 12))
    for inter in (False, True):
        a = S.rope(q, np.arange(5) + 7, f, interleaved=inter)
        assert np.allclose((a ** 2).sum(-1), (q ** 2).sum(-1), atol=1e-12)
        assert np.array_equal(a[..., 8:], q[..., 8:])
        # scores depend on the difference of positions alone
        s1 = a @ np.swapaxes(S.rope(k, np.arange(5) + 7, f, interleaved=inter), -1, -2)
        s2 = S.rope(q, np.arange(5) + 107, f, interleaved=inter) @ \
            np.swapaxes(S.rope(k, np.arange(5) + 107, f, interleaved=inter), -1, -2)
        assert np.allclose(s1, s2, atol=1e-9)
        # backward inverts forward (mscale 1), and position 0 is the identity
        assert np.allclose(S.rope(a, np.arange(5) + 7, f, interleaved=inter, backward=True), q)
        assert np.allclose(S.rope(q, np.zeros(5), f, interleaved=inter), q)


def test_rope_worked_example():
    x = np.zeros((1, 1, 1, 8))
    x[..., 0] = 1.0
    f = np.array([np.pi / 2, 1, 1, 1])
    half = S.rope(x, [1], f, mscale=2.0)[0, 0, 0]
    assert np.allclose(half, [0, 0, 0, 0, 2, 0, 0, 0], atol=1e-15)
    inter = S.rope(x, [1], f, interleaved=True)[0, 0, 0]
    assert np.allclose(inter, [0, 1, 0, 0, 0, 0, 0, 0], atol=1e-15)


def test_rope_gradient_by_differences():
    rng = np.random.default_rng(2)
    f, _ = S.rope_freqs(8)
    x, g = rng.normal(size=(2, 1, 2, 3, 10))
    pos = np.array([3, 11, 4])
    for inter in (False, True):
        dx = S.rope(g, pos, f, 1.3, inter, backward=True)
        for at in np.ndindex(x.shape):
            e = np.zeros(x.shape)
            e[at] = 1e-6
            num = ((S.rope(x + e, pos, f, 1.3, inter) - S.rope(x - e, pos, f, 1.3, inter)) * g).sum() / 2e-6
            assert abs(num - dx[at]) < 1e-7


def test_rope_freqs_scalings():
    f, m = S.rope_freqs(16)
    assert m == 1.0 and f[0] == 1.0 and np.isclose(f[-1], 10000.0 ** (-14 / 16))
    assert np.allclose(S.rope_freqs(16, kind="linear", factor=4)[0], f / 4)
    n = S.rope_freqs(16, kind="ntk", factor=4)[0]
    assert n[0] == 1.0 and np.isclose(n[-1], f[-1] / 4)     # the slowest pair is stretched by factor
    y, m = S.rope_freqs(128, kind="yarn", factor=16)
    f = S.rope_freqs(128)[0]
    assert np.isclose(m, 0.1 * np.log(16) + 1)
    assert np.isclose(y[0], f[0]) and np.isclose(y[-1], f[-1] / 16)
    assert ((y <= f * (1 + 1e-15)) & (y >= f / 16 * (1 - 1e-15))).all()


def test_block_scale():
    assert S.block_scale(0.0) == S.SCALE_MIN
    for a in (448.0, 449.0, 1.0, 0.875, np.nextafter(0.875, 1), 3e38, 1e-30, 7.0, 2.0 ** -100):
        s = S.block_scale(a)
        assert a <= 448 * s and (s == S.SCALE_MIN or a > 448 * s / 2)
        assert np.log2(s) == np.round(np.log2(s))
    assert S.block_scale(448.0) == 1.0 and S.block_scale(np.nextafter(448.0, 449)) == 2.0


def test_encode_matches_torch():
    x = np.concatenate([np.linspace(-448, 448, 20001), 2.0 ** np.arange(-14.0, 8) * 1.0625,
                        [0.0, -0.0, np.nan, 2.0 ** -10, 1.5 * 2.0 ** -9]]).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = S._encode(x)
    assert np.array_equal(np.where(np.isnan(x), 0, got), np.where(np.isnan(x), 0, ref))
    assert np.isnan(oracle_decode(got[np.isnan(x)])).all()
    assert S._encode(np.array([np.inf]))[0] == 0x7E and S._encode(np.array([-np.inf]))[0] == 0xFE


def oracle_decode(c):
    from oracle.fp8 import e4m3_decode
    return e4m3_decode(c)


def test_append_in_pieces_equals_at_once_when_the_scale_does_not_grow():
    rng = np.random.default_rng(3)
    x = rng.uniform(0.5, 1, size=(1, 2, 40, 4))
    x[0, :, ::16] = 1.0            # every page's largest value comes first
    table = [[2, 0, 1]]
    once = [np.zeros((3, 2, 16, 4), np.uint8), np.zeros((3, 2))]
    S.cache_append(x, *once, table, [0], None, 16)
    by_one = [np.full((3, 2, 16, 4), 0x7F, np.uint8), np.ones((3, 2))]
    for t in range(40):
        S.cache_append(x[:, :, t:t + 1], *by_one, table, [t], None, 16)
    assert np.array_equal(once[1], by_one[1])
    assert np.array_equal(S.cache_tokens(*once, table[0], 40, 16), S.cache_tokens(*by_one, table[0], 40, 16))
    err = np.abs(S.cache_tokens(*once, table[0], 40, 16) - x[0])
    assert (err <= 2.0 ** -4 * np.abs(x[0])).all()


def test_append_grows_scale_and_keeps_values():
    cache, scale = np.zeros((1, 1, 16, 2), np.uint8), np.zeros((1, 1))
    S.cache_append(np.full((1, 1, 3, 2), 1.0), cache, scale, [[0]], [0], None, 16)
    s0 = scale[0, 0]
    S.cache_append(np.full((1, 1, 1, 2), 100.0), cache, scale, [[0]], [3], None, 16)
    assert s0 == 2.0 ** -8 and scale[0, 0] == 2.0 ** -2
    got = S.cache_tokens(cache, scale, [0], 4, 16)[0]
    assert np.allclose(got[:3], 1.0) and np.allclose(got[3], 100.0, rtol=2 ** -4)
    assert (cache[0, 0, 4:] == 0).all()


def test_cache_attention_equals_dense():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(2, 1, 2, 50, 8))
    caches = []
    table = [[3, 1, 0, 2]]
    for k in range(2):
        c = [np.full((4, 2, 16, 8), 0x7F, np.uint8), np.ones((4, 2))]
        S.cache_append(x[k], *c, table, [0], None, 16)
        caches.append(c)
    q = rng.normal(size=(1, 4, 3, 8))
    o, lse, w, amp, unit = S.cache_attention(q, caches[0][0], caches[1][0], caches[0][1], caches[1][1], table, [50],
                                       16, 0.3, True)
    k = S.cache_tokens(*caches[0], table[0], 50, 16)[None]
    v = S.cache_tokens(*caches[1], table[0], 50, 16)[None]
    o_ref, l_ref = oracle.forward(q, k, v, 0.3, True, 47)
    assert np.allclose(o, o_ref, atol=1e-12) and np.allclose(lse, l_ref, atol=1e-12)
    assert (w >= np.abs(o) - 1e-12).all() and (unit >= w - 1e-12).all() and (amp > 0).all()


def test_cache_attention_rows_without_keys():
    c, s = np.full((1, 1, 16, 4), 0x38, np.uint8), np.ones((1, 1))
    o, lse, _, _, _ = S.cache_attention(np.ones((2, 1, 3, 4)), c, c, s, s, [[0], [0]], [2, 0], 16, 1.0, True)
    assert (o[0, 0, 0] == 0).all() and lse[0, 0, 0] == -np.inf      # length 2, query 0 of 3 stands before it
    assert np.allclose(o[0, 0, 1:], 1.0) and (lse[1] == -np.inf).all() and (o[1] == 0).all()


@pytest.mark.parametrize("bad", [-1, 7])
def test_pages_out_of_range_are_left_out(bad):
    c, s = np.full((2, 1, 16, 4), 0x38, np.uint8), np.ones((2, 1))
    before = c.copy()
    S.cache_append(np.ones((1, 1, 20, 4)), c, s, [[bad, 1]], [0], None, 16)
    assert np.array_equal(c[0], before[0])
    o, lse, _, _, _ = S.cache_attention(np.ones((1, 1, 1, 4)), c, c, s, s, [[bad, 1]], [20], 16, 1.0, False)
    assert np.allclose(lse, 4.0 + np.log(4))
