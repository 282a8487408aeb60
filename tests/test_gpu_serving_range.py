"""Attention over the paged E4M3 cache at the ends of its range: pages whose V has
very different scales, hidden ones among them, or the least one; scores of any size; NaN,
bad pages and empty batches there.  Appending to pages whose older scale is no power of two.  Calls
that share buffers.

Tolerances are those of test_gpu_serving.py (a weight rounded once to 11 bits, the
scores' error e_s through the exponential, float32 sums, weights below 2^-26 of a row's
largest to steps of it, half a step of the output) plus what tiny results add: half
a step of bfloat16's subnormals, 2^-134, and float32's in the partial results and their
products, less than 2^-140 in all.
"""
import numpy as np
import pytest
import torch

import exact_io_aware_50_b200 as F
from oracle import serving as S
from oracle.fp8 import e4m3_decode
from test_gpu_serving import U16, f64, i32, new_cache, np_cache

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -134 + 2.0 ** -140


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    F.lib()
    yield


def cache_of(k, v, lens, page, wide=0):
    """Sequences' tokens k, v [B, H, n, d] (float32) in a cache whose pages stand in
    no order and whose free slots hold NaN codes; the table has room for `wide` more
    tokens, on pages that are none."""
    B, H, n, d = k.shape
    width = (n + page - 1) // page
    cache = new_cache(B * width + 1, H, page, d)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(n)).reshape(B, width).to(torch.int32)
    F.cache_append(k.cuda(), v.cuda(), *cache, table.cuda(), i32([0] * B), i32(lens))
    return cache, torch.cat([table, torch.full((B, wide // page), -1, dtype=torch.int32)], dim=1)


def check(q, cache, table, lens, page, causal, scale, exact_scores=False):
    """exact_scores: the scores' differences are 0 or many times their error, so that the
    error of a score does not enter O."""
    out = o, lse = F.forward_cache(q.cuda(), *cache, table.cuda(), i32(lens), scale=scale, causal=causal)
    torch.cuda.synchronize()
    assert F.fa_device_status() == F.FA_OK
    ref_o, ref_l, w, amp, unit = S.cache_attention(f64(q), *np_cache(cache), table.tolist(), lens, page, scale, causal)
    o, lse, d = f64(o), f64(lse), q.shape[3]
    none = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
    e_s = amp * (d * 2.0 ** -23 + 2.0 ** -20)
    e_o = 0 * e_s if exact_scores else e_s
    assert e_o.max() < 0.1
    tol = np.abs(ref_o) * U16 + w * (2.0 ** -11 + 2.0 ** -13 + np.expm1(2 * e_o[..., None])) + unit * 2.0 ** -37 + TINY
    bad = np.abs(o - ref_o) - tol
    at = np.unravel_index(np.argmax(np.where(np.isfinite(bad), bad, np.inf)), bad.shape)
    assert np.isfinite(o).all() and (bad <= 0).all(), f"O[{at}] = {o[at]:.6g}, not {ref_o[at]:.6g} within {tol[at]:.3g}"
    lse, ref_l, e_s = lse[~none], ref_l[~none], e_s[~none]
    assert (np.abs(lse - ref_l) <= e_s + 2.0 ** -18 * (1 + np.abs(ref_l))).all()
    return out


ROWS = [(1, 1), (4, 5), (1, 130)]    # query heads, queries: one row, two 16-row tiles, 128-row tiles


@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "x".join(map(str, r)))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("gap,first,others", [
    (80, 0, 8000), (80, 0, 1e20), (20, 0, 1e30), (80, 1e-25, 1e10), (-80, 1e20, 0), (-80, 1e10, 1e-25),
    (88, 0, 8000), (96, 0, 8000), (88, 0, 1e20), (120, 0, 1e20), (88, 1e-25, 1e12), (120, 3e-30, 1e20), (-88, 1e20, 0)])
def test_v_scales_far_apart(gap, first, others, d, rows):
    """The first page's keys score `gap` nats above the others; its V is of size
    `first`, the others' of size `others`.  Early causal queries see the first
    page alone, with the others hidden beside it."""
    Hq, Nq = rows
    g = torch.Generator().manual_seed(d + Nq)
    lens, page = [66, 140, 200], 16
    k, v = torch.randn(2, 3, 1, 200, d, generator=g)
    k[..., 0] = 0
    k[:, :, :page] = 0
    k[:, :, :page, 0] = gap
    v[:, :, :page] *= first
    v[:, :, page:] *= others
    q = 0.1 * torch.randn(3, Hq, Nq, d, generator=g)
    q[..., 0] = 1.0
    for wide in (0, 4096):
        cache, table = cache_of(k, v, lens, page, wide)
        check(q.to(torch.bfloat16), cache, table, lens, page, True, 1.0)


SIZES = [1e3, 1e5, 1e6, 3e6, 1.2e7, 4e7, 1e8, 2.5e8, 1e9, 1e12, 1e30]


def large_scores(size, B, Hq, Nq, d, g):
    """q whose product with a key (1, 0, ..) is about +-size / 0.7, no two rows alike."""
    q = torch.randn(B, Hq, Nq, d, generator=g)
    q[..., 0] = (1 + torch.rand(B, Hq, Nq, generator=g)) * size * torch.tensor([1.0, -1.0])[torch.arange(Nq) % 2]
    return q.to(torch.bfloat16)


@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "x".join(map(str, r)))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("size", SIZES)
def test_equal_keys_of_large_scores(size, d, rows):
    """Equal scores, however large, share the weight equally, whatever the pages' scales:
    a row that sees one key returns its V."""
    Hq, Nq = rows
    g = torch.Generator().manual_seed(d + Nq)
    lens, page = [1, 64, 256], 16
    k = torch.zeros(3, 1, 256, d)
    k[..., 0] = 1.0
    v = torch.randn(3, 1, 256, d, generator=g)
    for b, f in enumerate((1.0, 2.0 ** 9, 2.0 ** -14)):
        v[b].view(16, page, d)[b::3] *= f
    cache, table = cache_of(k, v, lens, page)
    q = large_scores(size, 3, Hq, Nq, d, g)
    o, _ = check(q, cache, table, lens, page, False, 0.7, exact_scores=True)
    one = e4m3_decode(cache[1][int(table[0, 0]), 0, 0].cpu().numpy()) * float(cache[3][int(table[0, 0]), 0])
    assert (f64(o[0]) == one).all()


@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "x".join(map(str, r)))
@pytest.mark.parametrize("size", SIZES)
def test_one_key_above_the_others(size, rows):
    """The largest of several scores, all large, takes the whole weight; one block may
    raise the maximum by any amount, and V's scales differ by up to 2^40."""
    Hq, Nq = rows
    g = torch.Generator().manual_seed(Nq)
    lens, page, d = [500, 333, 190], 32, 64
    k = torch.zeros(3, 1, 500, d)
    k[..., 0] = (torch.rand(3, 1, 500, generator=g) - 0.5) * torch.logspace(-6, 0, 500)[None, None, :]
    k[:, 0, 7, 0], k[:, 0, 401, 0], k[:, 0, 150, 0], k[:, 0, 155, 0] = 1.5, 2.0, -1.5, -2.0
    k[2, 0, 20] *= 0
    v = torch.randn(3, 1, 500, d, generator=g)
    v[..., 64:96, :] *= 2.0 ** 20
    v[..., 384:416, :] *= 2.0 ** -20
    for wide in (0, 4096):
        cache, table = cache_of(k, v, lens, page, wide)
        check(large_scores(max(size, 1e4), 3, Hq, Nq, d, g), cache, table, lens, page, False, 0.7, exact_scores=True)


@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "x".join(map(str, r)))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,wide", [(17, 0), (100, 0), (17, 4096), (1000, 4096), (3000, 8192)])
def test_equal_keys_fall_apart_unevenly(n, wide, d, rows):
    """Equal keys that warps and CTAs share unevenly are one mean all the same, whatever
    the scores' size."""
    Hq, Nq = rows
    g = torch.Generator().manual_seed(d + Nq)
    k = torch.zeros(1, 1, n, d)
    k[..., 0] = 1.0
    v = 1.0 + torch.randn(1, 1, n, d, generator=g)
    cache, table = cache_of(k, v, [n], 16, wide)
    for size in (1.0, 4e7, 1e9):
        check(large_scores(size, 1, Hq, Nq, d, g), cache, table, [n], 16, False, 0.7, exact_scores=True)


CODES = e4m3_decode(np.arange(0x7F, dtype=np.uint8))
TIES = (CODES[1:] + CODES[:-1]) / 2            # what lies between two codes, all on a float32


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("T", [6, 40])
def test_append_to_pages_of_any_scale(dt, d, T):
    """New tokens, multiples of an older scale that lie on a tie between two codes among
    them, are rounded once; equal codes and scales."""
    scales = [m / 128 for m in (41, 47, 51, 52, 55, 56, 60, 61, 63, 95, 104, 109, 112, 122, 127)] + [0.7, 1e-3, 3e7, 0.5]
    scales = np.asarray(scales, np.float32)
    H, page, start = len(scales), 64, 5
    cache = new_cache(1, H, page, d)
    cache[0].random_(0, 0x7F)
    cache[1].random_(0x80, 0xFF)
    cache[2][0] = cache[3][0] = torch.from_numpy(scales)
    g = torch.Generator().manual_seed(d)
    t = torch.from_numpy(TIES[TIES <= 224])
    pick = t[torch.randint(len(t), (2, 1, H, T, d), generator=g)] * (1 - 2 * torch.randint(2, (2, 1, H, T, d), generator=g))
    near = 1 + 2.0 ** -20 * torch.randint(-1, 2, pick.shape, generator=g)
    k, v = (pick * near * torch.from_numpy(scales).double()[:, None, None]).to(dt)
    ref, table = np_cache(cache), torch.tensor([[0]], dtype=torch.int32)
    F.cache_append(k.cuda(), v.cuda(), *cache, table.cuda(), i32([start]))
    torch.cuda.synchronize()
    for x, i in ((k, 0), (v, 1)):
        S.cache_append(f64(x), ref[i], ref[i + 2], table.tolist(), [start], None, page)
        assert np.array_equal(ref[i + 2][0], scales)        # the older scales are the larger ones
        assert np.array_equal(f64(cache[i + 2]), ref[i + 2])
        assert np.array_equal(cache[i].cpu().numpy(), ref[i])


@pytest.mark.parametrize("d", [64, 128])
def test_append_grows_a_scale_that_is_no_power_of_two(d):
    """Older codes times such a scale, next to a tie between two codes of the new one, are
    rounded once."""
    code = np.arange(0x31, 0x41)                            # 0.5625 to 2
    tie = TIES[0x30:0x38]                                   # 0.53 to 0.97
    scales = np.float32(tie[None, :] / CODES[code][:, None]).ravel()
    scales = scales[(scales < 1) & (np.frexp(scales)[0] != 0.5)]
    H, page = len(scales), 16
    cache = new_cache(1, H, page, d)
    for i in (0, 1):
        cache[i][:] = torch.from_numpy(code.astype(np.uint8))[torch.arange(d) % 16] + 0x80 * i
        cache[i + 2][0] = torch.from_numpy(scales)
    x = torch.full((1, H, 2, d), 448.0)                     # the new scale: 1
    ref, table = np_cache(cache), torch.tensor([[0]], dtype=torch.int32)
    F.cache_append(x.cuda(), x.cuda(), *cache, table.cuda(), i32([9]))
    torch.cuda.synchronize()
    for i in (0, 1):
        S.cache_append(f64(x), ref[i], ref[i + 2], table.tolist(), [9], None, page)
        assert (ref[i + 2] == 1).all() and np.array_equal(f64(cache[i + 2]), ref[i + 2])
        assert np.array_equal(cache[i].cpu().numpy(), ref[i])


# -------------------------------------------------- hidden, missing and empty
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "x".join(map(str, r)))
@pytest.mark.parametrize("size,first", [(1.0, 0.0), (1e9, 1.0), (1e9, 0.0)])
def test_masks_beside_far_scales_and_large_scores(size, first, rows):
    """Causal rows, NaN codes behind each length, and a page that is none among pages of
    large V, where weights are formed apart from the common path."""
    Hq, Nq = rows
    g = torch.Generator().manual_seed(Nq)
    lens, page, d, n = [140, 300, 133], 16, 128, 300
    k = torch.zeros(3, 1, n, d)
    k[..., 0] = 1.0
    v = torch.randn(3, 1, n, d, generator=g) * 1e4
    v[:, :, :page] *= first
    for wide in (0, 4096):
        cache, table = cache_of(k, v, lens, page, wide)
        table[0, 5] = table[1, 0] = -1
        q = large_scores(size, 3, Hq, Nq, d, g)
        q[..., 0] = q[..., 0].abs()
        o, lse = F.forward_cache(q.cuda(), *cache, table.cuda(), i32(lens), scale=0.7)
        assert F.fa_device_status() == F.FA_ERR_PAGE
        ref_o, ref_l, w, _, unit = S.cache_attention(f64(q), *np_cache(cache), table.tolist(), lens, page, 0.7, True)
        tol = np.abs(ref_o) * U16 + w * (2.0 ** -11 + 2.0 ** -13) + unit * 2.0 ** -37 + TINY
        assert (np.abs(f64(o) - ref_o) <= tol).all()
        assert np.array_equal(np.isneginf(f64(lse)), np.isneginf(ref_l))


@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "x".join(map(str, r)))
@pytest.mark.parametrize("wide", [0, 4096])
def test_nan_key_reaches_only_the_rows_that_see_it(wide, rows):
    """A NaN code of K makes the rows that see its token NaN, O and L, and no others."""
    Hq, Nq = rows
    g = torch.Generator().manual_seed(3)
    n, page, d = 260, 32, 64
    k, v = torch.randn(2, 1, 1, n, d, generator=g)
    cache, table = cache_of(k, v, [n], page, wide)
    q = torch.randn(1, Hq, Nq, d, generator=g).to(torch.bfloat16).cuda()
    ref = F.forward_cache(q, *cache, table.cuda(), i32([n]))
    at = n - 1 - Nq // 2
    cache[0][int(table[0, at // page]), 0, at % page, 7] = 0xFF
    o, lse = F.forward_cache(q, *cache, table.cuda(), i32([n]))
    torch.cuda.synchronize()
    assert F.fa_device_status() == F.FA_OK
    sees = torch.arange(Nq) + n - Nq >= at
    assert torch.isnan(o[:, :, sees]).all() and torch.isnan(lse[:, :, sees]).all()
    assert torch.equal(o[:, :, ~sees], ref[0][:, :, ~sees]) and torch.equal(lse[:, :, ~sees], ref[1][:, :, ~sees])


@pytest.mark.parametrize("B", [1, 40, 200])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "x".join(map(str, r)))
def test_batches_without_a_token(rows, B):
    """Every sequence is empty: O = 0 and L = -inf all over, line or whole units."""
    Hq, Nq = rows
    for wide in (64, 8192):
        cache = new_cache(3, 2, 16, 128)
        table = torch.full((B, wide // 16), -1, dtype=torch.int32, device="cuda")
        q = torch.randn(B, 2 * Hq, Nq, 128, device="cuda").to(torch.bfloat16)
        o, lse = F.forward_cache(q, *cache, table, i32([0] * B))
        torch.cuda.synchronize()
        assert F.fa_device_status() == F.FA_OK
        assert not o.any() and torch.isneginf(lse).all()


# ------------------------------------------------------------ shared buffers
@pytest.mark.parametrize("Nq", [1, 200])
def test_one_workspace_for_graphs_replayed_in_turn(Nq):
    """Two captured calls on one caller's workspace, replayed one behind the other, whatever
    the workspace held."""
    g = torch.Generator().manual_seed(4)
    n, page, d = 3000, 64, 64
    need = F.fa_fwd_cache_workspace_size(1, 4, 2, Nq, d, page, -(-n // page))
    work = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    calls = []
    for _ in range(2):
        k, v = torch.randn(2, 1, 2, n, d, generator=g)
        cache, table = cache_of(k, v, [n], page)
        calls.append((torch.randn(1, 4, Nq, d, generator=g).to(torch.bfloat16).cuda(), *cache, table.cuda(), i32([n])))
    alone = [F.forward_cache(*c) for c in calls]
    graphs = []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = F.forward_cache(*c, workspace=work)
        graphs.append((graph, out))
    for i in (0, 1, 1, 0, 1, 0):
        for t in graphs[i][1]:
            t.fill_(1.0)
        graphs[i][0].replay()
        graphs[1 - i][0].replay()
        torch.cuda.synchronize()
        for (_, out), ref in zip(graphs, alone):
            assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    assert F.fa_device_status() == F.FA_OK


@pytest.mark.parametrize("rot", [32, 64, 128])
def test_rope_with_one_tensor_in_place(rot):
    """q turned where it stands, k into another tensor, and the other way round."""
    q, k = (torch.randn(2, H, 33, 128, device="cuda").to(torch.bfloat16) for H in (4, 2))
    freqs, ms = F.rope_freqs(rot)
    pos = i32(list(range(33)))
    want = F.rope(q, k, pos, freqs, ms)
    for which in (0, 1):
        a, b = q.clone(), k.clone()
        out = (a, torch.empty_like(b)) if which == 0 else (torch.empty_like(a), b)
        got = F.rope(a, b, pos, freqs, ms, out=out)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(b, k) if which == 0 else torch.equal(a, q)


@pytest.mark.parametrize("B,Nq", [(300, 1), (148, 130)])
def test_tiny_values_over_millions_of_tokens(B, Nq):
    """V of the least scale there is, 2^-112, over 3 * 2^20 equal tokens, one page named again
    and again: their mean is the value itself, though the sum's reciprocal times the scale
    lies far below float32's normal numbers.  (Sums of equal powers of two are exact.)"""
    page, d, n = 128, 64, 3 * 2 ** 20
    cache = [torch.full((1, 1, page, d), c, dtype=torch.uint8, device="cuda") for c in (0, 0x38)]   # K 0, V 1
    cache += [torch.ones(1, 1, device="cuda"), torch.full((1, 1), S.SCALE_MIN, device="cuda")]
    table = torch.zeros(B, n // page, dtype=torch.int32, device="cuda")
    q = torch.randn(B, 1, Nq, d, device="cuda").to(torch.bfloat16)
    o, lse = F.forward_cache(q, *cache, table, i32([n] * B), causal=False)
    torch.cuda.synchronize()
    assert F.fa_device_status() == F.FA_OK
    assert float((o.double() / S.SCALE_MIN - 1).abs().max()) <= U16 + 2.0 ** -11
    assert float((lse.double() - np.log(n)).abs().max()) <= 2.0 ** -18 * (1 + np.log(n))
