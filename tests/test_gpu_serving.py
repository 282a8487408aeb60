"""GPU parity of the serving operators (rotary positions, the paged E4M3 cache,
attention over it) with the float64 oracle, at the sizes and masks where they
can go wrong, and of a run of them together.

Tolerances (u16 = 2^-8 and u32 = 2^-24: half a step of bfloat16 and float32,
relative to the value):
* rope: cos and sin of a float64 angle rounded to float32 err by at most
  pi 2^-25 (the angle) + 2^-23 (two units of the function) + 2^-24 (times
  mscale); two products and one sum add 3 u32: below 2^-20 m (|x| + |y|) in
  all, plus u16 |result| for bfloat16.
* cache codes and scales: equal.
* cache_read: power-of-two scales give codes exactly; any scale: one float32
  product, one rounding: (u32 + u16) |value|.
* attention: a score's error is at most e_s = A (d 2^-23 + 2^-20), A the
  largest scale * sum |q k| of the row (d accumulations of the matrix unit,
  which may truncate, and the argument of the exponential); a weight is rounded
  once to 11 bits: 2^-11; the float32 sums of weights and of O stay below
  2^-13.  Score errors within +-e_s change a normalised weight by a factor
  within e^{+-2 e_s} (e^{+-e_s} in the numerator, the same in the sum), which is
  1 + 2 e_s only while e_s is small: scores of 1e6 and up have e_s > 1.  So
  |O - O_ref| <= u16 |O_ref| + W (2^-11 + 2^-13 + e^{2 e_s} - 1) + 2^-37 U with
  W = sum_j p_j |v_j|, U = max_j (p_j sv_j) sum_j |code_j|, and |L - L_ref| <= e_s + 2^-18 (1 + |L_ref|).
"""
import numpy as np
import pytest
import torch

import exact_io_aware_50_b200 as F
from oracle import serving as S
from oracle.fp8 import e4m3_decode

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    F.lib()
    yield


@pytest.fixture(autouse=True)
def _seed():
    torch.manual_seed(17)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rope
ROPE = [  # B, Hq, Hkv, N, d, rot, dtype, interleaved, positions from, shared positions
    (1, 1, 1, 1, 64, 64, "bf16", False, 0, False),
    (2, 4, 2, 7, 128, 128, "bf16", True, 1000000, False),
    (3, 5, 1, 33, 64, 32, "f32", False, 70, False),
    (1, 3, 3, 130, 256, 64, "f32", True, 2**31 - 200, True),
    (2, 2, 2, 65, 128, 16, "bf16", False, -40, False),
    (1, 8, 2, 19, 100, 40, "bf16", True, 5, True),      # rows that are no multiple of 16 bytes
    (1, 2, 2, 19, 100, 40, "bf16", False, 5, True),
    (2, 2, 1, 9, 36, 8, "f32", False, 5, False),
    (5, 33, 0, 3, 128, 64, "bf16", True, 4000, False),  # q alone
    (1, 40, 8, 300, 128, 128, "bf16", False, 131000, False),
    (16, 6, 6, 1, 20, 8, "bf16", True, 7, False),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("c", ROPE, ids=lambda c: "x".join(map(str, c)))
def test_rope(c, backward):
    B, Hq, Hkv, N, d, rot, dt, inter, first, shared = c
    g = torch.Generator().manual_seed(N + d)
    q = torch.randn(B, Hq, N, d, generator=g).to(DT[dt])
    k = torch.randn(B, Hkv, N, d, generator=g).to(DT[dt]) if Hkv else None
    pos = torch.arange(first, first + N, dtype=torch.int64).to(torch.int32)
    if not shared:
        pos = torch.stack([pos.roll(3 * b) for b in range(B)])
    freqs, ms = F.rope_freqs(rot, scaling="yarn", factor=8.0, original_len=2048)
    fn = F.rope_backward if backward else F.rope
    qg, kg = q.cuda(), None if k is None else k.cuda()
    outs = fn(qg, kg, pos.cuda(), freqs, ms, inter)
    again = fn(qg, kg, pos.cuda(), freqs, ms, inter, out=(qg, kg))   # in place
    assert again[0] is qg and again[1] is kg
    torch.cuda.synchronize()
    assert F.fa_device_status() == F.FA_OK
    ms32 = float(np.float32(ms))
    for x, y, z in ((q, outs[0], again[0]), (k, outs[1], again[1])):
        if x is None:
            assert y is None
            continue
        assert y.shape == x.shape and y.dtype == x.dtype and torch.equal(y, z)
        x = f64(x)
        ref = S.rope(x, pos.numpy(), f64(freqs), ms32, inter, backward)
        pair = S.rope(np.abs(x), np.zeros(N), np.zeros(rot // 2), ms32, inter)   # m |x| at its own column
        i = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
        j = i + (1 if inter else rot // 2)
        size = np.zeros(x.shape)
        size[..., i] = size[..., j] = pair[..., i] + pair[..., j]
        tol = size * 2.0 ** -20 + (np.abs(ref) * U16 if dt == "bf16" else 0)
        assert (np.abs(f64(y) - ref) <= tol).all(), float((np.abs(f64(y) - ref) - tol).max())
        assert np.array_equal(f64(y)[..., rot:], x[..., rot:])


def test_rope_backward_by_differences():
    """sum(rope(x) * g) changes along any direction u by sum(u * rope_backward(g))."""
    torch.manual_seed(3)
    x, g, u = (torch.randn(1, 2, 9, 64, device="cuda") for _ in range(3))
    freqs, _ = F.rope_freqs(48)
    pos = i32(list(range(100, 109)))
    dx, _ = F.rope_backward(g, None, pos, freqs, 1.25)
    hi, lo = (F.rope(x + s * u, None, pos, freqs, 1.25)[0].double() for s in (0.5, -0.5))
    num = ((hi - lo) * g.double()).sum()
    # the map is linear: only float32 rounding of x +- u / 2 and of the results
    bound = 8 * 2.0 ** -20 * float((g.abs() * (x.abs() + u.abs())).sum())
    assert abs(float(num - (u.double() * dx.double()).sum())) <= bound


# ------------------------------------------------------------------ cache
def new_cache(num_pages, H, page, d, fill=0x7F):
    return [torch.full((num_pages, H, page, d), fill, dtype=torch.uint8, device="cuda"),
            torch.full((num_pages, H, page, d), fill, dtype=torch.uint8, device="cuda"),
            torch.rand(num_pages, H, device="cuda").log2().floor().exp2(),
            torch.rand(num_pages, H, device="cuda").log2().floor().exp2()]


def np_cache(c):
    return [c[0].cpu().numpy().copy(), c[1].cpu().numpy().copy(), f64(c[2]), f64(c[3])]


def table_for(B, width, num_pages, seed=0):
    g = torch.Generator().manual_seed(seed)
    assert B * width <= num_pages
    return torch.randperm(num_pages, generator=g)[:B * width].reshape(B, width).to(torch.int32)


APPEND = [  # B, H, T, d, page, dtype, starts, counts
    (1, 1, 1, 64, 16, "bf16", [0], None),
    (3, 2, 1, 128, 64, "bf16", [0, 63, 64], None),
    (2, 3, 1, 256, 16, "f32", [17, 15], [1, 0]),
    (4, 1, 16, 64, 16, "f32", [0, 1, 15, 16], [16, 16, 3, 0]),
    (2, 2, 200, 128, 32, "bf16", [5, 96], [200, 131]),
    (2, 5, 130, 64, 128, "bf16", [0, 127], [129, 130]),
    (1, 2, 300, 256, 128, "f32", [77], None),
    (2, 1, 33, 128, 16, "bf16", [0, 3], [-5, 99]),       # counts are clamped to [0, T]
]


@pytest.mark.parametrize("c", APPEND, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_append(c):
    B, H, T, d, page, dt, start, count = c
    g = torch.Generator().manual_seed(T)
    k, v = ((torch.randn(B, H, T, d, generator=g) * torch.exp(3 * torch.randn(B, H, T, 1, generator=g))).to(DT[dt])
            for _ in range(2))
    width = max((s + T + page - 1) // page for s in start)
    table = table_for(B, width, B * width + 2)
    cache = new_cache(B * width + 2, H, page, d)
    cache[0].random_(0, 0x7F)       # older tokens: any codes
    cache[1].random_(0x80, 0xFF)
    ref = np_cache(cache)
    F.cache_append(k.cuda(), v.cuda(), *cache, table.cuda(), i32(start), None if count is None else i32(count))
    torch.cuda.synchronize()
    assert F.fa_device_status() == F.FA_OK
    for x, i in ((k, 0), (v, 1)):
        S.cache_append(f64(x), ref[i], ref[i + 2], table.tolist(), start, count, page)
        assert np.array_equal(cache[i].cpu().numpy(), ref[i])
        assert np.array_equal(f64(cache[i + 2]), ref[i + 2])


def test_append_values_at_the_edges():
    """Zeros, values next to a scale's border, subnormals, infinities, NaN."""
    edge = [0.0, -0.0, 448.0, 449.0, float("inf"), -float("inf"), float("nan"), 1e-40, 3e38, -3.4e38, 2.0 ** -112,
            448 * 2.0 ** -112, 0.875, 0.8750001, 1e-30, 7.0]
    x = torch.zeros(len(edge), 1, 16, 64)
    for i, e in enumerate(edge):
        x[i, 0, ::3, ::2] = e
        x[i, 0, 1, 1] = e * 0.3 if np.isfinite(e) else 1.5
    x[0, 0, 3:5] = 0.0
    cache = new_cache(len(edge), 1, 16, 64)
    table = table_for(len(edge), 1, len(edge))
    ref = np_cache(cache)
    F.cache_append(x.cuda(), (-x).cuda(), *cache, table.cuda(), i32([0] * len(edge)))
    torch.cuda.synchronize()
    for y, i in ((x, 0), (-x, 1)):
        S.cache_append(f64(y), ref[i], ref[i + 2], table.tolist(), [0] * len(edge), None, 16)
        assert np.array_equal(f64(cache[i + 2]), ref[i + 2])
        a, b = e4m3_decode(cache[i].cpu().numpy()), e4m3_decode(ref[i])
        assert np.array_equal(a, b, equal_nan=True)


def test_append_token_by_token_follows_the_definition():
    """A page's scale grows while it fills; the codes are those of the oracle's
    own token-by-token run."""
    g = torch.Generator().manual_seed(11)
    H, d, page = 2, 128, 16
    x = torch.randn(2, H, 40, d, generator=g) * torch.logspace(-3, 3, 40)[None, None, :, None]
    x = x.to(torch.bfloat16)
    cache = new_cache(8, H, page, d)
    table, ref = table_for(2, 4, 8), np_cache(cache)
    t_dev = table.cuda()
    for t in range(40):
        F.cache_append(x[:, :, t:t + 1].contiguous().cuda(), x[:, :, t:t + 1].contiguous().cuda(), *cache, t_dev,
                       i32([t, t + 5]))
        for i in (0, 1):
            S.cache_append(f64(x[:, :, t:t + 1]), ref[i], ref[i + 2], table.tolist(), [t, t + 5], None, page)
    for i in (0, 1):
        assert np.array_equal(cache[i].cpu().numpy(), ref[i]) and np.array_equal(f64(cache[i + 2]), ref[i + 2])


def test_append_leaves_out_what_is_out_of_range():
    H, d, page = 2, 64, 16
    cache = new_cache(6, H, page, d)
    ref = np_cache(cache)
    table = torch.tensor([[0, 1], [2, -1], [99, 3], [4, 5], [4, 5]], dtype=torch.int32)
    start = [0, 0, 0, 20, -3]
    x = torch.randn(5, H, 30, d).to(torch.bfloat16)
    assert F.fa_device_status() == F.FA_OK
    F.cache_append(x.cuda(), x.cuda(), *cache, table.cuda(), i32(start))
    assert F.fa_device_status() == F.FA_ERR_PAGE
    assert F.fa_device_status() == F.FA_OK         # read and cleared
    for i in (0, 1):
        S.cache_append(f64(x), ref[i], ref[i + 2], table.tolist(), start, None, page)
        assert np.array_equal(cache[i].cpu().numpy(), ref[i]) and np.array_equal(f64(cache[i + 2]), ref[i + 2])


READ = [  # B, H, d, page, dtype, lens, N
    (1, 1, 64, 16, "bf16", [1], 1),
    (3, 2, 128, 64, "bf16", [0, 65, 130], 131),
    (2, 3, 256, 16, "f32", [40, 17], 33),
    (2, 1, 64, 128, "f32", [128, 300], 300),
    (2, 5, 128, 32, "bf16", [7, 500], 517),
]


@pytest.mark.parametrize("any_scale", [False, True])
@pytest.mark.parametrize("c", READ, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_read(c, any_scale):
    B, H, d, page, dt, lens, N = c
    width = (max(max(lens), N) + page - 1) // page
    cache = new_cache(B * width, H, page, d)
    cache[0].random_(0, 0x7F)
    cache[1].random_(0x80, 0xFF)
    if any_scale:
        cache[2].uniform_(1e-3, 3.0)
        cache[3].uniform_(1e-3, 3.0)
    table = table_for(B, width, B * width)
    out = F.cache_read(*cache, table.cuda(), i32(lens), N, dtype=DT[dt])
    torch.cuda.synchronize()
    assert F.fa_device_status() == F.FA_OK
    ref = np_cache(cache)
    for i in (0, 1):
        want = np.zeros((B, H, N, d))
        for b in range(B):
            n = min(lens[b], N)
            want[b, :, :n] = S.cache_tokens(ref[i], ref[i + 2], table[b].tolist(), n, page)
        got = f64(out[i])
        assert out[i].dtype == DT[dt] and got.shape == want.shape
        tol = np.abs(want) * ((U32 + (U16 if dt == "bf16" else 0)) if any_scale else 0)
        assert (np.abs(got - want) <= tol).all()


def test_read_leaves_out_bad_pages():
    cache = new_cache(4, 1, 16, 64, fill=0x38)
    cache[2].fill_(1.0)
    table = torch.tensor([[0, -1, 2], [3, 1, 4]], dtype=torch.int32, device="cuda")
    k, v = F.cache_read(*cache, table, i32([48, 90]), 60)
    assert F.fa_device_status() == F.FA_ERR_PAGE
    want = torch.zeros(2, 60)
    want[0, :16] = want[0, 32:48] = want[1, :32] = 1.0
    assert torch.equal(k[:, 0, :, 0].float().cpu(), want)


# ------------------------------------------------------------------ attention
def attention_case(B, Hkv, d, page, lens, seed, any_scale=False, spread=1.0):
    """A cache of random tokens for sequences of the given lengths; every slot
    behind a length, and every page no sequence owns, holds NaN codes."""
    g = torch.Generator().manual_seed(seed)
    width = max(1, max((n + page - 1) // page for n in lens)) + 1
    total = B * width + 1
    table = table_for(B, width, total, seed)
    cache = new_cache(total, Hkv, page, d)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        x = torch.randn(2, 1, Hkv, n, d, generator=g) * torch.exp(spread * torch.randn(2, 1, Hkv, n, 1, generator=g))
        F.cache_append(x[0].cuda(), x[1].cuda(), *cache, table[b:b + 1].cuda(), i32([0]))
    if any_scale:
        cache[2].mul_(torch.rand(total, Hkv, device="cuda") + 0.5)
        cache[3].mul_(torch.rand(total, Hkv, device="cuda") + 0.5)
    return cache, table


def check_attention(q, cache, table, lens, page, causal, scale=None):
    d = q.shape[3]
    scale = d ** -0.5 if scale is None else scale
    o, lse = F.forward_cache(q.cuda(), *cache, table.cuda(), i32(lens), scale=scale, causal=causal)
    torch.cuda.synchronize()
    assert F.fa_device_status() == F.FA_OK
    compare_attention(o, lse, q, cache, table, lens, page, causal, scale)
    return o, lse


def compare_attention(o, lse, q, cache, table, lens, page, causal, scale):
    d = q.shape[3]
    ref_o, ref_l, w, amp, unit = S.cache_attention(f64(q), *np_cache(cache), table.tolist(), lens, page, scale, causal)
    o, lse = f64(o), f64(lse)
    none = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
    e_s = amp * (d * 2.0 ** -23 + 2.0 ** -20)
    tol = np.abs(ref_o) * U16 + w * (2.0 ** -11 + 2.0 ** -13 + np.expm1(np.minimum(2 * e_s[..., None], 50))) + unit * 2.0 ** -37
    bad = np.abs(o - ref_o) - tol
    at = np.unravel_index(np.nanargmax(bad), bad.shape)
    good = bool(np.isfinite(o).all() and (bad <= 0).all())
    assert good, f"O[{at}] = {o[at]:.6g}, not {ref_o[at]:.6g}: off by {bad[at]:.3g} beyond {tol[at]:.3g}"
    lse, ref_l, e_s = lse[~none], ref_l[~none], e_s[~none]
    err = np.abs(lse - ref_l) - (e_s + 2.0 ** -18 * (1 + np.abs(ref_l)))
    assert (err <= 0).all(), "L off beyond its bound"


ATTN = [  # B, Hq, Hkv, Nq, d, page, lens, causal
    (1, 1, 1, 1, 64, 16, [1], True),
    (1, 1, 1, 1, 128, 16, [0], True),
    (4, 8, 2, 1, 128, 64, [0, 1, 63, 65], True),
    (3, 4, 4, 1, 64, 16, [15, 16, 17], False),
    (2, 16, 1, 1, 128, 128, [129, 700], True),       # 16 query heads on one key/value head
    (2, 17, 1, 1, 64, 32, [31, 333], True),          # rows that do not fill a tile
    (3, 6, 2, 5, 128, 32, [3, 5, 200], True),        # lengths below the number of queries
    (2, 10, 2, 7, 256, 16, [2, 100], True),
    (1, 8, 8, 1, 256, 64, [1001], True),
    (2, 4, 1, 33, 64, 64, [33, 400], True),
    (1, 4, 2, 130, 128, 16, [500], True),
    (1, 4, 2, 130, 128, 16, [500], False),
    (1, 2, 1, 200, 256, 128, [263], True),
    (2, 8, 8, 64, 64, 32, [64, 190], False),
    (2, 3, 3, 150, 64, 64, [150, 90], True),         # a square causal block, and one shorter than its queries
    (1, 2, 2, 1, 128, 64, [20000], True),            # split over the whole GPU
    (9, 2, 1, 2, 64, 16, [0, 5000, 3, 0, 17, 900, 1, 2, 260], True),
]


@pytest.mark.parametrize("c", ATTN, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_attention(c):
    B, Hq, Hkv, Nq, d, page, lens, causal = c
    cache, table = attention_case(B, Hkv, d, page, lens, seed=Nq + d)
    q = torch.randn(B, Hq, Nq, d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    check_attention(q, cache, table, lens, page, causal)


def check_wide_table(c, more):
    """The same lengths in a block table with room for many more tokens, whose
    other entries are no pages."""
    B, Hq, Hkv, Nq, d, page, lens, causal = c
    cache, table = attention_case(B, Hkv, d, page, lens, seed=Nq + d)
    table = torch.cat([table, torch.full((B, more // page), -1, dtype=torch.int32)], dim=1)
    assert F.fa_fwd_cache_workspace_size(B, Hq, Hkv, Nq, d, page, table.shape[1]) > 0
    q = torch.randn(B, Hq, Nq, d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    check_attention(q, cache, table, lens, page, causal)


@pytest.mark.parametrize("c", ATTN, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_attention_wide_table(c):
    check_wide_table(c, 700)


MANY = [  # many tiles of 128 or 256 rows a head
    (2, 3, 1, 700, 64, 16, [700, 90], True),         # an odd group; most queries of the second see nothing
    (1, 5, 1, 301, 128, 32, [1000], True),
    (3, 8, 1, 220, 128, 64, [0, 221, 5], True),
    (1, 7, 1, 120, 256, 128, [450], True),
    (1, 6, 6, 517, 64, 64, [517], True),
    (1, 4, 1, 1100, 128, 16, [1100], False),
    (2, 64, 1, 400, 64, 32, [600, 433], True),       # 100 tiles; a warp of the merge takes several rows
    (8, 64, 2, 200, 64, 16, [900, 0, 130, 201, 1, 77, 640, 0], True),   # far more units than CTAs, some of them empty
    (3, 32, 8, 400, 256, 64, [600, 0, 250], True),
    (8, 64, 2, 200, 128, 16, [900, 0, 1, 201, 0, 64, 500, 30], False),
]


@pytest.mark.parametrize("c", MANY, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_many_tiles(c):
    test_attention(c)


@pytest.mark.parametrize("c", MANY, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_many_tiles_wide_table(c):
    check_wide_table(c, 2100)


def test_whole_units_many_and_empty():
    """Tables of few tokens, where CTAs take units from end to end: more units than
    CTAs, and sequences and queries that see nothing."""
    for c in [(40, 16, 8, 1, 64, 16, [(37 * b) % 300 if b % 3 else 0 for b in range(40)], True),
              (150, 3, 3, 1, 128, 32, [(11 * b) % 97 for b in range(150)], False),
              (9, 6, 2, 70, 128, 16, [0, 1, 69, 70, 71, 200, 5, 0, 31], True),
              (5, 2, 2, 130, 256, 64, [0, 64, 129, 1, 130], True)]:
        assert F.fa_fwd_cache_workspace_size(c[0], c[1], c[2], c[3], c[4], c[5], max(c[6]) // c[5] + 2) == 0
        test_attention(c)


@pytest.mark.parametrize("spread", [0.0, 4.0])
def test_attention_any_scales(spread):
    """Scales that are no powers of two; pages and heads of very different size."""
    for Nq in (1, 40):
        cache, table = attention_case(2, 2, 128, 16, [300, 77], 3, any_scale=True, spread=spread)
        q = torch.randn(2, 8, Nq, 128, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
        check_attention(q, cache, table, [300, 77], 16, True, scale=0.01 if spread else None)


@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** 30])
def test_attention_of_small_and_large_values(size):
    """Keys and queries far from 1 (their product is not), values too."""
    cache, table = attention_case(1, 1, 64, 16, [100], 8)
    for i, f in ((2, size), (3, size)):
        cache[i].mul_(f)
    q = (torch.randn(1, 2, 1, 64, generator=torch.Generator().manual_seed(6)) / size).to(torch.bfloat16)
    q[..., 0] = 0.0
    q[..., 1] *= 2.0 ** -20          # a row whose entries differ by a factor of a million
    check_attention(q, cache, table, [100], 16, True)


def test_attention_sharp_and_rising_scores():
    """Each later key scores higher, so the running maximum moves at every step."""
    for Nq in (1, 48):
        cache, table = attention_case(1, 1, 128, 64, [900], 4, spread=0.0)
        x = torch.zeros(1, 1, 900, 128)
        x[0, 0, :, 0] = torch.linspace(0, 440, 900)
        v = torch.randn(1, 1, 900, 128, generator=torch.Generator().manual_seed(2))
        F.cache_append(x.cuda(), v.cuda(), *cache, table.cuda(), i32([0]))
        q = torch.zeros(1, 4, Nq, 128)
        q[..., 0] = torch.tensor([1.0, -1.0, 8.0, -30.0])[None, :, None]
        check_attention(q.to(torch.bfloat16), cache, table, [900], 64, True, scale=0.25)


def test_attention_zero_queries_and_zero_pages():
    """Rows of q that are zero see every key alike; a head whose K or V is zero
    (whose pages then have the least scale there is) beside hidden tokens."""
    for Nq in (1, 5, 40):
        cache, table = attention_case(1, 3, 64, 16, [90], 14)
        x = torch.randn(1, 3, 90, 64, generator=torch.Generator().manual_seed(3))
        k, v = x.clone(), x.flip(2).contiguous()
        k[:, 0], v[:, 1], v[:, 2, 32:64] = 0, 0, 0
        F.cache_append(k.cuda(), v.cuda(), *cache, table.cuda(), i32([0]))
        assert float(cache[2][int(table[0, 0]), 0]) == S.SCALE_MIN
        q = torch.randn(1, 6, Nq, 64, generator=torch.Generator().manual_seed(7))
        q[:, ::2] = 0
        check_attention(q.to(torch.bfloat16), cache, table, [90], 16, True)


@pytest.mark.parametrize("Nq", [1, 30])
def test_attention_one_long_sequence_among_many(Nq):
    """More sequences than lanes; nearly all of the work in one of them, so that
    its units are cut into many pieces while the others have one or none."""
    B = 70
    lens = [[0, 1, 5, 17, 40][b % 5] for b in range(B)]
    lens[41] = 9000
    cache, table = attention_case(B, 1, 64, 64, lens, 15)
    q = torch.randn(B, 2, Nq, 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    check_attention(q, cache, table, lens, 64, True)


def test_cache_beyond_four_gigabytes():
    """Pages whose codes lie past 2^32 bytes: append, attention of few and of
    many rows, read."""
    H, page, d = 8, 128, 256
    num_pages = 2 ** 32 // (H * page * d) + 6
    if torch.cuda.mem_get_info()[0] < 4 * num_pages * H * page * d:
        pytest.skip("not enough device memory")
    cache = [torch.empty(num_pages, H, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones(num_pages, H, device="cuda") for _ in range(2)]
    table = torch.tensor([[num_pages - 1, 0, num_pages - 3]], dtype=torch.int32)
    g = torch.Generator().manual_seed(16)
    x = torch.randn(2, 1, H, 300, d, generator=g)
    F.cache_append(x[0].cuda(), x[1].cuda(), *cache, table.cuda(), i32([0]))
    small = [c[table[0].long()].contiguous() for c in cache]     # the three pages alone
    ref = np_cache(new_cache(3, H, page, d))
    for i in (0, 1):
        S.cache_append(f64(x[i]), ref[i], ref[i + 2], [[0, 1, 2]], [0], None, page)
        assert np.array_equal(f64(small[i + 2]), ref[i + 2])
        for p in range(3):
            n = min(page, 300 - page * p)
            assert np.array_equal(small[i][p, :, :n].cpu().numpy(), ref[i][p, :, :n])
    first = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    for Nq in (1, 100):
        q = torch.randn(1, H, Nq, d, generator=g).to(torch.bfloat16).cuda()
        a = F.forward_cache(q, *cache, table.cuda(), i32([300]))
        b = F.forward_cache(q, *small, first, i32([300]))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = F.cache_read(*cache, table.cuda(), i32([300]), 300), F.cache_read(*small, first, i32([300]), 300)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert F.fa_device_status() == F.FA_OK


def test_attention_shared_and_repeated_pages():
    """Two sequences that share a prefix's pages, and one whose table names a page twice."""
    cache, table = attention_case(3, 2, 64, 16, [80, 80, 80], 9)
    table[1, :3] = table[0, :3]
    table[2, 1] = table[2, 0]
    q = torch.randn(3, 4, 3, 64, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    check_attention(q, cache, table, [80, 71, 60], 16, True)


@pytest.mark.parametrize("Nq", [1, 50])
def test_attention_leaves_out_what_is_out_of_range(Nq):
    cache, table = attention_case(4, 1, 128, 16, [100, 100, 100, 100], 10)
    table[0, 2], table[1, 0] = -1, 10 ** 6
    lens = [100, 100, -7, 10 ** 6]
    q = torch.randn(4, 2, Nq, 128, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    table[3, 6:] = table[3, 0]       # the eighth page of its table exists: length is cut at the table's end
    o, lse = F.forward_cache(q.cuda(), *cache, table.cuda(), i32(lens))
    assert F.fa_device_status() == F.FA_ERR_PAGE
    cut = [100, 100, 0, table.shape[1] * 16]
    compare_attention(o, lse, q, cache, table, cut, 16, True, 128 ** -0.5)


@pytest.mark.parametrize("Nq", [1, 60])
@pytest.mark.parametrize("page_number", [-2 ** 31, 2 ** 31 - 1, 5])
def test_attention_reports_each_page_that_is_none(Nq, page_number):
    """Whatever the number outside [0, num_pages), alone in its table, line or whole units."""
    for more in (0, 60):
        cache, table = attention_case(1, 1, 64, 16, [60], 10)
        assert len(cache[0]) == 6
        table[0, 2] = page_number
        table = torch.cat([table, torch.full((1, more), -1, dtype=torch.int32)], dim=1)
        q = torch.randn(1, 2, Nq, 64, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
        o, lse = F.forward_cache(q.cuda(), *cache, table.cuda(), i32([60]))
        assert F.fa_device_status() == (F.FA_ERR_PAGE if page_number != 5 else F.FA_OK)
        if page_number != 5:
            compare_attention(o, lse, q, cache, table, [60], 16, True, 64 ** -0.5)


@pytest.mark.parametrize("Nq", [1, 12, 40])
def test_attention_nan_reaches_only_the_rows_that_see_it(Nq):
    """A NaN code of V in token t makes column c of the rows that see t NaN and no other value."""
    cache, table = attention_case(1, 1, 128, 32, [200], 12)
    t, col = 190, 5
    ref = F.forward_cache(torch.ones(1, 2, Nq, 128, device="cuda", dtype=torch.bfloat16), *cache, table.cuda(), i32([200]))
    cache[1][int(table[0, t // 32]), 0, t % 32, col] = 0x7F
    o, lse = F.forward_cache(torch.ones(1, 2, Nq, 128, device="cuda", dtype=torch.bfloat16), *cache, table.cuda(), i32([200]))
    torch.cuda.synchronize()
    sees = torch.arange(Nq) + 200 - Nq >= t
    want = torch.zeros(1, 2, Nq, 128, dtype=torch.bool)
    want[:, :, sees, col] = True
    assert torch.equal(torch.isnan(o).cpu(), want)
    assert torch.equal(lse, ref[1])
    assert torch.equal(o.cpu()[~want], ref[0].cpu()[~want])


# ------------------------------------------------------------------ together
def test_serving_run_together_eager_and_captured():
    """A prompt in two chunks, then decode steps: rope, append, attention, as
    a server calls them; the decode step is captured once and replayed.  Each
    attention is checked against the oracle on the cache as it then is, and the
    cache against the oracle's own."""
    B, Hq, Hkv, d, page, steps = 2, 8, 2, 128, 16, 6
    prompt, width = [37, 21], 6
    g = torch.Generator().manual_seed(21)
    freqs, ms = F.rope_freqs(d, scaling="ntk", factor=2.0)
    table = table_for(B, width, B * width)
    t_dev = table.cuda()
    cache = new_cache(B * width, Hkv, page, d)
    ref = np_cache(cache)

    def draw(T):
        return [torch.randn(B, H, T, d, generator=g).to(torch.bfloat16).cuda() for H in (Hq, Hkv, Hkv)]

    def follow(k, v, start, count):
        for x, i in ((k, 0), (v, 1)):
            S.cache_append(f64(x), ref[i], ref[i + 2], table.tolist(), start, count, page)
            assert np.array_equal(cache[i].cpu().numpy(), ref[i]) and np.array_equal(f64(cache[i + 2]), ref[i + 2])

    done = [0, 0]
    for T in (16, 21):                      # chunks of the prompt, padded to the longest
        count = [max(0, min(T, p - n)) for p, n in zip(prompt, done)]
        q, k, v = draw(T)
        pos = i32([[n + t for t in range(T)] for n in done])
        q, k = F.rope(q, k, pos, freqs, ms)
        F.cache_append(k, v, *cache, t_dev, i32(done), i32(count))
        torch.cuda.synchronize()
        follow(k, v, done, count)
        done = [n + c for n, c in zip(done, count)]
        o, lse = F.forward_cache(q, *cache, t_dev, i32(done))
        compare_attention(o, lse, q, cache, table, done, page, True, d ** -0.5)

    # the decode step: fixed buffers, captured once
    q, k, v = draw(1)
    pos, lens = i32([[n] for n in done]), i32([n + 1 for n in done])

    def step():
        F.rope(q, k, pos, freqs, ms, out=(q, k))
        F.cache_append(k, v, *cache, t_dev, pos[:, 0].contiguous())
        out = F.forward_cache(q, *cache, t_dev, lens)
        lens.add_(1)
        pos.add_(1)
        return out

    side = torch.cuda.Stream()
    saved = [t.clone() for t in (*cache, q, k, v, pos, lens)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):           # warm-up on another stream, then undone
        step()
        for t, s in zip((*cache, q, k, v, pos, lens), saved):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for _ in range(steps):
        for t, s in zip((q, k, v), draw(1)):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert F.fa_device_status() == F.FA_OK
        follow(k, v, done, None)            # k as rope left it
        done = [n + 1 for n in done]
        compare_attention(o, lse, q, cache, table, done, page, True, d ** -0.5)


def test_read_back_equals_attention_through_the_dense_forward():
    """cache_read feeds the split-KV forward: both paths agree to bfloat16."""
    cache, table = attention_case(1, 2, 128, 64, [1000], 13, spread=0.0)
    q = torch.randn(1, 4, 96, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    k, v = F.cache_read(*cache, table.cuda(), i32([1000]), 1000)
    o1, l1 = F.forward_splitkv(q, k, v, causal=True)
    o2, l2 = F.forward_cache(q, *cache, table.cuda(), i32([1000]))
    torch.cuda.synchronize()
    # O: two bfloat16 roundings, P rounded to bfloat16 on one side, terms of size |v| <= 5
    assert float((o1.float() - o2.float()).abs().max()) <= 2 * U16 * float(o1.float().abs().max()) + 5 * U16
    assert float((l1 - l2).abs().max()) <= 1e-3


def test_calls_on_two_streams_do_not_meet():
    """The wrapper's own workspaces: two calls in flight on two streams give what each gives alone."""
    cases = [attention_case(2, 2, 128, 64, [3000, 2500], s) for s in (1, 2)]
    qs = [torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).cuda() for s in (1, 2)]
    tabs = [t.cuda() for _, t in cases]
    lens = i32([3000, 2500])
    alone = [F.forward_cache(q, *c, t, lens) for q, (c, _), t in zip(qs, cases, tabs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(F.forward_cache(qs[i], *cases[i][0], tabs[i], lens))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(lse, alone[i][1])
