"""Host-side checks of the serving entry points that need no GPU: argument
errors of the C ABI and of the Python wrappers, the host-side frequency table."""
import ctypes

import numpy as np
import pytest
import torch

import exact_io_aware_50_b200 as F
from oracle import serving as S
from test_abi import FAKE, _FakeCuda


@pytest.mark.parametrize("fn", ["fa_rope", "fa_rope_f32", "fa_rope_bwd", "fa_rope_bwd_f32"])
def test_rope_argument_errors(fn):
    f = getattr(F, fn)

    def call(ptrs=(FAKE,) * 6, B=2, Hq=4, Hkv=2, N=8, d=64, rot=32, mscale=1.0):
        return f(*ptrs, B, Hq, Hkv, N, d, rot, 1, 0, mscale)

    for i in (0, 2, 4, 5):
        assert call(ptrs=tuple(0 if j == i else FAKE for j in range(6))) == F.FA_ERR_INVALID_ARG
    # k and k_out come together
    assert call(ptrs=(FAKE, 0, FAKE, FAKE, FAKE, FAKE)) == F.FA_ERR_INVALID_ARG
    assert call(ptrs=(FAKE, FAKE, FAKE, 0, FAKE, FAKE)) == F.FA_ERR_INVALID_ARG
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(N=-1), dict(d=0), dict(rot=0), dict(mscale=0.0),
               dict(mscale=float("nan")), dict(mscale=float("inf")), dict(mscale=-1.0)):
        assert call(**kw) == F.FA_ERR_INVALID_ARG, kw
    for kw in (dict(d=260), dict(d=66), dict(rot=72), dict(rot=12), dict(Hq=70000), dict(N=2**31 - 1, B=4)):
        assert call(**kw) == F.FA_ERR_UNSUPPORTED, kw
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 8), (4, 2), (5, 4)):
        assert call(ptrs=tuple(FAKE + off if j == i else FAKE for j in range(6))) == F.FA_ERR_ALIGNMENT


def test_rope_freqs_on_the_host():
    def call(rot=32, theta=10000.0, kind=0, factor=4.0, orig=4096, fast=32.0, slow=1.0, n=128):
        t, m = (ctypes.c_double * n)(), ctypes.c_float(-1)
        st = F.fa_rope_freqs(ctypes.addressof(t), ctypes.addressof(m), rot, theta, kind, factor, orig, fast, slow)
        return st, np.array(t[:rot // 2]), m.value

    for kind, name in enumerate(("none", "linear", "ntk", "yarn")):
        for rot in (8, 64, 128, 256):
            st, f, m = call(rot=rot, kind=kind)
            ref, mr = S.rope_freqs(rot, kind=name, factor=4.0)
            assert st == F.FA_OK and np.allclose(f, ref, rtol=1e-13, atol=0) and abs(m - mr) < 1e-6
    assert F.fa_rope_freqs(0, 0, 32, 1e4, 0, 1.0, 1, 2.0, 1.0) == F.FA_ERR_INVALID_ARG
    nan, inf = float("nan"), float("inf")
    for kw in (dict(rot=0), dict(theta=0.0), dict(theta=nan), dict(theta=inf), dict(kind=4), dict(kind=-1),
               dict(kind=1, factor=0.5), dict(kind=2, factor=nan), dict(kind=3, orig=0), dict(kind=3, fast=1.0),
               dict(kind=3, slow=nan), dict(kind=3, fast=inf)):
        assert call(**kw)[0] == F.FA_ERR_INVALID_ARG, kw
    assert call(rot=12)[0] == F.FA_ERR_UNSUPPORTED
    assert call(rot=264, n=256)[0] == F.FA_ERR_UNSUPPORTED
    f, m = F.rope_freqs(64, scaling="yarn", factor=8.0, device="cpu")
    ref, mr = S.rope_freqs(64, kind="yarn", factor=8.0)
    assert f.dtype == torch.float64 and np.allclose(f.numpy(), ref, rtol=1e-13) and abs(m - mr) < 1e-6
    with pytest.raises(ValueError, match="scaling"):
        F.rope_freqs(64, scaling="dynamic")
    with pytest.raises(F.FaError):
        F.rope_freqs(20, device="cpu")


SIZES = dict(B=2, Hkv=2, T=8, d=64, page=16, num_pages=9, max_pages=4)


def _size_errors(call):
    for kw in ([{k: 0} for k in SIZES] + [{k: -1} for k in SIZES]):
        assert call(**kw) == F.FA_ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(d=32), dict(d=512), dict(page=8), dict(page=24), dict(page=256),
               dict(max_pages=2**28), dict(T=2**28 + 1), dict(B=2**20, Hkv=2**10), dict(num_pages=2**31 - 1)):
        assert call(**kw) == F.FA_ERR_UNSUPPORTED, kw


@pytest.mark.parametrize("fn", ["fa_cache_append", "fa_cache_append_f32"])
def test_append_argument_errors(fn):
    def call(ptrs=(FAKE,) * 9, **kw):
        a = {**SIZES, **kw}
        return getattr(F, fn)(*ptrs, a["B"], a["Hkv"], a["T"], a["d"], a["page"], a["num_pages"], a["max_pages"])

    for i in range(8):   # the ninth, count, may be null
        assert call(ptrs=tuple(0 if j == i else FAKE for j in range(9))) == F.FA_ERR_INVALID_ARG
    _size_errors(call)
    assert call(B=256, Hkv=257) == F.FA_ERR_UNSUPPORTED
    for i in range(9):
        off = 8 if i < 4 else 2
        assert call(ptrs=tuple(FAKE + off if j == i else FAKE for j in range(9))) == F.FA_ERR_ALIGNMENT


@pytest.mark.parametrize("fn", ["fa_cache_read", "fa_cache_read_f32"])
def test_read_argument_errors(fn):
    def call(ptrs=(FAKE,) * 8, **kw):
        a = {**SIZES, **kw}
        return getattr(F, fn)(*ptrs, a["B"], a["Hkv"], a["T"], a["d"], a["page"], a["num_pages"], a["max_pages"])

    for i in range(8):
        assert call(ptrs=tuple(0 if j == i else FAKE for j in range(8))) == F.FA_ERR_INVALID_ARG
    _size_errors(call)
    assert call(B=256, Hkv=257) == F.FA_ERR_UNSUPPORTED
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 2), (4, 2), (5, 2), (6, 8), (7, 8)):
        assert call(ptrs=tuple(FAKE + off if j == i else FAKE for j in range(8))) == F.FA_ERR_ALIGNMENT


def test_forward_cache_argument_errors():
    def call(ptrs=(FAKE,) * 10, Hq=4, scale=0.125, **kw):
        a = {**SIZES, **kw}
        return F.fa_fwd_cache(*ptrs, a["B"], Hq, a["Hkv"], a["T"], a["d"], a["page"], a["num_pages"],
                              a["max_pages"], scale, 1)

    for i in range(9):
        assert call(ptrs=tuple(0 if j == i else FAKE for j in range(10))) == F.FA_ERR_INVALID_ARG
    _size_errors(call)
    # more pieces of work than int32 counts, were every sequence to fill its table
    assert call(B=1024, Hkv=1024, Hq=1024, max_pages=2**20) == F.FA_ERR_UNSUPPORTED
    for kw in (dict(Hq=3), dict(Hq=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == F.FA_ERR_INVALID_ARG, kw
    for i in range(9):
        off = 8 if i in (0, 1, 2, 7) else 2
        assert call(ptrs=tuple(FAKE + off if j == i else FAKE for j in range(10))) == F.FA_ERR_ALIGNMENT
    assert F.fa_fwd_cache_workspace_size(2, 4, 2, 8, 64, 64, 9) > 0
    assert call(ptrs=(FAKE,) * 9 + (0,), max_pages=99) == F.FA_ERR_INVALID_ARG
    assert call(ptrs=(FAKE,) * 9 + (FAKE + 64,), max_pages=99) == F.FA_ERR_ALIGNMENT
    for bad in ((0, 4, 2, 8, 64, 64, 9), (1, 4, 3, 8, 64, 64, 9), (1, 4, 2, 8, 96, 64, 9), (1, 4, 2, 8, 64, 24, 9),
                (1, 4, 2, 8, 64, 64, 0), (1, 0, 2, 8, 64, 64, 9)):
        assert F.fa_fwd_cache_workspace_size(*bad) == 0


def _cache(idx=0, H=2, d=64, pages=9, page=16, B=2):
    def t(shape, dtype):
        return _FakeCuda(shape, dtype, idx)
    return [t((pages, H, page, d), torch.uint8), t((pages, H, page, d), torch.uint8),
            t((pages, H), torch.float32), t((pages, H), torch.float32), t((B, 4), torch.int32)]


def test_wrappers_reject_bad_tensors():
    bf, i32 = torch.bfloat16, torch.int32

    def t(shape, dtype=bf, idx=0):
        return _FakeCuda(shape, dtype, idx)

    q, k = t((2, 4, 8, 64)), t((2, 2, 8, 64))
    pos, fr = t((2, 8), i32), t((16,), torch.float64)
    for args, match in (((t((2, 4, 64)), k, pos, fr), "q must be"), ((t((2, 4, 8, 64), torch.half), k, pos, fr), "q must be"),
                        ((q, t((2, 2, 9, 64)), pos, fr), "k must be"), ((q, t((2, 2, 8, 64), torch.float32), pos, fr), "k must be"),
                        ((q, k, t((2, 8), torch.int64), fr), "positions"), ((q, k, t((8, 2), i32), fr), "positions"),
                        ((q, k, t((9,), i32), fr), "positions"), ((q, k, pos, t((16,), torch.float32)), "freqs"),
                        ((q, t((2, 2, 8, 64), idx=1), pos, fr), "q's device"), ((q, k, pos, t((16,), torch.float64, 1)), "q's device")):
        for fn in (F.rope, F.rope_backward):
            with pytest.raises(ValueError, match=match):
                fn(*args, out=(q, k))
    with pytest.raises(ValueError, match="out must be"):
        F.rope(q, k, pos, fr, out=(q, None))
    with pytest.raises(ValueError, match="out must be"):
        F.rope(q, k, pos, fr, out=(q, q))

    start = t((2,), i32)
    for args, match in (((t((2, 2, 8)), k), "k and v must"), ((k, t((2, 2, 9, 64))), "k and v must"),
                        ((t((2, 2, 8, 64), torch.half),) * 2, "k and v must"),
                        ((t((2, 3, 8, 64)),) * 2, "E4M3"), ((t((2, 2, 8, 128)),) * 2, "E4M3")):
        with pytest.raises(ValueError, match=match):
            F.cache_append(*args, *_cache(), start)
    for at, bad, match in ((0, t((9, 2, 16, 64), bf), "E4M3"), (1, t((8, 2, 16, 64), torch.uint8), "E4M3"),
                           (2, t((9, 3), torch.float32), "k_scale"), (3, t((9, 2), torch.float64), "k_scale"),
                           (4, t((3, 4), i32), "block_table"), (4, t((2, 4), torch.int64), "block_table"),
                           (0, t((9, 2, 16, 64), torch.uint8, 1), "q's device"), (4, t((2, 4), i32, 1), "q's device")):
        c = _cache()
        c[at] = bad
        with pytest.raises(ValueError, match=match):
            F.cache_append(k, k, *c, start)
        with pytest.raises(ValueError, match=match):
            F.forward_cache(q, *c, start)
        if at:
            with pytest.raises(ValueError):
                F.cache_read(*c, start, 8)
    for bad in (t((3,), i32), t((2,), torch.int64), t((2, 1), i32)):
        for call in (lambda: F.cache_append(k, k, *_cache(), bad), lambda: F.cache_append(k, k, *_cache(), start, bad),
                     lambda: F.forward_cache(q, *_cache(), bad), lambda: F.cache_read(*_cache(), bad, 8)):
            with pytest.raises(ValueError, match=r"int32 \[B\]"):
                call()
    for call in (lambda: F.cache_append(k, k, *_cache(), None), lambda: F.forward_cache(q, *_cache(), None),
                 lambda: F.cache_read(*_cache(), None, 8), lambda: F.cache_read(*_cache(), start, 8, dtype=torch.half),
                 lambda: F.forward_cache(t((2, 4, 8, 64), torch.float32), *_cache(), start),
                 lambda: F.forward_cache(q, *_cache(), start, workspace=t((1 << 30,), torch.uint8, 1))):
        with pytest.raises(ValueError):
            call()


def test_strerror_covers_the_page_error():
    assert "page" in F.fa_strerror(F.FA_ERR_PAGE)
