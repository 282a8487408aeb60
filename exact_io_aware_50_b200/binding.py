"""ctypes binding of libfa.so -- argument marshalling only.

The ``fa_*`` functions mirror the C ABI one to one (raw device pointers as
ints, sizes, a CUDA stream handle) and return the status code.  ``forward``
and ``backward`` take torch CUDA tensors, allocate outputs/workspace with
torch (device memory only), pass pointers and torch's current stream, and
raise ``FaError`` on a non-zero status.  Every step of the computation runs in
the library's CUDA kernels; there is no other code path.
"""
from __future__ import annotations

import ctypes
import functools
import os

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_ALIGNMENT = 3
FA_ERR_ARCH = 4
FA_ERR_CUDA = 5
FA_ERR_TIMEOUT = 6
FA_ERR_PAGE = 7

FA_ROPE_KINDS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libfa.so")
_lib = None
# torch and what the serving operators' wrappers use of it, once one has run
_torch = _F32 = _BF16 = _I32 = _F8 = _get_device = _get_stream = None

EXPORTS = ("fa_fwd", "fa_fwd_pair", "fa_fwd_fp8", "fa_fwd_dropout", "fa_bwd_dropout", "fa_fwd_splitkv",
           "fa_fwd_splitkv_num_splits",
           "fa_fwd_splitkv_workspace_size", "fa_bwd", "fa_bwd_workspace_size", "fa_bwd_prep",
           "fa_bwd_dkdv",
           "fa_bwd_dq", "fa_fwd_f32", "fa_bwd_f32", "fa_device_status", "fa_wait_selftest",
           "fa_rope", "fa_rope_f32", "fa_rope_bwd", "fa_rope_bwd_f32", "fa_rope_freqs",
           "fa_cache_append", "fa_cache_append_f32", "fa_cache_read", "fa_cache_read_f32",
           "fa_fwd_cache", "fa_fwd_cache_workspace_size", "fa_strerror")


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({fa_strerror(status)})")


def lib():
    """Load libfa.so (once).  Raises if the built library is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is missing: build it with "
                               "`python -m exact_io_aware_50_b200.build`")
        L = ctypes.CDLL(lib_path)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        dims = [I, I, I, I, I, I, F, I, P]
        L.fa_fwd.argtypes = [P] * 5 + dims
        L.fa_fwd.restype = I
        L.fa_fwd_pair.argtypes = [P] * 5 + dims
        L.fa_fwd_pair.restype = I
        L.fa_fwd_f32.argtypes = [P] * 5 + dims
        L.fa_fwd_f32.restype = I
        U64 = ctypes.c_ulonglong
        L.fa_fwd_fp8.argtypes = [P] * 5 + [I, I, I, I, I, F, F, F, F, I, P]
        L.fa_fwd_fp8.restype = I
        L.fa_fwd_dropout.argtypes = [P] * 5 + [I, I, I, I, I, I, F, I, F, U64, U64, P]
        L.fa_fwd_dropout.restype = I
        L.fa_bwd_dropout.argtypes = [P] * 10 + [I, I, I, I, I, I, F, I, F, U64, U64, P]
        L.fa_bwd_dropout.restype = I
        L.fa_fwd_splitkv.argtypes = [P] * 6 + [I, I, I, I, I, I, F, I, I, P]
        L.fa_fwd_splitkv.restype = I
        L.fa_fwd_splitkv_num_splits.argtypes = [I] * 5
        L.fa_fwd_splitkv_num_splits.restype = I
        L.fa_fwd_splitkv_workspace_size.argtypes = [I] * 5
        L.fa_fwd_splitkv_workspace_size.restype = S
        L.fa_bwd.argtypes = [P] * 10 + dims
        L.fa_bwd.restype = I
        L.fa_bwd_f32.argtypes = [P] * 10 + dims
        L.fa_bwd_f32.restype = I
        L.fa_bwd_prep.argtypes = [P] * 6 + [I, I, I, I, I, I, F, P]
        L.fa_bwd_prep.restype = I
        L.fa_bwd_dkdv.argtypes = [P] * 7 + dims
        L.fa_bwd_dkdv.restype = I
        L.fa_bwd_dq.argtypes = [P, P, I, I, I, I, F, P]
        L.fa_bwd_dq.restype = I
        L.fa_bwd_workspace_size.argtypes = [I, I, I, I]
        L.fa_bwd_workspace_size.restype = S
        D = ctypes.c_double
        for fn in (L.fa_rope, L.fa_rope_f32, L.fa_rope_bwd, L.fa_rope_bwd_f32):
            fn.argtypes = [P] * 6 + [I] * 8 + [F, P]
            fn.restype = I
        L.fa_rope_freqs.argtypes = [P, P, I, D, I, D, I, D, D]
        L.fa_rope_freqs.restype = I
        for fn in (L.fa_cache_append, L.fa_cache_append_f32):
            fn.argtypes = [P] * 9 + [I] * 7 + [P]
            fn.restype = I
        for fn in (L.fa_cache_read, L.fa_cache_read_f32):
            fn.argtypes = [P] * 8 + [I] * 7 + [P]
            fn.restype = I
        L.fa_fwd_cache.argtypes = [P] * 10 + [I] * 8 + [F, I, P]
        L.fa_fwd_cache.restype = I
        L.fa_fwd_cache_workspace_size.argtypes = [I] * 7
        L.fa_fwd_cache_workspace_size.restype = S
        L.fa_device_status.argtypes = [P]
        L.fa_device_status.restype = I
        L.fa_wait_selftest.argtypes = [ctypes.c_longlong, P]
        L.fa_wait_selftest.restype = I
        L.fa_strerror.argtypes = [I]
        L.fa_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


# ----------------------------------------------------------------- raw ABI
def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=0):
    return lib().fa_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, int(causal), stream)


def fa_fwd_pair(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=0):
    return lib().fa_fwd_pair(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, int(causal), stream)


def fa_fwd_fp8(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, descale_q, descale_k, descale_v, causal,
               stream=0):
    return lib().fa_fwd_fp8(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, float(descale_q),
                            float(descale_k), float(descale_v), int(causal), stream)


def fa_fwd_dropout(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, p_drop, seed, offset,
                   stream=0):
    return lib().fa_fwd_dropout(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, int(causal),
                                float(p_drop), int(seed), int(offset), stream)


def fa_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d, scale, causal,
                   p_drop, seed, offset, stream=0):
    return lib().fa_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d,
                                scale, int(causal), float(p_drop), int(seed), int(offset), stream)


def fa_fwd_splitkv(q, k, v, o, lse, ws, B, Hq, Hkv, Nq, Nk, d, scale, causal, num_splits,
                   stream=0):
    return lib().fa_fwd_splitkv(q, k, v, o, lse, ws, B, Hq, Hkv, Nq, Nk, d, scale, int(causal),
                                int(num_splits), stream)


def fa_fwd_splitkv_num_splits(B, Hq, Nq, Nk, d):
    return int(lib().fa_fwd_splitkv_num_splits(B, Hq, Nq, Nk, d))


def fa_fwd_splitkv_workspace_size(B, Hq, Nq, d, num_splits):
    return int(lib().fa_fwd_splitkv_workspace_size(B, Hq, Nq, d, num_splits))


def fa_fwd_f32(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=0):
    return lib().fa_fwd_f32(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, int(causal), stream)


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=0):
    return lib().fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d, scale,
                        int(causal), stream)


def fa_bwd_f32(q, k, v, o, lse, dout, dq, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d, scale, causal,
               stream=0):
    return lib().fa_bwd_f32(q, k, v, o, lse, dout, dq, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d, scale,
                            int(causal), stream)


def fa_bwd_prep(q, k, o, lse, dout, ws, B, Hq, Hkv, Nq, Nk, d, scale, stream=0):
    return lib().fa_bwd_prep(q, k, o, lse, dout, ws, B, Hq, Hkv, Nq, Nk, d, scale, stream)


def fa_bwd_dkdv(q, k, v, dout, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=0):
    return lib().fa_bwd_dkdv(q, k, v, dout, dk, dv, ws, B, Hq, Hkv, Nq, Nk, d, scale,
                             int(causal), stream)


def fa_bwd_dq(ws, dq, B, Hq, Nq, d, scale, stream=0):
    return lib().fa_bwd_dq(ws, dq, B, Hq, Nq, d, scale, stream)


def fa_bwd_workspace_size(B, Hq, Nq, d):
    return int(lib().fa_bwd_workspace_size(B, Hq, Nq, d))


def fa_rope(q, k, q_out, k_out, positions, freqs, B, Hq, Hkv, N, d, rot_dim, pos_per_batch,
            interleaved, mscale, stream=0):
    return lib().fa_rope(q, k, q_out, k_out, positions, freqs, B, Hq, Hkv, N, d, rot_dim,
                         int(pos_per_batch), int(interleaved), mscale, stream)


def fa_rope_f32(q, k, q_out, k_out, positions, freqs, B, Hq, Hkv, N, d, rot_dim, pos_per_batch,
                interleaved, mscale, stream=0):
    return lib().fa_rope_f32(q, k, q_out, k_out, positions, freqs, B, Hq, Hkv, N, d, rot_dim,
                             int(pos_per_batch), int(interleaved), mscale, stream)


def fa_rope_bwd(dq_out, dk_out, dq, dk, positions, freqs, B, Hq, Hkv, N, d, rot_dim,
                pos_per_batch, interleaved, mscale, stream=0):
    return lib().fa_rope_bwd(dq_out, dk_out, dq, dk, positions, freqs, B, Hq, Hkv, N, d, rot_dim,
                             int(pos_per_batch), int(interleaved), mscale, stream)


def fa_rope_bwd_f32(dq_out, dk_out, dq, dk, positions, freqs, B, Hq, Hkv, N, d, rot_dim,
                    pos_per_batch, interleaved, mscale, stream=0):
    return lib().fa_rope_bwd_f32(dq_out, dk_out, dq, dk, positions, freqs, B, Hq, Hkv, N, d,
                                 rot_dim, int(pos_per_batch), int(interleaved), mscale, stream)


def fa_rope_freqs(freqs, mscale, rot_dim, theta, kind, factor, original_len, beta_fast, beta_slow):
    return lib().fa_rope_freqs(freqs, mscale, rot_dim, theta, kind, factor, original_len,
                               beta_fast, beta_slow)


def fa_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, start, count, B, Hkv, T,
                    d, page, num_pages, max_pages, stream=0):
    return lib().fa_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, start,
                                 count, B, Hkv, T, d, page, num_pages, max_pages, stream)


def fa_cache_append_f32(k, v, k_cache, v_cache, k_scale, v_scale, block_table, start, count, B,
                        Hkv, T, d, page, num_pages, max_pages, stream=0):
    return lib().fa_cache_append_f32(k, v, k_cache, v_cache, k_scale, v_scale, block_table, start,
                                     count, B, Hkv, T, d, page, num_pages, max_pages, stream)


def fa_cache_read(k_cache, v_cache, k_scale, v_scale, block_table, lens, k, v, B, Hkv, N, d, page,
                  num_pages, max_pages, stream=0):
    return lib().fa_cache_read(k_cache, v_cache, k_scale, v_scale, block_table, lens, k, v, B, Hkv,
                               N, d, page, num_pages, max_pages, stream)


def fa_cache_read_f32(k_cache, v_cache, k_scale, v_scale, block_table, lens, k, v, B, Hkv, N, d,
                      page, num_pages, max_pages, stream=0):
    return lib().fa_cache_read_f32(k_cache, v_cache, k_scale, v_scale, block_table, lens, k, v, B,
                                   Hkv, N, d, page, num_pages, max_pages, stream)


def fa_fwd_cache_workspace_size(B, Hq, Hkv, Nq, d, page, max_pages):
    return int(lib().fa_fwd_cache_workspace_size(B, Hq, Hkv, Nq, d, page, max_pages))


def fa_fwd_cache(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, o, lse, ws, B, Hq, Hkv,
                 Nq, d, page, num_pages, max_pages, scale, causal, stream=0):
    return lib().fa_fwd_cache(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, o, lse, ws,
                              B, Hq, Hkv, Nq, d, page, num_pages, max_pages, scale, int(causal),
                              stream)


def fa_device_status(stream=0):
    return lib().fa_device_status(stream)


def fa_wait_selftest(timeout_ns, stream=0):
    return lib().fa_wait_selftest(int(timeout_ns), stream)


def fa_strerror(status):
    try:
        return lib().fa_strerror(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


# ----------------------------------------------------------- torch helpers
def _check(status, where):
    if status != FA_OK:
        raise FaError(status, where)


# Argument checks of the wrappers: shapes and dtypes first, then device and
# layout; each raises ValueError before the library is called.
def _check_qkv(where, q, k, v, dtypes):
    """q [B, Hq, Nq, d]; k, v [B, Hkv, Nk, d]; one dtype among `dtypes`."""
    if q.dim() != 4 or k.dim() != 4 or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"{where}: q must be [B, Hq, Nq, d] and k, v both [B, Hkv, Nk, d]")
    if q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError(f"{where}: q and k disagree on B or d")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in dtypes:
        raise ValueError(f"{where}: q, k, v must share one dtype among {tuple(map(str, dtypes))}")


def _check_bwd_in(where, q, o, lse, dout):
    """o and dout shaped and typed like q; lse float32 [B, Hq, Nq]."""
    import torch
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError(f"{where}: o and dout must have q's shape")
    if o.dtype != q.dtype or dout.dtype != q.dtype:
        raise ValueError(f"{where}: o and dout must have q's dtype")
    if tuple(lse.shape) != tuple(q.shape[:3]) or lse.dtype != torch.float32:
        raise ValueError(f"{where}: lse must be float32 [B, Hq, Nq]")


def _check_cuda(where, q, *others):
    """q and every other tensor: contiguous, on CUDA, and on q's device.  The
    library launches on the current device, which the wrappers set to q's
    (``_on``), so a tensor on another GPU would be read by kernels running on
    the wrong one."""
    for t in (q,) + others:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{where}: inputs must be contiguous CUDA tensors")
        if t.device != q.device:
            raise ValueError(f"{where}: every tensor must be on q's device ({q.device}); "
                             f"got one on {t.device}")


def _on(q):
    """Context that makes q's device current for one library call."""
    import torch
    return torch.cuda.device(q.device)


def _workspace(where, workspace, B, Hq, Nq, d, device):
    """The caller's backward workspace, checked against fa_bwd_workspace_size
    (the C entry points take a bare pointer and cannot), or a new one."""
    import torch
    need = fa_bwd_workspace_size(B, Hq, Nq, d)
    if workspace is None:
        return torch.empty(need, device=device, dtype=torch.uint8)
    if (not workspace.is_cuda or not workspace.is_contiguous()
            or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"{where}: workspace must be a contiguous CUDA buffer of at least "
                         f"{need} bytes")
    if workspace.device != device:
        raise ValueError(f"{where}: workspace must be on q's device ({device}); "
                         f"got {workspace.device}")
    return workspace


# The serving operators' wrappers are called once a layer and token, so they
# keep their own time down: torch's names are looked up once, the context switch
# and the stream object are skipped where the device is current already.
def _t():
    global _torch, _F32, _BF16, _I32, _F8, _get_device, _get_stream
    if _torch is None:
        import torch
        _F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
        _F8 = (torch.float8_e4m3fn, torch.uint8)
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _torch = torch
    return _torch


def _call(fn, name, dev, *args):
    """fn(*args, stream) on CUDA device number `dev` and its current stream;
    raises FaError."""
    if _get_device() == dev:
        st = fn(*args, _get_stream(dev))
    else:
        with _torch.cuda.device(dev):
            st = fn(*args, _get_stream(dev))
    if st:
        raise FaError(st, name)


def _check_place(where, ref, others):
    """ref and others: contiguous CUDA tensors on one device, as _check_cuda
    asks, found in one pass where they are.  Returns the device's number."""
    dev = ref.device
    if dev.type == "cuda" and ref.is_contiguous():
        for t in others:
            if t.device != dev or not t.is_contiguous():
                break
        else:
            return dev.index
    _check_cuda(where, ref, *others)
    return dev.index


def _shape(q, k):
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if Bk != B or dk != d:
        raise ValueError("q and k shapes disagree")
    return B, Hq, Hkv, Nq, Nk, d


def _stream(t):
    import torch
    return torch.cuda.current_stream(t.device).cuda_stream


def forward(q, k, v, scale=None, causal=False, out=None, lse=None, cta_pair=False):
    """O, L = attention(q, k, v) for contiguous CUDA tensors [B, H, N, d]
    (bf16 -> fa_fwd, or fa_fwd_pair with cta_pair=True; float32 ->
    fa_fwd_f32)."""
    import torch
    _check_qkv("forward", q, k, v, (torch.bfloat16, torch.float32))
    _check_cuda("forward", q, k, v)
    B, Hq, Hkv, Nq, Nk, d = _shape(q, k)
    scale = d ** -0.5 if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    L = torch.empty(B, Hq, Nq, device=q.device, dtype=torch.float32) if lse is None else lse
    if (tuple(o.shape) != tuple(q.shape) or o.dtype != q.dtype or tuple(L.shape) != (B, Hq, Nq)
            or L.dtype != torch.float32):
        raise ValueError("forward: out must be shaped and typed like q, lse float32 [B, Hq, Nq]")
    _check_cuda("forward", q, o, L)
    if cta_pair and q.dtype != torch.bfloat16:
        raise ValueError("forward: cta_pair=True needs bf16 tensors")
    fn = (fa_fwd_pair if cta_pair else fa_fwd) if q.dtype == torch.bfloat16 else fa_fwd_f32
    with _on(q):
        _check(fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), L.data_ptr(), B, Hq, Hkv,
                  Nq, Nk, d, scale, causal, _stream(q)), fn.__name__)
    return o, L


def forward_splitkv(q, k, v, scale=None, causal=False, num_splits=None, workspace=None):
    """O, L for bf16 q [B, Hq, Nq, d] against k, v [B, Hkv, Nk, d] with the key
    range cut into pieces merged by their log-sum-exp (fa_fwd_splitkv).
    Causal is bottom-right aligned (Nq <= Nk).  num_splits=None picks
    fa_fwd_splitkv_num_splits."""
    import torch
    _check_qkv("forward_splitkv", q, k, v, (torch.bfloat16,))
    _check_cuda("forward_splitkv", q, k, v)
    B, Hq, Hkv, Nq, Nk, d = _shape(q, k)
    scale = d ** -0.5 if scale is None else float(scale)
    if num_splits is None:
        num_splits = fa_fwd_splitkv_num_splits(B, Hq, Nq, Nk, d)
    need = max(fa_fwd_splitkv_workspace_size(B, Hq, Nq, d, num_splits), 1)
    if workspace is None:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    elif (not workspace.is_cuda or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"forward_splitkv: workspace must be a contiguous CUDA buffer of at "
                         f"least {need} bytes")
    elif workspace.device != q.device:
        raise ValueError(f"forward_splitkv: workspace must be on q's device ({q.device}); "
                         f"got {workspace.device}")
    o = torch.empty_like(q)
    L = torch.empty(B, Hq, Nq, device=q.device, dtype=torch.float32)
    with _on(q):
        _check(fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              L.data_ptr(), workspace.data_ptr(), B, Hq, Hkv, Nq, Nk, d, scale,
                              causal, num_splits, _stream(q)), "fa_fwd_splitkv")
    return o, L


def forward_fp8(q, k, v, descale_q, descale_k, descale_v, scale=None, causal=False):
    """O (bf16), L from E4M3 inputs (fa_fwd_fp8).  q, k, v: contiguous CUDA
    tensors of dtype float8_e4m3fn or uint8 (the codes); descale_*: the
    per-tensor dequantisation factors."""
    import torch
    _check_qkv("forward_fp8", q, k, v, (torch.float8_e4m3fn, torch.uint8))
    B, Hq, Hkv, Nq, Nk, d = _shape(q, k)
    if Nq != Nk:
        raise ValueError("forward_fp8: Nq must equal Nk")
    _check_cuda("forward_fp8", q, k, v)
    scale = d ** -0.5 if scale is None else float(scale)
    o = torch.empty(q.shape, device=q.device, dtype=torch.bfloat16)
    L = torch.empty(B, Hq, Nq, device=q.device, dtype=torch.float32)
    with _on(q):
        _check(fa_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), L.data_ptr(),
                          B, Hq, Hkv, Nq, d, scale, descale_q, descale_k, descale_v, causal,
                          _stream(q)), "fa_fwd_fp8")
    return o, L


def forward_dropout(q, k, v, p_drop, seed, offset=0, scale=None, causal=False):
    """O, L with dropout on P (bf16, fa_fwd_dropout)."""
    import torch
    _check_qkv("forward_dropout", q, k, v, (torch.bfloat16,))
    _check_cuda("forward_dropout", q, k, v)
    B, Hq, Hkv, Nq, Nk, d = _shape(q, k)
    scale = d ** -0.5 if scale is None else float(scale)
    o = torch.empty_like(q)
    L = torch.empty(B, Hq, Nq, device=q.device, dtype=torch.float32)
    with _on(q):
        _check(fa_fwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              L.data_ptr(), B, Hq, Hkv, Nq, Nk, d, scale, causal, p_drop, seed,
                              offset, _stream(q)), "fa_fwd_dropout")
    return o, L


def backward_dropout(q, k, v, o, lse, dout, p_drop, seed, offset=0, scale=None, causal=False,
                     workspace=None):
    """dQ, dK, dV of forward_dropout with the same seed and offset."""
    import torch
    _check_qkv("backward_dropout", q, k, v, (torch.bfloat16,))
    _check_bwd_in("backward_dropout", q, o, lse, dout)
    _check_cuda("backward_dropout", q, k, v, o, lse, dout)
    B, Hq, Hkv, Nq, Nk, d = _shape(q, k)
    scale = d ** -0.5 if scale is None else float(scale)
    workspace = _workspace("backward_dropout", workspace, B, Hq, Nq, d, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    with _on(q):
        _check(fa_bwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                              dv.data_ptr(), workspace.data_ptr(), B, Hq, Hkv, Nq, Nk, d, scale,
                              causal, p_drop, seed, offset, _stream(q)), "fa_bwd_dropout")
    return dq, dk, dv


def backward(q, k, v, o, lse, dout, scale=None, causal=False, workspace=None):
    """dQ, dK, dV for f = sum(O * dout); o and lse from ``forward``."""
    import torch
    _check_qkv("backward", q, k, v, (torch.bfloat16, torch.float32))
    _check_bwd_in("backward", q, o, lse, dout)
    _check_cuda("backward", q, k, v, o, lse, dout)
    B, Hq, Hkv, Nq, Nk, d = _shape(q, k)
    scale = d ** -0.5 if scale is None else float(scale)
    workspace = _workspace("backward", workspace, B, Hq, Nq, d, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fn = fa_bwd if q.dtype == torch.bfloat16 else fa_bwd_f32
    with _on(q):
        _check(fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                  dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                  workspace.data_ptr(), B, Hq, Hkv, Nq, Nk, d, scale, causal, _stream(q)),
               fn.__name__)
    return dq, dk, dv


# ------------------------------------------------- rotary positions, 8-bit cache
def rope_freqs(rot_dim, theta=10000.0, scaling="none", factor=1.0, original_len=4096,
               beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(freqs, mscale) for ``rope``: the float64 frequency table [rot_dim / 2]
    on `device` and the factor on the rotated values, scaled for long contexts
    ("none", "linear", "ntk" or "yarn", fa_rope_freqs).  "yarn" blends by each
    pair's turns within original_len, as its paper does; ``rope`` takes any
    float64 table, so one that ramps over the pairs' indexes, as some
    checkpoints' code does, is passed as it is."""
    import torch
    if scaling not in FA_ROPE_KINDS:
        raise ValueError(f"rope_freqs: scaling must be one of {tuple(FA_ROPE_KINDS)}")
    if rot_dim <= 0:
        raise ValueError("rope_freqs: rot_dim must be positive")
    table = (ctypes.c_double * (rot_dim // 2 + 1))()
    mscale = ctypes.c_float(1.0)
    _check(fa_rope_freqs(ctypes.addressof(table), ctypes.addressof(mscale), rot_dim, float(theta),
                         FA_ROPE_KINDS[scaling], float(factor), int(original_len),
                         float(beta_fast), float(beta_slow)), "fa_rope_freqs")
    return (torch.tensor(table[:rot_dim // 2], dtype=torch.float64, device=device),
            float(mscale.value))


def _rope(where, q, k, positions, freqs, mscale, interleaved, out, name):
    torch = _t()
    shape, dtype = q.shape, q.dtype
    if len(shape) != 4 or (dtype is not _BF16 and dtype is not _F32):
        raise ValueError(f"{where}: q must be [B, Hq, N, d], bfloat16 or float32")
    B, Hq, N, d = shape
    Hkv = 0
    if k is not None:
        ks = k.shape
        if len(ks) != 4 or k.dtype is not dtype or ks[0] != B or ks[2] != N or ks[3] != d:
            raise ValueError(f"{where}: k must be [B, Hkv, N, d] of q's dtype")
        Hkv = ks[1]
    ps = positions.shape
    per_batch = len(ps) == 2
    if positions.dtype is not _I32 or ps != ((B, N) if per_batch else (N,)):
        raise ValueError(f"{where}: positions must be int32 [B, N] or [N]")
    fs = freqs.shape
    if len(fs) != 1 or freqs.dtype is not torch.float64:
        raise ValueError(f"{where}: freqs must be float64 [rot_dim / 2]")
    place = [positions, freqs] if k is None else [k, positions, freqs]
    if out is not None:
        qo, ko = out
        for t, o in ((q, qo), (k, ko)):
            if (o is None) != (t is None) or (t is not None and (o.shape != t.shape
                                                                 or o.dtype != t.dtype)):
                raise ValueError(f"{where}: out must be shaped and typed like (q, k)")
        place += [qo] if ko is None else [qo, ko]
    dev = _check_place(where, q, place)
    if out is None:   # contiguous, as q and k are
        qo = torch.empty_like(q)
        ko = None if k is None else torch.empty_like(k)
    if dtype is _F32:
        name += "_f32"
    _call(getattr(_lib or lib(), name), name, dev, q.data_ptr(), 0 if k is None else k.data_ptr(),
          qo.data_ptr(), 0 if k is None else ko.data_ptr(), positions.data_ptr(), freqs.data_ptr(),
          B, Hq, Hkv, N, d, 2 * fs[0], per_batch, 1 if interleaved else 0, mscale)
    return qo, ko


def rope(q, k, positions, freqs, mscale=1.0, interleaved=False, out=None):
    """(q', k'): rotary positions on q [B, Hq, N, d] and k [B, Hkv, N, d] (k
    may be None), bfloat16 or float32, in one launch (fa_rope, fa_rope_f32).
    positions: int32 [B, N] or [N]; freqs, mscale: ``rope_freqs``.  out=(q, k)
    turns in place."""
    return _rope("rope", q, k, positions, freqs, mscale, interleaved, out, "fa_rope")


def rope_backward(dq, dk, positions, freqs, mscale=1.0, interleaved=False, out=None):
    """Gradients of ``rope``'s inputs from those of its outputs (fa_rope_bwd,
    fa_rope_bwd_f32); dk may be None."""
    return _rope("rope_backward", dq, dk, positions, freqs, mscale, interleaved, out,
                 "fa_rope_bwd")


def _check_cache(where, ref, k_cache, v_cache, k_scale, v_scale, block_table, B, Hkv, d, name,
                 lens, *more):
    """The cache's tensors against B, Hkv, d; lens (called `name`): int32 [B];
    more: tensors whose place alone is checked.  Returns (page, num_pages,
    max_pages, device number)."""
    shape = k_cache.shape
    if (len(shape) != 4 or shape[1] != Hkv or shape[3] != d or v_cache.shape != shape
            or k_cache.dtype not in _F8 or v_cache.dtype not in _F8):
        raise ValueError(f"{where}: k_cache and v_cache must be E4M3 [num_pages, Hkv, page, d]")
    num_pages, _, page, _ = shape
    shape = (num_pages, Hkv)
    if (k_scale.shape != shape or v_scale.shape != shape or k_scale.dtype is not _F32
            or v_scale.dtype is not _F32):
        raise ValueError(f"{where}: k_scale and v_scale must be float32 [num_pages, Hkv]")
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != B or block_table.dtype is not _I32:
        raise ValueError(f"{where}: block_table must be int32 [B, max_pages]")
    if lens is None or lens.shape != (B,) or lens.dtype is not _I32:
        raise ValueError(f"{where}: {name} must be int32 [B]")
    dev = _check_place(where, ref, (k_cache, v_cache, k_scale, v_scale, block_table, lens) + more)
    return page, num_pages, shape[1], dev


def cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, start, count=None):
    """Write new tokens k, v [B, Hkv, T, d] (bfloat16 or float32) of each
    sequence at positions start[b] .. into the paged E4M3 cache, with one
    power-of-two scale per page and head (fa_cache_append).  count: int32 [B]
    tokens of each sequence that count (None: all T).  A sequence whose start
    is negative is left out.  The cache tensors are updated in place."""
    _t()
    shape, dtype = k.shape, k.dtype
    if (len(shape) != 4 or v.shape != shape or v.dtype is not dtype
            or (dtype is not _BF16 and dtype is not _F32)):
        raise ValueError("cache_append: k and v must both be [B, Hkv, T, d], bfloat16 or float32")
    B, Hkv, T, d = shape
    more = (v,)
    if count is not None:
        if count.shape != (B,) or count.dtype is not _I32:
            raise ValueError("cache_append: count must be int32 [B]")
        more = (v, count)
    page, num_pages, max_pages, dev = _check_cache("cache_append", k, k_cache, v_cache, k_scale,
                                                   v_scale, block_table, B, Hkv, d, "start", start,
                                                   *more)
    name = "fa_cache_append_f32" if dtype is _F32 else "fa_cache_append"
    _call(getattr(_lib or lib(), name), name, dev, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
          start.data_ptr(), 0 if count is None else count.data_ptr(), B, Hkv, T, d, page,
          num_pages, max_pages)


def cache_read(k_cache, v_cache, k_scale, v_scale, block_table, lens, N, dtype=None):
    """Dense k, v [B, Hkv, N, d] (bfloat16, or dtype=torch.float32): the first
    N tokens of each sequence out of the cache, zeros from lens[b] on
    (fa_cache_read)."""
    torch = _t()
    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("cache_read: dtype must be bfloat16 or float32")
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("cache_read: k_cache must be [num_pages, Hkv, page, d], block_table "
                         "int32 [B, max_pages]")
    _, Hkv, _, d = k_cache.shape
    B = block_table.shape[0]
    page, num_pages, max_pages, dev = _check_cache("cache_read", k_cache, k_cache, v_cache,
                                                   k_scale, v_scale, block_table, B, Hkv, d,
                                                   "lens", lens)
    k = torch.empty(B, Hkv, N, d, device=k_cache.device, dtype=dtype)
    v = torch.empty_like(k)
    name = "fa_cache_read_f32" if dtype is torch.float32 else "fa_cache_read"
    _call(getattr(_lib or lib(), name), name, dev, k_cache.data_ptr(), v_cache.data_ptr(),
          k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
          k.data_ptr(), v.data_ptr(), B, Hkv, N, d, page, num_pages, max_pages)
    return k, v


@functools.lru_cache(maxsize=256)   # a step's layers ask for the same sizes
def _fwd_cache_bytes(*sizes):
    return lib().fa_fwd_cache_workspace_size(*sizes)


def forward_cache(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, scale=None, causal=True,
                  workspace=None):
    """O (bfloat16), L of query tokens q [B, Hq, Nq, d] (bfloat16) over the
    first lens[b] tokens of each sequence of the paged E4M3 cache
    (fa_fwd_cache).  Causal is bottom-right aligned: the queries are the last
    Nq of those tokens.  A query that sees no key gets O = 0, L = -inf."""
    torch = _t()
    shape = q.shape
    if len(shape) != 4 or q.dtype is not _BF16 or k_cache.dim() != 4:
        raise ValueError("forward_cache: q must be bfloat16 [B, Hq, Nq, d], k_cache "
                         "[num_pages, Hkv, page, d]")
    B, Hq, Nq, d = shape
    Hkv = k_cache.shape[1]
    page, num_pages, max_pages, dev = _check_cache("forward_cache", q, k_cache, v_cache, k_scale,
                                                   v_scale, block_table, B, Hkv, d, "lens", lens)
    L = _lib or lib()
    place = q.device
    need = _fwd_cache_bytes(B, Hq, Hkv, Nq, d, page, max_pages)
    if workspace is None:
        if need:
            workspace = torch.empty(need, device=place, dtype=torch.uint8)
    elif (not workspace.is_cuda or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"forward_cache: workspace must be a contiguous CUDA buffer of at least "
                         f"{need} bytes")
    elif workspace.device != place:
        raise ValueError(f"forward_cache: workspace must be on q's device ({place}); "
                         f"got {workspace.device}")
    o = torch.empty_like(q)
    lse = torch.empty(B, Hq, Nq, device=place, dtype=_F32)
    _call(L.fa_fwd_cache, "fa_fwd_cache", dev, q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
          lens.data_ptr(), o.data_ptr(), lse.data_ptr(), workspace.data_ptr() if need else None, B, Hq, Hkv, Nq, d,
          page, num_pages, max_pages, d ** -0.5 if scale is None else scale,
          1 if causal else 0)
    return o, lse
