"""What is measured of the serving operators: rotary positions, the 8-bit paged key/value cache, attention over it.

A cache is two tensors [pages, Hkv, page, d] of E4M3 codes and two [pages, Hkv] of float32 scales: a page is the
block of tokens that shares one scale per head.  block_table [B, max_pages] names each sequence's pages in order.
"""
import math

import torch

own = False

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "f32": F32}
SCALE_MIN = 2.0 ** -112  # the scale of a page whose values are all zero (or smaller than this allows)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 32 sequences, positions far past the trained length: latency
        dict(name="rope_decode", op="rope", B=32, Hq=32, Hkv=8, N=1, d=128, rot=128, dtype="bf16", interleaved=False,
             backward=False, scaling="yarn", factor=16.0, far=120000),
        # the training step's q and k, causal B4 H16 N4096 d128
        dict(name="rope_train", op="rope", B=4, Hq=16, Hkv=16, N=4096, d=128, rot=128, dtype="bf16", interleaved=True,
             backward=False, scaling="none", factor=1.0, far=0),
        # the gradient in float32, half of each head rotated, an odd length
        dict(name="rope_grad_f32_partial", op="rope", B=2, Hq=16, Hkv=4, N=1999, d=64, rot=32, dtype="f32",
             interleaved=False, backward=True, scaling="linear", factor=4.0, far=5000),
        # a decode step of 64 sequences writes one token each, mostly into pages already begun
        dict(name="append_decode", op="append", B=64, Hkv=8, T=1, d=128, page=64, dtype="bf16", start_lo=1, start_hi=2000,
             ragged=False),
        # four prompts of up to 4096 tokens enter the cache, ragged, some after a shared prefix
        dict(name="append_prefill", op="append", B=4, Hkv=8, T=4096, d=128, page=64, dtype="bf16", start_lo=0,
             start_hi=333, ragged=True),
        # the cache of four long sequences back as bf16, for a kernel that wants dense K and V
        dict(name="read_long", op="read", B=4, Hkv=8, d=128, page=64, dtype="bf16", len_lo=5001, len_hi=8192),
        # a short one in float32, small pages
        dict(name="read_f32_pages_of_16", op="read", B=3, Hkv=2, d=256, page=16, dtype="f32", len_lo=17, len_hi=777),
        # one short sequence, one token: latency alone
        dict(name="attn_short", op="attn", B=1, Hq=8, Hkv=8, Nq=1, d=64, page=16, len_lo=300, len_hi=300, causal=True),
        # one long sequence, one token, grouped heads: the cache is split over the whole GPU
        dict(name="attn_long_gqa", op="attn", B=1, Hq=32, Hkv=8, Nq=1, d=128, page=64, len_lo=16384, len_hi=16384,
             causal=True),
        # a full decode batch of ragged lengths: the cache is far larger than L2
        dict(name="attn_batch", op="attn", B=32, Hq=32, Hkv=8, Nq=1, d=128, page=64, len_lo=2047, len_hi=16384,
             causal=True),
        # five drafted tokens a sequence checked at once, wide heads
        dict(name="attn_draft_d256", op="attn", B=8, Hq=16, Hkv=4, Nq=5, d=256, page=32, len_lo=501, len_hi=4000,
             causal=True),
        # a chunk of a prompt against the cache of what came before it
        dict(name="attn_chunk", op="attn", B=1, Hq=8, Hkv=8, Nq=512, d=128, page=128, len_lo=16384, len_hi=16384,
             causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attn", "attn"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        N = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(64, 60000 // (N * Hkv * (group + 1)))))
        return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, N=N, d=d, rot=rng.choice([d, d // 2, d // 4]), dtype=dtype,
                    interleaved=rng.random() < 0.5, backward=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=float(rng.choice([2, 4, 8, 32])),
                    far=rng.choice([0, 1000, 1000000]))
    if op == "append":
        T = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(128, 40000 // (T * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype, start_lo=rng.choice([0, 1, 50]),
                    start_hi=rng.choice([50, 500, 3000]), ragged=rng.random() < 0.5)
    hi = _log(rng, 1, 16384)
    lo = rng.choice([0, hi // 2, hi])
    if op == "read":
        B = _log(rng, 1, max(1, min(64, 60000 // (hi * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, dtype=dtype, len_lo=lo, len_hi=hi)
    Nq = rng.choice([1, 1, 1, 2, 3, 7, _log(rng, 1, 512)])
    most = 8 * 512 * 16384 * 128 // (hi * Hkv * group * d)  # tokens of queries: the work of the largest listed case
    Nq = max(1, min(Nq, most))
    B = _log(rng, 1, max(1, min(64, 120000 // (hi * Hkv), most // Nq)))
    return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, Nq=Nq, d=d, page=page, len_lo=lo, len_hi=hi,
                causal=rng.random() < 0.8)


def _spread(B, lo, hi):
    """B lengths from lo to hi, the longest first, the others in no order."""
    return [hi if b == 0 else lo + (hi - lo) * ((b * 37 + 11) % 101) // 100 for b in range(B)]


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        x = case["B"] * (case["Hq"] + case["Hkv"]) * case["N"] * d
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * es * x + 4 * case["B"] * case["N"] + 4 * case["rot"], "flops": 3 * x * case["rot"] // d}
    if case["op"] == "append":
        n = sum(_counts(case)) * case["Hkv"] * d
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * (es + 1) + 12 * case["B"], "flops": 4 * n}
    lens = _spread(case["B"], case["len_lo"], case["len_hi"])
    pages = sum(-(-n // case["page"]) for n in lens)
    cache = 2 * sum(lens) * case["Hkv"] * d + 8 * pages * case["Hkv"] + 4 * pages + 4 * case["B"]
    if case["op"] == "read":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": cache + 2 * es * case["B"] * case["Hkv"] * max(lens) * d, "flops": 2 * sum(lens) * case["Hkv"] * d}
    Nq, Hq = case["Nq"], case["Hq"]
    seen = sum(_seen(n, Nq, case["causal"]) for n in lens)
    rows = case["B"] * Hq * Nq
    return {"bytes": cache + rows * (4 * d + 4), "flops": 4 * Hq * d * seen}


def _seen(n, Nq, causal):
    """Pairs of a query and a key it sees: query i stands at position n - Nq + i."""
    if not causal:
        return n * Nq
    first = n - Nq + 1  # keys seen by the first query
    if first >= 0:
        return Nq * first + Nq * (Nq - 1) // 2
    return n * (n + 1) // 2


def _counts(case):
    return _spread(case["B"], case["T"] // 2, case["T"]) if case["ragged"] else [case["T"]] * case["B"]


# ------------------------------------------------------------------ inputs
def _rope_table(case):
    """Frequencies (float64, one for each rotated pair) and the factor on the rotated values, scaled for long contexts."""
    rot, s, theta = case["rot"], case["factor"], 10000.0
    if case["scaling"] == "ntk":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "yarn":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return (1 - keep) * f / s + keep * f, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _quantise(x):
    """E4M3 codes and power-of-two scales of pages [pages, H, page, d]."""
    m, e = torch.frexp(x.float().abs().amax((2, 3)))
    s = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int())).clamp(min=SCALE_MIN)
    return (x.float() / s[:, :, None, None]).to(F8), s


def _cache(case, tokens, g):
    """A cache of random pages with room for `tokens` of each sequence, its pages in no order, and its table."""
    page, H, d = case["page"], case["Hkv"], case["d"]
    need = [max(1, -(-n // page)) for n in tokens]
    width, total = max(need), sum(need) + 2
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    ends = torch.tensor(need, device="cuda").cumsum(0)
    col = torch.arange(width, device="cuda")[None, :]
    at = (ends - torch.tensor(need, device="cuda"))[:, None] + col
    table = torch.where(at < ends[:, None], perm[at.clamp(max=total - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    pages = []
    for k in range(2):
        x = torch.randn(total, H, page, d, generator=g, device="cuda", dtype=BF16)
        x = x * torch.exp(torch.randn(total, H, 1, 1, generator=g, device="cuda", dtype=F32)).to(BF16)
        pages.append(_quantise(x))
    return dict(k_cache=pages[0][0], v_cache=pages[1][0], k_scale=pages[0][1], v_scale=pages[1][1],
                table=table.contiguous())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)

    def randn(*shape, dtype):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32).to(dtype)

    s = dict(case=case)
    if case["op"] == "rope":
        dt = DTYPES[case["dtype"]]
        s["q"] = randn(case["B"], case["Hq"], case["N"], case["d"], dtype=dt)
        s["k"] = randn(case["B"], case["Hkv"], case["N"], case["d"], dtype=dt)
        first = torch.randint(0, case["far"] + 1, (case["B"], 1), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(case["N"], device="cuda")[None, :]).to(torch.int32)
        freqs, s["mscale"] = _rope_table(case)
        s["freqs"] = freqs.cuda()
        return s
    if case["op"] == "append":
        dt = DTYPES[case["dtype"]]
        start, count = _spread(case["B"], case["start_lo"], case["start_hi"]), _counts(case)
        s.update(_cache(case, [a + n for a, n in zip(start, count)], g))
        for name in ("k", "v"):  # a few channels of a head are larger than the others, as trained ones are
            s[name] = randn(case["B"], case["Hkv"], case["T"], case["d"], dtype=dt)
            s[name] *= torch.exp(randn(1, case["Hkv"], 1, case["d"], dtype=F32)).to(dt)
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        s["count"] = torch.tensor(count, dtype=torch.int32, device="cuda") if case["ragged"] else None
        return s
    lens = _spread(case["B"], case["len_lo"], case["len_hi"])
    s.update(_cache(case, lens, g))
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["N"] = max(lens)
    if case["op"] == "attn":
        s["q"] = randn(case["B"], case["Hq"], case["Nq"], case["d"], dtype=BF16)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if case["op"] == "rope":
        return _rope(s, case)
    if case["op"] == "append":
        return _append(s, case)
    if case["op"] == "read":
        return _read(s, case)
    return _attn(s, case)


def _rope(s, case):
    if own:
        import exact_io_aware_50_b200 as fa
        fn = fa.rope_backward if case["backward"] else fa.rope
        return fn(s["q"], s["k"], s["positions"], s["freqs"], mscale=s["mscale"], interleaved=case["interleaved"])
    angle = s["positions"].double()[:, None, :, None] * s["freqs"]  # far positions: the angle in 64 bits
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
    if case["backward"]:
        sin = -sin
    return _rotate(s["q"], cos, sin, case), _rotate(s["k"], cos, sin, case)


def _rotate(t, cos, sin, case):
    rot = case["rot"]
    z = t[..., :rot].float()
    if case["interleaved"]:
        x, y = z[..., 0::2], z[..., 1::2]
        z = torch.stack((x * cos - y * sin, y * cos + x * sin), -1).flatten(-2)
    else:
        x, y = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat((x * cos - y * sin, y * cos + x * sin), -1)
    return torch.cat((z.to(t.dtype), t[..., rot:]), -1)


def _append(s, case):
    if own:
        import exact_io_aware_50_b200 as fa
        fa.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["start"],
                        s["count"])
    else:
        _append_plain(s["k"], s["k_cache"], s["k_scale"], s, case)
        _append_plain(s["v"], s["v_cache"], s["v_scale"], s, case)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _append_plain(x, cache, scale, s, case):
    P, T = case["page"], case["T"]
    t = torch.arange(T, device="cuda")[None, :]
    pos = s["start"].long()[:, None] + t
    live = (t < s["count"][:, None]) if s["count"] is not None else torch.ones_like(pos, dtype=torch.bool)
    index = torch.gather(s["table"].long(), 1, (pos // P).clamp(max=s["table"].shape[1] - 1))
    page, slot = index[live], (pos % P)[live]                      # one entry for each token that is written
    rows = x.float().transpose(1, 2)[live]                         # [tokens, H, d]
    top = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), rows.abs().amax(-1), "amax")
    m, e = torch.frexp(top)
    need = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int()).clamp(min=SCALE_MIN)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    begun = torch.zeros_like(touched).index_fill_(0, page[slot == 0], True)
    new = torch.where(touched[:, None], torch.where(begun[:, None], need, torch.maximum(need, scale)), scale)
    at = torch.gather(s["table"].long(), 1, (s["start"].long()[:, None] // P).clamp(max=s["table"].shape[1] - 1))[:, 0]
    first = (s["start"] % P)[(s["start"] % P != 0) & live[:, 0]]
    at = at[(s["start"] % P != 0) & live[:, 0]]                    # pages that hold older tokens: their codes follow the scale
    kept = cache.view(torch.uint8)[at]
    old = (kept.view(F8).float() * (scale[at] / new[at])[:, :, None, None]).to(F8).view(torch.uint8)
    older = torch.arange(P, device="cuda") < first[:, None]
    cache.view(torch.uint8)[at] = torch.where(older[:, None, :, None], old, kept)
    codes = (rows / new[page][:, :, None]).to(F8)
    cache.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
    scale.copy_(new)


def _dense(cache, scale, s, case, N):
    """The first N tokens of each sequence as float32 [B, H, N, d], zero behind its length."""
    table = s["table"].long()
    x = cache.view(torch.uint8)[table].view(F8).float() * scale[table][..., None, None]  # [B, pages, H, page, d]
    x = x.permute(0, 2, 1, 3, 4).reshape(table.shape[0], case["Hkv"], -1, case["d"])[:, :, :N]
    live = torch.arange(N, device="cuda") < s["lens"][:, None]
    return torch.where(live[:, None, :, None], x, torch.zeros((), device="cuda"))


def _read(s, case):
    dt = DTYPES[case["dtype"]]
    if own:
        import exact_io_aware_50_b200 as fa
        return fa.cache_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"], s["N"], dtype=dt)
    return (_dense(s["k_cache"], s["k_scale"], s, case, s["N"]).to(dt),
            _dense(s["v_cache"], s["v_scale"], s, case, s["N"]).to(dt))


def _attn(s, case):
    if own:
        import exact_io_aware_50_b200 as fa
        return fa.forward_cache(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                                causal=case["causal"])
    B, Hq, Nq, d, N = case["B"], case["Hq"], case["Nq"], case["d"], s["N"]
    k, v = _dense(s["k_cache"], s["k_scale"], s, case, N), _dense(s["v_cache"], s["v_scale"], s, case, N)
    q = s["q"].float().reshape(B, case["Hkv"], -1, d)
    z = (q @ k.transpose(-1, -2)).reshape(B, Hq, Nq, N) * d ** -0.5
    j = torch.arange(N, device="cuda")
    seen = (j < s["lens"][:, None])[:, None, None, :]
    if case["causal"]:
        last = s["lens"][:, None] - Nq + torch.arange(Nq, device="cuda")
        seen = seen & (j <= last[..., None])[:, None]
    z = torch.where(seen, z, torch.full((), -math.inf, device="cuda"))
    top = z.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros((), device="cuda"))
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, case["Hkv"], -1, N) @ v).reshape(B, Hq, Nq, d) / total.clamp(min=1e-30)
    return o.to(BF16), (top + torch.log(total))[..., 0]


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [_exact_rope(s[n].double(), s, case) for n in ("q", "k")]
    if case["op"] == "append":
        out = {}
        for n in ("k", "v"):
            out[n + "_cache"], out[n + "_scale"] = _exact_append(s[n].double(), s[n + "_cache"], s[n + "_scale"], s, case)
        return out
    if case["op"] == "read":
        out = []
        for n in ("k", "v"):
            x = torch.zeros(case["B"], case["Hkv"], s["N"], case["d"], dtype=torch.float64, device="cuda")
            for b, length in enumerate(s["lens"].tolist()):
                x[b, :, :length] = _exact_tokens(s[n + "_cache"], s[n + "_scale"], s["table"][b], length)
            out.append(x)
        return out
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    group, Nq = case["Hq"] // case["Hkv"], case["Nq"]
    for b, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        k = _exact_tokens(s["k_cache"], s["k_scale"], s["table"][b], length).repeat_interleave(group, 0)
        v = _exact_tokens(s["v_cache"], s["v_scale"], s["table"][b], length).repeat_interleave(group, 0)
        z = torch.matmul(s["q"][b].double(), k.mT) / math.sqrt(case["d"])
        if case["causal"]:
            hidden = torch.ones(Nq, length, dtype=torch.bool, device="cuda").triu(length - Nq + 1)
            z.masked_fill_(hidden, -math.inf)
        lse[b] = torch.logsumexp(z, -1)
        w = torch.where(torch.isfinite(lse[b])[..., None], torch.exp(z - lse[b][..., None]), torch.zeros((), dtype=torch.float64, device="cuda"))
        o[b] = torch.matmul(w, v)
    return [o, lse]


def _exact_rope(x, s, case):
    rot = case["rot"]
    turn = torch.polar(torch.full((), float(s["mscale"]), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[..., None] * s["freqs"] * (-1.0 if case["backward"] else 1.0))[:, None]
    even = torch.arange(0, rot, 2) if case["interleaved"] else torch.arange(rot // 2)
    odd = even + (1 if case["interleaved"] else rot // 2)
    z = torch.complex(x[..., even], x[..., odd]) * turn
    x[..., even], x[..., odd] = z.real, z.imag
    return x


def _exact_tokens(cache, scale, table, length):
    """The tokens of one sequence in 64 bits, [H, length, d]."""
    H, P, d = cache.shape[1:]
    pages = table[: -(-length // P)].long()
    x = cache.view(torch.uint8)[pages].view(F8).double() * scale[pages].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(H, -1, d)[:, :length]


def _exact_append(x, cache, scale, s, case):
    """Page by page, with E4M3 by its definition: 3 bits of fraction, exponents from -6, at most 448."""
    P = case["page"]
    value, scale = cache.double(), scale.double()
    counts = s["count"].tolist() if s["count"] is not None else [case["T"]] * case["B"]

    def e4m3(t):
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(t / step) * step).clamp(-448, 448)

    for b, (start, count) in enumerate(zip(s["start"].tolist(), counts)):
        t = 0
        while t < count:
            slot = (start + t) % P
            n = min(P - slot, count - t)
            page = int(s["table"][b, (start + t) // P])
            new = x[b, :, t:t + n]
            top = new.abs().amax((1, 2))
            need = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -140) / 448)) - 1)
            need = torch.where(448 * need < top, 2 * need, need)       # a logarithm may be off next to a power of two
            need = torch.where(448 * need < top, 2 * need, need)
            need = torch.where(448 * need < top, 2 * need, need).clamp(min=SCALE_MIN)
            if slot:
                need = torch.maximum(need, scale[page])
                value[page, :, :slot] = e4m3(value[page, :, :slot] * (scale[page] / need)[:, None, None])
            scale[page] = need
            value[page, :, slot:slot + n] = e4m3(new / need[:, None, None])
            t += n
    return value, scale
