"""What is measured of the prompt-side operators: the rotated append, the cache copy and the chunk attention.

Three operators, each in its plain form (elementary torch operations in 32 bits, angles in 64) and, where `own` is
true, as the library's calls:

  append   RMS norm of every query and key head, rotary position, and the write of the key and value rows of ragged new
           tokens into a cache (bf16, or e4m3 codes with one power-of-two scale for 32 values; contiguous or paged)
  copy     rows of one cache into another: quantised rows read back into the bf16 cache that decoding reads, bf16 rows
           quantised to park a sequence, pages gathered into a contiguous cache
  attend   causal attention of ragged new tokens (from one token to a whole prompt) over a contiguous or paged cache,
           with optional score cap and sliding window

Cases hold sizes only; ragged lengths follow from the sizes, contents from the seed.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension
BLOCK = 32       # values that share a scale in a quantised row
EPS = 1e-6
THETA = 1e6


# ---- cases -----------------------------------------------------------------------------------------------------------
def _append(name, B, T, L, Hq=28, Hkv=4, mx8=False, page=0, interleaved=False, norm=True, rot=D):
    c = dict(op="append", B=B, T=T, L=L, Hq=Hq, Hkv=Hkv, mx8=mx8, page=page, interleaved=interleaved, norm=norm, rot=rot)
    return dict(c, name=name) if name else c


def _copy(name, B, L, Hkv=4, src_mx8=True, src_page=64, dst_mx8=False, dst_page=0):
    c = dict(op="copy", B=B, L=L, Hkv=Hkv, src_mx8=src_mx8, src_page=src_page, dst_mx8=dst_mx8, dst_page=dst_page)
    return dict(c, name=name) if name else c


def _attend(name, B, T, L, Hq=28, Hkv=4, page=0, cap=0.0, window=0, lse=False):
    c = dict(op="attend", B=B, T=T, L=L, Hq=Hq, Hkv=Hkv, page=page, cap=cap, window=window, lse=lse)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one sequence: a decode step's norm, rotation and append, all latency
        _append("append 1 token", 1, 1, 16384),
        # a decode step of a batch into a quantised paged cache
        _append("append 61 tokens mx8", 61, 61, 5000, Hq=32, Hkv=8, mx8=True, page=64, interleaved=True),
        # a ragged batch of prompt chunks into pages
        _append("append 8191 ragged", 5, 8191, 3000, page=16, rot=64),
        # a whole long prompt, quantised as it is written
        _append("append 131072 mx8", 1, 131072, 0, mx8=True, page=256),
        # a few parked sequences of ordinary length come back for decoding
        _copy("read back 3 x 4099", 3, 4099),
        # the library's 1M-key history comes back
        _copy("read back 1048576", 1, 1048576, src_page=256),
        # idle sequences are parked: contiguous rows quantised into pages
        _copy("park 7 x 40000", 7, 40000, Hkv=8, src_mx8=False, src_page=0, dst_mx8=True, dst_page=128),
        # dense decoding of one short sequence: all latency
        _attend("attend 1 over 300", 1, 1, 300, lse=True),
        # dense decoding of one sequence at the library's 128K length
        _attend("attend 1 over 131072", 1, 1, 131072),
        # dense decoding of a ragged batch over pages
        _attend("attend 61 ragged decode", 61, 61, 9000, Hq=32, Hkv=8, page=64),
        # chunks of a ragged batch behind long prefixes, capped scores in a sliding window
        _attend("attend 3x333 capped window", 3, 1000, 33000, Hq=16, Hkv=2, page=48, cap=30.0, window=4096),
        # a large chunk of a long prompt
        _attend("attend 4096 over 32768", 1, 4096, 32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ((28, 4), (32, 8), (16, 2), (8, 8), (16, 1), (7, 1))
PAGES = (0, 16, 48, 64, 128, 256)


def draw(rng):
    op = rng.choice(("append", "copy", "attend", "attend"))
    Hq, Hkv = rng.choice(HEADS)
    page = rng.choice(PAGES)
    if op == "append":
        T = _log(rng, 1, 100000 if Hq <= 28 else 60000)
        B = min(T, _log(rng, 1, 64))
        return _append("", B, T, rng.randrange(0, 20000 // B + 2), Hq, Hkv, rng.random() < 0.5, page, rng.random() < 0.5,
                       rng.random() < 0.75, rng.choice((D, D, 64, 32)))
    if op == "copy":
        L = _log(rng, 1, 1000000 * 4 // max(4, Hkv))
        B = max(1, min(64, _log(rng, 1, max(1, 1000000 * 4 // Hkv // L))))
        src_mx8 = rng.random() < 0.6
        return _copy("", B, L, Hkv, src_mx8, page, not src_mx8 and rng.random() < 0.7, rng.choice(PAGES))
    cap, window = rng.choice((0.0, 0.0, 0.0, 50.0)), rng.choice((0, 0, 0, _log(rng, 64, 8192)))
    if rng.random() < 0.5:    # decoding: a token, or a few, for every sequence
        B = _log(rng, 1, 128)
        L = _log(rng, 16, max(17, min(500000, 3000000 // (B * Hkv))))
        return _attend("", B, B * rng.choice((1, 1, 1, 3)), L, Hq, Hkv, page, cap, window, rng.random() < 0.3)
    L = _log(rng, 128, 100000)
    most = max(2, min(L, int(2.5e9 / (L * Hq))))
    T = _log(rng, 2, most)
    B = min(T, rng.choice((1, 1, 2, 3, 5)))
    return _attend("", B, T, max(1, L // B), Hq, Hkv, page, cap, window, rng.random() < 0.3)


def _lengths(case):
    """(tokens of each sequence, rows in the cache before the call, or in all for attend): ragged, from the sizes alone."""
    r = np.random.RandomState((case["B"] * 7919 + case["L"]) % (1 << 31))
    B, L = case["B"], case["L"]
    T = case.get("T", 0)
    if T:
        cut = np.sort(r.choice(np.arange(1, T), B - 1, replace=False)) if B > 1 else np.zeros(0, np.int64)
        n = np.diff(np.concatenate([[0], cut, [T]])).astype(np.int64)
        if T % B == 0 and T // B <= 4:
            n[:] = T // B
    else:
        n = np.zeros(B, np.int64)
    rows = np.full(B, L, np.int64)
    if B > 1 and L > 1:
        rows = r.randint(max(1, L // 4), L + 1, B).astype(np.int64)
        rows[0] = L
    if case["op"] == "attend":
        rows = np.maximum(rows, n)
    return n, rows


def _pairs(case):
    """(query-key pairs that the mask leaves, keys that some query sees), summed over the sequences."""
    n, L = _lengths(case)
    w = case["window"]
    pairs = keys = 0
    for ni, Li in zip(n.tolist(), L.tolist()):
        first = Li - ni
        seen = np.arange(first + 1, Li + 1, dtype=np.int64)
        pairs += int((np.minimum(seen, w) if w else seen).sum())
        keys += min(Li, ni - 1 + w) if w else Li
    return pairs, keys


def work(case):
    n, rows = _lengths(case)
    row = lambda mx8: D + D // BLOCK if mx8 else 2 * D  # noqa: E731
    if case["op"] == "append":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        return {"bytes": T * 2 * D * (2 * Hq + 2 * Hkv) + T * 2 * Hkv * row(case["mx8"]), "flops": T * (Hq + Hkv) * D * 7}
    if case["op"] == "copy":
        total = int(rows.sum()) * case["Hkv"] * 2
        return {"bytes": total * (row(case["src_mx8"]) + row(case["dst_mx8"])), "flops": total * D}
    pairs, keys = _pairs(case)
    T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
    return {"bytes": T * Hq * D * 4 + keys * Hkv * D * 4 + (T * Hq * 4 if case["lse"] else 0), "flops": pairs * Hq * D * 4}


# ---- inputs ----------------------------------------------------------------------------------------------------------
def _normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _power(e):
    """2^e in 64 bits, exactly, for whole e above -1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantised(x):
    """bf16 or fp32 rows -> (e4m3 codes, scale bytes): the smallest power of two that keeps 32 values within 448."""
    blocks = x.float().unflatten(-1, (D // BLOCK, BLOCK))
    m, e = torch.frexp(blocks.abs().amax(-1).double() / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    codes = (blocks.double() * _power(-e[..., None])).float().to(torch.float8_e4m3fn)
    return codes.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8)


def _cache(g, B, Hkv, most, page, mx8, filled=True):
    """Caches for B sequences of at most `most` rows: [pages, Hkv, rows, 128] and the page table, or None."""
    if page:
        width = -(-most // page)
        spare = 3
        table = torch.randperm(B * width + spare, generator=g, device="cuda")[: B * width].to(torch.int32).view(B, width)
        shape = (B * width + spare, Hkv, page, D)
    else:
        table, shape = None, (B, Hkv, most, D)
    c = {"table": table, "mx8": mx8}
    for n in ("k", "v"):
        if mx8 and filled:
            size = torch.exp2(torch.randint(-3, 4, shape[:-1] + (1,), generator=g, device="cuda").float())
            c[n], c[n + "_scale"] = _quantised(_normal(g, shape) * size)
        elif mx8:
            c[n] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
            c[n + "_scale"] = torch.zeros(shape[:-1] + (D // BLOCK,), dtype=torch.uint8, device="cuda")
        else:
            c[n] = _normal(g, shape) if filled else torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    return c


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _handle(c):
    from top_sparse_attention_exact_gb300 import retopk
    return retopk.KVCache(c["k"], c["v"], table=c["table"], k_scale=c.get("k_scale"), v_scale=c.get("v_scale"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, rows = _lengths(case)
    s = {"case": case}
    if case["op"] == "append":
        T, B, Hq, Hkv = case["T"], case["B"], case["Hq"], case["Hkv"]
        qkv = _normal(g, (T, (Hq + 2 * Hkv) * D), 1.5)      # the rows of one fused projection
        s["q"], s["k"], s["v"] = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
        s["q_weight"], s["k_weight"] = (1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")).to(torch.bfloat16)
        s["inv_freq"] = (THETA ** (-torch.arange(0, case["rot"], 2, device="cuda").double() / case["rot"])).float()
        s["cu"], s["start"] = _int32(np.concatenate([[0], np.cumsum(n)])), _int32(rows)
        s["end"] = torch.zeros_like(s["start"])
        s["cache"] = _cache(g, B, Hkv, int((rows + n).max()), case["page"], case["mx8"], filled=False)
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "copy":
        B, Hkv = case["B"], case["Hkv"]
        s["src"] = _cache(g, B, Hkv, case["L"], case["src_page"], case["src_mx8"])
        s["dst"] = _cache(g, B, Hkv, case["L"] + 256, case["dst_page"], case["dst_mx8"], filled=False)
        s["first"], s["last"] = torch.zeros(B, dtype=torch.int32, device="cuda"), _int32(rows)
    else:
        T, B, Hq, Hkv = case["T"], case["B"], case["Hq"], case["Hkv"]
        s["q"] = _normal(g, (T, Hq, D), 2.0)
        s["cache"] = _cache(g, B, Hkv, int(rows.max()) + 5, case["page"], False)
        s["cu"], s["lens"] = _int32(np.concatenate([[0], np.cumsum(n)])), _int32(rows)
        s["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda") if case["lse"] else None
    if own:     # handles that a user's program keeps: they describe the tensors above
        from top_sparse_attention_exact_gb300 import retopk
        for n in ("cache", "src", "dst"):
            if n in s:
                s[n + "_handle"] = _handle(s[n])
        if case["op"] == "append":
            w = case["norm"]
            s["rope"] = retopk.QKRope(inv_freq=s["inv_freq"], q_weight=s["q_weight"] if w else None,
                                      k_weight=s["k_weight"] if w else None, eps=EPS, interleaved=case["interleaved"])
        elif case["op"] == "attend":
            s["ws"] = torch.empty(retopk.chunk_attention_workspace_bytes(T, B, Hq, Hkv) + 256, dtype=torch.uint8,
                                  device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------
def _positions(cu, lens, T):
    """(sequence, index within it) of every token, and the position of its row behind `lens` rows."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t.to(torch.int32), right=True) - 1
    i = t - cu[b].long()
    return b, i, lens[b].long() + i


def _place(c, b, pos):
    """(page, row in it) of rows `pos` of sequences `b`."""
    if c["table"] is None:
        return b, pos
    page = c["k"].shape[2]
    return c["table"][b, pos // page].long(), pos % page


def _rotated(x, weight, case, cos, sin):
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    r, rest = x[..., : case["rot"]], x[..., case["rot"]:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r.chunk(2, -1)
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _plain_append(s):
    case, c = s["case"], s["cache"]
    b, _, pos = _positions(s["cu"], s["start"], case["T"])
    angle = pos.double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"].copy_(_rotated(s["q"], s["q_weight"], case, cos, sin))
    p, r = _place(c, b, pos)
    for name, x in (("k", _rotated(s["k"], s["k_weight"], case, cos, sin)), ("v", s["v"])):
        if case["mx8"]:
            c[name][p, :, r], c[name + "_scale"][p, :, r] = _quantised(x)
        else:
            c[name][p, :, r] = x.to(torch.bfloat16)
    torch.add(s["start"], s["cu"].diff(), out=s["end"])


def _plain_copy(s):
    src, dst = s["src"], s["dst"]
    b, pos = (torch.arange(s["case"]["L"], device="cuda") < s["last"][:, None]).nonzero(as_tuple=True)
    (p, r), (u, w) = _place(src, b, pos), _place(dst, b, pos)
    for name in ("k", "v"):
        x = src[name][p, :, r]
        if src["mx8"]:
            e = src[name + "_scale"][p, :, r].int()
            size = torch.where(e == 0, torch.full_like(e, 1 << 22), e << 23).view(torch.float32)
            x = (x.view(torch.float8_e4m3fn).float().unflatten(-1, (D // BLOCK, BLOCK)) * size[..., None]).flatten(-2)
        if dst["mx8"]:
            dst[name][u, :, w], dst[name + "_scale"][u, :, w] = _quantised(x)
        else:
            dst[name][u, :, w] = x.to(torch.bfloat16)


def _plain_attend(s):
    case, c = s["case"], s["cache"]
    B, T, Hq, Hkv = case["B"], case["T"], case["Hq"], case["Hkv"]
    n, L = _lengths(case)
    n, L, G = int(n.max()), int(L.max()), Hq // Hkv
    b, i, _ = _positions(s["cu"], s["lens"], T)
    q = torch.zeros((B, n, Hkv, G, D), device="cuda")
    q[b, i] = s["q"].float().view(T, Hkv, G, D)
    j = torch.arange(L, device="cuda")
    p, r = _place(c, torch.arange(B, device="cuda")[:, None], j[None, :].expand(B, L))
    k, v = c["k"][p, :, r].float(), c["v"][p, :, r].float()                     # [B, L, Hkv, D]
    score = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D), k.permute(0, 2, 3, 1)) / math.sqrt(D)
    score = score.view(B, Hkv, n, G, L)
    if case["cap"]:
        score = case["cap"] * torch.tanh(score / case["cap"])
    pos = (s["lens"].long() - s["cu"].diff().long())[:, None] + torch.arange(n, device="cuda")     # [B, n]
    seen = j <= pos[..., None]
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.view(B, Hkv, n * G, L), v.permute(0, 2, 1, 3)).view(B, Hkv, n, G, D) / total
    s["out"].copy_(out.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)[b, i])
    if s["lse"] is not None:
        s["lse"].copy_((top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(B, n, Hq)[b, i])


# ---- the library's calls -----------------------------------------------------------------------------------------------
def _own(s):
    from top_sparse_attention_exact_gb300 import retopk
    case = s["case"]
    if case["op"] == "append":
        retopk.qkv_append(s["rope"], s["q"], s["k"], s["v"], s["cache_handle"], s["start"], s["end"], s["q_out"],
                          cu_tokens=s["cu"])
    elif case["op"] == "copy":
        retopk.cache_copy(s["src_handle"], s["dst_handle"], s["first"], s["last"], case["L"])
    else:
        retopk.chunk_attention(s["q"], s["cache_handle"], s["lens"], s["out"], cu_tokens=s["cu"], softcap=case["cap"],
                               window=case["window"], lse=s["lse"], workspace=s["ws"])


def _rows(c):
    """A cache's buffers as the values they hold: codes and scales are 8-bit floats."""
    if not c["mx8"]:
        return {"k": c["k"], "v": c["v"]}
    return {"k": c["k"].view(torch.float8_e4m3fn), "v": c["v"].view(torch.float8_e4m3fn),
            "k_scale": c["k_scale"].view(torch.float8_e8m0fnu), "v_scale": c["v_scale"].view(torch.float8_e8m0fnu)}


def run(s):
    if own:
        _own(s)
    else:
        {"append": _plain_append, "copy": _plain_copy, "attend": _plain_attend}[s["case"]["op"]](s)
    if s["case"]["op"] == "append":
        return {"q": s["q_out"], "end": s["end"], **_rows(s["cache"])}
    if s["case"]["op"] == "copy":
        return _rows(s["dst"])
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


# ---- 64-bit values -----------------------------------------------------------------------------------------------------
def _spans(c, b, count, start=0):
    """(page, first row, last row, offset in the sequence) of rows start .. start+count-1 of sequence b."""
    page = c["k"].shape[2]
    table = None if c["table"] is None else c["table"][b].tolist()
    at = start
    while at < start + count:
        upto = min(start + count, (at // page + 1) * page)
        yield (b if table is None else table[at // page]), at % page, at % page + upto - at, at - start
        at = upto


def _values(c, name):
    """All rows of a cache in 64 bits."""
    if not c["mx8"]:
        return c[name].double()
    scale = _power(c[name + "_scale"].int() - 127)
    return c[name].view(torch.float8_e4m3fn).double() * scale.repeat_interleave(BLOCK, -1)


def _steps(x):
    """64-bit rows -> (e4m3 code values, scale values), from the grid's definition: 3 bits below the leading one, 2^-9 at least."""
    a = x.reshape(x.shape[:-1] + (D // BLOCK, BLOCK))
    top = a.abs().amax(-1, keepdim=True)
    e = torch.frexp(top.clamp_min(2.0 ** -140))[1] - 9
    e = torch.where(top > 448.0 * _power(e), e + 1, e).clamp(-127, 127)
    y = a / _power(e)
    ulp = _power(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
    return (torch.round(y / ulp) * ulp).reshape(x.shape), _power(e[..., 0])


def exact(case, seed):
    s = prepare(case, seed)
    n, rows = _lengths(case)
    if case["op"] == "append":
        out, half, c = torch.empty_like(s["q"], dtype=torch.float64), case["rot"] // 2, s["cache"]
        got = {"k": c["k"].double(), "v": c["v"].double()}
        scales = {x: torch.full(c["k"].shape[:-1] + (D // BLOCK,), 2.0 ** -127, dtype=torch.float64, device="cuda") for x in got}
        at = 0
        for b in range(case["B"]):
            m = int(n[b])
            turn = torch.outer(torch.arange(m, device="cuda").double() + float(rows[b]), s["inv_freq"].double())
            turn = torch.polar(torch.ones_like(turn), turn)[:, None]
            new = {"v": s["v"][at:at + m].double()}
            for name in ("q", "k"):
                x = s[name][at:at + m].double()
                if case["norm"]:
                    x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * s[name + "_weight"].double()
                first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
                z = torch.complex(x[..., first], x[..., second]) * turn
                x[..., first], x[..., second] = z.real, z.imag
                if name == "q":
                    out[at:at + m] = x
                else:
                    new["k"] = x
            for name in got:
                codes, size = _steps(new[name]) if case["mx8"] else (new[name], None)
                for page, r0, r1, o in _spans(c, b, m, int(rows[b])):
                    got[name][page, :, r0:r1] = codes[o:o + r1 - r0].transpose(0, 1)
                    if case["mx8"]:
                        scales[name][page, :, r0:r1] = size[o:o + r1 - r0].transpose(0, 1)
            at += m
        ends = torch.from_numpy(rows + n).to(torch.int32)
        if case["mx8"]:     # a rotated key next to a border of the 8-bit grid has no one value
            return {"q": out, "end": ends, "k": None, "v": got["v"], "k_scale": None, "v_scale": scales["v"]}
        return {"q": out, "end": ends, **got}
    if case["op"] == "copy":
        src, dst, got = s["src"], s["dst"], {}
        for name in ("k", "v"):
            x = _values(src, name)
            y = torch.zeros(dst[name].shape, dtype=torch.float64, device="cuda")
            for b in range(case["B"]):
                mine = torch.cat([x[p, :, r0:r1] for p, r0, r1, _ in _spans(src, b, int(rows[b]))], 1)
                for p, r0, r1, o in _spans(dst, b, int(rows[b])):
                    y[p, :, r0:r1] = mine[:, o:o + r1 - r0]
            if dst["mx8"]:
                y, e = _steps(y)
                got[name + "_scale"] = e
            got[name] = y
        return got
    pairs, _ = _pairs(case)
    if pairs * case["Hq"] * D * 4 > 4e12:
        return None
    T, Hq, Hkv, c = case["T"], case["Hq"], case["Hkv"], s["cache"]
    out = torch.empty((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, Hq), dtype=torch.float64, device="cuda")
    at, G = 0, Hq // Hkv
    for b in range(case["B"]):
        m, L = int(n[b]), int(rows[b])
        spans = list(_spans(c, b, L))
        k, v = (torch.cat([c[x][p, :, r0:r1] for p, r0, r1, _ in spans], 1).double() for x in ("k", "v"))    # [Hkv, L, D]
        for h in range(Hkv):
            for i0 in range(0, m, 256):
                i1 = min(m, i0 + 256)
                where = torch.arange(L - m + i0, L - m + i1, device="cuda")[:, None, None]
                z = torch.einsum("igd,jd->igj", s["q"][at + i0:at + i1, h * G:(h + 1) * G].double(), k[h]) * D ** -0.5
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                j = torch.arange(L, device="cuda")
                hidden = j > where
                if case["window"]:
                    hidden = hidden | (where - j >= case["window"])
                z = z.masked_fill(hidden, -math.inf)
                lse[at + i0:at + i1, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[at + i0:at + i1, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", torch.softmax(z, -1), v[h])
        at += m
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
