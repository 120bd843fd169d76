"""What is measured of the 4-bit cache: the rotated append into it, the copies from and to it, and the attention over it.

Three operators, each in its plain form (elementary torch operations in 32 bits, angles in 64) and, where `own` is
true, as the library's calls:

  append   RMS norm of every query and key head, rotary position, and the write of the key and value rows of ragged new
           tokens into a 4-bit cache, contiguous or paged
  copy     bf16 rows into a 4-bit cache (to park a sequence), and 4-bit rows back into the bf16 cache that sparse
           decoding reads
  attend   causal attention of ragged new tokens (from one token to a large chunk) over a 4-bit cache, contiguous or
           paged, with optional score cap and sliding window

A row of a 4-bit cache is 128 codes, two a byte (element 2 i in the low half of byte i), and a scale byte for each 16 of
them.  A code is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale byte is an unsigned float of 5 exponent and 3
mantissa bits, bias 15: the upper bits of an fp16.  A block's scale is its largest size over 6, rounded to nearest, at
most 10240; a value is its quotient by the scale, rounded to nearest, ties to the even code.

Cases hold sizes only; ragged lengths follow from the sizes, contents from the seed.  Where codes are outputs they are
returned as the 8-bit floats of the same values, scales as fp16: a lookup of the packed bytes, within the pass.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension
BLOCK = 16       # values that share a scale
EPS = 1e-6
THETA = 1e6


# ---- cases -----------------------------------------------------------------------------------------------------------
def _append(name, B, T, L, Hq=28, Hkv=4, page=0, interleaved=False, norm=True, rot=D):
    c = dict(op="append", B=B, T=T, L=L, Hq=Hq, Hkv=Hkv, page=page, interleaved=interleaved, norm=norm, rot=rot)
    return dict(c, name=name) if name else c


def _copy(name, B, L, Hkv=4, back=True, src_page=64, dst_page=0):
    c = dict(op="copy", B=B, L=L, Hkv=Hkv, back=back, src_page=src_page, dst_page=dst_page)
    return dict(c, name=name) if name else c


def _attend(name, B, T, L, Hq=28, Hkv=4, page=0, cap=0.0, window=0, lse=False):
    c = dict(op="attend", B=B, T=T, L=L, Hq=Hq, Hkv=Hkv, page=page, cap=cap, window=window, lse=lse)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step of a batch: norm, rotation and append of a token a sequence into pages, all latency
        _append("append 61 tokens", 61, 61, 300, Hq=32, Hkv=8, page=64, interleaved=True),
        # a ragged batch of prompt chunks into small pages
        _append("append 8191 ragged", 5, 8191, 300, page=16, rot=64),
        # a whole long prompt
        _append("append 131072", 1, 131072, 0, page=256),
        # the library's 1M-key history comes back for sparse decoding
        _copy("read back 1048576", 1, 1048576, src_page=256),
        # idle sequences are parked: contiguous rows into pages
        _copy("park 7 x 40000", 7, 40000, Hkv=8, back=False, src_page=0, dst_page=128),
        # decoding of one short sequence: all latency
        _attend("attend 1 over 300", 1, 1, 300, lse=True),
        # decoding of one sequence at the library's 128K length
        _attend("attend 1 over 131072", 1, 1, 131072),
        # decoding of a ragged batch over pages
        _attend("attend 61 ragged decode", 61, 61, 9000, Hq=32, Hkv=8, page=64),
        # a few drafted tokens of each sequence are verified at once
        _attend("attend 16 x 3 over 20000", 16, 48, 20000, page=64),
        # chunks of a ragged batch behind long prefixes, capped scores in a sliding window
        _attend("attend 3x333 capped window", 3, 1000, 33000, Hq=16, Hkv=2, page=48, cap=30.0, window=4096),
        # a prompt by itself
        _attend("attend a prompt of 2000", 1, 2000, 2000, page=16),
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
        return _append("", B, T, rng.randrange(0, 20000 // B + 2), Hq, Hkv, page, rng.random() < 0.5,
                       rng.random() < 0.75, rng.choice((D, D, 64, 32)))
    if op == "copy":
        L = _log(rng, 1, 1000000 * 4 // max(4, Hkv))
        B = max(1, min(64, _log(rng, 1, max(1, 1000000 * 4 // Hkv // L))))
        return _copy("", B, L, Hkv, rng.random() < 0.6, page, rng.choice(PAGES))
    cap, window = rng.choice((0.0, 0.0, 0.0, 50.0)), rng.choice((0, 0, 0, _log(rng, 64, 8192)))
    if rng.random() < 0.6:    # decoding: a token, or a few, for every sequence
        B = _log(rng, 1, 128)
        L = _log(rng, 16, max(17, min(500000, 8000000 // (B * Hkv))))
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


ROW = D // 2 + D // BLOCK     # bytes of a 4-bit row


def work(case):
    n, rows = _lengths(case)
    if case["op"] == "append":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        return {"bytes": T * 2 * D * (2 * Hq + 2 * Hkv) + T * 2 * Hkv * ROW, "flops": T * (Hq + Hkv) * D * 7}
    if case["op"] == "copy":
        total = int(rows.sum()) * case["Hkv"] * 2
        return {"bytes": total * (2 * D + ROW), "flops": total * D}
    pairs, keys = _pairs(case)
    T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
    return {"bytes": T * Hq * D * 4 + keys * Hkv * 2 * ROW + (T * Hq * 4 if case["lse"] else 0), "flops": pairs * Hq * D * 4}


# ---- inputs ----------------------------------------------------------------------------------------------------------
def _normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _power(e):
    """2^e in 32 bits, exactly, for whole e above -126."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x):
    """bf16 or fp32 rows [..., 128] -> (packed codes [..., 64], scale bytes [..., 8])."""
    blocks = x.float().unflatten(-1, (D // BLOCK, BLOCK))
    top = blocks.abs().amax(-1) / 6.0
    step = _power(torch.frexp(top)[1].clamp(-13, 20) - 4)
    scale = (torch.round(top / step) * step).clamp(max=10240.0)
    size = scale.half().view(torch.int16) >> 7
    y = torch.where(scale[..., None] > 0, blocks / scale[..., None], torch.zeros_like(blocks))
    step = _power(torch.frexp(y)[1].clamp(1, 3) - 2)
    r = (torch.round(y.abs() / step) * step).clamp(max=6.0)
    code = torch.where(r <= 2, 2 * r, torch.where(r <= 3, r + 2, r / 2 + 4)).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), size.to(torch.uint8)


def _cache(g, B, Hkv, most, page, fp4, filled=True, sized=False):
    """Caches for B sequences of at most `most` rows, keys and values in one pool [2, pages, Hkv, rows, .], and the
    page table, or None.  sized: rows of sizes 1/8 to 8, as those of several layers."""
    if page:
        width = -(-most // page)
        spare = 3
        table = torch.randperm(B * width + spare, generator=g, device="cuda")[: B * width].to(torch.int32).view(B, width)
        shape = (2, B * width + spare, Hkv, page, D)
    else:
        table, shape = None, (2, B, Hkv, most, D)
    c = {"table": table, "fp4": fp4}
    if fp4 and filled:
        parts = []
        for _ in range(2):
            x = _normal(g, shape[1:])
            if sized:
                x = x * torch.exp2(torch.randint(-3, 4, shape[1:-1] + (1,), generator=g, device="cuda").float()).to(torch.bfloat16)
            parts.append(_quantised(x))
        c["codes"], c["scales"] = (torch.stack(p) for p in zip(*parts))
    elif fp4:
        c["codes"] = torch.zeros(shape[:-1] + (D // 2,), dtype=torch.uint8, device="cuda")
        c["scales"] = torch.zeros(shape[:-1] + (D // BLOCK,), dtype=torch.uint8, device="cuda")
    else:
        c["rows"] = _normal(g, shape) if filled else torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    return c


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _handle(c):
    from top_sparse_attention_exact_gb300 import retopk
    if c["fp4"]:
        return retopk.KVCache(c["codes"][0], c["codes"][1], table=c["table"], k_scale=c["scales"][0], v_scale=c["scales"][1])
    return retopk.KVCache(c["rows"][0], c["rows"][1], table=c["table"])


SIZES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _codes_of_bytes():
    """What two packed bytes stand for, as four 8-bit floats: a row for each 16-bit number."""
    one = torch.tensor(SIZES + tuple(-x for x in SIZES), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    n = torch.arange(1 << 16, device="cuda")
    return torch.stack([one[(n >> s) & 15] for s in (0, 4, 8, 12)], -1).contiguous().view(torch.int32).flatten()


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
        s["cache"] = _cache(g, B, Hkv, int((rows + n).max()), case["page"], True, filled=False)
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "copy":
        B, Hkv, back = case["B"], case["Hkv"], case["back"]
        s["src"] = _cache(g, B, Hkv, case["L"], case["src_page"], back, sized=True)
        s["dst"] = _cache(g, B, Hkv, case["L"] + 256, case["dst_page"], not back, filled=False)
        s["first"], s["last"] = torch.zeros(B, dtype=torch.int32, device="cuda"), _int32(rows)
    else:
        T, B, Hq, Hkv = case["T"], case["B"], case["Hq"], case["Hkv"]
        s["q"] = _normal(g, (T, Hq, D), 2.0)
        s["cache"] = _cache(g, B, Hkv, int(rows.max()) + 5, case["page"], True)
        s["cu"], s["lens"] = _int32(np.concatenate([[0], np.cumsum(n)])), _int32(rows)
        s["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda") if case["lse"] else None
    if case["op"] == "append" or (case["op"] == "copy" and not case["back"]):
        s["values"], s["up"] = _codes_of_bytes(), torch.full((1,), 128, dtype=torch.int16, device="cuda")
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
    page = (c["codes"] if c["fp4"] else c["rows"]).shape[3]
    return c["table"][b, pos // page].long(), pos % page


def _values32(codes, scales):
    """Packed rows in 32 bits."""
    one = torch.tensor(SIZES + tuple(-x for x in SIZES), device="cuda")
    x = torch.stack((one[(codes & 15).int()], one[(codes >> 4).int()]), -1).flatten(-2)
    size = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (x.unflatten(-1, (D // BLOCK, BLOCK)) * size[..., None]).flatten(-2)


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
    c["codes"][0][p, :, r], c["scales"][0][p, :, r] = _quantised(_rotated(s["k"], s["k_weight"], case, cos, sin))
    c["codes"][1][p, :, r], c["scales"][1][p, :, r] = _quantised(s["v"])
    torch.add(s["start"], s["cu"].diff(), out=s["end"])


def _plain_copy(s):
    src, dst = s["src"], s["dst"]
    b, pos = (torch.arange(s["case"]["L"], device="cuda") < s["last"][:, None]).nonzero(as_tuple=True)
    (p, r), (u, w) = _place(src, b, pos), _place(dst, b, pos)
    if src["fp4"]:
        dst["rows"][0][u, :, w] = _values32(src["codes"][0][p, :, r], src["scales"][0][p, :, r]).to(torch.bfloat16)
        dst["rows"][1][u, :, w] = _values32(src["codes"][1][p, :, r], src["scales"][1][p, :, r]).to(torch.bfloat16)
    else:
        dst["codes"][0][u, :, w], dst["scales"][0][u, :, w] = _quantised(src["rows"][0][p, :, r])
        dst["codes"][1][u, :, w], dst["scales"][1][u, :, w] = _quantised(src["rows"][1][p, :, r])


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
    k = _values32(c["codes"][0][p, :, r], c["scales"][0][p, :, r])                     # [B, L, Hkv, D]
    v = _values32(c["codes"][1][p, :, r], c["scales"][1][p, :, r])
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


def _rows(s, c):
    """A cache's buffers as the values they hold."""
    if not c["fp4"]:
        return {"k": c["rows"][0], "v": c["rows"][1]}
    codes = s["values"][c["codes"].view(torch.int16).int()].view(torch.float8_e4m3fn)
    scales = (c["scales"] * s["up"]).view(torch.float16)
    return {"k": codes[0], "v": codes[1], "k_scale": scales[0], "v_scale": scales[1]}


def run(s):
    if own:
        _own(s)
    else:
        {"append": _plain_append, "copy": _plain_copy, "attend": _plain_attend}[s["case"]["op"]](s)
    if s["case"]["op"] == "append":
        return {"q": s["q_out"], "end": s["end"], **_rows(s, s["cache"])}
    if s["case"]["op"] == "copy":
        return _rows(s, s["dst"])
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


# ---- 64-bit values -----------------------------------------------------------------------------------------------------
def _spans(c, b, count, start=0):
    """(page, first row, last row, offset in the sequence) of rows start .. start+count-1 of sequence b."""
    page = (c["codes"] if c["fp4"] else c["rows"]).shape[3]
    table = None if c["table"] is None else c["table"][b].tolist()
    at = start
    while at < start + count:
        upto = min(start + count, (at // page + 1) * page)
        yield (b if table is None else table[at // page]), at % page, at % page + upto - at, at - start
        at = upto


def _decoded(codes, scales):
    """Packed rows in 64 bits, from the fields of a code and of a scale byte."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).int()
    e, m = (n // 2) % 4, n % 2
    x = torch.where(e == 0, m * 0.5, (1 + 0.5 * m.double()) * torch.exp2((e - 1).double()))
    x = torch.where(n >= 8, -x, x)
    e, m = scales.int() // 8, (scales.int() % 8).double() / 8
    size = torch.where(e == 0, m * 2.0 ** -14, (1 + m) * torch.exp2((e - 15).double()))
    return x * size.repeat_interleave(BLOCK, -1)


def _grid():
    """The scales that are written, in order: byte i is grid[i]."""
    e, m = np.divmod(np.arange(227), 8)
    return torch.from_numpy(np.where(e == 0, m / 8 * 2.0 ** -14, (1 + m / 8) * 2.0 ** (e - 15.0))).cuda()


def _steps(x):
    """64-bit rows -> (code values, scale values): the nearest ones, by the borders between neighbours."""
    grid, a = _grid(), x.unflatten(-1, (D // BLOCK, BLOCK))
    top = a.abs().amax(-1).contiguous()
    border = 3.0 * (grid[1:] + grid[:-1])                      # of a block's largest size
    i = torch.searchsorted(border, top)                         # borders below it
    tie = border[i.clamp(max=225)] == top
    size = grid[torch.where(tie & (i % 2 == 1), i + 1, i).clamp(max=226)]
    sizes = torch.tensor(SIZES, dtype=torch.float64, device="cuda")
    got = torch.zeros(a.shape, dtype=torch.int64, device="cuda")
    for n in range(7):
        edge = 0.5 * (sizes[n] + sizes[n + 1]) * size[..., None]
        got += (a.abs() >= edge if n % 2 else a.abs() > edge).long()
    got = torch.where(size[..., None] > 0, got, torch.zeros_like(got))
    return (sizes[got] * torch.where(a < 0, -1.0, 1.0)).flatten(-2), size


def exact(case, seed):
    s = prepare(case, seed)
    n, rows = _lengths(case)
    if case["op"] == "append":
        out, half, c = torch.empty_like(s["q"], dtype=torch.float64), case["rot"] // 2, s["cache"]
        codes = torch.zeros(c["codes"].shape[1:-1] + (D,), dtype=torch.float64, device="cuda")
        scales = torch.zeros(c["scales"].shape[1:], dtype=torch.float64, device="cuda")
        at = 0
        for b in range(case["B"]):
            m = int(n[b])
            turn = torch.outer(torch.arange(m, device="cuda").double() + float(rows[b]), s["inv_freq"].double())
            turn = torch.polar(torch.ones_like(turn), turn)[:, None]
            x = s["q"][at:at + m].double()
            if case["norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * s["q_weight"].double()
            first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            out[at:at + m] = x
            got, size = _steps(s["v"][at:at + m].double())
            for page, r0, r1, o in _spans(c, b, m, int(rows[b])):
                codes[page, :, r0:r1] = got[o:o + r1 - r0].transpose(0, 1)
                scales[page, :, r0:r1] = size[o:o + r1 - r0].transpose(0, 1)
            at += m
        ends = torch.from_numpy(rows + n).to(torch.int32)
        # a rotated key next to a border of the 4-bit grid has no one value
        return {"q": out, "end": ends, "k": None, "v": codes, "k_scale": None, "v_scale": scales}
    if case["op"] == "copy":
        src, dst, found = s["src"], s["dst"], {}
        for i, name in enumerate(("k", "v")):
            x = _decoded(src["codes"][i], src["scales"][i]) if src["fp4"] else src["rows"][i].double()
            shape = (dst["codes"] if dst["fp4"] else dst["rows"]).shape[1:-1] + (D,)
            y = torch.zeros(shape, dtype=torch.float64, device="cuda")
            for b in range(case["B"]):
                mine = torch.cat([x[p, :, r0:r1] for p, r0, r1, _ in _spans(src, b, int(rows[b]))], 1)
                for p, r0, r1, o in _spans(dst, b, int(rows[b])):
                    y[p, :, r0:r1] = mine[:, o:o + r1 - r0]
            if dst["fp4"]:
                y, found[name + "_scale"] = _steps(y)
            found[name] = y
        return found
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
        k, v = (_decoded(torch.cat([c["codes"][x][p, :, r0:r1] for p, r0, r1, _ in spans], 1),
                         torch.cat([c["scales"][x][p, :, r0:r1] for p, r0, r1, _ in spans], 1)) for x in range(2))    # [Hkv, L, D]
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
