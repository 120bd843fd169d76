"""The 4-bit cache (RETOPK_CACHE_FP4): rotated append into it, copies from and to it, attention over it, against plain
64-bit formulas (GPU).

Tolerances.  u = 2^-24 is half a step of fp32, half a step of bf16 is 2^-8 relative to the value.
  codes      of values that are exact (values, bf16 rows) scale and codes have one right answer: ties go to even.
             A rotated key is off by at most 2^-18 of the head's largest element (see the prompt-side tests): its
             scale may be a neighbour of the right one only where a sixth of the largest lies that near the border, its
             code is off by at most half the codes' gap and that error.
  attention  a 4-bit value is exact in fp16 and bf16, so keys and values add no rounding of their own.  A score is a sum of 128
             products, off by at most 128 u sum|q k| scale <= 2^-17 times that sum, and the exponential's argument and
             result by 2^-20 more: d; a capped score is off by no more.  The weights are rounded to fp16 once: by 2^-11 of
             each, or by half of fp16's smallest step, 2^-25, where that is more.  They are taken so that the row's
             largest is at least 2^7, so that is 2^-32 of p at most.  The output is rounded to bf16:
             |out - exact| <= 2^-8 |exact| + (2^-11 + 2 d + 2^-14) sum_j p_j |v_j| + 2^-32 sum_j |v_j|.
             lse is off by d + 2^-20 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

from top_sparse_attention_exact_gb300 import retopk

pytestmark = pytest.mark.gpu
D = 128
SIZES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def offsets(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


def f64(x):
    return torch.tensor(x, dtype=torch.float64, device="cuda")


def scale_of(byte):
    """What scale bytes stand for, in 64 bits, from their fields."""
    e, m = byte.int() // 8, (byte.int() % 8).double() / 8
    s = torch.where(e == 0, m * 2.0 ** -14, (1 + m) * torch.exp2((e - 15).double()))
    s = torch.where(byte.int() == 248, f64(math.inf), s)
    return torch.where(byte.int() > 248, f64(math.nan), s)


def value4(codes, scales):
    """Packed rows [..., 64] and scale bytes [..., 8] in 64 bits."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    x = f64(SIZES)[n % 8] * torch.where(n >= 8, -1.0, 1.0)
    return (x.unflatten(-1, (8, 16)) * scale_of(scales)[..., None]).flatten(-2)


def quantise4(x):
    """fp64 rows -> (sizes' indices with the sign in bit 3, scale bytes): nearest, by the exact borders between neighbours."""
    a = x.unflatten(-1, (8, 16))
    top = a.abs().amax(-1)
    grid = scale_of(torch.arange(227, device="cuda"))
    border = 3.0 * (grid[1:] + grid[:-1])
    i = torch.searchsorted(border, top.contiguous())
    tie = border[i.clamp(max=225)] == top
    byte = torch.where(tie & (i % 2 == 1), i + 1, i).clamp(max=226)
    s = grid[byte][..., None]
    code = torch.zeros(a.shape, dtype=torch.long, device="cuda")
    for n in range(7):
        edge = 0.5 * (SIZES[n] + SIZES[n + 1]) * s
        code += (a.abs() >= edge if n % 2 else a.abs() > edge).long()
    code = torch.where(s > 0, code, torch.zeros_like(code))
    bad = ~a.isfinite().all(-1)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return (code + 8 * torch.signbit(a).long()).flatten(-2), byte


class Cache:
    """A cache of B sequences with `rows` capacity, contiguous or in shuffled pages, filled with odd bytes."""

    def __init__(self, B, Hkv, rows, page=0, form="fp4", seed=0):
        self.page, self.form = page, form
        if page:
            width = -(-rows // page)
            perm = np.random.default_rng(seed).permutation(B * width + 2)[:B * width].reshape(B, width)
            self.table, shape = i32(perm), (B * width + 2, Hkv, page)
        else:
            self.table, shape = None, (B, Hkv, rows)
        full = lambda n, x: torch.full(shape + (n,), x, dtype=torch.uint8, device="cuda")  # noqa: E731
        if form == "bf16":
            self.k, self.v = (torch.full(shape + (D,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.ks = self.vs = None
        else:
            n, m = (64, 8) if form == "fp4" else (128, 4)
            self.k, self.v, self.ks, self.vs = full(n, 0x55), full(n, 0x55), full(m, 0xff), full(m, 0xff)
        self.h = retopk.KVCache(self.k, self.v, table=self.table, k_scale=self.ks, v_scale=self.vs)

    def at(self, b, n):
        pos = torch.arange(n, device="cuda")
        return (self.table[b, pos // self.page].long(), pos % self.page) if self.page else (torch.full_like(pos, b), pos)

    def put(self, b, k, v):
        """Rows 0.. of sequence b: bf16 [n, Hkv, 128], or a pair (codes, scales)."""
        for x, s, y in ((self.k, self.ks, k), (self.v, self.vs, v)):
            if self.form == "bf16":
                p, r = self.at(b, y.shape[0])
                x[p, :, r] = y
            else:
                p, r = self.at(b, y[0].shape[0])
                x[p, :, r], s[p, :, r] = y

    def rows(self, b, n):
        p, r = self.at(b, n)
        if self.form == "bf16":
            return [x[p, :, r].double() for x in (self.k, self.v)]
        if self.form == "fp4":
            return [value4(x[p, :, r], s[p, :, r]) for x, s in ((self.k, self.ks), (self.v, self.vs))]
        out = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            e = torch.exp2((s[p, :, r].int() - 127).double())
            out.append((x[p, :, r].view(torch.float8_e4m3fn).double().unflatten(-1, (4, 32)) * e[..., None]).flatten(-2))
        return out

    def parts(self):
        return [x for x in (self.k, self.v, self.ks, self.vs) if x is not None]

    def snapshot(self):
        return [x.clone() for x in self.parts()]


def packed(g, *shape, sizes=(0.5, 3.0)):
    """Random 4-bit rows: (codes [..., 64], scales [..., 8])."""
    lo, hi = (math.log2(x) for x in sizes)
    s = torch.exp2(torch.rand(*shape, 8, generator=g, device="cuda") * (hi - lo) + lo).half()
    return (torch.randint(0, 256, (*shape, 64), generator=g, device="cuda", dtype=torch.uint8),
            (s.view(torch.int16) >> 7).to(torch.uint8))


def freqs(rot, theta=1e6):
    return (theta ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)).float()


def rotated(x, w, inv_freq, pos, interleaved, eps):
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    top = x.abs().amax(-1, keepdim=True)
    if inv_freq is not None:
        m = inv_freq.numel()
        t = pos.double()[:, None, None] * inv_freq.double()
        i = torch.arange(m, device="cuda")
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
        y = x.clone()
        y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
        y[..., b] = x[..., b] * t.cos() + x[..., a] * t.sin()
        x = y
    return x, 2.0 ** -18 * top


# ---- copies ----------------------------------------------------------------------------------------------------------
def rows_of_all_kinds(g, n, Hkv):
    """bf16 rows of many sizes: normal ones, ones on the codes' borders, zeros, very small and very large ones."""
    x = normal(g, n, Hkv, D) * torch.exp2(torch.randint(-12, 12, (n, Hkv, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
    if n > 8:
        x[1::4] = torch.randint(-24, 25, x[1::4].shape, generator=g, device="cuda").to(torch.bfloat16) / 4
        x[2::8] = torch.randint(-240, 241, x[2::8].shape, generator=g, device="cuda").to(torch.bfloat16) * 2.0 ** -20
        x[4::8, :, ::3] = 0
        x[5] = 0
        x[6, :, ::5] = 3e38
        x[7] = 2.0 ** -133
    return x


@pytest.mark.parametrize("n,Hkv,page,page2", [([1], 1, 0, 0), ([17, 0, 130], 3, 16, 48), ([40, 333], 8, 0, 64), ([65], 2, 256, 0)])
def test_rows_are_parked_and_read_back(n, Hkv, page, page2):
    g = gen(sum(n))
    B, most = len(n), max(n) + 3
    src, dst, back = Cache(B, Hkv, most, page, "bf16"), Cache(B, Hkv, most, page2, seed=1), Cache(B, Hkv, most, page, "bf16", seed=2)
    for b in range(B):
        src.put(b, rows_of_all_kinds(g, n[b], Hkv), rows_of_all_kinds(g, n[b], Hkv))
    before, st = dst.snapshot(), torch.zeros(1, dtype=torch.int32, device="cuda")
    first, last = i32([min(2, x) for x in n]), i32(n)
    retopk.cache_copy(src.h, dst.h, first, last, status=st)
    retopk.cache_copy(dst.h, back.h, first, last, status=st)
    assert st.item() == 0
    for b in range(B):
        f = min(2, n[b])
        p, r = dst.at(b, n[b])
        p, r = p[f:], r[f:]
        for x, codes, scales, z in zip(src.rows(b, n[b]), (dst.k, dst.v), (dst.ks, dst.vs), back.rows(b, n[b])):
            code, byte = quantise4(x[f:])
            got = torch.stack((codes[p, :, r] % 16, codes[p, :, r] // 16), -1).flatten(-2).long()
            assert torch.equal(scales[p, :, r].long(), byte)
            # (the sign of a zero code is not looked at)
            assert torch.equal(got % 8, code % 8) and torch.equal((got >= 8) & (got % 8 > 0), (code >= 8) & (code % 8 > 0))
            assert torch.equal(z[f:], value4(codes[p, :, r], scales[p, :, r]))      # exact in bf16
        for x, old in zip(dst.parts(), before):
            x[p, :, r] = old[p, :, r]
    for x, old in zip(dst.parts(), before):      # nothing else was written
        assert torch.equal(x, old)


@pytest.mark.parametrize("page,page2", [(0, 16), (64, 48)])
def test_copies_between_coded_forms(page, page2):
    g, B, Hkv, n = gen(page), 2, 2, 100
    a, b, c8, c4 = Cache(B, Hkv, n, page), Cache(B, Hkv, n, page2, seed=3), Cache(B, Hkv, n, page2, "mx8", seed=4), Cache(B, Hkv, n, page, seed=5)
    for i in range(B):
        a.put(i, packed(g, n, Hkv), packed(g, n, Hkv, sizes=(2.0 ** -14, 8000.0)))
    zero, last = i32([0] * B), i32([n] * B)
    retopk.cache_copy(a.h, b.h, zero, last)      # bits
    retopk.cache_copy(a.h, c8.h, zero, last)     # one rounding to 8 bits
    retopk.cache_copy(c8.h, c4.h, zero, last)    # one rounding back
    for i in range(B):
        for x, y in zip(a.rows(i, n), b.rows(i, n)):
            assert torch.equal(x, y)
        for x, y, z, codes, scales in zip(a.rows(i, n), c8.rows(i, n), c4.rows(i, n), (c4.k, c4.v), (c4.ks, c4.vs)):
            # the smallest power of two with max <= 448 of it, codes of 4 bits or half a subnormal step of 2^-9
            top = x.unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True)
            e = torch.exp2(torch.ceil(torch.log2(top / 448)))
            assert ((y - x).abs().unflatten(-1, (4, 32)) <= torch.maximum(2.0 ** -4 * x.abs().unflatten(-1, (4, 32)), 2.0 ** -10 * e)).all()
            code, byte = quantise4(y)
            p, r = c4.at(i, n)
            assert torch.equal(scales[p, :, r].long(), byte)
            assert torch.equal(z.abs(), f64(SIZES)[code % 8] * scale_of(byte).repeat_interleave(16, -1))


def test_blocks_that_are_not_finite():
    x = torch.ones((4, 1, D), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 127] = float("inf"), float("nan"), float("-inf")
    src, dst, back = Cache(1, 1, 4, 0, "bf16"), Cache(1, 1, 4), Cache(1, 1, 4, 0, "bf16")
    src.put(0, x, x)
    retopk.cache_copy(src.h, dst.h, i32([0]), i32([4]))
    retopk.cache_copy(dst.h, back.h, i32([0]), i32([4]))
    assert [dst.ks[0, 0, r].tolist().index(255) for r in range(3)] == [0, 2, 7] and (dst.ks == 255).sum() == 3
    bad = [0, 16], [32, 48], [112, 128]
    for r, (lo, hi) in enumerate(bad):
        y = back.k[0, 0, r].float()
        assert y[lo:hi].isnan().all() and (torch.cat((y[:lo], y[hi:])) == 1.03125).sum() + (torch.cat((y[:lo], y[hi:])) == 1.0).sum() == 112
    assert not back.k[0, 0, 3].isnan().any()


@pytest.mark.parametrize("by", ["copy", "append"])
def test_blocks_at_the_ends_of_the_scales(by):
    # (largest of a block, its scale byte, what comes back of it), by hand.  Below 6 x 2^-14 scales are 2^-17 apart, ties go to even
    u = 2.0 ** -17                                                   # the smallest scale
    cases = [(0.0, 0, 0.0), (2.0 ** -133, 0, 0.0), (2.0 ** -19, 0, 0.0), (2.0 ** -16, 0, 0.0),
             (3 * u, 0, 0.0),                                        # 6 x 2^-18: the tie between no scale and the smallest
             ((1.5 + 2.0 ** -7) * 2 * u, 1, 3 * u),                  # the next bf16
             (6 * u, 1, 6 * u), (8.9375 * u, 1, 6 * u),              # (1.49 of it: the code is held at 6)
             (9 * u, 2, 8 * u),                                      # the tie between 1 and 2; 4.5 of 2, nearest code 4
             (15 * u, 2, 12 * u), (6 * 8 * u, 8, 6 * 8 * u),         # 2.5: a tie to 2; 6 x 2^-14, the smallest normal scale
             (48.25 * u, 8, 6 * 8 * u), (61440.0, 226, 61440.0), (61440.0 + 256, 226, 61440.0), (3e38, 226, 61440.0)]
    g = gen(77)
    x = torch.zeros((len(cases), 1, D), dtype=torch.bfloat16, device="cuda")
    for r, (top, byte, back) in enumerate(cases):
        at = torch.randint(0, 16, (8,), generator=g, device="cuda") + 16 * torch.arange(8, device="cuda")
        x[r, 0, at] = torch.tensor([top, -top] * 4, dtype=torch.bfloat16, device="cuda")
    n = len(cases)
    c, flat = Cache(1, 1, n), Cache(1, 1, n, 0, "bf16")
    if by == "copy":
        flat.put(0, x, x)
        retopk.cache_copy(flat.h, c.h, i32([0]), i32([n]))
    else:
        retopk.qkv_append(retopk.QKRope(), x, x, x, c.h, i32([0]), cu_tokens=offsets([n]))
    retopk.cache_copy(c.h, flat.h, i32([0]), i32([n]))
    for r, (top, byte, back) in enumerate(cases):
        for scales, rows in ((c.ks, flat.k), (c.vs, flat.v)):
            assert scales[0, 0, r].tolist() == [byte] * 8, (top, scales[0, 0, r])
            assert torch.equal(rows[0, 0, r].double(), back * x[r, 0].double().sign()), top


@pytest.mark.parametrize("form", ["fp4", "mx8"])
def test_keys_that_are_the_values_keep_one_pool(form):
    src, two, one = Cache(2, 2, 40, 16, "bf16"), Cache(2, 2, 40, 48, form), Cache(2, 2, 40, 48, form)
    for b in range(2):
        x = normal(gen(80 + b), 40, 2, D)
        src.put(b, x, x)
    one.h = retopk.KVCache(one.k, one.k, table=one.table, k_scale=one.ks, v_scale=one.ks)
    for c in (one, two):
        retopk.cache_copy(src.h, c.h, i32([0, 3]), i32([40, 17]))
    assert torch.equal(one.k, two.k) and torch.equal(one.ks, two.ks)
    bad = retopk.KVCache(one.k, two.k, table=one.table, k_scale=one.ks, v_scale=one.ks)      # one's scales for both are refused
    with pytest.raises(retopk.RetopkError):
        retopk.cache_copy(src.h, bad, i32([0]), i32([1]))


@pytest.mark.parametrize("form", ["fp4", "mx8"])
def test_keys_and_values_by_turns_in_one_pool(form):
    # pages 2 i of a pool are keys, pages 2 i + 1 values: the pools overlap, no row does
    g, B, rows = gen(81), 2, 40
    src, c, near = Cache(B, 2, rows, 16, "bf16"), Cache(2 * B, 2, rows, 16, form), Cache(B, 2, rows, 16, form)
    for b in range(B):
        src.put(b, normal(g, rows, 2, D), normal(g, rows, 2, D))
    pages = c.k.shape[0] // 2 * 2
    table = 2 * torch.randperm(pages // 2, generator=torch.Generator().manual_seed(3))[:B * 3].view(B, 3).to(torch.int32).cuda()
    h = retopk.KVCache(c.k[:pages - 1], c.k[1:pages], table=table, k_scale=c.ks[:pages - 1], v_scale=c.ks[1:pages])
    x = normal(g, B, 8, D)
    for to in (h, near.h):
        retopk.cache_copy(src.h, to, i32([0] * B), i32([rows - 2] * B))
        retopk.qkv_append(retopk.QKRope(), x, x[:, :2], x[:, 2:4], to, i32([rows - 2, 20]))
    for b in range(B):
        pos = torch.arange(rows - 2 + (b == 0), device="cuda")
        p, r = table[b, pos // 16].long(), pos % 16
        pn, rn = near.at(b, len(pos))
        for codes, scales, want, want_scales, odd in ((c.k, c.ks, near.k, near.ks, 0), (c.k, c.ks, near.v, near.vs, 1)):
            assert torch.equal(codes[p + odd, :, r], want[pn, :, rn]) and torch.equal(scales[p + odd, :, r], want_scales[pn, :, rn])
    if form == "fp4":
        q = normal(g, B, 8, D)
        assert torch.equal(retopk.chunk_attention(q, h, i32([rows - 1, 30])), retopk.chunk_attention(q, near.h, i32([rows - 1, 30])))


def test_a_pool_past_2_31_elements():
    pages, g = 70000, gen(2)                              # 64 bytes x 512 rows a page: 2.3e9
    k, v = (torch.zeros((pages, 1, 512, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, 1, 512, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = i32([[pages - 1, 3]])
    far = retopk.KVCache(k, v, table=table, k_scale=ks, v_scale=vs)
    src, back = Cache(1, 1, 600, 0, "bf16"), Cache(1, 1, 600, 0, "bf16")
    x, y = normal(g, 600, 1, D), normal(g, 600, 1, D)
    src.put(0, x, y)
    retopk.cache_copy(src.h, far, i32([0]), i32([600]))
    retopk.cache_copy(far, back.h, i32([0]), i32([600]))
    code, byte = quantise4(x[:, 0].double())
    assert torch.equal(ks[pages - 1, 0].long(), byte[:512]) and torch.equal(ks[3, 0, :88].long(), byte[512:])
    assert torch.equal(back.k[0, 0].double().abs(), f64(SIZES)[code % 8] * scale_of(byte).repeat_interleave(16, -1))


# ---- rotated append --------------------------------------------------------------------------------------------------
APPEND = [  # tokens of each sequence, rows before, Hq, Hkv, page, rot, interleaved, norm
    ([1], [0], 28, 4, 0, 128, False, True),
    ([1, 1, 1], [5, 127, 128], 8, 8, 16, 128, True, True),
    ([7, 0, 1, 130], [0, 3, 16, 500], 7, 1, 48, 64, False, True),
    ([7, 0, 1, 130], [0, 3, 16, 500], 28, 4, 48, 64, True, False),
    ([300], [1], 32, 8, 0, 32, False, False),
    ([33, 65], [100, 31], 16, 1, 64, 16, False, True),
    ([20], [9], 3, 3, 0, 0, False, False),                         # quantisation alone
]


@pytest.mark.parametrize("n,start,Hq,Hkv,page,rot,inter,norm", APPEND)
@pytest.mark.parametrize("in_place", [False, True])
def test_append(n, start, Hq, Hkv, page, rot, inter, norm, in_place):
    g = gen(len(n) * 100 + Hq + rot)
    B, T, pad = len(n), sum(n), 3
    proj = normal(g, T + pad, (Hq + 2 * Hkv) * D, scale=2.0)
    q, k, v = (x.view(T + pad, -1, D) for x in proj.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    qw, kw = (normal(g, D) for _ in range(2)) if norm else (None, None)
    inv = freqs(rot) if rot else None
    c = Cache(B, Hkv, max(a + b for a, b in zip(n, start)) + 5, page)
    before = c.snapshot()
    sl, st = i32(start), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sl if in_place else torch.full_like(sl, -1)
    qo = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rope = retopk.QKRope(inv, qw, kw, eps=1e-5, interleaved=inter)
    retopk.qkv_append(rope, q, k, v, c.h, sl, None if in_place else out, qo, cu_tokens=offsets(n), status=st)
    assert out.tolist() == [a + b for a, b in zip(n, start)] and st.item() == 0 and (qo[T:] == 7).all()
    t0 = 0
    for b in range(B):
        sel = slice(t0, t0 + n[b])
        t0 += n[b]
        if n[b] == 0:
            continue
        pos = start[b] + torch.arange(n[b], device="cuda")
        ref, tol = rotated(q[sel], qw, inv, pos, inter, 1e-5)
        assert ((qo[sel].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + tol).all()
        p, r = c.at(b, start[b] + n[b])
        p, r = p[start[b]:], r[start[b]:]
        # values: one right answer
        code, byte = quantise4(v[sel].double())
        assert torch.equal(c.vs[p, :, r].long(), byte)
        assert torch.equal(value4(c.v[p, :, r], c.vs[p, :, r]).abs(), f64(SIZES)[code % 8] * scale_of(byte).repeat_interleave(16, -1))
        # keys: the nearest ones to a value that is off by tol at most
        ref, tol = rotated(k[sel], kw, inv, pos, inter, 1e-5)
        got, s = c.ks[p, :, r].long(), scale_of(c.ks[p, :, r])
        top = ref.unflatten(-1, (8, 16)).abs().amax(-1)
        low, high = (quantise4((ref + d * tol * ref.sign()).clamp(-3e38, 3e38))[1] for d in (-1, 1))
        assert ((got >= low) & (got <= high)).all() and (top > 0).all()
        wide = s.repeat_interleave(16, -1)
        y = value4(c.k[p, :, r], c.ks[p, :, r])
        a = ref.abs() / wide
        half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, torch.where(a <= 6, 1.0, a - 6))) * wide
        assert ((y - ref).abs() <= half * (1 + 2.0 ** -20) + 2 * tol).all()
    for now, old in zip(c.snapshot(), before):      # what belongs to no new row is as it was
        for b in range(B):
            p, r = c.at(b, start[b] + n[b])
            now[p[start[b]:], :, r[start[b]:]] = old[p[start[b]:], :, r[start[b]:]]
        assert torch.equal(now, old)


def test_append_without_norm_or_rotation_is_what_a_copy_parks():
    g = gen(9)
    n, start = [40, 1, 25], [0, 77, 12]
    q, k, v = normal(g, 66, 8, D), rows_of_all_kinds(g, 66, 2), rows_of_all_kinds(g, 66, 2)
    rows, parked, c = Cache(3, 2, 100, 16, "bf16"), Cache(3, 2, 100, 48), Cache(3, 2, 100, 48)
    for cache in (rows, c):
        retopk.qkv_append(retopk.QKRope(), q, k, v, cache.h, i32(start), cu_tokens=offsets(n))
    retopk.cache_copy(rows.h, parked.h, i32(start), i32([a + b for a, b in zip(n, start)]))
    for x, y in zip(c.parts(), parked.parts()):
        assert torch.equal(x, y)


def test_append_full_sequences_and_bad_pages():
    g = gen(5)
    n, start = [4, 4, 4], [28, 29, 0]
    q, k, v = normal(g, 12, 4, D), normal(g, 12, 2, D), normal(g, 12, 2, D)
    c, st = Cache(3, 2, 32, 16), torch.zeros(1, dtype=torch.int32, device="cuda")
    before, sl = c.snapshot(), i32(start)
    retopk.qkv_append(retopk.QKRope(freqs(128)), q, k, v, c.h, sl, cu_tokens=offsets(n), status=st)
    assert sl.tolist() == [32, 29, 4] and st.item() == retopk.STATUS_KV_FULL
    for x, old in zip(c.parts(), before):      # the second sequence's pages are as they were
        assert torch.equal(x[c.table[1].long()], old[c.table[1].long()])
    good = c.table.clone()
    c.table[0, 1], c.table[2, 0] = c.k.shape[0], -1
    before = c.snapshot()
    st.zero_()
    retopk.qkv_append(retopk.QKRope(freqs(128)), q, k, v, c.h, i32([12, 0, 14]), cu_tokens=offsets([6, 0, 6]), status=st)
    assert st.item() == retopk.STATUS_BAD_PAGE
    for x, old in zip(c.parts(), before):
        for page in range(x.shape[0]):
            assert torch.equal(x[page], old[page]) == (page not in (good[0, 0].item(), good[2, 1].item()))


def test_append_captured_and_replayed_advances_each_time():
    g, B = gen(31), 3
    q, k, v = normal(g, B, 4, D), normal(g, B, 2, D), normal(g, B, 2, D)
    c, sl, qo = Cache(B, 2, 40, 16), i32([0, 5, 38]), torch.empty((B, 4, D), dtype=torch.bfloat16, device="cuda")
    rope, st = retopk.QKRope(freqs(128)), torch.zeros(1, dtype=torch.int32, device="cuda")
    retopk.qkv_append(rope, q, k, v, c.h, sl, q_out=qo, status=st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        retopk.qkv_append(rope, q, k, v, c.h, sl, q_out=qo, status=st)
    for _ in range(3):
        graph.replay()
    assert sl.tolist() == [4, 9, 42] and st.item() == 0
    code, byte = quantise4(v.double())
    for b, rows in enumerate((range(4), range(5, 9), range(38, 42))):
        p, r = c.at(b, 42)
        for i in rows:
            assert torch.equal(c.vs[p[i], :, r[i]].long(), byte[b])


# ---- attention -------------------------------------------------------------------------------------------------------
def check(q, n, lens, c, out, lse, scale, cap, window):
    """Against 64-bit attention over the values that the rows stand for."""
    t, Hkv = 0, c.k.shape[1]
    for b, (m, L) in enumerate(zip(n, lens)):
        sel = slice(t, t + m)
        t += m
        if m == 0:
            continue
        G = q.shape[1] // Hkv
        k, v = (x.repeat_interleave(G, 1) for x in c.rows(b, L))
        x = q[sel].double()
        pos = torch.arange(L - m, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        seen = (j <= pos) & ((j > pos - window) if window else True)
        s = torch.einsum("thd,jhd->htj", x, k) * scale
        d = 2.0 ** -17 * scale * torch.einsum("thd,jhd->htj", x.abs(), k.abs())
        if cap:
            s = cap * torch.tanh(s / cap)
        s = s.masked_fill(~seen, -math.inf)
        d = d.masked_fill(~seen, 0.0).amax(-1).T[..., None] if L else torch.zeros((m, q.shape[1], 1), device="cuda", dtype=torch.float64)
        d = d + 2.0 ** -20
        p = torch.softmax(s, -1).nan_to_num(0.0)
        ref, size = torch.einsum("htj,jhd->thd", p, v), torch.einsum("htj,jhd->thd", p, v.abs())
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * d + 2.0 ** -14) * size + 2.0 ** -32 * v.abs().sum(0)
        err = (out[sel].double() - ref).abs()
        assert (err <= tol).all().item(), (b, float((err - tol).max()), float((err / (size + 1e-30)).max()))
        if lse is not None:
            rl = torch.logsumexp(s, -1).T
            none = rl == -math.inf
            assert torch.equal(lse[sel] == -math.inf, none)
            assert ((lse[sel].double() - rl).abs() <= d[..., 0] + 2.0 ** -20 * (1 + rl.abs()))[~none].all()


ATTEND = [  # tokens of each sequence, rows in all, Hq, Hkv, page, window, cap
    ([1], [1], 1, 1, 0, 0, 0.0),                                    # a single key
    ([1], [300], 28, 4, 0, 0, 0.0),
    ([1], [129], 7, 1, 16, 0, 0.0),
    ([1] * 9, [1, 2, 15, 16, 17, 31, 32, 33, 1000], 16, 1, 48, 0, 0.0),
    ([1] * 9, [63, 64, 65, 127, 128, 129, 255, 256, 257], 8, 1, 0, 0, 0.0),
    ([1] * 5, [0, 5, 400, 17, 16], 32, 8, 64, 0, 50.0),             # a sequence without rows
    ([3] * 4, [3, 64, 500, 2], 8, 8, 0, 0, 0.0),                    # the last: fewer rows than tokens
    ([1, 1], [70001, 333], 28, 4, 256, 0, 0.0),                     # a long history beside a short one
    ([1] * 3, [30011, 30000, 5], 5, 1, 0, 0, 0.0),
    ([5], [40000], 16, 2, 0, 0, 30.0),
    ([2, 4], [9000, 700], 7, 1, 16, 0, 0.0),
    ([1, 2], [9000, 9000], 12, 4, 0, 100, 0.0),
    ([1], [20000], 28, 4, 64, 5000, 0.0),                           # a window of a long history
    ([1, 1], [2000, 50], 9, 1, 0, 1, 2.0),
    ([77], [77], 4, 2, 0, 0, 0.0),
    ([9, 12, 11], [4000, 12, 700], 28, 4, 64, 0, 0.0),              # around half a tile of tokens
    ([10, 9, 8], [4000, 12, 700], 28, 4, 16, 0, 7.0),
    ([65, 66], [3000, 66], 2, 2, 0, 0, 0.0),
    ([300], [300], 28, 4, 128, 0, 0.0),
    ([129], [1300], 16, 1, 16, 0, 0.0),
    ([64, 0, 1, 200], [64, 50, 700, 900], 10, 2, 48, 0, 0.0),
    ([200, 37], [1000, 37], 6, 6, 0, 33, 0.0),                      # a window inside one tile
    ([150], [900], 14, 2, 64, 257, 20.0),
    ([260], [100], 2, 1, 0, 0, 0.0),                                # tokens 0..159 see no key
    ([700], [5000], 15, 5, 112, 1, 0.0),                            # each token sees itself only
    ([513], [2050], 13, 1, 0, 0, 5.0),
    ([1] * 700, [(37 * i) % 600 for i in range(700)], 4, 2, 0, 0, 0.0),     # more sequences than a block has threads
    ([i % 3 for i in range(900)], [(53 * i) % 300 for i in range(900)], 2, 1, 16, 0, 0.0),
    ([40] * 400, [40 + i % 90 for i in range(400)], 8, 8, 0, 0, 0.0),
    ([1] * 63 + [900], [700 + 9 * i for i in range(63)] + [900], 28, 4, 64, 0, 0.0),     # a prompt among single tokens
    ([1] * 90 + [70] + [1] * 20, [300 + 31 * i for i in range(90)] + [2000] + [1500] * 20, 28, 4, 16, 0, 0.0),     # the mean is below two
    ([3, 70], [600, 1500], 40, 40, 0, 0, 0.0),                      # many KV heads
    ([1], [512], 6, 2, 0, 0, 0.0),                                  # a cache of a few tiles, with rows past the length
    ([130], [515], 3, 3, 64, 0, 0.0),
    ([2, 90], [800, 700], 8, 2, 0, 0, 1e6),                         # a cap far above all scores
    ([2, 90], [800, 700], 8, 2, 0, 0, 1e-3),                        # and far below
    ([1, 1], [800, 700], 8, 2, 0, 0, 1e6),
    ([1, 1], [800, 700], 8, 2, 0, 0, 1e-3),
    ([1, 2], [800, 700], 8, 2, 0, 200, 1e-30),
    ([1, 2], [800, 700], 8, 2, 0, 0, 3e38),
    ([2, 90], [800, 700], 8, 2, 0, 200, 1e-30),
    ([2, 90], [800, 700], 8, 2, 0, (1 << 31) - 1, 0.0),             # a window wider than any history
    ([1, 1], [800, 700], 8, 2, 0, 1 << 23, 12.0),
]


def setup(n, lens, Hq, Hkv, page, seed, pad=2, qscale=2.0, strided=True, sizes=(0.05, 0.4)):
    g = gen(seed)
    T = sum(n)
    wide = normal(g, T + pad, Hq + 3, D, scale=qscale)
    q = wide[:, :Hq] if strided else wide[:, :Hq].contiguous()
    c = Cache(len(n), Hkv, max(max(lens), 1) + 7, page, seed=seed)  # rows past the lengths are NaN
    for b, L in enumerate(lens):
        c.put(b, packed(g, L, Hkv, sizes=sizes), packed(g, L, Hkv, sizes=sizes))
    return q, c


@pytest.mark.parametrize("n,lens,Hq,Hkv,page,window,cap", ATTEND)
def test_attention(n, lens, Hq, Hkv, page, window, cap):
    q, c = setup(n, lens, Hq, Hkv, page, sum(lens) + Hq)
    T = sum(n)
    wide = torch.full((T + 2, Hq + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")
    out, lse = wide[:, :Hq], torch.full((T + 2, Hq), 9.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    retopk.chunk_attention(q, c.h, i32(lens), out, cu_tokens=offsets(n), softcap=cap, window=window, lse=lse, status=st)
    assert st.item() == 0
    check(q, n, lens, c, out, lse, 1 / math.sqrt(D), cap, window)
    # rows behind the last sequence and columns beside the heads are as they were
    assert (wide[T:] == 9).all() and (lse[T:] == 9).all() and (wide[:, Hq:] == 9).all()


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 1, 1), (9, 1, 1), (16, 1, 1), (8, 1, 2), (6, 2, 5), (17, 17, 17), (8, 1, 3), (12, 2, 4), (5, 1, 5), (14, 2, 4),
                                      (32, 2, 2), (2, 1, 16), (11, 1, 3), (1, 1, 32), (1, 1, 33), (1, 1, 7), (10, 10, 9)])
@pytest.mark.parametrize("page,window,cap", [(0, 0, 0.0), (16, 0, 0.0), (64, 300, 0.0), (48, 0, 20.0)])
def test_attention_rows_by_the_tile(Hq, Hkv, n, page, window, cap):
    # 1 to 33 rows a sequence and head: tiles that are full, one row past, ragged by token; histories cut and joined, and
    # sequences with fewer tokens than the mean, or more
    n = [n, max(1, n - 1), n, 1, n + 2, 0]
    lens = [5003, 40, 1300, 7001, 1030, 77]
    q, c = setup(n, lens, Hq, Hkv, page, Hq + sum(n))
    lse = torch.full((sum(n) + 2, Hq), 9.0, device="cuda")
    out = retopk.chunk_attention(q, c.h, i32(lens), cu_tokens=offsets(n), softcap=cap, window=window, lse=lse)
    check(q, n, lens, c, out, lse, 1 / math.sqrt(D), cap, window)
    assert (lse[sum(n):] == 9).all()


@pytest.mark.parametrize("B,L", [(1, 260), (6, 1000)])
def test_attention_one_token_each_without_offsets(B, L):
    q, c = setup([1] * B, [L] * B, 8, 2, 0, B, pad=0, strided=False)
    out = retopk.chunk_attention(q, c.h, i32([L] * B), scale=0.3)
    check(q, [1] * B, [L] * B, c, out, None, 0.3, 0.0, 0)
    same = q.clone()
    assert retopk.chunk_attention(same, c.h, i32([L] * B), same, scale=0.3) is same      # out may be q
    assert torch.equal(same, out)


@pytest.mark.parametrize("n", [[1, 1], [1, 40]])
def test_attention_zero_scores_under_any_cap(n):
    L = [300, 600]
    q, c = setup(n, L, 8, 2, 0, 25)
    q.zero_()
    for cap in (1e-38, 1e-30, 1e-8, 3.0, 1e30, 3e38):
        out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n), softcap=cap)
        check(q, n, L, c, out, None, 1 / math.sqrt(D), 0.0, 0)     # all weights equal


@pytest.mark.parametrize("n", [[1, 1], [3, 2], [1, 40]])
@pytest.mark.parametrize("sizes", [(2.0 ** -15, 2.0 ** -11), (2.0 ** -12, 6000.0), (0.1, 0.1), (1.0, 60.0)])
def test_attention_scales_of_all_sizes(n, sizes):
    # small ones (among fp16's subnormals, code by scale), ones that differ by 2^24 within a row, large scores
    L = [600, 3100]
    q, c = setup(n, L, 14, 2, 0, 3, sizes=sizes)
    q.mul_(0.05 / sizes[1])
    lse = torch.empty((sum(n) + 2, 14), device="cuda")
    for scale in (None, 20.0):
        out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n), lse=lse, scale=scale)
        check(q, n, L, c, out, lse, scale or 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("n", [[1, 1], [1, 40]])
def test_attention_queries_of_all_sizes(n):
    # elements and rows that differ by far more than fp16 holds
    L = [500, 900]
    q, c = setup(n, L, 8, 2, 16, 5)
    size = torch.exp2(torch.randint(-60, 3, q.shape[:2] + (1,), generator=gen(6), device="cuda").float())
    q.mul_(size.to(torch.bfloat16))
    q[:, :, ::2] *= 2.0 ** -30
    out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n))
    check(q, n, L, c, out, None, 1 / math.sqrt(D), 0.0, 0)
    up = (q.float() * 2.0 ** 62).to(torch.bfloat16)       # the same scores from far larger queries
    out = retopk.chunk_attention(up, c.h, i32(L), cu_tokens=offsets(n), scale=2.0 ** -62 / math.sqrt(D))
    check(q, n, L, c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("n,L,window", [([200], [3000], 0), ([1], [9000], 0), ([90, 3], [2500, 6000], 700), ([1, 2], [9000, 2000], 1500)])
@pytest.mark.parametrize("cap", [0.0, 4.0, 30.0, 1000.0])
def test_attention_scores_whose_size_comes_and_goes(n, L, window, cap):
    # stretches of small and of large scores: maxima that jump and stay, capped ones far below the cap and at it by turns
    q, c = setup(n, L, 7, 1, 0, 33, qscale=1.0)
    for b, rows in enumerate(L):
        wave = torch.exp2(6 * torch.sin(torch.arange(rows, device="cuda") / 211.0) - 3)[:, None, None]
        codes, scales = packed(gen(34 + b), rows, 1, sizes=(0.3, 0.31))
        s = (scale_of(scales) * wave).half().view(torch.int16) >> 7
        c.put(b, (codes, s.to(torch.uint8)), packed(gen(36 + b), rows, 1))
    lse = torch.empty((sum(n) + 2, 7), device="cuda")
    out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n), softcap=cap, window=window, lse=lse)
    check(q, n, L, c, out, lse, 1 / math.sqrt(D), cap, window)


@pytest.mark.parametrize("n,L", [([1], [20000]), ([3], [20000]), ([200], [6000])])
def test_attention_scores_that_grow_along_the_history(n, L):
    q, c = setup(n, L, 8, 1, 0, 4, qscale=1.0)
    q.copy_(q.abs())
    ramp = torch.linspace(0.02, 0.6, L[0], device="cuda")[:, None, None]
    codes = torch.randint(0, 256, (L[0], 1, 64), generator=gen(9), device="cuda", dtype=torch.uint8) & 0x77      # no signs
    c.put(0, (codes, (ramp.expand(-1, 1, 8).half().view(torch.int16) >> 7).to(torch.uint8)), packed(gen(10), L[0], 1))
    out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n))
    check(q, n, L, c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("n", [1, 3, 30])
def test_attention_a_wide_tail_beside_a_peak(n):
    # one key of weight 1 and 60000 of 2^-21 .. 2^-18 with values of one sign: their sum is far from lost
    L = 60000
    q, c = setup([n], [L], 8, 1, 0, 7)
    q.fill_(0.125)
    codes = torch.full((L, 1, 64), 0x22, dtype=torch.uint8, device="cuda")      # ones
    scales = torch.full((L, 1, 8), 0, dtype=torch.uint8, device="cuda")
    scales[77] = 0x3c << 1                                                       # 1: a score of 16, times the scale
    c.put(0, (codes, scales), (codes, torch.full_like(scales, 0x3c << 1)))
    c.vs[0, 0, 77] = 0                                                           # the peak's own value: 0
    for scale in (14.0 / 16, 12.5 / 16):
        out = retopk.chunk_attention(q, c.h, i32([L]), cu_tokens=offsets([n]), scale=scale)
        check(q, [n], [L], c, out, None, scale, 0.0, 0)
        assert out[:n].float().mean() > 0.01


def test_attention_lengths_beyond_the_capacity_are_clamped():
    for n in ([1], [40]):
        q, c = setup(n, [64], 4, 1, 0, 12, pad=0)
        c.put(0, packed(gen(1), 71, 1), packed(gen(2), 71, 1))
        out = retopk.chunk_attention(q, c.h, i32([5000]), cu_tokens=offsets(n))
        check(q, n, [71], c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("cu,lens", [([0, 5, 3, 9], [50, 60, 70]), ([2, 4, 6, 40], [10, 20, 30]), ([0, 0, 0, 0], [9, 9, 9]), ([-4, 2, 7, 7], [9, -9, 3]),
                                     ([-(1 << 31), 2, (1 << 31) - 1, 9], [9, (1 << 31) - 1, -(1 << 31)]), ([0, 1, 2, 3], [90, 50, 100])])
@pytest.mark.parametrize("T", [9, 3])
def test_attention_odd_offsets_and_lengths_stay_inside(cu, lens, T):
    # offsets that decrease, leave tokens out or pass the last token; a negative length: no row outside is written
    q, _ = setup([T], [90], 8, 2, 16, 26, pad=0, strided=False)
    c = Cache(3, 2, 100, 16)
    for b in range(3):
        c.put(b, packed(gen(b), 112, 2), packed(gen(b + 9), 112, 2))
    out = torch.full((T + 2, 8, D), 9.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    retopk.chunk_attention(q, c.h, i32(lens), out[1:T + 1], cu_tokens=i32(cu), status=st)
    assert st.item() == 0 and (out[0] == 9).all() and (out[T + 1] == 9).all() and not out.isnan().any()
    flat = {t for b in range(3) for t in range(max(cu[b], 0), min(cu[b + 1], T))}
    for t in range(T):
        if t not in flat:
            assert (out[1 + t] == 9).all()


@pytest.mark.parametrize("n", [[1, 1], [30, 40]])
def test_attention_reports_bad_pages(n):
    q, c = setup(n, [100, 100], 4, 1, 16, 13, pad=0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: retopk.chunk_attention(q, c.h, i32([100, 100]), cu_tokens=offsets(n), status=st)  # noqa: E731
    good = call().clone()
    c.table[0, 2], c.table[0, 3] = c.k.shape[0], -7
    out = call()
    assert st.item() == retopk.STATUS_BAD_PAGE
    assert torch.equal(out[n[0]:], good[n[0]:]) and not out.isnan().any()


@pytest.mark.parametrize("n", [[1, 1], [20, 90]])
def test_attention_shared_pages(n):
    q, c = setup(n, [200, 150], 4, 2, 16, 14, pad=0)
    c.table[1, :9] = c.table[0, :9]
    out = retopk.chunk_attention(q, c.h, i32([200, 150]), cu_tokens=offsets(n))
    check(q, n, [200, 150], c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("n,L", [([1, 1], [301, 7001]), ([200, 3], [901, 2051])])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_queries_that_are_not_finite_stay_in_their_rows(n, L, cap, bad):
    q, c = setup(n, L, 14, 2, 64, 47, pad=0, qscale=6.0, strided=False)
    T = sum(n)
    hit = torch.zeros((T, 14), dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[n[0], 0] = hit[T - 1, 13] = True
    clean = q.clone()
    q[..., 5][hit] = bad
    lse = torch.empty((T, 14), device="cuda")
    out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n), lse=lse, softcap=cap)
    if math.isnan(bad):
        assert out[hit].isnan().all() and lse[hit].isnan().all()
    want = retopk.chunk_attention(clean, c.h, i32(L), cu_tokens=offsets(n), softcap=cap)
    assert ((out.float() - want.float()).abs()[~hit] <= 2.0 ** -7 * want.float().abs()[~hit] + 0.01).all() and lse[~hit].isfinite().all()


@pytest.mark.parametrize("n", [[1], [40]])
def test_attention_a_pool_past_2_31_elements(n):
    pages = 70000                                          # 64 bytes x 512 rows a page: 2.3e9
    k, v = (torch.zeros((pages, 1, 512, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, 1, 512, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    q, c = setup(n, [600], 4, 1, 0, 15, pad=0)
    for far, near in ((k, c.k), (v, c.v), (ks, c.ks), (vs, c.vs)):
        far[pages - 1, 0], far[3, 0, :88] = near[0, 0, :512], near[0, 0, 512:600]
    h = retopk.KVCache(k, v, table=i32([[pages - 1, 3]]), k_scale=ks, v_scale=vs)
    out = retopk.chunk_attention(q, h, i32([600]), cu_tokens=offsets(n))
    check(q, n, [600], c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("n", [[1, 1, 1], [3, 3, 3], [100, 1, 30]])
def test_attention_captured_follows_lengths_and_two_graphs_share_a_workspace(n):
    L = [700, 5000, 40]
    q, c = setup(n, L, 28, 4, 64, 21, pad=0, strided=False)
    T, lens, at = sum(n), i32(L), offsets(n)
    ws = torch.empty(retopk.chunk_attention_workspace_bytes(T, 3, 28, 4) + 256, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    call = lambda o: retopk.chunk_attention(q, c.h, lens, o, cu_tokens=at, workspace=ws)  # noqa: E731
    call(outs[0])
    graphs = []
    for o in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(o)
    for new in ([700, 5000, 40], [100, 4000, 30], [512, 64, 35]):
        lens.copy_(i32(new))
        for o in outs:
            o.fill_(7)
        for x in (0, 1, 0, 1):
            graphs[x].replay()
        for o in outs:
            check(q, n, new, c, o, None, 1 / math.sqrt(D), 0.0, 0)
    assert torch.equal(*outs)


@pytest.mark.parametrize("n", [[1] * 4, [2] * 4, [90] * 4])
def test_attention_on_another_stream_and_two_calls_at_once(n):
    L = [3000, 100, 2047, 901]
    q, c = setup(n, L, 8, 2, 0, 22, pad=0, strided=False)
    want = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n)).clone()
    lens, at = i32(L), offsets(n)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            got.append(retopk.chunk_attention(q, c.h, lens, cu_tokens=at, stream=s))
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x, want)      # the order of every sum follows from the lengths alone


def test_a_sequence_from_prompt_to_sparse_decoding():
    # a prompt and single tokens are appended in 4 bits and attended, then read back for the decode steps
    g, Hq, Hkv, n0, steps = gen(40), 8, 2, 200, 5
    c, flat = Cache(1, Hkv, 256, 16), Cache(1, Hkv, 256, 0, "bf16")
    sl, rope = i32([0]), retopk.QKRope(freqs(128), normal(g, D), normal(g, D))
    for n in [n0] + [1] * steps:
        x = normal(g, n, Hq + 2 * Hkv, D)
        q = retopk.qkv_append(rope, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], c.h, sl, cu_tokens=i32([0, n]))
        out = retopk.chunk_attention(q, c.h, sl, cu_tokens=i32([0, n]))
        check(q, [n], [sl.item()], c, out, None, 1 / math.sqrt(D), 0.0, 0)
    L = sl.item()
    assert L == n0 + steps
    retopk.cache_copy(c.h, flat.h, i32([0]), sl)
    for x, y in zip(flat.rows(0, L), c.rows(0, L)):
        assert torch.equal(x, y)
    again = retopk.chunk_attention(q, flat.h, sl)
    assert ((again.float() - out.float()).abs() <= 2.0 ** -6 * out.float().abs() + 2.0 ** -8).all()
    full = torch.empty((1, Hq, D), dtype=torch.bfloat16, device="cuda")
    retopk.exact_topk_attention_step(q, flat.k, flat.v, sl, 256, full)      # every key is among the best 256
    assert ((full.float() - out.float()).abs() <= 2.0 ** -6 * out.float().abs() + 2.0 ** -8).all()
