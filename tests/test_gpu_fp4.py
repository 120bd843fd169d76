"""The 4-bit cache (RETOPK_CACHE_FP4): rotated append into it and copies from and to it, against plain 64-bit
formulas (GPU).

Tolerances.  u = 2^-24 is half a step of fp32, half a step of bf16 is 2^-8 relative to the value.
  codes      of values that are exact (values, bf16 rows) scale and codes have one right answer: ties go to even.
             A rotated key is off by at most 2^-18 of the head's largest element (see the prompt-side tests): its
             scale may be a neighbour of the right one only where a sixth of the largest lies that near the border, its
             code is off by at most half the codes' gap and that error.
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
