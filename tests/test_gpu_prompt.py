"""Rotated append, cache copy and chunk attention against plain 64-bit formulas (GPU).

Tolerances.  u = 2^-24 is half a step of fp32, half a step of bf16 is 2^-8 and of e4m3 2^-4, relative to the value.
  rotation   a' = a c - b s in fp32 from a norm of 128 terms: each of a, b is off by less than 16 u relative, c and s
             by 2^-22, so a' is off by at most 2^-19 (|a| + |b|) <= 2^-18 of the head's largest element; then one
             rounding to the output's type.
  attention  a score is a sum of 128 products, off by at most 128 u sum|q k| scale <= 2^-17 times that sum, and the
             exponential's argument and result by 2^-20 more: d; a capped score is off by no more.  The weights are rounded to bf16 once
             (2^-8), the output once more: |out - exact| <= 2^-8 |exact| + (2^-8 + 2 d + 2^-14) sum_j p_j |v_j|.
             lse is off by d + 2^-20 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

from top_sparse_attention_exact_gb300 import retopk

pytestmark = pytest.mark.gpu
D = 128


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


class Cache:
    """A cache of B sequences with `rows` capacity, contiguous or in shuffled pages, filled with `fill`."""

    def __init__(self, B, Hkv, rows, page=0, mx8=False, fill=float("nan"), seed=0):
        self.page, self.mx8 = page, mx8
        if page:
            width = -(-rows // page)
            perm = np.random.default_rng(seed).permutation(B * width + 2)[:B * width].reshape(B, width)
            self.table, shape = i32(perm), (B * width + 2, Hkv, page, D)
        else:
            self.table, shape = None, (B, Hkv, rows, D)
        if mx8:
            self.k, self.v = (torch.full(shape, 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.ks, self.vs = (torch.full(shape[:3] + (4,), 0x66, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.h = retopk.KVCache(self.k, self.v, table=self.table, k_scale=self.ks, v_scale=self.vs)
        else:
            self.k, self.v = (torch.full(shape, fill, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.ks = self.vs = None
            self.h = retopk.KVCache(self.k, self.v, table=self.table)

    def at(self, b, n):
        pos = torch.arange(n, device="cuda")
        return (self.table[b, pos // self.page].long(), pos % self.page) if self.page else (torch.full_like(pos, b), pos)

    def put(self, b, k, v):
        """Rows 0.. of sequence b (k, v: [n, Hkv, 128])."""
        p, r = self.at(b, k.shape[0])
        self.k[p, :, r], self.v[p, :, r] = k, v

    def rows(self, b, n):
        p, r = self.at(b, n)
        out = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            y = x[p, :, r]
            if self.mx8:
                y = value8(y, s[p, :, r])
            out.append(y.double())
        return out

    def snapshot(self):
        return [x.clone() for x in (self.k, self.v, self.ks, self.vs) if x is not None]


def value8(codes, scale):
    s = torch.ldexp(torch.ones((), dtype=torch.float64), scale.cpu().int() - 127).cuda()
    s = torch.where(scale == 255, torch.full_like(s, math.nan), s)
    return (codes.view(torch.float8_e4m3fn).double().unflatten(-1, (4, 32)) * s[..., None]).flatten(-2)


def scale8(x):
    """The smallest e with max|x| <= 448 * 2^e for each 32 values of fp64 rows, by search over exact powers."""
    top = x.unflatten(-1, (4, 32)).abs().amax(-1)
    e = torch.frexp(top / 448.0)
    return torch.where(top == 0, torch.full_like(e.exponent, -127),
                       torch.where(e.mantissa == 0.5, e.exponent - 1, e.exponent).clamp(min=-127))


# ---- rotated append --------------------------------------------------------------------------------------------------
def rotated(x, w, inv_freq, pos, interleaved, eps):
    """(exact rows, bound on the fp32 error) of [n, heads, 128] bf16 rows."""
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


def freqs(rot, theta=1e6):
    return (theta ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)).float()


APPEND = [  # tokens of each sequence, rows before, Hq, Hkv, page, rot, interleaved, norm, mx8
    ([1], [0], 28, 4, 0, 128, False, True, False),
    ([1], [8000000], 2, 1, 0, 128, False, True, False),            # a far position
    ([1, 1, 1], [5, 127, 128], 8, 8, 16, 128, True, True, True),
    ([7, 0, 1, 130], [0, 3, 16, 500], 7, 1, 48, 64, False, True, False),
    ([7, 0, 1, 130], [0, 3, 16, 500], 7, 1, 48, 64, True, False, True),
    ([300], [1], 32, 8, 0, 32, False, False, True),
    ([33, 65], [100, 31], 16, 1, 64, 16, False, True, True),
    ([20], [9], 3, 3, 32, 0, False, True, False),                  # norm alone
    ([20], [9], 1, 1, 0, 0, False, False, True),                   # quantisation alone
]


@pytest.mark.parametrize("n,start,Hq,Hkv,page,rot,inter,norm,mx8", APPEND)
@pytest.mark.parametrize("in_place", [False, True])
def test_append(n, start, Hq, Hkv, page, rot, inter, norm, mx8, in_place):
    g = gen(len(n) * 100 + Hq + rot)
    B, T = len(n), sum(n)
    pad = 3                                                        # rows behind the last sequence
    proj = normal(g, T + pad, (Hq + 2 * Hkv) * D, scale=2.0)
    q, k, v = (x.view(T + pad, -1, D) for x in proj.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    qw, kw = (normal(g, D) for _ in range(2)) if norm else (None, None)
    inv = freqs(rot) if rot else None
    c = Cache(B, Hkv, max(a + b for a, b in zip(n, start)) + 5, page, mx8, fill=3.0)
    before = c.snapshot()
    sl, st = i32(start), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sl if in_place else torch.full_like(sl, -1)
    qo = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rope = retopk.QKRope(inv, qw, kw, eps=1e-5, interleaved=inter)
    retopk.qkv_append(rope, q, k, v, c.h, sl, None if in_place else out, qo, cu_tokens=offsets(n), status=st)
    assert out.tolist() == [a + b for a, b in zip(n, start)] and st.item() == 0
    if not in_place:
        assert sl.tolist() == start
    assert (qo[T:] == 7).all()
    t0 = 0
    for b in range(B):
        sel = slice(t0, t0 + n[b])
        t0 += n[b]
        if n[b] == 0:
            continue
        pos = start[b] + torch.arange(n[b], device="cuda")
        ref, tol = rotated(q[sel], qw, inv, pos, inter, 1e-5)
        assert ((qo[sel].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + tol).all()
        ref, tol = rotated(k[sel], kw, inv, pos, inter, 1e-5)
        p, r = c.at(b, start[b] + n[b])
        p, r = p[start[b]:], r[start[b]:]
        if not mx8:
            assert ((c.k[p, :, r].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + tol).all()
            assert torch.equal(c.v[p, :, r].view(torch.int16), v[sel].contiguous().view(torch.int16))
            continue
        for x, exact, slack, codes, scale in ((k, ref, tol, c.k, c.ks), (v, v[sel].double(), 0.0 * tol, c.v, c.vs)):
            e = scale8(exact)
            near = ((scale8(exact * (1 + 2.0 ** -17)) != e) | (scale8(exact * (1 - 2.0 ** -17)) != e)) & (slack.amax() > 0)
            got = scale[p, :, r].int() - 127
            assert (got == e)[~near].all() and ((got - e).abs() <= 1).all()
            y = value8(codes[p, :, r], scale[p, :, r])
            step = torch.ldexp(torch.ones((), dtype=torch.float64), (got.cpu() - 10)).cuda().repeat_interleave(32, -1)
            assert ((y - exact).abs() <= torch.maximum(2.0 ** -4 * exact.abs(), step) * (1 + 2.0 ** -10) + slack).all()
    # what belongs to no new row is as it was
    for now, old in zip(c.snapshot(), before):
        for b in range(B):
            p, r = c.at(b, start[b] + n[b])
            now[p[start[b]:], :, r[start[b]:]] = old[p[start[b]:], :, r[start[b]:]]
        assert torch.equal(now.view(torch.uint8), old.view(torch.uint8))


def test_append_full_sequence_keeps_rows_and_length():
    g = gen(5)
    n, start = [4, 4, 4], [28, 29, 0]
    q, k, v = normal(g, 12, 4, D), normal(g, 12, 2, D), normal(g, 12, 2, D)
    c = Cache(3, 2, 32, 16, fill=1.0)
    sl, st = i32(start), torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = retopk.qkv_append(retopk.QKRope(freqs(128)), q, k, v, c.h, sl, cu_tokens=offsets(n), status=st)
    assert sl.tolist() == [32, 29, 4] and st.item() == retopk.STATUS_KV_FULL
    assert (c.rows(1, 32)[0] == 1).all() and (c.rows(1, 32)[1] == 1).all()
    ref, tol = rotated(q[4:8], None, freqs(128), 29 + torch.arange(4, device="cuda"), False, 0)
    assert ((qo[4:8].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + tol).all()


def test_append_keeps_out_of_bad_pages():
    g = gen(6)
    q, k, v = normal(g, 40, 2, D), normal(g, 40, 1, D), normal(g, 40, 1, D)
    c = Cache(2, 1, 48, 16, fill=1.0)
    good = c.table.clone()
    c.table[0, 1], c.table[1, 0] = c.k.shape[0], -1                # outside the pool on either side
    before, st = c.snapshot(), torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = i32([0, 0])
    retopk.qkv_append(retopk.QKRope(), q, k, v, c.h, sl, cu_tokens=offsets([33, 7]), status=st)
    assert st.item() == retopk.STATUS_BAD_PAGE and sl.tolist() == [33, 7]
    now = c.snapshot()
    for page in range(c.k.shape[0]):
        written = page in (good[0, 0].item(), good[0, 2].item())
        assert torch.equal(now[0][page], before[0][page]) != written


def test_append_of_blocks_that_are_not_finite_or_zero():
    g = gen(7)
    k, v, q = normal(g, 4, 1, D), normal(g, 4, 1, D), normal(g, 4, 1, D)
    v[0, 0, 3], v[1, 0, 40], v[2, 0, 64:96] = float("inf"), float("nan"), 0.0
    v[3, 0, :32] = 0
    v[3, 0, 5] = 2.0 ** -133                                        # the smallest bf16
    c = Cache(1, 1, 8, mx8=True)
    retopk.qkv_append(retopk.QKRope(), q, k, v, c.h, i32([0]), cu_tokens=offsets([4]))
    y = c.rows(0, 4)[1][:, 0]
    assert y[0, :32].isnan().all() and y[1, 32:64].isnan().all() and not y[0, 32:].isnan().any()
    assert (y[2, 64:96] == 0).all() and c.vs[0, 0, 2, 2] == 0 and c.vs[0, 0, 0, 0] == 255
    assert y[3, 5] == 2.0 ** -133 and (y[3, :5] == 0).all()


@pytest.mark.parametrize("inter", [False, True])
def test_an_infinity_stays_in_its_pair(inter):
    # without a norm an element reaches its partner of the rotation and no other
    k = torch.ones((2, 1, D), dtype=torch.bfloat16, device="cuda")
    k[0, 0, 100], k[1, 0, 3] = float("inf"), float("nan")
    c = Cache(2, 1, 8, fill=0.0)
    retopk.qkv_append(retopk.QKRope(freqs(64), interleaved=inter), k, k, k, c.h, i32([1, 1]))
    bad = lambda b: (~c.k[b, 0, 1].isfinite()).nonzero().flatten().tolist()  # noqa: E731
    assert bad(0) == [100] and bad(1) == ([2, 3] if inter else [3, 35])


def test_append_odd_offsets_and_lengths_stay_inside():
    for cu, start in (([0, 5, 3, 9], [3, 4, 5]), ([2, 4, 6, 40], [0, 1, 2]), ([-3, 2, 2, 8], [7, -2, 30]), ([9, 9, 9, 9], [1, 2, 3])):
        q = normal(gen(3), 9, 2, D)
        c = Cache(3, 2, 32, 16, fill=1.0)
        out = torch.full((11, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
        sl = i32([0, 0, 0, 77])
        retopk.qkv_append(retopk.QKRope(freqs(128)), q, q, q, c.h, i32(start), sl[:3], out[1:10], cu_tokens=i32(cu))
        assert (out[0] == 9).all() and (out[10] == 9).all() and sl[3] == 77


def test_append_offsets_and_lengths_at_the_ends_of_their_type():
    # differences of these pass 32 bits: no sequence whose tokens do not fit is written or advances
    low, high = -(1 << 31), (1 << 31) - 1
    for cu, start in (([low, 2, 4, 9], [3, 4, 5]), ([0, 2, 4, high], [3, high, 5]), ([low, high, high, high], [0, low, 2])):
        q = normal(gen(3), 9, 2, D)
        c = Cache(3, 2, 32, 16, fill=1.0)
        before, st = c.snapshot(), torch.zeros(1, dtype=torch.int32, device="cuda")
        out, sl = torch.full((11, 2, D), 9.0, dtype=torch.bfloat16, device="cuda"), i32([0, 0, 0, 77])
        retopk.qkv_append(retopk.QKRope(freqs(128)), q, q, q, c.h, i32(start), sl[:3], out[1:10], cu_tokens=i32(cu), status=st)
        fits = [s >= 0 and 0 <= b - a and s + b - a <= 32 for a, b, s in zip(cu, cu[1:], start)]
        assert sl.tolist() == [s + b - a if f else s for a, b, s, f in zip(cu, cu[1:], start, fits)] + [77]
        assert (out[0] == 9).all() and (out[10] == 9).all() and st.item() in (0, retopk.STATUS_KV_FULL)
        for b in range(3):      # pages of sequences that do not fit are as they were
            if not fits[b]:
                pages = c.table[b].long()
                assert all(torch.equal(x[pages], y[pages]) for x, y in zip(c.snapshot(), before))


def test_append_captured_and_replayed_advances_each_time():
    g = gen(31)
    B = 3
    q, k, v = normal(g, B, 4, D), normal(g, B, 2, D), normal(g, B, 2, D)
    c, sl, qo = Cache(B, 2, 40, fill=0.0), i32([0, 5, 38]), torch.empty((B, 4, D), dtype=torch.bfloat16, device="cuda")
    rope, st = retopk.QKRope(freqs(128)), torch.zeros(1, dtype=torch.int32, device="cuda")
    retopk.qkv_append(rope, q, k, v, c.h, sl, q_out=qo, status=st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        retopk.qkv_append(rope, q, k, v, c.h, sl, q_out=qo, status=st)
    for _ in range(3):
        graph.replay()
    assert sl.tolist() == [4, 9, 40] and st.item() == retopk.STATUS_KV_FULL
    for b, rows in enumerate((range(4), range(5, 9), range(38, 40))):
        for r in rows:
            assert torch.equal(c.v[b, :, r], v[b])


@pytest.mark.parametrize("rot,inter", [(128, False), (64, True)])
def test_qk_rope_is_appends_rows_and_works_in_place(rot, inter):
    g = gen(8)
    B, Hq, Hkv = 5, 14, 2
    q, k, v = normal(g, B, Hq, D), normal(g, B, Hkv, D), normal(g, B, Hkv, D)
    qw, kw = normal(g, D), normal(g, D)
    sl = i32([0, 1, 77, 4000, 12])
    rope = retopk.QKRope(freqs(rot), qw, kw, interleaved=inter)
    c = Cache(B, Hkv, 4096)
    qo = retopk.qkv_append(rope, q, k, v, c.h, sl, torch.empty_like(sl))
    q2, k2 = retopk.qk_rope(rope, q, k, sl)
    assert torch.equal(q2, qo)
    for b, pos in enumerate(sl.tolist()):
        assert torch.equal(k2[b], c.k[b, :, pos])
    retopk.qk_rope(rope, q, k, sl, q, k)
    assert torch.equal(q, q2) and torch.equal(k, k2)


@pytest.mark.parametrize("rot,inter,norm", [(128, False, True), (64, True, False), (32, False, True), (0, False, True)])
def test_qk_rope_of_ragged_tokens(rot, inter, norm):
    g = gen(11 + rot)
    n, start, Hq, Hkv = [7, 0, 1, 130, 33], [0, 3, 16, 500, 1 << 20], 28, 4
    T = sum(n)
    proj = normal(g, T + 3, (Hq + Hkv) * D, scale=2.0)
    q, k = (x.view(T + 3, -1, D) for x in proj.split([Hq * D, Hkv * D], dim=1))
    qw, kw = (normal(g, D) for _ in range(2)) if norm else (None, None)
    inv = freqs(rot) if rot else None
    qo, ko = (torch.full((T + 3, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for H in (Hq, Hkv))
    sl = i32(start)
    retopk.qk_rope(retopk.QKRope(inv, qw, kw, interleaved=inter), q, k, sl, qo, ko, cu_tokens=offsets(n))
    assert sl.tolist() == start and (qo[T:] == 7).all() and (ko[T:] == 7).all()
    t = 0
    for b in range(len(n)):
        sel, pos = slice(t, t + n[b]), start[b] + torch.arange(n[b], device="cuda")
        t += n[b]
        for x, w, out in ((q, qw, qo), (k, kw, ko)):
            ref, tol = rotated(x[sel], w, inv, pos, inter, 1e-6)
            assert ((out[sel].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + tol).all()


def test_append_nothing_moves_lengths_over():
    c = Cache(2, 2, 32)
    e = torch.empty((0, 4, D), dtype=torch.bfloat16, device="cuda")
    sl, out = i32([3, 9]), i32([0, 0])
    retopk.qkv_append(retopk.QKRope(), e, e[:, :2], e[:, :2], c.h, sl, out, cu_tokens=i32([0, 0, 0]))
    assert out.tolist() == [3, 9]


# ---- cache copy ------------------------------------------------------------------------------------------------------
def filled(g, B, Hkv, rows, page, mx8, seed):
    c = Cache(B, Hkv, rows, page, mx8, seed=seed)
    for x, s in ((c.k, c.ks), (c.v, c.vs)):
        if mx8:
            x.copy_(torch.randint(0, 256, x.shape, generator=g, device="cuda"))
            x[(x & 127) == 127] = 0                                 # the two NaN codes are never written
            s.copy_(torch.randint(0, 250, s.shape, generator=g, device="cuda"))
        else:
            size = torch.exp2(torch.randint(-40, 40, x.shape[:3] + (1,), generator=g, device="cuda").float())
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * size)
    return c


@pytest.mark.parametrize("src8,dst8", [(True, False), (False, True), (False, False), (True, True)])
@pytest.mark.parametrize("Hkv,sp,dp,first,last", [
    (1, 0, 0, [0], [1]), (4, 16, 0, [0, 5, 200], [300, 5, 201]), (2, 0, 48, [1, 130], [128, 263]), (3, 64, 256, [0], [1025]),
    (1, 128, 16, [7, 0, 0, 90], [90, 0, 513, 80])])
def test_copy(src8, dst8, Hkv, sp, dp, first, last):
    g = gen(sum(last) + Hkv)
    B = len(first)
    src = filled(g, B, Hkv, max(last) + 9, sp, src8, 1)
    dst = Cache(B, Hkv, max(last) + 2, dp, dst8, fill=2.0, seed=2)
    old = dst.snapshot()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    retopk.cache_copy(src.h, dst.h, i32(first), i32(last), max(1, max(l - f for f, l in zip(first, last))), status=st)
    assert st.item() == 0
    now = dst.snapshot()
    for b in range(B):
        f, l = first[b], max(first[b], last[b])
        (p, r), (u, w) = (x[f:l] for x in src.at(b, l)), (x[f:l] for x in dst.at(b, l))
        for x, xs, y, ys in ((src.k, src.ks, dst.k, dst.ks), (src.v, src.vs, dst.v, dst.vs)):
            if src8 == dst8:
                assert torch.equal(y[u, :, w].view(torch.uint8), x[p, :, r].view(torch.uint8))
                assert not src8 or torch.equal(ys[u, :, w], xs[p, :, r])
            elif src8:     # representable in bf16 but for the last bits of the smallest scales
                assert torch.equal(y[u, :, w], value8(x[p, :, r], xs[p, :, r]).to(torch.bfloat16))
            else:
                exact = x[p, :, r].double()
                e = scale8(exact)
                assert torch.equal(ys[u, :, w].int() - 127, e)
                one = torch.ldexp(torch.ones((), dtype=torch.float64), -e.cpu()).cuda().repeat_interleave(32, -1)
                assert torch.equal(y[u, :, w], (exact * one).float().to(torch.float8_e4m3fn).view(torch.uint8))
        for new, was in zip(now, old):
            new[u, :, w] = was[u, :, w]
    for new, was in zip(now, old):
        assert torch.equal(new.view(torch.uint8), was.view(torch.uint8))


def test_copy_stops_at_max_rows():
    src, dst = filled(gen(4), 2, 2, 300, 16, True, 1), Cache(2, 2, 300, fill=2.0)
    retopk.cache_copy(src.h, dst.h, i32([0, 100]), i32([300, 300]), 77)
    for b, f in enumerate((0, 100)):
        new, old = dst.rows(b, 300)[0], src.rows(b, 300)[0].to(torch.bfloat16).double()
        assert torch.equal(new[f:f + 77], old[f:f + 77]) and (new[:f] == 2).all() and (new[f + 77:] == 2).all()


def test_copy_reports_rows_out_of_range_and_bad_pages():
    src, dst = filled(gen(3), 2, 1, 64, 16, True, 1), Cache(2, 1, 40, fill=2.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    retopk.cache_copy(src.h, dst.h, i32([0, -3]), i32([60, 8]), 64, status=st)
    assert st.item() == retopk.STATUS_GATHER
    assert torch.equal(dst.rows(0, 40)[0], src.rows(0, 40)[0].to(torch.bfloat16).double())
    st.zero_()
    src.table[0, 0] = 1 << 30
    dst.k.fill_(2.0)
    retopk.cache_copy(src.h, dst.h, i32([0, 0]), i32([32, 0]), 64, status=st)
    assert st.item() == retopk.STATUS_BAD_PAGE
    assert (dst.k[0, 0, :16] == 2).all() and not (dst.k[0, 0, 16:32] == 2).all() and (dst.k[0, 0, 32:] == 2).all()


# ---- chunk attention -------------------------------------------------------------------------------------------------
def reference(q, k, v, first, scale, cap, window):
    """(out, lse, sum p|v|, score error) in fp64 of q [n, Hq, 128] at positions first.., over k, v [L, Hkv, 128]."""
    n, Hq, _ = q.shape
    L, Hkv, _ = k.shape
    q, k, v = q.double(), k.double().repeat_interleave(Hq // Hkv, 1), v.double().repeat_interleave(Hq // Hkv, 1)
    s = torch.einsum("ihd,jhd->hij", q, k) * scale
    size = torch.einsum("ihd,jhd->hij", q.abs(), k.abs()).amax((0, 1, 2)) * scale if L and n else torch.zeros(())
    if cap:
        s = cap * torch.tanh(s / cap)
    pos, j = first + torch.arange(n, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
    seen = (j <= pos) & ((j > pos - window) if window else torch.ones_like(j <= pos))
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if L else torch.full((Hq, n), -math.inf, dtype=torch.float64, device="cuda")
    p = torch.nan_to_num(torch.exp(s - lse[..., None]), nan=0.0)
    out, mass = (torch.einsum("hij,jhd->ihd", p, x) for x in (v, v.abs()))
    return out, lse.transpose(0, 1), mass, 2.0 ** -17 * float(size) + 2.0 ** -20


def check(q, qoff, n, lens, c, out, lse, scale, cap, window):
    t = qoff
    for b in range(len(n)):
        L = max(0, lens[b])
        k, v = c.rows(b, L)
        sel = slice(t, t + n[b])
        t += n[b]
        if n[b] == 0:
            continue
        ref, rl, mass, d = reference(q[sel], k, v, L - n[b], scale, cap, window)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * d + 2.0 ** -14) * mass
        err = (out[sel].double() - ref).abs()
        assert (err <= tol).all(), (b, float((err - tol).max()), float((err / (mass + 1e-30)).max()))
        if lse is not None:
            none = rl == -math.inf
            assert torch.equal(lse[sel] == -math.inf, none)
            assert ((lse[sel].double() - rl).abs() <= d + 2.0 ** -20 * (1 + rl.abs()))[~none].all()


ATTEND = [  # tokens of each sequence, rows in all, Hq, Hkv, page, window, cap
    ([1], [1], 1, 1, 0, 0, 0.0),                                    # a single key
    ([1], [300], 28, 4, 0, 0, 0.0),
    ([1], [129], 7, 1, 16, 0, 0.0),
    ([1] * 9, [1, 2, 127, 128, 129, 255, 256, 257, 1000], 16, 1, 48, 0, 0.0),
    ([1] * 5, [0, 5, 400, 17, 16], 32, 8, 64, 0, 50.0),             # a sequence without rows
    ([3] * 4, [3, 64, 500, 2], 8, 8, 0, 0, 0.0),                    # the last: fewer rows than tokens
    ([1, 1], [70001, 333], 28, 4, 256, 0, 0.0),                     # a long history beside a short one
    ([5], [40000], 16, 2, 0, 0, 30.0),
    ([1, 2], [9000, 9000], 12, 4, 0, 100, 0.0),
    ([77], [77], 4, 2, 0, 0, 0.0),
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
    ([3, 70], [600, 1500], 40, 40, 0, 0, 0.0),                      # many KV heads
    ([1], [512], 6, 2, 0, 0, 0.0),                                  # a cache of a few tiles, with rows past the length
    ([130], [515], 3, 3, 64, 0, 0.0),
    ([2, 90], [800, 700], 8, 2, 0, 0, 1e6),                         # a cap far above all scores
    ([2, 90], [800, 700], 8, 2, 0, 0, 1e-3),                        # and far below
    ([2, 90], [800, 700], 8, 2, 0, 200, 1e-30),
    ([2, 90], [800, 700], 8, 2, 0, (1 << 31) - 1, 0.0),             # a window wider than any history
    ([2, 90], [800, 700], 8, 2, 0, 1 << 23, 12.0),
]


def setup(n, lens, Hq, Hkv, page, seed, pad=2, qscale=2.0, strided=True):
    g = gen(seed)
    T = sum(n)
    wide = normal(g, T + pad, Hq + 3, D, scale=qscale)
    q = wide[:, :Hq] if strided else wide[:, :Hq].contiguous()
    c = Cache(len(n), Hkv, max(max(lens), 1) + 7, page, seed=seed)  # rows past the lengths are NaN
    for b, L in enumerate(lens):
        c.put(b, normal(g, L, Hkv, D), normal(g, L, Hkv, D))
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
    check(q, 0, n, lens, c, out, lse, 1 / math.sqrt(D), cap, window)
    # rows behind the last sequence and columns beside the heads are as they were
    assert (wide[T:] == 9).all() and (lse[T:] == 9).all() and (wide[:, Hq:] == 9).all()


@pytest.mark.parametrize("B,L", [(1, 260), (6, 1000)])
def test_attention_one_token_each_without_offsets(B, L):
    q, c = setup([1] * B, [L] * B, 8, 2, 0, B, pad=0, strided=False)
    out = retopk.chunk_attention(q, c.h, i32([L] * B), scale=0.3)
    check(q, 0, [1] * B, [L] * B, c, out, None, 0.3, 0.0, 0)


def test_attention_large_and_tiny_scores():
    # scores over a range of hundreds: one key takes all the weight; then all weights equal
    q, c = setup([1, 40], [600, 600], 8, 2, 0, 3, qscale=60.0)
    lse = torch.empty((43, 8), device="cuda")
    out = retopk.chunk_attention(q, c.h, i32([600, 600]), cu_tokens=offsets([1, 40]), lse=lse)
    check(q, 0, [1, 40], [600, 600], c, out, lse, 1 / math.sqrt(D), 0.0, 0)
    zero = torch.zeros_like(q)
    out = retopk.chunk_attention(zero, c.h, i32([600, 600]), cu_tokens=offsets([1, 40]), lse=lse)
    check(zero, 0, [1, 40], [600, 600], c, out, lse, 1 / math.sqrt(D), 0.0, 0)


def test_attention_scores_that_grow_along_the_history():
    # every later tile raises the running maximum, so the accumulators are rescaled all along
    n, L, Hq, Hkv = [200], [3000], 8, 1
    q, c = setup(n, L, Hq, Hkv, 0, 4, qscale=1.0)
    ramp = torch.linspace(0, 4, L[0], device="cuda")[:, None, None]
    q.copy_(q.abs())
    k = (torch.rand((L[0], Hkv, D), generator=gen(9), device="cuda") * ramp).to(torch.bfloat16)
    c.put(0, k, normal(gen(10), L[0], Hkv, D))
    out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n))
    check(q, 0, n, L, c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("n,L,window", [([200], [3000], 0), ([1], [9000], 0), ([90, 3], [2500, 6000], 700)])
@pytest.mark.parametrize("cap", [0.0, 4.0, 30.0, 1000.0])
def test_attention_scores_whose_size_comes_and_goes(n, L, window, cap):
    # stretches of small and of large scores: far below the cap and at it by turns, maxima that jump and stay
    q, c = setup(n, L, 7, 1, 0, 33, qscale=1.0)
    for b, rows in enumerate(L):
        wave = torch.exp2(6 * torch.sin(torch.arange(rows, device="cuda") / 211.0) - 3)[:, None, None]
        c.put(b, (normal(gen(34 + b), rows, 1, D) * wave).to(torch.bfloat16), normal(gen(36 + b), rows, 1, D))
    lse = torch.empty((sum(n) + 2, 7), device="cuda")
    out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n), softcap=cap, window=window, lse=lse)
    check(q, 0, n, L, c, out, lse, 1 / math.sqrt(D), cap, window)


def test_attention_lengths_beyond_the_capacity_are_clamped():
    q, c = setup([1], [64], 4, 1, 0, 12, pad=0)
    c.put(0, normal(gen(1), 71, 1, D), normal(gen(2), 71, 1, D))
    out = retopk.chunk_attention(q, c.h, i32([5000]))
    check(q, 0, [1], [71], c, out, None, 1 / math.sqrt(D), 0.0, 0)


def test_attention_zero_scores_under_a_tiny_cap():
    q, c = setup([1, 40], [300, 600], 8, 2, 0, 25)
    q.zero_()
    for cap in (1e-30, 1e-8, 3.0, 1e30):
        out = retopk.chunk_attention(q, c.h, i32([300, 600]), cu_tokens=offsets([1, 40]), softcap=cap)
        check(q, 0, [1, 40], [300, 600], c, out, None, 1 / math.sqrt(D), 0.0, 0)     # all weights equal


@pytest.mark.parametrize("cu,lens", [([0, 5, 3, 9], [50, 60, 70]), ([2, 4, 6, 40], [10, 20, 30]), ([0, 0, 0, 0], [9, 9, 9]), ([-4, 2, 7, 7], [9, -9, 3])])
def test_attention_odd_offsets_and_lengths_stay_inside(cu, lens):
    # offsets that decrease, leave tokens out or pass the last token; a negative length: no row outside is written
    q, c = setup([9], [90], 8, 2, 16, 26, pad=0, strided=False)
    c = Cache(3, 2, 100, 16, fill=0.5)
    out = torch.full((11, 8, D), 9.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    retopk.chunk_attention(q, c.h, i32(lens), out[1:10], cu_tokens=i32(cu), status=st)
    assert st.item() == 0 and (out[0] == 9).all() and (out[10] == 9).all() and not out.isnan().any()
    flat = sorted({t for b in range(3) for t in range(max(cu[b], 0), min(cu[b + 1], 9))})
    for t in range(9):
        if t not in flat:
            assert (out[1 + t] == 9).all()


def test_attention_reports_bad_pages():
    q, c = setup([1, 1], [100, 100], 4, 1, 16, 13, pad=0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = retopk.chunk_attention(q, c.h, i32([100, 100]), status=st).clone()
    c.table[0, 2], c.table[0, 3] = c.k.shape[0], -7
    out = retopk.chunk_attention(q, c.h, i32([100, 100]), status=st)
    assert st.item() == retopk.STATUS_BAD_PAGE
    assert torch.equal(out[1], good[1]) and not out.isnan().any()


def test_attention_shared_pages():
    # two sequences with the same first pages
    q, c = setup([1, 1], [200, 150], 4, 2, 16, 14, pad=0)
    c.table[1, :9] = c.table[0, :9]
    out = retopk.chunk_attention(q, c.h, i32([200, 150]))
    check(q, 0, [1, 1], [200, 150], c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("Hq,Hkv", [(7, 1), (28, 4), (3, 1), (16, 1)])
@pytest.mark.parametrize("n,page", [(1, 0), (1, 16), (2, 48), (30, 0)])
@pytest.mark.parametrize("tail", [float("nan"), float("inf")])
def test_attention_past_the_length_in_tiles_that_some_warps_have_no_token_for(Hq, Hkv, n, page, tail):
    # The last tile ends among keys 32..63: values past the length there are cleared by lanes whose warp may have no
    # row of its own (few heads, few tokens), and reach the product's first half.
    lens = [33, 44, 47, 63, 128 + 34, 256 + 44, 384 + 61, 1280 + 50]
    q, c = setup([n] * len(lens), lens, Hq, Hkv, page, 41 + n + Hq)
    for x in (c.k, c.v):
        x.copy_(torch.where(x.isnan(), torch.full_like(x, tail), x))
    lse = torch.empty((len(lens) * n + 2, Hq), device="cuda")
    out = retopk.chunk_attention(q, c.h, i32(lens), cu_tokens=offsets([n] * len(lens)), lse=lse)
    check(q, 0, [n] * len(lens), lens, c, out, lse, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("Hq,Hkv", [(7, 1), (28, 4), (16, 1)])
@pytest.mark.parametrize("n,page,window", [(1, 0, 0), (1, 16, 100), (3, 48, 0), (40, 0, 0), (64, 16, 57)])
@pytest.mark.parametrize("cap", [5.0, 1e-3])
def test_attention_capped_scores_beside_keys_past_the_length(Hq, Hkv, n, page, window, cap):
    # Scores past half the cap, and lengths that end between two neighbouring keys: the last key, and each token's own,
    # have a hidden one beside them, whose score is NaN or infinite where it lies past the length.
    lens = [n, 129, 301, 128 + 33, 256 + 63, 2051]
    q, c = setup([n] * len(lens), lens, Hq, Hkv, page, 43 + n + Hq, qscale=6.0)
    lse = torch.empty((len(lens) * n + 2, Hq), device="cuda")
    for tail in (float("nan"), float("inf"), -float("inf")):
        for x in (c.k, c.v):
            x.copy_(torch.where(x.isfinite(), x, torch.full_like(x, tail)))
        out = retopk.chunk_attention(q, c.h, i32(lens), cu_tokens=offsets([n] * len(lens)), softcap=cap, window=window, lse=lse)
        check(q, 0, [n] * len(lens), lens, c, out, lse, 1 / math.sqrt(D), cap, window)


@pytest.mark.parametrize("n,L", [([1, 1], [301, 7001]), ([200, 3], [901, 2051])])
def test_attention_capped_queries_that_are_not_finite_stay_in_their_rows(n, L):
    # the same of scores past half the cap, with odd lengths and NaN behind them: rows of such a query are NaN, no others
    q, c = setup(n, L, 14, 2, 64, 47, pad=0, qscale=6.0, strided=False)
    T, at, lens = sum(n), offsets(n), i32(L)
    hit = torch.zeros((T, 14), dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[n[0], 0] = hit[T - 1, 13] = True
    clean = q.clone()
    q[hit] = float("nan")
    lse = torch.empty((T, 14), device="cuda")
    for cap in (5.0, 1e-3):
        out = retopk.chunk_attention(q, c.h, lens, cu_tokens=at, lse=lse, softcap=cap)
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        t = 0
        for b in range(len(n)):
            sel, rows = slice(t, t + n[b]), c.rows(b, L[b])
            t += n[b]
            ref, rl, mass, d = reference(clean[sel], *rows, L[b] - n[b], 1 / math.sqrt(D), cap, 0)
            bad = (out[sel].double() - ref).abs() > 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * d + 2.0 ** -14) * mass
            off = (lse[sel].double() - rl).abs() > d + 2.0 ** -20 * (1 + rl.abs())
            assert not out[sel][~hit[sel]].isnan().any() and not lse[sel][~hit[sel]].isnan().any()
            assert not bad[~hit[sel]].any() and not off[~hit[sel]].any()


def test_attention_captured_and_replayed_with_new_lengths():
    lens, n = [900, 333], [1, 1]
    q, c = setup(n, lens, 28, 4, 64, 15, pad=0, strided=False)
    sl, out = i32([10, 20]), torch.empty_like(q)
    ws = torch.empty(retopk.chunk_attention_workspace_bytes(2, 2, 28, 4) + 256, dtype=torch.uint8, device="cuda")
    retopk.chunk_attention(q, c.h, sl, out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        retopk.chunk_attention(q, c.h, sl, out, workspace=ws)
        retopk.chunk_attention(q, c.h, sl, out, workspace=ws)      # the same workspace, one after another
    for L in (lens, [1, 2], [129, 128]):
        sl.copy_(i32(L))
        out.fill_(9.0)
        g.replay()
        for b in range(2):
            k, v = c.rows(b, L[b])
            ref, _, mass, d = reference(q[b:b + 1], k, v, L[b] - 1, 1 / math.sqrt(D), 0.0, 0)
            assert ((out[b:b + 1].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * d + 2.0 ** -14) * mass).all()


def test_attention_on_two_streams_at_once():
    a, b = setup([1, 1], [5000, 100], 28, 4, 0, 16, pad=0), setup([300], [2000], 8, 8, 128, 17, pad=0)
    la, lb, cu = i32([5000, 100]), i32([2000]), offsets([300])
    one = [retopk.chunk_attention(a[0], a[1].h, la).clone(), retopk.chunk_attention(b[0], b[1].h, lb, cu_tokens=cu).clone()]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        x = retopk.chunk_attention(a[0], a[1].h, la, stream=s[0])
        y = retopk.chunk_attention(b[0], b[1].h, lb, cu_tokens=cu, stream=s[1])
        torch.cuda.synchronize()
        assert torch.equal(x, one[0]) and torch.equal(y, one[1])


def test_attention_repeats_bit_for_bit():
    q, c = setup([1, 90, 4], [30000, 2000, 700], 28, 4, 64, 18)
    cu, sl = offsets([1, 90, 4]), i32([30000, 2000, 700])
    first = retopk.chunk_attention(q, c.h, sl, cu_tokens=cu)[:95].clone()
    for _ in range(4):
        assert torch.equal(retopk.chunk_attention(q, c.h, sl, cu_tokens=cu)[:95], first)


@pytest.mark.parametrize("n,L", [([1, 1, 1], [300, 70000, 5]), ([200, 1, 40], [900, 20000, 700])])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_attention_of_queries_that_are_not_finite_stays_in_their_rows(n, L, cap):
    q, c = setup(n, L, 14, 2, 64, 31, pad=0, strided=False)
    T, at, lens = sum(n), offsets(n), i32(L)
    lse, lse2 = (torch.empty((T, 14), device="cuda") for _ in range(2))
    good = retopk.chunk_attention(q, c.h, lens, cu_tokens=at, lse=lse, softcap=cap)
    bad = q.clone()
    rows = [(0, 3), (n[0], 0), (T - 1, 13)]     # one in each sequence: whole, cut and short histories
    for t, h in rows:
        bad[t, h] = float("nan")
    out = retopk.chunk_attention(bad, c.h, lens, cu_tokens=at, lse=lse2, softcap=cap)
    hit = torch.zeros((T, 14), dtype=torch.bool, device="cuda")
    for t, h in rows:
        hit[t, h] = True
    assert out[hit].isnan().all() and lse2[hit].isnan().all()
    # the rows beside them may take another way to the same sums, so they are held to the formula
    check(q, 0, n, L, c, torch.where(hit[..., None], good, out), torch.where(hit, lse, lse2), 1 / math.sqrt(D), cap, 0)


@pytest.mark.parametrize("n,L", [([1, 1], [300, 70000]), ([300, 40], [3000, 4000])])
def test_attention_into_its_queries(n, L):
    q, c = setup(n, L, 28, 4, 0, 32, pad=0)
    at, lens = offsets(n), i32(L)
    want = retopk.chunk_attention(q, c.h, lens, cu_tokens=at)
    assert torch.equal(retopk.chunk_attention(q, c.h, lens, q, cu_tokens=at), want)


@pytest.mark.parametrize("n,L", [([1, 1], [300, 7000]), ([300, 40], [900, 400])])
def test_attention_between_its_queries(n, L):
    # queries and outputs by turns in the rows of one buffer
    q, c = setup(n, L, 28, 4, 0, 33, pad=0)
    T, at, lens = sum(n), offsets(n), i32(L)
    want = retopk.chunk_attention(q, c.h, lens, cu_tokens=at)
    for first, second in ((0, 28), (28, 0)):
        both = torch.zeros((T, 56, D), dtype=torch.bfloat16, device="cuda")
        x, y = both[:, first:first + 28], both[:, second:second + 28]
        x.copy_(q)
        assert torch.equal(retopk.chunk_attention(x, c.h, lens, y, cu_tokens=at), want) and torch.equal(x, q)


def test_numbers_beyond_32_bits_are_not_taken_for_others():
    q, c = setup([1], [600], 4, 1, 0, 20, pad=0)
    lens, flat = i32([600]), Cache(1, 1, 600, fill=0.0)
    want = retopk.chunk_attention(q, c.h, lens)
    assert torch.equal(retopk.chunk_attention(q, c.h, lens, window=(1 << 32) + 5), want)
    for kw in (dict(window=-(1 << 32)), dict(softcap=1e-50), dict(scale=1e-50), dict(softcap=1e39), dict(scale=-1.0)):
        with pytest.raises(retopk.RetopkError):
            retopk.chunk_attention(q, c.h, lens, **kw)
    for rows in ((1 << 32) + 5, -(1 << 32) + 5):
        with pytest.raises(retopk.RetopkError):
            retopk.cache_copy(c.h, flat.h, i32([0]), lens, rows)


@pytest.mark.parametrize("n,L,Hq,Hkv,page", [([1], [70001], 28, 4, 0), ([1, 1], [40000, 30001], 16, 1, 16), ([40], [20011], 7, 1, 48),
                                             ([3, 9], [9000, 25003], 8, 8, 0), ([300], [8300], 28, 4, 64)])
def test_attention_counts_every_tile_of_a_long_history_once(n, L, Hq, Hkv, page):
    # Column d of V is 1 in one tile of 128 keys and 0 elsewhere, other tiles each time: an output is that tile's share of
    # the weights, and its bound is relative to it.
    q, c = setup(n, L, Hq, Hkv, page, 50, pad=0, qscale=0.5)
    at, lens = offsets(n), i32(L)
    for first in range(0, -(-max(L) // 128), D):
        for b, rows in enumerate(L):
            tile = torch.arange(rows, device="cuda") // 128 - first
            p, r = c.at(b, rows)
            c.v[p, :, r] = (tile[:, None] == torch.arange(D, device="cuda")).to(torch.bfloat16)[:, None]
        out = retopk.chunk_attention(q, c.h, lens, cu_tokens=at)
        check(q, 0, n, L, c, out, None, 1 / math.sqrt(D), 0.0, 0)


@pytest.mark.parametrize("n,L", [([600] + [1] * 40, [700] + [50 * i for i in range(1, 41)]), ([1] * 20 + [1500], [900] * 20 + [1700]),
                                 ([2049], [2049]), ([1] * 30 + [64, 257], [100 * i for i in range(30)] + [64, 3001])])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_attention_of_prompts_among_single_tokens(n, L, cap):
    q, c = setup(n, L, 14, 2, 48, 51)
    lse = torch.empty((sum(n) + 2, 14), device="cuda")
    out = retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n), softcap=cap, lse=lse)
    check(q, 0, n, L, c, out, lse, 1 / math.sqrt(D), cap, 0)


def test_attention_of_several_batches_in_one_workspace():
    # the largest call's workspace serves smaller ones, with more and with fewer sequences
    ws = torch.empty(retopk.chunk_attention_workspace_bytes(900, 512, 28, 4) + 256, dtype=torch.uint8, device="cuda")
    calls = []
    for i, (n, L) in enumerate((([3] * 300, [60 + i for i in range(300)]), ([900], [2000]), ([1], [30000]), ([20, 5], [4000, 900]))):
        q, c = setup(n, L, 28, 4, 16, 60 + i, pad=0)
        calls.append((q, c, i32(L), offsets(n), retopk.chunk_attention(q, c.h, i32(L), cu_tokens=offsets(n))))
    graphs = []
    for q, c, lens, at, want in calls:
        out = torch.empty_like(want)
        assert torch.equal(retopk.chunk_attention(q, c.h, lens, out, cu_tokens=at, workspace=ws), want)
        graphs.append((torch.cuda.CUDAGraph(), out))
        with torch.cuda.graph(graphs[-1][0]):
            retopk.chunk_attention(q, c.h, lens, out, cu_tokens=at, workspace=ws)
    for _ in range(2):      # captured calls that share it, one behind the other
        for g, out in graphs:
            out.zero_()
            g.replay()
        for (g, out), call in zip(graphs, calls):
            assert torch.equal(out, call[4])


def test_calls_refuse_tensors_elsewhere():
    q, c = setup([1], [10], 4, 1, 0, 19, pad=0)
    with pytest.raises(retopk.RetopkError):
        retopk.chunk_attention(q.cpu(), c.h, i32([10]))
    with pytest.raises(retopk.RetopkError):
        retopk.chunk_attention(q, c.h, i32([10]).cpu())
    with pytest.raises(retopk.RetopkError):
        retopk.chunk_attention(q, c.h, i32([10]), lse=torch.empty((2, 4), device="cuda"))
    with pytest.raises(retopk.RetopkError):
        retopk.chunk_attention(q, c.h, i32([10]), workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24))


# ---- far offsets -------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("contiguous", [False, True])
def test_rows_past_two_to_the_31_elements(contiguous):
    """Appended, attended, parked and read back in pools of more than 2^31 elements, in their last pages."""
    g = gen(70)
    Hq, n = 8, [40, 3]
    if contiguous:      # sequences 0 and 2 lie below, 1 (and the last rows of 2) beyond
        B, Hkv, page, rows, start = 3, 1, 0, 1 << 23, [5, 7, (1 << 23) - 40]
        n, pages, table = [3, 40, 40], 3, None
    else:
        B, Hkv, page, rows, start = 2, 4, 256, 1024, [500, 250]
        pages = (1 << 31) // (Hkv * page * D) + 9
        table = i32([[pages - 1 - 2 * i, pages - 2 - 2 * i][b] for b in range(2) for i in range(4)]).view(2, 4)
    T, last = sum(n), [a + b for a, b in zip(start, n)]
    shape = (pages, Hkv, page or rows, D)
    assert pages * Hkv * (page or rows) * D > 1 << 31
    kv = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c = Cache.__new__(Cache)
    c.page, c.mx8, c.table, c.k, c.v, c.ks, c.vs = page, False, table, kv[0], kv[1], None, None
    c.h = retopk.KVCache(*kv, table=table)
    q, k, v = normal(g, T, Hq, D), normal(g, T, Hkv, D), normal(g, T, Hkv, D)
    sl, at, st = i32(start), offsets(n), torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = retopk.QKRope()      # (rows as they are)
    retopk.qkv_append(rope, q, k, v, c.h, sl, cu_tokens=at, status=st)
    assert sl.tolist() == last and st.item() == 0
    new = [slice(a - b, a) for a, b in zip(np.cumsum(n).tolist(), n)]

    def place(b):
        pos = torch.arange(start[b], last[b], device="cuda")
        return (table[b, pos // page].long(), pos % page) if page else (torch.full_like(pos, b), pos)

    for b in range(B):
        p, r = place(b)
        assert torch.equal(c.k[p, :, r], k[new[b]]) and torch.equal(c.v[p, :, r], v[new[b]])
    out = retopk.chunk_attention(q, c.h, sl, cu_tokens=at, window=30)
    for b in range(B):      # rows before the new ones are zeros: 29 of them, where there are as many
        zeros = torch.zeros((min(start[b], 29), Hkv, D), dtype=torch.bfloat16, device="cuda")
        ref, _, mass, d = reference(q[new[b]], torch.cat([zeros, k[new[b]]]), torch.cat([zeros, v[new[b]]]), len(zeros), 1 / math.sqrt(D), 0.0, 30)
        assert ((out[new[b]].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * d + 2.0 ** -14) * mass).all()
    codes = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(shape[:3] + (4,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    parked = retopk.KVCache(*codes, table=table, k_scale=scales[0], v_scale=scales[1])
    retopk.cache_copy(c.h, parked, i32(start), sl, 64, status=st)
    for x in kv:
        x.zero_()
    retopk.cache_copy(parked, c.h, i32(start), sl, 64, status=st)
    again = [[x[p, :, r].clone() for x in kv] for p, r in map(place, range(B))]
    for b in range(B):
        for x, y in zip(again[b], (k[new[b]], v[new[b]])):
            top = y.double().unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, 4, 32).flatten(-2)
            assert ((x.double() - y.double()).abs() <= torch.maximum(2.0 ** -4 * y.double().abs(), top * 2.0 ** -17)).all()
    # the same rows from the 8-bit append
    for x in codes + scales + kv:
        x.zero_()
    retopk.qkv_append(rope, q, k, v, parked, i32(start), cu_tokens=at, status=st)
    retopk.cache_copy(parked, c.h, i32(start), sl, 64, status=st)
    assert st.item() == 0
    for b in range(B):
        assert all(torch.equal(x[place(b)[0], :, place(b)[1]], y) for x, y in zip(kv, again[b]))


# ---- together --------------------------------------------------------------------------------------------------------
def test_prompt_in_chunks_then_sparse_decoding():
    """A prompt is appended to pages and attended in chunks, gathered into the contiguous cache, and decoded with
    retopk_decode_step_kv; the sequence is then parked in 8 bits and read back."""
    g = gen(21)
    B, Hq, Hkv, L0, K, C = 2, 8, 2, 700, 2000, 8
    w = (torch.randn(2, D, generator=g, device="cuda") * 0.1 + 1).to(torch.bfloat16)
    rope = retopk.QKRope(freqs(128, 1e4), w[0], w[1])
    paged = Cache(B, Hkv, 800, 48, fill=0.0)
    proj = normal(g, L0 + 4, B, (Hq + 2 * Hkv) * D)
    sl = i32([0] * B)
    qs = []
    for f, l in ((0, 333), (333, 334), (334, 700)):
        x = proj[f:l].transpose(0, 1).reshape(B * (l - f), -1)
        q, k, v = (y.view(x.shape[0], -1, D) for y in x.split([Hq * D, Hkv * D, Hkv * D], dim=1))
        cu = offsets([l - f] * B)
        qr = retopk.qkv_append(rope, q, k, v, paged.h, sl, cu_tokens=cu)
        out = retopk.chunk_attention(qr, paged.h, sl, cu_tokens=cu)
        check(qr, 0, [l - f] * B, [l] * B, paged, out, None, 1 / math.sqrt(D), 0.0, 0)
        qs.append(qr.view(B, l - f, Hq, D))
    assert sl.tolist() == [L0] * B
    flat = Cache(B, Hkv, 800, fill=0.0)
    retopk.cache_copy(paged.h, flat.h, i32([0] * B), sl, 800)
    for b in range(B):
        assert all(torch.equal(x, y) for x, y in zip(paged.rows(b, L0), flat.rows(b, L0)))
    # with K beyond every length the sparse step is dense attention: the two agree
    ctx = retopk.ReTopK(B, Hq, Hkv, 800, K=K, C=C, W=8, R=2, T_r=1, tau=2.0)
    q_last = torch.cat(qs, 1)[:, -C:].transpose(1, 2).contiguous()
    ctx.retopk_init_cache(q_last, flat.k, sl)
    for t in range(4):
        x = proj[L0 + t].view(B, Hq + 2 * Hkv, D)
        q, k = retopk.qk_rope(rope, x[:, :Hq], x[:, Hq:Hq + Hkv], sl)
        sparse = torch.empty_like(q)
        ctx.retopk_decode_step_kv(k, x[:, Hq + Hkv:].contiguous(), q, flat.k, flat.v, sl, sparse)
        dense = retopk.chunk_attention(q, flat.h, sl)
        check(q, 0, [1] * B, [L0 + t + 1] * B, flat, dense, None, 1 / math.sqrt(D), 0.0, 0)
        check(q, 0, [1] * B, [L0 + t + 1] * B, flat, sparse, None, 1 / math.sqrt(D), 0.0, 0)
    parked, back = Cache(B, Hkv, 800, 64, mx8=True, seed=5), Cache(B, Hkv, 800, fill=0.0)
    zero = i32([0] * B)
    retopk.cache_copy(flat.h, parked.h, zero, sl, 800)
    retopk.cache_copy(parked.h, back.h, zero, sl, 800)
    for b in range(B):
        for x, y in zip(flat.rows(b, L0 + 4), back.rows(b, L0 + 4)):
            top = x.unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, 4, 32).flatten(-2)
            assert ((x - y).abs() <= torch.maximum(2.0 ** -4 * x.abs(), top * 2.0 ** -17)).all()
