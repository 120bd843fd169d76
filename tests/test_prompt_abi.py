"""Refusals of the prompt-side entry points: answered on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from top_sparse_attention_exact_gb300 import retopk

P = 1 << 20     # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    return retopk.load()


def cache(**kw):
    d = dict(k=P, v=P, k_scale=None, v_scale=None, table=None, format=0, n_pages=2, n_kv_heads=4, page_rows=100, table_width=0)
    d.update(kw)
    return retopk.retopk_cache(*[d[f] for f, _ in retopk.retopk_cache._fields_])


def rope(**kw):
    d = dict(q_weight=None, k_weight=None, inv_freq=P, eps=1e-6, rot_dim=128, interleaved=0)
    d.update(kw)
    return retopk.retopk_rope(*[d[f] for f, _ in retopk.retopk_rope._fields_])


def append(lib, r=None, c=None, T=2, B=2, Hq=8, q=P, qs=1024, k=P, ks=512, v=P, vs=512, cu=None, sl=P, so=P, qo=P + 4096, st=None):
    r, c = r or rope(), c or cache()
    return lib.retopk_qkv_append(ctypes.addressof(r), q, qs, k, ks, v, vs, cu, T, B, Hq, ctypes.addressof(c), sl, so, qo, st, None)


def attend(lib, c=None, q=P, qs=1024, cu=None, T=2, B=2, Hq=8, sl=P, scale=0.0, cap=0.0, window=0, out=P, os=1024, lse=None, ws=P, n=None):
    c = c or cache()
    n = lib.retopk_chunk_attention_workspace_bytes(2, 2, 8, 4) if n is None else n
    return lib.retopk_chunk_attention(q, qs, ctypes.addressof(c), cu, T, B, Hq, sl, scale, cap, window, out, os, lse, ws, n, None, None)


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(format=2), -1), (dict(format=1), -1), (dict(n_pages=1), -1),
              (dict(n_pages=0), -1), (dict(page_rows=0), -1), (dict(n_kv_heads=0), -1), (dict(table=P, table_width=0, page_rows=16), -1),
              (dict(table=P, table_width=3, page_rows=24), -1), (dict(page_rows=(1 << 23) + 1), -2),
              (dict(table=P, table_width=1 << 20, page_rows=16), -2), (dict(k=P + 8), -5), (dict(v=P + 2), -5),
              (dict(table=P + 2, table_width=2, page_rows=16), -5), (dict(format=1, k_scale=P + 1, v_scale=P), -5)]


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_caches_are_checked(lib, kw, rc):
    assert append(lib, c=cache(**kw)) == rc
    assert attend(lib, c=cache(**kw)) == rc
    good = cache(k=P + 65536, v=P + 65536)
    a, b = cache(**kw), good
    for x, y in ((a, b), (b, a)):
        assert lib.retopk_cache_copy(ctypes.addressof(x), ctypes.addressof(y), P, P, 2, 10, None, None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), -1), (dict(B=0), -1), (dict(T=3), -1), (dict(Hq=6), -1), (dict(Hq=0), -1), (dict(q=None), -1), (dict(k=None), -1),
    (dict(v=None), -1), (dict(qo=None), -1), (dict(sl=None), -1), (dict(so=None), -1), (dict(qs=1016), -1), (dict(ks=504), -1),
    (dict(qs=1028), -5), (dict(vs=516), -5), (dict(q=P + 8), -5), (dict(qo=P + 8), -5), (dict(sl=P + 1), -5), (dict(st=P + 2), -5),
    (dict(Hq=128), -2), (dict(T=(1 << 22) + 1, cu=P), -2), (dict(qo=P, qs=2048), -1)])
def test_append_refuses(lib, kw, rc):
    assert append(lib, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(inv_freq=None), -1), (dict(rot_dim=24), -2), (dict(rot_dim=144), -2), (dict(rot_dim=-16), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(q_weight=P + 8), -5), (dict(inv_freq=P + 2), -5)])
def test_rope_refuses(lib, kw, rc):
    assert append(lib, r=rope(**kw)) == rc
    r = rope(**kw)
    assert lib.retopk_qk_rope(ctypes.addressof(r), P, 1024, P, 512, None, 2, 2, 8, 4, P, P + 8192, P + 16384, None) == rc


def test_in_place_rope_needs_the_outputs_strides(lib):
    r = rope()
    call = lambda qs, ks, qo, ko: lib.retopk_qk_rope(ctypes.addressof(r), P, qs, P + 65536, ks, None, 2, 2, 8, 4, P, qo, ko, None)  # noqa: E731
    assert call(2048, 512, P, P + 131072) == -1
    assert call(1024, 1024, P + 131072, P + 65536) == -1
    assert call(1024, 512, None, P) == -1


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), -1), (dict(T=3), -1), (dict(B=0), -1), (dict(Hq=6), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(sl=None), -1),
    (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(cap=-1.0), -1),
    (dict(cap=float("nan")), -1), (dict(window=-1), -1), (dict(qs=1020), -1), (dict(os=1000), -1), (dict(qs=1028), -5), (dict(os=1028), -5),
    (dict(q=P + 2), -5), (dict(out=P + 4), -5), (dict(lse=P + 2), -5), (dict(ws=None), -3), (dict(ws=P + 128), -3), (dict(n=0), -3),
    (dict(Hq=128), -2)])
def test_attention_refuses(lib, kw, rc):
    assert attend(lib, **kw) == rc


def test_attention_over_quantised_rows_is_refused(lib):
    assert attend(lib, c=cache(format=1, k_scale=P, v_scale=P)) == -2


def test_attention_workspace_sizes(lib):
    n = lib.retopk_chunk_attention_workspace_bytes
    assert n(1, 1, 28, 4) > 0 and n(0, 1, 28, 4) > 0
    for bad in ((-1, 1, 28, 4), (1, 0, 28, 4), (1, 1, 28, 5), (1, 1, 17, 1), (1, 1, 0, 1), ((1 << 22) + 1, 1, 28, 4)):
        assert n(*bad) == 0


@pytest.mark.parametrize("Hq,Hkv", [(28, 4), (32, 8), (16, 1), (8, 8), (7, 1)])
def test_a_workspace_of_the_largest_call_is_enough_for_smaller_ones(lib, Hq, Hkv):
    n = lib.retopk_chunk_attention_workspace_bytes
    sizes = [1, 2, 7, 17, 18, 27, 28, 36, 128, 192, 193, 512, 4096, 1 << 20]
    at = {(T, B): n(T, B, Hq, Hkv) for T in sizes for B in sizes[:-1]}
    for (T, B), most in at.items():
        assert most > 0 and all(size <= most for (T2, _), size in at.items() if T2 <= T)


def test_outputs_that_overlap_what_is_read_are_refused(lib):
    far, c = P + (1 << 20), cache(k=P + (1 << 24), v=P + (1 << 25))
    ok = dict(c=c, q=P, k=P + 65536, v=P + 131072, qo=far, sl=P + 262144, so=P + 262144)
    for kw in (dict(qo=P + 2048), dict(qo=P + 65536 + 1024), dict(qo=P + 131072 - 1024), dict(q=P + 1024, qo=P), dict(so=P + 262144 + 4),
               dict(so=P + 262144 - 4)):
        assert append(lib, **{**ok, **kw}) == -1
    r = rope()
    turn = lambda qo, ko, k=P + 65536: lib.retopk_qk_rope(  # noqa: E731
        ctypes.addressof(r), P, 1024, k, 512, None, 2, 2, 8, 4, P + 262144, qo, ko, None)
    for qo, ko in ((P + 16, far), (far, P + 2048), (P + 65536, far), (far, far + 2048), (far + 1024, far), (P, P)):
        assert turn(qo, ko) == -1
    # rows of 1024 elements in the same or another stride
    for q, qs, out, os in ((P, 2048, P, 1024), (P, 1024, P, 2048), (P, 2048, P + 1024, 2048), (P, 2048, P + 2064, 2048),
                           (P + 1024, 2048, P, 2048), (P, 1024, P + 2048, 1024), (P, 2048, P + 2048, 1024)):
        assert attend(lib, c=c, q=q, qs=qs, out=out, os=os, sl=P + 65536, ws=P + 131072) == -1
    a = cache()     # 2 pages of 102400 bytes
    for b in (cache(k=P + 65536, v=far), cache(k=far, v=P + 204784), cache(k=far, v=P), cache(k=P - 204784, v=far)):
        for x, y in ((a, b), (b, a)):
            assert lib.retopk_cache_copy(ctypes.addressof(x), ctypes.addressof(y), P, P, 2, 10, None, None) == -1


def test_copy_refuses(lib):
    a, b, other = cache(), cache(k=P + 65536, v=P + 65536), cache(k=P + 65536, v=P + 65536, n_kv_heads=2)
    call = lambda x, y, first=P, last=P, B=2, rows=10, st=None: lib.retopk_cache_copy(  # noqa: E731
        ctypes.addressof(x), ctypes.addressof(y), first, last, B, rows, st, None)
    assert call(a, a) == -1 and call(a, other) == -1
    assert call(a, b, first=None) == -1 and call(a, b, last=None) == -1 and call(a, b, B=0) == -1 and call(a, b, rows=-1) == -1
    assert call(a, b, rows=(1 << 23) + 1) == -2 and call(a, b, first=P + 2) == -5 and call(a, b, st=P + 1) == -5
    assert call(a, b, B=3) == -1
    assert call(a, b, rows=0) == 0


def test_empty_calls_need_no_tokens(lib):
    assert attend(lib, T=0, cu=P, q=None, out=None) == 0
    r = rope()
    assert lib.retopk_qk_rope(ctypes.addressof(r), None, 0, None, 0, P, 0, 2, 8, 4, P, None, None, None) == 0


def test_python_handles_check_their_tensors():
    k = torch.zeros((2, 4, 32, 128), dtype=torch.bfloat16)
    c8, s8 = torch.zeros((2, 4, 32, 128), dtype=torch.uint8), torch.zeros((2, 4, 32, 4), dtype=torch.uint8)
    assert retopk.KVCache(k, k.clone()).rows == 32
    c = retopk.KVCache(c8, c8.clone(), table=torch.zeros((3, 2), dtype=torch.int32), k_scale=s8, v_scale=s8.clone())
    assert (c.B, c.rows, c.Hkv) == (3, 64, 4)
    for bad in (lambda: retopk.KVCache(k, k[:1]), lambda: retopk.KVCache(k.float(), k.float()), lambda: retopk.KVCache(k, k, k_scale=s8, v_scale=s8),
                lambda: retopk.KVCache(c8, c8), lambda: retopk.KVCache(c8, c8, k_scale=s8, v_scale=s8[..., :2]),
                lambda: retopk.KVCache(k[..., :64], k[..., :64]), lambda: retopk.KVCache(k.transpose(1, 2), k.transpose(1, 2)),
                lambda: retopk.KVCache(k, k, table=torch.zeros((3, 2))), lambda: retopk.QKRope(q_weight=torch.zeros(64, dtype=torch.bfloat16)),
                lambda: retopk.QKRope(inv_freq=torch.zeros(64, dtype=torch.float64)), lambda: retopk._tokens(k[0].transpose(0, 1), "q"),
                lambda: retopk._tokens(k[0, :, :, :64], "q"), lambda: retopk._lens(torch.zeros(3), 3, "n"),
                lambda: retopk._lens(torch.zeros(4, dtype=torch.int32), 3, "n"), lambda: retopk._status(torch.zeros(1)),
                lambda: retopk.KVCache(k, k)._holds(3, "call")):
        with pytest.raises(retopk.RetopkError):
            bad()


def test_python_numbers_do_not_wrap_into_others():
    for n in ((1 << 32) + 4, 1 << 31, -(1 << 32) + 1, -1):
        with pytest.raises(retopk.RetopkError):
            retopk.chunk_attention_workspace_bytes(n, 1, 28, 4)
    assert retopk._bound((1 << 32) + 5) == (1 << 31) - 1 and retopk._bound(-(1 << 32)) == -1 and retopk._bound(7) == 7
    assert retopk._real(0.0, "x") == 0.0 and retopk._real(1e-30, "x") == 1e-30
    for bad in (lambda: retopk.QKRope(eps=1e-50), lambda: retopk._real(-1e-50, "x")):
        with pytest.raises(retopk.RetopkError):
            bad()
