"""Refusals of the 4-bit cache (RETOPK_CACHE_FP4): answered on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from top_sparse_attention_exact_gb300 import retopk

P = 1 << 20     # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    return retopk.load()


def cache(**kw):
    d = dict(k=P, v=P + (1 << 24), k_scale=P + (1 << 25), v_scale=P + (1 << 26), table=None, format=2, n_pages=2, n_kv_heads=4, page_rows=100,
             table_width=0)
    d.update(kw)
    return retopk.retopk_cache(*[d[f] for f, _ in retopk.retopk_cache._fields_])


def append(lib, c):
    r = retopk.retopk_rope(None, None, P, 1e-6, 128, 0)
    return lib.retopk_qkv_append(ctypes.addressof(r), P, 1024, P, 512, P, 512, None, 2, 2, 8, ctypes.addressof(c), P, P, P + 4096, None, None)


def copy(lib, a, b):
    return lib.retopk_cache_copy(ctypes.addressof(a), ctypes.addressof(b), P, P, 2, 10, None, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(k=None), -1), (dict(format=3), -1), (dict(format=-1), -1), (dict(n_pages=1), -1),
    (dict(k_scale=P + 4), -5), (dict(v_scale=P + 2), -5), (dict(k=P + 8), -5), (dict(v=P + 4), -5), (dict(page_rows=(1 << 23) + 1), -2),
    (dict(table=P, table_width=2, page_rows=24), -1)])
def test_caches_are_checked(lib, kw, rc):
    assert append(lib, cache(**kw)) == rc
    good = cache(k=P + (1 << 27), v=P + (1 << 28), format=0)
    assert copy(lib, cache(**kw), good) == rc and copy(lib, good, cache(**kw)) == rc


def test_copies_between_pools_that_overlap_are_refused(lib):
    a = cache()                                             # codes of 51200 bytes
    for b in (cache(k=P + 51184), cache(v=P + (1 << 24) - 51184), cache(k=P + (1 << 24) + 16, v=P), cache(format=0, k=P - 204784, v=P + (1 << 30))):
        assert copy(lib, a, b) == -1 and copy(lib, b, a) == -1


def test_copies_between_scales_that_overlap_are_refused(lib):
    a, far = cache(), dict(k=P + (1 << 27), v=P + (1 << 28), k_scale=P + (1 << 29), v_scale=P + (1 << 30))   # scales of 6400 bytes
    for kw in (dict(k_scale=P + (1 << 25) + 6392), dict(v_scale=P + (1 << 25)), dict(v_scale=P + (1 << 26) - 6392), dict(k_scale=P + 51192),
               dict(v=P + (1 << 25) - 51184)):
        b = cache(**{**far, **kw})
        assert copy(lib, a, b) == -1 and copy(lib, b, a) == -1
    b = cache(format=1, **{**far, "k_scale": P + (1 << 26) + 3196})       # of 3200 bytes
    assert copy(lib, a, b) == -1 and copy(lib, b, a) == -1


@pytest.mark.parametrize("format", [1, 2])
def test_caches_with_one_pool_of_scales_for_keys_and_values_are_not_written(lib, format):
    src = cache(k=P + (1 << 27), v=P + (1 << 28), format=0)
    for kw in (dict(v_scale=P + (1 << 25)), dict(k_scale=P + (1 << 26)), dict(v=P + 64 * 800, v_scale=P + (1 << 25))):
        bad = cache(format=format, **kw)
        assert append(lib, bad) == -1 and copy(lib, src, bad) == -1


def test_attention_takes_4_bit_caches_and_checks_them(lib):
    n = lib.retopk_chunk_attention_workspace_bytes(2, 2, 8, 4)

    def attend(c, q=P + (1 << 27), ws=P + (1 << 28), size=n):
        return lib.retopk_chunk_attention(q, 1024, ctypes.addressof(c), None, 2, 2, 8, P, 0.0, 0.0, 0, P + (1 << 29), 1024, None, ws, size, None, None)
    for kw, rc in ((dict(k_scale=None), -1), (dict(v_scale=P + 4), -5), (dict(k=P + 8), -5), (dict(page_rows=0), -1), (dict(format=1), -2)):
        assert attend(cache(**kw)) == rc
    assert attend(cache(), q=P + 2) == -5 and attend(cache(), size=n - 1) == -3 and attend(cache(), ws=P + 128) == -3


@pytest.mark.parametrize("Hq,Hkv", [(28, 4), (32, 8), (16, 1), (8, 8), (7, 1)])
def test_a_workspace_of_the_largest_call_is_enough_for_smaller_ones(lib, Hq, Hkv):
    n = lib.retopk_chunk_attention_workspace_bytes
    sizes = [1, 2, 5, 64, 608, 4096]
    at = {(T, B): n(T, B, Hq, Hkv) for T in sizes for B in sizes}
    for (T, B), most in at.items():
        assert all(size <= most for (T2, _), size in at.items() if T2 <= T)


def test_python_handles_check_their_tensors():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    c, s = z(2, 4, 32, 64), z(2, 4, 32, 8)
    h = retopk.KVCache(c, c.clone(), table=torch.zeros((3, 2), dtype=torch.int32), k_scale=s, v_scale=s.clone())
    assert (h.B, h.rows, h.Hkv, h.struct.format) == (3, 64, 4, retopk.CACHE_FP4)
    assert retopk.KVCache(z(2, 4, 32, 128), z(2, 4, 32, 128), k_scale=z(2, 4, 32, 4), v_scale=z(2, 4, 32, 4)).struct.format == retopk.CACHE_MX8
    for bad in (lambda: retopk.KVCache(c, c), lambda: retopk.KVCache(c, c, k_scale=s, v_scale=s[..., :4]),
                lambda: retopk.KVCache(c, z(2, 4, 32, 128), k_scale=s, v_scale=s), lambda: retopk.KVCache(c, c, k_scale=s, v_scale=z(2, 4, 16, 8)),
                lambda: retopk.KVCache(c[..., :32], c[..., :32], k_scale=s, v_scale=s), lambda: retopk.KVCache(c, c, k_scale=s, v_scale=None),
                lambda: retopk.KVCache(c, c, k_scale=s.int(), v_scale=s.int())):
        with pytest.raises(retopk.RetopkError):
            bad()
