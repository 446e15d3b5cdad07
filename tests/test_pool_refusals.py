"""Host checks of the calls on a cache's pages (no GPU work): every refusal returns before a launch."""
import ctypes

import pytest
import torch

from test_serving_devices import on, sdcp as stood_in  # noqa: F401  (a fixture: the library's calls are stood in for)

INVALID, WORKSPACE, ALIGN, TOO_LARGE = 1, 2, 3, 4
P = 4096  # an address that is never touched


@pytest.fixture(scope="module")
def sdcp():
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    from speculative_decoding_verification_sdcp_gb300 import sdcp as m
    return m


def pool(m, **kw):
    a = dict(n_pages=9, page_tokens=16, n_slots=3, max_pages=4, page_table=P, held=P, refs=P)
    a.update(kw)
    return m.KvPoolDesc(a.pop("size", ctypes.sizeof(m.KvPoolDesc)), **a)


def fork(m, p=None, **kw):
    a = dict(parent=P, length=P, st=P)
    a.update(kw)
    return m.lib.sdcp_fork_kv(ctypes.byref(p or pool(m)), a["parent"], a["length"], a["st"], None)


def reserve(m, p=None, **kw):
    a = dict(lens=P, upto=P, copies=P, most=3, n=P, st=P, ws=P, wb=1 << 20)
    a.update(kw)
    return m.lib.sdcp_reserve_kv(ctypes.byref(p or pool(m)), a["lens"], a["upto"], a["copies"], a["most"], a["n"], a["st"], a["ws"], a["wb"], None)


def release(m, p=None, **kw):
    a = dict(keep=P, st=P)
    a.update(kw)
    return m.lib.sdcp_release_kv(ctypes.byref(p or pool(m)), a["keep"], a["st"], None)


def compact(m, p=None, **kw):
    a = dict(copies=P, most=3, n=P, live=P, ws=P, wb=1 << 20)
    a.update(kw)
    return m.lib.sdcp_compact_kv(ctypes.byref(p or pool(m)), a["copies"], a["most"], a["n"], a["live"], a["ws"], a["wb"], None)


def copy(m, cache=None, **kw):
    a = dict(copies=P, most=3, n=P, st=P)
    a.update(kw)
    c = dict(n_pages=4, page_tokens=16, kv_heads=2, head_dim=64, max_pages=0, page_table=None, pages=P)
    c.update(cache or {})
    desc = m.KvCacheDesc(c.pop("size", ctypes.sizeof(m.KvCacheDesc)), **c)
    return m.lib.sdcp_copy_pages(ctypes.byref(desc), a["copies"], a["most"], a["n"], a["st"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(size=8), INVALID), (dict(n_pages=0), INVALID), (dict(page_tokens=8), INVALID), (dict(page_tokens=48), INVALID),
    (dict(page_tokens=2048), INVALID), (dict(n_slots=-1), INVALID), (dict(max_pages=0), INVALID), (dict(page_table=None), INVALID),
    (dict(held=None), INVALID), (dict(refs=None), INVALID), (dict(max_pages=2**27), TOO_LARGE), (dict(n_pages=2**30 + 1), TOO_LARGE),
    (dict(n_slots=2**30 + 1), TOO_LARGE), (dict(page_table=P + 2), ALIGN), (dict(held=P + 1), ALIGN), (dict(refs=P + 3), ALIGN)])
def test_pools(sdcp, kw, rc):
    for call in (fork, reserve, release, compact):
        assert call(sdcp, p=pool(sdcp, **kw)) == rc
    assert sdcp.lib.sdcp_fork_kv(None, P, P, P, None) == INVALID


@pytest.mark.parametrize("call,kw,rc", [
    (fork, dict(parent=None), INVALID), (fork, dict(length=None), INVALID), (fork, dict(st=None), INVALID), (fork, dict(st=P + 1), ALIGN),
    (fork, dict(length=P + 2), ALIGN), (release, dict(keep=None), INVALID), (release, dict(st=None), INVALID), (release, dict(keep=P + 2), ALIGN),
    (reserve, dict(lens=None), INVALID), (reserve, dict(upto=None), INVALID), (reserve, dict(copies=None), INVALID), (reserve, dict(n=None), INVALID),
    (reserve, dict(st=None), INVALID), (reserve, dict(most=2), INVALID), (reserve, dict(most=-1), INVALID), (reserve, dict(most=2**31 - 1), TOO_LARGE),
    (reserve, dict(copies=P + 8), ALIGN), (reserve, dict(n=P + 2), ALIGN), (reserve, dict(lens=P + 2), ALIGN), (reserve, dict(ws=None), WORKSPACE),
    (reserve, dict(ws=P + 128), WORKSPACE), (reserve, dict(wb=1023), WORKSPACE), (compact, dict(copies=None), INVALID), (compact, dict(n=None), INVALID),
    (compact, dict(live=None), INVALID), (compact, dict(most=-1), INVALID), (compact, dict(live=P + 2), ALIGN), (compact, dict(copies=P + 4), ALIGN),
    (compact, dict(ws=None), WORKSPACE), (compact, dict(wb=0), WORKSPACE), (copy, dict(copies=None), INVALID), (copy, dict(n=None), INVALID),
    (copy, dict(st=None), INVALID), (copy, dict(most=-1), INVALID), (copy, dict(most=2**30 + 1), TOO_LARGE), (copy, dict(copies=P + 8), ALIGN),
    (copy, dict(st=P + 2), ALIGN)])
def test_calls(sdcp, call, kw, rc):
    assert call(sdcp, **kw) == rc


@pytest.mark.parametrize("kw,rc", [(dict(size=8), INVALID), (dict(n_pages=0), INVALID), (dict(page_tokens=8), INVALID), (dict(kv_heads=0), INVALID),
                                   (dict(head_dim=96), INVALID), (dict(pages=None), INVALID), (dict(pages=P + 8), ALIGN)])
def test_caches(sdcp, kw, rc):
    assert copy(sdcp, cache=kw) == rc


def test_nothing_to_do(sdcp):
    empty = pool(sdcp, n_slots=0, page_table=None, held=None)
    assert fork(sdcp, p=empty, parent=None) == 0 and release(sdcp, p=empty, keep=None) == 0


def test_workspace(sdcp):
    size = sdcp.lib.sdcp_pool_workspace_bytes
    assert size(0, 1) == 0 and size(1, -1) == 0 and size(9, 0) > 0
    for a, b in ((1, 0), (9, 3), (1000, 70), (1 << 20, 4096)):
        assert size(a, b) <= size(a + 1, b) and size(a, b) <= size(a, b + 1) and size(a, b) % 256 == 0


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_what_the_library_cannot_see(sdcp):
    p = sdcp.KvPool(9, 16, 3, 4, "cpu")
    for bad in (dict(page_table=ints(3, 4).long()), dict(page_table=ints(3)), dict(page_table=ints(3, 4), held=ints(2)),
                dict(page_table=ints(3, 8)[:, ::2]), dict(page_table=ints(3, 4), refs=ints(8))):
        with pytest.raises((TypeError, ValueError)):
            sdcp.KvPool(9, 16, **bad)
    c = sdcp.KvCache(9, 16, 1, 64, "cpu")
    ws = torch.zeros(4096, dtype=torch.uint8)
    calls = [lambda x: sdcp.sdcp_fork_kv(p, x, ints(3), ints(3)), lambda x: sdcp.sdcp_fork_kv(p, ints(3), x, ints(3)),
             lambda x: sdcp.sdcp_fork_kv(p, ints(3), ints(3), x), lambda x: sdcp.sdcp_release_kv(p, x, ints(3)),
             lambda x: sdcp.sdcp_release_kv(p, ints(3), x), lambda x: sdcp.sdcp_reserve_kv(p, x, ints(3), ints(3, 4), ints(1), ints(3), ws),
             lambda x: sdcp.sdcp_reserve_kv(p, ints(3), x, ints(3, 4), ints(1), ints(3), ws),
             lambda x: sdcp.sdcp_reserve_kv(p, ints(3), ints(3), ints(3, 4), ints(1), x, ws)]
    for call in calls:
        for x in (ints(2), ints(3).long(), ints(6)[::2]):
            with pytest.raises((TypeError, ValueError)):
                call(x)
    lists = [lambda l, n: sdcp.sdcp_reserve_kv(p, ints(3), ints(3), l, n, ints(3), ws), lambda l, n: sdcp.sdcp_compact_kv(p, l, n, ints(1), ws),
             lambda l, n: sdcp.sdcp_copy_pages(c, l, n, ints(1))]
    for call in lists:
        for l, n in ((ints(3, 3), ints(1)), (ints(12), ints(1)), (ints(3, 4).long(), ints(1)), (ints(3, 4), ints(0)), (ints(4, 3).t(), ints(1))):
            with pytest.raises((TypeError, ValueError)):
                call(l, n)
    with pytest.raises(ValueError):
        sdcp.sdcp_copy_pages(c, ints(3, 4), ints(1), ints(0))
    with pytest.raises(ValueError):
        sdcp.sdcp_compact_kv(p, ints(3, 4), ints(1), ints(0), ws)


def _calls(m):
    """Each call's tensors by name, and the call."""
    def make(t, table=None):
        return m.KvPool(9, 16, page_table=t["table"], held=t["held"], refs=t["refs"])

    base = dict(status=ints(3), table=ints(3, 4), held=ints(3), refs=ints(9))
    ws = torch.zeros(4096, dtype=torch.uint8)
    pages = torch.zeros((9, 1, 2, 16 * 34), dtype=torch.uint8)
    return [
        (dict(base, a=ints(3), b=ints(3)), lambda t: m.sdcp_fork_kv(make(t), t["a"], t["b"], t["status"])),
        (dict(base, a=ints(3), b=ints(3), l=ints(3, 4), n=ints(1), ws=ws),
         lambda t: m.sdcp_reserve_kv(make(t), t["a"], t["b"], t["l"], t["n"], t["status"], t["ws"])),
        (dict(base, a=ints(3)), lambda t: m.sdcp_release_kv(make(t), t["a"], t["status"])),
        (dict(base, l=ints(3, 4), n=ints(1), ws=ws, status=ints(1)), lambda t: m.sdcp_compact_kv(make(t), t["l"], t["n"], t["status"], t["ws"])),
        (dict(status=ints(1), l=ints(3, 4), n=ints(1), pages=pages),
         lambda t: m.sdcp_copy_pages(m.KvCache(9, 16, 1, 64, None, pages=t["pages"]), t["l"], t["n"], t["status"]))]


@pytest.mark.parametrize("k", range(5))
def test_every_tensor_is_on_the_device(stood_in, monkeypatch, k):  # noqa: F811
    def reached(*a):
        raise AssertionError("the library was called")

    for name in ("sdcp_fork_kv", "sdcp_reserve_kv", "sdcp_release_kv", "sdcp_compact_kv", "sdcp_copy_pages"):
        monkeypatch.setattr(stood_in.lib, name, reached)
    t, call = _calls(stood_in)[k]
    good = {k: on(v) for k, v in t.items()}
    with pytest.raises(AssertionError, match="library was called"):
        call(good)
    for name in t:
        for other in (t[name], on(t[name], 1)):
            with pytest.raises(ValueError, match="device"):
                call({**good, name: other})
