"""Host checks of sdcp_attend_shared_kv (no GPU work): every refusal returns before a launch."""
import ctypes
import itertools

import pytest
import torch

from test_serving_devices import ints, on, sdcp as stood_in  # noqa: F401  (a fixture: the library's calls are stood in for)
from test_serving_refusals import ALIGN, BAD_CACHES, INVALID, P, TOO_LARGE, WORKSPACE, cache


@pytest.fixture(scope="module")
def sdcp():
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    from speculative_decoding_verification_sdcp_gb300 import sdcp as m
    return m


def attend(m, c=None, **kw):
    a = dict(B=2, off=P, total=3, lens=P, ng=1, groups=P, q=P, qs=256, nq=4, scale=0.1, out=P, st=P, ws=P, wb=1 << 40)
    a.update(kw)
    c = cache(m) if c is None else c
    return m.lib.sdcp_attend_shared_kv(ctypes.byref(c), a["B"], a["off"], a["total"], a["lens"], a["ng"], a["groups"], a["q"], a["qs"], a["nq"],
                                       a["scale"], a["out"], a["st"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(ng=-1), INVALID), (dict(ng=0), INVALID), (dict(groups=None), INVALID),
    (dict(nq=3), INVALID), (dict(nq=0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("-inf")), INVALID),
    (dict(total=2**30), TOO_LARGE), (dict(total=2**29), TOO_LARGE), (dict(nq=1 << 21, qs=1 << 28), TOO_LARGE), (dict(off=None), INVALID),
    (dict(lens=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(st=None), INVALID), (dict(qs=255), INVALID),
    (dict(qs=260), ALIGN), (dict(q=P + 8), ALIGN), (dict(out=P + 2), ALIGN), (dict(off=P + 2), ALIGN), (dict(lens=P + 1), ALIGN),
    (dict(groups=P + 2), ALIGN), (dict(st=P + 3), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=P + 128), WORKSPACE), (dict(wb=0), WORKSPACE),
    (dict(B=0, off=None), 0)])
def test_calls(sdcp, kw, rc):
    assert attend(sdcp, **kw) == rc


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_caches(sdcp, kw, rc):
    assert attend(sdcp, c=cache(sdcp, **kw)) == rc


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(32, 8, 128), (28, 4, 64), (128, 1, 128)])
def test_a_smaller_batch_needs_no_more(sdcp, q_heads, kv_heads, head_dim):
    size = sdcp.lib.sdcp_attend_shared_workspace_bytes
    sizes = [(B, total, g) for B in (0, 1, 63, 512) for total in (0, 8, 1024, 70000) for g in (0, 1, 40, 512)]
    need = {s: size(*s, q_heads, kv_heads, head_dim) for s in sizes}
    assert min(need.values()) > 0 and all(v % 256 == 0 for v in need.values())
    for a, b in itertools.product(sizes, sizes):
        if all(x <= y for x, y in zip(a, b)):
            assert need[a] <= need[b]
    for bad in ((-1, 0, 0, 4, 2, 64), (1, -1, 0, 4, 2, 64), (1, 0, -1, 4, 2, 64), (1, 0, 0, 5, 2, 64), (1, 0, 0, 4, 0, 64), (1, 0, 0, 4, 2, 96),
                (1, 2**30, 0, 1, 1, 64), (1, 2**28, 0, 8, 1, 64)):
        assert size(*bad) == 0


def _call(m, t):
    return m.sdcp_attend_shared_kv(m.KvCache(2, 16, 1, 64, None, pages=t["pages"]), t["table"], t["off"], 1, t["lens"], t["groups"], t["q"], t["out"],
                                   t["status"], t["ws"])


def _tensors():
    vec = torch.zeros((3, 1, 64)).bfloat16()
    return dict(table=ints(2, 1), off=ints(3), lens=ints(2), status=ints(2), pages=torch.zeros((2, 1, 2, 16 * 34), dtype=torch.uint8), groups=ints(2),
                q=vec, out=vec.clone(), ws=torch.zeros(1 << 10, dtype=torch.uint8))


def test_every_tensor_is_on_the_device(stood_in, monkeypatch):  # noqa: F811
    def reached(*a):
        raise AssertionError("the library was called")

    monkeypatch.setattr(stood_in.lib, "sdcp_attend_shared_kv", reached)
    good = {k: on(v) for k, v in _tensors().items()}
    with pytest.raises(AssertionError, match="library was called"):
        _call(stood_in, good)
    for name in good:
        for other in (_tensors()[name], on(_tensors()[name], 1)):
            with pytest.raises(ValueError, match="device"):
                _call(stood_in, {**good, name: other})


@pytest.mark.parametrize("kw", [dict(groups=ints(0)), dict(groups=ints(1)), dict(groups=ints(2).long()), dict(groups=ints(4)[::2]),
                                dict(out=torch.zeros((3, 1, 64))), dict(out=torch.zeros((2, 1, 64)).bfloat16()), dict(q=torch.zeros((3, 2, 64)).bfloat16()),
                                dict(lens=ints(1)), dict(off=ints(2)), dict(status=ints(2).long()), dict(table=ints(1, 1))])
def test_binding_refuses_what_the_library_cannot_see(sdcp, kw):
    with pytest.raises((TypeError, ValueError)):
        _call(sdcp, {**_tensors(), **kw})


def test_workspace_of_invalid_sizes(sdcp):
    with pytest.raises(sdcp.SdcpError):
        sdcp.alloc_attend_shared_workspace(1, 0, 1, 5, 2, 64, "cpu")
