"""Host checks of the serving operators (no GPU work): every refusal returns before a launch."""
import ctypes

import pytest

INVALID, WORKSPACE, ALIGN, TOO_LARGE = 1, 2, 3, 4
P = 4096  # an address that is never touched


@pytest.fixture(scope="module")
def sdcp():
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    from speculative_decoding_verification_sdcp_gb300 import sdcp as m
    return m


def adjust(m, **kw):
    a = dict(logits=P, out=P, dtype=0, V=100, B=2, rows=0, off=P, total=4, tok=P, ctl=P, hist=P, stride=8, bt=P, bv=P, nb=3, masks=P,
             ms=4, nm=2, mr=P, st=P)
    a.update(kw)
    return m.lib.sdcp_adjust_logits(a["logits"], a["out"], a["dtype"], a["V"], a["B"], a["rows"], a["off"], a["total"], a["tok"], a["ctl"],
                                    a["hist"], a["stride"], a["bt"], a["bv"], a["nb"], a["masks"], a["ms"], a["nm"], a["mr"], a["st"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(V=0), INVALID), (dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(dtype=2), INVALID), (dict(rows=2), INVALID),
    (dict(stride=-1), INVALID), (dict(nb=-1), INVALID), (dict(nm=-1), INVALID), (dict(V=(1 << 24) + 1), TOO_LARGE),
    (dict(total=2**30), TOO_LARGE), (dict(logits=None), INVALID), (dict(out=None), INVALID), (dict(off=None), INVALID),
    (dict(ctl=None), INVALID), (dict(st=None), INVALID), (dict(tok=None), INVALID), (dict(hist=None), INVALID), (dict(bt=None), INVALID),
    (dict(bv=None), INVALID), (dict(masks=None), INVALID), (dict(ms=3), INVALID), (dict(logits=P + 2), ALIGN),
    (dict(out=P + 1, dtype=1), ALIGN), (dict(B=0, off=None), 0)])
def test_adjust(sdcp, kw, rc):
    assert adjust(sdcp, **kw) == rc


def cache(m, **kw):
    a = dict(n_pages=4, page_tokens=16, kv_heads=2, head_dim=64, max_pages=2, page_table=P, pages=P)
    a.update(kw)
    return m.KvCacheDesc(a.pop("size", ctypes.sizeof(m.KvCacheDesc)), **a)


BAD_CACHES = [(dict(size=8), INVALID), (dict(n_pages=0), INVALID), (dict(page_tokens=8), INVALID), (dict(page_tokens=24), INVALID),
              (dict(page_tokens=2048), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=257), INVALID), (dict(head_dim=96), INVALID),
              (dict(max_pages=0), INVALID), (dict(page_table=None), INVALID), (dict(pages=None), INVALID), (dict(pages=P + 8), ALIGN),
              (dict(max_pages=2**27), TOO_LARGE)]


def rotary(m, **kw):
    a = dict(layout=0, rot_dim=64, n_positions=10, table=P)
    a.update(kw)
    return m.RotaryDesc(a.pop("size", ctypes.sizeof(m.RotaryDesc)), **a)


def append(m, c=None, rot=None, **kw):
    a = dict(B=2, off=P, total=3, lens=P, dtype=1, k=P, ks=128, v=P, vs=128, q=P, qs=256, nq=4, qo=P, st=P)
    a.update(kw)
    c = cache(m) if c is None else c
    return m.lib.sdcp_append_kv(ctypes.byref(c), a["B"], a["off"], a["total"], a["lens"], a["dtype"], a["k"], a["ks"], a["v"], a["vs"],
                                None if rot is None else ctypes.byref(rot), a["q"], a["qs"], a["nq"], a["qo"], a["st"], None)


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_caches(sdcp, kw, rc):
    c = cache(sdcp, **kw)
    assert append(sdcp, c=c) == rc and read(sdcp, c=c) == rc and attend(sdcp, c=c) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(dtype=5), INVALID), (dict(total=2**30), TOO_LARGE), (dict(off=None), INVALID),
    (dict(lens=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(st=None), INVALID), (dict(q=None), INVALID),
    (dict(qo=None), INVALID), (dict(nq=0), INVALID), (dict(nq=-1), INVALID), (dict(ks=120), INVALID), (dict(vs=64), INVALID),
    (dict(qs=248), INVALID), (dict(ks=129), ALIGN), (dict(vs=132), ALIGN), (dict(qs=260), ALIGN), (dict(k=P + 8), ALIGN),
    (dict(v=P + 2), ALIGN), (dict(q=P + 4), ALIGN), (dict(qo=P + 8), ALIGN), (dict(B=0, off=None), 0)])
def test_append(sdcp, kw, rc):
    assert append(sdcp, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(size=4), INVALID), (dict(layout=2), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=7), INVALID), (dict(rot_dim=66), INVALID),
    (dict(n_positions=0), INVALID), (dict(table=None), INVALID), (dict(table=P + 2), ALIGN)])
def test_rotary(sdcp, kw, rc):
    assert append(sdcp, rot=rotary(sdcp, **kw)) == rc


def read(m, c=None, **kw):
    a = dict(B=2, off=P, n=5, start=P, dtype=1, k=P, v=P, st=P)
    a.update(kw)
    c = cache(m) if c is None else c
    return m.lib.sdcp_read_kv(ctypes.byref(c), a["B"], a["off"], a["n"], a["start"], a["dtype"], a["k"], a["v"], a["st"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(n=-1), INVALID), (dict(dtype=9), INVALID), (dict(n=2**30), TOO_LARGE), (dict(off=None), INVALID),
    (dict(start=None), INVALID), (dict(st=None), INVALID), (dict(k=None, v=None), INVALID), (dict(k=P + 8), ALIGN), (dict(v=P + 4), ALIGN),
    (dict(B=0, off=None), 0)])
def test_read(sdcp, kw, rc):
    assert read(sdcp, **kw) == rc


def attend(m, c=None, **kw):
    a = dict(B=2, off=P, total=3, lens=P, q=P, qs=256, nq=4, scale=0.1, window=0, out=P, st=P, ws=P, wb=1 << 40)
    a.update(kw)
    c = cache(m) if c is None else c
    return m.lib.sdcp_attend_kv(ctypes.byref(c), a["B"], a["off"], a["total"], a["lens"], a["q"], a["qs"], a["nq"], a["scale"], a["window"],
                                a["out"], a["st"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(nq=3), INVALID), (dict(nq=0), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(total=2**30), TOO_LARGE), (dict(off=None), INVALID),
    (dict(lens=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(st=None), INVALID), (dict(qs=255), INVALID),
    (dict(qs=260), ALIGN), (dict(q=P + 8), ALIGN), (dict(out=P + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=P + 128), WORKSPACE),
    (dict(wb=0), WORKSPACE), (dict(B=0, off=None), 0)])
def test_attend(sdcp, kw, rc):
    assert attend(sdcp, **kw) == rc


def test_sizes(sdcp):
    L = sdcp.lib
    assert L.sdcp_kv_page_bytes(16, 2, 64) == 2 * 2 * 16 * 34 and L.sdcp_kv_page_bytes(64, 8, 128) == 2 * 8 * 64 * 68
    assert L.sdcp_kv_page_bytes(17, 2, 64) == 0 and L.sdcp_kv_page_bytes(16, 2, 80) == 0
    for bad in ((-1, 0, 4, 2, 64), (1, -1, 4, 2, 64), (1, 0, 5, 2, 64), (1, 0, 4, 0, 64), (1, 0, 4, 2, 96)):
        assert L.sdcp_attend_workspace_bytes(*bad) == 0
    assert L.sdcp_attend_workspace_bytes(0, 0, 4, 2, 64) > 0


def test_binding_refuses_what_the_library_cannot_see(sdcp):
    torch = pytest.importorskip("torch")
    z = lambda *s, **k: torch.zeros(*s, **{"dtype": torch.int32, **k})  # noqa: E731
    with pytest.raises(sdcp.SdcpError):
        sdcp.KvCache(1, 17, 1, 64, "cpu")
    c = sdcp.KvCache(2, 16, 1, 64, "cpu")
    with pytest.raises(ValueError):
        sdcp.KvCache(2, 16, 1, 64, "cpu", pages=c.pages[:1])
    f = torch.zeros((3, 64))
    with pytest.raises(TypeError):
        sdcp.sdcp_adjust_logits(f, f.bfloat16(), z(3), 1, z(1), z(64, dtype=torch.uint8), None, z(2))
    with pytest.raises(TypeError):
        sdcp.sdcp_adjust_logits(f.t(), f.t(), z(3), 1, z(1), z(64, dtype=torch.uint8), None, z(2))
    with pytest.raises(ValueError):
        sdcp.sdcp_adjust_logits(f, f, z(3), 2, z(2), z(64, dtype=torch.uint8), None, z(2))
    h = torch.zeros((3, 1, 64))
    with pytest.raises(TypeError):
        sdcp.sdcp_append_kv(c, z(2, 1), z(3), 1, z(2), h, h.bfloat16(), z(2))
    with pytest.raises(ValueError):
        sdcp.sdcp_append_kv(c, z(2, 1), z(3), 1, z(2), h, h[:, :, :32], z(2))
    with pytest.raises(ValueError):
        sdcp.sdcp_append_kv(c, z(1, 1), z(3), 1, z(2), h, h, z(2))
    with pytest.raises(TypeError):
        sdcp.sdcp_attend_kv(c, z(2, 1), z(3), 1, z(2), h, h, z(2), z(1))
    with pytest.raises(TypeError):
        sdcp.sdcp_read_kv(c, z(2, 1), z(3), 1, z(2), None, None, z(2))
