"""A bounded wait of the attention kernel that runs out reports SDCP_S_INTERNAL for every session and
leaves the device usable.

The library is built once more with the test-only flag SDCP_TEST_WAIT_EXPIRY (as in
tests/test_zz_wait_expiry.py): waits give up after 20 ms, and every fourth CTA never hands the weights
of its first tile over.  Its product warp's wait for them runs out, and its other warps' waits for that
product; they agree on it, wait for their own copies, give the tensor memory back and return.  No
fault, trap or endless loop is involved, and the ordinary library gives the same output before and
after."""
import ctypes
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def waitlib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    path = build_ext.build(extra_flags=["-DSDCP_TEST_WAIT_EXPIRY"],
                           lib=os.path.join(build_ext.PKG, "libsdcp_waittest.so"),
                           build_dir=os.path.join(build_ext.BUILD, "waittest"))
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    fn = ctypes.CDLL(path).sdcp_attend_kv
    fn.argtypes, fn.restype = sdcp.lib.sdcp_attend_kv.argtypes, ctypes.c_int
    return fn


# one tile a CTA; several tiles a CTA, copies of the next one under way; the wide shape; many sessions
@pytest.mark.parametrize("B,m,ctx,share,dim", [(1, 0, 200, 4, 128), (4, 0, 20000, 4, 128), (4, 8, 20000, 8, 64), (300, 1, 300, 4, 64)])
def test_waits_that_run_out_report_internal(waitlib, monkeypatch, B, m, ctx, share, dim):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    P, heads = 64, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(B)
    per = -(-(ctx + m + 1) // P)
    cache = sdcp.KvCache(B * per, P, heads, dim, DEV)
    cache.pages.random_(0, 256, generator=g)
    cache.pages[..., P * dim // 2:].random_(100, 120, generator=g)
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).view(B, per)
    off = torch.arange(B + 1, dtype=torch.int32, device=DEV) * m
    lens = torch.full((B,), ctx, dtype=torch.int32, device=DEV)
    q = torch.randn((B * (m + 1), heads * share, dim), generator=g, device=DEV).to(torch.bfloat16)
    ws = sdcp.alloc_attend_workspace(B, B * m, heads * share, heads, dim, DEV)

    def call():
        out, st = torch.empty_like(q), torch.full((B,), -9, dtype=torch.int32, device=DEV)
        sdcp.sdcp_attend_kv(cache, table, off, B * m, lens, q, out, st, ws)
        torch.cuda.synchronize()  # raises if the device had faulted
        return out, set(st.tolist())

    before, ok = call()
    assert ok == {sdcp.S_OK} and bool(torch.isfinite(before.float()).all())
    with monkeypatch.context() as mp:
        mp.setattr(sdcp.lib, "sdcp_attend_kv", waitlib)
        assert call()[1] == {sdcp.S_INTERNAL}
    after, ok = call()
    assert ok == {sdcp.S_OK} and torch.equal(before.view(torch.int16), after.view(torch.int16))
