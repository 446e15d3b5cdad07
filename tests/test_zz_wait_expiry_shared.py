"""A bounded wait of the shared attention's kernel that runs out reports SDCP_S_INTERNAL for every session
and leaves the device usable.

The library is built with the test-only flag SDCP_TEST_WAIT_EXPIRY (as in tests/test_zz_wait_expiry_attend.py):
waits give up after 20 ms, and every fourth CTA keeps the weights of its first step to itself.  Its product
warp's wait for them runs out, the others' waits see it; copies and products under way end, the tensor memory
is given back.  No fault, trap or endless loop is involved, and the ordinary library gives the same output
before and after."""
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
    fn = ctypes.CDLL(path).sdcp_attend_shared_kv
    fn.argtypes, fn.restype = sdcp.lib.sdcp_attend_shared_kv.argtypes, ctypes.c_int
    return fn


# a step a CTA; several, copies of the next tile under way; two blocks of pairs; many groups
@pytest.mark.parametrize("groups,size,m,ctx,share,dim", [(1, 2, 0, 200, 4, 128), (1, 2, 0, 40000, 4, 128), (2, 8, 8, 6000, 8, 64), (150, 2, 1, 300, 4, 64)])
def test_waits_that_run_out_report_internal(waitlib, monkeypatch, groups, size, m, ctx, share, dim):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    P, heads, B = 64, 8, groups * size
    g = torch.Generator(device=DEV)
    g.manual_seed(B)
    common, per = ctx // P, -(-(ctx + m + 1) // P)
    cache = sdcp.KvCache(groups * common + B * (per - common), P, heads, dim, DEV)
    cache.pages.random_(0, 256, generator=g)
    cache.pages[..., P * dim // 2:].random_(100, 120, generator=g)
    table = torch.empty((B, per), dtype=torch.int32, device=DEV)
    table[:, :common] = torch.arange(groups * common, dtype=torch.int32, device=DEV).view(groups, common).repeat_interleave(size, 0)
    table[:, common:] = groups * common + torch.arange(B * (per - common), dtype=torch.int32, device=DEV).view(B, -1)
    off = torch.arange(B + 1, dtype=torch.int32, device=DEV) * m
    lens = torch.full((B,), ctx, dtype=torch.int32, device=DEV)
    group_offsets = torch.arange(groups + 1, dtype=torch.int32, device=DEV) * size
    q = torch.randn((B * (m + 1), heads * share, dim), generator=g, device=DEV).to(torch.bfloat16)
    ws = sdcp.alloc_attend_shared_workspace(B, B * m, groups, heads * share, heads, dim, DEV)

    def call():
        out, st = torch.empty_like(q), torch.full((B,), -9, dtype=torch.int32, device=DEV)
        sdcp.sdcp_attend_shared_kv(cache, table, off, B * m, lens, group_offsets, q, out, st, ws)
        torch.cuda.synchronize()  # raises if the device had faulted
        return out, set(st.tolist())

    before, ok = call()
    assert ok == {sdcp.S_OK} and bool(torch.isfinite(before.float()).all())
    with monkeypatch.context() as mp:
        mp.setattr(sdcp.lib, "sdcp_attend_shared_kv", waitlib)
        assert call()[1] == {sdcp.S_INTERNAL}
    after, ok = call()
    assert ok == {sdcp.S_OK} and torch.equal(before.view(torch.int16), after.view(torch.int16))
