"""The attention's workspace: one that is large enough for a program's largest batch is for its others
too (no GPU work)."""
import itertools

import pytest


@pytest.fixture(scope="module")
def sdcp():
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    from speculative_decoding_verification_sdcp_gb300 import sdcp as m
    return m


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(32, 8, 128), (28, 4, 64), (8, 8, 64), (64, 8, 128), (128, 1, 128)])
def test_a_smaller_batch_needs_no_more(sdcp, q_heads, kv_heads, head_dim):
    sizes = [(B, total) for B in (0, 1, 2, 7, 63, 64, 512, 1024) for total in (0, 1, 8, 192, 1024, 4096, 70000)]
    need = {s: sdcp.sdcp_attend_workspace_bytes(s[0], s[1], q_heads, kv_heads, head_dim) for s in sizes}
    assert min(need.values()) > 0
    for (B, total), (b, t) in itertools.product(sizes, sizes):
        if b <= B and t <= total:
            assert need[(b, t)] <= need[(B, total)]
