"""The calls on pages and the shared attention together, as examples/branch_round.py runs them.

What a continuation has cached is its own: forks share pages and rounds write beside one another, and no
committed token changes.  The shared attention agrees with the attention of sessions by themselves, and a pool
that is full refuses sessions and leaves them as they were."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def examples():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import branch_round
    import verify_round
    return branch_round, verify_round


@pytest.mark.parametrize("length", [3, 16, 33, 230])
def test_continuations_keep_their_pages_apart(examples, length):
    branch_round, verify_round = examples
    rng = np.random.default_rng(length)
    model = verify_round.Model(vocab=300)
    prompts = [rng.integers(0, 300, length + s).tolist() for s in range(3)]
    run = branch_round.Branches(model, prompts, 4, pool_pages=300)
    refs = run.pool.refs.tolist()
    assert max(refs) == (4 if length > 1 else 0) and sum(refs) == sum(run.pool.held.tolist())
    first = [run.cached(s) for s in range(run.B)]
    for s in range(run.B):  # a fork holds its session's tokens
        assert all(torch.equal(x, y) for x, y in zip(first[s], first[s - s % 4]))
    for r in range(1, 5):
        before = [run.cached(s) for s in range(run.B)]
        lens = list(run.kv_len)
        run.round([rng.integers(0, 300, int(rng.integers(1, 20))).tolist() for _ in range(run.B)], r)
        assert not run.refused
        for s in range(run.B):  # what was committed is not touched by the round, the slot's own or another's
            assert all(torch.equal(x[:lens[s]], y) for x, y in zip(run.cached(s), before[s]))
        held, refs, table = run.pool.held.tolist(), run.pool.refs.tolist(), run.pool.page_table.tolist()
        assert held == [-(-n // 16) for n in run.kv_len]
        count = np.zeros(300, dtype=int)
        for s in range(run.B):
            np.add.at(count, table[s][:held[s]], 1)
            assert set(table[s][held[s]:]) <= {-1}
        assert count.tolist() == refs
    kept = [1, 0, 3]
    before = [run.cached(4 * s + k) for s, k in enumerate(kept)]
    live = run.keep(kept)
    assert live == sum(-(-run.kv_len[4 * s + k] // 16) for s, k in enumerate(kept))
    refs = run.pool.refs.tolist()
    assert refs == [1] * live + [0] * (300 - live)
    for (s, k), want in zip(enumerate(kept), before):
        assert all(torch.equal(x, y) for x, y in zip(run.cached(4 * s + k), want))
    # the pool is usable on: the kept ones go on, with pages past them
    run.kv_len = [n if s % 4 == kept[s // 4] else 0 for s, n in enumerate(run.kv_len)]
    status = run.score([[1, 2, 3] if s % 4 == kept[s // 4] else [] for s in range(run.B)], grouped=False)[3]
    assert status.tolist() == [0] * 3


def test_attention_of_forks_is_the_attention_of_copies(examples):
    """The rows of forked sessions, attended in groups, against sdcp_attend_kv over the same pages."""
    branch_round, verify_round = examples
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    rng = np.random.default_rng(5)
    model = verify_round.Model(vocab=300)
    run = branch_round.Branches(model, [rng.integers(0, 300, n).tolist() for n in (450, 301)], 5, pool_pages=200)
    rows = [rng.integers(0, 300, int(rng.integers(1, 9))).tolist() for _ in range(run.B)]
    calls = []
    shared = sdcp.sdcp_attend_shared_kv

    def both(cache, table, off, total, kv_len, groups, q, out, status, ws):
        shared(cache, table, off, total, kv_len, groups, q, out, status, ws)
        other, st = torch.empty_like(out), torch.empty_like(status)
        sdcp.sdcp_attend_kv(cache, table, off, total, kv_len, q, other, st,
                            sdcp.alloc_attend_workspace(status.numel(), total, q.shape[1], cache.kv_heads, cache.head_dim, q.device))
        calls.append((out.double(), other.double(), status.tolist() + st.tolist()))

    sdcp.sdcp_attend_shared_kv = both
    try:
        run.score(rows)
    finally:
        sdcp.sdcp_attend_shared_kv = shared
    (x, y, status), = calls
    assert set(status) == {0}
    # both are within 2^-8 of their value and 2^-10 of the largest value that is summed of the exact sum
    most = max(float(run.cached(s)[1].abs().max()) for s in range(run.B)) * 1.5
    assert bool(((x - y).abs() <= 2 * (2.0**-8 * torch.maximum(x.abs(), y.abs()) + 2.0**-10 * most)).all())


def test_a_pool_that_is_full_refuses_and_goes_on(examples):
    branch_round, verify_round = examples
    rng = np.random.default_rng(6)
    model = verify_round.Model(vocab=300)
    run = branch_round.Branches(model, [rng.integers(0, 300, 41).tolist() for _ in range(2)], 2, pool_pages=9)
    lens, before = list(run.kv_len), [run.cached(s) for s in range(4)]
    run.round([rng.integers(0, 300, 30).tolist() for _ in range(4)], 1)  # 3 pages each shared by two, 3 free
    for s in range(4):  # nobody's tokens are written over
        assert all(torch.equal(x[:lens[s]], y) for x, y in zip(run.cached(s), before[s]))
    assert run.refused and not all(s in run.refused for s in range(4))
    assert all(run.kv_len[s] == lens[s] for s in run.refused) and all(run.kv_len[s] > lens[s] for s in range(4) if s not in run.refused)
