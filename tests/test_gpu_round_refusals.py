"""A session that one of a round's calls refuses commits nothing, whatever the calls after it say."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_round
    return verify_round


def test_a_position_past_the_rotation_is_refused_for_good(example):
    """The table of pages holds 64 positions, the rotation's 40: the append refuses what the attention
    does not."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    rng = np.random.default_rng(4)
    s = example.Rounds(example.Model(vocab=300), [rng.integers(0, 300, n).tolist() for n in (37, 3)], max_tokens=40, page_tokens=32)
    for r in range(1, 4):  # session 0 has kv_len 36 .. 40, and each round takes it further by at least one
        before = [list(h) for h in s.history], list(s.kv_len), s.state.cpu().numpy().reshape(2, -1).copy()
        got = s.round([[1, 2, 3], [5]], r)
        past = before[1][0] + 3 >= 40
        assert got[1] and s.kv_len[1] > before[1][1]
        assert bool(got[0]) != past
        if past:
            assert s.refused == {0: sdcp.S_LIMIT}
            assert s.history[0] == before[0][0] and s.kv_len[0] == before[1][0]
            assert np.array_equal(s.state.cpu().numpy().reshape(2, -1)[0], before[2][0])
    assert past


def test_a_prompt_past_the_rotation_is_refused(example):
    with pytest.raises(ValueError):
        example.Rounds(example.Model(vocab=300), [[1, 2], [3] * 50], max_tokens=40, page_tokens=32)


def test_a_prompt_of_one_token_leaves_the_others_their_context(example):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    rng = np.random.default_rng(5)
    prompts = [rng.integers(0, 300, n).tolist() for n in (20, 1, 33, 2)]
    model = example.Model(vocab=300)
    s = example.Rounds(model, prompts, max_tokens=64, page_tokens=32)
    assert s.kv_len == [19, 0, 32, 1]
    off = np.concatenate([[0], np.cumsum(s.kv_len)])
    v = torch.zeros((int(off[-1]), model.kv_heads, model.head_dim), device="cuda:0")
    sdcp.sdcp_read_kv(s.cache, s.page_table, s._int(off.tolist()), int(off[-1]), s._int([0] * 4), None, v, s._int([0] * 4))
    rows = [t for p in prompts for t in p[:-1]]
    want = model.qkv(model.embed[torch.tensor(rows, device="cuda:0")])[2].float()
    # a value is within half a scale of what was appended, and a scale is at most 9/8 of a seventh of the
    # group's largest; the same product over other rows may differ by a bfloat16 rounding
    most = want.unflatten(2, (-1, 32)).abs().amax(dim=3, keepdim=True).expand(-1, -1, -1, 32).flatten(2)
    assert ((v - want).abs() <= most * (9 / 8 / 14 + 2.0**-7)).all()
    assert all(s.round([[7]] * 4, 1)) and not s.refused


def test_an_empty_prompt_is_refused(example):
    with pytest.raises(ValueError):
        example.Rounds(example.Model(vocab=300), [[1, 2], []])
