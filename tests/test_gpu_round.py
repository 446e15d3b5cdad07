"""The serving operators together, as examples/verify_round.py runs them: under Rule 1 the tokens of
a session do not depend on its drafter (SDCP draft Section 6.4), so rounds with different drafts emit
the same text; a drafter that proposes what the verifier will say has everything accepted."""
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


def _text(example, drafter, tokens=14, banned=()):
    rng = np.random.default_rng(3)
    model = example.Model(vocab=500)
    prompts = [rng.integers(0, 500, n).tolist() for n in (2, 40, 131, 17)]
    s = example.Rounds(model, prompts, banned=banned)
    r = 0
    accepted = 0
    while min(len(h) - len(p) for h, p in zip(s.history, prompts)) < tokens:
        r += 1
        drafts = drafter(s, r)
        got = s.round(drafts, r)
        accepted += sum(len(g) - 1 for g in got)
    return [h[len(p):len(p) + tokens] for h, p in zip(s.history, prompts)], accepted


def test_the_text_does_not_depend_on_the_drafter(example):
    rng = np.random.default_rng(9)
    a, _ = _text(example, lambda s, r: [rng.integers(0, 500, 1).tolist() for _ in range(4)])
    b, _ = _text(example, lambda s, r: [rng.integers(0, 500, int(rng.integers(1, 9))).tolist() for _ in range(4)])
    assert a == b

    def knowing(s, r):
        done = [len(h) - n for h, n in zip(s.history, s.prompt_len)]
        return [(t[d:d + 5] + [0])[:5] for t, d in zip(a, done)]

    c, accepted = _text(example, knowing)
    assert a == c and accepted >= 4 * 10


def test_a_banned_token_is_never_emitted(example):
    rng = np.random.default_rng(9)
    a, _ = _text(example, lambda s, r: [rng.integers(0, 500, 2).tolist() for _ in range(4)])
    banned = {t for text in a for t in text[:3]}
    b, _ = _text(example, lambda s, r: [rng.integers(0, 500, 2).tolist() for _ in range(4)], banned=sorted(banned))
    assert not banned & {t for text in b for t in text}
