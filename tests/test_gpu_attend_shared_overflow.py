"""Scores beyond binary32's range: one that becomes minus infinity has no weight, wherever it stands.

Keys are 7 times their scale in every channel and queries -2^120 in all 64, so the score of a token of scale s is
-2^120 * 64 * 7 s: beyond 2^128 from s = 2^-6 on (byte 72), and 2^114.8 for s = 2^-14 (byte 8).  One token is of
byte 8, the others' scales are at least twice its, so it leads by 2^114 or more and has all the weight: the
output is its value, rounded once to bfloat16 (2^-8 of it)."""
import numpy as np
import pytest

from test_gpu_attend_shared import Shared, _built  # noqa: F401  (a fixture: the library is built)
import serving_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64])
@pytest.mark.parametrize("best", [1, 37, 200, 700, 1663, 1666])
@pytest.mark.parametrize("members,common", [(1, 0), (2, 13), (40, 13)])
def test_a_score_of_minus_infinity_has_no_weight(members, common, best, D):
    r = np.random.default_rng(best)
    c = Shared([members], [common], [1] * members, [1700 + b for b in range(members)], P=128, Hkv=1, share=4, D=D, seed=best, scale=1.0)
    for b in range(members):
        for t in range(c.lens[b] + 2):
            page, slot = c.pages[c.table[b, t // 128], 0, 0], t % 128
            # whole tiles beyond the range, and tokens among others, a tile's and a call's first among them
            huge = t // 128 in (0, 3, 12) or t % 5 == 0 or t >= c.lens[b]
            page[128 * 32 + slot * 2:128 * 32 + slot * 2 + 2] = 8 if t == best else int(r.integers(160, 168) if huge else r.integers(16, 40))
            for g in range(2):
                page[(g * 128 + slot) * 16:(g * 128 + slot) * 16 + 16] = 0xFF
    c.q[:] = np.float32(-2.0**120)
    out, st = c.run()
    assert st.tolist() == [0] * members
    got = out.double().cpu().numpy()
    for b in range(members):
        want = ref.block_values(c.pages[c.table[b, best // 128], 0, 1], 128, D)[best % 128]
        assert (np.abs(got[2 * b:2 * b + 2] - want) <= 2.0**-8 * np.abs(want)).all()


@pytest.mark.parametrize("members,common", [(1, 0), (2, 13), (40, 13)])
def test_a_query_with_an_infinity_gives_nan_in_its_row_alone(members, common):
    """All its scores are infinite, of one sign: no weight at all, or infinite ones."""
    c = Shared([members], [common], [1] * members, [1700 + b for b in range(members)], P=128, Hkv=1, share=4, D=64, seed=members, scale=1.0, q_scale=0.1)
    for b in range(members):
        for t in range(c.lens[b] + 2):
            page, slot = c.pages[c.table[b, t // 128], 0, 0], t % 128
            for g in range(2):
                page[(g * 128 + slot) * 16:(g * 128 + slot) * 16 + 16] = 0xFF
    some = range(0, 2 * members, 3)
    for r in some:
        c.q[r, r % 4, r % 64] = -np.inf if r % 2 == 0 else np.inf
    c.check(*c.run(), nan_rows={(r, r % 4) for r in some})
