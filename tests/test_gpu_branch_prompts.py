"""Prompts of a token in examples/branch_round.py."""
import pytest

from test_gpu_branch_round import examples  # noqa: F401  (a fixture: the library is built, the examples are on the path)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[1], [1, 1, 1], [1, 40, 1]])
def test_prompts_of_one_token(examples, lengths):  # noqa: F811
    """All of a prompt but its last token is cached before the first round: nothing, of a prompt of one."""
    branch_round, verify_round = examples
    run = branch_round.Branches(verify_round.Model(vocab=300), [list(range(5, 5 + n)) for n in lengths], 2, pool_pages=40)
    assert run.kv_len == [n - 1 for n in lengths for _ in range(2)]
    for r in range(1, 4):
        emitted = run.round([[7, 9, 11]] * run.B, r)
        assert not run.refused and all(emitted)
