"""Which rows sdcp_attend_shared_kv attends together, seen from its workspace.

The output is the same up to rounding whether a group's pages are read once or for each session.  The workspace
holds a reference and a sum for each pair of a row and a head that has a session's part beside a group's; a pair
that has none keeps the mark (0, -1), which no reference and sum can be (a sum of weights is not negative)."""
import numpy as np
import pytest
import torch

from test_gpu_attend_shared import Shared, _built  # noqa: F401  (a fixture: the library is built)

pytestmark = pytest.mark.gpu
MARK = -0x4080000000000000  # the floats (0, -1) as a whole number


def case(n=6, common=10, refuse=(), seed=40, D=64):
    r = np.random.default_rng(seed)
    lens = (common * 128 + r.integers(0, 900, n)).tolist()
    c = Shared([n], [common], r.integers(0, 4, n).tolist(), lens, P=128, Hkv=2, share=4, D=D, seed=seed)
    for b, how in refuse:
        if how == "ended":  # as sdcp_release_kv leaves a slot's row, and a round keeps it out
            c.lens[b] = -1
            c.table[b] = -1
        elif how == "entry":
            c.table[b, 0] = -1
        elif how == "late entry":
            c.table[b, common - 1] = c.n_pages
        else:
            c.lens[b] = 2**31 - 1
    return c


def joined(c, offsets, bad=()):
    """The number of rows that have two parts; the output is checked."""
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    c.group_offsets = np.array(offsets, dtype=np.int32)
    t = c.tensors(workspace_fill=0)
    sdcp.sdcp_attend_shared_kv(*t, scale=c.scale)
    torch.cuda.synchronize()
    c.check(t[7], t[8].cpu().numpy(), bad)
    pairs = (c.total + len(c.ms)) * c.Hq - int((t[9].view(torch.int64) == MARK).sum())
    assert pairs % c.Hq == 0
    return pairs // c.Hq


def rows(c, b0, b1, bad=()):
    return sum(c.ms[b] + 1 for b in range(b0, b1) if b not in bad)


@pytest.mark.parametrize("D", [64, 128])
def test_a_group_is_attended_together(D):
    c = case(D=D)
    assert joined(c, range(7)) == 0
    assert joined(c, [0, 6]) == rows(c, 0, 6)
    assert joined(c, [0, 2, 3, 6]) == rows(c, 0, 2) + rows(c, 3, 6)
    # one entry apart: what is before it is shared, and nothing where it is the first
    c.table[3, 7] = c.table[3, 10]
    assert joined(c, [0, 6]) == rows(c, 0, 6)
    c.table[3, 0] = c.table[3, 10]
    assert joined(c, [0, 6]) == 0


@pytest.mark.parametrize("refuse", [[(1, "ended")], [(0, "ended")], [(0, "entry")], [(0, "late entry")], [(0, "limit")],
                                    [(0, "ended"), (1, "entry"), (2, "limit")], [(0, "entry"), (3, "ended")]])
def test_a_refused_member_does_not_end_the_sharing(refuse):
    c, bad = case(refuse=refuse), [b for b, _ in refuse]
    assert joined(c, [0, 6], bad) == rows(c, 0, 6, bad)


def test_many_refused_members_before_the_first_that_is_not():
    n, how = 310, ("ended", "entry", "limit")
    c = case(n=n, common=2, refuse=[(b, how[b % 3]) for b in range(300)])
    assert joined(c, [0, n], range(300)) == rows(c, 300, n)
    c = case(n=n, common=2, refuse=[(b, how[b % 3]) for b in range(n)])
    assert joined(c, [0, n], range(n)) == 0
