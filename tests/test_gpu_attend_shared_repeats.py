"""sdcp_attend_shared_kv, called over and over: every output is the first one's, bit for bit.

The warp that issues the products waits for two barriers at once; what both stand for has to be there before a
product reads it."""
import pytest
import torch

from test_gpu_attend_shared import Shared, _built  # noqa: F401  (a fixture: the library is built)

pytestmark = pytest.mark.gpu


# items of one block and of two, whole ones and cut ones
@pytest.mark.parametrize("members,m,share,D", [(2, 0, 4, 128), (24, 3, 8, 64), (24, 3, 8, 128), (3, 60, 7, 64)])
def test_repeats_are_bit_equal(members, m, share, D):
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    c = Shared([members], [20], [m] * members, [1280 + 40 * b for b in range(members)], P=64, Hkv=2, share=share, D=D, seed=members)
    t = c.tensors()
    sdcp.sdcp_attend_shared_kv(*t, scale=c.scale)
    first = t[7].clone().view(torch.int16)
    different = torch.zeros((), dtype=torch.int64, device=first.device)
    for _ in range(300):
        t[7].fill_(float("nan"))
        sdcp.sdcp_attend_shared_kv(*t, scale=c.scale)
        different += (t[7].view(torch.int16) != first).sum()
    assert different.item() == 0 and t[8].tolist() == [0] * members
    assert bool(torch.isfinite(t[7].float()).all())
