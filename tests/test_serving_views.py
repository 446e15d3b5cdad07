"""What the binding takes as rows of heads: the stride of a dimension of size one says nothing."""
import pytest
import torch


@pytest.fixture(scope="module")
def heads():
    from speculative_decoding_verification_sdcp_gb300 import build_ext
    build_ext.build()
    from speculative_decoding_verification_sdcp_gb300 import sdcp
    return lambda t, rows, n: sdcp._heads(t, rows, n, 64, "k")


def test_strides_of_single_heads_and_rows(heads):
    one = torch.zeros((1, 5, 64)).transpose(0, 1)          # [5, 1, 64], the head's stride is 5 * 64
    assert one.stride() == (64, 320, 1) and heads(one, 5, 1) == 64
    wide = torch.zeros((5, 3 * 64)).as_strided((5, 1, 64), (192, 7, 1))
    assert heads(wide, 5, 1) == 192
    row = torch.zeros((4, 64)).as_strided((1, 4, 64), (1, 64, 1))
    assert heads(row, 1, 4) == 4 * 64
    assert heads(torch.zeros((6, 10, 64))[:, 2:5], 6, 3) == 640


def test_gaps_are_refused(heads):
    for bad in (torch.zeros((5, 4, 64))[:, ::2], torch.zeros((5, 2, 128))[:, :, ::2], torch.zeros((2, 5, 64)).transpose(0, 1),
                torch.zeros((5, 2, 32)), torch.zeros((4, 2, 64)), torch.zeros((5, 128))):
        with pytest.raises(ValueError):
            heads(bad, 5, 2)
