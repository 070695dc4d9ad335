"""The layouts of q, k, v and outputs that the binding accepts, and the row stride
that it passes on."""
import pytest
import torch

from hstu_pointwise_attention_b200.ops import _row_stride

H, D = 2, 8


def strided(shape, strides):
    return torch.as_strided(torch.zeros(400), shape, strides)


@pytest.mark.parametrize("t,want", [
    (torch.zeros(5, H, D), H * D), (torch.zeros(5, H * D), H * D),
    (strided((5, H, D), (40, D, 1)), 40), (strided((5, H * D), (40, 1)), 40),
    (strided((1, H * D), (40, 1)), H * D),
    # strides without a meaning: of an empty tensor, and of a dimension of size 1
    (torch.zeros(0, H, D), H * D), (strided((0, H, D), (3, 5, 7)), H * D),
    (strided((0, H * D), (3, 7)), H * D), (strided((1, H, D), (3, D, 1)), H * D)])
def test_accepted(t, want):
    assert _row_stride(t, H, D, "x") == want


@pytest.mark.parametrize("t", [
    torch.zeros(()), torch.zeros(16), torch.zeros(5, H, D, 1), torch.zeros(5, D, H),
    torch.zeros(5, H * D + 1), torch.zeros(0, H, D + 1), torch.zeros(0, H * D + 1),
    torch.zeros(0), torch.zeros(5, D, H).transpose(1, 2),
    strided((5, H, D), (40, D + 1, 1)), strided((5, H, D), (40, D, 2)),
    strided((5, H * D), (40, 2))])
def test_refused(t):
    with pytest.raises(ValueError, match="^x: "):
        _row_stride(t, H, D, "x")
