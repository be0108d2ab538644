"""What the block-scaled bindings hand to the C interface (CPU: no device is needed)."""
import pytest
import torch

from bit_quantized_b200 import build as q8build

q8build.build()
from bit_quantized_b200 import q8  # noqa: E402


@pytest.mark.parametrize("stride", [0, 1, 65, 1000])
def test_the_stride_of_a_single_row_does_not_matter(stride):
    # torch leaves it as it was made: an unaligned one is no reason to refuse the call
    t = torch.empty_strided((1, 64), (stride, 1), dtype=torch.bfloat16)
    assert q8._ld(t) == 64
    assert q8._ld(torch.empty_strided((2, 64), (72, 1))) == 72
