"""That the fp32 check of the paged attention tells two bf16 parts of the
softmax weights from three."""
import pytest

from tests import _paged_fp32 as F


@pytest.mark.parametrize("d", [64, 128])
def test_check_sees_the_third_part(d):
    c, q = F.inputs(5, [0, 1, 24, 64, 100, 128], 2, 4, d, 32)
    three = F.check(c, q, F.expected(c, q, 3), unit=128)
    two = F.check(c, q, F.expected(c, q, 2), unit=128)
    assert (three < 0.1).all(), three
    assert (two[2:] > 1.5).all(), two
