"""Layouts of outputs whose rows lie between one another without sharing memory are
served; those that share are refused."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_packed import sa  # noqa: E402, F401
from tests.test_rotary_outputs_cpu import collide  # noqa: E402

pytestmark = pytest.mark.gpu


def test_rows_between_one_another(sa):  # noqa: F811
    rot = sa.Rotary(64)
    served = refused = 0
    for tokens, heads, st, sh in ((2, 2, 128, 192), (3, 2, 64, 192), (4, 2, 64, 192), (3, 3, 72, 216), (3, 3, 72, 208),
                                  (5, 4, 64, 320), (6, 4, 64, 320), (2, 5, 320, 64), (2, 6, 320, 64), (3, 2, 200, 264),
                                  (300, 2, 64, 64 * 300), (301, 2, 64, 64 * 300)):
        q = torch.randn(tokens, heads, 64, device="cuda").bfloat16()
        k = torch.randn(tokens, 1, 64, device="cuda").bfloat16()
        pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
        out = torch.zeros(tokens * st + heads * sh + 64, dtype=torch.bfloat16, device="cuda").as_strided(
            (tokens, heads, 64), (st, sh, 1))
        if collide(tokens, heads, st, sh, 64):
            refused += 1
            with pytest.raises(sa.SparseAttnError):
                rot(q, k, pos, q_out=out)
            assert (out == 0).all()
        else:
            served += 1
            rot(q, k, pos, q_out=out)
            assert torch.equal(out, rot(q, k, pos)[0])
    assert served >= 4 and refused >= 4
