"""What PackedAttention reserves."""
import pytest

torch = pytest.importorskip("torch")

from tests import _packed as tp  # noqa: E402
from tests.test_gpu_packed import run, sa  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def need(sa, heads, d, tokens, keys, batch):  # noqa: F811
    return sa.sparse_attn_packed_workspace_size(sa.PackedShape(
        total_q=tokens, total_k=keys, batch=batch, num_q_heads=heads, num_kv_heads=heads, head_dim=d, scale=1.0))


def test_a_short_prompt_reserves_no_rounds(sa):  # noqa: F811
    # 16 KV heads of 128: from 8192 keys on their states take several rounds' room
    att = sa.PackedAttention(16, 16, 128)
    q, k, v, cq, ck = tp.inputs(110, [41], [41], 16, 16, 128, device="cuda")
    tp.same(att(q, k, v, cq), run(sa, 16, 16, 128, q, k, v, cq, cq)[0])
    assert att._ws_bytes <= need(sa, 16, 128, 8192, 8192, 64) < 30e6
    # and as many keys as there are make it grow
    q, k, v, cq, ck = tp.inputs(111, [300], [40000], 16, 16, 128, device="cuda")
    att(q, k, v, cq, ck)
    assert need(sa, 16, 128, 8192, 40000, 64) <= att._ws_bytes
    assert att._ws_bytes > 150e6 and int(att.dev_status.item()) == 0


def test_rounds_by_the_size_of_keys_and_values(sa):  # noqa: F811
    # (sizes of 16 heads of 128: 8192 bytes a key)
    one = need(sa, 16, 128, 100, 8192, 1)
    for keys, rounds in ((8193, 2), (16384, 2), (16385, 4), (32768, 4), (32769, 8), (1 << 20, 8)):
        assert abs(need(sa, 16, 128, 100, keys, 1) / one - rounds) < 0.05
    assert 19e6 < one < 23e6 and 9.5e6 < need(sa, 16, 64, 100, 100, 1) < 12e6
