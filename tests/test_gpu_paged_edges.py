"""The paged cache operators on the GPU where calls meet their limits: waits
that give up, aliased arguments, bad pages, other streams and devices."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    return sa, torch


def _q(torch, seed, b, hq, d):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(b, hq, d, generator=g).bfloat16()


def test_attend_of_short_sequences_ends_when_waits_give_up(env):
    # every tile is a segment's first and last, and the waits give up at
    # different tiles; each launch ends, and the next one is right
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(60, [1 + 37 * x % 120 for x in range(400)], 4, 128, 16)
    dev, cache = P.to_gpu(c, sa, with_weights=False)
    q = _q(torch, 50, 400, 32, 128)
    gq = q.cuda()
    out, lse = torch.empty(400, 32, 128, device="cuda"), torch.empty(400, 32, device="cuda")
    try:
        for limit in (1, 200, 500, 1000, 1500, 2000, 3000, 5000):
            sa.sparse_attn_set_wait_limit(limit)
            for _ in range(4):
                cache.attend(gq, out=out, lse=lse)
            torch.cuda.synchronize()
            if limit == 1:
                assert int(cache.dev_status.item()) & sa.SA_DEV_TIMEOUT
    finally:
        sa.sparse_attn_set_wait_limit(0)
    cache.dev_status.zero_()
    cache.attend(gq, out=out, lse=lse)
    assert int(cache.dev_status.item()) == 0
    P.check_attend(c, q, out, lse)
