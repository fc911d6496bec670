"""Wait limits far below a copy's time end the decode step's waits every time."""
import pytest

pytestmark = pytest.mark.gpu


def test_decode_step_wait_timeouts_are_reported_every_time():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    from tests._parity import to_dev
    from workloads import generate, workload
    w = workload(5)
    x = generate.decode_inputs(w)
    shape = sa.Shape.decode(w.seq_len, w.block, w.num_q_heads, w.num_kv_heads, w.head_dim, w.batch)
    plan = sa.sparse_attn_plan(shape, w.budget_tokens // w.block, head_kind=generate.head_kinds(w),
                               window_blocks=w.window_tokens // w.block, num_workers=1)
    plan.upload()
    kmax = plan.info()["kmax"]
    q, k, v = (to_dev(x[n]) for n in "qkv")
    rows = w.batch * w.num_q_heads
    kbar = torch.empty(w.batch * w.num_kv_heads * w.nb * w.head_dim, device="cuda")
    sa.sparse_attn_pool_kcache(shape, k, kbar)
    idx = torch.empty(rows, kmax, dtype=torch.int32, device="cuda")
    cnt = torch.empty(rows, dtype=torch.int32, device="cuda")
    out = torch.empty(rows, w.head_dim, device="cuda")
    st = torch.zeros(300, dtype=torch.int32, device="cuda")
    flush = torch.zeros(256 * 1024 * 1024, dtype=torch.uint8, device="cuda")

    def step(status):
        sa.sparse_attn_decode_step(shape, plan, q, kbar, k, v, None, idx, cnt, kmax, out, None, status)

    step(st[:1])
    assert int(st[0]) == 0
    want = out.clone()
    sa.sparse_attn_set_wait_limit(1)
    try:
        for i in range(len(st)):
            flush.max()                    # the copies come from memory, not L2
            step(st[i:])
        torch.cuda.synchronize()
    finally:
        sa.sparse_attn_set_wait_limit(0)
    late = (st & sa.SA_DEV_TIMEOUT) == 0
    assert not late.any(), f"{int(late.sum())} of {len(st)} launches did not time out"
    st.zero_()
    step(st[:1])
    assert int(st[0]) == 0 and torch.equal(out, want)
