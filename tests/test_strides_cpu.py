"""The native calls name the tensor whose strides or address a kernel cannot take
(CPU tensors: what is asked of a device comes last)."""
import pytest

torch = pytest.importorskip("torch")

P = 1 << 20


@pytest.fixture(scope="module")
def calls():
    import __graft_entry__
    __graft_entry__.build()
    from head_heterogeneous_block_gb300._device import calls
    return calls


def rows(tokens, heads, d, st, sh, offset=0):
    return torch.zeros(tokens * max(st, 1) + heads * max(sh, 1) + d + offset, dtype=torch.bfloat16).as_strided(
        (tokens, heads, d), (st, sh, 1), offset)


Q, K = (4, 8, 64), (4, 2, 64)


def packed(calls, **kw):
    t = {"q": rows(*Q, 512, 64), "k": rows(*K, 128, 64), "v": rows(*K, 128, 64), "out": rows(*Q, 512, 64), **kw}
    cu = torch.tensor([0, 4], dtype=torch.int32)
    return calls.packed(0, 8, 2, 64, 0.125, 100, 4, 100, t["q"], t["k"], t["v"], cu, None, t["out"], None, P, 1 << 40, P, 0)


def rotary(calls, **kw):
    t = {"q": rows(*Q, 512, 64), "k": rows(*K, 128, 64), "q_out": rows(*Q, 512, 64), "k_out": rows(*K, 128, 64), **kw}
    return calls.rotary(P, 0, 64, t["q"], t["k"], torch.zeros(4, dtype=torch.int32), t["q_out"], t["k_out"], 0)


def store(calls, **kw):
    t = {"q": rows(*Q, 512, 64), "k": rows(*K, 128, 64), "v": rows(*K, 128, 64), "q_out": rows(*Q, 512, 64),
         "k_out": rows(*K, 128, 64), **kw}
    return calls.rotary_store(P, 0, 64, 2, t["q"], t["k"], t["v"], torch.zeros(4, dtype=torch.int32), P,
                              torch.zeros(2, 4, dtype=torch.int64), t["q_out"], t["k_out"], P, 0)


@pytest.mark.parametrize("call", [packed, rotary, store])
def test_strides_and_address_of_the_first_tensor(calls, call):
    with pytest.raises(ValueError, match="q must be on cuda:0"):
        call(calls)                               # nothing wrong but the device
    for st, sh, what in ((512, 60, "heads"), (500, 64, "tokens")):
        with pytest.raises(ValueError, match=f"^q has a stride of .* between {what}"):
            call(calls, q=rows(*Q, st, sh))
    with pytest.raises(ValueError, match="^q must start on a 16-byte boundary"):
        call(calls, q=rows(*Q, 512, 64, offset=1))
    # rows that are one in memory: an input of rotary positions may have them, attention's may not
    for st, sh, what in ((512, 0, "heads"), (0, 64, "tokens"), (512, 56, "heads")):
        with pytest.raises(ValueError, match=f"^q has a stride of .* between {what}" if call is packed else "cuda:0"):
            call(calls, q=rows(*Q, st, sh))


def test_the_stride_of_an_extent_of_one_is_not_used(calls):
    with pytest.raises(ValueError, match="must be on cuda:0"):
        calls.packed(0, 1, 1, 64, 0.125, 100, 4, 100, *[rows(1, 1, 64, 3, 5)] * 3, torch.tensor([0, 1], dtype=torch.int32),
                     None, rows(1, 1, 64, 7, 1), None, P, 1 << 40, P, 0)
