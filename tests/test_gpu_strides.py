"""Refusals of strides and addresses name the tensor, and change nothing."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_packed import sa  # noqa: E402, F401

pytestmark = pytest.mark.gpu

Q, K = (4, 8, 64), (4, 2, 64)


def rows(shape, st, sh, offset=0):
    t, h, d = shape
    return torch.zeros(t * max(st, 1) + h * max(sh, 1) + d + offset, dtype=torch.bfloat16, device="cuda").as_strided(
        shape, (st, sh, 1), offset)


@pytest.mark.parametrize("which", ["packed", "rotary", "store"])
def test_strides_and_addresses(sa, which):  # noqa: F811
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, pos = torch.tensor([0, 4], **i32), torch.zeros(4, **i32)
    att, rot = sa.PackedAttention(8, 2, 64), sa.Rotary(64)
    pools = [torch.zeros(4, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = sa.PagedCache(*pools, torch.zeros(1, 2, 2, **i32), torch.zeros(1, 2, **i32))
    slots = torch.arange(8, device="cuda").view(2, 4)

    def call(**kw):
        t = {n: torch.ones(Q if n in ("q", "out", "q_out") else K, dtype=torch.bfloat16, device="cuda")
             for n in ("q", "k", "v", "out", "q_out", "k_out")}
        t.update(kw)
        if which == "packed":
            att(t["q"], t["k"], t["v"], cu, out=t["out"])
        elif which == "rotary":
            rot(t["q"], t["k"], pos, q_out=t["q_out"], k_out=t["k_out"])
        else:
            rot.store(t["q"], t["k"], t["v"], pos, cache, slots, q_out=t["q_out"], k_out=t["k_out"])

    names = {"packed": ("q", "k", "v", "out"), "rotary": ("q", "k", "q_out", "k_out"),
             "store": ("q", "k", "v", "q_out", "k_out")}[which]
    for name in names:
        shape = Q if name in ("q", "out", "q_out") else K
        least = which == "packed" or name.endswith("out")
        for st, sh, what in ((512, 60, "heads"), (500, 64, "tokens")) + (
                ((512, 0, "heads"), (0, 64, "tokens"), (512, 56, "heads")) if least else ()):
            with pytest.raises(ValueError, match=f"^{name} has a stride of .* between {what}"):
                call(**{name: rows(shape, st, sh)})
        with pytest.raises(ValueError, match=f"^{name} must start on a 16-byte boundary"):
            call(**{name: rows(shape, 512, 64, offset=1)})
        if not least:
            call(**{name: rows(shape, 0, 0)})
    call()
    torch.cuda.synchronize()
    assert int(att.dev_status.item()) == 0 and int(rot.dev_status.item()) == 0
