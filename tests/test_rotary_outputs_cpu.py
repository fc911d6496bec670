"""Outputs of rotary positions that would be written twice are refused (nothing
touches a device: the addresses are read by nobody)."""
import itertools

import pytest

from tests.test_serving_cpu import P, _desc, _rot, _rotary, _store, sa  # noqa: F401


@pytest.mark.parametrize("change", [dict(qo=5 * P), dict(ko=5 * P)])
def test_an_output_at_the_values(sa, change):  # noqa: F811
    assert _store(sa, _rot(sa), _desc(sa), **change) == 1


def collide(tokens, heads, st, sh, d):
    at = sorted(t * st + h * sh for t in range(tokens) for h in range(heads))
    return any(b - a < d for a, b in zip(at, at[1:]))


def test_outputs_whose_rows_share_memory(sa):  # noqa: F811
    # every small layout, by comparing all rows: the ones that share are refused, of both outputs; one that does not
    # goes on to what is refused after it (the address of another input, or a missing status word)
    seen = set()
    for tokens, heads, st, sh in itertools.product((1, 2, 3, 5, 9), (1, 2, 3, 8), range(128, 1100, 72), range(128, 1100, 56)):
        shares = collide(tokens, heads, st, sh, 128)
        seen.add(shares)
        if not shares:
            continue
        r = _rot(sa)
        assert _rotary(sa, r, tokens=tokens, hq=heads, qos=(st, sh)) == 1
        assert _rotary(sa, r, tokens=tokens, hkv=heads, ks=(256, 128), kos=(st, sh)) == 1
        assert _store(sa, r, _desc(sa, num_kv_heads=heads), tokens=tokens, kos=(st, sh)) == 1
    assert seen == {True, False}
