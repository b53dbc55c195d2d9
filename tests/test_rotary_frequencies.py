"""The scaled rotary frequencies (host): where the ramp over the pairs' indices begins and ends, and what is refused."""
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build
    build()
    import paged_kv_cache_261_gb300 as pa
    return pa


def by_index(rd, base, scale, length, low, high):
    """Pair by pair: the index at which a pair makes n turns over the length, a ramp between that of `high` turns,
    rounded down, and that of `low`, rounded up, within [0, rd - 1]."""
    at = [rd * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high, low)]
    a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
    f = []
    for j in range(rd // 2):
        w = base ** (-2.0 * j / rd)
        r = min(1.0, max(0.0, (j - a) / max(b - a, 0.001)))          # how far down the ramp
        f.append(w * (1 - r) + w / scale * r)
    return f


@pytest.mark.parametrize("rd,base,scale,length,low,high", [
    (128, 1e4, 8.0, 65536, 1.0, 32.0),       # the last pair makes more than `low` turns: the ramp ends behind it
    (128, 1e4, 8.0, 10 ** 6, 1.0, 32.0), (64, 1e4, 4.0, 131072, 2.0, 64.0), (32, 500.0, 16.0, 32768, 1.0, 4.0),
    (16, 100.0, 2.0, 10 ** 9, 1.0, 2.0),     # and begins behind it
    (128, 1e4, 40.0, 4096, 1.0, 32.0), (128, 1e6, 4.0, 32768, 1.0, 32.0), (64, 5e5, 8.0, 8192, 1.0, 4.0)])
def test_by_index(pa, rd, base, scale, length, low, high):
    got = pa.rotary_frequencies(rd, base, "by_index", scale, length, low, high)
    assert np.allclose(got, by_index(rd, base, scale, length, low, high), rtol=1e-12, atol=0)


def test_by_index_at_the_last_pair(pa):
    """65536 tokens, base 10,000, 64 pairs: a turn belongs to index 64.3, so the ramp ends at 65, not at the last pair's
    63, which is two steps of 65 - 40 short of it. (32 turns belong to index 40.2.)"""
    f = pa.rotary_frequencies(128, 1e4, "by_index", 8.0, 65536, 1.0, 32.0)
    plain = 1e4 ** (-63 / 64)
    r = (63 - 40) / (65 - 40)
    assert math.isclose(f[63], plain * (1 - r) + plain / 8 * r, rel_tol=1e-12)
    assert math.isclose(f[40], 1e4 ** (-40 / 64), rel_tol=1e-12) and f[41] < 0.99 * 1e4 ** (-41 / 64)


@pytest.mark.parametrize("scaling", ["by_turns", "by_index"])
@pytest.mark.parametrize("bad", [dict(original_len=0), dict(original_len=-8192), dict(original_len=float("nan")),
                                 dict(high=float("inf")), dict(high=float("nan")), dict(scale=float("nan")),
                                 dict(base=float("inf")), dict(original_len=float("inf")), dict(scale=float("inf"))])
def test_what_gives_no_frequencies_is_refused(pa, scaling, bad):
    with pytest.raises(ValueError):
        pa.rotary_frequencies(8, scaling=scaling, **{**dict(scale=2.0), **bad})
