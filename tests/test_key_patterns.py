"""On the CPU: the patterns find a key, a unit or a tile that is left out or counted twice."""
import numpy as np
import pytest

from key_patterns import marks, shares, turns, wrong


@pytest.mark.parametrize("n,unit,channels", [(1, 32, 64), (33, 32, 64), (4100, 32, 128), (20000, 32, 64),
                                             (1000, 1, 128), (3000, 1, 80)])
def test_every_key_and_unit_is_seen(n, unit, channels):
    sets = [marks(n, unit, channels, t) for t in range(turns(n, unit, channels))]
    want = [shares([n], unit, channels, t)[0] for t in range(len(sets))]
    for m, w in zip(sets, want):
        assert np.allclose(m.sum(0) / n, w, rtol=1e-15)
    assert sum(m.sum() for m in sets) == n          # every key in one channel of one set
    edges = [p for u in range(0, n, 32) for p in (u - 1, u, u + 1) if 0 <= p < n]
    for lo, hi in [(p, p + 1) for p in edges] + [(u, min(n, u + 32)) for u in range(0, n, 32)]:
        if hi - lo == n:
            continue
        at = lo // unit // channels
        part = sets[at][lo:hi].sum(0)
        left_out = (sets[at].sum(0) - part) / (n - (hi - lo))
        twice = (sets[at].sum(0) + part) / (n + (hi - lo))
        assert wrong(left_out, want[at]).any() and wrong(twice, want[at]).any()


def test_shares_of_late_starts():
    m = marks(700, 32, 64, 0)
    assert np.allclose(m[37:650].sum(0) / 613, shares([650], 32, 64, 0, first=37)[0])
