"""Values that show which keys an attention counted.  Queries are zero, so every visible key has the
same weight; a value row is 1 in the channel of its key's unit and 0 elsewhere.  An output is then the
share of the visible keys that belong to the channel's unit: exact up to the last rounding, and a key
that is left out or counted twice moves it by one part in `unit`.

Roundings: weights are 1 and products, counts and sums exact in 32 bits; the division and the scaling
by it are under 2^-20 together, the output's rounding is half a step of bf16, 2^-8."""
import numpy as np

STEP = 2.0 ** -8 + 2.0 ** -20


def turns(n, unit, channels):
    """How many sets of values mark every unit of n keys once."""
    return max(1, -(-n // (unit * channels)))


def marks(n, unit, channels, turn):
    """[n, channels]: 1 where the key's unit is the channel's in this turn."""
    c = np.arange(n) // unit - turn * channels
    return (c[:, None] == np.arange(channels)).astype(np.float64)


def shares(seen, unit, channels, turn, first=0):
    """[len(seen), channels]: the share of keys first .. seen - 1 in each channel's unit."""
    seen = np.asarray(seen, np.int64)[:, None]
    lo = (turn * channels + np.arange(channels)) * unit
    hits = np.clip(np.minimum(seen, lo + unit) - np.maximum(first, lo), 0, None)
    return hits / np.maximum(seen - first, 1)


def wrong(got, want):
    return np.abs(got - want) > np.abs(want) * STEP
