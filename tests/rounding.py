"""Whether bf16 outputs are fp32 results rounded once.

An output that is off by `err` before its rounding differs from the bf16 nearest the
64-bit value where that value lies within `err` of the middle between two bf16 numbers:
with probability err / step.  So the number of outputs that differ says how far off they
were, hundreds of times below the rounding itself, where a bound on each output alone
must allow for half a step."""
import numpy as np


def step(v):
    """The distance of bf16 numbers at |v|."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - 7)


def nearest(v):
    """The bf16 number nearest to a float64 (ties to even)."""
    s = step(v)
    return np.rint(v / s) * s


def faults(got, want, err):
    """What is wrong with bf16 outputs `got` of 64-bit values `want` that are known to
    `err` (a standard deviation, for each): None, or a sentence."""
    s = step(np.maximum(np.abs(want), np.abs(got)))
    off = np.abs(got - want)
    if not (off <= s / 2 + 16 * err).all():
        return f"an output is off by {(off / (s / 2 + 16 * err)).max()} times half a step and 16 err"
    chance = np.minimum(1.0, err / s).sum()
    most = chance + 6 * chance ** 0.5 + 6  # six deviations of a count of rare events
    differ = int((got != nearest(want)).sum())
    return None if differ <= most else \
        f"{differ} of {got.size} outputs are not the nearest bf16; {most:.0f} at most expected"
