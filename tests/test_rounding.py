"""The check of bf16 outputs against itself (CPU): what it passes and what it finds."""
import numpy as np
import pytest
import torch

import rounding


def _values(n=200_000):
    r = np.random.default_rng(0)
    return r, r.normal(size=n)


def test_steps_and_nearest():
    v = np.array([1.0, 1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, -1.999, 0.0, 3e-3])
    assert rounding.step(v[:2]).tolist() == [2.0 ** -7, 2.0 ** -7]
    assert rounding.nearest(v).tolist() == torch.tensor(v).float().bfloat16().tolist()


@pytest.mark.parametrize("err", [0.0, 1e-7, 1e-5])
def test_passes_what_is_as_good_as_it_says(err):
    r, v = _values()
    assert rounding.faults(rounding.nearest(v + err * r.normal(size=v.size)), v, np.full(v.size, err)) is None


@pytest.mark.parametrize("name,spoil", [
    ("cut to two bf16 parts before the rounding", lambda v: v * (1 - 2.0 ** -16)),
    ("a sum of which 2^-15 is lost", lambda v: v - 2.0 ** -15),
    ("scaled by 1.01", lambda v: v * 1.01),
    ("zeros", lambda v: 0 * v)])
def test_finds(name, spoil):
    _, v = _values()
    err = 40 * 2.0 ** -24 * np.abs(v)
    assert rounding.faults(rounding.nearest(spoil(v)), v, err) is not None
    assert rounding.faults(rounding.nearest(v), v, err) is None


def test_finds_one_output_a_step_off():
    _, v = _values(1000)
    got = rounding.nearest(v)
    got[3] += 2 * rounding.step(got[3])
    assert rounding.faults(got, v, 1e-6 * np.abs(v)) is not None
