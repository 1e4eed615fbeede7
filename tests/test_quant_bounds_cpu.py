"""How far the 8-bit form's values may be from the rows they hold, as the header states it, in every binade of fp32."""
import os

import numpy as np
from tests import _quant as Q


def test_the_stated_bound():
    rng = np.random.default_rng(149)
    for binade in list(range(-149, 127)) * 4:
        x = (np.clip(rng.standard_normal(64), -1.9, 1.9) * 2.0 ** binade).astype(np.float32).astype(np.float64)
        b = Q.exponent(x)
        far, top = np.abs(Q.nearest(x, b) - x), np.abs(x).max()
        of_largest = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -17 * top)
        assert (far <= np.maximum(of_largest, 2.0 ** -136)).all()
        assert b <= 1 or (far <= of_largest).all()  # the last of the three is for rows at the least exponent alone


def test_the_header_states_it():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "mfs.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    assert "at most 2^-4 of a value, or 2^-17 of the row's largest, or 2^-136" in text
