"""The precision cases of the attention tell the mistakes apart that they are there for (planted here, in numpy)."""
import numpy as np

from tests.serve_precision import CHUNK, JOINS, RUN, SMALL, TWO_SLOTS, drift, parts


def test_two_parts_of_a_probability_are_outside_the_bound_and_three_inside():
    p = np.exp2(-4 * np.random.default_rng(1).random(4000))
    err = lambda k: np.abs(parts(p, k) / p - 1).max()
    assert err(3) < TWO_SLOTS / 4 and err(2) > 1.5 * TWO_SLOTS


def test_truncated_runs_are_outside_the_bound_and_rounded_ones_inside():
    assert np.float64(np.float32(CHUNK.sum())) == CHUNK.sum() and SMALL * 2**15 == 15
    for r in (RUN, RUN + 1):
        assert abs(drift(r)) < 40 * 2.0**-24 and abs(drift(r, truncate=True)) > abs(drift(r)) + 3 * JOINS
