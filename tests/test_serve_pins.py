"""Pins of oracle.serve: hand-worked values, closed forms and brute force, on the CPU."""
import itertools

import numpy as np
import pytest
from scipy.special import logsumexp, softmax

from oracle import serve


def test_reserve_by_hand():
    """Two sequences of one layer and two heads, pages of 4; lengths 3, 4 | 0, 9; counts 2 and 1."""
    bt = np.array([[5, -1, -1], [6, -1, -1], [-1, -1, -1], [0, 1, 2]], dtype=np.int32)
    free = np.array([9, 8, 7, 4, 3], dtype=np.int32)
    pos = np.zeros((4, 12), dtype=np.int32)
    r = serve.reserve_slots(bt, np.array([3, 4, 0, 9], dtype=np.int32), pos, None, np.ones((4, 12)),
                            np.array([2, 1]), np.array([10, 20]), 1, free, 5, 4, 1, 2, 4, 10)
    # rows 0, 1 and 2 open a page each (slots 4, 4 and 0); row 3's slot 9 lies in page 2, which it holds
    assert r["bt"].tolist() == [[5, 7, -1], [6, 4, -1], [3, -1, -1], [0, 1, 2]] and r["depth"] == 2
    assert r["slot_map"][:, 0].tolist() == [[23, 16], [28, 17], [12, 9], [-1, -1]]
    assert r["token_pos"].tolist() == [10, 11, 20, -1] and r["token_start"].tolist() == [0, 2, 3]
    assert r["row_len"].tolist() == [5, 6, 1, 10] and r["slot_pos"][0, 3:5].tolist() == [10, 11]
    assert r["crf"][3].tolist() == [1] * 9 + [0, 1, 1]
    short = serve.reserve_slots(bt, np.array([3, 4, 0, 9], dtype=np.int32), pos, None, None, np.array([2, 1]),
                                np.array([10, 20]), 1, free, 2, 4, 1, 2, 4, 10)
    assert short["depth"] == 2 and np.array_equal(short["bt"], bt) and (short["slot_map"] == -1).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 1, 2, 16))
    pos, f = np.array([0, 5, 11]), np.array([1.0, 0.25, 0.1, 0.03])
    y, reach = serve.norm_rope(x, None, 0.0, pos, f, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])
    a, b = (0, 1) if interleaved else (0, 4)
    want = np.cos(5.0) * x[1, 0, 0, a] - np.sin(5.0) * x[1, 0, 0, b]
    assert abs(y[1, 0, 0, a] - want) < 1e-14 and (np.abs(y) <= reach + 1e-12).all()
    # q . k of rotated vectors depends on the distance of their positions alone
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    dots = [(serve.norm_rope(q, None, 0, np.array([i + 7]), f, interleaved)[0] *
             serve.norm_rope(k, None, 0, np.array([i]), f, interleaved)[0])[..., :8].sum() for i in (0, 3, 1000)]
    assert np.ptp(dots) < 1e-10
    w = np.full((1, 16), 2.0)
    n = serve.norm_rope(x, w, 0.0, pos, f, interleaved)[0]
    assert np.allclose((n * n).mean(-1), 4.0)


def test_bounds_hold_for_every_key_and_query():
    rng = np.random.default_rng(2)
    keys, q = rng.standard_normal((22, 8)), rng.standard_normal((3, 8))
    for b, (lo, hi, first) in enumerate(serve.block_bounds(keys, np.arange(22)[::-1], 5)):
        top = np.maximum(q * lo, q * hi).sum()
        assert (keys[5 * b:5 * b + 5] @ q.T).sum(1).max() <= top + 1e-12
        assert first == 21 - min(21, 5 * b + 4)


def test_choice_by_brute_force():
    """The chosen pages have the largest total score of all choices of that many, and hold the pinned ones."""
    rng = np.random.default_rng(3)
    for trial in range(30):
        keys, q = rng.standard_normal((27, 4)), rng.standard_normal((2, 4))
        bounds = serve.block_bounds(keys, np.arange(27), 4)
        sink, recent, k = trial % 2, trial % 3, 3 + trial % 3
        got = serve.select_blocks(bounds, q, 23, k, sink, recent)
        scores = [np.maximum(q * lo, q * hi).sum() for lo, hi, _ in bounds]
        seen = [b for b in range(7) if 4 * b <= 23]
        pinned = {b for b in seen if b < sink or b >= 7 - recent}
        best = max((c for c in itertools.combinations(seen, k) if pinned <= set(c)), key=lambda c: sum(scores[b] for b in c))
        assert got == list(best)
    same = [(np.zeros(4), np.zeros(4), 0)] * 6
    assert serve.select_blocks(same, q, 0, 3, 0, 1) == [0, 1, 5]
    assert serve.select_blocks(same, q, -1, 3, 0, 1) == []


def test_attention_against_scipy():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 8)), rng.standard_normal((20, 8)), rng.standard_normal((20, 8))
    pos = np.arange(20)
    out, lse, reach, _ = serve.attention(q, k, v, pos, 12, [0, 1, 2, 10, 11, 12, 13])
    logit = q @ k[[0, 1, 2, 10, 11, 12]].T / np.sqrt(8)
    assert np.allclose(lse, logsumexp(logit, axis=1)) and np.allclose(out, softmax(logit, axis=1) @ v[[0, 1, 2, 10, 11, 12]])
    assert (np.abs(out) <= reach).all()
    assert serve.attention(q, k, v, pos, -1)[1].tolist() == [-np.inf] * 3


@pytest.mark.parametrize("mistake", ["stack bottom", "row order", "floor", "scale", "swap", "mask"])
def test_planted_mistakes_are_caught(mistake, monkeypatch):
    if mistake in ("stack bottom", "row order", "floor"):
        real = serve.reserve_slots

        def wrong(bt, row_len, *a):
            r = real(bt, row_len, *a)
            if mistake == "stack bottom":
                r["depth"] += 1
            elif mistake == "row order":
                r["bt"][[0, 1]] = r["bt"][[1, 0]]
            else:
                r["slot_map"] = np.where(r["slot_map"] >= 0, r["slot_map"] // 4 * 4, -1)
            return r
        monkeypatch.setattr(serve, "reserve_slots", wrong)
        check = test_reserve_by_hand
    elif mistake == "swap":
        real = serve.norm_rope
        monkeypatch.setattr(serve, "norm_rope", lambda *a: real(*a[:-1], not a[-1]))

        def check():
            test_rotation_is_a_rotation(False)
    else:
        real = serve.attention

        def wrong(q, k, v, pos, q_pos, slots=None):
            return real(q * (1.1 if mistake == "scale" else 1), k, v, pos, q_pos + (mistake == "mask"), slots)
        monkeypatch.setattr(serve, "attention", wrong)
        check = test_attention_against_scipy
    with pytest.raises(AssertionError):
        check()
