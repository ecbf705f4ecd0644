"""Pins of the logits-adjustment and token-table oracles (no GPU)."""
import math

import numpy as np

import oracle


def test_one_row_by_hand():
    x = np.array([2.0, -2.0, 0.0, 4.0, 1.0, np.nan, -np.inf, 3.0])
    prompt = np.array([1, 1, 1, 0, 0, 1, 1, 0], dtype=bool)
    times = np.array([0, 3, 0, 2, 0, 0, 1, 0])
    bias = np.array([0, 0, 0, 0.5, -1, 0, 0, 0.0])
    allowed = np.array([1, 1, 1, 1, 1, 0, 1, 0], dtype=bool)
    y = oracle.adjust_row(x, prompt, times, 2.0, 0.25, 0.125, bias, allowed)
    assert y.tolist() == [1.0, -4.0 - (0.375 + 0.25), 0.0, 2.0 - 0.5 + 0.5, 0.0, -math.inf,
                          -math.inf, -math.inf]


def test_rows_see_the_drafts_before_them():
    cu = np.array([0, 3, 4])
    t = np.zeros((4, 4), dtype=np.float32)
    d = np.zeros((2, 4), dtype=np.float32)
    counts = np.zeros((2, 4), dtype=np.int32)
    counts[1, 2] = 5
    out, dout, st = oracle.adjust_logits(t, cu, d, [1, 1], counts, slots=[0, 1], frequency=1.0,
                                         ctx=[[3, -1]])
    assert st == 0
    assert out.tolist() == [[0, 0, 0, -1], [0, -1, 0, -1], [0, -2, 0, -1], [0, 0, -5, 0]]
    assert dout.tolist() == [[0, 0, 0, -1], [0, -1, 0, -1]]


def test_failing_sequences_are_nan_and_alone():
    cu = np.array([0, 1, 2, 3])
    t = np.ones((3, 4), dtype=np.float32)
    out, _, st = oracle.adjust_logits(t, cu, repetition=np.array([1.0, 0.0, 2.0], np.float32),
                                      bias=[[(9, 1.0)], [], [(1, 2.0), (1, 3.0)]])
    assert st == oracle.DEV_BAD_PARAM | oracle.sampling.DEV_BAD_TOKEN
    assert np.isnan(out[1]).all() and out[0].tolist() == [1] * 4 and out[2].tolist() == [1, 4, 1, 1]


def test_count_table():
    counts = np.zeros((3, 40), dtype=np.int32)
    c, seen, st = oracle.count_tokens(counts, [5, 5, 39, 7, 41, 0], [0, 3, 6], slots=[2, 0],
                                      prompt=True)
    assert st == oracle.DEV_BAD_TOKEN
    assert c[2, 5] == c[2, 39] == c[0, 7] == c[0, 0] == np.int32(-2 ** 31) and (c != 0).sum() == 4
    assert seen.tolist() == [[1 << 7 | 1, 0], [0, 0], [1 << 5, 1 << 7]]
    c, seen, st = oracle.count_tokens(c, [5, 5, 39, 7, 7, 0], [0, 3, 6], num_accepted=[1, -1],
                                      slots=[2, 0])
    assert st == 0 and c[2, 5] == np.int32(-2 ** 31 + 2) and c[2, 39] == np.int32(-2 ** 31)
    assert c[0, 7] == np.int32(-2 ** 31)
    c, seen, _ = oracle.count_tokens(c, [1], [0, 1], slots=[2], reset=True)
    assert (c[2] != 0).sum() == 1 and c[2, 1] == 1 and seen[2].tolist() == [2, 0]
    assert c[0, 7] == np.int32(-2 ** 31)


def test_bits_round_trip():
    rng = np.random.default_rng(2)
    counts = (rng.random((3, 77)) < 0.3).astype(np.int32)
    seen = oracle.seen_bits(counts)
    assert seen.shape == (3, 3)
    for s in range(3):
        assert np.array_equal(oracle.allowed_tokens(seen[s], 77), counts[s] != 0)
        by_hand = [(int(seen[s, t >> 5]) >> (t & 31)) & 1 for t in range(77)]
        assert by_hand == (counts[s] != 0).astype(int).tolist()
