"""The beam oracle against an exhaustive search and by hand."""

import itertools
import math

import numpy as np
import pytest

from oracle import beam as ob


def test_by_hand():
    # beam 0: probabilities 1/2, 1/4, 1/4; beam 1: 3/4, 1/8, 1/8 behind a score of ln 1/2
    x = np.log(np.array([[[2.0, 1.0, 1.0], [6.0, 1.0, 1.0]]]))
    s = ob.select(x, [[0.0, math.log(0.5)]], 4, eos=1)
    assert s["parents"].tolist() == [0, 1, 0, 0] and s["tokens"].tolist() == [0, 0, 1, 2]
    assert np.allclose(s["scores"], np.log([0.5, 0.375, 0.25, 0.25]))
    assert s["finished"].tolist() == [False, False, True, False]
    # a finished beam is one candidate; the other beam has no score
    s = ob.select(x, [[-1.0, -math.inf]], 2, finished=[[True, False]], pad=7)
    assert s["tokens"].tolist() == [7, 7] and s["scores"].tolist() == [-1.0, -math.inf]
    assert s["finished"].tolist() == [True, False] and s["parents"].tolist() == [0, 0]


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_without_candidates(bad):
    x = np.zeros((1, 2, 3))
    x[0, 0, 1] = bad
    s = ob.select(x, [[0.0, -1.0]], 2)
    assert s["parents"].tolist() == [1, 1] and s["tokens"].tolist() == [0, 1]


@pytest.mark.parametrize("seed", range(5))
def test_wide_beams_find_the_best_sequences(seed):
    """With as many beams as there are prefixes nothing is lost: the result is the best of all sequences."""
    rng = np.random.default_rng(seed)
    vocab, steps = 3, 3
    tables = [rng.normal(size=(vocab ** t, vocab)) for t in range(steps)]        # logits given the tokens before
    width = vocab ** (steps - 1)
    scores, history, lens = np.full((1, width), -np.inf), np.zeros((1, width, steps), int), np.zeros((1, width), int)
    scores[0, 0] = 0.0
    for t in range(steps):
        prefix = [int("".join(map(str, h[:t])) or "0", vocab) for h in history[0]]
        s = ob.select(tables[t][prefix][None], scores, width, history=history, lens=lens)
        scores, history, lens = s["scores"][None], s["history"][None], s["lens"][None]
    brute = []
    for seq in itertools.product(range(vocab), repeat=steps):
        total = sum(ob.log_probabilities(tables[t][int("".join(map(str, seq[:t])) or "0", vocab)])[seq[t]]
                    for t in range(steps))
        brute.append((total, seq))
    brute.sort(key=lambda b: -b[0])
    assert [tuple(h) for h in history[0]] == [seq for _, seq in brute[:width]]
    assert np.allclose(scores[0], [b for b, _ in brute[:width]])
