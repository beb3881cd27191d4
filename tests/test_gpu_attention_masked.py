"""What masked keys and vanishing weights must not change: windows without end, NaN values far below the
largest score."""

import numpy as np
import pytest
import torch

from tests.test_gpu_attention import Problem
from tests.test_gpu_attention_variants import FORMS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [(1 << 63) - 1, 1 << 62, 1 << 31, 5000])
@pytest.mark.parametrize("form", FORMS)
def test_windows_past_every_length_are_none(form, window):
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs, heads, hk, 64, 16, seed=5)
    out, lse = p.run()
    got, got_lse = p.run(window=window)
    assert torch.equal(out, got) and torch.equal(lse, got_lse)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q_len", [1, 40])
def test_nan_values_under_vanishing_weights(q_len, dtype):
    """A visible NaN value is in the sum however small its weight, in calls that split the keys as in others: here its
    score lies some 370 powers of two below those of the later keys, in the first of several splits."""
    p = Problem([(q_len, 3000)], 4, 2, 64, dtype=dtype, seed=2)
    k = np.where(np.arange(3000) < 300, -4.0, 4.0)[:, None, None] * np.ones((3000, 2, 64))
    slots = p.table[0, np.arange(3000) // 16].astype(np.int64) * 16 + np.arange(3000) % 16
    v = np.random.default_rng(1).standard_normal((3000, 2, 64)).astype(np.float32)
    p.put(k.astype(np.float32), v, slots)
    p.q.fill_(4.0)
    page, at = p.slot(0, 70)
    p.cache[2][page, 1, at, 11] = 0x7F
    p.check()
