"""Softmax weights enter the product with the values in more bits than the outputs have: an output is off
by its own rounding and by FP32 arithmetic, no more.

Bound: half a step u of the output, and of sum_j p_j |v_j| the weights' u^2 (two terms of the type
of q, the second of the first one's rounding error), FP32 sums over n keys (n 2^-23) and twice the error of
a score.  F16 weights are 2^7 or more at the largest key and lose what is below 2^-25: 2^-32 of sum_j |v_j|."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_attention import HALF_STEP, Problem
from tests.test_gpu_attention_variants import FORMS, oracle_at, sample_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("form", [f for f in FORMS if "tiles of" not in f])
def test_outputs_are_off_by_their_own_rounding(form, dim, dtype):
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs + [(1, 2), (2, 5)], heads, hk, dim, 16, dtype, seed=dim + 9)
    at = sample_of(p)
    out = p.run()[0][torch.tensor(at, device=dev())].double().cpu().numpy()
    want, _, mag, big, seen = oracle_at(p, at)
    u = HALF_STEP[dtype]
    score = big * (dim + 8) * 2.0 ** -24 + 2.0 ** -20
    tol = u * np.abs(want) + mag * (u * u + seen * 2.0 ** -23 + 2 * score)[..., None] + 1e-30
    if dtype == "f16":                               # no value here is above 2^6
        tol += seen[..., None] * 2.0 ** (6 - 32)
    over = np.abs(out - want) > tol
    assert not over.any(), f"{over.sum()} of {over.size} outputs are off by up to {(np.abs(out - want) / tol)[over].max()} bounds"
