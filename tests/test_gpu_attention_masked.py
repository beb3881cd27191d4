"""What masked keys and vanishing weights must not change: windows without end."""

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
