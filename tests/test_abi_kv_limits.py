"""Further refusals of the cache entry points, checked without a GPU."""

import pytest
import torch

from tests.test_abi_kv import LAUNCH, NULL, attention, mxa  # noqa: F401

if torch.cuda.is_available():
    pytest.skip("argument-validation tests use fake device addresses; CPU only", allow_module_level=True)


def test_attention_needs_the_columns_that_it_is_told_of():
    """A kernel may read any of the table's columns before it knows a request's length, so a table of four columns has
    to be there even where no request may have a token; a table without columns is never read."""
    assert attention(table=None, max_kv=0) == NULL
    assert attention(table=None, max_kv=0, cols=0) == LAUNCH      # accepted: no device here to launch on
    assert attention(table=None, cols=0) == LAUNCH
