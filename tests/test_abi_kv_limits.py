"""Further refusals of the cache entry points, checked without a GPU."""

import pytest
import torch

from tests.test_abi_kv import FAKE, LAUNCH, NULL, append, attention, cache, mxa  # noqa: F401

if torch.cuda.is_available():
    pytest.skip("argument-validation tests use fake device addresses; CPU only", allow_module_level=True)


def test_attention_needs_the_columns_that_it_is_told_of():
    """A kernel may read any of the table's columns before it knows a request's length, so a table of four columns has
    to be there even where no request may have a token; a table without columns is never read."""
    assert attention(table=None, max_kv=0) == NULL
    assert attention(table=None, max_kv=0, cols=0) == LAUNCH      # accepted: no device here to launch on
    assert attention(table=None, cols=0) == LAUNCH


def test_flags_without_a_truth_value():
    """Whose __bool__ raises: that error, not a result with an error set."""
    x, pos, t = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 32, 2)
    c = mxa.KVCache(*(torch.zeros((2, 2, 16, n), dtype=torch.uint8) for n in (64, 2, 64, 2)))
    both = torch.zeros(2, dtype=torch.bool)
    with pytest.raises(RuntimeError, match="ambiguous"):
        mxa.mx_rope(x, pos, t, inverse=both)
    with pytest.raises(RuntimeError, match="ambiguous"):
        mxa.mx_paged_attention(x.bfloat16(), c, pos.view(2, 2), torch.zeros(3, dtype=torch.int32), pos[:2], lse=both, max_q=1,
                               max_kv=1)


@pytest.mark.parametrize("kw", [dict(tokens=1 << 26, heads=1, q=FAKE + 2), dict(tokens=1 << 31),
                                dict(tokens=1 << 26, cache=cache(kv_heads=64))])
def test_appends_of_any_length(kw):
    """Lengths beyond one launch's thread numbers are cut into several; there is no device here to launch on."""
    assert append(**kw) == LAUNCH


def test_append_refuses_a_table_without_rows():
    """It has no address, which the library takes for a call without rotation: the keys would be stored unturned."""
    x, pos = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    c = mxa.KVCache(*(torch.zeros((2, 2, 16, n), dtype=torch.uint8) for n in (64, 2, 64, 2)))
    with pytest.raises(ValueError, match="rows"):
        mxa.mx_kv_append(x, x, c, pos.long(), pos, torch.zeros(0, 32, 2))
