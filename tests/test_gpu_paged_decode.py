"""The serving example: outputs of mixed steps over the MXFP8 cache against the same
layer with float32 attention.  E4M3 elements are off by at most 2^-4 of their value; the
keys' errors enter the scores and the values' the outputs, both averaged over channels
and tokens, then the output projection quantizes its input once more on either side.  The
bound is one such step for each of keys, values and that input: 3 x 2^-4."""

import importlib.util
import os

import pytest

from tests.gpu_util import import_library

pytestmark = pytest.mark.gpu

mxa = import_library()

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dim,kv_heads", [(64, 2), (128, 2), (128, 8)])
def test_steps_agree_with_the_whole_layer(dim, kv_heads):
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, steps, tokens = example.serve(requests=4, dim=dim, kv_heads=kv_heads, chunk=32)
    assert steps > 4 and tokens > 64
    assert worst < 3 * 2.0 ** -4
