"""Beam selection, forks, appends, attention, compaction and freeing together, as the example uses them.

The scores of a search over shared pages have to be the log-probabilities of the sequences found, fed alone.  Attention
over the same keys may add them in another order where a call has other sizes (the prompts: few sequences against many),
and its outputs are rounded to BF16 (2^-9 of their value) before the next layer: an output that falls to the other
side of a rounding moves a logit by 2^-8 of one of 256 channels of one of the layers, some 4 x 2^-8 / 16 = 1e-3 of the
logits' spread of about 4.  A sequence of up to 40 tokens that read wrong keys is off by more than 0.1 a token."""

import importlib.util
import os

import pytest
import torch

from tests.gpu_util import import_library

pytestmark = pytest.mark.gpu

mxa = import_library()

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("beams,steps,page,layers,kv_heads,dim,lengths", [
    (4, 40, 16, 2, 2, 64, (5, 33, 64)), (1, 20, 16, 1, 4, 64, (1, 17)), (8, 24, 32, 3, 1, 64, (31,)),
    (3, 36, 64, 2, 2, 128, (1, 2, 70, 128, 40))])
def test_scores_are_those_of_the_sequences(beams, steps, page, layers, kv_heads, dim, lengths):
    e = example()
    model = e.Model(layers=layers, kv_heads=kv_heads, dim=dim, seed=beams)
    g = torch.Generator().manual_seed(beams)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in lengths]
    step, most = e.search(model, prompts, beams, steps, page)
    alone = e.replay(model, prompts, step.history, step.lens, page)
    assert step.lens.eq(steps).all()
    assert (step.scores[:, :-1] >= step.scores[:, 1:]).all()
    assert (alone - step.scores).abs().max() < 0.05 * steps / 10
    assert beams == 1 or most < sum(-(-(n + steps) // page) for n in lengths) * beams


def test_finished_beams_stay():
    e = example()
    model = e.Model(seed=3)
    prompts = [[1, 2, 3], [7] * 20]
    step, _ = e.search(model, prompts, 4, 30, eos=int(e.search(model, prompts, 4, 30)[0].history[0, 0, 4]))
    assert step.finished.any()
    alone = e.replay(model, prompts, step.history, step.lens)
    assert (alone - step.scores).abs().max() < 0.15
