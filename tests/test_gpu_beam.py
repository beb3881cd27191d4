"""Beam selection on the GPU against the 64-bit oracle.

Tokens and parents are whole numbers and must be equal.  The GPU's ln sum exp(x - m) is off by at most:
the argument d = x - m and its product with log2 e, three roundings of 2^-24 |d|, weighted by the
probabilities (mean |d| <= ln vocab, 12 here): 2.2e-6; the exponential, 2^-23; 65 FP32 additions before the sum goes
on in FP64, 2^-24 each: 3.9e-6; 6.2e-6 together.  Candidates of different beams that are nearer than 8e-6 may
come in another order (see `unsure`); those of one beam may not.  A score is rounded to FP32 once more: 2^-24 of itself."""

import numpy as np
import pytest
import torch

from oracle import beam as ob
from tests.gpu_util import dev, import_library

pytestmark = pytest.mark.gpu

mxa = import_library()
NEAR = 8e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def check(x, scores, width=None, finished=None, eos=-1, pad=0, history=None, lens=None):
    """x [requests][beams][vocab] on the GPU; the others numpy or None."""
    up = lambda a, d: None if a is None else torch.tensor(a, dtype=d, device=dev())  # noqa: E731
    got = mxa.mx_beam_select(x, up(scores, torch.float32), width, up(finished, torch.bool), eos, pad, up(history, torch.int32),
                             up(lens, torch.int32))
    r, b = x.shape[:2]
    w = b if width is None else width
    scores = np.asarray(scores, dtype=np.float32).astype(np.float64)
    want = ob.select(x.double().cpu().numpy(), scores, w, finished, eos, pad, history, lens)
    z = want["scores"].reshape(r, w)
    sure = unsure(x, scores, w, finished, z)
    for name in ("parents", "tokens", "finished"):
        g = getattr(got, name).cpu().numpy()
        assert np.array_equal(g[sure], want[name].reshape(r, w)[sure]), name
    s = got.scores.double().cpu().numpy()
    finite = np.isfinite(z)
    assert np.array_equal(finite, np.isfinite(s)) and (s[~finite] == -np.inf).all()
    assert (np.abs(s[finite] - z[finite]) <= NEAR + 2.0 ** -24 * np.abs(z[finite])).all()
    if history is not None:
        c = np.asarray(history).shape[-1]
        assert np.array_equal(got.history.cpu().numpy()[sure], want["history"].reshape(r, w, c)[sure])
        assert np.array_equal(got.lens.cpu().numpy()[sure], want["lens"].reshape(r, w)[sure])
    else:
        assert got.history is None and got.lens is None
    return got, sure


def unsure(x, scores, w, finished, z):
    """Which of the oracle's choices no other beam's candidate comes near (the next one behind the last included)."""
    more = ob.select(x.double().cpu().numpy(), scores, w + 1, finished)
    r = x.shape[0]
    s, p = more["scores"].reshape(r, w + 1), more["parents"].reshape(r, w + 1)
    with np.errstate(invalid="ignore"):
        near = (np.abs(np.diff(s, axis=1)) < NEAR) & (np.diff(p, axis=1) != 0)
    return ~(near | np.concatenate([np.zeros((r, 1), bool), near[:, :-1]], 1))


def logits(shape, dtype, seed, spread=2.5):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev()) * spread).to(DT[dtype])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1023, 1024, 1025, 4095, 4096, 4097, 5003])
def test_vocabularies(vocab, dtype):
    rng = np.random.default_rng(vocab)
    for seed, (r, b, w) in enumerate(((1, 1, 1), (3, 4, 4), (2, 3, 6))):
        _, sure = check(logits((r, b, vocab), dtype, vocab + seed), rng.uniform(-9, 0, (r, b)), w)
        assert sure.mean() > 0.8


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("r,b,w,vocab", [(1, 4, 4, 50001), (2, 64, 64, 777), (1, 1, 64, 131075), (5, 7, 13, 9999), (700, 3, 5, 130),
                                        (64, 8, 16, 3001), (40, 16, 16, 20000)])
def test_sizes(r, b, w, vocab, dtype):
    rng = np.random.default_rng(r)
    _, sure = check(logits((r, b, vocab), dtype, r), rng.uniform(-9, 0, (r, b)), w)
    assert sure.mean() > 0.8


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab", [5, 700, 4097, 20000])
def test_equal_logits_go_by_token(vocab, dtype):
    """All alike, alike but for a few, and a few values many times over; beams apart by their scores."""
    scores = [[0.0, -0.5, -40.0]]
    x = torch.full((1, 3, vocab), 1.5, dtype=DT[dtype], device=dev())
    got, _ = check(x, scores, 8)
    assert got.tokens[0, :min(5, vocab)].tolist() == list(range(min(5, vocab)))
    x[0, 1, vocab // 2:] = 1.75
    check(x, scores, 16)
    g = torch.Generator(device=dev()).manual_seed(vocab)
    x = torch.randint(-2, 3, (1, 3, vocab), generator=g, device=dev()).to(DT[dtype])
    check(x, scores, 33)
    # both zeros are one value
    check(torch.where(x < 0, -0.0, 0.0).to(DT[dtype]), scores, 9)
    # falling and rising: the best come last
    x = (torch.arange(vocab, device=dev()) // 40).to(DT[dtype]).expand(1, 3, vocab) / 64
    check(x, scores, 20)
    check(x.flip(-1).contiguous(), scores, 20)


def test_equal_scores_go_to_the_lower_beam():
    x = logits((2, 1, 900), "f32", 4).expand(2, 5, 900)
    s = torch.full((2, 5), -3.0, device=dev())
    got = mxa.mx_beam_select(x, s, 10)
    assert got.parents.tolist() == [[0, 1, 2, 3, 4] * 2, [5, 6, 7, 8, 9] * 2]
    # 4096 candidates: of 64 beams alike (the 64 best logits' score each 64 times), and all of one score
    x = logits((1, 1, 900), "f32", 5).expand(2, 64, 900)
    s = torch.full((2, 64), -3.0, device=dev())
    got = mxa.mx_beam_select(x, s, 64)
    assert got.parents.tolist() == [list(range(64)), list(range(64, 128))]
    assert (got.tokens == x[0, 0].argmax()).all()
    got = mxa.mx_beam_select(x * 0.0, s, 64)
    assert (got.parents == torch.tensor([[0], [64]], device=dev())).all()
    assert got.tokens.tolist() == [list(range(64))] * 2
    # 15 beams, 20 to be chosen: 300 candidates, fewer than 20 of them real
    x = torch.full((1, 15, 40), -float("inf"), device=dev())
    x[0, ::2, 7] = 1.0
    got = mxa.mx_beam_select(x, -torch.arange(15.0, device=dev())[None], 20)
    assert got.parents[0].tolist() == list(range(0, 15, 2)) + [0] * 12 and got.tokens[0].tolist() == [7] * 8 + [0] * 12
    assert got.scores[0].tolist() == [-float(i) for i in range(0, 15, 2)] + [-float("inf")] * 12


@pytest.mark.parametrize("beams", [4, 40])
def test_a_score_of_minus_zero_equals_zero(beams):
    """A finished beam's -0 comes before the zeros of higher beams, few candidates or many."""
    x = torch.full((1, beams, 9), -float("inf"), device=dev())
    x[:, :, 5] = 0.0
    scores = torch.zeros(1, beams, device=dev())
    scores[0, 0] = -0.0
    finished = torch.zeros(1, beams, dtype=torch.bool, device=dev())
    finished[0, 0] = True
    got = mxa.mx_beam_select(x, scores, 4, finished, pad=2)
    assert got.parents.tolist() == [[0, 1, 2, 3]] and got.tokens.tolist() == [[2, 5, 5, 5]]
    assert got.scores.tolist() == [[0.0] * 4]


@pytest.mark.parametrize("dtype", list(DT))
def test_masked_and_bad_rows(dtype):
    """Banned tokens, rows with nothing left, NaN and infinities; scores that are none."""
    x = logits((4, 4, 3000), dtype, 1)
    lowest = torch.finfo(DT[dtype]).min
    x[0, 0] = -np.inf                          # nothing left
    x[0, 1, 5:] = -np.inf                      # five left
    x[0, 2, ::2] = lowest                      # masked with the lowest value: of no weight, but there
    x[1, 0, 2999] = np.nan
    x[1, 1, 0] = np.inf
    x[1, 2, 7] = -np.nan
    x[1, 3] = -np.inf
    x[1, 3, 2998] = 3.0                        # one left: probability 1
    x[2] = -np.inf                             # a request without candidates
    x[3, 0] = lowest                           # all alike, however low
    scores = np.array([[-1.0, -1.5, -2.0, -np.inf], [0.0, -1.0, -2.0, -3.0], [-1.0, -2.0, -3.0, -4.0],
                       [-1.0, np.nan, np.inf, -np.inf]])
    history, lens = np.arange(4 * 4 * 6).reshape(4, 4, 6), np.array([[0, 3, 6, 9], [-1, 2, 5, 6], [1] * 4, [5] * 4])
    got, _ = check(x, scores, 12, history=history, lens=lens)
    assert got.scores[1].tolist()[:2] == [-3.0, -np.inf] and got.tokens[1, 0] == 2998
    assert got.tokens[3].tolist() == list(range(12))


def test_finished_beams():
    x = logits((3, 4, 500), "bf16", 2)
    x[0, 0] = np.nan                           # a finished beam's logits are not looked at
    finished = np.array([[1, 0, 0, 1], [1, 1, 1, 1], [0, 0, 0, 0]], dtype=bool)
    scores = np.array([[-1.0, -2.0, -2.5, -90.0], [-4.0, -1.0, -np.inf, -2.0], [-1.0, -1.1, -1.2, -1.3]])
    history, lens = np.arange(3 * 4 * 5).reshape(3, 4, 5), np.array([[1, 2, 3, 4], [5, 4, 3, 2], [0, 5, 4, 1]])
    top = int(x[2, 0].float().argmax())
    got, _ = check(x, scores, 4, finished, eos=top, pad=top, history=history, lens=lens)
    assert got.finished[1].tolist() == [True, True, True, False]         # the fourth is empty
    assert got.tokens[1].tolist() == [top] * 4
    check(x, scores, 7, finished, eos=top, pad=3)


@pytest.mark.parametrize("cols", [0, 1, 63, 64, 65, 1000, 70001])
def test_histories(cols):
    rng = np.random.default_rng(cols)
    r, b, w = 2, 3, 5
    check(logits((r, b, 300), "f32", 3), rng.uniform(-3, 0, (r, b)), w, history=rng.integers(0, 300, (r, b, cols)),
          lens=rng.integers(0, cols + 1, (r, b)))


def test_large_values_and_narrow_sums():
    """Logits of +-1e30 and of one great value beside thousands of small ones."""
    x = logits((2, 3, 2500), "f32", 6) * 1e30
    check(x, np.zeros((2, 3)) - [[0, 1, 2]], 4)
    # subnormal logits: all equally likely to 64 bits, but in an order
    x = torch.randint(-900, 900, (2, 3, 2500), device=dev()) * 2.0 ** -149
    assert x.abs().max() > 0
    check(x, np.zeros((2, 3)) - [[0, 1, 2]], 4)
    x = logits((2, 3, 2500), "f32", 7) * 1e-3
    x[:, :, 1234] = 40.0
    check(x, np.zeros((2, 3)) - [[0, 1, 2]], 9)


@pytest.mark.parametrize("dtype", list(DT))
def test_strided_logits(dtype):
    """Part of a wider projection, rows at any alignment of their type, requests and beams in either order."""
    base = logits((4 * 3 * 1207 + 5,), dtype, 8)
    for start in (0, 1, 3):
        x = base[start:start + 4 * 3 * 1207].view(4, 3, 1207)
        for y in (x[:, :, 2:1201], x.transpose(0, 1)[:, :, :1100], x[1:2, :, :5], x[:, 1:2, 7:]):
            check(y, np.random.default_rng(start).uniform(-5, 0, y.shape[:2]), 4)


def test_logits_past_32_bits():
    """2.5e9 logits: the last request's, and histories of 1.2e9 tokens."""
    r, b, v, c = 300, 64, 131072, 65536
    x, s = torch.zeros((r, b, v), dtype=torch.bfloat16, device=dev()), torch.zeros((r, b), device=dev())
    x[-1] = logits((b, v), "bf16", 1)
    s[-1] = -torch.rand(b, device=dev())
    history = torch.zeros((r, b, c), dtype=torch.int32, device=dev())
    history[-1] = torch.arange(b * c, device=dev()).view(b, c) % 50000
    lens = torch.full((r, b), 7, dtype=torch.int32, device=dev())
    got = mxa.mx_beam_select(x, s, 16, history=history, lens=lens)
    want = mxa.mx_beam_select(x[-1:], s[-1:], 16, history=history[-1:], lens=lens[-1:])
    for name in ("tokens", "finished", "history", "lens"):
        assert torch.equal(getattr(got, name)[-1:], getattr(want, name)), name
    # a call of other sizes sums in other segments: each is off by at most NEAR and its rounding (see above)
    assert ((got.scores[-1:] - want.scores).abs() <= 2 * NEAR + 2.0 ** -23 * want.scores.abs()).all()
    assert torch.equal(got.parents[-1:], want.parents + (r - 1) * b)
    assert got.tokens[0].tolist() == list(range(16)) and got.parents[0].tolist() == [0] * 16


def test_a_history_of_the_most_columns():
    """2^31 - 1 columns: the count of the last step passes 31 bits."""
    cols = (1 << 31) - 1
    history = torch.empty(1, 1, cols, dtype=torch.int32, device=dev())
    at = [0, 63, 64, 65, 1 << 30, cols - 65, cols - 2, cols - 1]
    history.fill_(-3)
    history[0, 0, at] = torch.arange(8, dtype=torch.int32, device=dev())
    x = torch.tensor([[[0.0, 1.0]]], device=dev())
    got = mxa.mx_beam_select(x, torch.zeros(1, 1, device=dev()), history=history,
                             lens=torch.tensor([[cols - 1]], dtype=torch.int32, device=dev()))
    assert got.lens.tolist() == [[cols]] and got.history[0, 0, at].tolist() == [0, 1, 2, 3, 4, 5, 6, 1]
    history[0, 0, cols - 1] = 1
    assert torch.equal(got.history, history)


def test_the_most_rows():
    """2^20 requests of 64 beams, a wave for each: 2^32 threads, more than a launch can have."""
    requests, beams, width = 1 << 20, 64, 3
    g = torch.Generator(device=dev()).manual_seed(8)
    # sixteenths, so that beams of a request tie
    scores = torch.randint(-2000, 0, (requests, beams), generator=g, device=dev()).float() / 16
    x = torch.randn(requests, beams, 1, generator=g, device=dev()).bfloat16()
    got = mxa.mx_beam_select(x, scores, width, pad=7)
    # of one token the log-probability is 0
    want, parents = scores.sort(dim=1, descending=True, stable=True)
    assert torch.equal(got.scores, want[:, :width])
    first = torch.arange(requests, device=dev())[:, None] * beams
    assert torch.equal(got.parents.long(), parents[:, :width] + first) and not got.tokens.any() and not got.finished.any()


def test_scores_of_one_beam_add_up():
    """With the vocabulary as wide as the beam every probability comes back: they sum to one."""
    x = logits((1, 1, 60), "f32", 9)
    got = mxa.mx_beam_select(x, torch.zeros((1, 1), device=dev()), 60)
    assert abs(got.scores.double().exp().sum().item() - 1.0) < 60 * 2.0 ** -22
    assert sorted(got.tokens[0].tolist()) == list(range(60))


def test_empty():
    x = logits((0, 3, 50), "f32", 1)
    got = mxa.mx_beam_select(x, torch.zeros((0, 3), device=dev()), 2)
    assert got.tokens.shape == (0, 2)


def test_replayed_graph_and_streams():
    x, scores = logits((3, 4, 9000), "bf16", 1), torch.zeros((3, 4), device=dev())
    call = lambda: mxa.mx_beam_select(x, scores, 6, eos=3)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(5):
        x.copy_(logits(x.shape, "bf16", seed + 20))
        scores.copy_(-torch.rand((3, 4), device=dev()) * 5)
        graph.replay()
        want = call()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = call()
        torch.cuda.current_stream().wait_stream(side)
        for a, b, c in zip(out[:4], want[:4], other[:4]):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    x, s = logits((2, 3, 50), "f32", 1), torch.zeros((2, 3), device=dev())
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device=dev())  # noqa: E731
    call = lambda **kw: mxa.mx_beam_select(**{**dict(logits=x, scores=s), **kw})  # noqa: E731
    for kw in ({"logits": x[0]}, {"logits": x.double()}, {"logits": x.transpose(1, 2), "scores": torch.zeros((2, 50), device=dev())},
               {"scores": s.double()}, {"scores": s[:1]}, {"scores": s.t()}, {"width": 0}, {"width": 65}, {"width": -1},
               {"finished": s}, {"finished": s[0].bool()}, {"eos": 2 ** 31}, {"pad": -2 ** 31 - 1}, {"history": i(2, 3, 4)},
               {"lens": i(2, 3)}, {"history": i(2, 3, 4), "lens": i(2, 4)}, {"history": i(2, 3), "lens": i(2, 3)},
               {"history": i(2, 3, 4).long(), "lens": i(2, 3)}, {"logits": x[:, :, :0]}, {"logits": x.cpu(), "scores": s.cpu()},
               {"logits": logits((1, 65, 5), "f32", 0), "scores": torch.zeros((1, 65), device=dev()), "width": 4}):
        with pytest.raises(ValueError):
            call(**kw)
