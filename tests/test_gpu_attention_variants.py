"""Every form of the paged attention kernels against the 64-bit oracle, with and without windows.

Which form a call takes depends on its sizes (256 CUs; G = heads per kv head, rows = new tokens x G):
up to 16 rows a request, one 16-row tile a wave; up to 32, two; more, 32 x 32 tiles in workgroups of
four waves, of eight where requests x ceil(rows / 256) x kv heads reach the number of CUs.  Requests
of few rows take four waves where requests x kv heads x ceil(keys / 256) is at most 64.  Long calls
are held to the oracle in a sample of their queries: a query at position p of its request is the only
new token of a request of p + 1 tokens."""

import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.gpu_util import dev
from tests.test_gpu_attention import HALF_STEP, Problem, mxa

pytestmark = pytest.mark.gpu


def sample_of(p, want=24):
    """Tokens to look at: the first and last of every request, and others spread over all."""
    edge = {int(t) for a, b in zip(p.cu[:-1], p.cu[1:]) for t in (a, a + 1, b - 2, b - 1) if a <= t < b}
    return sorted(edge | {int(t) for t in np.linspace(0, p.cu[-1] - 1, want)})


def oracle_at(p, tokens, **kw):
    """The oracle's results of single tokens of a problem."""
    q = p.q[torch.tensor(tokens, device=dev())].double().cpu().numpy()
    r = np.searchsorted(p.cu, tokens, side="right") - 1
    pos = p.lens[r] - (p.cu[r + 1] - p.cu[r]) + np.array(tokens) - p.cu[r]
    with np.errstate(invalid="ignore"):
        return oa.attention(q, p.cache, p.table[r], np.arange(len(tokens) + 1), pos + 1, p.window, **kw)


def check_sample(p, got=None, spoiled=None):
    """Outputs and log-sum-exps of a sample of tokens, to the bounds of an output's derivation.  `spoiled` [tokens][heads][dim]
    holds +-1 where a visible value decodes to an infinity of that sign, 2 where infinities of both signs meet."""
    out, lse = p.run() if got is None else got
    assert out.shape == p.q.shape
    at = sample_of(p)
    want, wl, mag, big, seen = oracle_at(p, at)
    out, lse = (x[torch.tensor(at, device=dev())].double().cpu().numpy() for x in (out, lse))
    u = HALF_STEP[p.dtype]
    if spoiled is not None:
        sign = spoiled[at]
        want = np.where(sign == 2, np.nan, np.where(sign != 0, np.inf * np.where(sign == 0, 1, sign), want))
    bad = np.isnan(want) != np.isnan(out)
    assert not bad.any(), f"NaN at other places: {bad.sum()}, first token {at[np.argwhere(bad)[0][0]]}, {np.argwhere(bad)[0]}"
    inf = np.isinf(want)
    assert np.array_equal(out[inf], want[inf]) and not np.isinf(out[~inf]).any()
    fin = np.isfinite(want)
    score = big * (p.dim + 8) * 2.0 ** -24 + 2.0 ** -20
    with np.errstate(invalid="ignore"):
        tol = u * np.abs(want) + mag * (u + seen * 2.0 ** -23 + 2 * score)[..., None] + 1e-30
        over = np.abs(np.where(fin, out - want, 0)) > np.where(fin, tol, 0)
    assert not over.any(), (f"{over.sum()} of {over.size} outputs are off; first token {at[np.argwhere(over)[0][0]]}: "
                            f"{out[over][0]} for {want[over][0]}, bound {tol[over][0]}")
    f = np.isfinite(wl)
    assert np.array_equal(np.isnan(wl), np.isnan(lse)) and np.array_equal(lse[~f & ~np.isnan(wl)], wl[~f & ~np.isnan(wl)])
    assert (np.abs(lse[f] - wl[f]) <= (score + seen * 2.0 ** -23)[f] + 2.0 ** -20 * (1 + np.abs(wl[f]))).all()


# heads, kv heads, requests (new tokens, cached tokens)
FORMS = {
    "one row tile, four waves": (8, 2, [(1, 300), (3, 91), (1, 1600)]),
    "one row tile, eight waves": (16, 4, [(1, 4500), (3, 2000), (1, 700), (4, 33)]),
    "two row tiles": (16, 2, [(4, 2500), (3, 900), (1, 40)]),
    "tiles of four waves": (8, 2, [(70, 2600), (40, 333), (9, 1900)]),
    "tiles of four waves beside few rows": (8, 2, [(1, 3000), (70, 700), (5, 1900), (1, 17)]),
    "tiles of eight waves": (64, 16, [(250, 900), (256, 256), (1, 500), (131, 700), (256, 1999)]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("window", [0, 37, 1500])
def test_forms(form, dim, dtype, window):
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs, heads, hk, dim, 16, dtype, window, seed=dim + window)
    for r, n in enumerate(p.lens):     # pages wholly before a window are gone
        first = max(0, int(n) - reqs[r][0] - window + 1) if window else 0
        p.table[r, :first // 16] = -3
    check_sample(p)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_forms_with_nan_values_and_bad_pages(form, dim):
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs, heads, hk, dim, 16, seed=dim + 1)
    for r, (m, n) in enumerate(reqs):
        page, at = p.slot(r, n - 1 - m // 2)          # a value that the request's later tokens see
        p.cache[2][page, hk - 1, at, r + 3] = 0x7F
        page, at = p.slot(r, n - 1)
        p.cache[3][page, 0, at, dim // 32 - 1] = 0xFF
    p.table[len(reqs) - 1, reqs[-1][1] // 16 // 2] = len(p.cache[0])
    check_sample(p)
