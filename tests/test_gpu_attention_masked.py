"""What masked keys and vanishing weights must not change: windows without end, values that decode to
infinities, NaN values far below the largest score."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_attention import Problem, mxa
from tests.test_gpu_attention_variants import FORMS, check_sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [(1 << 63) - 1, 1 << 62, 1 << 31, 5000])
@pytest.mark.parametrize("form", FORMS)
def test_windows_past_every_length_are_none(form, window):
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs, heads, hk, 64, 16, seed=5)
    out, lse = p.run()
    got, got_lse = p.run(window=window)
    assert torch.equal(out, got) and torch.equal(lse, got_lse)


# E4M3 code and scale code of an element that the type of q cannot hold: 256 x 2^8 for F16, 448 x 2^120 for BF16
INFINITE = {"f16": (0x78, 135), "bf16": (0x7E, 247)}


def spoil(p, reqs):
    """Puts such elements into values of every request: its newest token, ones that a half and a third of its queries
    see, and an older one.  Returns for every output the sign of the infinities that it sees, 2 where both meet."""
    code, scale = INFINITE[p.dtype]
    sees = np.zeros((2, int(p.cu[-1]), p.heads, p.dim), dtype=bool)
    group = p.heads // p.hk
    for r, (m, n) in enumerate(reqs):
        cleared = set()
        pos = n - m + np.arange(m)                     # of the queries
        for back, ch, minus in ((0, 5, 0), (m // 2, 6, 1), (m // 2, 7, 0), (m // 3, 7, 1), (min(n - 1, m + 20), 9, 1)):
            key, head = n - 1 - back, r % p.hk
            if minus and ch == 7 and m // 3 == m // 2:
                continue                               # the place is taken by the other sign
            page, at = p.slot(r, key)
            if key not in cleared:
                p.cache[2][page, head, at, :32] = 0
                p.cache[3][page, head, at, 0] = scale
                cleared.add(key)
            p.cache[2][page, head, at, ch] = code | minus << 7
            q = pos >= key
            if p.window:
                q &= pos < key + p.window
            sees[minus, p.cu[r] + np.flatnonzero(q), head * group:(head + 1) * group, ch] = True
    return np.where(sees[0] & sees[1], 2, sees[0].astype(int) - sees[1])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("window", [0, 25])
def test_infinite_values_reach_only_rows_that_see_them(form, dim, dtype, window):
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs, heads, hk, dim, 16, dtype, window, seed=dim + 3)
    check_sample(p, spoiled=spoil(p, reqs))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("form", FORMS)
def test_nan_values_with_f16_queries(form, dim):
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs, heads, hk, dim, 16, "f16", seed=dim + 4)
    for r, (m, n) in enumerate(reqs):
        page, at = p.slot(r, n - 1 - m // 2)
        p.cache[2][page, hk - 1, at, r + 3] = 0xFF
        p.cache[3][page, 0, at, dim // 32 - 1] = 0xFF
    check_sample(p)


@pytest.mark.parametrize("tokens", [6, 40])
def test_appended_values_that_round_up_to_infinity(tokens):
    """The newest token's 65504 is stored as 65536, which F16 does not hold: only its own query sees it."""
    g = torch.Generator(device=dev()).manual_seed(tokens)
    cache = mxa.new_kv_cache(4, 2, 16, 64)
    k, v = (torch.randn((tokens, 2, 64), device=dev(), generator=g).half() for _ in range(2))
    q = torch.randn((tokens, 8, 64), device=dev(), generator=g).half()
    v[-1, 1, 3] = 65504.0
    mxa.mx_kv_append(k, v, cache, torch.arange(tokens, device=dev()))
    table = torch.arange(4, dtype=torch.int32, device=dev())[None]
    cu, lens = (torch.tensor(t, dtype=torch.int32, device=dev()) for t in ([0, tokens], [tokens]))
    out = mxa.mx_paged_attention(q, cache, table, cu, lens, max_q=tokens, max_kv=tokens)
    assert out[:-1].isfinite().all()
    assert (out[-1, 4:, 3] == float("inf")).all()
    out[-1, 4:, 3] = 0
    assert out.isfinite().all()


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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", ["one row tile, four waves", "one row tile, eight waves", "two row tiles", "tiles of four waves"])
def test_large_values_under_vanishing_weights(form, dtype):
    """Values near the type's largest whose weight is 2^-369 of the others': nothing of them is in the sum."""
    heads, hk, reqs = FORMS[form]
    p = Problem(reqs, heads, hk, 64, dtype=dtype, seed=12)
    for r, (m, n) in enumerate(reqs):
        low = np.arange(5, n - m, 9)
        k = np.full((n, hk, 64), 4.0, np.float32)
        k[low] = -4.0
        v = np.random.default_rng(r).standard_normal((n, hk, 64)).astype(np.float32)
        p.put(k, v, p.table[r, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16)
        for key in low:
            page, at = p.slot(r, int(key))
            p.cache[2][page, :, at, ::2] = 0x7E          # 448 x 2^119, 448 x 2^7
            p.cache[3][page, :, at] = 246 if dtype == "bf16" else 134
    p.q.fill_(4.0)
    check_sample(p)
