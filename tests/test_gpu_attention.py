"""Attention over the paged MXFP8 cache on the GPU against the 64-bit oracle.

Bound of an output: one rounding to its type (half a step: u = 2^-8 for BF16, 2^-11
for F16), and the error of the weights times sum_j p_j |v_j|: one rounding u to the
same type, FP32 sums over n keys (n 2^-23), and twice (numerator and denominator) the
error of a score, dim + 8 roundings of 2^-24 of the largest sum |q k| and the
exponential's 2^-20.  The log-sum-exp has the score's error, the sum's, and its own rounding."""

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import mx as omx
from tests.gpu_util import dev, import_library

pytestmark = pytest.mark.gpu

mxa = import_library()

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


class Problem:
    """Requests (new tokens, cached tokens) over shuffled pages; bytes that belong to nobody are E4M3 and
    E8M0 NaNs, and table entries that nobody needs are out of range."""

    def __init__(self, reqs, heads=8, hk=2, dim=128, page=16, dtype="bf16", window=0, seed=0, spare=2, shift=0):
        g = np.random.default_rng(seed)
        self.dtype, self.window, self.dim, self.page, self.hk, self.heads = dtype, window, dim, page, hk, heads
        need = [-(-n // page) for _, n in reqs]
        pages = sum(need) + spare
        order = g.permutation(pages).astype(np.int32)
        self.table = np.full((len(reqs), max(need + [1])), -7, np.int32)
        self.cache = [np.full((pages, hk, page, w), 0xFF, np.uint8) for w in (dim, dim // 32, dim, dim // 32)]
        at = 0
        for r, (m, n) in enumerate(reqs):
            self.table[r, :need[r]] = order[at:at + need[r]]
            at += need[r]
            ch = np.exp2(g.uniform(-1.5, 1.5, dim))
            k = (g.standard_normal((n, hk, dim)) * ch).astype(np.float32)
            v = (g.standard_normal((n, hk, dim)) * np.exp2(g.uniform(-3, 3, (n, 1, 1)))).astype(np.float32)
            slots = self.table[r, np.arange(n) // page] * page + np.arange(n) % page
            self.put(k, v, slots)
        self.cu = np.cumsum([0] + [m for m, _ in reqs]).astype(np.int32)
        self.lens = np.array([n for _, n in reqs], np.int32)
        self.max_q, self.max_kv = max([m for m, _ in reqs]), max([n for _, n in reqs])
        q = torch.from_numpy(g.standard_normal((self.cu[-1], heads + shift, dim)).astype(np.float32)).to(DT[dtype])
        self.q = q.to(dev())[:, shift:]

    def put(self, k, v, slots):
        for n, x in ((0, k), (2, v)):
            if len(x):
                q, s = omx.quantize_rowwise(x.reshape(-1, self.dim), "e4m3", "ceil")
                self.cache[n][slots // self.page, :, slots % self.page] = q.reshape(len(slots), self.hk, -1)
                self.cache[n + 1][slots // self.page, :, slots % self.page] = s.reshape(len(slots), self.hk, -1)

    def slot(self, r, key):
        return int(self.table[r, key // self.page]), key % self.page

    def gpu_args(self):
        up = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
        return (mxa.KVCache(*map(up, self.cache)), up(self.table), up(self.cu), up(self.lens))

    def run(self, **kw):
        kw = {"window": self.window, "lse": True, "max_q": self.max_q, "max_kv": self.max_kv, **kw}
        return mxa.mx_paged_attention(self.q, *self.gpu_args(), **kw)

    def check(self, got=None, scale=None):
        out, lse = self.run(scale=scale) if got is None else got
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            want, wl, mag, big, seen = oa.attention(self.q.double().cpu().numpy(), self.cache, self.table, self.cu, self.lens,
                                                    self.window, scale)
        u = HALF_STEP[self.dtype]
        score = big * (self.dim + 8) * 2.0 ** -24 + 2.0 ** -20
        tol = u * np.abs(want) + mag * (u + seen * 2.0 ** -23 + 2 * score)[..., None] + 1e-30
        bad = np.isnan(want) != np.isnan(out)
        assert not bad.any(), f"NaN at other places, first {np.argwhere(bad)[0]}"
        over = np.abs(out - want) > tol
        assert not over.any(), (f"{over.sum()} of {over.size} outputs are off; first {np.argwhere(over)[0]}: "
                                f"{out[over][0]} for {want[over][0]}, bound {tol[over][0]}")
        fin = np.isfinite(wl)
        assert np.array_equal(np.isnan(wl), np.isnan(lse)) and np.array_equal(lse[~fin & ~np.isnan(wl)], wl[~fin & ~np.isnan(wl)])
        tol = score + seen * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(wl))
        assert (np.abs(lse[fin] - wl[fin]) <= tol[fin]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,hk", [(4, 4), (7, 1), (16, 2)])
def test_decode(dim, heads, hk, dtype):
    Problem([(1, n) for n in (1, 2, 16, 31, 32, 33, 100, 257)], heads, hk, dim, 16, dtype, seed=dim).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_chunks(dim, dtype):
    Problem([(45, 45), (70, 131), (3, 500), (1, 1), (129, 129)], 8, 2, dim, 32, dtype, seed=dim).check()


@pytest.mark.parametrize("page", [16, 48, 64, 128])
@pytest.mark.parametrize("group", [1, 3, 7, 8])
def test_pages_and_groups(page, group):
    Problem([(5, 300), (1, 77), (20, 20), (2, 129)], 2 * group, 2, 64, page, seed=page + group).check()


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 1000])
@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_windows(window, q_len):
    """Pages wholly before a window may have gone: their table entries are taken out."""
    p = Problem([(q_len, 700), (min(q_len, 2), 5), (1, 90)], 8, 2, 128, 16, window=window, seed=window)
    for r, n in enumerate(p.lens):
        m = p.cu[r + 1] - p.cu[r]
        p.table[r, :max(0, n - m - window + 1) // 16] = -3
    p.check()


@pytest.mark.parametrize("q_len", [1, 2, 8, 9, 16, 17])
def test_row_tiles(q_len):
    """Around 16, 32 and 64 rows a request (8 heads to a kv head)."""
    Problem([(q_len, 200), (max(1, q_len - 1), 90)], 16, 2, 128, seed=q_len).check()


@pytest.mark.parametrize("q_len,kv", [(1, 9000), (1, 2049), (16, 5000), (33, 4000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_contexts(q_len, kv, dtype):
    Problem([(q_len, kv), (1, kv // 3), (1, 1)], 4, 1, 64, 64, dtype, seed=kv).check()


def test_scale():
    p = Problem([(4, 60), (1, 33)], seed=4)
    p.check(scale=0.02)
    p.check(scale=1.0)


def test_rows_that_see_nothing():
    """A request without cached tokens, one with fewer than new tokens, one without new tokens."""
    p = Problem([(2, 0), (5, 3), (0, 40), (1, 17)], seed=1)
    p.check()
    out, lse = p.run()
    assert (out[:4] == 0).all() and (lse[:4] == -float("inf")).all()


def test_growing_scores():
    """Scores that rise along the keys move the reference exponent many times."""
    p = Problem([(1, 2000), (30, 1500)], 4, 2, 64, seed=9)
    k = np.linspace(-1, 1, 2000)[:, None, None] * np.ones((2000, 2, 64)) * 4
    for r, n in enumerate(p.lens):
        slots = p.table[r, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
        v = np.random.default_rng(r).standard_normal((n, 2, 64)).astype(np.float32)
        p.put(k[:n].astype(np.float32), v, slots)
    p.q.copy_(p.q.abs() * 2)
    p.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tiny_and_zero_blocks(dtype):
    p = Problem([(1, 50), (20, 40)], 4, 2, 128, dtype=dtype, seed=3)
    p.cache[2][:, :, 3] = 0
    p.cache[3][:, :, 3] = 0            # code 0 in all of a token's values
    p.cache[0][:, :, 5] = 0
    p.cache[1][:, :, 5] = 0
    p.cache[3][:, :, 7] = 0            # values of 2^-127 and below
    p.check()


@pytest.mark.parametrize("q_len", [1, 6, 40])
def test_nan_values_reach_only_rows_that_see_them(q_len):
    p = Problem([(q_len, 100), (q_len, 64)], 8, 2, 96, seed=q_len)
    page, at = p.slot(0, 99)           # the newest token: only the last query sees it
    p.cache[2][page, 1, at, 40] = 0x7F
    page, at = p.slot(1, 64 - (q_len + 1) // 2)
    p.cache[3][page, 0, at, 2] = 0xFF
    p.cache[2][page, 0, at, 64:] = 0x7F
    p.check()


def test_nan_keys_reach_only_rows_that_see_them():
    p = Problem([(40, 100)], 8, 2, 64, seed=5)
    page, at = p.slot(0, 80)
    p.cache[0][page, 1, at, 3] = 0xFF
    p.check()


@pytest.mark.parametrize("q_len", [1, 40])
def test_bad_pages_give_nan(q_len):
    p = Problem([(q_len, 100), (q_len, 100), (q_len, 64), (q_len, 50)], 8, 2, 64, seed=5)
    p.table[0, 5] = -1
    p.table[1, 6] = len(p.cache[0])
    p.check()
    p.table = p.table[:, :5].copy()    # a table too narrow for the first two
    p.check()


@pytest.mark.parametrize("kv", [40, 3000])
def test_requests_beyond_the_announced_sizes_give_nan(kv):
    p = Problem([(1, kv), (3, kv), (1, kv + 1), (2, 20)], 4, 2, 64, seed=6)
    out, lse = p.run(max_q=2, max_kv=kv)
    assert out[1:5].isnan().all() and lse[1:5].isnan().all()
    keep = [0, 5, 6]
    want, wl = p.run()
    assert out[keep].isfinite().all()
    assert torch.allclose(out[keep].float(), want[keep].float(), rtol=2 ** -6, atol=1e-2)
    assert torch.allclose(lse[keep], wl[keep], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("kv", [40, 5000])
def test_tokens_outside_all_requests_are_left(kv):
    p = Problem([(2, 30), (1, kv), (3, 50)], 4, 2, 64, seed=6)
    cache, table, cu, lens = p.gpu_args()
    out = torch.full_like(p.q, 7.0)
    mxa.mx_paged_attention(p.q, cache, table[1:2], cu[1:3].contiguous(), lens[1:2].contiguous(), max_q=2, max_kv=kv, out=out)
    assert (out[:2] == 7).all() and (out[3:] == 7).all() and not (out[2] == 7).all()


def test_sliced_queries_defaults_and_streams():
    p = Problem([(5, 90), (1, 300)], 8, 2, 128, seed=8, shift=3)
    assert not p.q.is_contiguous()
    p.check()
    want = p.run()
    args = p.gpu_args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mxa.mx_paged_attention(p.q, *args, lse=True)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(mxa.mx_paged_attention(p.q, *args), want[0])


@pytest.mark.parametrize("kv", [90, 6000])
def test_graph_replays(kv):
    """Captured append and attention, replayed with eager work between, repeat the eager bits."""
    p = Problem([(1, kv), (1, 40)], 8, 2, 128, seed=8)
    cache, table, cu, lens = p.gpu_args()
    rope = mxa.mx_rope_table(8192, 128)
    k = torch.randn((2, 2, 128), device=dev()).bfloat16()
    slots = torch.tensor([int(p.table[r, (n - 1) // 16]) * 16 + (int(n) - 1) % 16 for r, n in enumerate(p.lens)], device=dev())
    pos = lens - 1

    def step():
        q = mxa.mx_kv_append(k, k, cache, slots, pos, rope, q=p.q)
        return mxa.mx_paged_attention(q, cache, table, cu, lens, lse=True, max_q=1, max_kv=kv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        k.copy_(torch.randn((2, 2, 128), device=dev()))
        p.q.copy_(torch.randn(p.q.shape, device=dev()))
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got]
        want = step()
        assert torch.equal(mine[0], want[0]) and torch.equal(mine[1], want[1]), f"replay {i}"


def test_same_bits_again_and_offsets_past_32_bits():
    """The same tokens in the first and in the last pages of a cache of over 2^32 bytes."""
    pages = (1 << 32) // (2 * 64 * 128) + 70
    cache = mxa.KVCache(*(torch.empty((pages, 2, 64, n), dtype=torch.uint8, device=dev()) for n in (128, 4, 128, 4)))
    table = mxa.mx_rope_table(8192, 128)
    n = 4000
    g = torch.Generator(device=dev()).manual_seed(1)
    k, v = (torch.randn((n, 2, 128), device=dev(), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((1, 8, 128), device=dev(), generator=g).bfloat16()
    pos = torch.arange(n, dtype=torch.int32, device=dev())
    got = []
    for first in (0, pages - 63):
        mxa.mx_kv_append(k, v, cache, first * 64 + torch.arange(n, device=dev()), pos, table)
        ids = first + torch.arange(63, dtype=torch.int32, device=dev())[None]
        for x, m in ((q, 1), (q, 1), (q.expand(40, 8, 128).contiguous(), 40)):
            cu = torch.tensor([0, m], dtype=torch.int32, device=dev())
            got.append(mxa.mx_paged_attention(x, cache, ids, cu, torch.tensor([n], dtype=torch.int32, device=dev()), lse=True,
                                              max_q=m, max_kv=n))
    for a, b in ((0, 1), (0, 3), (0, 4), (2, 5)):
        assert torch.equal(got[a][0], got[b][0]) and torch.equal(got[a][1], got[b][1])
