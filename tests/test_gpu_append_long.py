"""An append of more threads than one launch takes."""

import pytest
import torch

from tests.gpu_util import dev, import_library

pytestmark = pytest.mark.gpu

mxa = import_library()


def test_more_tokens_than_a_launch():
    """45 million tokens, 32 threads each for an unaligned query and 8 each for a key and a value: 2.16e9.  All are one
    token repeated (stride 0) at positions of their own; those around the cut at 2^31 / 48 and the last are stored."""
    n, cut = 45_000_000, 0x7FFFFC00 // 48
    g = torch.Generator(device=dev()).manual_seed(1)
    flat = torch.randn(65, device=dev(), generator=g).bfloat16()
    q = flat[1:].view(1, 1, 64).expand(n, 1, 64)
    k, v = (torch.randn((1, 1, 64), device=dev(), generator=g).bfloat16().expand(n, 1, 64) for _ in range(2))
    table = mxa.mx_rope_table(1000, 64)
    pos = torch.arange(n, dtype=torch.int32, device=dev()) % 1000
    slots = torch.full((n,), -1, dtype=torch.int64, device=dev())
    at = torch.tensor([0, 1, cut - 2, cut - 1, cut, cut + 1, n - 2, n - 1], device=dev())
    slots[at] = torch.arange(8, device=dev())
    cache, small = mxa.new_kv_cache(1, 1, 16, 64), mxa.new_kv_cache(1, 1, 16, 64)
    out = mxa.mx_kv_append(k, v, cache, slots, pos, table, q=q)
    want = mxa.mx_kv_append(k[:8], v[:8], small, torch.arange(8, device=dev()), pos[at], table, q=q[:8])
    assert torch.equal(out[at], want)
    for a, b in zip(cache, small):
        assert torch.equal(a, b)
    rows = mxa.mx_kv_append(k[:1000], v[:1000], small, slots[2:1002], pos[:1000], table, q=q[:1000])
    assert torch.equal(out.view(n // 1000, 1000, 1, 64)[::4999], rows.expand(n // 1000, -1, -1, -1).view(-1, 1000, 1, 64)[::4999])
    assert torch.equal(out[cut - 500:cut + 500], rows[pos[cut - 500:cut + 500].long()])
