"""Page tables without columns: nobody's tokens have a place."""

import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_attention import Problem, mxa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 40])
def test_tables_without_columns(m):
    p = Problem([(m, 50), (m, 0), (m, 1)], 8, 2, 64)
    cache, _, cu, lens = p.gpu_args()
    out, lse = mxa.mx_paged_attention(p.q, cache, torch.zeros((3, 0), dtype=torch.int32, device=dev()), cu, lens, lse=True,
                                      max_q=m, max_kv=50)
    sees = torch.zeros(3 * m, dtype=torch.bool, device=dev())
    sees[:m] = torch.arange(m, device=dev()) >= m - 50
    sees[-1] = True
    assert out[sees].isnan().all() and lse[sees].isnan().all()
    assert (out[~sees] == 0).all() and (lse[~sees] == -float("inf")).all()


@pytest.mark.parametrize("heads", [8, 1])
def test_strides_of_single_tokens_and_heads(heads):
    """The stride of a dimension of one element means nothing, though it is no multiple of 16 bytes."""
    p = Problem([(1, 50)] if heads > 1 else [(3, 50)], heads, 1, 64)
    q = p.q.contiguous()
    odd = q.as_strided(q.shape, (3, 64, 1) if heads > 1 else (64, 3, 1))
    args = p.gpu_args()
    want = mxa.mx_paged_attention(q, *args, max_q=3, max_kv=50)
    assert torch.equal(mxa.mx_paged_attention(odd, *args, max_q=3, max_kv=50), want)
    table, pos = mxa.mx_rope_table(64, 64), args[3][:1] if heads > 1 else torch.arange(3, dtype=torch.int32, device=dev())
    assert torch.equal(mxa.mx_rope(odd, pos, table), mxa.mx_rope(q, pos, table))
    assert odd.data_ptr() == q.data_ptr()
