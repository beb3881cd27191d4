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
