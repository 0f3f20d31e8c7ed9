"""Sizes past what an attention counts are refused, also where they would come
back small in 32 bits."""
import pytest
import torch

import decode_kv_cache_02_gb300 as pkg
from tests.test_gpu_cache import BF, DEV, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [0, -1, (1 << 30) + 1, 1 << 31, (1 << 32) + 100])
def test_rows_past_the_limit(rows):
    K = torch.zeros(4, 1, 16, 64, dtype=BF, device=DEV)
    table, lens = torch.zeros(1, 4, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    q = rnd((1, 1, 1, 64), BF, 1)
    with pytest.raises(ValueError):
        pkg.rkv_paged_attention(q, K, K.clone(), table, lens, max_rows=rows)
    with pytest.raises(ValueError):
        pkg.rkv_attention_workspace_size(q, 1, rows)


def test_a_table_of_more_rows_than_32_bits_count():
    """2^22 + 1 blocks of 1024 rows: the default bound is 2^32 + 1024, which a C
    int holds as 1024; a bound of the caller's own is taken."""
    K = rnd((3, 1, 1024, 64), BF, 2)
    V = rnd((3, 1, 1024, 64), BF, 3)
    table = torch.zeros(1, (1 << 22) + 1, dtype=torch.int32, device=DEV)
    table[0, :3] = torch.tensor([2, 0, 1])
    lens = torch.full((1,), 2000, dtype=torch.int32, device=DEV)
    q = rnd((1, 1, 2, 64), BF, 1)
    with pytest.raises(ValueError):
        pkg.rkv_paged_attention(q, K, V, table, lens)
    a = pkg.rkv_paged_attention(q, K, V, table, lens, max_rows=2000)
    b = pkg.rkv_paged_attention(q, K, V, table[:, :3].contiguous(), lens, max_rows=2000)
    assert torch.equal(a, b)
