"""Corners of the attention calls: what a caller may do and seldom does (needs a GB300).

Inputs, results in 64 bits and their tolerances are those of test_attention_gpu.py.
"""

import pytest
import torch

from test_attention_gpu import Want, b2b, ints, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# ----------------------------------------------------------------- page tables
@pytest.mark.parametrize("pages", [0, 2, 5])
@pytest.mark.parametrize("prefix", [0, 150])
def test_a_page_table_without_columns_holds_no_keys(prefix, pages):
    """No request has a page yet: lengths are clamped to the table, also where the pool has as many pages as there are
    requests (an empty tensor's address is null, as that of no table)."""
    q, k, v = normal(1, 2, 4, 64), normal(2, prefix, 2, 64), normal(3, prefix, 2, 64)
    pool, lengths = normal(4, pages, 16, 2, 64), ints([5, 9])
    plan = b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    want = Want(2, 4, 64)
    for b in range(2):
        want.rows(b, q[b:b + 1], k, v, [prefix], 1 / 8, "f16")
    for table in (torch.empty(2, 0, dtype=torch.int32, device="cuda"), ints([[0, 1], [1, 0]])[:, :0]):
        want.check(*plan.run(q, k, v, pool, pool, lengths, table, return_lse=True))
        out, lse = torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device="cuda")
        want.check(*plan.run(q, k, v, pool, pool, lengths, table, out=out, lse=lse))
    assert plan.status() == 0
