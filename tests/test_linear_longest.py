"""The longest rows of a projection: K up to 2^24 is accepted, more is refused (no GPU)."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

OK, INVALID = 0, 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from mh_prefetch_subtree_gb300.build import build
    build()


@pytest.mark.parametrize("K, status", [(2 ** 24, OK), (2 ** 24 + 8, INVALID), (2 ** 31 - 8, INVALID)])
def test_longest(K, status):
    w = torch.zeros(8, 8, dtype=torch.bfloat16)
    lin = ps.make_linear(w=w)
    lin.N, lin.K, lin.w_ld = 1, K, K
    # no rows: what is wrong with the projection itself is said all the same
    assert ps.lib().ps_linear_rows(lin, None, 0, 0, None, 0, None, 0, 0, None) == status
