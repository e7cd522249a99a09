"""The caps of a projection: 2^-60 to 2^60 (no GPU)."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

OK, INVALID = 0, 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from mh_prefetch_subtree_gb300.build import build
    build()


@pytest.mark.parametrize("cap, status", [(30.0, OK), (2.0 ** -60, OK), (2.0 ** 60, OK), (2.0 ** 61, INVALID), (3e38, INVALID),
                                         (2.0 ** -61, INVALID), (1e-39, INVALID), (0.0, INVALID), (-1.0, INVALID),
                                         (float("inf"), INVALID), (float("nan"), INVALID)])
def test_caps(cap, status):
    lin = ps.make_linear(w=torch.zeros(8, 8, dtype=torch.bfloat16), act="cap", cap=cap)
    assert ps.lib().ps_linear_rows(lin, None, 0, 0, None, 0, None, 0, 0, None) == status
    lin.act = ps.PS_ACTS["none"]                # not read
    assert ps.lib().ps_linear_rows(lin, None, 0, 0, None, 0, None, 0, 0, None) == OK
