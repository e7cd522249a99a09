"""Matrices of a projection that would span more than 2^40 elements are refused before anything is counted in bytes (no GPU)."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

INVALID = 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from mh_prefetch_subtree_gb300.build import build
    build()


@pytest.mark.parametrize("rows, x_ld, w_rows, w_ld, ld", [
    (2 ** 26, 2 ** 38, 8, 8, 8),                # x
    (2 ** 31 - 1, 2 ** 38, 8, 8, 8),
    (3, 8, 2 ** 27, 2 ** 38, 2 ** 27),          # w
    (3, 8, 2 ** 29, 2 ** 12, 2 ** 29),
    (0, 8, 2 ** 27, 2 ** 38, 2 ** 27),          # before any row is asked for
    (2 ** 31 - 1, 8, 8, 8, 2 ** 30),            # out
    (0, 8, 1, 2 ** 39, 8),                      # a row, and the next one further than a tile's rows may be
])
def test_spans(rows, x_ld, w_rows, w_ld, ld):
    x, w, out = (torch.zeros(64, dtype=torch.bfloat16) for _ in range(3))
    lin = ps.make_linear(w=torch.zeros(8, 8, dtype=torch.bfloat16))
    lin.N, lin.K, lin.w_ld, lin.w = w_rows, 8, w_ld, w.data_ptr()
    assert ps.lib().ps_linear_rows(lin, x.data_ptr(), x_ld, rows, None, 0, out.data_ptr(), ld, 0, None) == INVALID
