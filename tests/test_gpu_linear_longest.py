"""ps_linear_rows with rows of 2^24 inputs, the longest that it takes: no wait runs out on the way.

Nearly all products are zero, whose additions are exact, and 64 are not: each of their additions is off by at most
2^-23 of the sum's size, as are the 8 of a divided k's parts; then a rounding to bfloat16."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("rows, N, dtype", [(1, 3, torch.float32), (40, 200, torch.bfloat16), (130, 300, torch.bfloat16),
                                            (260, 130, torch.float32)])
def test_longest(rows, N, dtype):
    K, g = 2 ** 24, torch.Generator(device=DEV).manual_seed(rows)
    at = torch.cat([torch.randperm(K - 2, device=DEV, generator=g)[:62] + 1, torch.tensor([0, K - 1], device=DEV)])
    x, w = (torch.zeros(n, K, dtype=torch.bfloat16, device=DEV) for n in (rows, N))
    x[:, at] = torch.randn(rows, 64, device=DEV, generator=g).to(torch.bfloat16)
    w[:, at] = torch.randn(N, 64, device=DEV, generator=g).to(torch.bfloat16)
    out = torch.full((rows, -(-N // 8) * 8), 77.0, dtype=dtype, device=DEV)
    ps.ps_linear_rows(ps.make_linear(w=w), x, out)
    a, b = x[:, at].double(), w[:, at].double()
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    err = (64 + 8) * 2.0 ** -23 * size + torch.finfo(dtype).eps / 2 * want.abs()
    assert ((out[:, :N].double() - want).abs() <= err * (1 + 2.0 ** -7)).all()
