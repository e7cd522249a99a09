"""Capped projections from the smallest cap to the largest, zeros and infinities among the sums.

Tolerance: that of test_gpu_linear.py: sums to (K / 16 + 16) 2^-23 of their size (the slope is at most 1), the
activation to 2^-20 of its value; with the largest cap z / cap is a multiple of 2^-149, so z one of 2^-89."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("cap", [2.0 ** -60, 1e-3, 0.1, 30.0, 1e6, 2.0 ** 60])
@pytest.mark.parametrize("scale", [1e-6, 1.0, 1e6])
@pytest.mark.parametrize("rows", [3, 150])
def test_caps(cap, scale, rows):
    cap = float(torch.tensor(cap))              # as the projection holds it
    N, K, g = 200, 64, torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, K, device=DEV, generator=g).to(torch.bfloat16)
    w = (scale * torch.randn(N, K, device=DEV, generator=g)).to(torch.bfloat16)
    x[1] = 0
    out = torch.full((rows, N), 77.0, device=DEV)
    ps.ps_linear_rows(ps.make_linear(w=w, act="cap", cap=cap), x, out)
    z, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    y = cap * torch.tanh(z / cap)
    assert ((out.double() - y).abs() <= (K / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -20 * y.abs() + 2.0 ** -89).all()
    assert (out[1] == 0).all()
    x[2, 0] = float("inf")
    ps.ps_linear_rows(ps.make_linear(w=w, act="cap", cap=cap), x, out)
    assert torch.equal(out[2].double(), cap * w[:, 0].double().sign())
