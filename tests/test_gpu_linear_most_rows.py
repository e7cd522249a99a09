"""ps_linear_rows with as many rows as its argument can say: 2^31 - 1 of 8 inputs and 8 outputs, 34 GB each.

Tolerance: as in test_gpu_linear.py, (K / 16 + 16) 2^-23 of the sum's size, then one rounding to bfloat16."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 256, 2 ** 30 + 3])
def test_most_rows(n):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    g = torch.Generator(device=DEV).manual_seed(n)
    K = N = 8
    w = torch.randn(N, K, device=DEV, generator=g).to(torch.bfloat16)
    bias = torch.randn(N, device=DEV, generator=g).to(torch.bfloat16)
    x = torch.zeros(n, K, dtype=torch.bfloat16, device=DEV)
    out = torch.full((n, N), 77.0, dtype=torch.bfloat16, device=DEV)
    some = [0, 2 ** 30 - 300, 2 ** 30, n - 600]
    for r in some:
        x[r:r + 600] = torch.randn(min(600, n - r), K, device=DEV, generator=g)
    ps.ps_linear_rows(ps.make_linear(w=w, bias=bias), x, out)
    torch.cuda.synchronize()
    for r in some:
        a = x[r:r + 600].double()
        want, size = a @ w.double().t() + bias.double(), a.abs() @ w.double().abs().t() + bias.double().abs()
        err = (K / 16 + 16) * 2.0 ** -23 * size * (1 + 2.0 ** -7) + 2.0 ** -8 * want.abs()
        assert ((out[r:r + 600].double() - want).abs() <= err).all(), r
    for r in some:
        out[r:r + 600] = bias
    # the others' inputs are zero
    step = 2 ** 27
    for r in range(0, n, step):
        assert bool((out[r:r + step] == bias).all()), r
    del x, out
    torch.cuda.empty_cache()
