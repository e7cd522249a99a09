"""ps_head_rows with as many rows as its argument can say: 2^31 - 1 of 32 inputs (137 GB) and 8 outputs (34 GB).

Tolerance: products are exact; 32 of them and a group's scale are float32, (32 + 2) 2^-24 of the sum's size, then one
rounding to bfloat16."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 30 + 3])
def test_most_rows(n):
    torch.cuda.empty_cache()
    K, V = 32, 8
    if torch.cuda.mem_get_info()[0] < n * (K + V) * 2 + (20 << 30):
        pytest.skip("needs up to 192 GB of free device memory")
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.rand(V, 1, device=DEV, generator=g)
    w = torch.stack([q & 15, q >> 4], 2).reshape(V, K).double().sub(8) * scales.double()
    hidden = torch.zeros(n, K, dtype=torch.bfloat16, device=DEV)
    logits = torch.full((n, V), 77.0, dtype=torch.bfloat16, device=DEV)
    some = [0, 2 ** 30 - 300, n - 600] if n > 2 ** 30 + 600 else [0, n - 600]
    for r in some:
        hidden[r:r + 600] = torch.randn(600, K, device=DEV, generator=g)
    ps.ps_head_rows(ps.make_head(q=q, scales=scales, group=32), hidden, logits)
    torch.cuda.synchronize()
    for r in some:
        a = hidden[r:r + 600].double()
        want, size = a @ w.t(), a.abs() @ w.abs().t()
        assert ((logits[r:r + 600].double() - want).abs() <= 34 * 2.0 ** -24 * size * 1.01 + 2.0 ** -8 * want.abs()).all(), r
        logits[r:r + 600] = 0
    step = 2 ** 27
    for r in range(0, n, step):                 # the others' hidden states are zero
        assert not bool(logits[r:r + step].any()), r
    del hidden, logits
    torch.cuda.empty_cache()
