"""Waits of the many-row head kernel that run out: no logit is wrong, each is the one of
an undisturbed call or NaN, and the next call is right."""

import time

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


# one block holds the hidden rows, or the two of a cluster half of them each; with two
# tiles of two units nothing but the weights' own hand-over could stop wrong ones
@pytest.mark.parametrize("K,blocks,tiles", [(256, 1, 2), (512, 1, 3), (1536, 2, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lost_copies_give_nan(K, blocks, tiles, dtype):
    n, group = 40, 128
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    V = tiles * 256 * sms - 8                              # of a pipeline
    g = torch.Generator(device=DEV).manual_seed(K)
    q = torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    s = (torch.rand(V, K // group, device=DEV, generator=g) / K ** 0.5).to(torch.bfloat16)
    h = torch.randn(n, K, device=DEV, generator=g).to(torch.bfloat16)
    head = ps.make_head(q=q, scales=s, group=group)
    want, got, after = (torch.full((n, V), 7.0, dtype=dtype, device=DEV) for _ in range(3))
    ps.ps_head_rows(head, h, want)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ps.ps_selftest_head_wait(head, h, got)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    nan = torch.isnan(got)
    assert torch.equal(got[~nan], want[~nan])
    # the first block's rows: of each tile pair 128 a pipeline, of a cluster's 256 the first
    rows = torch.arange(V, device=DEV)
    pair, first = rows // (256 * blocks), rows // 128 % blocks == 0
    lost = first & (pair % (sms // blocks) == 0) & (pair > 0)
    assert int(lost.sum()) == (tiles - 1) * 256
    assert nan[:, lost].all()
    # what the failure cannot reach is there
    assert not nan[:, pair % (sms // blocks) != 0].any()
    ps.ps_head_rows(head, h, after)
    torch.cuda.synchronize()
    assert torch.equal(after, want)


def test_refusals():
    head = lambda K, group, scale: ps.make_head(                         # noqa: E731
        q=torch.zeros(64, K // 2, dtype=torch.uint8, device=DEV),
        scales=torch.zeros(64, K // group, dtype=scale, device=DEV), group=group)
    for n, K, group, scale in ((32, 512, 128, torch.bfloat16), (65, 512, 128, torch.bfloat16),
                               (40, 128, 128, torch.bfloat16), (40, 4096, 128, torch.bfloat16),
                               (40, 512, 64, torch.bfloat16), (40, 512, 128, torch.float32)):
        h = torch.zeros(n, K, dtype=torch.bfloat16, device=DEV)
        assert ps.ps_selftest_head_wait(head(K, group, scale), h, torch.zeros(n, 64, device=DEV),
                                        check=False) == 1
