"""The head called first thing in a host thread that has used no CUDA before."""

import threading

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("n,V", [(1, 512), (40, 39000), (20, 39000)])
def test_first_call_of_a_thread(n, V):
    K, group = 512, 64
    g = torch.Generator(device=DEV).manual_seed(n)
    q = torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    s = torch.rand(V, K // group, device=DEV, generator=g) / K ** 0.5
    h = torch.randn(n, K, device=DEV, generator=g).to(torch.bfloat16)
    head = ps.make_head(q=q, scales=s, group=group)
    out = [torch.zeros(n, V, device=DEV) for _ in range(4)]
    ps.ps_head_rows(head, h, out[0])
    torch.cuda.synchronize()
    stream = torch.cuda.Stream().cuda_stream               # a number: the threads make no CUDA objects
    status = []
    for o in out[1:]:
        t = threading.Thread(
            target=lambda: status.append(ps.ps_head_rows(head, h, o, stream=stream, check=False)))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert status == [ps.PS_OK] * 3
    assert all(torch.equal(o, out[0]) for o in out[1:])
