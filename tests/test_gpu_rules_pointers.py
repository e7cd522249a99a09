"""Host memory where a matrix of the device is expected is refused before any launch."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("pinned", [False, True])
def test_host_rows_are_refused(pinned):
    host = torch.zeros(4, 64, dtype=torch.bfloat16, pin_memory=pinned)
    dev = torch.full((4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    u = ps.make_rules()
    assert ps.ps_process_rows(u, host, dev, st, stream=0, check=False) == 1
    assert ps.ps_process_rows(u, dev, host, st, stream=0, check=False) == 1
    assert ps.ps_process_rows(u, host, host, st, stream=0, check=False) == 1
    assert ps.ps_process_rows(u, dev.clone(), dev, st, stream=0, check=False) == 0
    torch.cuda.synchronize()
    assert bool((dev == 3.0).all()) and int(st.item()) == 0


@pytest.mark.parametrize("pinned", [False, True])
def test_host_matrices_of_a_head_are_refused(pinned):
    make = lambda *shape, dtype, on: (torch.zeros(*shape, dtype=dtype, device=DEV) if on else       # noqa: E731
                                      torch.zeros(*shape, dtype=dtype, pin_memory=pinned))
    for hidden, q, out in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1)):
        head = ps.make_head(q=make(40, 32, dtype=torch.uint8, on=q),
                            scales=torch.zeros(40, 1, device=DEV), group=64)
        h = make(2, 64, dtype=torch.bfloat16, on=hidden)
        y = make(2, 40, dtype=torch.float32, on=out)
        want = 0 if hidden and q and out else 1
        assert ps.ps_head_rows(head, h, y, stream=0, check=False) == want
    torch.cuda.synchronize()
