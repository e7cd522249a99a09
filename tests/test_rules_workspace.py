"""The workspace of scoring under rules: what is enough for a batch is enough for every
smaller one."""

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps
from oracle import rules as O
from tests import rules_cases as C


@pytest.fixture(scope="module", autouse=True)
def built():
    from mh_prefetch_subtree_gb300.build import build
    build()


def batch(n, V, dtype):
    b = ps.PsSubtreeBatch()
    b.V, b.n_rows, b.dtype = V, n, dtype
    return b


@pytest.mark.parametrize("dtype", [ps.PS_BF16, ps.PS_F32])
@pytest.mark.parametrize("V", [1, 1000, 1024, 1025, 2048, 5003, 12289, 24577, 50021, 128256, 151936,
                               262144, 1 << 22, 1 << 27])
def test_workspace_rises_with_the_rows(V, dtype):
    rows = list(range(0, 400)) + [1000, 1001, 65536, 100000]
    need = [ps.ps_rules_workspace_bytes(batch(n, V, dtype)) for n in rows]
    assert all(a <= b for a, b in zip(need, need[1:]))


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(50021, "bf16"), (13001, "f32")])
def test_one_workspace_serves_all_smaller_batches(V, dtype):
    """Also shows that no count writes past its own size: what lies behind it stays."""
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(51)
    most = 40
    x = C.logits(rng, most, V, dtype)
    r = C.random_rules(rng, V, most, n_masks=0)
    xd, tok = x.to(dev), rng.integers(0, V, most)
    one = lambda *v: torch.tensor(v, device=dev)
    pad = 1 << 14
    for k, n in enumerate([40, 1, 2, 3, 5, 8, 16, 20, 31, 40]):
        s = {a: getattr(r, a) for a in vars(r)}
        s.update(row_seq=r.row_seq[:n], row_len=r.row_len[:n])
        b = ps.make_batch(V=V, T=n, alpha=4.0, tau=0.5, chain_seg0=one(0, 1).int(), seg_row0=one(0, n),
                          seg_cut=one(0).int(), seg_src=one(-1).int(), logits=xd[:n],
                          tokens=torch.from_numpy(tok[:n].astype(np.int32)).to(dev))
        need = ps.ps_rules_workspace_bytes(b)
        if k == 0:
            ws = torch.empty(need + pad, dtype=torch.uint8, device=dev)
            total = need
        ws.fill_(0x5A)
        lp0, lq = (torch.zeros(n, dtype=torch.float64, device=dev) for _ in range(2))
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        ps.ps_score_rows_rules(b, C.device_rules(O.Rules(**s), dev), lp0, lq, st, ws[:total])
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and bool((ws[need:] == 0x5A).all())
        y, _ = O.process_rows(C.host(x[:n], V), O.Rules(**s))
        want, _, _ = O.logprobs(y, tok[:n], 0.5)
        assert np.allclose(lp0.cpu().numpy(), want, rtol=1e-4, atol=1e-300)
