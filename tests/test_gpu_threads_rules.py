"""The operators for proposals under rules from several host threads, each on its own
stream: every call is accepted, and its results are those of the same call alone,
bit for bit.  The heads of two threads share a kernel and differ in its shared memory."""

import threading

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps
from tests import rules_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


def _head(n, V, K, group, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    s = (torch.rand(V, K // group, device=DEV, generator=g) / K ** 0.5).to(torch.bfloat16)
    h = torch.randn(n, K, device=DEV, generator=g).to(torch.bfloat16)
    out = torch.zeros(n, -(-V // 8) * 8, dtype=torch.bfloat16, device=DEV)
    head = ps.make_head(q=q, scales=s, group=group)
    return (lambda stream: ps.ps_head_rows(head, h, out, stream=stream)), [out]


def _process(V, n, seed):
    rng = np.random.default_rng(seed)
    x = C.logits(rng, n, V, "bf16").to(DEV)
    rules = C.device_rules(C.random_rules(rng, V, n), DEV)
    out, st = torch.zeros_like(x), torch.zeros(1, dtype=torch.int32, device=DEV)
    return (lambda stream: ps.ps_process_rows(rules, x, out, st, V=V, stream=stream)), [out, st]


def _score(V, n, seed):
    rng = np.random.default_rng(seed)
    x = C.logits(rng, n, V, "bf16").to(DEV)
    rules = C.device_rules(C.random_rules(rng, V, n), DEV)
    one = lambda *v: torch.tensor(v, device=DEV)
    b = ps.make_batch(V=V, T=n, alpha=4.0, tau=0.25, chain_seg0=one(0, 1).int(), seg_row0=one(0, n),
                      seg_cut=one(0).int(), seg_src=one(-1).int(), logits=x,
                      tokens=torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).to(DEV))
    f = [torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(3)]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(ps.ps_rules_workspace_bytes(b), dtype=torch.uint8, device=DEV)
    return (lambda stream: ps.ps_score_rows_rules(b, rules, f[0], f[1], st, ws, stream=stream,
                                                  entropy=f[2])), f + [st]


def _together(makers, rounds):
    jobs = [m() for m in makers]
    alone = []
    for call, outs in jobs:
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    errors, gate = [], threading.Barrier(len(jobs))

    def run(call):
        try:
            s = torch.cuda.Stream(device=DEV)
            gate.wait()
            for i in range(rounds):
                call(s)
                if i % 200 == 199:
                    s.synchronize()
            s.synchronize()
        except Exception as e:          # reported below
            errors.append(e)

    th = [threading.Thread(target=run, args=(call,)) for call, _ in jobs]
    for t in th:
        t.start()
    for t in th:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, outs), want in zip(jobs, alone):
        for o, w in zip(outs, want):
            # bits, so that NaN compares too
            as_int = {2: torch.int16, 4: torch.int32, 8: torch.int64}[o.element_size()]
            assert torch.equal(o.view(as_int), w.view(as_int))


@pytest.mark.parametrize("n,V,K", [(1, 512, (256, 8192)), (12, 512, (256, 4096)), (24, 512, (256, 2048)),
                                   (64, 39000, (256, 1024))])
def test_heads_of_two_widths(n, V, K):
    makers = [lambda k=k, i=i: _head(n, V, k, 128, i) for i, k in enumerate(K + K)]
    _together(makers, 4000 if V < 1000 else 1000)


def test_all_operators_at_once():
    _together([lambda: _head(1, 4096, 1024, 64, 1), lambda: _head(40, 39000, 512, 64, 2),
               lambda: _process(20001, 30, 3), lambda: _score(20001, 30, 4),
               lambda: _score(1001, 300, 5)], 300)
