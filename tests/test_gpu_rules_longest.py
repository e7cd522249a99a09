"""Histories of 2^31 - 1 tokens, the longest that a row can see: the indexes of the loops
over them pass 2^31."""

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps
from oracle import rules as O
from tests import rules_cases as C
from tests.test_gpu_rules import check_process, check_score

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
L, TAIL, MADE, V = 2 ** 31 - 1, 3000, 1000, 1000


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


def test_longest_history():
    if torch.cuda.get_device_properties(DEV).total_memory < 40 << 30:
        pytest.skip("9 GB of tokens")
    rng = np.random.default_rng(61)
    g = torch.Generator(device=DEV).manual_seed(61)
    n = 304                                               # two rows a block, one after the other
    hist = torch.randint(0, 500, (L,), dtype=torch.int32, device=DEV, generator=g)
    tail = rng.integers(480, 700, TAIL).astype(np.int32)
    hist[-TAIL:] = torch.from_numpy(tail).to(DEV)
    short = np.concatenate([np.arange(500), tail]).astype(np.int32)    # as many seen, the same tail
    lens = np.sort(rng.integers(L - 40, L + 1, n))
    lens[::2] = np.minimum(lens[::2], lens[1::2])
    lens[1::2] = np.minimum(lens[1::2], lens[::2] + 6)
    lens[-2:] = L - 3, L
    kw = dict(repetition=np.array([1.2], np.float32), frequency=np.array([0.3], np.float32),
              presence=np.array([0.4], np.float32), row_seq=np.zeros(n, np.int32))
    r = O.Rules(seq_begin=np.array([0, 500 + TAIL]), seq_tokens=short,
                seq_prompt=np.array([500 + TAIL - MADE], np.int32),
                row_len=(lens - (L - 500 - TAIL)).astype(np.int32), **kw)
    dev = lambda a: torch.from_numpy(np.asarray(a)).to(DEV)              # noqa: E731
    rules = ps.make_rules(seq_begin=dev(np.array([0, L])), seq_tokens=hist,
                          seq_prompt=dev(np.array([L - MADE], np.int32)),
                          row_len=dev(lens.astype(np.int32)), **{k: dev(a) for k, a in kw.items()})
    x = C.logits(rng, n, V, "f32")
    xd, st = x.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(xd)
    ps.ps_process_rows(rules, xd, out, st, V=V)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_process(out.cpu()[:, :V], x, r, V, "f32")
    few = xd[:4].clone()
    ps.ps_process_rows(rules, few, few, st, V=V)          # in place
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(few, out[:4])
    tok = rng.integers(0, V, n)
    one = lambda *v: torch.tensor(v, device=DEV)                         # noqa: E731
    b = ps.make_batch(V=V, T=n, alpha=4.0, tau=0.25, chain_seg0=one(0, 1).int(), seg_row0=one(0, n),
                      seg_cut=one(0).int(), seg_src=one(-1).int(), logits=xd,
                      tokens=dev(tok.astype(np.int32)))
    res = [torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(3)]
    ws = torch.empty(ps.ps_rules_workspace_bytes(b), dtype=torch.uint8, device=DEV)
    ps.ps_score_rows_rules(b, rules, res[0], res[1], st, ws, entropy=res[2])
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_score(dict(zip(("lp0", "lq", "entropy"), (a.cpu().numpy() for a in res))), x, r, V, tok, 0.25)
