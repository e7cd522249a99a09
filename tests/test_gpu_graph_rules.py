"""The operators for proposals under rules captured in a CUDA graph: a replay reads its
inputs afresh (a decoding loop writes the next hidden states, lengths, masks and tokens
into the same tensors) and gives the bits of the same calls made one by one."""

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


@pytest.mark.parametrize("n,V,K", [(3, 2000, 256), (12, 2000, 512), (40, 39000, 512)])
def test_a_decoding_step_replays(n, V, K):
    rng = np.random.default_rng(n)
    g = torch.Generator(device=DEV).manual_seed(n)
    group, ld = 64, -(-V // 8) * 8
    head = ps.make_head(
        q=torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device=DEV, generator=g),
        scales=torch.rand(V, K // group, device=DEV, generator=g) / K ** 0.5, group=group)
    hidden = torch.randn(n, K, device=DEV, generator=g).to(torch.bfloat16)
    r = C.random_rules(rng, V, n)
    rules = C.device_rules(r, DEV)
    row_len, row_mask, toks = rules._keep[11], rules._keep[12], rules._keep[1]
    rows, out, inplace = (torch.zeros(n, ld, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    one = lambda *v: torch.tensor(v, device=DEV)                         # noqa: E731
    tok = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).to(DEV)
    b = ps.make_batch(V=V, T=n, alpha=4.0, tau=0.25, chain_seg0=one(0, 1).int(), seg_row0=one(0, n),
                      seg_cut=one(0).int(), seg_src=one(-1).int(), logits=rows, tokens=tok)
    res = [torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(3)]
    ws = torch.empty(ps.ps_rules_workspace_bytes(b), dtype=torch.uint8, device=DEV)

    def step(stream):
        ps.ps_head_rows(head, hidden, rows, stream=stream)
        ps.ps_process_rows(rules, rows, out, st, V=V, stream=stream)
        inplace.copy_(rows)
        ps.ps_process_rows(rules, inplace, inplace, st, V=V, stream=stream)
        ps.ps_score_rows_rules(b, rules, res[0], res[1], st, ws, stream=stream, entropy=res[2])

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (rows, out, inplace, *res)]

    def same(xs, ys):
        as_int = {2: torch.int16, 8: torch.int64}
        for x, y in zip(xs, ys):
            assert torch.equal(x.view(as_int[x.element_size()]), y.view(as_int[y.element_size()]))

    s = torch.cuda.Stream(device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(s)
    eager = [results()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    graph.replay()
    same(results(), eager[0])
    # the next step's contents in the same tensors
    hidden.copy_(torch.randn(n, K, device=DEV, generator=g))
    row_len.copy_(torch.from_numpy(np.array([rng.integers(0, e + 1) for e in np.diff(r.seq_begin)[r.row_seq]],
                                            np.int32)))
    row_mask.copy_(torch.from_numpy(rng.integers(-1, 4, n).astype(np.int32)))
    toks.copy_(toks.flip(0))
    tok.copy_(torch.from_numpy(rng.integers(0, V, n).astype(np.int32)))
    graph.replay()
    replayed = results()
    for t in (rows, out, inplace, *res):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step(s)
    again = results()
    same(replayed, again)
    assert not torch.equal(again[0], eager[0][0]) and int(st.item()) == 0
