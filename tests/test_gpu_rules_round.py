"""A whole round under rules: the example's, and DeviceSubtree against the oracle."""

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps
import oracle
from oracle import rules as O
from synth.trees import assemble_layout, bfs_tree
from tests import gpu_harness as H
from tests import rules_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


def test_the_example_scores_what_it_drew():
    from examples.rules_round import main
    r = main(V=2000, T=40, n_pf=6)
    req = ~r["layout"].is_root()
    T = 40
    # the draws took bfloat16 rows after the rules, the scores float32 ones: each logit
    # is off by 2^-8 of its size at most (|l| < 16 here), twice (token and normaliser),
    # divided by tau = 1/4
    n = T - r["layout"].seg_cut[req]
    assert (np.abs(r["drawn_lq"] - r["lq_y"])[req] <= n * 2 * 16 * 2.0 ** -8 / 0.25).all()
    assert np.isfinite(r["lq_y"][req]).all() and (r["log_accept"][req] <= 0).all()


def test_round_under_rules_against_the_oracle():
    rng = np.random.default_rng(31)
    V = 3000
    lay = assemble_layout([bfs_tree(rng, 24, 5) for _ in range(3)])
    n = lay.n_rows
    r = C.random_rules(rng, V, n, n_seqs=7)
    x = C.logits(rng, n, V, "bf16")
    y, _ = O.process_rows(C.host(x, V), r)
    # every token allowed, so that all sums are finite
    tok = np.array([rng.choice(np.nonzero(np.isfinite(row))[0]) for row in y]).astype(np.int32)
    u = 1.0 - rng.random(lay.n_seg)
    d = ps.DeviceSubtree.create(layout=lay, u=u, logits=x.to(DEV), tokens=torch.from_numpy(tok).to(DEV),
                                V=V, alpha=4.0, tau=0.25, max_steps=20, entropy=True, per_row=False,
                                rules=C.device_rules(r, DEV))
    d.step()
    torch.cuda.synchronize()
    assert int(d.t["status"].item()) == 0 and int(d.t["wstatus"].item()) == 0
    lp0, lq, ent = O.logprobs(y, tok, 0.25)
    g = {k: d.t[k].cpu().numpy() for k in ("lp0", "lq", "entropy", "log_accept", "path", "k_delta",
                                           "state_seg")}
    H.check_rows(g, dict(lp0=lp0, lq=lq, entropy=ent))
    sums = oracle.suffix_sums(lay, lp0, lq)
    _, la = oracle.log_accept(sums, 4.0)
    req = ~lay.is_root()
    assert (np.abs(g["log_accept"] - la)[req] <= H.LA_ATOL).all()
    wk = oracle.walk(lay, g["log_accept"], u, 20)
    assert np.array_equal(g["k_delta"], wk["k_delta"]) and np.array_equal(g["state_seg"], wk["state_seg"])
    # the carried values are those of the rules' distribution
    out = d.carry({k: torch.zeros(3, 24, dtype=torch.float64, device=DEV) for k in ("lp0", "lq", "entropy")})
    torch.cuda.synchronize()
    assert int(out["status"].item()) == 0


def test_rules_that_are_too_few_are_refused():
    rng = np.random.default_rng(32)
    lay = assemble_layout([bfs_tree(rng, 8, 2)])
    x = torch.zeros(lay.n_rows, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        ps.DeviceSubtree.create(layout=lay, u=np.ones(lay.n_seg), logits=x,
                                tokens=torch.zeros(lay.n_rows, dtype=torch.int32, device=DEV), V=64,
                                alpha=1.0, tau=0.5, max_steps=4,
                                rules=ps.make_rules(seq_begin=torch.zeros(2, dtype=torch.int64, device=DEV),
                                                    seq_tokens=torch.zeros(0, dtype=torch.int32, device=DEV),
                                                    row_seq=torch.zeros(3, dtype=torch.int32, device=DEV)))
