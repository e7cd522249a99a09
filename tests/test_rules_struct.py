"""A ps_logit_rules that the caller fills field by field, as the other structs may be."""

import torch

import mh_prefetch_subtree_gb300 as ps


def test_rules_filled_by_field_reach_the_library():
    from mh_prefetch_subtree_gb300.build import build
    build()
    u = ps.PsLogitRules()
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32)
    # accepted by the binding; host memory is then refused as not being the device's
    assert ps.ps_process_rows(u, x, torch.zeros_like(x), st, stream=0, check=False) == 1
    u.n_seqs = -1
    assert ps.ps_process_rows(u, x[:0], x[:0], st, stream=0, check=False) == 1
    u.n_seqs = 0
    assert ps.ps_process_rows(u, x[:0], x[:0], st, stream=0, check=False) == 0
