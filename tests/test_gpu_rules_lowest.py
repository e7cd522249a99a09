"""Scoring under rules where processed logits of seen or biased ids are finite but
as low as the type goes: a suppressed id that is in the history, a bias of the
type's lowest value.  They carry no mass and may not reach the row's other sums."""

import numpy as np
import pytest
import torch

from oracle import rules as O
from tests import rules_cases as C
from tests.test_gpu_rules import check_score, score

pytestmark = pytest.mark.gpu
F32_MIN = float(torch.finfo(torch.float32).min)
LOW = [F32_MIN, -3.0e38, -2.4e38, -2.3e38, -1.0e38, -1.0e35, -1.1e30, -8.0e29, -1.0e25, -1.0e9]


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


def check(r, x, V, tok):
    for tau in (0.25, 0.7, 1.0):
        for entropy in (True, False):
            g = score(r, x, V, tok, tau, entropy)
            assert g["status"] == 0, (tau, entropy)
            check_score(g, x, r, V, tok, tau)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ids_left", ["all", "few"])
def test_low_logits_that_no_rule_touches(dtype, ids_left):
    """Most of the vocabulary suppressed by values far from the others', and with a mask
    that leaves two ids of it and the token."""
    rng = np.random.default_rng(45)
    values = [-1.0e8, -3.0e8, -1.0e9, -7.7e9, -1.0e10, -3.3e10, -1.0e12, -2.0e12, -1.0e20, -1.0e25,
              -8.0e29, -1.0e30]
    V, n = 20000, len(values)
    x = C.logits(rng, n, V, dtype)
    for i, low in enumerate(values):
        x[i, :19000] = low
    r = O.Rules()
    if ids_left == "few":
        mask = np.zeros((1, V // 32), np.uint32)
        for v in (70, 9000, 19500):
            mask[0, v // 32] |= np.uint32(1 << (v % 32))
        r = O.Rules(mask=mask, row_mask=np.zeros(n, np.int32))
    check(r, x, V, np.full(n, 19500))
