"""Warps that keep the reference of the row before, at both ends of the range in which
they may: the ids of one warp far below its reference, those of another as far above, so
that the references differ by more than the exponents of the sums."""

import numpy as np
import pytest
import torch

from oracle import rules as O
from tests import rules_cases as C
from tests.test_gpu_rules import check_score, score

pytestmark = pytest.mark.gpu
WARPS = 12


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype,V,ids", [("bf16", 24576, 11), ("f32", 12288, 10)])
@pytest.mark.parametrize("tau", [1.0, 0.5, 0.3, 0.25, 0.125])
@pytest.mark.parametrize("low,high", [(-59, 63), (-44, 48), (-46, 50), (-30, 60), (-20, 40)])
def test_references_far_apart(dtype, V, ids, tau, low, high):
    g, ln2 = 1.0 / tau, np.log(2.0)
    # a warp has 2^ids ids of the row, in blocks of 32 that skew from lane to lane
    b = np.arange(V) // 32
    warp = (b % WARPS - b // WARPS) % WARPS
    a_ids, b_ids = warp == 0, warp == 1
    # log2 of the sums of 2^(g y): `low` in warp 0, `high` in warp 1, whose ids are 2^-6
    # of warp 0's in mass
    up, down, less = -(low - ids) / g * ln2, (high - ids) / g * ln2, 6.0 / g * ln2
    rows = np.full((3, V), -300.0)
    rows[:, 64 * WARPS] = 0.0                               # a token with some mass
    rows[0, a_ids], rows[0, b_ids] = up + 150.0, -200.0     # references to start from
    rows[1, a_ids], rows[1, b_ids] = up, -less - down       # as the next row will find them
    rows[2, a_ids], rows[2, b_ids] = 0.0, -less
    # three rows a block, one after the other
    x = torch.from_numpy(np.tile(rows, (152, 1))).to(C.NP[dtype])
    tok = np.full(len(x), 64 * WARPS)
    gpu = score(O.Rules(), x, V, tok, tau, entropy=False)
    assert gpu["status"] == 0
    few = slice(300, 306)
    check_score({k: v if k in ("status", "entropy") else v[few] for k, v in gpu.items()},
                x[few], O.Rules(), V, tok[few], tau)
    for k in ("lp0", "lq"):
        assert np.array_equal(gpu[k], np.tile(gpu[k][300:303], 152))
