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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rho", [0.8, 1.0, 1.3])
def test_lowest_logits_of_seen_ids(dtype, rho):
    rng = np.random.default_rng(41)
    V, n = 9001, len(LOW)
    ids = rng.choice(V, 24, replace=False)
    x = C.logits(rng, n, V, dtype)
    lowest = float(torch.finfo(C.NP[dtype]).min)
    for i, low in enumerate(LOW):
        x[i, torch.from_numpy(ids[:20])] = max(low, lowest)
    r = O.Rules(seq_begin=np.array([0, 24]), seq_tokens=ids.astype(np.int32),
                repetition=np.array([rho], np.float32), frequency=np.array([0.25], np.float32),
                row_seq=np.zeros(n, np.int32))
    tok = rng.integers(0, V, n)
    tok[np.isin(tok, ids[:20])] = ids[20]                 # a token with some mass
    check(r, x, V, tok)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lowest_biases(dtype):
    rng = np.random.default_rng(42)
    V, n = 5003, len(LOW)
    ids = np.sort(rng.choice(V, (n, 30), replace=True), 1)
    ids = [np.unique(row) for row in ids]
    r = O.Rules(bias_begin=np.concatenate([[0], np.cumsum([len(k) for k in ids])]),
                bias_ids=np.concatenate(ids).astype(np.int32),
                bias_values=np.concatenate([np.full(len(k), v) for k, v in zip(ids, LOW)]).astype(np.float32))
    x = C.logits(rng, n, V, dtype)
    tok = np.array([int(np.setdiff1d(np.arange(V), k)[i * 7]) for i, k in enumerate(ids)])
    check(r, x, V, tok)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_lowest_logits(dtype):
    """Thousands of seen ids, most of them suppressed."""
    rng = np.random.default_rng(43)
    V, n = 4000, len(LOW)
    ids = rng.permutation(V)[:3600]
    x = C.logits(rng, n, V, dtype)
    lowest = float(torch.finfo(C.NP[dtype]).min)
    for i, low in enumerate(LOW):
        x[i, torch.from_numpy(ids[:3000])] = max(low, lowest)
    r = O.Rules(seq_begin=np.array([0, 3600]), seq_tokens=ids.astype(np.int32),
                presence=np.array([0.5], np.float32), row_seq=np.zeros(n, np.int32))
    check(r, x, V, ids[3100 + np.arange(n)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lowest_logit_alone_among_masked_ones(dtype):
    """The mask leaves the token and, far from it, one suppressed id that was seen."""
    rng = np.random.default_rng(44)
    V, n = 20000, 2 * len(LOW)
    x = C.logits(rng, n, V, dtype)
    seen, tok = 137, 16001
    lowest = float(torch.finfo(C.NP[dtype]).min)
    for i in range(n):
        x[i, seen] = max(LOW[i // 2], lowest)
    mask = np.zeros((2, V // 32), np.uint32)
    for v in (seen, tok, tok + 40):
        mask[0, v // 32] |= np.uint32(1 << (v % 32))
    mask[1] = mask[0]
    mask[1, 100:120] = 0xFFFFFFFF
    r = O.Rules(seq_begin=np.array([0, 1]), seq_tokens=np.array([seen], np.int32),
                repetition=np.array([1.0], np.float32), row_seq=np.zeros(n, np.int32),
                mask=mask, row_mask=(np.arange(n) % 2).astype(np.int32))
    check(r, x, V, np.full(n, tok))
