"""Cuts and numbers that divide equal ids exactly: of n equal ids, p = j / n keeps j and u = k / j draws the kth of them,
for any value, temperature and type, and however the row is divided.  These are whole numbers, without a tolerance."""

import numpy as np
import pytest
import torch

from .test_gpu_sampling import DEV, TYPES, run_sample, run_score, sampling_of

pytestmark = pytest.mark.gpu


def rows(V, n, values, dtype, rng):
    """Rows with n equal largest ids; the others are out, or far below."""
    ids = np.stack([np.sort(rng.permutation(V)[:n]) for _ in values])
    x = np.full((len(values), -(-V // 8) * 8), -np.inf, np.float32)
    x[::2] = np.minimum(values[::2] - 4000, -3e4)[:, None]
    x[:, V:] = np.nan
    np.put_along_axis(x, ids, values[:, None].astype(np.float32), 1)
    return torch.from_numpy(x).to(DEV).to(TYPES[dtype]), ids


VALUES = np.array([0.0, 1.0, 40.003, -7.1, 1e-3, -1e-3, 2.0 ** -12, 0.37, 59.0, -300.25, 9470.181640625, 3e5, -1e-30, 88.0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [0.01, 0.25, 1.0, 2.2153697, 30.0, 400.0])
@pytest.mark.parametrize("V, n", [(2, 2), (40, 8), (700, 64), (5000, 512), (50000, 4096)])
def test_equal_ids_are_divided(V, n, tau, dtype):
    rng = np.random.default_rng(V + int(100 * tau))
    values = np.tile(VALUES, 4 if V < 50000 else 1)
    x, ids = rows(V, n, values, dtype, rng)
    at = np.arange(len(values))
    for part in (0.5, 1.0, 0.25 if n > 2 else 0.5, 3 / 8 if n > 2 else 1.0):
        j = int(n * part)
        s = sampling_of([(tau, 0, part, 0.0)])
        k = rng.integers(1, j + 1, len(values))
        k[::3] = j
        # the least and the greatest number that draw the kth, where they are not rounded
        for u in (k / j, (k - 1) / j + 1e-5 / n):
            if not j & (j - 1) or (u == 1).all():
                tok, out, status = run_sample(x, s, torch.from_numpy(u).to(DEV), V)
                assert status == 0 and np.array_equal(tok, ids[at, k - 1]), (part, np.nonzero(tok != ids[at, k - 1]))
                assert np.abs(out[1] + np.log(j)).max() <= 1e-8 * (1 + np.log(j))
        last, st = run_score(x, s, torch.from_numpy(ids[:, j - 1].astype(np.int32)).to(DEV), V)
        assert st == 0 and np.abs(last[1] + np.log(j)).max() <= 1e-8 * (1 + np.log(j))
        if j < n:
            out_of, st = run_score(x, s, torch.from_numpy(ids[:, j].astype(np.int32)).to(DEV), V)
            assert st == 0 and np.all(np.isneginf(out_of[1])), np.nonzero(~np.isneginf(out_of[1]))
        # a top-k before it
        s = sampling_of([(tau, j, 0.5, 0.0)])
        if j % 2 == 0:
            tok, out, _ = run_sample(x, s, torch.ones(len(values), dtype=torch.float64, device=DEV), V)
            assert np.array_equal(tok, ids[at, j // 2 - 1])
