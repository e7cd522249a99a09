"""Rows with many values on both sides of zero, equally far: a bin around zero is halved at zero, and what lies below
does not hold the zeros again.  Tolerances: as in test_gpu_sampling.py."""

import numpy as np
import pytest
import torch

from oracle import sampling as O

from .test_gpu_sampling import DEV, TYPES, check_drawn, close_lp, close_lq, eps_of, exact_choice, run_sample, run_score, sampling_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size, tau", [(0.012, 146.64177), (7.2e-5, 0.0755281), (3e-4, 1.0), (1e-38, 0.3), (0.4, 300.0)])
@pytest.mark.parametrize("V, n, negative_zeros", [(300, 400, False), (560, 30, False), (9000, 5, True), (560, 40, True)])
def test_symmetric_rows(V, n, negative_zeros, size, tau, dtype):
    rng = np.random.default_rng(V + n)
    steps = np.clip(np.round(rng.normal(0, 2, (n, V))), -6, 6)
    steps[:, 0], steps[:, 1], steps[:, 2] = 6, -6, 0
    x = steps * (size / 6)
    if negative_zeros:
        x = np.where((x == 0) & (rng.random((n, V)) < 0.5), -0.0, x)
    d = torch.full((n, -(-V // 8) * 8), float("nan"), dtype=TYPES[dtype], device=DEV)
    d[:, :V] = torch.from_numpy(x.astype(np.float32)).to(DEV).to(TYPES[dtype])
    x = d[:, :V].double().cpu().numpy()
    u = 1.0 - rng.random(n)
    for choice in ((tau, 0, 1.0, 0.0), (tau, 0, 0.8088308, 1e-4), (tau, V * 4 // 5, 1.0, 0.0), (tau, V * 4 // 5, 0.917, 0.0)):
        s = sampling_of([choice])
        tok, out, status = run_sample(d, s, torch.from_numpy(u).to(DEV), V)
        given = rng.integers(0, V, n).astype(np.int32)
        sc, status2 = run_score(d, s, torch.from_numpy(given).to(DEV), V)
        assert status == status2 == 0
        for r in range(0, n, max(1, n // 40)):
            t = O.truncate(x[r], *exact_choice(choice))
            if 1e-15 < t.margin < eps_of(V):
                continue
            check_drawn(t, int(tok[r]), u[r], V)
            for got, v in ((out, int(tok[r])), (sc, int(given[r]))):
                assert close_lq(got[1, r], O.log_q(t, v), V), (choice, r, got[1, r], O.log_q(t, v))
                assert close_lp(got[0, r], O.log_p0(x[r], v), V)
