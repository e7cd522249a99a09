"""log p0 and the entropy of bfloat16 rows with many values around zero, which share a bin: p0 is the softmax at
temperature 1, whatever the temperature of q.

Tolerance.  Every e^l of the bin is added up to 2^-24, an average of float32 exponentials (2^-22) is around it:
1e-6, where test_gpu_sampling.py allows 3e-6.  The same inputs twice: the same bits."""

import numpy as np
import pytest
import torch

from oracle import sampling as O

from .test_gpu_sampling import DEV, close_lq, exact_choice, run_sample, run_score, sampling_of

pytestmark = pytest.mark.gpu


def row(kind, V, n, tau, rng):
    x = np.full(V, -np.inf) if kind != "others" else rng.normal(-4, 2, V)
    near = 2.0 ** -10 * max(tau, 1.0)
    ids = rng.permutation(V)[:n]
    if kind == "two":
        x[ids] = np.where(np.arange(n) % 2, 0.97, -0.97) * near
    else:
        x[ids] = rng.uniform(-1, 1, n) * near
    x[ids[0]] = 2.1 * near                   # the largest, outside the bin
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["two", "spread", "others"])
@pytest.mark.parametrize("tau", [1 / 128, 0.01, 0.02, 0.05, 0.3, 1.0, 4.0])
@pytest.mark.parametrize("V, n, copies", [(300, 251, 1), (300, 251, 400), (40000, 900, 2), (9000, 4, 1)])
def test_values_around_zero(V, n, copies, tau, kind):
    rng = np.random.default_rng(n + int(1000 * tau))
    x = torch.from_numpy(row(kind, V, n, tau, rng)).to(DEV)
    d = torch.full((copies, -(-V // 8) * 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    d[:, :V] = x.to(torch.bfloat16)
    x = d[0, :V].double().cpu().numpy()
    choice = (tau, 0, 1.0, 0.0)
    s = sampling_of([choice])
    u = torch.from_numpy(1.0 - rng.random(copies)).to(DEV)
    tok, out, status = run_sample(d, s, u, V)
    again = run_sample(d, s, u, V)
    assert status == 0 and np.array_equal(tok, again[0]) and np.array_equal(out, again[1])
    given = torch.full((copies,), int(np.argsort(-x)[n // 2]), dtype=torch.int32, device=DEV)
    sc, status = run_score(d, s, given, V)
    only, _ = run_score(d, s, given, V, entropy=False)
    assert status == 0 and np.array_equal(only[:2], sc[:2])
    t, h = O.truncate(x, *exact_choice(choice)), O.entropy(x)
    for r in range(copies):
        for got, id_ in ((out, int(tok[r])), (sc, int(given[0]))):
            want = O.log_p0(x, id_)
            assert abs(got[0, r] - want) <= 1e-6 * (1 + abs(want)), (got[0, r], want)
            assert close_lq(got[1, r], O.log_q(t, id_), V)
            assert abs(got[2, r] - h) <= 2e-6 * (1 + h), (got[2, r], h)
