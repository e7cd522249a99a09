"""float32 rows in which more than 2^18 ids share one value, or one bin of values: a bin's mass, added up
over the blocks of a cluster, has more than 32 bits.  Tolerances: as in test_gpu_sampling.py."""

import numpy as np
import pytest
import torch

from oracle import sampling as O

from .test_gpu_sampling import DEV, check_drawn, close_lp, close_lq, exact_choice, run_sample, run_score, sampling_of

pytestmark = pytest.mark.gpu

# shares that fall between two of the equal ids, not next to a border
OPEN, POWER, USUAL = (1.0, 0, 1.0, 0.0), (0.25, 0, 0.8767123, 0.0), (0.8, 280001, 0.9312345, 0.001)


def row(kind, V, rng):
    if kind == "zeros":
        x = np.zeros(V)
    elif kind == "negative":                 # a padded row with one id ahead
        x = np.full(V, -3.0)
        x[rng.integers(V)] = 2.0
    elif kind == "close":                    # several values of one bin
        x = 20 + rng.integers(0, 4, V) * 2.0 ** -9
    elif kind == "masked":                   # most ids equal, the others out
        x = np.where(rng.random(V) < 0.05, -np.inf, 1.5)
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["zeros", "negative", "close", "masked"])
@pytest.mark.parametrize("V", [2 ** 18 + 1, 300000, 2 ** 20])
def test_many_equal_ids(V, kind):
    rng = np.random.default_rng(V)
    u = np.array([1e-300, 0.1, 0.3, 0.5, 0.9, 0.999, 1.0])
    x = row(kind, V, rng)
    ld = -(-V // 4) * 4
    d = torch.full((len(u), ld), float("nan"), device=DEV)
    d[:, :V] = torch.from_numpy(x).to(DEV)
    x = x.astype(np.float64)
    for choice in (OPEN, POWER, USUAL):
        t = O.truncate(x, *exact_choice(choice))
        s = sampling_of([choice])
        tok, out, status = run_sample(d, s, torch.from_numpy(u).to(DEV), V)
        assert status == 0
        given = np.array([t.order[0], t.order[t.n_kept // 2], t.order[t.n_kept - 1], t.order[-1]] + list(rng.integers(0, V, 3)))
        sc, status = run_score(d, s, torch.from_numpy(given.astype(np.int32)).to(DEV), V)
        assert status == 0
        h = O.entropy(x)
        for r in range(len(u)):
            check_drawn(t, int(tok[r]), u[r], V)
            assert close_lq(out[1, r], O.log_q(t, int(tok[r])), V) and close_lp(out[0, r], O.log_p0(x, int(tok[r])), V)
            # the last place that the cuts leave is a border
            place = O.place_of(t, int(given[r]))
            if abs(place - (t.n_kept - 1)) > 1 or choice == OPEN:
                assert close_lq(sc[1, r], O.log_q(t, int(given[r])), V), (choice, r, sc[1, r], O.log_q(t, int(given[r])))
            assert close_lp(sc[0, r], O.log_p0(x, int(given[r])), V)
            assert abs(out[2, r] - h) <= 1e-4 * h + 2e-6
