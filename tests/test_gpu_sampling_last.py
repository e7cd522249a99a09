"""Draws whose number is 1, or next to it: they end in the row's tail, where a bin of several values may have a
mass although each of its ids, rounded by itself, has none.  Every row has a token all the same.
Tolerances: as in test_gpu_sampling.py; an id of the tail weighs less than they allow."""

import numpy as np
import pytest
import torch

from oracle import sampling as O

from .test_gpu_sampling import DEV, TYPES, check_drawn, close_lp, close_lq, eps_of, exact_choice, run_sample, sampling_of

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(d, V, choice, u):
    x = d[:, :V].double().cpu().numpy()
    tok, out, status = run_sample(d, sampling_of([choice]), torch.from_numpy(u).to(DEV), V)
    assert status == 0
    assert ((tok >= 0) & (tok < V)).all(), tok
    for r in range(len(u)):
        t = O.truncate(x[r], *exact_choice(choice))
        if 1e-15 < t.margin < eps_of(V):        # whose cut is a border in itself
            continue
        check_drawn(t, int(tok[r]), u[r], V)
        assert close_lq(out[1, r], O.log_q(t, int(tok[r])), V), (r, out[1, r], O.log_q(t, int(tok[r])))
        assert close_lp(out[0, r], O.log_p0(x[r], int(tok[r])), V)


@pytest.mark.parametrize("dtype, M, tau, tail", [("f32", 10.0, 1.0, [-21.95, -21.96]), ("f32", 10.0, 1.0, [-21.95] * 2),
                                                 ("bf16", 32.0, 1.003591, [0.0, 0.0]), ("f32", 32.0, 1.003591, [0.0, 0.0])])
@pytest.mark.parametrize("V", [3, 9000])
def test_a_tail_of_ids_without_a_mass(V, dtype, M, tau, tail):
    """About half a unit of mass each: the bin has one unit, its ids round to none."""
    n, at = 4, [V - 1, 0, V // 2]
    d = torch.full((n, -(-V // 8) * 8), -INF, dtype=TYPES[dtype], device=DEV)
    for i, v in zip(at, [M] + tail):
        d[:, i] = v
    for choice in ((tau, 0, 1.0, 0.0), (tau, 0, 1.0 - 2.0 ** -24, 0.0), (tau, 3, 1.0, 0.0), (tau, 0, 1.0, 1e-30)):
        check(d, V, choice, np.array([1.0, 1.0 - 2.0 ** -53, 0.5, 1.0]))


@pytest.mark.parametrize("V, n", [(5000, 3), (700, 400)])
def test_many_ids_of_a_tail_without_a_mass(V, n):
    """More than are listed, of one value and of several."""
    rng = np.random.default_rng(V)
    one = np.full(V, -21.95)
    some = rng.choice([-21.95, -21.951, -21.96], V)
    for tail in (one, some):
        tail[V // 3] = 10.0
        d = torch.from_numpy(np.tile(tail.astype(np.float32), (n, 1))).to(DEV)
        check(d, V, (1.0, 0, 1.0, 0.0), np.resize([1.0, 1.0 - 2.0 ** -53, 1.0 - 2.0 ** -46], n))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V, tau, n", [(1000, 0.25, 320), (4097, 0.5, 60), (16384, 0.25, 60), (50021, 0.7, 60)])
def test_normal_rows(V, tau, n, dtype):
    g = torch.Generator(device=DEV).manual_seed(V)
    d = (3 * torch.randn(n, -(-V // 8) * 8, device=DEV, generator=g)).to(TYPES[dtype])
    u = np.resize([1.0, 1.0 - 2.0 ** -53, 1.0 - 2.0 ** -46, 1.0 - 2.0 ** -40], n)
    check(d, V, (tau, 0, 1.0, 0.0), u)
    check(d, V, (tau, 0, 1.0 - 2.0 ** -24, 0.0), u)
