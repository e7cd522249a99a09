"""The mass of a float32 row's bin is the sum of its elements' weights, each rounded to 28 bits of the weight of the
bin's largest value.

Tolerance.  The rows hold one largest id and many equal ones at the lower end of a bin, whose weight is 0.37 of the
bin's largest and lies 0.14 to 0.18 below a multiple of 2^-28: rounded to nearest it is off by 0.18 2^-28 / 0.37 =
1.8e-9 of itself.  The exponentials of the bin's largest value and of the weight add 2^-31 each, the logarithm 2^-30:
3.7e-9 in all.  Rounded down the weight would be off by 8.3e-9."""

import numpy as np
import pytest
import torch

from .test_gpu_sampling import DEV, run_score, sampling_of

pytestmark = pytest.mark.gpu
M, TAU = 40.25, 0.25


def values(n):
    """Float32 values from 40 on whose weight, relative to the largest below 40.25, is as said."""
    x = (40 + np.arange(6000) * 2.0 ** -18).astype(np.float64)
    ref = float(np.nextafter(np.float32(40.25), np.float32(0)))
    part = np.exp((x - ref) / TAU) * 2.0 ** 28 % 1.0
    x = x[(part > 0.82) & (part < 0.86)]
    return x[np.linspace(0, len(x) - 1, n).astype(int)]


@pytest.mark.parametrize("copies", [1, 30])
def test_weights_are_rounded_to_nearest(copies):
    V, xs = 100001, np.repeat(values(12), copies)
    d = torch.full((len(xs), -(-V // 4) * 4), float("nan"), device=DEV)
    d[:, :V] = torch.from_numpy(xs).to(DEV, torch.float32)[:, None]
    d[:, 77] = M
    tok = torch.arange(100, 100 + len(xs), dtype=torch.int32, device=DEV)
    out, status = run_score(d, sampling_of([(TAU, 0, 1.0, 0.0)]), tok, V, entropy=False)
    y = (xs - M) / TAU
    assert status == 0 and np.abs(out[1] - (y - np.log1p((V - 1) * np.exp(y)))).max() <= 4e-9
