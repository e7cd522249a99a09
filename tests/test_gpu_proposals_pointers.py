"""Arrays that do not lie on their elements' boundaries are refused by draws and scores under truncation."""

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

from .test_gpu_sampling import DEV, batch_of, sampling_of

pytestmark = pytest.mark.gpu


def test_misaligned_arrays():
    x = torch.zeros(2, 64, device=DEV)
    s, L = sampling_of([(1.0, 0, 1.0, 0.0)]), ps.lib()
    space = torch.zeros(64, dtype=torch.float64, device=DEV)
    space[:4] = 0.5
    tok = torch.zeros(8, dtype=torch.int32, device=DEV)
    index = torch.zeros(4, dtype=torch.int64, device=DEV)
    p = space.data_ptr()
    arg = [s, 64, 1, 2, x.data_ptr(), 64, p, tok.data_ptr(), p + 64, p + 128, p + 192, p + 256, None]
    assert L.ps_sample_rows(*arg) == 0
    for i, by in ((6, 4), (7, 2), (8, 4), (9, 4), (10, 4), (11, 2)):
        a = list(arg)
        a[i] += by
        assert L.ps_sample_rows(*a) == 1, i
    batch = batch_of(x, tok[:2], 64, row_index=index[:2])
    arg = [batch, s, p + 64, p + 128, p + 192, p + 256, None]
    assert L.ps_score_rows_truncated(*arg) == 0
    for i, by in ((2, 4), (3, 4), (4, 4), (5, 2)):
        a = list(arg)
        a[i] += by
        assert L.ps_score_rows_truncated(*a) == 1, i
    for name, by in (("tokens", 2), ("row_index", 4)):
        batch = batch_of(x, tok[:2], 64, row_index=index[:2])
        setattr(batch, name, getattr(batch, name) + by)
        assert L.ps_score_rows_truncated(batch, s, *arg[2:]) == 1, name
    torch.cuda.synchronize()
