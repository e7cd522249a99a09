"""Waits of a projection that run out: no output is wrong, each is the one of an undisturbed call or NaN, NaN where
copies were left out, and the next call is right."""

import time

import pytest
import torch

import mh_prefetch_subtree_gb300 as ps

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


# (rows, N, K, blocks of a tile, rows of x a tile, whether k is divided): one block a tile, a divided k, and pairs of
# blocks; K of 1024 is 16 steps, more than a ring holds, so that the first block makes no tile
CASES = [(50, 128 * 300, 1024, 1, 64, False), (300, 128 * 20, 1024, 1, 256, False), (600, 128 * 200 - 8, 1024, 2, 256, False),
         (900, 128 * 400, 1024, 2, 256, False), (34, 1000, 8192, 1, 64, True), (60, 400, 8192, 1, 64, True)]


def run(rows, N, K, dtype, residual, act="silu"):
    g = torch.Generator(device=DEV).manual_seed(rows + K)
    x = torch.randn(rows, K, device=DEV, generator=g).to(torch.bfloat16)
    w = (torch.randn(N, K, device=DEV, generator=g) / K ** 0.5).to(torch.bfloat16)
    r = torch.randn(rows, N, device=DEV, generator=g).to(dtype) if residual else None
    lin = ps.make_linear(w=w, act=act, bias=torch.randn(N, device=DEV, generator=g))
    want, got, after = (torch.full((rows, N), 7.0, dtype=dtype, device=DEV) for _ in range(3))
    ps.ps_linear_rows(lin, x, want, residual=r)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ps.ps_selftest_linear_wait(lin, x, got, residual=r)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    nan = torch.isnan(got)
    assert not torch.isnan(want).any() and torch.equal(got[~nan], want[~nan])
    ps.ps_linear_rows(lin, x, after, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(after, want)
    return nan


def first_blocks(rows, N, C, tile_rows):
    """The place in its order of each output's tile among those of the first block (or pair), or -1."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    n_cols, n_tiles = -(-rows // tile_rows), -(-N // (128 * C))
    step = min(n_cols * n_tiles, sms // C)
    unit = (torch.arange(N, device=DEV) // (128 * C))[None] * n_cols + (torch.arange(rows, device=DEV) // tile_rows)[:, None]
    return torch.where(unit % step == 0, unit // step, -1)


@pytest.mark.parametrize("rows, N, K, C, tile_rows, divided", CASES)
@pytest.mark.parametrize("dtype, residual", [(torch.bfloat16, False), (torch.float32, True)])
def test_lost_copies_give_nan(rows, N, K, C, tile_rows, divided, dtype, residual):
    nan = run(rows, N, K, dtype, residual)
    if divided:                                 # the first cluster has the first tile
        lost = (torch.arange(N, device=DEV) < 128).expand(rows, N)
    else:
        lost = first_blocks(rows, N, C, tile_rows) >= 0
    assert torch.equal(nan, lost)


@pytest.mark.parametrize("rows, N, C, tile_rows", [(40, 128 * 152 * 14, 1, 64), (600, 128 * 152 * 6, 2, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tiles_made_before_are_kept(rows, N, C, tile_rows, dtype):
    """One step a tile: those that the ring held are there, later ones of the first block are not."""
    nan = run(rows, N, 64, dtype, False)
    place = first_blocks(rows, N, C, tile_rows)
    assert int(place.max()) > 11
    assert not nan[place < 1].any() and nan[place > 10].all()
    # from some place on, all
    first = int(place[nan].min())
    assert torch.equal(nan, place >= first)
