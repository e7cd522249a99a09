"""The 4-bit head on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps
from oracle.rules import head_rows

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


def case(n, V, K, group, scale, zeros, seed=0, hidden_ld=None):
    g = torch.Generator().manual_seed(seed)
    h = torch.full((n, hidden_ld or K), float("nan"), dtype=torch.bfloat16)
    h[:, :K] = torch.randn(n, K, generator=g).to(torch.bfloat16)
    q = torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, generator=g)
    s = ((0.2 + torch.rand(V, K // group, generator=g)) / K ** 0.5).to(scale)
    z = torch.randint(0, 16, (V, K // group), dtype=torch.uint8, generator=g) if zeros else None
    return h, q, s, z


def run(h, q, s, z, group, dtype, ld=None, stream=None):
    V = q.shape[0]
    out = torch.full((h.shape[0], ld or -(-V // 8) * 8), 7.0, dtype=dtype, device=DEV)
    head = ps.make_head(q=q.to(DEV), scales=s.to(DEV), zeros=None if z is None else z.to(DEV),
                        group=group)
    ps.ps_head_rows(head, h.to(DEV), out, stream=stream)
    torch.cuda.synchronize()
    assert (out[:, V:] == 7.0).all()                      # the padding is not written
    return out.cpu()[:, :V]


def check(got, h, q, s, z, group):
    K = 2 * q.shape[1]
    want, size = head_rows(h[:, :K].double().numpy(), q.numpy(), s.double().numpy(),
                           None if z is None else z.numpy(), group)
    # exact products; a float32 sum loses at most one unit (2^-23, also where it
    # truncates) of the running magnitude at each of its steps: at most K within a
    # dot product, whatever its order, and a scaling and an addition a group
    bound = (K + 2 * K / min(group, 128)) * 2.0 ** -23 * size
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)     # half a unit of 8 significant bits
    err = np.abs(got.double().numpy() - want)
    assert (err <= bound).all(), (err - bound).max()
    # and as a whole far closer: errors of single steps do not line up
    if got.dtype == torch.float32 and want.size >= 64:
        assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(want)


SHAPES = [  # rows, V, K, group
    (1, 1, 32, 32), (1, 17, 64, 64), (3, 100, 128, 128), (8, 1000, 96, 32), (9, 333, 192, 64),
    (16, 515, 256, 256), (1, 4097, 1024, 128), (5, 2050, 2080, 32), (17, 1040, 512, 64),
    (33, 777, 640, 128), (64, 1500, 1024, 32), (65, 300, 384, 128), (130, 129, 256, 64),
    # long rows of hidden states, 17 rows and more
    (40, 515, 2048, 128), (64, 1111, 4096, 128), (50, 200, 4608, 64), (100, 130, 4096, 512),
]


@pytest.mark.parametrize("n,V,K,group", SHAPES)
@pytest.mark.parametrize("scale,zeros,dtype", [
    (torch.bfloat16, True, torch.float32), (torch.float32, False, torch.float32),
    (torch.float32, True, torch.bfloat16)])
def test_head_rows(n, V, K, group, scale, zeros, dtype):
    h, q, s, z = case(n, V, K, group, scale, zeros, seed=n + V)
    check(run(h, q, s, z, group, dtype), h, q, s, z, group)


@pytest.mark.parametrize("n", [2, 20])
@pytest.mark.parametrize("K,group", [(16384, 128), (8192 + 4096 + 128, 128), (8192 + 32, 32),
                                     (24576, 8192)])
def test_wide_hidden_states(n, K, group):
    h, q, s, z = case(n, 200, K, group, torch.float32, True, seed=K)
    check(run(h, q, s, z, group, torch.float32), h, q, s, z, group)


def test_many_vocabulary_rows():
    for n in (1, 12, 40):
        h, q, s, z = case(n, 60001, 256, 64, torch.bfloat16, True, seed=5)
        check(run(h, q, s, z, 64, torch.bfloat16, ld=60032), h, q, s, z, 64)


@pytest.mark.parametrize("n", [4, 24])
def test_strided_hidden_and_extremes(n):
    h, q, s, z = case(n, 257, 128, 64, torch.float32, True, seed=6, hidden_ld=136)
    q[:64], q[64:128] = 0, 255
    z[:32], z[32:64] = 0, 15
    s[3] = 0.0
    s[4] = -s[4]
    check(run(h, q, s, z, 64, torch.float32), h, q, s, z, 64)
    h[1, :128] = 0
    assert (run(h, q, s, z, 64, torch.float32)[1] == 0).all()


@pytest.mark.parametrize("n", [3, 40])
def test_a_row_does_not_reach_the_others(n):
    """A NaN or an infinity in one hidden row, or in one vocabulary row's scale,
    stays there."""
    h, q, s, z = case(n, 100, 128, 32, torch.float32, True, seed=7)
    want = run(h, q, s, z, 32, torch.float32)
    h[1, 5] = float("nan")
    s[50, 1] = float("inf")
    got = run(h, q, s, z, 32, torch.float32)
    assert torch.isnan(got[1]).all()
    rest, cols = [i for i in range(n) if i != 1], [i for i in range(100) if i != 50]
    assert torch.equal(got[rest][:, cols], want[rest][:, cols])
    assert not torch.isfinite(got[rest][:, 50]).any()


def test_same_bits_again_and_on_another_stream():
    for n in (1, 16, 50):
        h, q, s, z = case(n, 5001, 512, 128, torch.bfloat16, True, seed=8)
        a = run(h, q, s, z, 128, torch.float32)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            b = run(h, q, s, z, 128, torch.float32)
        assert torch.equal(a, b)
        # a row's result does not depend on the rows next to it within a call of the same size
        p = torch.randperm(n)
        assert torch.equal(run(h[p].contiguous(), q, s, z, 128, torch.float32), a[p])


# heads large enough for the tensor memory kernel: one block's hidden rows and two
# blocks', 32 and 64 at a time, several times, parts of a copy and of a tile left over
LARGE = [(17, 40000, 256, 64), (33, 40009, 288, 32), (32, 41111, 640, 128), (64, 39999, 1024, 512),
         (130, 39000, 320, 64), (64, 39425, 1120, 32), (50, 40321, 1216, 64), (20, 40000, 2304, 256),
         (70, 39900, 2112, 64)]


@pytest.mark.parametrize("n,V,K,group", LARGE)
@pytest.mark.parametrize("scale,zeros,dtype", [
    (torch.bfloat16, True, torch.float32), (torch.float32, False, torch.bfloat16)])
def test_large_heads(n, V, K, group, scale, zeros, dtype):
    h, q, s, z = case(n, V, K, group, scale, zeros, seed=n + V, hidden_ld=K + 8)
    check(run(h, q, s, z, group, dtype), h, q, s, z, group)


@pytest.mark.parametrize("n,K", [(40, 512), (40, 1280)])
def test_large_heads_keep_rows_apart(n, K):
    """Extremes, a NaN and an infinity of one row stay there; the same bits again,
    for rows in another order, and on another stream."""
    V = 39300
    h, q, s, z = case(n, V, K, 64, torch.float32, True, seed=9)
    q[:64], q[64:128] = 0, 255
    z[:32], z[32:64] = 0, 15
    s[3], s[4] = 0.0, -s[4]
    h[2] *= 2.0 ** 100
    h[3] *= 2.0 ** -100
    h[4] = 0
    want = run(h, q, s, z, 64, torch.float32)
    check(want, h, q, s, z, 64)
    assert (want[4] == 0).all()
    p = torch.randperm(n, generator=torch.Generator().manual_seed(1))
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        assert torch.equal(run(h[p].contiguous(), q, s, z, 64, torch.float32, stream=st), want[p])
    h[1, 5], s[50, 1], h[7, K - 1] = float("nan"), float("inf"), float("-inf")
    got = run(h, q, s, z, 64, torch.float32)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[7]).any()
    rest = [i for i in range(n) if i not in (1, 7)]
    cols = [i for i in range(V) if i != 50]
    assert torch.equal(got[rest][:, cols], want[rest][:, cols])
    assert not torch.isfinite(got[rest][:, 50]).any()


def test_more_groups_of_rows_than_blocks():
    """Each block takes several groups of hidden rows, one after another."""
    n, V, K, group = 5003, 39001, 1056, 32
    h, q, s, z = case(n, V, K, group, torch.bfloat16, True, seed=10)
    out = torch.empty((n, 39008), dtype=torch.bfloat16, device=DEV)
    head = ps.make_head(q=q.to(DEV), scales=s.to(DEV), zeros=z.to(DEV), group=group)
    ps.ps_head_rows(head, h.to(DEV), out)
    rows = [0, 31, 63, 64, 2500, 4863, 4864, 4900, 4991, 4992, 5002]
    check(out[rows].cpu()[:, :V], h[rows], q, s, z, group)


def test_no_rows():
    h, q, s, z = case(0, 40, 32, 32, torch.float32, False)
    assert run(h, q, s, z, 32, torch.float32).shape == (0, 40)
