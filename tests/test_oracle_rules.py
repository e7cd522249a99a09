"""The rules' and the head's oracle against hand-worked values (CPU)."""

import numpy as np

from oracle.rules import Rules, head_rows, logprobs, process_row, process_rows


def test_penalties_by_hand():
    x = np.array([2.0, -2.0, 0.0, 4.0, 1.0])
    y, size = process_row(x, history=[0, 1, 3, 3, 3], prompt=2, repetition=2.0, frequency=0.5,
                          presence=0.25, bias=[(1, 1.0), (4, -3.0)], mask=None)
    # 0: prompt only, 2/2; 1: prompt only, -2*2 + 1; 3: three times generated
    assert y.tolist() == [1.0, -3.0, 0.0, 4.0 / 2 - 1.5 - 0.25, -2.0]
    assert size.tolist() == [1.0, 5.0, 0.0, 3.75, 4.0]


def test_mask_wins_over_everything():
    x = np.array([np.nan, 1.0, np.inf, 2.0])
    y, _ = process_row(x, history=[0, 2], prompt=0, repetition=1.5, frequency=0.0, presence=0.0,
                       bias=[(2, 5.0)], mask=np.array([0b1010], np.uint32))
    assert y.tolist() == [-np.inf, 1.0, -np.inf, 2.0]


def test_rows_see_their_prefix_only():
    r = Rules(seq_begin=np.array([0, 3]), seq_tokens=np.array([1, 1, 2]),
              frequency=np.array([1.0], np.float32), row_seq=np.zeros(4, np.int32),
              row_len=np.arange(4, dtype=np.int32))
    y, _ = process_rows(np.zeros((4, 3)), r)
    assert y.tolist() == [[0, 0, 0], [0, -1, 0], [0, -2, 0], [0, -2, -1]]


def test_logprobs_against_the_plain_softmax():
    rng = np.random.default_rng(5)
    x = rng.normal(0, 2, (6, 50))
    x[0, 3:9] = -np.inf
    tok = rng.integers(0, 50, 6)
    tok[0] = 4
    lp0, lq, ent = logprobs(x, tok, 0.5)
    for i in range(6):
        p = np.exp(x[i] - x[i].max())
        p /= p.sum()
        q = np.exp(2 * (x[i] - x[i].max()))
        q /= q.sum()
        if i == 0:
            assert lp0[i] == lq[i] == -np.inf
        else:
            assert abs(lp0[i] - np.log(p[tok[i]])) < 1e-12
            assert abs(lq[i] - np.log(q[tok[i]])) < 1e-12
        nz = p > 0
        assert abs(ent[i] + (p[nz] * np.log(p[nz])).sum()) < 1e-12


def test_empty_and_nonfinite_rows_are_nan():
    x = np.array([[-np.inf, -np.inf], [0.0, np.nan], [0.0, np.inf], [0.0, -np.inf]])
    lp0, lq, ent = logprobs(x, [0, 0, 0, 0], 1.0)
    assert np.isnan(lp0[:3]).all() and np.isnan(lq[:3]).all() and np.isnan(ent[:3]).all()
    assert lp0[3] == 0.0 and ent[3] == 0.0


def test_head_by_hand():
    # one vocabulary row of 32 elements: q = 9, zero 8 everywhere, but element 1 is 15
    q = np.full((1, 16), 0x99, np.uint8)
    q[0, 0] = 0xF9
    h = np.zeros((2, 32))
    h[0, 0], h[0, 1], h[1, 31] = 2.0, 3.0, -1.0
    y, size = head_rows(h, q, np.array([[0.5]]), None, 32)
    assert y.tolist() == [[0.5 * (2 + 3 * 7)], [-0.5]]
    assert size.tolist() == [[11.5], [0.5]]
    y, _ = head_rows(h, q, np.array([[0.5]]), np.array([[15]], np.uint8), 32)
    assert y.tolist() == [[0.5 * (2 * -6)], [0.5 * 6]]
