"""Blocks that walk down many rows and from one slice of the vocabulary to the next:
histories that grow by 0 to 7 tokens a row and pass the places where a block changes how
it keeps them, masks wide and narrow that come again down the rows, and hundreds of
biases.  The expected rows are formed here a row at a time, with arrays over the
vocabulary; a few of them are checked against the oracle's id-by-id form."""

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps
from oracle import rules as O
from tests import gpu_harness as H
from tests import rules_cases as C

DEV = torch.device("cuda:0")
V = 50021                       # words of a mask row: 1564, a multiple of 4


def setup_module(module):
    if torch.cuda.is_available():
        import __graft_entry__
        __graft_entry__.build()


def one_row(x, r, i):
    """(processed float64 row, magnitude of its rounding errors) of row i."""
    s, n = int(r.row_seq[i]), int(r.row_len[i])
    b = int(r.seq_begin[s])
    hist, prompt = r.seq_tokens[b:b + n], int(r.seq_prompt[s])
    y = x.astype(np.float64).copy()
    seen = np.unique(hist)
    rho, f, p = (float(a[s]) for a in (r.repetition, r.frequency, r.presence))
    y[seen] = np.where(y[seen] > 0, y[seen] / rho, y[seen] * rho)
    size = np.abs(y)
    ids, c = np.unique(hist[min(prompt, n):], return_counts=True)
    y[ids] += -f * c - p
    size[ids] += abs(f) * c + abs(p)
    b, e = int(r.bias_begin[s]), int(r.bias_begin[s + 1])
    y[r.bias_ids[b:e]] += r.bias_values[b:e]
    size[r.bias_ids[b:e]] += np.abs(r.bias_values[b:e])
    m = int(r.row_mask[i])
    if m >= 0:
        bits = np.unpackbits(r.mask[m].view(np.uint8), bitorder="little")[:x.shape[0]]
        y[bits == 0] = -np.inf
    return y, size


def logprobs(y, t, tau):
    """(lp0, lq, entropy) of one row as in the oracle, with one exponential a logit."""
    top = y.max()
    d = y - top
    e = np.exp(d)
    z = e.sum()

    def logp(g):
        if np.isneginf(y[t]):
            return -np.inf
        w = np.exp(g * (np.delete(y, t) - y[t])) if y[t] == top else None
        if w is not None:
            return -np.log1p(w.sum())
        return g * d[t] - np.log(np.exp(g * d).sum())

    ok = e > 0
    return logp(1.0), logp(1.0 / tau), np.log(z) - (e[ok] * d[ok]).sum() / z


def case(seed, dtype, rows_each=240):
    """Five sequences: histories that pass 96 and 896 touched ids of a patching warp as
    they grow (a slice is a third of the vocabulary here, for float32 a fifth, a warp's
    share of it a fourth), one that begins far past them, one that begins empty, and one
    of common tokens."""
    rng = np.random.default_rng(seed)
    shares = 4 * (3 if dtype == "bf16" else 5)
    starts = [96 * shares - 250, 896 * shares - 450, 1500 * shares, 0, 3000]
    hists, lens = [], []
    for k, start in enumerate(starts):
        grow = rng.integers(0, 8, rows_each)               # 7 is more than is handed on one by one
        grow[rng.random(rows_each) < 0.3] = 1
        n = start + np.concatenate([[0], np.cumsum(grow)[:-1]])
        n[rows_each // 2] = max(0, n[rows_each // 2] - 40)  # and once back
        if k < 3:                                          # all different
            toks = rng.permutation(V)[:start + 8 * rows_each]
        else:
            toks = np.minimum(V - 1, (rng.random(start + 8 * rows_each) ** -0.9).astype(np.int64) * (1 + k % 2))
        hists.append(toks)
        lens.append(n)
    begin = np.concatenate([[0], np.cumsum([len(h) for h in hists])]).astype(np.int64)
    n_seq, n_rows = len(starts), len(starts) * rows_each
    n_bias = [0, 30, 1500, 700, 4000]
    bias = [np.sort(rng.choice(V, k, replace=False)) for k in n_bias]
    words = V // 32 + 1
    bits = np.zeros((8, words * 32), bool)
    bits[0] = rng.random(words * 32) < 0.9
    bits[1] = rng.random(words * 32) < 0.5
    bits[2] = rng.random(words * 32) < 0.03
    bits[3, rng.choice(V, 150, replace=False)] = True
    bits[4, rng.choice(V, 12, replace=False)] = True
    bits[5, [0, V - 1]] = True
    bits[6, 20000] = True
    bits[7, :900] = True                                   # all in the first segment
    mask = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)
    r = O.Rules(
        seq_begin=begin, seq_tokens=np.concatenate(hists).astype(np.int32),
        seq_prompt=np.array([1000, 10000, 10 ** 6, 0, 2900], np.int32),
        repetition=np.array([1.2, 0.9, 1.1, 1.3, 1.0], np.float32),
        frequency=np.array([0.3, 0.0, 0.2, 0.01, -0.05], np.float32),
        presence=np.array([0.4, 0.5, 0.0, -0.3, 0.2], np.float32),
        bias_begin=np.concatenate([[0], np.cumsum(n_bias)]).astype(np.int64),
        bias_ids=np.concatenate(bias).astype(np.int32),
        bias_values=rng.normal(0, 2, sum(n_bias)).astype(np.float32),
        mask=mask, row_seq=np.repeat(np.arange(n_seq), rows_each).astype(np.int32),
        row_len=np.concatenate(lens).astype(np.int32),
        row_mask=(np.arange(n_rows) % 10 - 2).clip(-1).astype(np.int32))
    # the other half of each sequence: one mask for many rows on end
    long_run = np.arange(n_rows) % rows_each >= rows_each // 2
    r.row_mask[long_run] = (np.arange(n_rows)[long_run] // 40 % 9) - 1
    return rng, r, n_rows


def tokens(rng, r, n_rows):
    tok = rng.integers(0, V, n_rows)
    for i in range(n_rows):
        m, kind = int(r.row_mask[i]), rng.integers(0, 3)
        if kind == 0 and r.row_len[i] > 0:                  # the last one of the history
            tok[i] = r.seq_tokens[r.seq_begin[r.row_seq[i]] + r.row_len[i] - 1]
        elif kind == 1 and m >= 0:                          # one that is allowed
            bits = np.unpackbits(r.mask[m].view(np.uint8), bitorder="little")[:V]
            tok[i] = rng.choice(np.nonzero(bits)[0])
    return tok


def test_the_row_form_is_the_oracles():
    rng, r, n_rows = case(1, "bf16", rows_each=4)
    x = rng.normal(0, 3, (n_rows, V))
    rows = [0, 5, 10, 14, 19]
    sub = O.Rules(**{**vars(r), "row_seq": r.row_seq[rows], "row_len": r.row_len[rows],
                     "row_mask": r.row_mask[rows]})
    want, size = O.process_rows(x[rows], sub)
    tok = tokens(rng, r, n_rows)
    lp0, lq, ent = O.logprobs(want, tok[rows], 0.25)
    for k, i in enumerate(rows):
        y, s = one_row(x[i], r, i)
        assert np.allclose(y, want[k], rtol=1e-14, atol=0) and np.allclose(s, size[k], rtol=1e-14, atol=0)
        assert np.allclose(logprobs(y, tok[i], 0.25), (lp0[k], lq[k], ent[k]), rtol=1e-10, atol=1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seed", [1, 2])
def test_process_walks(dtype, seed):
    rng, r, n_rows = case(seed, dtype)
    x = C.logits(rng, n_rows, V, dtype, ld=50048)
    rules, xd = C.device_rules(r, DEV), x.to(DEV)
    out, st = torch.full_like(xd, 7.0), torch.zeros(1, dtype=torch.int32, device=DEV)
    ps.ps_process_rows(rules, xd, out, st, V=V)
    again = torch.full_like(xd, 7.0)
    ps.ps_process_rows(rules, xd, again, st, V=V)
    ps.ps_process_rows(rules, xd, xd, st, V=V)              # in place
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(out, again) and torch.equal(out[:, :V], xd[:, :V])
    assert (out[:, V:] == 7.0).all()
    got, xs = out.cpu(), x[:, :V]
    for i in range(n_rows):
        want, size = one_row(xs[i].double().numpy(), r, i)
        g = got[i, :V].double().numpy()
        inf = np.isinf(want)
        assert np.array_equal(g[inf], want[inf]), i
        ok = ~inf
        assert (np.abs(g[ok] - want[ok]) <= C.process_bound(want[ok], size[ok], dtype)).all(), i


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [0.25, 0.7])
def test_score_walks(dtype, tau):
    rng, r, n_rows = case(int(tau * 100), dtype)
    x = C.logits(rng, n_rows, V, dtype, ld=50048)
    tok = tokens(rng, r, n_rows)
    one = lambda *v: torch.tensor(v, device=DEV)
    b = ps.make_batch(V=V, T=n_rows, alpha=4.0, tau=tau, chain_seg0=one(0, 1).int(),
                      seg_row0=one(0, n_rows), seg_cut=one(0).int(), seg_src=one(-1).int(),
                      logits=x.to(DEV), tokens=torch.from_numpy(tok.astype(np.int32)).to(DEV))
    rules = C.device_rules(r, DEV)
    ws = torch.empty(ps.ps_rules_workspace_bytes(b), dtype=torch.uint8, device=DEV)
    want = np.array([logprobs(one_row(x[i, :V].double().numpy(), r, i)[0], tok[i], tau)
                     for i in range(n_rows)])
    for entropy in (True, False):
        runs = []
        for _ in range(2):
            lp0, lq, ent = (torch.full((n_rows,), 5.0, dtype=torch.float64, device=DEV) for _ in range(3))
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            ps.ps_score_rows_rules(b, rules, lp0, lq, st, ws, entropy=ent if entropy else None)
            torch.cuda.synchronize()
            assert int(st.item()) == 0
            runs.append(dict(lp0=lp0.cpu().numpy(), lq=lq.cpu().numpy(),
                             entropy=ent.cpu().numpy() if entropy else None))
        for k in ("lp0", "lq") + (("entropy",) if entropy else ()):
            assert np.array_equal(runs[0][k], runs[1][k], equal_nan=True)
        H.check_rows(runs[0], dict(lp0=want[:, 0], lq=want[:, 1], entropy=want[:, 2]))
