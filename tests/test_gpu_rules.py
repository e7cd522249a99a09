"""Rules on logits rows on the GPU: ps_process_rows and ps_score_rows_rules against
the float64 oracle, at the sizes and masks where they can go wrong."""

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps
from oracle import rules as O
from tests import gpu_harness as H
from tests import rules_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EDGES = (1, 7, 8, 31, 32, 1023, 1024, 2047, 2048, 4095, 4096, 8191, 8192, 8199, 16383, 16384)


def setup_module(module):
    import __graft_entry__
    __graft_entry__.build()


def process(r, x, V, out=None, stream=None):
    """(rows [n, V] as the device wrote them, out tensor, status)."""
    xd = x.to(DEV)
    out = torch.full_like(xd, 7.0) if out is None else out
    if isinstance(out, str):
        out = xd
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ps.ps_process_rows(C.device_rules(r, DEV), xd, out, st, V=V, stream=stream)
    torch.cuda.synchronize()
    return out.cpu()[:, :V], out.cpu(), int(st.item())


def check_process(got, x, r, V, dtype):
    want, size = O.process_rows(C.host(x, V), r)
    g = got.double().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(g[inf], want[inf])
    ok = ~np.isnan(want) & ~inf
    err = np.abs(g[ok] - want[ok])
    assert (err <= C.process_bound(want, size, dtype)[ok]).all(), err.max()
    # what no rule touches keeps its bits
    same = (want == C.host(x, V)) & ok & (size == np.abs(want))
    assert np.array_equal(g[same], C.host(x, V)[same])


def score(r, x, V, tokens, tau, entropy=True, row_index=None, stream=None):
    n = len(tokens)
    xd = x.to(DEV)
    one = lambda *v: torch.tensor(v, device=DEV)
    b = ps.make_batch(V=V, T=max(1, n), alpha=4.0, tau=tau, chain_seg0=one(0, 1).int(),
                      seg_row0=one(0, n).long(), seg_cut=one(0).int(), seg_src=one(-1).int(),
                      logits=xd, tokens=torch.from_numpy(np.asarray(tokens, np.int32)).to(DEV),
                      row_index=None if row_index is None
                      else torch.from_numpy(np.asarray(row_index, np.int64)).to(DEV))
    f = lambda: torch.full((n,), 5.0, dtype=torch.float64, device=DEV)
    lp0, lq, ent = f(), f(), f()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    nb = ps.ps_rules_workspace_bytes(b)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device=DEV)
    ps.ps_score_rows_rules(b, C.device_rules(r, DEV), lp0, lq, st, ws, stream=stream,
                           entropy=ent if entropy else None)
    torch.cuda.synchronize()
    return dict(lp0=lp0.cpu().numpy(), lq=lq.cpu().numpy(),
                entropy=ent.cpu().numpy() if entropy else None, status=int(st.item()))


def check_score(g, x, r, V, tokens, tau, rows=None):
    v = C.host(x, V)
    v = v if rows is None else v[rows]
    y, _ = O.process_rows(v, r)
    lp0, lq, ent = O.logprobs(y, tokens, tau)
    H.check_rows(g, dict(lp0=lp0, lq=lq, entropy=ent))


# (V, rows): one id, odd sizes, the ends of 16-byte vectors, mask words and slices
SIZES = [(1, 1), (7, 3), (33, 5), (1000, 9), (8191, 4), (8192, 4), (8201, 4), (50021, 6),
         (151936, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", SIZES)
def test_process_rows(V, n, dtype):
    rng = np.random.default_rng(V + n)
    r = C.random_rules(rng, V, n, edge_ids=EDGES)
    x = C.logits(rng, n, V, dtype)
    got, whole, st = process(r, x, V)
    assert st == 0
    check_process(got, x, r, V, dtype)
    assert (whole[:, V:] == 7.0).all()                   # the padding is not written
    inplace, whole, st = process(r, x, V, out="in place")
    assert st == 0 and torch.equal(inplace, got)
    assert torch.isnan(whole[:, V:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", SIZES)
def test_score_rows(V, n, dtype):
    rng = np.random.default_rng(V + 2 * n)
    r = C.random_rules(rng, V, n, edge_ids=EDGES)
    x = C.logits(rng, n, V, dtype)
    # tokens: anywhere, among the touched ids, and at the ends
    tok = rng.integers(0, V, n)
    tok[: n // 2] = rng.choice(r.seq_tokens, n // 2)
    tok[-1] = V - 1
    for tau, entropy in ((0.25, True), (0.25, False), (0.7, True), (1.0, False)):
        g = score(r, x, V, tok, tau, entropy)
        assert g["status"] == 0
        check_score(g, x, r, V, tok, tau)


@pytest.mark.parametrize("tau", [1.0, 0.5, 0.25, 0.125, 0.3, 1.7])
def test_score_temperatures(tau):
    rng = np.random.default_rng(int(100 * tau))
    V, n = 3001, 12
    r = C.random_rules(rng, V, n)
    x = C.logits(rng, n, V, "bf16")
    tok = rng.integers(0, V, n)
    for entropy in (True, False):
        check_score(score(r, x, V, tok, tau, entropy), x, r, V, tok, tau)


def test_dominant_token_keeps_its_digits():
    # log p near 0: the penalty leaves the token far above the rest
    rng = np.random.default_rng(3)
    V, n = 9001, 6
    x = C.logits(rng, n, V, "f32", sigma=1.0)
    tok = np.array([5, 8191, 8192, 9000, 17, 42])
    x[torch.arange(n), torch.from_numpy(tok)] = 40.0
    r = C.random_rules(rng, V, n, n_masks=0)
    r.seq_tokens[:] = rng.choice(tok, r.seq_tokens.shape[0])
    r.frequency[:] = 0.01
    g = score(r, x, V, tok, 0.5)
    check_score(g, x, r, V, tok, 0.5)


@pytest.mark.parametrize("op", ["process", "score"])
def test_every_part_alone_and_none(op):
    rng = np.random.default_rng(11)
    V, n = 4099, 6
    full = C.random_rules(rng, V, n, n_seqs=n)
    # lengths that both a row's sequence and sequence r have
    own = np.diff(full.seq_begin)
    full.row_len = np.minimum(full.row_len, own).astype(np.int32)
    x = C.logits(rng, n, V, "bf16")
    tok = rng.integers(0, V, n)
    parts = [(), ("seq_begin", "seq_tokens"),
             ("seq_begin", "seq_tokens", "repetition", "row_len"),
             ("seq_begin", "seq_tokens", "seq_prompt", "frequency", "row_seq"),
             ("seq_begin", "seq_tokens", "presence"),
             ("bias_begin", "bias_ids", "bias_values"),
             ("bias_begin", "bias_ids", "bias_values", "row_seq"), ("mask", "row_mask")]
    for keep in parts:
        r = O.Rules(**{k: getattr(full, k) for k in keep})
        if op == "process":
            got, _, st = process(r, x, V)
            check_process(got, x, r, V, "bf16")
        else:
            g = score(r, x, V, tok, 0.25)
            st = g["status"]
            check_score(g, x, r, V, tok, 0.25)
        assert st == 0, keep
    r = O.Rules(mask=np.ascontiguousarray(np.tile(full.mask, (2, 1))[:n]))   # row r has mask r
    got, _, st = process(r, x, V)
    assert st == 0
    check_process(got, x, r, V, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_places_may_hold_anything(dtype):
    rng = np.random.default_rng(12)
    V, n = 8233, 5
    r = C.random_rules(rng, V, n)
    r.row_mask[:] = 1
    r.mask[1] = rng.integers(0, 2 ** 32, r.mask.shape[1], dtype=np.uint32)
    r.mask[1, 0] |= 1 << 9
    x = C.logits(rng, n, V, dtype)
    off = np.array([not (int(r.mask[1, v // 32]) >> (v % 32)) & 1 for v in range(V)])
    bad = torch.tensor([float("nan"), float("inf"), float("-inf"),
                        float(torch.finfo(C.NP[dtype]).min)])
    for i in range(n):
        x[i, :V][torch.from_numpy(off)] = bad[i % 4].to(C.NP[dtype])
    x[:, :V][:, 9] = 1.0                                  # allowed
    got, _, st = process(r, x, V)
    assert st == 0
    check_process(got, x, r, V, dtype)
    on = np.nonzero(~off)[0]
    tok = on[rng.integers(0, len(on), n)]
    tok[0] = np.nonzero(off)[0][0]                        # a forbidden token: -inf
    for entropy in (True, False):
        g = score(r, x, V, tok, 0.25, entropy)
        assert g["status"] == 0 and g["lp0"][0] == -np.inf
        check_score(g, x, r, V, tok, 0.25)


def test_rows_that_keep_nothing_or_one_id():
    rng = np.random.default_rng(13)
    V, n = 5000, 4
    r = O.Rules(mask=np.zeros((2, 157), np.uint32), row_mask=np.array([0, 1, -1, 0], np.int32))
    r.mask[1, 100] = 1 << 5
    r.mask[0, 156] = 0xFFFFFF00                           # bits from V on only
    x = C.logits(rng, n, V, "f32")
    got, _, st = process(r, x, V)
    assert st == 0 and torch.isneginf(got[[0, 3]]).all()
    check_process(got, x, r, V, "f32")
    tok = np.array([3205, 3205, 3205, 1])
    for entropy in (True, False):
        g = score(r, x, V, tok, 0.25, entropy)
        assert g["status"] == 0x02                        # a row without a finite logit
        assert g["lp0"][1] == 0.0 and g["lq"][1] == 0.0
        check_score(g, x, r, V, tok, 0.25)


def test_nonfinite_logits_that_count():
    rng = np.random.default_rng(14)
    V, n = 20000, 6
    r = C.random_rules(rng, V, n, n_masks=0)
    x = C.logits(rng, n, V, "bf16")
    x[1, 9000] = float("nan")
    x[2, 100] = float("inf")
    x[3, :V] = float("-inf")
    x[4, : V // 2] = float("-inf")
    x[5, int(r.seq_tokens[0])] = float("nan")             # on a touched id
    tok = rng.integers(V // 2, V, n)
    for entropy in (True, False):
        g = score(r, x, V, tok, 0.25, entropy)
        assert g["status"] == 0x02
        check_score(g, x, r, V, tok, 0.25)
    got, _, st = process(r, x, V)
    assert st == 0
    check_process(got, x, r, V, "bf16")


def test_infinite_biases():
    rng = np.random.default_rng(15)
    V, n = 300, 2
    r = O.Rules(bias_begin=np.array([0, 3, 3]), bias_ids=np.array([0, 7, 299], np.int32),
                bias_values=np.array([-np.inf, 2.0, -np.inf], np.float32))
    x = C.logits(rng, n, V, "f32")
    got, _, _ = process(r, x, V)
    check_process(got, x, r, V, "f32")
    tok = np.array([7, 0])
    check_score(score(r, x, V, tok, 0.5), x, r, V, tok, 0.5)
    assert score(r, x, V, [0, 1], 0.5)["lp0"][0] == -np.inf


@pytest.mark.parametrize("op", ["process", "score"])
def test_growing_prefixes_and_long_histories(op):
    """Consecutive positions of two sequences (each row sees one token more), and
    histories far longer than the vocabulary slice."""
    rng = np.random.default_rng(16)
    V, n = 12000, 40
    r = C.random_rules(rng, V, n, n_seqs=2, longest=30000)
    r.seq_begin = np.array([0, 20000, 30000])
    r.seq_tokens = rng.integers(0, V, 30000).astype(np.int32)
    r.seq_prompt = np.array([15000, 50000], np.int32)     # a prompt longer than the sequence too
    r.row_seq = np.repeat([0, 1], n // 2).astype(np.int32)
    r.row_len = np.concatenate([19960 + np.arange(20), np.arange(20)]).astype(np.int32)
    r.row_len[5] = 3                                      # and one step back
    x = C.logits(rng, n, V, "bf16")
    if op == "process":
        got, _, st = process(r, x, V)
        assert st == 0
        check_process(got, x, r, V, "bf16")
    else:
        tok = rng.integers(0, V, n)
        g = score(r, x, V, tok, 0.25, False)
        assert g["status"] == 0
        check_score(g, x, r, V, tok, 0.25)


def test_one_token_all_the_time():
    V, n = 2048, 3
    rng = np.random.default_rng(17)
    r = O.Rules(seq_begin=np.array([0, 70000]), seq_tokens=np.full(70000, 2047, np.int32),
                frequency=np.array([0.001], np.float32), row_seq=np.zeros(3, np.int32),
                row_len=np.array([70000, 65536, 1], np.int32))
    x = C.logits(rng, n, V, "f32")
    got, _, st = process(r, x, V)
    assert st == 0
    check_process(got, x, r, V, "f32")
    tok = np.array([2047, 2047, 0])
    check_score(score(r, x, V, tok, 0.5), x, r, V, tok, 0.5)


def test_row_index_and_shared_rows():
    rng = np.random.default_rng(18)
    V, pool, n = 5003, 7, 25
    r = C.random_rules(rng, V, n)
    x = C.logits(rng, pool, V, "bf16", ld=5064)
    ri = rng.integers(0, pool, n)
    tok = rng.integers(0, V, n)
    g = score(r, x, V, tok, 0.25, row_index=ri)
    assert g["status"] == 0
    check_score(g, x, r, V, tok, 0.25, rows=ri)


@pytest.mark.parametrize("n", [400, 1000])
def test_many_rows(n):
    """More rows than blocks; a repeated call and another stream give the same bits."""
    rng = np.random.default_rng(n)
    V = 777
    r = C.random_rules(rng, V, n, longest=300, n_seqs=5)
    order = np.lexsort((r.row_len, r.row_seq))
    r.row_seq, r.row_len = r.row_seq[order], r.row_len[order]
    x = C.logits(rng, n, V, "bf16")
    tok = rng.integers(0, V, n)
    got, _, st = process(r, x, V)
    assert st == 0
    check_process(got, x, r, V, "bf16")
    g = score(r, x, V, tok, 0.25)
    check_score(g, x, r, V, tok, 0.25)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, _, _ = process(r, x, V)
        h = score(r, x, V, tok, 0.25)
    assert torch.equal(torch.nan_to_num(again), torch.nan_to_num(got))
    for k in ("lp0", "lq", "entropy"):
        assert np.array_equal(g[k], h[k], equal_nan=True)


def test_no_rules_agree_with_plain_scoring():
    rng = np.random.default_rng(20)
    V, n = 40001, 30
    x = C.logits(rng, n, V, "bf16")
    tok = rng.integers(0, V, n)
    g = score(O.Rules(), x, V, tok, 0.25)
    check_score(g, x, O.Rules(), V, tok, 0.25)
    got, _, _ = process(O.Rules(), x, V)
    assert torch.equal(got, x[:, :V])


def test_no_rows():
    r = O.Rules()
    assert process(r, torch.zeros(0, 64, dtype=torch.bfloat16), 64)[2] == 0
    assert score(r, torch.zeros(0, 64, dtype=torch.bfloat16), 64, np.zeros(0, np.int32), 0.5)["status"] == 0


def _broken(kind, r, n):
    """One fault in the rules of row 1 (or of its sequence); the bits it sets and
    the rows whose results are NaN."""
    s = int(r.row_seq[1])
    if kind == "token":
        r.row_len[:] = np.minimum(r.row_len, 5)
        r.row_len[1] = 20
        r.seq_tokens[r.seq_begin[s] + 19] = 10 ** 6
        return 0x01, [1]
    if kind == "negative token":
        r.row_len[:] = np.minimum(r.row_len, 5)
        r.row_len[1] = 20
        r.seq_tokens[r.seq_begin[s] + 12] = -3
        return 0x01, [1]
    if kind in ("sequence", "negative sequence"):
        r.row_seq[1] = 10 ** 6 if kind == "sequence" else -1
        return 0x100, [1]
    if kind in ("length", "negative length"):
        r.row_len[1] = 10 ** 6 if kind == "length" else -1
        return 0x100, [1]
    if kind in ("mask", "negative mask"):
        r.row_mask[1] = 99 if kind == "mask" else -2
        return 0x100, [1]
    same = [i for i in range(n) if r.row_seq[i] == s]
    if kind == "repetition":
        r.repetition[s] = 0.0
    elif kind == "presence":
        r.presence[s] = np.nan
    elif kind == "frequency":
        r.frequency[s] = np.inf
    elif kind == "begin":
        r.seq_begin[s + 1] = 10 ** 9
        same = [i for i in range(n) if r.row_seq[i] in (s, s + 1)]
    elif kind == "bias order":
        b = int(r.bias_begin[s])
        r.bias_ids[b], r.bias_ids[b + 1] = r.bias_ids[b + 1], r.bias_ids[b]
    elif kind == "bias twice":
        b = int(r.bias_begin[s])
        r.bias_ids[b + 1] = r.bias_ids[b]
    elif kind == "bias id":
        r.bias_ids[int(r.bias_begin[s + 1]) - 1] = 10 ** 6
    return 0x100, same


@pytest.mark.parametrize("kind", [
    "token", "negative token", "sequence", "negative sequence", "length", "negative length",
    "mask", "negative mask", "repetition", "presence", "frequency", "begin", "bias order",
    "bias twice", "bias id"])
def test_faults_are_flagged_and_stay_in_their_rows(kind):
    rng = np.random.default_rng(21)
    V, n = 9000, 8
    r = C.random_rules(rng, V, n, n_seqs=4, longest=30)
    r.seq_begin = np.arange(5).astype(np.int64) * 30      # equal lengths, three biases each
    r.seq_tokens = rng.integers(0, V, 120).astype(np.int32)
    r.row_seq = np.array([0, 1, 2, 3, 1, 2, 0, 3], np.int32)
    r.row_len = rng.integers(0, 31, n).astype(np.int32)
    r.bias_begin = np.arange(5).astype(np.int64) * 3
    r.bias_ids = np.concatenate([np.sort(rng.choice(V, 3, replace=False)) for _ in range(4)]).astype(np.int32)
    r.bias_values = rng.normal(0, 1, 12).astype(np.float32)
    x = C.logits(rng, n, V, "bf16")
    tok = rng.integers(0, V, n)
    good, _, _ = process(r, x, V)
    good_s = score(r, x, V, tok, 0.25)
    import copy
    bad = copy.deepcopy(r)
    bits, rows = _broken(kind, bad, n)
    if kind in ("token", "negative token"):
        r.row_len = bad.row_len
        good, _, _ = process(O.Rules(**{**vars(r)}), x, V)
        good_s = score(r, x, V, tok, 0.25)
    got, _, st = process(bad, x, V)
    assert st == bits
    inplace, _, st = process(bad, x, V, out="in place")
    assert st == bits
    assert torch.isnan(got[rows]).all() and torch.isnan(inplace[rows]).all()
    rest = [i for i in range(n) if i not in rows]
    assert torch.equal(got[rest], good[rest]) and torch.equal(inplace[rest], good[rest])
    g = score(bad, x, V, tok, 0.25)
    assert g["status"] == bits
    for k in ("lp0", "lq", "entropy"):
        assert np.isnan(g[k][rows]).all()
        assert np.array_equal(g[k][rest], good_s[k][rest])


def test_bad_scored_token_and_row_index():
    rng = np.random.default_rng(22)
    V, n = 600, 4
    r = C.random_rules(rng, V, n)
    x = C.logits(rng, n, V, "f32")
    g = score(r, x, V, [0, V, 1, -1], 0.25)
    assert g["status"] == 0x01 and np.isnan(g["lp0"][[1, 3]]).all() and np.isfinite(g["entropy"][[0, 2]]).all()
    g = score(r, x, V, [0, 1, 2, 3], 0.25, row_index=[0, 9, 2, -1])
    assert g["status"] == 0x40 and np.isnan(g["lq"][[1, 3]]).all() and np.isfinite(g["entropy"][[0, 2]]).all()
