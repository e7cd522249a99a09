"""Inputs of the tests of rules on logits rows: host descriptions, their device
form, and the tolerances of what is computed from them."""

import numpy as np
import torch

import mh_prefetch_subtree_gb300 as ps
from oracle.rules import Rules

U32 = 2.0 ** -24          # half a unit in the last place of float32, relative
UBF = 2.0 ** -8           # of bfloat16 (8 significant bits)

NP = {"bf16": torch.bfloat16, "f32": torch.float32}


def random_rules(rng, V, n_rows, *, n_seqs=None, longest=64, n_masks=4, n_bias=6, edge_ids=()):
    """Rules with sequences of length 0 and 1 among them, repeated tokens, ids at
    the ends of the vocabulary and at edge_ids, biases on seen, unseen and masked
    ids, wide and narrow masks, and rows of every sequence in no order."""
    n_seqs = n_seqs or max(1, n_rows // 2)
    lens = rng.integers(0, longest + 1, n_seqs)
    lens[0] = longest
    if n_seqs > 1:
        lens[1] = 0
    if n_seqs > 2:
        lens[2] = 1
    begin = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    pool = np.unique(np.concatenate([rng.integers(0, V, 24), [0, V - 1],
                                     [e for e in edge_ids if 0 <= e < V]]).astype(np.int64))
    toks = rng.choice(pool, int(begin[-1])).astype(np.int32)
    few = rng.random(toks.shape[0]) < 0.3
    toks[few] = pool[0]                                  # one id very often
    row_seq = rng.integers(0, n_seqs, n_rows).astype(np.int32)
    row_len = np.array([rng.integers(0, lens[s] + 1) for s in row_seq], np.int32)
    row_len[0] = lens[row_seq[0]]
    bias = [np.sort(rng.choice(pool, min(len(pool), int(k)), replace=False))
            for k in rng.integers(0, n_bias + 1, n_seqs)]
    ids = np.concatenate(bias).astype(np.int32) if n_bias else np.zeros(0, np.int32)
    r = Rules(
        seq_begin=begin, seq_tokens=toks, seq_prompt=rng.integers(0, longest, n_seqs).astype(np.int32),
        repetition=rng.choice([0.8, 1.0, 1.3], n_seqs).astype(np.float32),
        frequency=rng.choice([-0.25, 0.0, 0.4], n_seqs).astype(np.float32),
        presence=rng.choice([-0.5, 0.0, 0.7], n_seqs).astype(np.float32),
        bias_begin=np.concatenate([[0], np.cumsum([len(b) for b in bias])]).astype(np.int64),
        bias_ids=ids, bias_values=rng.normal(0, 3, ids.shape[0]).astype(np.float32),
        row_seq=row_seq, row_len=row_len)
    if n_masks:
        words = (V + 31) // 32
        share = rng.choice([1.0, 0.9, 0.5, 0.03], n_masks)
        bits = rng.random((n_masks, words * 32)) < share[:, None]
        bits[:, :V][:, rng.integers(0, V, 4)] = True
        r.mask = (bits.reshape(n_masks, words, 32).astype(np.uint64)
                  << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
        r.row_mask = rng.integers(-1, n_masks, n_rows).astype(np.int32)
    return r


def device_rules(r: Rules, dev) -> ps.PsLogitRules:
    kw = {}
    for k, a in vars(r).items():
        if a is None:
            continue
        a = np.ascontiguousarray(a.view(np.int32) if a.dtype == np.uint32 else a)
        kw[k] = torch.from_numpy(a.copy()).to(dev)
    return ps.make_rules(**kw)


def logits(rng, n_rows, V, dtype, ld=None, sigma=3.0):
    """(host float64 values, CPU tensor [n_rows, ld]) of normal logits; the padding
    holds NaN."""
    ld = ld or -(-V // 8) * 8
    x = torch.full((n_rows, ld), float("nan"), dtype=NP[dtype])
    x[:, :V] = torch.from_numpy(rng.normal(0, sigma, (n_rows, V))).to(NP[dtype])
    return x


def host(x, V):
    return x[:, :V].double().numpy()


def process_bound(want, size, dtype):
    """Float32 arithmetic of at most five operations on terms whose magnitudes add
    up to `size`, then one rounding to the rows' type."""
    b = 5 * U32 * size
    with np.errstate(invalid="ignore"):
        if dtype == "bf16":
            b = b + UBF * (np.abs(want) + b)
    return b
