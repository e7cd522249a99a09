"""Float64 oracle of the rules on logits rows and of the 4-bit head.

Written from their definitions, one id and one row at a time where that is
affordable; shares no code with the CUDA library.

* ``process_row``    one row under penalties, biases and a mask;
* ``process_rows``   every row of a ``Rules`` description, with the magnitude that
                     its rounding errors scale with;
* ``logprobs``       log p0, log q_tau and entropy of processed rows;
* ``head_rows``      the head's products, with the same kind of magnitude.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np


@dataclass
class Rules:
    """Host arrays under the names of ps_logit_rules; None where NULL."""

    seq_begin: np.ndarray | None = None
    seq_tokens: np.ndarray | None = None
    seq_prompt: np.ndarray | None = None
    repetition: np.ndarray | None = None
    frequency: np.ndarray | None = None
    presence: np.ndarray | None = None
    bias_begin: np.ndarray | None = None
    bias_ids: np.ndarray | None = None
    bias_values: np.ndarray | None = None
    mask: np.ndarray | None = None            # uint32 [n_masks, words]
    row_seq: np.ndarray | None = None
    row_len: np.ndarray | None = None
    row_mask: np.ndarray | None = None


def process_row(x, *, history, prompt, repetition, frequency, presence, bias, mask):
    """(l', magnitude) of one float64 row: bias is a list of (id, value), mask a
    row of 32-bit words or None."""
    x = np.array(x, dtype=np.float64)
    V = x.shape[0]
    seen = set(int(t) for t in history)
    made: dict[int, int] = {}
    for t in history[prompt:]:
        made[int(t)] = made.get(int(t), 0) + 1
    size = np.abs(x)
    with np.errstate(invalid="ignore"):
        for v in seen:
            x[v] = x[v] / repetition if x[v] > 0 else x[v] * repetition
            size[v] = abs(x[v])
        for v, c in made.items():
            x[v] = x[v] - frequency * c - presence
            size[v] += abs(frequency) * c + abs(presence)
        for v, b in bias:
            x[v] += b
            size[v] += abs(b)
    if mask is not None:
        for v in range(V):
            if not (int(mask[v // 32]) >> (v % 32)) & 1:
                x[v] = -np.inf
    return x, size


def process_rows(x, r: Rules):
    """(l' [n_rows, V], magnitude) for float64 rows x under r."""
    n_rows = x.shape[0]
    out, size = np.empty_like(x), np.empty_like(x)
    for i in range(n_rows):
        s = i if r.row_seq is None else int(r.row_seq[i])
        history, prompt = [], 0
        one = lambda a, d: d if a is None else float(a[s])
        if r.seq_begin is not None:
            b, e = int(r.seq_begin[s]), int(r.seq_begin[s + 1])
            n = e - b if r.row_len is None else int(r.row_len[i])
            history = list(r.seq_tokens[b:b + n])
            prompt = 0 if r.seq_prompt is None else int(r.seq_prompt[s])
        bias = []
        if r.bias_begin is not None:
            b, e = int(r.bias_begin[s]), int(r.bias_begin[s + 1])
            bias = list(zip(r.bias_ids[b:e].tolist(), r.bias_values[b:e].astype(np.float64)))
        mask = None
        if r.mask is not None:
            m = i if r.row_mask is None else int(r.row_mask[i])
            mask = None if m < 0 else r.mask[m]
        out[i], size[i] = process_row(
            x[i], history=history, prompt=prompt, repetition=one(r.repetition, 1.0),
            frequency=one(r.frequency, 0.0), presence=one(r.presence, 0.0), bias=bias, mask=mask)
    return out, size


def logprobs(x, tokens, tau):
    """(lp0, lq, entropy) of float64 rows x; NaN for a row without a finite logit
    or with a NaN or +inf one."""
    n = x.shape[0]
    lp0, lq, ent = (np.empty(n) for _ in range(3))
    for i in range(n):
        row, t = x[i], int(tokens[i])
        if not np.isfinite(row).any() or np.isnan(row).any() or np.isposinf(row).any():
            lp0[i] = lq[i] = ent[i] = np.nan
            continue
        # relative to the token where it can be, so that a token that holds nearly
        # all the mass keeps its digits
        def logp(y):
            if np.isneginf(y[t]):
                return -np.inf
            d = np.delete(y, t) - y[t]
            m = max(0.0, float(d.max())) if d.size else 0.0
            if m == 0.0:
                return -np.log1p(np.exp(d).sum())
            return -(m + np.log(np.exp(d - m).sum() + np.exp(-m)))

        lp0[i], lq[i] = logp(row), logp(row / tau)
        y = row[np.isfinite(row)]
        y = y - y.max()
        e = np.exp(y)
        z = e.sum()
        ent[i] = np.log(z) - (e * y).sum() / z
    return lp0, lq, ent


def head_rows(hidden, q, scales, zeros, group):
    """(logits, sum of |products|) in float64: hidden [n, K], q [V, K/2] uint8."""
    V, half = q.shape
    w = np.empty((V, 2 * half))
    w[:, 0::2], w[:, 1::2] = q & 15, q >> 4
    z = np.full((V, 2 * half // group), 8.0) if zeros is None else zeros.astype(np.float64)
    w = (w - np.repeat(z, group, 1)) * np.repeat(scales.astype(np.float64), group, 1)
    h = hidden.astype(np.float64)
    return h @ w.T, np.abs(h) @ np.abs(w).T
