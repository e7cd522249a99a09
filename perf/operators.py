"""Cases for measuring the operators around the scoring of logits rows.

Three operators, each with a plain form (elementary torch operations, 32 bits) and
the library's own calls:

head     ps_head_rows: the output head with 4-bit weights and group scales, which
         makes the logits rows while proposals are decoded.
process  ps_process_rows: penalties for repeated tokens, biases and grammar masks
         on logits rows.
score    ps_score_rows_rules: log p0, log q_tau and entropy of each row's token
         under the same rules, without writing the processed rows.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _head(name, rows, V, K, group, scale="bf16", out="bf16", zeros=True):
    return {"name": name, "op": "head", "rows": rows, "V": V, "K": K, "group": group,
            "scale": scale, "out": out, "zeros": zeros}


def _process(name, rows, V, dtype, per_seq, hist, masks, bias):
    return {"name": name, "op": "process", "rows": rows, "V": V, "dtype": dtype,
            "per_seq": per_seq, "hist": hist, "masks": masks, "bias": bias}


def _score(name, rows, V, dtype, per_seq, hist, masks, bias, tau, entropy):
    c = _process(name, rows, V, dtype, per_seq, hist, masks, bias)
    c.update({"op": "score", "tau": tau, "entropy": entropy})
    return c


def listed():
    return [
        # one chain decoding alone: the whole head is read for a single token
        _head("head-one-token", 1, 151936, 4096, 128),
        # the 16 requests of a round decode together
        _head("head-16-requests", 16, 151936, 4096, 128),
        # 64 requests, the largest round, with a larger vocabulary and a narrower model
        _head("head-64-requests", 64, 262144, 2048, 64, zeros=False),
        # a tiny vocabulary and model: what a call costs
        _head("head-tiny", 4, 1024, 1024, 32, scale="f32", out="f32"),
        # one chain, tiny vocabulary, no grammar: what a call costs
        _process("process-tiny", 1, 1024, "f32", 1, 64, 0, 0),
        # one decoding step of a round's 16 requests, after a prompt and half an answer
        _process("process-16-requests", 16, 151936, "bf16", 1, 2048, 12, 32),
        # the suffixes of one request after another, all positions at once
        _process("process-suffixes", 1000, 151936, "bf16", 250, 512, 24, 32),
        # float32 rows of an odd vocabulary, long histories, few rows for each
        _process("process-long-f32", 150, 50021, "f32", 3, 16384, 6, 8),
        # the token of every request, just drawn, with the entropy of its row
        _score("score-16-requests", 16, 151936, "bf16", 1, 2048, 12, 32, 0.25, True),
        # a subtree's segments: every position of every suffix
        _score("score-subtree", 8000, 151936, "bf16", 600, 512, 24, 32, 0.25, False),
        # a larger vocabulary, another temperature and the entropy
        _score("score-entropy", 1500, 262144, "bf16", 400, 2048, 24, 8, 0.7, True),
        # float32 rows of an odd vocabulary without a grammar
        _score("score-odd-f32", 777, 50021, "f32", 100, 1024, 0, 16, 0.5, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("head", "process", "score"))
    if op == "head":
        group = rng.choice((32, 64, 128))
        rows, V = _log(rng, 1, 64), _log(rng, 1000, 262144)
        most = 151936 * 4096 // V
        K = group * max(1, _log(rng, 512, min(8192, max(most, 513))) // group)
        return {"op": op, "rows": rows, "V": V, "K": K, "group": group,
                "scale": rng.choice(("bf16", "f32")), "out": rng.choice(("bf16", "f32")),
                "zeros": rng.random() < 0.5}
    dtype = rng.choice(("bf16", "bf16", "f32"))
    V = _log(rng, 1000, 262144)
    most = (150_000_000 if op == "process" else 1_200_000_000) // (V * (2 if dtype == "f32" else 1))
    rows = _log(rng, 1, max(2, min(6000, most)))
    c = {"op": op, "rows": rows, "V": V, "dtype": dtype,
         "per_seq": rng.choice((1, _log(rng, 1, 1000))), "hist": _log(rng, 16, 16384),
         "masks": rng.choice((0, rng.randint(1, 32))), "bias": rng.choice((0, rng.randint(1, 64)))}
    # the plain form holds rows * (history + suffix) token places
    while c["rows"] * (c["hist"] + 2 * c["per_seq"]) > 40_000_000:
        c["hist"] = max(16, c["hist"] // 2)
        c["per_seq"] = max(1, c["per_seq"] // 2)
    if op == "score":
        c["tau"] = rng.choice((0.125, 0.25, 0.5, 1.0, round(rng.uniform(0.2, 1.5), 3)))
        c["entropy"] = rng.random() < 0.4
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _prepare_head(c, seed):
    g = _gen(seed)
    V, K, G = c["V"], c["K"], c["group"]
    s = {"case": c}
    # hidden states after a norm: about one in size, some channels far larger
    h = torch.randn(c["rows"], K, device=DEV, generator=g)
    h = h * torch.exp(0.5 * torch.randn(K, device=DEV, generator=g))
    s["hidden"] = h.to(torch.bfloat16)
    s["q"] = torch.randint(0, 256, (V, K // 2), device=DEV, dtype=torch.uint8, generator=g)
    sc = (0.5 + torch.rand(V, K // G, device=DEV, generator=g)) * (0.6 / math.sqrt(K))
    s["scales"] = sc.to(TYPES[c["scale"]])
    s["zeros"] = (torch.randint(5, 11, (V, K // G), device=DEV, dtype=torch.uint8, generator=g)
                  if c["zeros"] else None)
    s["ld"] = -(-V // 8) * 8
    if own:
        import mh_prefetch_subtree_gb300 as ps

        s["out"] = torch.zeros(c["rows"], s["ld"], dtype=TYPES[c["out"]], device=DEV)
        s["head"] = ps.make_head(q=s["q"], scales=s["scales"], zeros=s["zeros"], group=G)
    return s


def _prepare_rows(c, seed):
    rng = np.random.default_rng(seed)
    g = _gen(seed)
    rows, V, per_seq, hist = c["rows"], c["V"], c["per_seq"], c["hist"]
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    # sequences: a prompt, generated tokens before the first row, then one row a token
    sizes = rng.integers(1, 2 * per_seq, rows) if per_seq > 1 else np.ones(rows, np.int64)
    n_seqs = int(np.searchsorted(np.cumsum(sizes), rows)) + 1
    sizes = sizes[:n_seqs]
    sizes[-1] -= int(sizes.sum()) - rows
    before = rng.integers(hist // 2, hist + 1, n_seqs)
    if n_seqs > 2:
        before[1] = 0                                   # a sequence that begins here
    prompt = (before * rng.uniform(0.2, 0.9, n_seqs)).astype(np.int64)
    seq_begin = np.concatenate([[0], np.cumsum(before + sizes)])
    row_seq = np.repeat(np.arange(n_seqs), sizes)
    first = np.repeat(np.cumsum(sizes) - sizes, sizes)
    row_len = before[row_seq] + np.arange(rows) - first
    n_tok = int(seq_begin[-1])
    # token ids as text has them: a few very often
    toks = torch.rand(n_tok, device=DEV, generator=g).pow(4).mul(V).to(torch.int64).clamp(max=V - 1)
    to = lambda a, t: torch.as_tensor(np.ascontiguousarray(a)).to(device=DEV, dtype=t)  # noqa: E731
    s["seq_begin"], s["seq_prompt"] = to(seq_begin, torch.int64), to(prompt, torch.int32)
    s["row_seq"], s["row_len"] = to(row_seq, torch.int32), to(row_len, torch.int32)
    s["longest"] = int(row_len.max()) if rows else 0
    s["repetition"] = to(rng.choice([1.0, 1.05, 1.1, 1.3], n_seqs), torch.float32)
    s["frequency"] = to(rng.choice([0.0, 0.1, 0.4], n_seqs), torch.float32)
    s["presence"] = to(rng.choice([0.0, 0.2, 0.5], n_seqs), torch.float32)
    # biases: distinct ids in rising order, per sequence
    s["bias_begin"] = s["bias_ids"] = s["bias_values"] = None
    if c["bias"]:
        n = rng.integers(0, c["bias"] + 1, n_seqs)
        ids = [np.sort(rng.choice(V, k, replace=False)) for k in n]
        s["bias_begin"] = to(np.concatenate([[0], np.cumsum(n)]), torch.int64)
        s["bias_ids"] = to(np.concatenate(ids), torch.int32)
        s["bias_values"] = to(rng.normal(0, 2, int(n.sum())), torch.float32)
    # a row for each state of the grammar: wide ones and narrow ones; some rows are free
    words = -(-V // 32)
    s["mask"] = s["row_mask"] = None
    keep = None
    if c["masks"]:
        share = rng.choice([0.95, 0.5, 0.02, 0.001], c["masks"])
        keep = torch.randint(0, V, (c["masks"], 32), device=DEV, generator=g)
        bits = torch.rand(c["masks"], words * 32, device=DEV, generator=g) < to(share, torch.float32)[:, None]
        bits.scatter_(1, keep, True)
        w = bits.view(c["masks"], words, 32).to(torch.int64) << torch.arange(32, device=DEV)
        w = w.sum(-1)
        s["mask"] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
        s["row_mask"] = to(rng.integers(-1, c["masks"], rows), torch.int32)
    # each row's token is the sequence's next one; a row with a mask mostly has an allowed one
    at = to(seq_begin[row_seq] + row_len, torch.int64)
    if keep is not None:
        m = s["row_mask"].long()
        pick = keep[m.clamp(min=0), torch.randint(0, 32, (rows,), device=DEV, generator=g)]
        free = (m < 0) | (torch.rand(rows, device=DEV, generator=g) < 0.02)
        toks[at] = torch.where(free, toks[at], pick)
    s["seq_tokens"] = toks.to(torch.int32)
    s["tokens"] = s["seq_tokens"][at].contiguous()
    # logits: normal, the row's token raised in most rows
    ld = -(-V // 8) * 8
    x = torch.empty(rows, ld, dtype=dt, device=DEV)
    for r in range(0, rows, 2000):
        y = torch.randn(min(2000, rows - r), ld, device=DEV, generator=g).mul_(3.0)
        up = 8.0 + 3.0 * torch.randn(y.shape[0], 1, device=DEV, generator=g)
        y.scatter_add_(1, s["tokens"][r:r + 2000, None].long(), up)
        x[r:r + 2000] = y.to(dt)
    s["logits"], s["ld"] = x, ld
    if own:
        import mh_prefetch_subtree_gb300 as ps

        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["rules"] = ps.make_rules(
            seq_begin=s["seq_begin"], seq_tokens=s["seq_tokens"], seq_prompt=s["seq_prompt"],
            repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
            bias_begin=s["bias_begin"], bias_ids=s["bias_ids"], bias_values=s["bias_values"],
            mask=s["mask"], row_mask=s["row_mask"], row_seq=s["row_seq"], row_len=s["row_len"])
        if c["op"] == "process":
            s["out"] = torch.zeros_like(x)
        else:
            one = lambda *v: torch.tensor(v, device=DEV)  # noqa: E731
            s["batch"] = ps.make_batch(
                V=V, T=rows, alpha=4.0, tau=c["tau"], chain_seg0=one(0, 1).int(),
                seg_row0=one(0, rows).long(), seg_cut=one(0).int(), seg_src=one(-1).int(),
                logits=x, tokens=s["tokens"])
            s["rows64"] = torch.zeros(3 if c["entropy"] else 2, rows, dtype=torch.float64, device=DEV)
            s["workspace"] = torch.empty(ps.ps_rules_workspace_bytes(s["batch"]), dtype=torch.uint8,
                                         device=DEV)
    return s


def prepare(case, seed):
    return _prepare_head(case, seed) if case["op"] == "head" else _prepare_rows(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_head(s):
    c = s["case"]
    V, K, G = c["V"], c["K"], c["group"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], -1).view(V, K // G, G).float()
    z = s["zeros"].float()[:, :, None] if s["zeros"] is not None else 8.0
    w = ((q - z) * s["scales"].float()[:, :, None]).view(V, K)
    return (s["hidden"].float() @ w.t()).to(TYPES[c["out"]])


def _plain_rules(s):
    """The processed rows, in 32 bits."""
    c = s["case"]
    rows, V = c["rows"], c["V"]
    x = s["logits"][:, :V].float()
    rs = s["row_seq"].long()
    col = lambda a: a[rs][:, None]  # noqa: E731
    if s["longest"]:
        at = torch.arange(s["longest"], device=DEV)[None, :]
        there = at < s["row_len"][:, None]
        made = there & (at >= col(s["seq_prompt"]))
        ids = s["seq_tokens"][torch.where(there, col(s["seq_begin"][:-1]) + at, 0)].long()
        count = torch.zeros(rows, V, device=DEV).scatter_add_(1, ids, made.float())
        seen = torch.zeros(rows, V, device=DEV).scatter_add_(1, ids, there.float()) > 0
        rho = col(s["repetition"])
        x = torch.where(seen, torch.where(x > 0, x / rho, x * rho), x)
        x = x - col(s["frequency"]) * count - col(s["presence"]) * (count > 0)
        del count, seen
    if s["bias_begin"] is not None:
        n_seqs = s["seq_begin"].numel() - 1
        n = s["bias_begin"][1:] - s["bias_begin"][:-1]
        of = torch.repeat_interleave(torch.arange(n_seqs, device=DEV), n,
                                     output_size=s["bias_ids"].numel())
        dense = torch.zeros(n_seqs, V, device=DEV)
        dense[of, s["bias_ids"].long()] = s["bias_values"]
        x = x + dense[rs]
    if s["mask"] is not None:
        bit = (s["mask"][:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        bit = bit.view(s["mask"].shape[0], -1)[:, :V].bool()
        m = s["row_mask"].long()
        x = torch.where(bit[m.clamp(min=0)] | (m < 0)[:, None], x, float("-inf"))
    return x


def _plain_score(s):
    c = s["case"]
    x = _plain_rules(s)
    x = x - x.amax(1, keepdim=True)
    lt = x.gather(1, s["tokens"].long()[:, None])[:, 0]
    e = x.exp()
    z = e.sum(1)
    got = {"lp0": lt - z.log()}
    if c["entropy"]:
        got["entropy"] = z.log() - torch.where(e > 0, e * x, 0.0).sum(1) / z
    del e
    got["lq"] = lt / c["tau"] - (x / c["tau"]).exp().sum(1).log()
    return got


def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "head":
            return _plain_head(state)
        if c["op"] == "process":
            return _plain_rules(state).to(TYPES[c["dtype"]])
        return _plain_score(state)
    import mh_prefetch_subtree_gb300 as ps

    if c["op"] == "head":
        ps.ps_head_rows(state["head"], state["hidden"], state["out"])
        return state["out"][:, :c["V"]]
    if c["op"] == "process":
        ps.ps_process_rows(state["rules"], state["logits"], state["out"], state["status"], V=c["V"])
        return state["out"][:, :c["V"]]
    r = state["rows64"]
    ps.ps_score_rows_rules(state["batch"], state["rules"], r[0], r[1], state["status"],
                           state["workspace"], entropy=r[2] if c["entropy"] else None)
    f = r.float()
    got = {"lp0": f[0], "lq": f[1]}
    if c["entropy"]:
        got["entropy"] = f[2]
    return got


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c, V = case, case["V"]
    if c["op"] == "head":
        k = c["K"] // c["group"]
        e = 2 if c["out"] == "bf16" else 4
        weights = V * c["K"] / 2 + V * k * ((2 if c["scale"] == "bf16" else 4) + (1 if c["zeros"] else 0))
        return {"bytes": weights + c["rows"] * (2 * c["K"] + e * V),
                "flops": 2 * c["rows"] * V * c["K"]}
    e = 2 if c["dtype"] == "bf16" else 4
    n_seqs = max(1, c["rows"] / c["per_seq"])
    tokens = n_seqs * (0.75 * c["hist"] + c["per_seq"])
    other = 4 * tokens + 12 * c["rows"] + n_seqs * (20 + 4 * c["bias"]) + c["masks"] * V / 8
    if c["op"] == "process":
        return {"bytes": 2 * c["rows"] * V * e + other, "flops": 2 * c["rows"] * V}
    per = (6 if c["tau"] != 1.0 else 4) + (2 if c["entropy"] else 0)
    return {"bytes": c["rows"] * (V * e + 20 + (8 if c["entropy"] else 0)) + other,
            "flops": per * c["rows"] * V}


def _exact_row(s, r, x, bits):
    """Row r's processed logits from `x`, the row in 64 bits."""
    b = s["host"]
    q, V = b["row_seq"][r], s["case"]["V"]
    lo, n, p = b["seq_begin"][q], b["row_len"][r], b["seq_prompt"][q]
    hist = s["seq_tokens"][lo:lo + n].long()
    seen = torch.bincount(hist, minlength=V) > 0
    cnt = torch.bincount(hist[min(p, n):], minlength=V).double()
    rho, fr, pr = (float(b[k][q]) for k in ("repetition", "frequency", "presence"))
    x = torch.where(seen & (x > 0), x / rho, torch.where(seen, x * rho, x))
    x = x - fr * cnt - pr * (cnt > 0).double()
    if s["bias_begin"] is not None:
        i, j = b["bias_begin"][q], b["bias_begin"][q + 1]
        x.index_add_(0, s["bias_ids"][i:j].long(), s["bias_values"][i:j].double())
    if bits is not None and b["row_mask"][r] >= 0:
        x = x.masked_fill(~bits[b["row_mask"][r]], float("-inf"))
    return x


def exact(case, seed):
    s = prepare(case, seed)
    c, V = case, case["V"]
    if c["op"] == "head":
        K, G = c["K"], c["group"]
        h = s["hidden"].double()
        out = torch.empty(c["rows"], V, dtype=torch.float64, device=DEV)
        for v in range(0, V, 16384):
            q = s["q"][v:v + 16384]
            n = q.shape[0]
            w = torch.empty(n, K, dtype=torch.float64, device=DEV)
            w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
            z = s["zeros"][v:v + 16384].double() if s["zeros"] is not None else torch.full(
                (n, K // G), 8.0, dtype=torch.float64, device=DEV)
            w -= z.repeat_interleave(G, 1)
            w *= s["scales"][v:v + 16384].double().repeat_interleave(G, 1)
            out[:, v:v + n] = h @ w.t()
        return out
    s["host"] = {k: s[k].cpu().numpy() for k in (
        "row_seq", "row_len", "seq_begin", "seq_prompt", "repetition", "frequency", "presence",
        "bias_begin", "row_mask") if s[k] is not None}
    bits = None
    if s["mask"] is not None:
        by = s["mask"].view(torch.uint8).long()
        bits = torch.stack([(by >> k) % 2 for k in range(8)], -1).reshape(by.shape[0], -1)[:, :V] == 1
    if c["op"] == "process":
        out = torch.empty(c["rows"], V, dtype=torch.float64, device=DEV)
        for r in range(c["rows"]):
            out[r] = _exact_row(s, r, s["logits"][r, :V].double(), bits)
        return out
    got = {k: torch.empty(c["rows"], dtype=torch.float64, device=DEV)
           for k in ("lp0", "lq") + (("entropy",) if c["entropy"] else ())}
    tok = s["tokens"].tolist()
    for r in range(c["rows"]):
        x = _exact_row(s, r, s["logits"][r, :V].double(), bits)
        lp = x - torch.logsumexp(x, 0)
        got["lp0"][r] = lp[tok[r]]
        t = x / c["tau"]
        got["lq"][r] = t[tok[r]] - torch.logsumexp(t, 0)
        if c["entropy"]:
            got["entropy"][r] = -torch.special.xlogy(lp.exp(), lp.exp()).sum()
    return got
