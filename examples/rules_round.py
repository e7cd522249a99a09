"""One prefetch round with a constrained proposal: decode, score, walk.

A toy model (the hidden state of a position is the embedding of the token before
it) with a 4-bit output head proposes the suffixes of a subtree under penalties for
repeated tokens, biases and a grammar.  The scores have to come from the same
distribution, so the round's rows are scored under the same rules:

    hidden --ps_head_rows--> logits --ps_process_rows--> drawn tokens
                                \\--ps_score_rows_rules--> log p0, log q_tau
                                                --> log A --> the walk

    python examples/rules_round.py
"""

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mh_prefetch_subtree_gb300 as ps  # noqa: E402
from synth.trees import assemble_layout, bfs_tree  # noqa: E402

DEV = torch.device("cuda:0")


def levels(layout):
    """Requests in the order in which their source states are complete."""
    level = {0: -1}
    while len(level) < layout.n_seg:
        for s in range(1, layout.n_seg):
            if s not in level and int(layout.seg_src[s]) in level:
                level[s] = level[int(layout.seg_src[s])] + 1
    return [[s for s in level if level[s] == k] for k in range(max(level.values()) + 1)]


def main(V=8000, K=256, group=64, T=96, prompt=32, n_pf=12, alpha=4.0, tau=0.25, seed=1):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    layout = assemble_layout([bfs_tree(rng, T, n_pf)])
    n_seg, n_rows = layout.n_seg, layout.n_rows
    row0, cuts = layout.seg_row0, layout.seg_cut

    # the model: embeddings, and a head of 4-bit weights with a scale and a zero a group
    embed = torch.randn(V, K, device=DEV, generator=gen).to(torch.bfloat16)
    head = ps.make_head(
        q=torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device=DEV, generator=gen),
        scales=(0.5 / K ** 0.5 * (0.5 + torch.rand(V, K // group, device=DEV, generator=gen))),
        zeros=torch.randint(6, 11, (V, K // group), dtype=torch.uint8, device=DEV, generator=gen),
        group=group)

    # one sequence per segment: the prompt and positions 1..T
    seqs = torch.randint(0, V, (n_seg, prompt + T), dtype=torch.int32, device=DEV, generator=gen)
    seqs[:, :prompt] = seqs[0, :prompt]
    # a grammar with two states that take turns: even ids, and all ids below 3/4 V
    ids = np.arange(-(-V // 32) * 32)
    bits = np.stack([ids % 2 == 0, ids < 3 * V // 4])
    words = (bits.reshape(2, -1, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
    state_of = lambda t: t % 2  # noqa: E731  (position t is 1..T)
    for t in range(1, T + 1):                      # the current state obeys it as well
        x = seqs[0, prompt + t - 1]
        seqs[0, prompt + t - 1] = x // 2 * 2 if state_of(t) == 0 else x % (3 * V // 4)
    i32 = lambda a: torch.as_tensor(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    shared = dict(
        seq_begin=torch.arange(n_seg + 1, device=DEV) * (prompt + T), seq_tokens=seqs.view(-1),
        seq_prompt=i32([prompt] * n_seg),
        repetition=torch.full((n_seg,), 1.2, device=DEV),
        frequency=torch.full((n_seg,), 0.1, device=DEV),
        presence=torch.full((n_seg,), 0.3, device=DEV),
        bias_begin=torch.arange(n_seg + 1, device=DEV) * 2, bias_ids=i32([0, 100] * n_seg),
        bias_values=torch.tensor([-2.0, 1.5] * n_seg, device=DEV),
        mask=i32(words.astype(np.uint32).view(np.int32)))
    rules_of = lambda seg, t: ps.make_rules(  # noqa: E731  rows (segment, position)
        row_seq=i32(seg), row_len=i32(np.asarray(t) + prompt - 1),
        row_mask=i32([state_of(x) for x in t]), **shared)

    # the logits of every scored row: the current state's, then each request's
    logits = torch.empty(n_rows, V, dtype=torch.bfloat16, device=DEV)
    root = np.arange(cuts[0] + 1, T + 1)
    ps.ps_head_rows(head, embed[seqs[0, prompt + root - 2].long()], logits[:int(row0[1])])
    drawn_lq = torch.zeros(n_seg, dtype=torch.float64, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for batch in levels(layout):
        for s in batch:                            # x_{0:c} comes from the source state
            seqs[s] = seqs[int(layout.seg_src[s])]
        for t in range(1, T + 1):
            live = [s for s in batch if cuts[s] < t]
            if not live:
                continue
            rows = torch.empty(len(live), V, dtype=torch.bfloat16, device=DEV)
            ps.ps_head_rows(head, embed[seqs[live, prompt + t - 2].long()], rows)
            for k, s in enumerate(live):
                logits[int(row0[s]) + t - 1 - int(cuts[s])] = rows[k]
            ps.ps_process_rows(rules_of(live, [t] * len(live)), rows, rows, status)   # in place
            logq = torch.log_softmax(rows.float() / tau, -1)
            tok = torch.multinomial(logq.exp(), 1, generator=gen)
            drawn_lq[live] += logq.gather(1, tok)[:, 0].double()
            seqs[live, prompt + t - 1] = tok[:, 0].int()

    # score the round under the rules, and walk it
    seg = np.repeat(np.arange(n_seg), np.diff(row0))
    pos = np.concatenate([np.arange(cuts[s] + 1, T + 1) for s in range(n_seg)])
    tokens = seqs[torch.as_tensor(seg, device=DEV), torch.as_tensor(pos + prompt - 1, device=DEV)]
    d = ps.DeviceSubtree.create(layout=layout, u=1.0 - rng.random(n_seg), logits=logits,
                                tokens=tokens.contiguous(), V=V, alpha=alpha, tau=tau,
                                max_steps=30, entropy=True, rules=rules_of(seg, pos))
    d.step()
    torch.cuda.synchronize()
    for name, word in (("decoding", status), ("scoring", d.t["status"]), ("walk", d.t["wstatus"])):
        assert int(word.item()) == 0, (name, ps.dev_status_names(int(word.item())))
    return dict(layout=layout, drawn_lq=drawn_lq.cpu().numpy(), lq_y=d.t["lq_y"].cpu().numpy(),
                log_accept=d.t["log_accept"].cpu().numpy(), k_delta=int(d.t["k_delta"][0]),
                state=int(d.t["state_seg"][0]), entropy=d.t["entropy"].cpu().numpy())


if __name__ == "__main__":
    r = main()
    print("log q of the proposals as drawn :", np.round(r["drawn_lq"][1:], 2))
    print("and as scored                   :", np.round(r["lq_y"][1:], 2))
    print("log A                           :", np.round(r["log_accept"][1:], 2))
    print(f"transitions {r['k_delta']}, reached segment {r['state']}")
