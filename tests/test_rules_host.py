"""Refusals of the entry points for rules and for the head: what the host can see
(no GPU calls), and the binding's own checks."""

import ctypes

import numpy as np
import pytest
import torch

import mh_prefetch_subtree_gb300 as ps


@pytest.fixture(scope="module", autouse=True)
def built():
    from mh_prefetch_subtree_gb300.build import build
    build()


def test_struct_sizes_match_the_header_layout():
    # int32 x2, int64 x3, 13 pointers; int32 x4, 3 pointers
    assert ctypes.sizeof(ps.PsLogitRules) == 2 * 4 + 3 * 8 + 13 * 8
    assert ctypes.sizeof(ps.PsHead) == 4 * 4 + 3 * 8


def rules(n_rows=4, V=100, **kw):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    d = dict(seq_begin=torch.tensor([0, 3, 5]), seq_tokens=i32(1, 2, 3, 4, 5),
             bias_begin=torch.tensor([0, 1, 2]), bias_ids=i32(3, 9),
             bias_values=torch.tensor([1.0, 2.0]),
             mask=torch.zeros(2, (V + 31) // 32, dtype=torch.int32),
             row_seq=torch.zeros(n_rows, dtype=torch.int32),
             row_len=torch.zeros(n_rows, dtype=torch.int32),
             row_mask=torch.zeros(n_rows, dtype=torch.int32))
    d.update(kw)
    return ps.make_rules(**d)


def process(u, x=None, out=None, V=100, st=True):
    x = torch.zeros(4, 104, dtype=torch.bfloat16) if x is None else x
    out = torch.zeros_like(x) if out is None else out
    return ps.ps_process_rows(u, x, out, torch.zeros(1, dtype=torch.int32), V=V, stream=0,
                              check=False)


def raw_process(u, **kw):
    """The C call with single arguments replaced."""
    x = torch.zeros(4, 104, dtype=torch.bfloat16)
    y = torch.zeros(4, 104, dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32)
    a = dict(rules=ctypes.byref(u) if u is not None else None, V=100, dtype=0, n=4,
             logits=x.data_ptr(), ld=104, out=y.data_ptr(), out_ld=104, status=st.data_ptr())
    a.update({k: (v(x, y) if callable(v) else v) for k, v in kw.items()})
    return ps.lib().ps_process_rows(a["rules"], a["V"], a["dtype"], a["n"], a["logits"], a["ld"],
                                    a["out"], a["out_ld"], a["status"], None)


def test_process_refusals():
    u = rules()
    # all host checks pass: host memory is then refused as not being the device's
    assert raw_process(u) == 1
    assert raw_process(None) == 1
    assert raw_process(u, dtype=2) == 4
    for bad in (dict(V=0), dict(n=-1), dict(logits=None), dict(out=None), dict(status=None),
                dict(ld=96), dict(ld=101), dict(out_ld=99), dict(ld=1 << 41),
                dict(logits=lambda x, y: x.data_ptr() + 2), dict(out=lambda x, y: y.data_ptr() + 8),
                dict(V=1 << 30, ld=1 << 30, out_ld=1 << 30)):
        assert raw_process(u, **bad) == 1, bad
    # overlapping, but not the same array
    assert raw_process(u, out=lambda x, y: x.data_ptr() + 16) == 1
    assert raw_process(u, out=lambda x, y: x.data_ptr(), out_ld=112) == 1
    assert raw_process(u, n=0) == 0
    assert raw_process(u, n=0, dtype=9) == 4


@pytest.mark.parametrize("field,value", [
    ("n_seqs", -1), ("n_masks", -1), ("n_tokens", -1), ("n_bias", -1), ("mask_ld", 3),
    ("seq_tokens", None), ("bias_ids", None), ("bias_values", None)])
def test_rules_refusals(field, value):
    u = rules()
    setattr(u, field, value)
    # n = 0 does not reach the device: only the rules can be refused
    assert raw_process(u, n=0) == 1


def test_rules_without_row_arrays_need_enough_sequences_and_masks():
    x = dict(row_seq=None, row_len=None)
    assert raw_process(rules(**x)) == 1                   # two sequences, four rows
    u = rules(row_mask=None)
    assert raw_process(u) == 1                            # two masks, four rows


def test_score_refusals():
    x = torch.zeros(4, 104, dtype=torch.bfloat16)
    tok = torch.zeros(4, dtype=torch.int32)
    a = lambda *v: torch.tensor(v)
    b = ps.make_batch(V=100, T=4, alpha=1.0, tau=0.5, chain_seg0=a(0, 1).int(),
                      seg_row0=a(0, 4), seg_cut=a(0).int(), seg_src=a(-1).int(), logits=x,
                      tokens=tok)
    f = torch.zeros(4, dtype=torch.float64)
    st = torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    al = (-ws.data_ptr()) % 256
    ws = ws[al:]

    def call(u, w=ws):
        return ps.ps_score_rows_rules(b, u, f, f, st, w, stream=0, check=False)

    need = ps.ps_rules_workspace_bytes(b)
    assert 0 < need <= ws.numel()
    assert call(rules()) == 1                             # host memory
    assert call(rules(), ws[:need - 1]) == 7
    assert call(rules(), ws[8:]) == 7
    u = rules()
    u.mask_ld = 1
    assert call(u) == 1
    b.tau = 0.0
    assert call(rules()) == 1
    b.tau, b.dtype = 0.5, 5
    assert call(rules()) == 4
    with pytest.raises(ValueError):
        b.dtype = 0
        call(rules(n_rows=3))


def test_binding_checks_rules():
    with pytest.raises(TypeError):
        rules(seq_tokens=torch.zeros(5, dtype=torch.int64))
    with pytest.raises(TypeError):
        rules(bias_values=torch.zeros(2, dtype=torch.float64))
    for bad in (dict(seq_tokens=None), dict(bias_ids=None), dict(seq_begin=None),
                dict(bias_begin=torch.tensor([0, 1, 2, 2])), dict(mask=None),
                dict(mask=torch.zeros(8, dtype=torch.int32)),
                dict(bias_values=torch.zeros(1)),
                dict(repetition=torch.ones(3))):
        with pytest.raises(ValueError):
            rules(**bad)
    x = torch.zeros(4, 104, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        process(rules(), x, torch.zeros(3, 104, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        process(rules(), x, torch.zeros(4, 104))
    with pytest.raises(TypeError):
        process(rules(), x.half())
    with pytest.raises(ValueError):
        process(rules(), torch.zeros(4, 208, dtype=torch.bfloat16)[:, ::2])
    with pytest.raises(ValueError):
        process(rules(n_rows=2), x)


def head(V=20, K=64, group=32, scale=torch.float32, zeros=True):
    return ps.make_head(q=torch.zeros(V, K // 2, dtype=torch.uint8),
                        scales=torch.zeros(V, K // group, dtype=scale), group=group,
                        zeros=torch.zeros(V, K // group, dtype=torch.uint8) if zeros else None)


def raw_head(h, **kw):
    hid = torch.zeros(2, 64, dtype=torch.bfloat16)
    out = torch.zeros(2, 24, dtype=torch.float32)
    a = dict(hidden=hid.data_ptr(), hidden_ld=64, n=2, logits=out.data_ptr(), ld=24, dtype=1)
    a.update({k: (v(hid, out) if callable(v) else v) for k, v in kw.items()})
    return ps.lib().ps_head_rows(ctypes.byref(h) if h is not None else None, a["hidden"],
                                 a["hidden_ld"], a["n"], a["logits"], a["ld"], a["dtype"], None)


def test_head_refusals():
    h = head()
    assert raw_head(h) == 1                               # host memory
    assert raw_head(h, n=0) == 0
    assert raw_head(None) == 1
    assert raw_head(h, dtype=2) == 4
    for bad in (dict(n=-1), dict(hidden=None), dict(hidden_ld=56), dict(hidden_ld=65),
                dict(logits=None), dict(ld=16), dict(ld=23), dict(hidden=lambda a, b: a.data_ptr() + 2),
                dict(logits=lambda a, b: b.data_ptr() + 4)):
        assert raw_head(h, **bad) == 1, bad
    for field, value, want in (("V", 0, 1), ("K", 0, 1), ("K", 48, 1), ("group", 16, 4),
                               ("group", 96, 4), ("group", 0, 4), ("group", 192, 4),
                               ("scale_dtype", 3, 4), ("q", None, 1), ("scales", None, 1)):
        h = head()
        setattr(h, field, value)
        assert raw_head(h, n=0) == want, (field, value)


def test_binding_checks_head():
    with pytest.raises(TypeError):
        ps.make_head(q=torch.zeros(4, 32, dtype=torch.int8), scales=torch.zeros(4, 2), group=32)
    with pytest.raises(TypeError):
        head(scale=torch.float16)
    with pytest.raises(ValueError):
        ps.make_head(q=torch.zeros(4, 32, dtype=torch.uint8), scales=torch.zeros(4, 1), group=32)
    with pytest.raises(ValueError):
        ps.make_head(q=torch.zeros(4, 32, dtype=torch.uint8), scales=torch.zeros(4, 2), group=32,
                     zeros=torch.zeros(4, 1, dtype=torch.uint8))
    h = head()
    with pytest.raises(TypeError):
        ps.ps_head_rows(h, torch.zeros(2, 64), torch.zeros(2, 24), stream=0)
    with pytest.raises(ValueError):
        ps.ps_head_rows(h, torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(3, 24), stream=0)
