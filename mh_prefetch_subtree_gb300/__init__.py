"""Python binding of libps (scoring and walking one prefetched subtree batch).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libps.so``; this module turns torch tensors into the C structs
of ``include/ps.h`` and calls the entry points of the same names.  There is
no CPU fallback: if the library is missing or fails to load, every call
raises.

Entry points (see include/ps.h for the contract):
    ps_score_workspace_bytes, ps_score_subtree, ps_score_rows,
    ps_assemble_subtree, ps_walk_subtree, ps_score_walk_subtree, ps_carry_state,
    ps_validate_subtree,
    ps_score_subtree_noalloc, ps_status_string, ps_version,
    ps_process_rows, ps_rules_workspace_bytes, ps_score_rows_rules, ps_head_rows,
    ps_linear_rows, ps_sample_rows, ps_score_rows_truncated
Convenience: ``make_batch``, ``make_score_out``, ``make_tree``,
``make_walk_out``, ``make_rules``, ``make_head``, ``make_linear``, ``make_sampling`` build
the structs from tensors;
``DeviceSubtree`` holds a whole batch on the GPU with its outputs and workspace.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libps.so")

PS_OK = 0
PS_FLAG_MASKED_LOGITS = 0x1
PS_ERR_INVALID_ARG, PS_ERR_INFEASIBLE, PS_ERR_BAD_TREE, PS_ERR_UNSUPPORTED = 1, 2, 3, 4
PS_ERR_CUDA, PS_ERR_TIMEOUT, PS_ERR_WORKSPACE = 5, 6, 7
PS_BF16, PS_F32 = 0, 1
PS_ACTS = {"none": 0, "cap": 1, "silu": 2, "gelu": 3}
PS_DEV_BITS = {
    0x01: "BAD_TOKEN", 0x02: "NONFINITE", 0x04: "INFEASIBLE", 0x08: "BAD_TREE",
    0x10: "BAD_LAYOUT", 0x20: "TIMEOUT", 0x40: "BAD_ROW_INDEX", 0x80: "BAD_UNIFORM",
    0x100: "BAD_RULES", 0x200: "BAD_SAMPLING",
}
PS_NODE_LEAF, PS_NODE_DEFERRED = -1, -2

_vp = ctypes.c_void_p


class PsSubtreeBatch(ctypes.Structure):
    _fields_ = [("V", ctypes.c_int32), ("T", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("n_chains", ctypes.c_int32), ("n_seg", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("n_rows", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("n_logit_rows", ctypes.c_int64),
                ("alpha", ctypes.c_double), ("tau", ctypes.c_double),
                ("eps", ctypes.c_double), ("chain_seg0", _vp), ("seg_row0", _vp), ("seg_cut", _vp), ("seg_src", _vp),
                ("logits", _vp), ("row_index", _vp), ("tokens", _vp),
                ("root_lp0", _vp), ("root_lq", _vp)]


class PsScoreOut(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("lp0", "lq", "lp_y", "lq_y", "lp_x", "lq_x",
                                   "log_ratio", "log_accept", "status", "entropy",
                                   "eps_class")]


class PsTree(ctypes.Structure):
    _fields_ = [("n_chains", ctypes.c_int32), ("n_nodes", ctypes.c_int32),
                ("n_seg", ctypes.c_int32), ("max_steps", ctypes.c_int32),
                ("chain_node0", _vp), ("chain_seg0", _vp), ("acc", _vp), ("rej", _vp),
                ("req", _vp), ("u", _vp)]


class PsWalkOut(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("state_seg", "end_node", "k_delta", "path", "status")]


class PsCarryIo(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("state_seg", "row_lp0", "row_lq", "row_entropy", "prev_lp0",
                                   "prev_lq", "prev_entropy", "next_lp0", "next_lq",
                                   "next_entropy", "loglik", "confidence", "status")]


class PsLogitRules(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_masks", ctypes.c_int32),
                ("n_tokens", ctypes.c_int64), ("n_bias", ctypes.c_int64),
                ("mask_ld", ctypes.c_int64)] + \
        [(n, _vp) for n in ("seq_begin", "seq_tokens", "seq_prompt", "repetition", "frequency",
                            "presence", "bias_begin", "bias_ids", "bias_values", "mask",
                            "row_seq", "row_len", "row_mask")]
    _rows = None        # rows that the row arrays hold, where make_rules has seen them


class PsSampling(ctypes.Structure):
    _rows = None                  # rows that row_set holds, where known
    _fields_ = [("n_sets", ctypes.c_int64), ("tau", _vp), ("top_k", _vp), ("top_p", _vp),
                ("min_p", _vp), ("row_set", _vp)]


class PsHead(ctypes.Structure):
    _fields_ = [("V", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("q", _vp), ("scales", _vp), ("zeros", _vp)]


class PsLinear(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("act", ctypes.c_int32),
                ("cap", ctypes.c_float), ("bias_dtype", ctypes.c_int32), ("w_ld", ctypes.c_int64),
                ("w", _vp), ("bias", _vp)]


class PsError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {ps_status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libps.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libps.so is not built ({LIB_PATH}); run "
                               "`python -m mh_prefetch_subtree_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.ps_score_workspace_bytes.argtypes = [ctypes.POINTER(PsSubtreeBatch)]
        L.ps_score_workspace_bytes.restype = ctypes.c_size_t
        L.ps_score_subtree.argtypes = [ctypes.POINTER(PsSubtreeBatch), ctypes.POINTER(PsScoreOut),
                                       _vp, ctypes.c_size_t, _vp]
        L.ps_score_subtree.restype = ctypes.c_int
        L.ps_score_rows.argtypes = [ctypes.POINTER(PsSubtreeBatch), _vp, _vp, _vp, _vp, _vp,
                                    ctypes.c_size_t, _vp]
        L.ps_score_rows.restype = ctypes.c_int
        L.ps_score_rows_multi.argtypes = [ctypes.POINTER(PsSubtreeBatch),
                                          ctypes.POINTER(ctypes.c_double), ctypes.c_int32,
                                          _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.ps_score_rows_multi.restype = ctypes.c_int
        L.ps_assemble_subtree.argtypes = [ctypes.POINTER(PsSubtreeBatch), _vp, _vp,
                                          ctypes.POINTER(PsScoreOut), _vp]
        L.ps_assemble_subtree.restype = ctypes.c_int
        L.ps_score_subtree_noalloc.argtypes = [ctypes.POINTER(PsSubtreeBatch),
                                               ctypes.POINTER(PsScoreOut), _vp]
        L.ps_score_subtree_noalloc.restype = ctypes.c_int
        L.ps_walk_subtree.argtypes = [ctypes.POINTER(PsTree), _vp, ctypes.POINTER(PsWalkOut), _vp]
        L.ps_walk_subtree.restype = ctypes.c_int
        L.ps_score_walk_subtree.argtypes = [ctypes.POINTER(PsSubtreeBatch), ctypes.POINTER(PsTree),
                                            ctypes.POINTER(PsScoreOut), ctypes.POINTER(PsWalkOut),
                                            _vp, ctypes.c_size_t, _vp]
        L.ps_score_walk_subtree.restype = ctypes.c_int
        L.ps_carry_state.argtypes = [ctypes.POINTER(PsSubtreeBatch), ctypes.POINTER(PsCarryIo),
                                     _vp]
        L.ps_carry_state.restype = ctypes.c_int
        i32p = ctypes.POINTER(ctypes.c_int32)
        L.ps_build_bfs_tree.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp,
                                        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32] + \
            [_vp] * 7 + [i32p, i32p, i32p]
        L.ps_build_bfs_tree.restype = ctypes.c_int
        L.ps_predictive_allocation.argtypes = [ctypes.c_int32, _vp, _vp, _vp, _vp,
                                               ctypes.c_int32, ctypes.POINTER(ctypes.c_double),
                                               _vp]
        L.ps_predictive_allocation.restype = ctypes.c_int
        L.ps_midpoint_branch_probability.argtypes = [ctypes.c_double, ctypes.c_double]
        L.ps_midpoint_branch_probability.restype = ctypes.c_double
        L.ps_validate_subtree.argtypes = [ctypes.POINTER(PsSubtreeBatch), ctypes.POINTER(PsTree),
                                          ctypes.c_char_p, ctypes.c_size_t]
        L.ps_validate_subtree.restype = ctypes.c_int
        L.ps_selftest_wait_timeout.argtypes = [ctypes.c_uint64, _vp, _vp]
        L.ps_selftest_wait_timeout.restype = ctypes.c_int
        L.ps_selftest_read.argtypes = [_vp, ctypes.c_size_t, _vp, _vp]
        L.ps_selftest_read.restype = ctypes.c_int
        L.ps_process_rows.argtypes = [ctypes.POINTER(PsLogitRules), ctypes.c_int32,
                                      ctypes.c_int32, ctypes.c_int64, _vp, ctypes.c_int64, _vp,
                                      ctypes.c_int64, _vp, _vp]
        L.ps_process_rows.restype = ctypes.c_int
        L.ps_rules_workspace_bytes.argtypes = [ctypes.POINTER(PsSubtreeBatch)]
        L.ps_rules_workspace_bytes.restype = ctypes.c_size_t
        L.ps_score_rows_rules.argtypes = [ctypes.POINTER(PsSubtreeBatch),
                                          ctypes.POINTER(PsLogitRules), _vp, _vp, _vp, _vp, _vp,
                                          ctypes.c_size_t, _vp]
        L.ps_score_rows_rules.restype = ctypes.c_int
        L.ps_linear_rows.argtypes = [ctypes.POINTER(PsLinear), _vp, ctypes.c_int64, ctypes.c_int32,
                                     _vp, ctypes.c_int64, _vp, ctypes.c_int64, ctypes.c_int32, _vp]
        L.ps_linear_rows.restype = ctypes.c_int
        L.ps_selftest_linear_wait.argtypes = L.ps_linear_rows.argtypes
        L.ps_selftest_linear_wait.restype = ctypes.c_int
        L.ps_sample_rows.argtypes = [ctypes.POINTER(PsSampling), ctypes.c_int32, ctypes.c_int32,
                                     ctypes.c_int64, _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp]
        L.ps_sample_rows.restype = ctypes.c_int
        L.ps_score_rows_truncated.argtypes = [ctypes.POINTER(PsSubtreeBatch),
                                              ctypes.POINTER(PsSampling), _vp, _vp, _vp, _vp, _vp]
        L.ps_score_rows_truncated.restype = ctypes.c_int
        L.ps_head_rows.argtypes = [ctypes.POINTER(PsHead), _vp, ctypes.c_int64, ctypes.c_int32,
                                   _vp, ctypes.c_int64, ctypes.c_int32, _vp]
        L.ps_head_rows.restype = ctypes.c_int
        L.ps_selftest_head_wait.argtypes = L.ps_head_rows.argtypes
        L.ps_selftest_head_wait.restype = ctypes.c_int
        L.ps_status_string.argtypes = [ctypes.c_int]
        L.ps_status_string.restype = ctypes.c_char_p
        L.ps_version.argtypes = []
        L.ps_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def ps_status_string(status: int) -> str:
    return lib().ps_status_string(int(status)).decode()


def ps_version() -> str:
    return lib().ps_version().decode()


def ps_score_workspace_bytes(batch: PsSubtreeBatch) -> int:
    return int(lib().ps_score_workspace_bytes(ctypes.byref(batch)))


def ps_score_subtree(batch: PsSubtreeBatch, out: PsScoreOut, workspace: torch.Tensor,
                     stream=None, check: bool = True) -> int:
    ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = lib().ps_score_subtree(ctypes.byref(batch), ctypes.byref(out), ws_ptr, ws_bytes,
                                _stream(stream, workspace))
    if check and st != PS_OK:
        raise PsError(st, "ps_score_subtree")
    return st


def ps_score_subtree_noalloc(batch: PsSubtreeBatch, out: PsScoreOut, stream=None,
                             check: bool = True) -> int:
    """Scoring for callers that cannot allocate device memory: no workspace
    argument; libps uses its own static device array (see include/ps.h for the
    row limit, the once-per-device set-up and why overlapping calls race)."""
    st = lib().ps_score_subtree_noalloc(ctypes.byref(batch), ctypes.byref(out),
                                        _stream(stream, None))
    if check and st != PS_OK:
        raise PsError(st, "ps_score_subtree_noalloc")
    return st


def ps_score_rows(batch: PsSubtreeBatch, lp0: torch.Tensor, lq: torch.Tensor,
                  status: torch.Tensor, workspace: torch.Tensor, stream=None,
                  check: bool = True, entropy: torch.Tensor | None = None) -> int:
    _need(lp0, torch.float64, "lp0")
    _need(lq, torch.float64, "lq")
    _need(entropy, torch.float64, "entropy", optional=True)
    _need(status, torch.int32, "status")
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().ps_score_rows(ctypes.byref(batch), _ptr(lp0), _ptr(lq), _ptr(entropy),
                             _ptr(status), _ptr(workspace), ws_bytes, _stream(stream, workspace))
    if check and st != PS_OK:
        raise PsError(st, "ps_score_rows")
    return st


def ps_score_rows_multi(batch: PsSubtreeBatch, taus, lp0: torch.Tensor, lq: torch.Tensor,
                        status: torch.Tensor, workspace: torch.Tensor, stream=None,
                        check: bool = True, entropy: torch.Tensor | None = None) -> int:
    """log p0 and log q_tau for several temperatures in one pass (each 1/tau
    in {1, 2, 4, 8}); lq is [len(taus), n_rows]."""
    taus = [float(t) for t in taus]
    _need(lp0, torch.float64, "lp0")
    _need(lq, torch.float64, "lq")
    _need(entropy, torch.float64, "entropy", optional=True)
    _need(status, torch.int32, "status")
    if len(lq.shape) != 2 or lq.shape[0] != len(taus) or lq.shape[1] != lp0.shape[0]:
        raise ValueError("lq must be [len(taus), n_rows]")
    arr = (ctypes.c_double * max(1, len(taus)))(*taus)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().ps_score_rows_multi(ctypes.byref(batch), arr, len(taus), _ptr(lp0), _ptr(lq),
                                   _ptr(entropy), _ptr(status), _ptr(workspace), ws_bytes,
                                   _stream(stream, workspace))
    if check and st != PS_OK:
        raise PsError(st, "ps_score_rows_multi")
    return st


def ps_selftest_wait_timeout(limit_ns: int, status: torch.Tensor, stream=None,
                             check: bool = True) -> int:
    """Diagnostic: a device wait that nothing completes gives up after limit_ns
    and sets PS_DEV_TIMEOUT in status (see include/ps.h)."""
    _need(status, torch.int32, "status")
    st = lib().ps_selftest_wait_timeout(int(limit_ns), _ptr(status), _stream(stream, status))
    if check and st != PS_OK:
        raise PsError(st, "ps_selftest_wait_timeout")
    return st


def ps_selftest_read(data: torch.Tensor, sink: torch.Tensor, stream=None,
                     check: bool = True) -> int:
    """Diagnostic: one plain streaming read of `data` (a contiguous device
    tensor, 16-byte aligned, a multiple of 16 bytes), folded into the int32
    `sink`; timing it gives the device's plain read rate (see include/ps.h)."""
    _need(sink, torch.int32, "sink")
    nbytes = data.numel() * data.element_size()
    st = lib().ps_selftest_read(_ptr(data), nbytes, _ptr(sink), _stream(stream, data))
    if check and st != PS_OK:
        raise PsError(st, "ps_selftest_read")
    return st


def ps_assemble_subtree(batch: PsSubtreeBatch, lp0: torch.Tensor, lq: torch.Tensor,
                        out: PsScoreOut, stream=None, check: bool = True) -> int:
    _need(lp0, torch.float64, "lp0")
    _need(lq, torch.float64, "lq")
    st = lib().ps_assemble_subtree(ctypes.byref(batch), _ptr(lp0), _ptr(lq), ctypes.byref(out),
                                   _stream(stream, lp0))
    if check and st != PS_OK:
        raise PsError(st, "ps_assemble_subtree")
    return st


def ps_walk_subtree(tree: PsTree, log_accept: torch.Tensor, out: PsWalkOut, stream=None,
                    check: bool = True) -> int:
    _need(log_accept, torch.float64, "log_accept")
    st = lib().ps_walk_subtree(ctypes.byref(tree), _ptr(log_accept), ctypes.byref(out),
                               _stream(stream, log_accept))
    if check and st != PS_OK:
        raise PsError(st, "ps_walk_subtree")
    return st


def ps_score_walk_subtree(batch: PsSubtreeBatch, tree: PsTree, out: PsScoreOut,
                          wout: PsWalkOut, workspace: torch.Tensor, stream=None,
                          check: bool = True) -> int:
    """Score, sum and walk one batch in one call (see include/ps.h)."""
    ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = lib().ps_score_walk_subtree(ctypes.byref(batch), ctypes.byref(tree), ctypes.byref(out),
                                     ctypes.byref(wout), ws_ptr, ws_bytes,
                                     _stream(stream, workspace))
    if check and st != PS_OK:
        raise PsError(st, "ps_score_walk_subtree")
    return st


def ps_carry_state(batch: PsSubtreeBatch, io: PsCarryIo, stream=None, check: bool = True) -> int:
    """The reached state's per-position values for the next round (see
    include/ps.h)."""
    st = lib().ps_carry_state(ctypes.byref(batch), ctypes.byref(io), _stream(stream, None))
    if check and st != PS_OK:
        raise PsError(st, "ps_carry_state")
    return st


def ps_process_rows(rules: PsLogitRules, logits: torch.Tensor, out: torch.Tensor,
                    status: torch.Tensor, V: int | None = None, stream=None,
                    check: bool = True) -> int:
    """out[r] = the rules applied to logits[r] (see include/ps.h); out may be
    logits itself.  V: ids of a row (default: the row length)."""
    dt = _row_dtype(logits, "logits")
    _need(out, logits.dtype, "out")
    _need(status, torch.int32, "status")
    shape, out_shape = logits.shape, out.shape
    if len(shape) != 2 or len(out_shape) != 2 or out_shape[0] != shape[0]:
        raise ValueError("logits and out must be [n_rows, ld] with the same n_rows")
    n_rows, ld = shape
    _need_rows(rules, n_rows)
    st = (_lib or lib()).ps_process_rows(rules, ld if V is None else V, dt, n_rows, _ptr(logits),
                                         ld, _ptr(out), out_shape[1], _ptr(status),
                                         _stream(stream, logits))
    if check and st != PS_OK:
        raise PsError(st, "ps_process_rows")
    return st


def ps_rules_workspace_bytes(batch: PsSubtreeBatch) -> int:
    return int(lib().ps_rules_workspace_bytes(ctypes.byref(batch)))


def ps_score_rows_rules(batch: PsSubtreeBatch, rules: PsLogitRules, lp0: torch.Tensor,
                        lq: torch.Tensor, status: torch.Tensor, workspace: torch.Tensor,
                        stream=None, check: bool = True,
                        entropy: torch.Tensor | None = None) -> int:
    """ps_score_rows under rules, without writing the processed rows; the
    workspace holds ps_rules_workspace_bytes(batch)."""
    _need(lp0, torch.float64, "lp0")
    _need(lq, torch.float64, "lq")
    _need(entropy, torch.float64, "entropy", optional=True)
    _need(status, torch.int32, "status")
    _need_rows(rules, batch.n_rows)
    st = (_lib or lib()).ps_score_rows_rules(batch, rules, _ptr(lp0), _ptr(lq), _ptr(entropy),
                                             _ptr(status), _ptr(workspace), workspace.nbytes,
                                             _stream(stream, workspace))
    if check and st != PS_OK:
        raise PsError(st, "ps_score_rows_rules")
    return st


def _linear_call(name: str, linear: PsLinear, x: torch.Tensor, out: torch.Tensor,
                 residual: torch.Tensor | None, stream, check: bool) -> int:
    _need(x, torch.bfloat16, "x")
    dt = _row_dtype(out, "out")
    shape, out_shape = x.shape, out.shape
    if len(shape) != 2 or len(out_shape) != 2 or out_shape[0] != shape[0]:
        raise ValueError("x and out must be matrices with the same number of rows")
    res_ld = 0
    if residual is not None:
        _need(residual, out.dtype, "residual")
        if residual.dim() != 2 or residual.shape[0] != shape[0]:
            raise ValueError("residual must be a matrix with as many rows as out")
        res_ld = residual.shape[1]
    st = getattr(_lib or lib(), name)(linear, _ptr(x), shape[1], shape[0], _ptr(residual), res_ld,
                                      _ptr(out), out_shape[1], dt, _stream(stream, out))
    if check and st != PS_OK:
        raise PsError(st, name)
    return st


def ps_linear_rows(linear: PsLinear, x: torch.Tensor, out: torch.Tensor,
                   residual: torch.Tensor | None = None, stream=None, check: bool = True) -> int:
    """out[:, :N] = act(x W^T + bias) + residual (see include/ps.h): x is [n_rows, >= K]
    bfloat16, out [n_rows, ld] bfloat16 or float32, residual None or of out's type; it may be
    out itself."""
    return _linear_call("ps_linear_rows", linear, x, out, residual, stream, check)


def ps_selftest_linear_wait(linear: PsLinear, x: torch.Tensor, out: torch.Tensor,
                            residual: torch.Tensor | None = None, stream=None, check: bool = True) -> int:
    """Diagnostic: ps_linear_rows with copies left out and short waits (see include/ps.h)."""
    return _linear_call("ps_selftest_linear_wait", linear, x, out, residual, stream, check)


def ps_sample_rows(sampling: PsSampling, logits: torch.Tensor, u: torch.Tensor,
                   tokens: torch.Tensor, status: torch.Tensor, V: int | None = None,
                   lp0: torch.Tensor | None = None, lq: torch.Tensor | None = None,
                   entropy: torch.Tensor | None = None, stream=None, check: bool = True) -> int:
    """Draws tokens[r] from the truncated distribution of logits[r] by u[r] (see
    include/ps.h).  V: ids of a row (default: the row length)."""
    dt = _row_dtype(logits, "logits")
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits must be [n_rows, ld]")
    n_rows, ld = shape
    _need_sets(sampling, n_rows)
    f64 = torch.float64
    st = (_lib or lib()).ps_sample_rows(
        sampling, ld if V is None else V, dt, n_rows, _ptr(logits), ld, _rows_ptr(u, f64, n_rows, "u"),
        _rows_ptr(tokens, torch.int32, n_rows, "tokens"),
        None if lp0 is None else _rows_ptr(lp0, f64, n_rows, "lp0"),
        None if lq is None else _rows_ptr(lq, f64, n_rows, "lq"),
        None if entropy is None else _rows_ptr(entropy, f64, n_rows, "entropy"),
        _rows_ptr(status, torch.int32, 1, "status"), _stream(stream, logits))
    if check and st != PS_OK:
        raise PsError(st, "ps_sample_rows")
    return st


def ps_score_rows_truncated(batch: PsSubtreeBatch, sampling: PsSampling, lp0: torch.Tensor,
                            lq: torch.Tensor, status: torch.Tensor, stream=None,
                            check: bool = True, entropy: torch.Tensor | None = None) -> int:
    """log p0 and log q of the rows' tokens, q truncated (see include/ps.h)."""
    n, f64 = batch.n_rows, torch.float64
    _need_sets(sampling, n)
    st = (_lib or lib()).ps_score_rows_truncated(
        batch, sampling, _rows_ptr(lp0, f64, n, "lp0"), _rows_ptr(lq, f64, n, "lq"),
        None if entropy is None else _rows_ptr(entropy, f64, n, "entropy"),
        _rows_ptr(status, torch.int32, 1, "status"), _stream(stream, lp0))
    if check and st != PS_OK:
        raise PsError(st, "ps_score_rows_truncated")
    return st


def _head_call(name: str, head: PsHead, hidden: torch.Tensor, logits: torch.Tensor, stream,
               check: bool) -> int:
    _need(hidden, torch.bfloat16, "hidden")
    dt = _row_dtype(logits, "logits")
    shape, out_shape = hidden.shape, logits.shape
    if len(shape) != 2 or len(out_shape) != 2 or out_shape[0] != shape[0]:
        raise ValueError("hidden and logits must be matrices with the same number of rows")
    st = getattr(_lib or lib(), name)(head, _ptr(hidden), shape[1], shape[0], _ptr(logits),
                                      out_shape[1], dt, _stream(stream, logits))
    if check and st != PS_OK:
        raise PsError(st, name)
    return st


def ps_head_rows(head: PsHead, hidden: torch.Tensor, logits: torch.Tensor, stream=None,
                 check: bool = True) -> int:
    """logits[:, :V] = hidden times the 4-bit head (see include/ps.h): hidden is
    [n_rows, >= K] bfloat16, logits [n_rows, ld] bfloat16 or float32."""
    return _head_call("ps_head_rows", head, hidden, logits, stream, check)


def ps_selftest_head_wait(head: PsHead, hidden: torch.Tensor, logits: torch.Tensor, stream=None,
                          check: bool = True) -> int:
    """Diagnostic: the many-row head kernel with weight copies left out (see include/ps.h)."""
    return _head_call("ps_selftest_head_wait", head, hidden, logits, stream, check)


def make_carry_io(*, state_seg, row_lp0, row_lq, next_lp0, next_lq, status, row_entropy=None,
                  prev_lp0=None, prev_lq=None, prev_entropy=None, next_entropy=None,
                  loglik=None, confidence=None) -> PsCarryIo:
    io = PsCarryIo()
    _need(state_seg, torch.int32, "state_seg")
    _need(status, torch.int32, "status")
    io.state_seg, io.status = _ptr(state_seg), _ptr(status)
    for name, x, opt in (("row_lp0", row_lp0, False), ("row_lq", row_lq, False),
                         ("row_entropy", row_entropy, True), ("prev_lp0", prev_lp0, True),
                         ("prev_lq", prev_lq, True), ("prev_entropy", prev_entropy, True),
                         ("next_lp0", next_lp0, False), ("next_lq", next_lq, False),
                         ("next_entropy", next_entropy, True), ("loglik", loglik, True),
                         ("confidence", confidence, True)):
        _need(x, torch.float64, name, optional=opt)
        setattr(io, name, _ptr(x))
    io._keep = (state_seg, row_lp0, row_lq, row_entropy, prev_lp0, prev_lq, prev_entropy,
                next_lp0, next_lq, next_entropy, loglik, confidence, status)
    return io


def ps_build_bfs_tree(T: int, n_pf: int, depth_cap: int | None, cuts) -> dict:
    """BFS request collection for one chain (host; see include/ps.h)."""
    cuts = np.ascontiguousarray(cuts, dtype=np.int32)
    n_cuts = int(cuts.shape[0])
    max_nodes, max_seg = 1 + 2 * n_cuts, n_pf + 1
    arr = {k: np.empty(max_nodes, np.int32) for k in ("acc", "rej", "req", "node_cut",
                                                      "deferred_cut")}
    seg = {k: np.empty(max_seg, np.int32) for k in ("seg_cut", "seg_src")}
    nn, ns, used = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    st = lib().ps_build_bfs_tree(int(T), int(n_pf), -1 if depth_cap is None else int(depth_cap),
                                 cuts.ctypes.data if n_cuts else None, n_cuts, max_nodes,
                                 max_seg, arr["acc"].ctypes.data, arr["rej"].ctypes.data,
                                 arr["req"].ctypes.data, arr["node_cut"].ctypes.data,
                                 arr["deferred_cut"].ctypes.data, seg["seg_cut"].ctypes.data,
                                 seg["seg_src"].ctypes.data, ctypes.byref(nn), ctypes.byref(ns),
                                 ctypes.byref(used))
    if st != PS_OK:
        raise PsError(st, "ps_build_bfs_tree")
    out = {k: v[:nn.value].copy() for k, v in arr.items()}
    out.update({k: v[:ns.value].copy() for k, v in seg.items()})
    out["cuts_used"] = used.value
    return out


def ps_predictive_allocation(acc, rej, candidate, h_acc, budget: int) -> tuple[float, np.ndarray]:
    """The eq. (19) dynamic program (host; see include/ps.h)."""
    acc = np.ascontiguousarray(acc, dtype=np.int32)
    rej = np.ascontiguousarray(rej, dtype=np.int32)
    cand = np.ascontiguousarray(candidate, dtype=np.uint8)
    h = np.ascontiguousarray(h_acc, dtype=np.float64)
    n = int(acc.shape[0])
    sel = np.zeros(n, np.uint8)
    val = ctypes.c_double()
    st = lib().ps_predictive_allocation(n, acc.ctypes.data, rej.ctypes.data, cand.ctypes.data,
                                        h.ctypes.data, int(budget), ctypes.byref(val),
                                        sel.ctypes.data)
    if st != PS_OK:
        raise PsError(st, "ps_predictive_allocation")
    return val.value, sel.astype(bool)


def ps_midpoint_branch_probability(p_accept: float, p_reject: float) -> float:
    return float(lib().ps_midpoint_branch_probability(float(p_accept), float(p_reject)))


def ps_validate_subtree(batch: PsSubtreeBatch | None, tree: PsTree | None) -> tuple[int, str]:
    buf = ctypes.create_string_buffer(256)
    st = lib().ps_validate_subtree(ctypes.byref(batch) if batch is not None else None,
                                   ctypes.byref(tree) if tree is not None else None, buf, 256)
    return int(st), buf.value.decode()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if not x.is_contiguous():
            raise ValueError("tensors passed to libps must be contiguous")
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        if not x.flags.c_contiguous:
            raise ValueError("arrays passed to libps must be C-contiguous")
        return x.ctypes.data
    raise TypeError(type(x))


def _rows_ptr(x, dtype: torch.dtype, n: int, name: str) -> int:
    """The address of a contiguous tensor of dtype with at least n elements."""
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if x.numel() < n:
        raise ValueError(f"{name} must hold {n} elements")
    if not x.is_contiguous():
        raise ValueError("tensors passed to libps must be contiguous")
    return x.data_ptr()


# the handle of a device's current stream without a Stream object for each call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, like: torch.Tensor | None):
    if stream is None:
        dev = like.device if like is not None else None
        if _raw_stream is not None and dev is not None and dev.index is not None:
            return _raw_stream(dev.index)
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_NP_OF = {torch.int32: np.int32, torch.int64: np.int64, torch.float64: np.float64,
          torch.int8: np.int8}


def _need(x, dtype: torch.dtype, name: str, optional: bool = False):
    if isinstance(x, torch.Tensor):
        if x.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    elif x is None:
        if not optional:
            raise ValueError(f"{name} is required")
    elif isinstance(x, np.ndarray):
        if x.dtype != _NP_OF[dtype]:
            raise TypeError(f"{name} must be {_NP_OF[dtype]}, got {x.dtype}")
    else:
        raise TypeError(f"{name}: tensor or ndarray expected")


def _row_dtype(x, name: str) -> int:
    if isinstance(x, torch.Tensor):
        if x.dtype == torch.bfloat16:
            return PS_BF16
        if x.dtype == torch.float32:
            return PS_F32
    raise TypeError(f"{name} must be a bf16 or f32 tensor")


def _need_rows(rules: PsLogitRules, n_rows: int) -> None:
    have = rules._rows
    if have is not None and have < n_rows:
        raise ValueError(f"the rules' row arrays hold {have} rows, {n_rows} are asked for")


def make_rules(*, seq_begin=None, seq_tokens=None, seq_prompt=None, repetition=None,
               frequency=None, presence=None, bias_begin=None, bias_ids=None, bias_values=None,
               mask=None, row_seq=None, row_len=None, row_mask=None) -> PsLogitRules:
    """Fill a ps_logit_rules from device tensors (see include/ps.h).  mask is
    [n_masks, words] int32 holding the 32-bit words; every argument may be left
    out where the C struct takes NULL."""
    i32 = (("seq_tokens", seq_tokens), ("seq_prompt", seq_prompt), ("bias_ids", bias_ids),
           ("mask", mask), ("row_seq", row_seq), ("row_len", row_len), ("row_mask", row_mask))
    i64 = (("seq_begin", seq_begin), ("bias_begin", bias_begin))
    f32 = (("repetition", repetition), ("frequency", frequency), ("presence", presence),
           ("bias_values", bias_values))
    u = PsLogitRules()
    for group, dt in ((i32, torch.int32), (i64, torch.int64), (f32, torch.float32)):
        for name, x in group:
            _need(x, dt, name, optional=True)
            setattr(u, name, _ptr(x))
    size = lambda x: 0 if x is None else int(x.shape[0])
    if seq_begin is None and any(x is not None for x in (seq_tokens, seq_prompt, repetition,
                                                         frequency, presence)):
        raise ValueError("a history and penalties need seq_begin")
    if (seq_begin is None) != (seq_tokens is None):
        raise ValueError("seq_begin and seq_tokens go together")
    if len({x is None for x in (bias_begin, bias_ids, bias_values)}) != 1:
        raise ValueError("bias_begin, bias_ids and bias_values go together")
    if bias_ids is not None and size(bias_ids) != size(bias_values):
        raise ValueError("bias_ids and bias_values must have the same length")
    per_seq = [x for x in (seq_begin, bias_begin) if x is not None]
    u.n_seqs = size(per_seq[0]) - 1 if per_seq else 0
    if any(size(x) < 1 for x in per_seq) or any(size(x) != size(per_seq[0]) for x in per_seq) or any(
            size(x) != u.n_seqs for x in (seq_prompt, repetition, frequency, presence)
            if x is not None):
        raise ValueError("the arrays of the sequences differ in length")
    u.n_tokens, u.n_bias = size(seq_tokens), size(bias_ids)
    if mask is not None:
        if mask.dim() != 2:
            raise ValueError("mask must be [n_masks, words]")
        u.n_masks, u.mask_ld = int(mask.shape[0]), int(mask.shape[1])
    elif row_mask is not None:
        raise ValueError("row_mask needs mask")
    rows = [size(x) for x in (row_seq, row_len, row_mask) if x is not None]
    u._rows = min(rows) if rows else None
    u._keep = (seq_begin, seq_tokens, seq_prompt, repetition, frequency, presence, bias_begin,
               bias_ids, bias_values, mask, row_seq, row_len, row_mask)
    return u


def _need_sets(sampling: PsSampling, n_rows: int) -> None:
    have = sampling._rows
    if have is not None and have < n_rows:
        raise ValueError(f"row_set holds {have} rows, {n_rows} are asked for")


def make_sampling(*, tau: torch.Tensor, top_k: torch.Tensor | None = None,
                  top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None,
                  row_set: torch.Tensor | None = None) -> PsSampling:
    """Fill a ps_sampling from device tensors (see include/ps.h): tau, top_p and min_p
    float32, top_k int32, one entry a set; row_set int32, one entry a row."""
    s = PsSampling()
    for name, x, dt in (("tau", tau, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32),
                        ("row_set", row_set, torch.int32)):
        _need(x, dt, name, optional=name != "tau")
        if x is not None and x.dim() != 1:
            raise ValueError(f"{name} must be a vector")
        setattr(s, name, _ptr(x))
    s.n_sets = int(tau.shape[0])
    if any(x is not None and x.shape[0] != s.n_sets for x in (top_k, top_p, min_p)):
        raise ValueError("the arrays of the sets differ in length")
    s._rows = None if row_set is None else int(row_set.shape[0])
    s._keep = (tau, top_k, top_p, min_p, row_set)
    return s


def make_linear(*, w: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
                cap: float = 0.0, K: int | None = None) -> PsLinear:
    """Fill a ps_linear from device tensors: w [N, >= K] bfloat16 (K: default all of a row),
    bias [N] bfloat16 or float32, act one of none, cap, silu, gelu."""
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise TypeError("w must be an [N, K] bfloat16 tensor")
    if act not in PS_ACTS:
        raise ValueError(f"act must be one of {', '.join(PS_ACTS)}")
    h = PsLinear()
    h.N, h.w_ld = int(w.shape[0]), int(w.shape[1])
    h.K = h.w_ld if K is None else int(K)
    h.act, h.cap = PS_ACTS[act], float(cap)
    if bias is not None:
        h.bias_dtype = _row_dtype(bias, "bias")
        if tuple(bias.shape) != (h.N,):
            raise ValueError("bias must be [N]")
    h.w, h.bias = _ptr(w), _ptr(bias)
    h._keep = (w, bias)
    return h


def make_head(*, q: torch.Tensor, scales: torch.Tensor, group: int,
              zeros: torch.Tensor | None = None) -> PsHead:
    """Fill a ps_head from device tensors: q [V, K/2] uint8, scales [V, K/group]
    bfloat16 or float32, zeros [V, K/group] uint8 or None."""
    if q.dtype != torch.uint8 or q.dim() != 2:
        raise TypeError("q must be a [V, K/2] uint8 tensor")
    h = PsHead()
    h.V, h.K, h.group = int(q.shape[0]), 2 * int(q.shape[1]), int(group)
    h.scale_dtype = _row_dtype(scales, "scales")
    shape = (h.V, h.K // h.group) if h.group > 0 and h.K % h.group == 0 else None
    if tuple(scales.shape) != shape:
        raise ValueError("scales must be [V, K / group]")
    if zeros is not None and (zeros.dtype != torch.uint8 or tuple(zeros.shape) != shape):
        raise ValueError("zeros must be [V, K / group] uint8")
    h.q, h.scales, h.zeros = _ptr(q), _ptr(scales), _ptr(zeros)
    h._keep = (q, scales, zeros)
    return h


def make_batch(*, V: int, T: int, alpha: float, tau: float, chain_seg0, seg_row0, seg_cut,
               seg_src, logits=None, tokens=None, row_index=None, n_rows: int | None = None,
               n_logit_rows: int | None = None, ld: int | None = None,
               dtype: int | None = None, eps: float = 0.01, root_lp0=None,
               root_lq=None, flags: int = 0) -> PsSubtreeBatch:
    """Fill a ps_subtree_batch from tensors (device for scoring, host for validation)."""
    _need(chain_seg0, torch.int32, "chain_seg0")
    _need(seg_row0, torch.int64, "seg_row0")
    _need(seg_cut, torch.int32, "seg_cut")
    _need(seg_src, torch.int32, "seg_src")
    _need(tokens, torch.int32, "tokens", optional=True)
    _need(row_index, torch.int64, "row_index", optional=True)
    _need(root_lp0, torch.float64, "root_lp0", optional=True)
    _need(root_lq, torch.float64, "root_lq", optional=True)
    b = PsSubtreeBatch()
    b.V, b.T = int(V), int(T)
    b.n_chains = int(chain_seg0.shape[0]) - 1
    b.n_seg = int(seg_cut.shape[0])
    b.flags = int(flags)
    if n_rows is None:
        n_rows = int(tokens.shape[0]) if tokens is not None else 0
    b.n_rows = int(n_rows)
    if logits is not None:
        if dtype is None:
            if logits.dtype == torch.bfloat16:
                dtype = PS_BF16
            elif logits.dtype == torch.float32:
                dtype = PS_F32
            else:
                raise TypeError(f"logits must be bf16 or f32, got {logits.dtype}")
        if ld is None:
            ld = int(logits.shape[-1])
        if n_logit_rows is None:
            n_logit_rows = int(logits.shape[0])
    b.dtype = int(PS_BF16 if dtype is None else dtype)
    if ld is None:                       # host-only validation: smallest legal stride
        per16 = 8 if b.dtype == PS_BF16 else 4
        ld = -(-int(V) // per16) * per16
    b.ld = int(ld)
    b.n_logit_rows = int(0 if n_logit_rows is None else n_logit_rows)
    b.alpha, b.tau, b.eps = float(alpha), float(tau), float(eps)
    b.chain_seg0, b.seg_row0 = _ptr(chain_seg0), _ptr(seg_row0)
    b.seg_cut, b.seg_src = _ptr(seg_cut), _ptr(seg_src)
    b.logits, b.row_index, b.tokens = _ptr(logits), _ptr(row_index), _ptr(tokens)
    b.root_lp0, b.root_lq = _ptr(root_lp0), _ptr(root_lq)
    b._keep = (chain_seg0, seg_row0, seg_cut, seg_src, logits, tokens, row_index, root_lp0,
               root_lq)
    return b


def make_score_out(*, log_accept, status, lp0=None, lq=None, lp_y=None, lq_y=None, lp_x=None,
                   lq_x=None, log_ratio=None, entropy=None, eps_class=None) -> PsScoreOut:
    o = PsScoreOut()
    for name, x in (("lp0", lp0), ("lq", lq), ("lp_y", lp_y), ("lq_y", lq_y), ("lp_x", lp_x),
                    ("lq_x", lq_x), ("log_ratio", log_ratio), ("log_accept", log_accept),
                    ("entropy", entropy)):
        _need(x, torch.float64, name, optional=name != "log_accept")
        setattr(o, name, _ptr(x))
    _need(status, torch.int32, "status")
    _need(eps_class, torch.int8, "eps_class", optional=True)
    o.status = _ptr(status)
    o.eps_class = _ptr(eps_class)
    o._keep = (lp0, lq, lp_y, lq_y, lp_x, lq_x, log_ratio, log_accept, status, entropy,
               eps_class)
    return o


def make_tree(*, chain_node0, chain_seg0, acc, rej, req, u, max_steps: int) -> PsTree:
    for name, x in (("chain_node0", chain_node0), ("chain_seg0", chain_seg0), ("acc", acc),
                    ("rej", rej), ("req", req)):
        _need(x, torch.int32, name)
    _need(u, torch.float64, "u")
    t = PsTree()
    t.n_chains = int(chain_node0.shape[0]) - 1
    t.n_nodes = int(acc.shape[0])
    t.n_seg = int(u.shape[0])
    t.max_steps = int(max_steps)
    t.chain_node0, t.chain_seg0 = _ptr(chain_node0), _ptr(chain_seg0)
    t.acc, t.rej, t.req, t.u = _ptr(acc), _ptr(rej), _ptr(req), _ptr(u)
    t._keep = (chain_node0, chain_seg0, acc, rej, req, u)
    return t


def make_walk_out(*, state_seg, end_node, k_delta, status, path=None) -> PsWalkOut:
    o = PsWalkOut()
    for name, x in (("state_seg", state_seg), ("end_node", end_node), ("k_delta", k_delta),
                    ("status", status)):
        _need(x, torch.int32, name)
        setattr(o, name, _ptr(x))
    _need(path, torch.int32, "path", optional=True)
    o.path = _ptr(path)
    o._keep = (state_seg, end_node, k_delta, status, path)
    return o


def dev_status_names(bits: int) -> list[str]:
    return [n for b, n in PS_DEV_BITS.items() if bits & b]


@dataclass
class DeviceSubtree:
    """A subtree batch resident on one GPU, with its outputs and workspace.

    Built from host arrays of the layout (chain_seg0, seg_row0, seg_cut,
    seg_src, chain_node0, acc, rej, req), the acceptance uniforms and the
    device tensors of logits and tokens.  With rules (make_rules, its row arrays
    in the order of the scored rows) the rows are scored under them; with sampling
    (make_sampling, row_set in that order) under its truncation, its temperatures taking the
    place of tau.  Under both, rows go through ps_process_rows first and are given here as
    processed, with sampling alone.
    """

    batch: PsSubtreeBatch
    tree: PsTree
    score_out: PsScoreOut
    walk_out: PsWalkOut
    workspace: torch.Tensor
    t: dict
    rules: PsLogitRules | None = None
    sampling: PsSampling | None = None

    @classmethod
    def create(cls, *, layout, u, logits: torch.Tensor, tokens: torch.Tensor, V: int,
               alpha: float, tau: float, max_steps: int, row_index: torch.Tensor | None = None,
               per_row: bool = True, sums: bool = True, path: bool = True,
               entropy: bool = False, eps: float | None = None,
               root_lp0: torch.Tensor | None = None,
               root_lq: torch.Tensor | None = None, flags: int = 0,
               rules: PsLogitRules | None = None,
               sampling: PsSampling | None = None) -> "DeviceSubtree":
        if rules is not None and sampling is not None:
            raise ValueError("process the rows with ps_process_rows, then score them with sampling alone")
        dev = logits.device
        i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).to(dev)
        t = dict(
            chain_seg0=i32(layout.chain_seg0),
            seg_row0=torch.as_tensor(np.ascontiguousarray(layout.seg_row0, dtype=np.int64)).to(dev),
            seg_cut=i32(layout.seg_cut), seg_src=i32(layout.seg_src),
            chain_node0=i32(layout.chain_node0), acc=i32(layout.acc), rej=i32(layout.rej),
            req=i32(layout.req),
            u=torch.as_tensor(np.ascontiguousarray(u, dtype=np.float64)).to(dev),
            logits=logits, tokens=tokens, row_index=row_index,
        )
        n_rows = int(layout.seg_row0[-1])
        n_seg = int(len(layout.seg_cut))
        n_chains = int(len(layout.chain_seg0)) - 1
        f64 = lambda n: torch.empty(n, dtype=torch.float64, device=dev)
        # their sums are formed from these
        per_row = per_row or rules is not None or sampling is not None
        t["lp0"] = f64(n_rows) if per_row else None
        t["lq"] = f64(n_rows) if per_row else None
        for k in ("lp_y", "lq_y", "lp_x", "lq_x", "log_ratio"):
            t[k] = f64(n_seg) if sums else None
        t["log_accept"] = f64(n_seg)
        t["entropy"] = f64(n_rows) if entropy else None
        t["eps_class"] = (torch.empty(n_seg, dtype=torch.int8, device=dev)
                          if eps is not None else None)
        t["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        t["wstatus"] = torch.zeros(1, dtype=torch.int32, device=dev)
        for k in ("state_seg", "end_node", "k_delta"):
            t[k] = torch.empty(n_chains, dtype=torch.int32, device=dev)
        t["path"] = (torch.empty(n_chains * (max_steps + 1), dtype=torch.int32, device=dev)
                     if path else None)
        batch = make_batch(V=V, T=layout.T, alpha=alpha, tau=tau, chain_seg0=t["chain_seg0"],
                           seg_row0=t["seg_row0"], seg_cut=t["seg_cut"], seg_src=t["seg_src"],
                           logits=logits, tokens=tokens, row_index=row_index, n_rows=n_rows,
                           eps=0.01 if eps is None else eps, root_lp0=root_lp0,
                           root_lq=root_lq, flags=flags)
        if rules is not None:
            _need_rows(rules, n_rows)
        if sampling is not None:
            _need_sets(sampling, n_rows)
        ws_bytes = (256 if sampling is not None else
                    ps_score_workspace_bytes(batch) if rules is None
                    else ps_rules_workspace_bytes(batch))
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        sout = make_score_out(log_accept=t["log_accept"], status=t["status"], lp0=t["lp0"],
                              lq=t["lq"], lp_y=t["lp_y"], lq_y=t["lq_y"], lp_x=t["lp_x"],
                              lq_x=t["lq_x"], log_ratio=t["log_ratio"], entropy=t["entropy"],
                              eps_class=t["eps_class"])
        tree = make_tree(chain_node0=t["chain_node0"], chain_seg0=t["chain_seg0"], acc=t["acc"],
                         rej=t["rej"], req=t["req"], u=t["u"], max_steps=max_steps)
        wout = make_walk_out(state_seg=t["state_seg"], end_node=t["end_node"],
                             k_delta=t["k_delta"], status=t["wstatus"], path=t["path"])
        return cls(batch=batch, tree=tree, score_out=sout, walk_out=wout, workspace=ws, t=t,
                   rules=rules, sampling=sampling)

    def score(self, stream=None) -> None:
        if self.rules is not None or self.sampling is not None:
            self.score_rows(stream)
            self.assemble(stream)
        else:
            ps_score_subtree(self.batch, self.score_out, self.workspace, stream)

    def score_rows(self, stream=None) -> None:
        """First half of score(): per-row log-probabilities into t['lp0'], t['lq']."""
        if self.rules is not None:
            ps_score_rows_rules(self.batch, self.rules, self.t["lp0"], self.t["lq"],
                                self.t["status"], self.workspace, stream,
                                entropy=self.t["entropy"])
        elif self.sampling is not None:
            ps_score_rows_truncated(self.batch, self.sampling, self.t["lp0"], self.t["lq"],
                                    self.t["status"], stream, entropy=self.t["entropy"])
        else:
            ps_score_rows(self.batch, self.t["lp0"], self.t["lq"], self.t["status"],
                          self.workspace, stream, entropy=self.t["entropy"])

    def assemble(self, stream=None) -> None:
        """Second half of score(): suffix sums and log A from t['lp0'], t['lq']."""
        ps_assemble_subtree(self.batch, self.t["lp0"], self.t["lq"], self.score_out, stream)

    def walk(self, stream=None) -> None:
        ps_walk_subtree(self.tree, self.t["log_accept"], self.walk_out, stream)

    def step(self, stream=None, fused: bool = True) -> None:
        """One pass of the whole path: score, sum and walk in one call
        (ps_score_walk_subtree), or with fused=False in two
        (ps_score_subtree, then ps_walk_subtree); under rules or truncation, in three."""
        if fused and self.rules is None and self.sampling is None:
            ps_score_walk_subtree(self.batch, self.tree, self.score_out, self.walk_out,
                                  self.workspace, stream)
        else:
            self.score(stream)
            self.walk(stream)

    def carry(self, prev: dict | None = None, stream=None) -> dict:
        """Per-position values of each chain's reached state for the next
        round (after step()); prev holds the current state's values for the
        positions below the root cut ("lp0", "lq" and optionally "entropy",
        each [n_chains, T])."""
        t = self.t
        n_chains = int(t["chain_seg0"].shape[0]) - 1
        T = int(self.batch.T)
        dev = t["log_accept"].device
        out = {k: torch.empty((n_chains, T), dtype=torch.float64, device=dev)
               for k in ("lp0", "lq")}
        ent = t.get("entropy") is not None
        if ent:
            out["entropy"] = torch.empty((n_chains, T), dtype=torch.float64, device=dev)
        out["loglik"] = torch.empty(n_chains, dtype=torch.float64, device=dev)
        if ent:
            out["confidence"] = torch.empty(n_chains, dtype=torch.float64, device=dev)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        prev = prev or {}
        io = make_carry_io(state_seg=t["state_seg"], row_lp0=t["lp0"], row_lq=t["lq"],
                           row_entropy=t.get("entropy"), prev_lp0=prev.get("lp0"),
                           prev_lq=prev.get("lq"), prev_entropy=prev.get("entropy"),
                           next_lp0=out["lp0"], next_lq=out["lq"],
                           next_entropy=out.get("entropy"), loglik=out["loglik"],
                           confidence=out.get("confidence"), status=status)
        ps_carry_state(self.batch, io, stream)
        out["status"] = status
        return out
