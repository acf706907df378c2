"""ctypes binding of libssv (include/ssv.h).  Argument marshalling only:
every step of the verification pass runs in the library's CUDA kernels.
PyTorch supplies device memory and streams.

The library is loaded from this package's ``lib/libssv.so`` (built in-tree
by ``build.build()``).  If it is missing every call raises ``SsvError``;
there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from contextlib import nullcontext
from typing import Optional

import numpy as np

from .build import LIB

SSV_OK, SSV_ERR_INVALID, SSV_ERR_UNSUPPORTED, SSV_ERR_CUDA = 0, 1, 2, 3
SSV_ERR_TIMEOUT, SSV_ERR_BAD_TAU, SSV_ERR_WORKSPACE, SSV_ERR_NOT_FINITE = 4, 5, 6, 7
SSV_ERR_NO_PAGES = 8
SSV_F32, SSV_BF16 = 0, 1
ARGMAX, GUMBEL, REJECT, GUMBEL_GEN = 0, 1, 2, 3

#: every symbol include/ssv.h declares
EXPORTS = ("ssv_rope_copy", "ssv_verify_attn_workspace", "ssv_verify_attn", "ssv_verify_step", "ssv_accept_workspace",
           "ssv_accept", "ssv_accept_noalloc", "ssv_commit", "ssv_lmhead_accept_workspace", "ssv_lmhead_accept",
           "ssv_get_status", "ssv_status_string", "ssv_version", "ssv_bench", "ssv_set_fault_injection",
           "ssv_tree_verify_attn_workspace", "ssv_tree_verify_attn", "ssv_tree_accept_workspace", "ssv_tree_accept",
           "ssv_stream_read", "ssv_page_plan", "ssv_norm_rope_copy", "ssv_verify_attn_fp8_workspace",
           "ssv_verify_attn_fp8", "ssv_commit_fp8", "ssv_logprobs", "ssv_distill", "ssv_distill_backward")
RENORM, REST = 0, 1
FAULT_NONE, FAULT_ATTN, FAULT_ACCEPT, FAULT_LMHEAD = 0, 1, 2, 3


class SsvError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} (code {code})")


class SeqC(C.Structure):
    _fields_ = [("cache_len", C.c_int32), ("new_len", C.c_int32), ("block", C.c_int32),
                ("q_off", C.c_int32), ("kv_off", C.c_int32), ("tau_off", C.c_int32)]


class RopeArgs(C.Structure):
    _fields_ = [("q_in", C.c_void_p), ("k_in", C.c_void_p), ("q_out", C.c_void_p), ("k_out", C.c_void_p),
                ("dtype", C.c_int), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("d", C.c_int32),
                ("base", C.c_double), ("seqs", C.c_void_p), ("batch", C.c_int32), ("total_rows", C.c_int32),
                ("positions", C.c_void_p), ("dev_status", C.c_void_p)]


class AttnArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k_cache", C.c_void_p), ("v_cache", C.c_void_p), ("k_new", C.c_void_p),
                ("v_new", C.c_void_p), ("o", C.c_void_p), ("in_dtype", C.c_int), ("out_dtype", C.c_int),
                ("Hq", C.c_int32), ("Hkv", C.c_int32), ("d", C.c_int32), ("scale", C.c_float),
                ("seqs", C.c_void_p), ("batch", C.c_int32), ("tau", C.c_void_p), ("total_rows", C.c_int32),
                ("total_cache", C.c_int32), ("total_slots", C.c_int32), ("max_cache", C.c_int32),
                ("max_new", C.c_int32), ("max_block", C.c_int32), ("dev_status", C.c_void_p)]


class AcceptArgs(C.Structure):
    _fields_ = [("mode", C.c_int), ("T", C.c_float), ("V", C.c_int32), ("batch", C.c_int32),
                ("total_slots", C.c_int32), ("max_block", C.c_int32), ("logits_dtype", C.c_int),
                ("logits", C.c_void_p), ("draft_logits", C.c_void_p), ("draft_tokens", C.c_void_p),
                ("tau", C.c_void_p), ("block", C.c_void_p), ("gamma", C.c_void_p), ("slot_off", C.c_void_p),
                ("noise", C.c_void_p), ("n_noise_rows", C.c_int32), ("noise_row", C.c_void_p),
                ("u_accept", C.c_void_p), ("u_sample", C.c_void_p), ("n_acc", C.c_void_p),
                ("n_out", C.c_void_p), ("tokens", C.c_void_p), ("dev_status", C.c_void_p),
                ("noise_seed", C.c_uint64)]


class CommitArgs(C.Structure):
    _fields_ = [("k_new", C.c_void_p), ("v_new", C.c_void_p), ("k_dst", C.c_void_p), ("v_dst", C.c_void_p),
                ("dtype", C.c_int), ("Hkv", C.c_int32), ("d", C.c_int32), ("seqs", C.c_void_p),
                ("batch", C.c_int32), ("tau", C.c_void_p), ("n_acc", C.c_void_p), ("dst_off", C.c_void_p),
                ("dst_cap", C.c_void_p), ("new_len", C.c_void_p), ("total_rows", C.c_int32),
                ("total_slots", C.c_int32), ("dst_rows", C.c_int32), ("dev_status", C.c_void_p)]


class TreeAttnArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k_cache", C.c_void_p), ("v_cache", C.c_void_p), ("k_new", C.c_void_p),
                ("v_new", C.c_void_p), ("o", C.c_void_p), ("in_dtype", C.c_int), ("out_dtype", C.c_int),
                ("Hq", C.c_int32), ("Hkv", C.c_int32), ("d", C.c_int32), ("scale", C.c_float), ("seqs", C.c_void_p),
                ("batch", C.c_int32), ("parent", C.c_void_p), ("pos", C.c_void_p), ("total_q", C.c_int32),
                ("total_k", C.c_int32), ("total_cache", C.c_int32), ("total_edges", C.c_int32),
                ("total_out", C.c_int32), ("max_cache", C.c_int32), ("dev_status", C.c_void_p)]


class TreeAcceptArgs(C.Structure):
    _fields_ = [("mode", C.c_int), ("T", C.c_float), ("V", C.c_int32), ("seqs", C.c_void_p), ("batch", C.c_int32),
                ("logits_dtype", C.c_int), ("logits", C.c_void_p), ("parent", C.c_void_p), ("pos", C.c_void_p),
                ("token", C.c_void_p), ("total_edges", C.c_int32), ("total_out", C.c_int32),
                ("noise", C.c_void_p), ("n_noise_rows", C.c_int32), ("noise_row", C.c_void_p),
                ("pos_off", C.c_void_p), ("total_positions", C.c_int32), ("n_acc", C.c_void_p), ("path", C.c_void_p),
                ("emit_pos", C.c_void_p), ("emit_tok", C.c_void_p), ("dev_status", C.c_void_p)]


class FaultInjection(C.Structure):
    _fields_ = [("kernel", C.c_int), ("skip", C.c_int32), ("wait_budget_cycles", C.c_int64)]


class LmheadArgs(C.Structure):
    _fields_ = [("mode", C.c_int), ("T", C.c_float), ("V", C.c_int32), ("hidden", C.c_int32),
                ("batch", C.c_int32), ("total_slots", C.c_int32), ("hidden_states", C.c_void_p),
                ("lm_head", C.c_void_p), ("draft_tokens", C.c_void_p), ("tau", C.c_void_p), ("block", C.c_void_p),
                ("gamma", C.c_void_p), ("slot_off", C.c_void_p), ("noise", C.c_void_p),
                ("n_noise_rows", C.c_int32), ("noise_row", C.c_void_p), ("n_acc", C.c_void_p),
                ("n_out", C.c_void_p), ("tokens", C.c_void_p), ("dev_status", C.c_void_p)]


class PagePlanArgs(C.Structure):
    _fields_ = [("cache_len", C.c_void_p), ("new_len", C.c_void_p), ("block", C.c_void_p), ("held", C.c_void_p),
                ("pages", C.c_void_p), ("free_list", C.c_void_p), ("n_free", C.c_void_p), ("batch", C.c_int32),
                ("max_pages", C.c_int32), ("page_size", C.c_int32), ("n_pages", C.c_int32),
                ("total_rows", C.c_int32), ("seqs", C.c_void_p), ("slot_map", C.c_void_p),
                ("slot_off", C.c_void_p), ("held_out", C.c_void_p), ("n_free_out", C.c_void_p),
                ("dev_status", C.c_void_p)]


class NormRopeArgs(C.Structure):
    _fields_ = [("q_in", C.c_void_p), ("k_in", C.c_void_p), ("q_out", C.c_void_p), ("k_out", C.c_void_p),
                ("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("q_in_stride", C.c_int64),
                ("k_in_stride", C.c_int64), ("q_out_stride", C.c_int64), ("k_out_stride", C.c_int64),
                ("dtype", C.c_int), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("d", C.c_int32), ("eps", C.c_float),
                ("base", C.c_double), ("seqs", C.c_void_p), ("batch", C.c_int32), ("total_rows", C.c_int32),
                ("positions", C.c_void_p), ("dev_status", C.c_void_p)]


class AttnFp8Args(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k_cache", C.c_void_p), ("v_cache", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("pages", C.c_void_p), ("k_new", C.c_void_p), ("v_new", C.c_void_p),
                ("o", C.c_void_p), ("k_stride", C.c_int64), ("v_stride", C.c_int64), ("Hq", C.c_int32),
                ("Hkv", C.c_int32), ("d", C.c_int32), ("page_size", C.c_int32), ("n_pages", C.c_int32),
                ("table_len", C.c_int32), ("scale", C.c_float), ("seqs", C.c_void_p), ("batch", C.c_int32),
                ("tau", C.c_void_p), ("total_rows", C.c_int32), ("total_slots", C.c_int32),
                ("max_cache", C.c_int32), ("max_new", C.c_int32), ("max_block", C.c_int32),
                ("dev_status", C.c_void_p)]


class CommitFp8Args(C.Structure):
    _fields_ = [("k_new", C.c_void_p), ("v_new", C.c_void_p), ("k_cache", C.c_void_p), ("v_cache", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p), ("pages", C.c_void_p), ("k_stride", C.c_int64),
                ("v_stride", C.c_int64), ("dtype", C.c_int), ("Hkv", C.c_int32), ("d", C.c_int32),
                ("page_size", C.c_int32), ("n_pages", C.c_int32), ("table_len", C.c_int32), ("seqs", C.c_void_p),
                ("batch", C.c_int32), ("tau", C.c_void_p), ("n_acc", C.c_void_p), ("new_len", C.c_void_p),
                ("total_rows", C.c_int32), ("total_slots", C.c_int32), ("max_new", C.c_int32),
                ("max_block", C.c_int32), ("dev_status", C.c_void_p), ("cache_len", C.c_void_p)]


class LogprobsArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("logits_stride", C.c_int64), ("dtype", C.c_int), ("V", C.c_int32),
                ("total_rows", C.c_int32), ("rows", C.c_void_p), ("tokens", C.c_void_p), ("n", C.c_int32),
                ("top_k", C.c_int32), ("T", C.c_float), ("logprob", C.c_void_p), ("rank", C.c_void_p),
                ("entropy", C.c_void_p), ("lse", C.c_void_p), ("top_logprob", C.c_void_p),
                ("top_token", C.c_void_p), ("dev_status", C.c_void_p)]


class DistillArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("logits_stride", C.c_int64), ("dtype", C.c_int), ("V", C.c_int32),
                ("n", C.c_int32), ("K", C.c_int32), ("teacher_token", C.c_void_p), ("teacher_logprob", C.c_void_p),
                ("T", C.c_float), ("mode", C.c_int), ("weight", C.c_void_p), ("loss", C.c_void_p),
                ("stats", C.c_void_p), ("grad_loss", C.c_void_p), ("grad", C.c_void_p), ("grad_stride", C.c_int64),
                ("dev_status", C.c_void_p)]


_lib = None


def lib():
    """Load libssv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise SsvError(SSV_ERR_UNSUPPORTED, f"libssv not built ({LIB} missing; run __graft_entry__.build())")
        L = C.CDLL(LIB)
        vp, sz = C.c_void_p, C.c_size_t
        L.ssv_rope_copy.argtypes = [C.POINTER(RopeArgs), vp]
        L.ssv_verify_attn_workspace.argtypes = [C.POINTER(AttnArgs), C.POINTER(sz)]
        L.ssv_verify_attn.argtypes = [C.POINTER(AttnArgs), vp, sz, vp]
        L.ssv_accept_workspace.argtypes = [C.POINTER(AcceptArgs), C.POINTER(sz)]
        L.ssv_accept.argtypes = [C.POINTER(AcceptArgs), vp, sz, vp]
        L.ssv_accept_noalloc.argtypes = [C.POINTER(AcceptArgs), vp]
        L.ssv_commit.argtypes = [C.POINTER(CommitArgs), vp]
        L.ssv_lmhead_accept_workspace.argtypes = [C.POINTER(LmheadArgs), C.POINTER(sz)]
        L.ssv_lmhead_accept.argtypes = [C.POINTER(LmheadArgs), vp, sz, vp]
        L.ssv_verify_step.argtypes = [C.POINTER(RopeArgs), C.POINTER(AttnArgs), vp, sz, C.POINTER(AcceptArgs), vp,
                                      sz, vp]
        L.ssv_get_status.argtypes = [vp, vp]
        L.ssv_status_string.argtypes = [C.c_int]
        L.ssv_status_string.restype = C.c_char_p
        L.ssv_version.restype = C.c_char_p
        L.ssv_bench.argtypes = [C.c_char_p, C.c_int32, C.c_char_p, sz]
        L.ssv_stream_read.argtypes = [vp, sz, vp, vp]
        L.ssv_set_fault_injection.argtypes = [C.POINTER(FaultInjection)]
        L.ssv_tree_verify_attn_workspace.argtypes = [C.POINTER(TreeAttnArgs), C.POINTER(sz)]
        L.ssv_tree_verify_attn.argtypes = [C.POINTER(TreeAttnArgs), vp, sz, vp]
        L.ssv_tree_accept_workspace.argtypes = [C.POINTER(TreeAcceptArgs), C.POINTER(sz)]
        L.ssv_tree_accept.argtypes = [C.POINTER(TreeAcceptArgs), vp, sz, vp]
        L.ssv_page_plan.argtypes = [C.POINTER(PagePlanArgs), vp]
        L.ssv_norm_rope_copy.argtypes = [C.POINTER(NormRopeArgs), vp]
        L.ssv_verify_attn_fp8_workspace.argtypes = [C.POINTER(AttnFp8Args), C.POINTER(sz)]
        L.ssv_verify_attn_fp8.argtypes = [C.POINTER(AttnFp8Args), vp, sz, vp]
        L.ssv_commit_fp8.argtypes = [C.POINTER(CommitFp8Args), vp]
        L.ssv_logprobs.argtypes = [C.POINTER(LogprobsArgs), vp]
        L.ssv_distill.argtypes = [C.POINTER(DistillArgs), vp]
        L.ssv_distill_backward.argtypes = [C.POINTER(DistillArgs), vp]
        for name in ("ssv_rope_copy", "ssv_verify_attn_workspace", "ssv_verify_attn", "ssv_verify_step",
                     "ssv_accept_workspace", "ssv_accept", "ssv_accept_noalloc", "ssv_commit",
                     "ssv_lmhead_accept_workspace", "ssv_lmhead_accept", "ssv_get_status", "ssv_bench",
                     "ssv_set_fault_injection", "ssv_tree_verify_attn_workspace", "ssv_tree_verify_attn",
                     "ssv_tree_accept_workspace", "ssv_tree_accept", "ssv_stream_read", "ssv_page_plan",
                     "ssv_norm_rope_copy", "ssv_verify_attn_fp8_workspace", "ssv_verify_attn_fp8",
                     "ssv_commit_fp8", "ssv_logprobs", "ssv_distill", "ssv_distill_backward"):
            getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    try:
        return lib().ssv_status_string(int(code)).decode()
    except SsvError:
        return "libssv unavailable"


def version() -> str:
    return lib().ssv_version().decode()


def _check(code: int, what: str):
    if code != SSV_OK:
        raise SsvError(code, what)


# ---------------------------------------------------------------------------
# torch plumbing
# ---------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _on(stream):
    """Where a call makes its outputs and its scratch: on the stream that it
    runs on.  They are then filled in that stream's order, and their memory goes
    back to that stream's allocations; like any tensor of that stream they are
    waited for before another one uses them."""
    return nullcontext() if stream is None else _torch().cuda.stream(stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SSV_F32
    if t.dtype == torch.bfloat16:
        return SSV_BF16
    raise SsvError(SSV_ERR_INVALID, f"unsupported dtype {t.dtype}")


class Batch:
    """A packed batch: host ssv_seq table + device copy + the bounds the library needs."""

    def __init__(self, seqs: np.ndarray, device="cuda"):
        torch = _torch()
        self.host = np.ascontiguousarray(np.asarray(seqs, dtype=np.int32).reshape(-1, 6))
        self.dev = torch.from_numpy(self.host.copy()).to(device)
        h = self.host
        self.batch = int(h.shape[0])
        self.total_rows = int(np.sum(h[:, 1] + 2 * h[:, 2])) if self.batch else 0
        self.total_cache = int(np.sum(h[:, 0])) if self.batch else 0
        self.total_slots = int(np.sum(h[:, 2])) if self.batch else 0
        self.max_cache = int(h[:, 0].max()) if self.batch else 0
        self.max_new = int(h[:, 1].max()) if self.batch else 0
        self.max_block = int(h[:, 2].max()) if self.batch else 1

    @classmethod
    def from_device(cls, seqs, total_rows: int, total_slots: int, max_cache: int, max_new: int, max_block: int):
        """A batch whose table exists on the device only (int32 [batch, 6], as
        page_plan writes it), with bounds that the caller states: the rows
        packed, the slots, and the largest C, N and B that any record may
        have.  For the operators over the paged cache."""
        x = cls.__new__(cls)
        x.host, x.dev, x.batch = None, seqs, seqs.shape[0]
        x.total_rows, x.total_cache, x.total_slots = total_rows, 0, total_slots
        x.max_cache, x.max_new, x.max_block = max_cache, max_new, max_block
        return x


def _workspace(nbytes: int, device, ws=None):
    torch = _torch()
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise SsvError(SSV_ERR_WORKSPACE, "workspace")
        return ws
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def rope_args(q, k, batch: Batch, base: float = 10000.0, q_out=None, k_out=None, positions=None, dev_status=None):
    """positions: optional int32 [rows] device table (fresh rows and data rows
    at their entries, mask rows at their data row's)."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    return RopeArgs(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _dtype_code(q), q.shape[1], k.shape[1], q.shape[2],
                    float(base), _ptr(batch.dev), batch.batch, q.shape[0], _ptr(positions), _ptr(dev_status))


def rope_copy(q, k, batch: Batch, base: float = 10000.0, q_out=None, k_out=None, stream=None, positions=None,
              dev_status=None):
    """Rotate Q [rows, Hq, d] and K_new [rows, Hkv, d]; returns (q_out, k_out)."""
    a = rope_args(q, k, batch, base, q_out, k_out, positions, dev_status)
    _check(lib().ssv_rope_copy(C.byref(a), _stream_ptr(stream)), "ssv_rope_copy")
    return (q if q_out is None else q_out), (k if k_out is None else k_out)


def verify_step(rope: "RopeArgs | None", attn: AttnArgs, attn_workspace, accept: "AcceptArgs | None" = None,
                accept_workspace=None, stream=None):
    """ssv_verify_step on prepared argument blocks (see rope_args, attn_args,
    accept_args): rotation, verification attention and acceptance as one call."""
    aw = _ptr(attn_workspace)
    awb = 0 if attn_workspace is None else attn_workspace.numel() * attn_workspace.element_size()
    cw = _ptr(accept_workspace)
    cwb = 0 if accept_workspace is None else accept_workspace.numel() * accept_workspace.element_size()
    _check(lib().ssv_verify_step(None if rope is None else C.byref(rope), C.byref(attn), aw, awb,
                                 None if accept is None else C.byref(accept), cw, cwb, _stream_ptr(stream)),
           "ssv_verify_step")


def attn_args(q, k_cache, v_cache, k_new, v_new, out, batch: Batch, tau, scale: float = 0.0, dev_status=None):
    return AttnArgs(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(out),
                    _dtype_code(q), _dtype_code(out), q.shape[1], k_new.shape[1], q.shape[2], float(scale),
                    _ptr(batch.dev), batch.batch, _ptr(tau), batch.total_rows,
                    batch.total_cache if k_cache is None else k_cache.shape[0], batch.total_slots, batch.max_cache, batch.max_new, batch.max_block, _ptr(dev_status))


def verify_attn_workspace_bytes(args: AttnArgs) -> int:
    n = C.c_size_t(0)
    _check(lib().ssv_verify_attn_workspace(C.byref(args), C.byref(n)), "ssv_verify_attn_workspace")
    return int(n.value)


def verify_attn(q, k_cache, v_cache, k_new, v_new, batch: Batch, tau, out=None, out_dtype=None,
                scale: float = 0.0, workspace=None, dev_status=None, stream=None):
    """Verification attention; returns O [rows, Hq, d]."""
    torch = _torch()
    with _on(stream):
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
        a = attn_args(q, k_cache, v_cache, k_new, v_new, out, batch, tau, scale, dev_status)
        ws = _workspace(verify_attn_workspace_bytes(a), q.device, workspace)
    _check(lib().ssv_verify_attn(C.byref(a), _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream)),
           "ssv_verify_attn")
    return out


def accept_args(mode, T, logits, draft_tokens, tau, block, gamma, slot_off, n_acc, n_out, tokens,
                draft_logits=None, noise=None, noise_row=None, u_accept=None, u_sample=None, max_block=64,
                dev_status=None, noise_seed=0):
    return AcceptArgs(int(mode), float(T), logits.shape[1], block.shape[0], draft_tokens.shape[0], int(max_block),
                      _dtype_code(logits), _ptr(logits), _ptr(draft_logits), _ptr(draft_tokens), _ptr(tau),
                      _ptr(block), _ptr(gamma), _ptr(slot_off), _ptr(noise),
                      0 if noise is None else noise.shape[0], _ptr(noise_row), _ptr(u_accept), _ptr(u_sample),
                      _ptr(n_acc), _ptr(n_out), _ptr(tokens), _ptr(dev_status), int(noise_seed))


def accept_workspace_bytes(args: AcceptArgs) -> int:
    n = C.c_size_t(0)
    _check(lib().ssv_accept_workspace(C.byref(args), C.byref(n)), "ssv_accept_workspace")
    return int(n.value)


def accept(mode, T, logits, draft_tokens, tau, block, gamma, slot_off, draft_logits=None, noise=None,
           noise_row=None, u_accept=None, u_sample=None, max_block=64, workspace=None, dev_status=None,
           stream=None, out=None, noise_seed=0):
    """Acceptance; returns (n_acc [batch], n_out [batch], tokens [slots]) int32 device tensors."""
    torch = _torch()
    dev = logits.device
    if out is None:
        with _on(stream):
            out = (torch.empty(block.shape[0], dtype=torch.int32, device=dev),
                   torch.empty(block.shape[0], dtype=torch.int32, device=dev),
                   torch.empty(draft_tokens.shape[0], dtype=torch.int32, device=dev))
    n_acc, n_out, tokens = out
    a = accept_args(mode, T, logits, draft_tokens, tau, block, gamma, slot_off, n_acc, n_out, tokens,
                    draft_logits, noise, noise_row, u_accept, u_sample, max_block, dev_status, noise_seed)
    with _on(stream):
        ws = _workspace(accept_workspace_bytes(a), dev, workspace)
    _check(lib().ssv_accept(C.byref(a), _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream)),
           "ssv_accept")
    return n_acc, n_out, tokens


def accept_noalloc(mode, T, logits, draft_tokens, tau, block, gamma, slot_off, draft_logits=None, noise=None,
                   noise_row=None, u_accept=None, u_sample=None, max_block=64, dev_status=None, stream=None,
                   out=None, noise_seed=0):
    """ssv_accept without a workspace: scratch comes from the library's fixed
    per-device array (for callers that cannot allocate).  Output tensors may
    be passed in ``out``; otherwise they are allocated here by torch."""
    torch = _torch()
    dev = logits.device
    if out is None:
        with _on(stream):
            out = (torch.empty(block.shape[0], dtype=torch.int32, device=dev),
                   torch.empty(block.shape[0], dtype=torch.int32, device=dev),
                   torch.empty(draft_tokens.shape[0], dtype=torch.int32, device=dev))
    n_acc, n_out, tokens = out
    a = accept_args(mode, T, logits, draft_tokens, tau, block, gamma, slot_off, n_acc, n_out, tokens,
                    draft_logits, noise, noise_row, u_accept, u_sample, max_block, dev_status, noise_seed)
    _check(lib().ssv_accept_noalloc(C.byref(a), _stream_ptr(stream)), "ssv_accept_noalloc")
    return n_acc, n_out, tokens


def commit_args(k_new, v_new, k_dst, v_dst, batch: Batch, tau, n_acc, dst_off, dst_cap, new_len,
                dev_status=None):
    return CommitArgs(_ptr(k_new), _ptr(v_new), _ptr(k_dst), _ptr(v_dst), _dtype_code(k_new), k_new.shape[1],
                      k_new.shape[2], _ptr(batch.dev), batch.batch, _ptr(tau), _ptr(n_acc), _ptr(dst_off),
                      _ptr(dst_cap), _ptr(new_len), k_new.shape[0], tau.shape[0], k_dst.shape[0],
                      _ptr(dev_status))


def commit(k_new, v_new, k_dst, v_dst, batch: Batch, tau, n_acc, dst_off, dst_cap, new_len=None, dev_status=None,
           stream=None):
    """Appends each sequence's fresh prompt rows and accepted data rows (stage
    order) to its cache in k_dst / v_dst (in place); returns new_len [batch]
    int32 device (-1 for a sequence rejected on the device)."""
    torch = _torch()
    if k_dst.dtype != k_new.dtype or v_dst.dtype != k_new.dtype or v_new.dtype != k_new.dtype:
        raise SsvError(SSV_ERR_INVALID, "ssv_commit: k_new, v_new, k_dst and v_dst must share one dtype")
    if tuple(k_dst.shape[1:]) != tuple(k_new.shape[1:]) or v_dst.shape != k_dst.shape or v_new.shape != k_new.shape:
        raise SsvError(SSV_ERR_INVALID, "ssv_commit: row shapes differ")
    if new_len is None:
        with _on(stream):
            new_len = torch.empty(batch.batch, dtype=torch.int32, device=k_new.device)
    a = commit_args(k_new, v_new, k_dst, v_dst, batch, tau, n_acc, dst_off, dst_cap, new_len, dev_status)
    _check(lib().ssv_commit(C.byref(a), _stream_ptr(stream)), "ssv_commit")
    return new_len


def lmhead_args(mode, T, hidden_states, lm_head, draft_tokens, tau, block, gamma, slot_off, n_acc, n_out, tokens,
                noise=None, noise_row=None, dev_status=None):
    return LmheadArgs(int(mode), float(T), lm_head.shape[0], lm_head.shape[1], block.shape[0],
                      draft_tokens.shape[0], _ptr(hidden_states), _ptr(lm_head), _ptr(draft_tokens), _ptr(tau),
                      _ptr(block), _ptr(gamma), _ptr(slot_off), _ptr(noise), 0 if noise is None else noise.shape[0],
                      _ptr(noise_row), _ptr(n_acc), _ptr(n_out), _ptr(tokens), _ptr(dev_status))


def lmhead_accept_workspace_bytes(args: LmheadArgs) -> int:
    n = C.c_size_t(0)
    _check(lib().ssv_lmhead_accept_workspace(C.byref(args), C.byref(n)), "ssv_lmhead_accept_workspace")
    return int(n.value)


def lmhead_accept(mode, T, hidden_states, lm_head, draft_tokens, tau, block, gamma, slot_off, noise=None,
                  noise_row=None, workspace=None, dev_status=None, stream=None, out=None):
    """LM head over the slots' hidden states fused with acceptance; returns
    (n_acc [batch], n_out [batch], tokens [slots]) int32 device tensors."""
    torch = _torch()
    if hidden_states.dtype != torch.bfloat16 or lm_head.dtype != torch.bfloat16:
        raise SsvError(SSV_ERR_INVALID, "ssv_lmhead_accept: hidden states and LM head must be bf16")
    if hidden_states.shape[1] != lm_head.shape[1] or hidden_states.shape[0] != draft_tokens.shape[0]:
        raise SsvError(SSV_ERR_INVALID, "ssv_lmhead_accept: shapes")
    dev = hidden_states.device
    if out is None:
        with _on(stream):
            out = (torch.empty(block.shape[0], dtype=torch.int32, device=dev),
                   torch.empty(block.shape[0], dtype=torch.int32, device=dev),
                   torch.empty(draft_tokens.shape[0], dtype=torch.int32, device=dev))
    n_acc, n_out, tokens = out
    a = lmhead_args(mode, T, hidden_states, lm_head, draft_tokens, tau, block, gamma, slot_off, n_acc, n_out,
                    tokens, noise, noise_row, dev_status)
    with _on(stream):
        ws = _workspace(lmhead_accept_workspace_bytes(a), dev, workspace)
    _check(lib().ssv_lmhead_accept(C.byref(a), _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream)),
           "ssv_lmhead_accept")
    return n_acc, n_out, tokens


def set_fault_injection(kernel=None, skip: int = -1, wait_budget_cycles: int = 1 << 31):
    """Test support: shorten the bounded waits of one kernel and make its CTA 0
    leave out one copy (see ssv_set_fault_injection); kernel None restores the
    defaults."""
    if kernel is None:
        _check(lib().ssv_set_fault_injection(None), "ssv_set_fault_injection")
        return
    f = FaultInjection(int(kernel), int(skip), int(wait_budget_cycles))
    _check(lib().ssv_set_fault_injection(C.byref(f)), "ssv_set_fault_injection")


def tree_attn_args(q, k_cache, v_cache, k_new, v_new, out, seqs, parent, pos, total_out, max_cache,
                   scale: float = 0.0, dev_status=None):
    """seqs: int32 [batch, 9] device tensor of ssv_tree_seq records."""
    return TreeAttnArgs(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(out), _dtype_code(q),
                        _dtype_code(out), q.shape[1], k_new.shape[1], q.shape[2], float(scale), _ptr(seqs),
                        seqs.shape[0], _ptr(parent), _ptr(pos), q.shape[0], k_new.shape[0],
                        0 if k_cache is None else k_cache.shape[0], 0 if parent is None else parent.shape[0],
                        int(total_out), int(max_cache), _ptr(dev_status))


def tree_verify_attn_workspace_bytes(args: TreeAttnArgs) -> int:
    n = C.c_size_t(0)
    _check(lib().ssv_tree_verify_attn_workspace(C.byref(args), C.byref(n)), "ssv_tree_verify_attn_workspace")
    return n.value


def tree_verify_attn(q, k_cache, v_cache, k_new, v_new, seqs, parent, pos, total_out, max_cache, out=None,
                     out_dtype=None, scale: float = 0.0, dev_status=None, stream=None, workspace=None):
    """Attention of the tree pass; returns O [total_out, Hq, d] (rows of
    committed positions are left as they were in `out`).  workspace: a zeroed
    uint8 device tensor of tree_verify_attn_workspace_bytes (allocated here
    when not given)."""
    torch = _torch()
    with _on(stream):
        if out is None:
            out = torch.zeros((int(total_out), q.shape[1], q.shape[2]), dtype=out_dtype or q.dtype, device=q.device)
        a = tree_attn_args(q, k_cache, v_cache, k_new, v_new, out, seqs, parent, pos, total_out, max_cache, scale,
                           dev_status)
        ws = _workspace(tree_verify_attn_workspace_bytes(a), q.device, workspace)
    _check(lib().ssv_tree_verify_attn(C.byref(a), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                      _stream_ptr(stream)), "ssv_tree_verify_attn")
    return out


def tree_accept_args(mode, T, logits, seqs, parent, pos, token, n_acc, path, emit_pos, emit_tok, noise=None,
                     noise_row=None, pos_off=None, dev_status=None):
    return TreeAcceptArgs(int(mode), float(T), logits.shape[1], _ptr(seqs), seqs.shape[0], _dtype_code(logits),
                          _ptr(logits), _ptr(parent), _ptr(pos), _ptr(token),
                          0 if parent is None else parent.shape[0], logits.shape[0], _ptr(noise),
                          0 if noise is None else noise.shape[0], _ptr(noise_row), _ptr(pos_off),
                          0 if noise_row is None else noise_row.shape[0], _ptr(n_acc), _ptr(path), _ptr(emit_pos),
                          _ptr(emit_tok), _ptr(dev_status))


def tree_accept(mode, T, logits, seqs, parent, pos, token, noise=None, noise_row=None, pos_off=None, workspace=None,
                dev_status=None, stream=None):
    """Acceptance of the tree by state equality; returns (n_acc [batch],
    path [batch, 64], emit_pos [batch], emit_tok [batch]) int32 device tensors."""
    torch = _torch()
    dev = logits.device
    b = seqs.shape[0]
    with _on(stream):
        n_acc = torch.empty(b, dtype=torch.int32, device=dev)
        path = torch.empty((b, 64), dtype=torch.int32, device=dev)
        ep = torch.empty(b, dtype=torch.int32, device=dev)
        et = torch.empty(b, dtype=torch.int32, device=dev)
    a = tree_accept_args(mode, T, logits, seqs, parent, pos, token, n_acc, path, ep, et, noise, noise_row, pos_off,
                         dev_status)
    n = C.c_size_t(0)
    _check(lib().ssv_tree_accept_workspace(C.byref(a), C.byref(n)), "ssv_tree_accept_workspace")
    with _on(stream):
        ws = _workspace(int(n.value), dev, workspace)
    _check(lib().ssv_tree_accept(C.byref(a), _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream)),
           "ssv_tree_accept")
    return n_acc, path, ep, et


# ---------------------------------------------------------------------------
# the paged 8-bit KV cache
# ---------------------------------------------------------------------------
# A serving loop calls these once per layer and pass, and the smallest of their kernels take a few
# microseconds: the argument block is packed in one go (the layout of the ctypes structure of the
# same name) instead of field by field, and the stream is read by its handle.
_CODES = {C.c_void_p: "P", C.c_int: "i", C.c_int32: "i", C.c_int64: "q", C.c_float: "f", C.c_double: "d"}


def _packer(cls):
    return struct.Struct("@" + "".join(_CODES[f] for _, f in cls._fields_)).pack


_pack_plan, _pack_norm = _packer(PagePlanArgs), _packer(NormRopeArgs)
_pack_attn, _pack_commit = _packer(AttnFp8Args), _packer(CommitFp8Args)
_pack_logprobs, _pack_distill = _packer(LogprobsArgs), _packer(DistillArgs)
_entries = {}


def _entry(name: str, workspace: bool = False):
    """Entry point `name` on packed argument blocks."""
    f = _entries.get(name)
    if f is None:
        types = [C.c_char_p] + ([C.c_void_p, C.c_size_t] if workspace else []) + [C.c_void_p]
        f = _entries[name] = C.CFUNCTYPE(C.c_int, *types)((name, lib()))
    return f


def _launch(what: str, tensors, block, stream, workspace=None):
    """Calls entry point `what` on the packed `block`, on the given stream or
    the current one of the device that holds the first of `tensors`; the others
    (None: left out) have to be there, too."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise SsvError(SSV_ERR_INVALID, f"{what}: tensors of one CUDA device")
    if workspace is not None and not workspace.is_contiguous():
        raise SsvError(SSV_ERR_WORKSPACE, f"{what}: the workspace is contiguous")
    _launch_on(what, dev, block, stream, workspace)


def _launch_on(what: str, dev: int, block, stream, workspace=None):
    if dev < 0:
        raise SsvError(SSV_ERR_INVALID, f"{what}: tensors of one CUDA device")
    cuda = _torch()._C
    if cuda._cuda_getDevice() != dev:
        with _torch().cuda.device(dev):
            return _launch_on(what, dev, block, stream, workspace)
    s = cuda._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if workspace is None:
        code = (_entries.get(what) or _entry(what))(block, s)
    else:
        code = (_entries.get(what) or _entry(what, True))(block, workspace.data_ptr(),
                                                          workspace.numel() * workspace.element_size(), s)
    if code:
        _check(code, what)


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _rows_strided(t, what: str) -> int:
    """Row stride (elements) of a [rows, heads, d] tensor whose heads are contiguous; 0: packed."""
    if t.dim() != 3:
        raise SsvError(SSV_ERR_INVALID, f"{what}: [rows, heads, d]")
    if t.is_contiguous():
        return 0
    (rows, heads, d), s = t.shape, t.stride()
    if rows and (s[2] != 1 or (s[1] != d and heads > 1)):
        raise SsvError(SSV_ERR_INVALID, f"{what}: [rows, heads, d] with contiguous heads")
    if rows > 1 and s[0] < heads * d:  # one row repeated (stride 0, which the library reads as packed), or rows that overlap
        raise SsvError(SSV_ERR_INVALID, f"{what}: rows that do not overlap")
    return s[0] if rows > 1 else heads * d


def _paged_cache(k_cache, v_cache, k_scale, v_scale, pages, what: str):
    """(Hkv, page_size, d, n_pages) of a paged e4m3 cache, checked."""
    torch = _torch()
    shape = k_cache.shape
    for x in (k_cache, v_cache):
        if x.dtype not in (torch.uint8, torch.float8_e4m3fn) or x.dim() != 4 or not x.is_contiguous() or \
                x.shape != shape:
            raise SsvError(SSV_ERR_INVALID, f"{what}: caches are contiguous e4m3 [n_pages, Hkv, page_size, d]")
    n, hkv, ps, d = shape
    for x in (k_scale, v_scale):
        if x.dtype != torch.float32 or x.shape != (n, hkv) or not x.is_contiguous():
            raise SsvError(SSV_ERR_INVALID, f"{what}: scales are contiguous fp32 [n_pages, Hkv]")
    return hkv, ps, d, n


def _int32(what: str, *tensors):
    i32 = _torch().int32
    for t in tensors:
        if t is not None and (t.dtype != i32 or not t.is_contiguous()):
            raise SsvError(SSV_ERR_INVALID, f"{what}: index tensors are contiguous int32")


def page_plan(cache_len, new_len, block, held, pages, free_list, n_free, page_size: int, total_rows: int, out=None,
              dev_status=None, stream=None):
    """Tables of a pass from the requests' lengths (ssv_page_plan).  cache_len
    [batch] (negative: the request has ended), new_len, block, held [batch],
    pages [batch, max_pages], free_list [n_pages], n_free [1]: int32 device
    tensors; pages and free_list are updated in place.  Returns (seqs
    [batch, 6], slot_map [total_rows], slot_off [batch], held [batch], n_free
    [1]), new tensors unless given in ``out``."""
    torch = _torch()
    what, i32, dev = "ssv_page_plan", torch.int32, cache_len.get_device()
    for t in (cache_len, new_len, block, held, pages, free_list, n_free) + (out or ()) + \
            (() if dev_status is None else (dev_status,)):
        if t.dtype != i32 or not t.is_contiguous():
            raise SsvError(SSV_ERR_INVALID, f"{what}: index tensors are contiguous int32")
        if t.get_device() != dev:
            raise SsvError(SSV_ERR_INVALID, f"{what}: tensors of one CUDA device")
    batch = cache_len.numel()
    if cache_len.dim() != 1 or new_len.numel() != batch or block.numel() != batch or held.numel() != batch or \
            pages.dim() != 2 or pages.shape[0] != batch or n_free.numel() != 1:
        raise SsvError(SSV_ERR_INVALID, f"{what}: shapes")
    total_rows = int(total_rows)
    if out is None:
        # one allocation: the table, the offsets, the counts, the stack height, the slot map
        with _on(stream):
            buf = torch.empty(8 * batch + 1 + total_rows, dtype=i32, device=cache_len.device)
        seqs, slot_off, held_out, n_out, slot_map = buf.split_with_sizes([6 * batch, batch, batch, 1, total_rows])
        out = (seqs.view(batch, 6), slot_map, slot_off, held_out, n_out)
        at = buf.data_ptr()
        outs = (at, at + 32 * batch + 4, at + 24 * batch, at + 28 * batch, at + 32 * batch)
    else:
        if tuple(x.numel() for x in out) != (6 * batch, total_rows, batch, batch, 1):
            raise SsvError(SSV_ERR_INVALID, f"{what}: output shapes")
        outs = tuple(x.data_ptr() for x in out)
    a = _pack_plan(cache_len.data_ptr(), new_len.data_ptr(), block.data_ptr(), held.data_ptr(), pages.data_ptr(),
                   free_list.data_ptr(), n_free.data_ptr(), batch, pages.shape[1], int(page_size), free_list.numel(),
                   total_rows, *outs, _addr(dev_status))
    _launch_on(what, dev, a, stream)
    if batch == 0:  # the call writes nothing: no rows, and the stack as it was
        with _on(stream):
            out[1].fill_(-1)
            out[4].copy_(n_free)
    return out


def norm_rope_copy(q, k, q_weight, k_weight, batch: Batch, base: float = 10000.0, eps: float = 1e-6, q_out=None,
                   k_out=None, positions=None, dev_status=None, stream=None):
    """RMS norm of every head of Q [rows, Hq, d] and K_new [rows, Hkv, d]
    (weights [d]) and rope_copy's rotation in one pass; in place unless
    outputs are given.  Rows may be strided (parts of a fused projection).
    Returns (q_out, k_out)."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    if q.dim() != 3 or k.dim() != 3 or q_out.shape != q.shape or k_out.shape != k.shape or \
            q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2]:
        raise SsvError(SSV_ERR_INVALID, "ssv_norm_rope_copy: shapes")
    what = "ssv_norm_rope_copy"
    dt = q.dtype
    if k.dtype != dt or q_out.dtype != dt or k_out.dtype != dt or q_weight.dtype != dt or k_weight.dtype != dt:
        raise SsvError(SSV_ERR_INVALID, "ssv_norm_rope_copy: one dtype")
    if q_weight.shape != q.shape[2:] or k_weight.shape != q.shape[2:] or not q_weight.is_contiguous() or \
            not k_weight.is_contiguous():
        raise SsvError(SSV_ERR_INVALID, "ssv_norm_rope_copy: weights are [d]")
    _int32(what, batch.dev, positions)
    if positions is not None and positions.shape[0] < q.shape[0]:
        raise SsvError(SSV_ERR_INVALID, "ssv_norm_rope_copy: one position per row")
    a = _pack_norm(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), q_weight.data_ptr(),
                   k_weight.data_ptr(), _rows_strided(q, what), _rows_strided(k, what), _rows_strided(q_out, what),
                   _rows_strided(k_out, what), _dtype_code(q), q.shape[1], k.shape[1], q.shape[2], eps, base,
                   batch.dev.data_ptr(), batch.batch, q.shape[0], _addr(positions), _addr(dev_status))
    _launch(what, (q, k, q_out, k_out, q_weight, k_weight, batch.dev, positions, dev_status), a, stream)
    return q_out, k_out


def _attn_fp8_fields(q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, out, batch, tau, scale, dev_status):
    what = "ssv_verify_attn_fp8"
    hkv, ps, d, n = _paged_cache(k_cache, v_cache, k_scale, v_scale, pages, what)
    bf16, shape = _torch().bfloat16, q.shape
    if q.dtype != bf16 or k_new.dtype != bf16 or v_new.dtype != bf16 or out.dtype != bf16:
        raise SsvError(SSV_ERR_INVALID, f"{what}: q, fresh rows and output are bf16")
    if q.dim() != 3 or not q.is_contiguous() or not out.is_contiguous() or out.shape != shape or \
            k_new.shape != (shape[0], hkv, d) or v_new.shape != k_new.shape or shape[2] != d:
        raise SsvError(SSV_ERR_INVALID, f"{what}: shapes")
    _int32(what, pages, batch.dev, tau)
    return (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            pages.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), out.data_ptr(), _rows_strided(k_new, what),
            _rows_strided(v_new, what), shape[1], hkv, d, ps, n, pages.numel(), scale, batch.dev.data_ptr(),
            batch.batch, tau.data_ptr(), shape[0], tau.shape[0], batch.max_cache, batch.max_new, batch.max_block,
            _addr(dev_status))


def attn_fp8_args(q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, out, batch: Batch, tau,
                  scale: float = 0.0, dev_status=None):
    return AttnFp8Args(*_attn_fp8_fields(q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, out, batch, tau,
                                         float(scale), dev_status))


def verify_attn_fp8_workspace_bytes(args: AttnFp8Args) -> int:
    n = C.c_size_t(0)
    _check(lib().ssv_verify_attn_fp8_workspace(C.byref(args), C.byref(n)), "ssv_verify_attn_fp8_workspace")
    return int(n.value)


def verify_attn_fp8_workspace(q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, batch: Batch, tau,
                              stream=None):
    """A zeroed workspace for verify_attn_fp8 on these arguments, to be kept
    for later calls on the same stream, of any sizes that ask for no more."""
    a = attn_fp8_args(q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, q, batch, tau)
    with _on(stream):
        return _workspace(verify_attn_fp8_workspace_bytes(a), q.device)


def verify_attn_fp8(q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, batch: Batch, tau, out=None,
                    scale: float = 0.0, workspace=None, dev_status=None, stream=None):
    """Verification attention with the cached keys in e4m3 pages; q, k_new,
    v_new bf16 (fresh rows may be strided).  Returns O [rows, Hq, d] bf16."""
    torch = _torch()
    if out is None:
        with _on(stream):
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    a = _attn_fp8_fields(q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, out, batch, tau, float(scale),
                         dev_status)
    ws = workspace
    if ws is None:
        with _on(stream):
            ws = _workspace(verify_attn_fp8_workspace_bytes(AttnFp8Args(*a)), q.device)
    _launch("ssv_verify_attn_fp8", (q, k_cache, v_cache, k_scale, v_scale, pages, k_new, v_new, out, batch.dev, tau, ws,
                                    dev_status), _pack_attn(*a), stream, ws)
    return out


def commit_fp8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, pages, batch: Batch, tau, n_acc, new_len=None,
               dev_status=None, stream=None, cache_len=None):
    """Quantises and appends each sequence's fresh prompt rows and accepted
    data rows (stage order) to its pages, in place; returns new_len [batch]
    int32 device.  cache_len: the lengths that page_plan was given, which the
    requests that it left idle and the sequences rejected here keep (a loop
    passes them; without them such a sequence gets its record's cache_len, 0
    in page_plan's idle records, or -1)."""
    torch = _torch()
    what = "ssv_commit_fp8"
    hkv, ps, d, n = _paged_cache(k_cache, v_cache, k_scale, v_scale, pages, what)
    rows = k_new.shape[0]
    if k_new.dtype != v_new.dtype or k_new.shape != (rows, hkv, d) or v_new.shape != k_new.shape:
        raise SsvError(SSV_ERR_INVALID, f"{what}: fresh rows")
    _int32(what, pages, batch.dev, tau, n_acc, new_len, cache_len)
    if n_acc.shape[0] != batch.batch or (new_len is not None and new_len.shape[0] != batch.batch) or \
            (cache_len is not None and cache_len.shape[0] != batch.batch):
        raise SsvError(SSV_ERR_INVALID, f"{what}: shapes")
    if new_len is None:
        with _on(stream):
            new_len = torch.empty(batch.batch, dtype=torch.int32, device=k_new.device)
    a = _pack_commit(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                     v_scale.data_ptr(), pages.data_ptr(), _rows_strided(k_new, what), _rows_strided(v_new, what),
                     _dtype_code(k_new), hkv, d, ps, n, pages.numel(), batch.dev.data_ptr(), batch.batch,
                     tau.data_ptr(), n_acc.data_ptr(), new_len.data_ptr(), rows, tau.shape[0], batch.max_new,
                     batch.max_block, _addr(dev_status), _addr(cache_len))
    _launch(what, (k_new, v_new, k_cache, v_cache, k_scale, v_scale, pages, batch.dev, tau, n_acc, new_len, dev_status,
                   cache_len), a, stream)
    return new_len


# ---------------------------------------------------------------------------
# log-probabilities and distillation
# ---------------------------------------------------------------------------
def _logit_rows(t, what: str) -> int:
    """Row stride (elements) of [rows, V] logits whose elements are contiguous; 0: packed."""
    if t.dim() != 2 or t.shape[1] < 1:
        raise SsvError(SSV_ERR_INVALID, f"{what}: logits are [rows, V]")
    if t.is_contiguous():
        return 0
    (rows, v), s = t.shape, t.stride()
    if v > 1 and s[1] != 1:
        raise SsvError(SSV_ERR_INVALID, f"{what}: the logits of a row are contiguous")
    if rows > 1 and s[0] < v:
        raise SsvError(SSV_ERR_INVALID, f"{what}: rows that do not overlap")
    return s[0] if rows > 1 else 0


def _like(what: str, shape, dtype, *tensors):
    for t in tensors:
        if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
            raise SsvError(SSV_ERR_INVALID, f"{what}: contiguous {dtype} {list(shape)}")


def logprobs(logits, tokens=None, top_k: int = 0, T: float = 1.0, rows=None, out=None, dev_status=None, stream=None):
    """Log-probabilities of tokens (int32 [n], -1: none) under softmax(logits
    / T), their ranks, the rows' entropies and log-sum-exps, and each row's
    top_k alternatives.  logits [rows, V] fp32 or bf16 (rows may be strided);
    entry i has logits row rows[i] (int32 [n]; without it row i).  Returns
    (logprob [n], rank [n], entropy [n], lse [n], top_logprob [n, top_k],
    top_token [n, top_k]); logprob and rank are None without tokens, the
    last two with top_k 0.  ``out``: six tensors (or None) of those shapes,
    for calls in a loop (making them is most of a short call's time).  Mask
    with -inf where alternatives are asked for: a row masked with a number
    that leaves fewer tokens than top_k takes milliseconds."""
    torch = _torch()
    what, f32, i32 = "ssv_logprobs", torch.float32, torch.int32
    stride, dt = _logit_rows(logits, what), _dtype_code(logits)
    _int32(what, tokens, rows)
    for t in (tokens, rows):
        if t is not None and t.dim() != 1:
            raise SsvError(SSV_ERR_INVALID, f"{what}: one token and one row per entry")
    n = (tokens if tokens is not None else rows if rows is not None else logits).shape[0]
    if rows is not None and rows.shape[0] != n:
        raise SsvError(SSV_ERR_INVALID, f"{what}: one token and one row per entry")
    top_k = int(top_k)
    if top_k < 0:
        raise SsvError(SSV_ERR_INVALID, f"{what}: top_k")
    if out is None:
        dev, empty = logits.device, torch.empty
        with _on(stream):
            out = (None if tokens is None else empty(n, dtype=f32, device=dev),
                   None if tokens is None else empty(n, dtype=i32, device=dev),
                   empty(n, dtype=f32, device=dev), empty(n, dtype=f32, device=dev),
                   empty((n, top_k), dtype=f32, device=dev) if top_k else None,
                   empty((n, top_k), dtype=i32, device=dev) if top_k else None)
    else:
        out = tuple(out)
        if len(out) != 6:
            raise SsvError(SSV_ERR_INVALID, f"{what}: six outputs")
        _like(what, (n,), f32, out[0], out[2], out[3])
        _like(what, (n,), i32, out[1])
        _like(what, (n, top_k), f32, out[4])
        _like(what, (n, top_k), i32, out[5])
    a = _pack_logprobs(logits.data_ptr(), stride, dt, logits.shape[1], logits.shape[0], _addr(rows), _addr(tokens), n,
                       top_k, T, *map(_addr, out), _addr(dev_status))
    _launch(what, (logits, rows, tokens, dev_status) + out, a, stream)
    return out


def _distill_fields(what, logits, teacher_token, teacher_logprob, T, mode, weight, loss, stats, grad_loss, grad, dev_status):
    torch = _torch()
    f32, n = torch.float32, logits.shape[0]
    stride, dt = _logit_rows(logits, what), _dtype_code(logits)
    if teacher_token.dim() != 2 or teacher_token.shape[0] != n:
        raise SsvError(SSV_ERR_INVALID, f"{what}: the target's tokens are [rows, K]")
    _int32(what, teacher_token)
    _like(what, teacher_token.shape, f32, teacher_logprob)
    _like(what, (n,), f32, weight, loss, grad_loss)
    _like(what, (n, 4), f32, stats)
    grad_stride = 0
    if grad is not None:
        if grad.dtype != logits.dtype or grad.shape != logits.shape:
            raise SsvError(SSV_ERR_INVALID, f"{what}: the gradient is as the logits")
        grad_stride = _logit_rows(grad, what)
    return _pack_distill(logits.data_ptr(), stride, dt, logits.shape[1], n, teacher_token.shape[1],
                         teacher_token.data_ptr(), teacher_logprob.data_ptr(), T, mode, _addr(weight), _addr(loss),
                         _addr(stats), _addr(grad_loss), _addr(grad), grad_stride, _addr(dev_status))


def _empty_rows(logits):
    """An uninitialised tensor of the logits' shape whose rows lie to 32-byte boundaries as theirs do, where that
    costs little memory."""
    torch = _torch()
    n, v = logits.shape
    s = logits.stride(0) if n > 1 else v
    lead = (logits.data_ptr() % 32) // logits.element_size()
    if (s == v and lead == 0) or not v <= s <= v + 64:
        return torch.empty((n, v), dtype=logits.dtype, device=logits.device)
    if lead == 0:
        return torch.empty_strided((n, v), (s, 1), dtype=logits.dtype, device=logits.device)
    return torch.empty(n * s + lead, dtype=logits.dtype, device=logits.device).as_strided((n, v), (s, 1), lead)


def distill(logits, teacher_token, teacher_logprob, T: float = 1.0, mode: int = RENORM, weight=None, grad=False,
            loss=None, stats=None, dev_status=None, stream=None):
    """Distillation loss of a drafter's logits [n, V] (fp32 or bf16; rows may
    be strided) against the target's alternatives (teacher_token int32,
    teacher_logprob fp32 [n, K], as logprobs returns them; token -1: absent),
    times weight [n].  Returns (loss [n], stats [n, 4], grad); grad is None
    unless it is asked for (True: rows may be strided as the logits' are) or
    given (a tensor like the logits, which may be the logits themselves).
    stats is what distill_backward takes.  Not part of autograd: no result has
    a grad_fn; the gradient goes on with logits.backward(grad)."""
    torch = _torch()
    what = "ssv_distill"
    if logits.dim() != 2:
        raise SsvError(SSV_ERR_INVALID, f"{what}: logits are [rows, V]")
    n = logits.shape[0]
    with _on(stream):
        if loss is None:
            loss = torch.empty(n, dtype=torch.float32, device=logits.device)
        if stats is None:
            stats = torch.empty((n, 4), dtype=torch.float32, device=logits.device)
        if grad is True:
            grad = _empty_rows(logits)
    if grad is False:
        grad = None
    a = _distill_fields(what, logits, teacher_token, teacher_logprob, T, mode, weight, loss, stats, None, grad, dev_status)
    _launch(what, (logits, teacher_token, teacher_logprob, weight, loss, stats, grad, dev_status), a, stream)
    return loss, stats, grad


def distill_backward(logits, teacher_token, teacher_logprob, stats, grad_loss=None, T: float = 1.0, mode: int = RENORM,
                     weight=None, grad=None, dev_status=None, stream=None):
    """Gradient of sum(grad_loss * loss) for distill's losses on the same
    arguments, from the statistics that it returned; grad_loss [n] fp32 (None:
    ones).  grad: a tensor like the logits, which may be the logits themselves
    (allocated here when not given, rows strided as theirs may be).  Returns
    grad, for logits.backward(grad)."""
    what = "ssv_distill_backward"
    if logits.dim() != 2:
        raise SsvError(SSV_ERR_INVALID, f"{what}: logits are [rows, V]")
    if grad is None:
        with _on(stream):
            grad = _empty_rows(logits)
    a = _distill_fields(what, logits, teacher_token, teacher_logprob, T, mode, weight, None, stats, grad_loss, grad,
                        dev_status)
    _launch(what, (logits, teacher_token, teacher_logprob, weight, stats, grad_loss, grad, dev_status), a, stream)
    return grad


def stream_read(buf, out, stream=None):
    """Reads every byte of the device tensor `buf` once (measurement reference
    for memory-bound kernels); XOR checksum into the int32 device tensor `out`."""
    nbytes = buf.numel() * buf.element_size()
    _check(lib().ssv_stream_read(_ptr(buf), nbytes, _ptr(out), _stream_ptr(stream)), "ssv_stream_read")


def get_status(dev_status, stream=None) -> int:
    """Waits for the stream and returns (and clears) the device status word."""
    return int(lib().ssv_get_status(_ptr(dev_status), _stream_ptr(stream)))


def bench(config: str, iters: int = 20) -> str:
    buf = C.create_string_buffer(4096)
    _check(lib().ssv_bench(config.encode(), int(iters), buf, 4096), "ssv_bench")
    return buf.value.decode()
