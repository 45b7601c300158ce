"""Thin Python binding of libmsa.so (C-ABI in include/msa.h).

Argument marshalling only: it checks dtypes and layouts, allocates outputs
and workspaces with torch (device memory), and passes raw pointers and the
current CUDA stream to the library (the paged calls through _paged_binding.so,
which does the same natively).  Every step of the computation runs in
the library's kernels; there is no fallback.  If libmsa.so has not been
built, the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import math
import os
import threading
from dataclasses import dataclass
from functools import cached_property
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

OP_INDEX_SELECT, OP_SPARSE_ATTN_FWD, OP_KL_FWD, OP_FUSED_BWD, OP_FUSED_BWD_KL, OP_TRAIN_STEP = 0, 1, 2, 3, 4, 5
OP_WARMUP_KL = 6
OP_PAGED_PLAN, OP_PAGED_APPEND, OP_PAGED_BLOCK_SCORES, OP_PAGED_BLOCK_TOPK, OP_PAGED_ATTN = 16, 17, 18, 19, 20
OP_PAGED_FORK, OP_PAGED_COMPACT, OP_PAGED_COPY, OP_PAGED_CHUNK_SCORES, OP_PAGED_CHUNK_ATTN = 32, 33, 34, 35, 36
PAGE = 128      # tokens of a cache page
STATUS = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARGUMENT", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_WORKSPACE",
          4: "MSA_ERR_CUDA", 5: "MSA_ERR_TIMEOUT", 6: "MSA_ERR_DEVICE"}
EXPORTS = ("msa_workspace_size", "msa_index_select", "msa_sparse_attn_fwd", "msa_kl_fwd", "msa_fused_bwd",
           "msa_fused_bwd_kl", "msa_train_step", "msa_train_step_staged", "msa_block_mask", "msa_warmup_kl",
           "msa_index_proj_workspace_size", "msa_index_proj_fwd", "msa_index_proj_bwd", "msa_kv_append",
           "msa_paged_workspace_size", "msa_paged_plan", "msa_paged_plan_held", "msa_paged_append", "msa_paged_block_scores",
           "msa_paged_block_topk", "msa_paged_attn", "msa_paged_fork", "msa_paged_compact", "msa_paged_copy",
           "msa_paged_chunk_scores", "msa_paged_chunk_attn", "msa_rotary_fwd", "msa_rotary_bwd", "msa_last_error", "msa_check_device_status",
           "msa_version", "msa_launch_count")


class MsaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class _CProjShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("T", "Dm", "Hkv", "d_idx")]


@dataclass
class ProjShape:
    """msa_proj_shape: T tokens of Dm features projected to Hkv index queries
    and one index key of d_idx features each."""
    T: int
    Dm: int
    Hkv: int
    d_idx: int

    def c(self) -> _CProjShape:
        return _CProjShape(self.T, self.Dm, self.Hkv, self.d_idx)


class _CShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Nq", "Nk", "q_offset", "Hq", "Hkv", "d", "d_idx", "block", "topk")] + [
        ("kv_rows", ctypes.c_longlong), ("scale", ctypes.c_float), ("scale_idx", ctypes.c_float)]


@dataclass
class Shape:
    """msa_shape: see include/msa.h for the meaning of each field."""
    B: int
    Nq: int
    Nk: int
    Hq: int
    Hkv: int
    d: int
    d_idx: int
    topk: int
    block: int = 128
    q_offset: int = 0
    kv_rows: int = 0
    scale: float = 0.0
    scale_idx: float = 0.0

    @property
    def nb(self) -> int:
        return (self.Nk + self.block - 1) // self.block

    @property
    def G(self) -> int:
        return self.Hq // self.Hkv

    @property
    def rows_kv(self) -> int:
        return self.kv_rows or self.Nk

    def c(self) -> _CShape:
        return _CShape(self.B, self.Nq, self.Nk, self.q_offset, self.Hq, self.Hkv, self.d, self.d_idx, self.block,
                       self.topk, self.kv_rows, self.scale, self.scale_idx)


class _CPagedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("R", "T", "max_blocks", "n_pages", "Hq", "Hkv", "d", "d_idx", "topk")] + [
        ("scale", ctypes.c_float), ("scale_idx", ctypes.c_float)]


@dataclass(frozen=True)
class PagedShape:
    """msa_paged_shape: R requests, T rows (query tokens) of a step, block tables
    of max_blocks columns, a pool of n_pages pages of 128 tokens."""
    R: int
    T: int
    max_blocks: int
    n_pages: int
    Hq: int
    Hkv: int
    d: int
    d_idx: int
    topk: int
    scale: float = 0.0
    scale_idx: float = 0.0

    @property
    def G(self) -> int:
        return self.Hq // self.Hkv

    @property
    def n_segs(self) -> int:
        """Entries of a plan's segment list before the last."""
        return min(self.T, 2 * self.R + self.T // PAGE)

    def c(self) -> _CPagedShape:
        return _CPagedShape(self.R, self.T, self.max_blocks, self.n_pages, self.Hq, self.Hkv, self.d, self.d_idx,
                            self.topk, self.scale, self.scale_idx)

    def __getstate__(self):
        return {n: getattr(self, n) for n in self.__dataclass_fields__}     # copies and pickles leave the handles behind

    @cached_property
    def _calls(self) -> dict:
        """By op, the binding's handle of the call: the shape and (name, shape, dtype, kind) of each tensor in the order of
        the C arguments."""
        i32, f32, bf, f8 = 0, 1, 2, 3                  # dtypes
        need, maybe, out = 0, 1, 2                     # kinds; an `out` that is None is allocated
        R, T, H, N, D = self.R, self.T, self.Hkv, self.n_pages, self.d
        row = lambda *names: [(n, (T,), i32, need) for n in names]  # noqa: E731
        table, starts = ("block_table", (R, self.max_blocks), i32, need), ("q_starts", (R + 1,), i32, need)
        cache = lambda kind: ([(n, (N, H, PAGE, D), f8, kind) for n in ("k8", "v8")]  # noqa: E731
                              + [(n, (N, H), f32, kind) for n in ("k_scale", "v_scale")])
        k_idx, sel, scores = (N, PAGE, self.d_idx), (T, H, self.topk), (T, H, self.max_blocks)
        specs = {
            OP_PAGED_PLAN: [("new_lens", (R,), i32, need), ("lens", (R,), i32, need), ("ended", (R,), i32, maybe), ("held", (R,), i32, maybe), table,
                            ("free_pages", (N,), i32, need), ("free_state", (2,), i32, need), ("lens", (R,), i32, out),
                            ("free_state", (2,), i32, out), ("q_starts", (R + 1,), i32, out), ("row_req", (T,), i32, out),
                            ("row_pos", (T,), i32, out), ("slots", (T,), i32, out), ("segs", (self.n_segs + 1,), i32, out)],
            OP_PAGED_APPEND: [("k_new", (T, H, D), bf, maybe), ("v_new", (T, H, D), bf, maybe), ("k_idx_new", (T, self.d_idx), bf, maybe),
                              *row("slots"), ("segs", (self.n_segs + 1,), i32, need), *cache(maybe), ("k_idx", k_idx, bf, maybe)],
            OP_PAGED_BLOCK_SCORES: [("q_idx", (T, H, self.d_idx), bf, need), ("k_idx", k_idx, bf, need), table, starts,
                                    *row("row_req", "row_pos"), ("block_scores", scores, f32, out)],
            OP_PAGED_BLOCK_TOPK: [("block_scores", scores, f32, need), *row("row_pos"), ("sel_idx", sel, i32, out)],
            OP_PAGED_ATTN: [("q", (T, self.Hq, D), bf, need), *cache(need), table, *row("row_req", "row_pos"),
                            ("sel_idx", sel, i32, maybe), ("o", (T, self.Hq, D), bf, out), ("lse", (T, self.Hq), f32, out)],
        }
        return {op: binding().prepare(op, self._fields, args) for op, args in specs.items()}

    @property
    def _fields(self) -> tuple:
        return (self.R, self.T, self.max_blocks, self.n_pages, self.Hq, self.Hkv, self.d, self.d_idx, self.topk, self.scale, self.scale_idx)

    @cached_property
    def _more_calls(self) -> dict:
        """As _calls, of the calls for shared pages and chunks."""
        i32, f32, bf, f8 = 0, 1, 2, 3
        need, maybe, out = 0, 1, 2
        R, T, H, N, D = self.R, self.T, self.Hkv, self.n_pages, self.d
        table = ("block_table", (R, self.max_blocks), i32, need)
        starts_pos = [table, ("q_starts", (R + 1,), i32, need), ("row_pos", (T,), i32, need)]
        cache = lambda kind: ([(n, (N, H, PAGE, D), f8, kind) for n in ("k8", "v8")]  # noqa: E731
                              + [(n, (N, H), f32, kind) for n in ("k_scale", "v_scale")])
        k_idx = (N, PAGE, self.d_idx)
        specs = {
            OP_PAGED_FORK: [("src", (R,), i32, need), ("fork_lens", (R,), i32, maybe), ("lens", (R,), i32, need), ("held", (R,), i32, maybe),
                            table, ("free_pages", (N,), i32, need), ("free_state", (2,), i32, need), ("shares", (N,), i32, need),
                            ("moves", (R, 3), i32, out)],
            OP_PAGED_COPY: [("moves", (-1, 3), i32, need), *cache(maybe), ("k_idx", k_idx, bf, maybe)],      # -1: any number
            OP_PAGED_CHUNK_SCORES: [("q_idx", (T, H, self.d_idx), bf, need), ("k_idx", k_idx, bf, need), *starts_pos,
                                    ("block_scores", (T, H, self.max_blocks), f32, out)],
            OP_PAGED_CHUNK_ATTN: [("q", (T, self.Hq, D), bf, need), *cache(need), *starts_pos, ("sel_idx", (T, H, self.topk), i32, maybe),
                                  ("o", (T, self.Hq, D), bf, out), ("lse", (T, self.Hq), f32, out)],
        }
        for op, given, made in ((OP_PAGED_COMPACT, need, out), ((OP_PAGED_COMPACT, None), maybe, maybe)):     # without shares none are written
            specs[op] = [("lens", (R,), i32, need), ("held", (R,), i32, maybe), table, ("shares", (N,), i32, given),
                         ("block_table", (R, self.max_blocks), i32, out), ("free_pages", (N,), i32, out), ("free_state", (2,), i32, out),
                         ("shares", (N,), i32, made), ("moves", (max(1, N // 2), 3), i32, out)]
        return {op: binding().prepare(op[0] if isinstance(op, tuple) else op, self._fields, args) for op, args in specs.items()}


class PagedPlan(NamedTuple):
    """What msa_paged_plan writes (int32 tensors): the lengths after the step
    [R], the ring's {head, count} [2], q_starts [R+1], row_req, row_pos, slots
    [T] and segs [n_segs+1]."""
    lens: torch.Tensor
    free_state: torch.Tensor
    q_starts: torch.Tensor
    row_req: torch.Tensor
    row_pos: torch.Tensor
    slots: torch.Tensor
    segs: torch.Tensor


class PagedCompact(NamedTuple):
    """What msa_paged_compact writes (int32 tensors): block_table [R, max_blocks],
    free_pages [n_pages], free_state [2], shares [n_pages] (None without any) and
    moves [max(1, n_pages // 2), 3]."""
    block_table: torch.Tensor
    free_pages: torch.Tensor
    free_state: torch.Tensor
    shares: torch.Tensor | None
    moves: torch.Tensor


class _CRotaryShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("T", "Hq", "Hkv", "d", "d_rot", "interleaved", "period", "offset")] + [
        ("scale", ctypes.c_float)] + [(n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")] + [
        ("zeros", ctypes.c_int)]


@dataclass(frozen=True)
class RotaryShape:
    """msa_rotary_shape: T tokens of Hq query and Hkv key heads of d features, the
    first d_rot (0: all) of which turn, paired with those d_rot/2 further on or,
    interleaved, with their neighbours.  Without positions token t is at offset
    + t % period (0: T).  scale (0: 1) multiplies the turned features.  The
    strides go by the tensors."""
    T: int
    Hq: int
    Hkv: int
    d: int
    d_rot: int = 0
    interleaved: bool = False
    period: int = 0
    offset: int = 0
    scale: float = 0.0

    def c(self) -> _CRotaryShape:
        return _CRotaryShape(self.T, self.Hq, self.Hkv, self.d, self.d_rot or self.d, self.interleaved, self.period, self.offset, self.scale)

    def __getstate__(self):
        return {n: getattr(self, n) for n in self.__dataclass_fields__}     # as PagedShape's

    @cached_property
    def _call(self):
        return binding().prepare_rotary(self.T, self.Hq, self.Hkv, self.d, self.d_rot or self.d, self.interleaved, self.period, self.offset,
                                        self.scale)


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libmsa.so (fails loudly if it is missing: there is no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(LIB_PATH)
            P, S = ctypes.c_void_p, ctypes.POINTER(_CShape)
            sz, f = ctypes.c_size_t, ctypes.c_float
            L.msa_workspace_size.argtypes = [S, ctypes.c_int]
            L.msa_workspace_size.restype = sz
            L.msa_index_select.argtypes = [S, P, P, P, P, P, sz, P]
            L.msa_sparse_attn_fwd.argtypes = [S, P, P, P, P, P, P, P, sz, P]
            L.msa_kl_fwd.argtypes = [S, P, P, P, P, P, P, f, P, P, P, P, sz, P]
            L.msa_fused_bwd.argtypes = [S, P, P, P, P, P, P, P, P, P, P, f, P, P, P, P, P, P, sz, P]
            L.msa_fused_bwd_kl.argtypes = [S, P, P, P, P, P, P, P, P, P, P, f, P, P, P, P, P, P, P, P, sz, P]
            L.msa_train_step.argtypes = [S, P, P, P, P, P, P, f, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
            L.msa_train_step_staged.argtypes = [S, P, P, P, P, P, P, f, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P,
                                                sz, P]
            L.msa_check_device_status.argtypes = [P, P]
            L.msa_block_mask.argtypes = [S, P, P, P, P, P]
            L.msa_kv_append.argtypes = [S, P, P, P, P, P, P, P]
            L.msa_warmup_kl.argtypes = [S, P, P, P, P, P, f, P, P, P, P, P, P, P, sz, P]
            PS = ctypes.POINTER(_CProjShape)
            L.msa_index_proj_workspace_size.argtypes = [PS]
            L.msa_index_proj_workspace_size.restype = sz
            L.msa_index_proj_fwd.argtypes = [PS, P, P, P, P, P, P, sz, P]
            L.msa_index_proj_bwd.argtypes = [PS, P, P, P, P, P, P, sz, P]
            GS = ctypes.POINTER(_CPagedShape)
            L.msa_paged_workspace_size.argtypes = [GS, ctypes.c_int]
            L.msa_paged_workspace_size.restype = sz
            for fn, ptrs in (("msa_paged_plan", 14), ("msa_paged_plan_held", 15), ("msa_paged_append", 11), ("msa_paged_block_scores", 8),
                             ("msa_paged_block_topk", 4), ("msa_paged_attn", 12), ("msa_paged_fork", 10), ("msa_paged_compact", 10),
                             ("msa_paged_chunk_scores", 7), ("msa_paged_chunk_attn", 12)):
                getattr(L, fn).argtypes = [GS] + [P] * ptrs + [sz, P]
            L.msa_paged_copy.argtypes = [GS, P, ctypes.c_int, P, P, P, P, P, P, sz, P]
            RS = ctypes.POINTER(_CRotaryShape)
            for fn in ("msa_rotary_fwd", "msa_rotary_bwd"):
                getattr(L, fn).argtypes = [RS] + [P] * 7
            L.msa_selftest_wait_timeout.argtypes = [P, ctypes.c_uint, P]
            for fn in ("msa_index_select", "msa_sparse_attn_fwd", "msa_kl_fwd", "msa_fused_bwd", "msa_fused_bwd_kl",
                       "msa_train_step", "msa_train_step_staged", "msa_check_device_status", "msa_block_mask",
                       "msa_warmup_kl", "msa_index_proj_fwd", "msa_index_proj_bwd", "msa_selftest_wait_timeout",
                       "msa_kv_append", "msa_paged_plan", "msa_paged_plan_held", "msa_paged_append", "msa_paged_block_scores",
                       "msa_paged_block_topk", "msa_paged_attn", "msa_paged_fork", "msa_paged_compact", "msa_paged_copy",
                       "msa_paged_chunk_scores", "msa_paged_chunk_attn", "msa_rotary_fwd", "msa_rotary_bwd"):
                getattr(L, fn).restype = ctypes.c_int
            L.msa_last_error.restype = ctypes.c_char_p
            L.msa_version.restype = ctypes.c_char_p
            L.msa_launch_count.restype = ctypes.c_ulonglong
            L.msa_kernel_timing.argtypes = [ctypes.c_int]
            L.msa_kernel_timing.restype = ctypes.c_int
            L.msa_kernel_timing_report.argtypes = [ctypes.c_char_p, sz]
            L.msa_kernel_timing_report.restype = sz
            _lib = L
        return _lib


_binding = None


def binding():
    """Load _paged_binding.so, the paged calls' marshalling (fails loudly if it is missing)."""
    global _binding
    lib()                                   # libmsa.so, which the binding is linked with
    with _lock:
        if _binding is None:
            path = os.path.join(_HERE, "_paged_binding.so")
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
            spec = importlib.util.spec_from_file_location("block_sparse_gqa_causal_gb300._paged_binding", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _binding = module
        return _binding


def _check(code: int) -> None:
    if code != 0:
        raise MsaError(code, lib().msa_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, name: str, shape, dtype) -> None:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: need a contiguous CUDA {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} cuda={t.is_cuda}")


def workspace_size(shape: Shape, op: int) -> int:
    n = lib().msa_workspace_size(ctypes.byref(shape.c()), op)
    if n == 0:
        _check(1)
    return int(n)


def new_workspace(shape: Shape, op: int, device=None) -> torch.Tensor:
    """A workspace with its 256-byte status word zeroed."""
    n = workspace_size(shape, op)
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    ws[:256].zero_()
    return ws


def _ws(ws, shape, op, device):
    if ws is None:
        ws = new_workspace(shape, op, device)
    return ws


def index_select(shape: Shape, q_idx, k_idx, *, sel_idx=None, block_scores=None, return_scores=False,
                 workspace=None, stream=None):
    """msa_index_select.  Returns sel_idx [B,Hkv,Nq,topk] int32 (and the block
    scores [B,Nq,Hkv,nb] fp32 when asked for)."""
    s = shape
    _need(q_idx, "q_idx", (s.B, s.Nq, s.Hkv, s.d_idx), torch.bfloat16)
    _need(k_idx, "k_idx", (s.B, s.rows_kv, s.d_idx), torch.bfloat16)
    dev = q_idx.device
    if sel_idx is None:
        sel_idx = torch.empty((s.B, s.Hkv, s.Nq, s.topk), dtype=torch.int32, device=dev)
    if return_scores and block_scores is None:
        block_scores = torch.empty((s.B, s.Nq, s.Hkv, s.nb), dtype=torch.float32, device=dev)
    ws = _ws(workspace, s, OP_INDEX_SELECT, dev)
    _check(lib().msa_index_select(ctypes.byref(s.c()), _ptr(q_idx), _ptr(k_idx), _ptr(sel_idx), _ptr(block_scores),
                                  _ptr(ws), ws.numel(), _stream(stream)))
    return (sel_idx, block_scores) if return_scores else sel_idx


def sparse_attn_fwd(shape: Shape, q, k, v, sel_idx, *, o=None, lse=None, workspace=None, stream=None):
    """msa_sparse_attn_fwd.  Returns (o [B,Nq,Hq,d] bf16, lse [B,Hq,Nq] fp32)."""
    s = shape
    _need(q, "q", (s.B, s.Nq, s.Hq, s.d), torch.bfloat16)
    _need(k, "k", (s.B, s.rows_kv, s.Hkv, s.d), torch.bfloat16)
    _need(v, "v", (s.B, s.rows_kv, s.Hkv, s.d), torch.bfloat16)
    _need(sel_idx, "sel_idx", (s.B, s.Hkv, s.Nq, s.topk), torch.int32)
    dev = q.device
    o = torch.empty((s.B, s.Nq, s.Hq, s.d), dtype=torch.bfloat16, device=dev) if o is None else o
    lse = torch.empty((s.B, s.Hq, s.Nq), dtype=torch.float32, device=dev) if lse is None else lse
    ws = _ws(workspace, s, OP_SPARSE_ATTN_FWD, dev)
    _check(lib().msa_sparse_attn_fwd(ctypes.byref(s.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(sel_idx), _ptr(o),
                                     _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
    return o, lse


def kl_fwd(shape: Shape, q, k, q_idx, k_idx, sel_idx, lse, kl_coef: float = 1.0, *, lse_idx=None, kl_rows=None,
           kl_loss=None, want_rows=True, lse_only=False, workspace=None, stream=None):
    """msa_kl_fwd.  Returns (kl_loss scalar tensor, lse_idx [B,Hkv,Nq], kl_rows [B,Hkv,Nq] or None).
    lse_only: compute lse_idx alone (kl_loss and kl_rows are None); the
    training step's form, whose loss then comes from fused_bwd(..., with_kl=True)."""
    s = shape
    _need(q, "q", (s.B, s.Nq, s.Hq, s.d), torch.bfloat16)
    _need(k, "k", (s.B, s.rows_kv, s.Hkv, s.d), torch.bfloat16)
    _need(q_idx, "q_idx", (s.B, s.Nq, s.Hkv, s.d_idx), torch.bfloat16)
    _need(k_idx, "k_idx", (s.B, s.rows_kv, s.d_idx), torch.bfloat16)
    _need(sel_idx, "sel_idx", (s.B, s.Hkv, s.Nq, s.topk), torch.int32)
    _need(lse, "lse", (s.B, s.Hq, s.Nq), torch.float32)
    dev = q.device
    lse_idx = torch.empty((s.B, s.Hkv, s.Nq), dtype=torch.float32, device=dev) if lse_idx is None else lse_idx
    if lse_only:
        kl_rows = kl_loss = None
    else:
        if want_rows and kl_rows is None:
            kl_rows = torch.empty((s.B, s.Hkv, s.Nq), dtype=torch.float32, device=dev)
        kl_loss = torch.empty((), dtype=torch.float32, device=dev) if kl_loss is None else kl_loss
    ws = _ws(workspace, s, OP_KL_FWD, dev)
    _check(lib().msa_kl_fwd(ctypes.byref(s.c()), _ptr(q), _ptr(k), _ptr(q_idx), _ptr(k_idx), _ptr(sel_idx),
                            _ptr(lse), ctypes.c_float(kl_coef), _ptr(lse_idx), _ptr(kl_rows), _ptr(kl_loss),
                            _ptr(ws), ws.numel(), _stream(stream)))
    return kl_loss, lse_idx, kl_rows


def fused_bwd(shape: Shape, q, k, v, o, d_o, lse, q_idx, k_idx, sel_idx, lse_idx, kl_coef: float = 1.0, *,
              grads=None, with_kl=False, kl_rows=None, kl_loss=None, workspace=None, stream=None):
    """msa_fused_bwd.  Returns (dq, dk, dv, dq_idx, dk_idx) bf16.
    with_kl: msa_fused_bwd_kl, which also gives the step's KL loss; returns
    (dq, dk, dv, dq_idx, dk_idx, kl_loss, kl_rows), kl_rows None unless a
    [B,Hkv,Nq] fp32 tensor is passed for it."""
    s = shape
    for t, n, shp in ((q, "q", (s.B, s.Nq, s.Hq, s.d)), (o, "o", (s.B, s.Nq, s.Hq, s.d)),
                      (d_o, "d_o", (s.B, s.Nq, s.Hq, s.d)), (k, "k", (s.B, s.Nk, s.Hkv, s.d)),
                      (v, "v", (s.B, s.Nk, s.Hkv, s.d)), (q_idx, "q_idx", (s.B, s.Nq, s.Hkv, s.d_idx)),
                      (k_idx, "k_idx", (s.B, s.Nk, s.d_idx))):
        _need(t, n, shp, torch.bfloat16)
    _need(lse, "lse", (s.B, s.Hq, s.Nq), torch.float32)
    _need(lse_idx, "lse_idx", (s.B, s.Hkv, s.Nq), torch.float32)
    _need(sel_idx, "sel_idx", (s.B, s.Hkv, s.Nq, s.topk), torch.int32)
    if grads is None:
        grads = tuple(torch.empty_like(t) for t in (q, k, v, q_idx, k_idx))
    dq, dk, dv, dqi, dki = grads
    if with_kl:
        kl_loss = torch.empty((), dtype=torch.float32, device=q.device) if kl_loss is None else kl_loss
        if kl_rows is not None:
            _need(kl_rows, "kl_rows", (s.B, s.Hkv, s.Nq), torch.float32)
        ws = _ws(workspace, s, OP_FUSED_BWD_KL, q.device)
        _check(lib().msa_fused_bwd_kl(ctypes.byref(s.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(d_o), _ptr(lse),
                                      _ptr(q_idx), _ptr(k_idx), _ptr(sel_idx), _ptr(lse_idx), ctypes.c_float(kl_coef),
                                      _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dqi), _ptr(dki), _ptr(kl_rows), _ptr(kl_loss),
                                      _ptr(ws), ws.numel(), _stream(stream)))
        return dq, dk, dv, dqi, dki, kl_loss, kl_rows
    ws = _ws(workspace, s, OP_FUSED_BWD, q.device)
    _check(lib().msa_fused_bwd(ctypes.byref(s.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(d_o), _ptr(lse),
                               _ptr(q_idx), _ptr(k_idx), _ptr(sel_idx), _ptr(lse_idx), ctypes.c_float(kl_coef),
                               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dqi), _ptr(dki), _ptr(ws), ws.numel(),
                               _stream(stream)))
    return dq, dk, dv, dqi, dki


def train_step(shape: Shape, q, k, v, q_idx, k_idx, d_o, kl_coef: float = 1.0, *, out=None, workspace=None,
               stream=None, input_ready=None):
    """msa_train_step: selection, forward, lse_idx, fused backward with the KL loss in one call.
    Returns a dict with sel, o, lse, lse_idx, kl_rows, kl_loss, dq, dk, dv, dq_idx, dk_idx
    (pass `out`, a dict of preallocated tensors with those keys, to reuse buffers).
    input_ready: three torch.cuda.Events (or None each), recorded after the writes
    of (q_idx, k_idx), (q, k, v) and d_o: msa_train_step_staged, whose stream waits
    on each just before the first phase reading those inputs."""
    s = shape
    for t, n, shp in ((q, "q", (s.B, s.Nq, s.Hq, s.d)), (d_o, "d_o", (s.B, s.Nq, s.Hq, s.d)),
                      (k, "k", (s.B, s.Nk, s.Hkv, s.d)), (v, "v", (s.B, s.Nk, s.Hkv, s.d)),
                      (q_idx, "q_idx", (s.B, s.Nq, s.Hkv, s.d_idx)), (k_idx, "k_idx", (s.B, s.Nk, s.d_idx))):
        _need(t, n, shp, torch.bfloat16)
    dev = q.device
    if out is None:
        out = {"sel": torch.empty((s.B, s.Hkv, s.Nq, s.topk), dtype=torch.int32, device=dev),
               "o": torch.empty_like(q), "lse": torch.empty((s.B, s.Hq, s.Nq), dtype=torch.float32, device=dev),
               "lse_idx": torch.empty((s.B, s.Hkv, s.Nq), dtype=torch.float32, device=dev),
               "kl_rows": torch.empty((s.B, s.Hkv, s.Nq), dtype=torch.float32, device=dev),
               "kl_loss": torch.empty((), dtype=torch.float32, device=dev),
               "dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
               "dq_idx": torch.empty_like(q_idx), "dk_idx": torch.empty_like(k_idx)}
    ws = _ws(workspace, s, OP_TRAIN_STEP, dev)
    args = [ctypes.byref(s.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx), _ptr(d_o),
            ctypes.c_float(kl_coef), _ptr(out["sel"]), _ptr(out["o"]), _ptr(out["lse"]), _ptr(out["lse_idx"]),
            _ptr(out.get("kl_rows")), _ptr(out["kl_loss"]), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
            _ptr(out["dq_idx"]), _ptr(out["dk_idx"])]
    if input_ready is None:
        _check(lib().msa_train_step(*args, _ptr(ws), ws.numel(), _stream(stream)))
    else:
        evs = [None if ev is None else ctypes.c_void_p(ev.cuda_event) for ev in input_ready]
        _check(lib().msa_train_step_staged(*args, *evs, _ptr(ws), ws.numel(), _stream(stream)))
    return out


def block_mask(shape: Shape, sel_idx, *, counts=False, blocks=False, stream=None):
    """msa_block_mask.  Returns the mask words [B, Hkv, ceil(Nq/128),
    ceil(nb/32)] as int32 (the uint32 bit patterns), plus the per-tile
    active-block counts [B, Hkv, T] and the ascending active-block lists
    [B, Hkv, T, nb] (-1 padded) when asked for."""
    s = shape
    _need(sel_idx, "sel_idx", (s.B, s.Hkv, s.Nq, s.topk), torch.int32)
    T, W = (s.Nq + 127) // 128, (s.nb + 31) // 32
    dev = sel_idx.device
    mask = torch.empty((s.B, s.Hkv, T, W), dtype=torch.int32, device=dev)
    cnt = torch.empty((s.B, s.Hkv, T), dtype=torch.int32, device=dev) if counts else None
    blk = torch.empty((s.B, s.Hkv, T, s.nb), dtype=torch.int32, device=dev) if blocks else None
    _check(lib().msa_block_mask(ctypes.byref(s.c()), _ptr(sel_idx), _ptr(mask), _ptr(cnt), _ptr(blk),
                                _stream(stream)))
    out = (mask,) + ((cnt,) if counts else ()) + ((blk,) if blocks else ())
    return out[0] if len(out) == 1 else out


def kv_append(shape: Shape, k_new, v_new, k_idx_new, k, v, k_idx, *, stream=None) -> None:
    """msa_kv_append: the Nq new tokens' K, V [B, Nq, Hkv, d] and K_idx
    [B, Nq, d_idx] rows into the caches k, v [B, kv_rows, Hkv, d] and k_idx
    [B, kv_rows, d_idx] at rows q_offset .. q_offset+Nq-1 (a pair given as
    None, None is skipped)."""
    s = shape
    for new, cache, row in ((k_new, k, (s.Hkv, s.d)), (v_new, v, (s.Hkv, s.d)), (k_idx_new, k_idx, (s.d_idx,))):
        if new is not None:
            _need(new, "new rows", (s.B, s.Nq) + row, torch.bfloat16)
        if cache is not None:
            _need(cache, "cache", (s.B, s.rows_kv) + row, torch.bfloat16)
    _check(lib().msa_kv_append(ctypes.byref(s.c()), _ptr(k_new), _ptr(v_new), _ptr(k_idx_new), _ptr(k), _ptr(v),
                               _ptr(k_idx), _stream(stream)))


def paged_workspace_size(shape: PagedShape, op: int) -> int:
    n = lib().msa_paged_workspace_size(ctypes.byref(shape.c()), op)
    if n == 0:
        _check(1)
    return int(n)


def new_paged_workspace(shape: PagedShape, op: int, device=None) -> torch.Tensor:
    """A workspace of a paged call, its first 4,096 bytes (status word, arrival counts) zeroed."""
    dev = torch.device("cuda" if device is None else device)
    with torch.cuda.device(dev) if dev.type == "cuda" else contextlib.nullcontext():     # its size goes by the device's SMs
        ws = torch.empty(paged_workspace_size(shape, op), dtype=torch.uint8, device=dev)
        ws[:4096].zero_()
    return ws


def _paged(shape: PagedShape, op: int, workspace, stream, *tensors):
    """A paged call through the binding, which checks the tensors, on their device and its current stream; the outputs."""
    if stream is not None:
        # outputs and workspace are allocated on the stream as well, so that they are not handed out again before the
        # call's kernels are done with them
        dev = next(t.device for t in tensors if t is not None)
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        with torch.cuda.stream(stream):
            return _paged(shape, op, workspace, None, *tensors)
    if workspace is None:
        dev = next(t.device for t in tensors if t is not None)
        workspace = new_paged_workspace(shape, op[0] if type(op) is tuple else op, dev)
    calls = shape._calls if op in shape._calls else shape._more_calls
    r = (_binding or binding()).call(calls[op], workspace, *tensors)
    if type(r) is int:
        _check(r)
    return r


def paged_plan(shape: PagedShape, new_lens, lens, block_table, free_pages, free_state, *, ended=None, held=None, out=None,
               workspace=None, stream=None) -> PagedPlan:
    """msa_paged_plan: the step's pages, block tables and slot maps from the
    requests' lengths.  new_lens, lens, ended [R], free_state [2] int32; block_table
    [R, max_blocks] and free_pages [n_pages] int32 are updated in place.  held [R]
    int32, the pages in each slot's row of the table, is updated in place too: with
    it (msa_paged_plan_held) lengths may be lowered between steps.  Returns a
    PagedPlan (pass `out` to reuse its tensors; its lens and free_state may be
    the tensors passed in)."""
    return PagedPlan(*_paged(shape, OP_PAGED_PLAN, workspace, stream, new_lens, lens, ended, held, block_table, free_pages, free_state,
                             *(out or (None,) * 7)))


def paged_append(shape: PagedShape, k_new, v_new, k_idx_new, slots, segs, k8, v8, k_scale, v_scale, k_idx, *,
                 workspace=None, stream=None) -> None:
    """msa_paged_append: the rows k_new, v_new [T, Hkv, d] and k_idx_new [T, d_idx]
    (bf16) into the caches k8, v8 [n_pages, Hkv, 128, d] (float8_e4m3fn) with
    k_scale, v_scale [n_pages, Hkv] (fp32), and k_idx [n_pages, 128, d_idx] (bf16),
    at a plan's slots and segs.  The K and V group, or the K_idx pair, may be None."""
    _paged(shape, OP_PAGED_APPEND, workspace, stream, k_new, v_new, k_idx_new, slots, segs, k8, v8, k_scale, v_scale, k_idx)


def paged_block_scores(shape: PagedShape, q_idx, k_idx, block_table, q_starts, row_req, row_pos, *, block_scores=None,
                       workspace=None, stream=None):
    """msa_paged_block_scores: [T, Hkv, max_blocks] fp32 of q_idx [T, Hkv, d_idx] and
    the pages k_idx [n_pages, 128, d_idx] (bf16)."""
    return _paged(shape, OP_PAGED_BLOCK_SCORES, workspace, stream, q_idx, k_idx, block_table, q_starts, row_req, row_pos,
                  block_scores)[0]


def paged_block_topk(shape: PagedShape, block_scores, row_pos, *, sel_idx=None, workspace=None, stream=None):
    """msa_paged_block_topk: sel_idx [T, Hkv, topk] int32 of block_scores [T, Hkv, max_blocks]."""
    return _paged(shape, OP_PAGED_BLOCK_TOPK, workspace, stream, block_scores, row_pos, sel_idx)[0]


def paged_attn(shape: PagedShape, q, k8, v8, k_scale, v_scale, block_table, row_req, row_pos, *, sel_idx=None, o=None,
               lse=None, workspace=None, stream=None):
    """msa_paged_attn: (o [T, Hq, d] bf16, lse [T, Hq] fp32) of q [T, Hq, d] bf16 over
    the 8-bit cache: the blocks of sel_idx [T, Hkv, topk], or all of them when it is None."""
    return _paged(shape, OP_PAGED_ATTN, workspace, stream, q, k8, v8, k_scale, v_scale, block_table, row_req, row_pos, sel_idx, o, lse)


def paged_fork(shape: PagedShape, src, lens, block_table, free_pages, free_state, shares, *, fork_lens=None, held=None, moves=None,
               workspace=None, stream=None):
    """msa_paged_fork: slot r goes on from slot src[r]'s cache (r: as it is, -1: it
    ends), from its first fork_lens[r] tokens (all of them).  src, fork_lens,
    lens, held [R], block_table [R, max_blocks], free_pages, shares [n_pages] and
    free_state [2] int32; all but src and fork_lens are updated in place.
    Returns moves [R, 3], the copies that paged_copy has to make in each layer's
    caches before anything is appended."""
    return _paged(shape, OP_PAGED_FORK, workspace, stream, src, fork_lens, lens, held, block_table, free_pages, free_state, shares, moves)[0]


def paged_compact(shape: PagedShape, lens, block_table, shares=None, *, held=None, out=None, workspace=None, stream=None) -> PagedCompact:
    """msa_paged_compact: the pages in use moved to the front of the pool, for
    paged_copy in each layer's caches.  lens, held [R], block_table [R, max_blocks],
    shares [n_pages] int32.  Pass `out` to reuse its tensors; its block_table
    and shares may be the tensors passed in."""
    o = list(out or (None,) * 5)
    if shares is None:
        t, f, s, m = _paged(shape, (OP_PAGED_COMPACT, None), workspace, stream, lens, held, block_table, None, o[0], o[1], o[2], None, o[4])
        return PagedCompact(t, f, s, None, m)
    return PagedCompact(*_paged(shape, OP_PAGED_COMPACT, workspace, stream, lens, held, block_table, shares, *o))


def paged_copy(shape: PagedShape, moves, k8, v8, k_scale, v_scale, k_idx, *, workspace=None, stream=None) -> None:
    """msa_paged_copy: the moves [n, 3] int32 of paged_fork or paged_compact, made in a
    layer's caches (as paged_append's).  The K and V group, or k_idx, may be None."""
    _paged(shape, OP_PAGED_COPY, workspace, stream, moves, k8, v8, k_scale, v_scale, k_idx)


def paged_chunk_scores(shape: PagedShape, q_idx, k_idx, block_table, q_starts, row_pos, *, block_scores=None, workspace=None, stream=None):
    """msa_paged_chunk_scores: paged_block_scores for chunks of new tokens."""
    return _paged(shape, OP_PAGED_CHUNK_SCORES, workspace, stream, q_idx, k_idx, block_table, q_starts, row_pos, block_scores)[0]


def paged_chunk_attn(shape: PagedShape, q, k8, v8, k_scale, v_scale, block_table, q_starts, row_pos, *, sel_idx=None, o=None, lse=None,
                     workspace=None, stream=None):
    """msa_paged_chunk_attn: paged_attn for chunks of new tokens, (o [T, Hq, d] bf16, lse [T, Hq] fp32)."""
    return _paged(shape, OP_PAGED_CHUNK_ATTN, workspace, stream, q, k8, v8, k_scale, v_scale, block_table, q_starts, row_pos, sel_idx, o, lse)


def rotary_freqs(d_rot: int, base: float = 10000.0, *, factor: float = 1.0, original_len: int = 0, low: float = 1.0, high: float = 4.0,
                 device=None) -> torch.Tensor:
    """The frequencies of msa_rotary_fwd, d_rot/2 64-bit fractions of a turn, of f_i =
    base^(-2i / d_rot) radians a position.  For contexts `factor` times longer: all
    divided by it (original_len 0), or only those that turn `low` times or less over
    the original_len tokens that the model was trained on; those that turn `high`
    times or more stay, and between the two the share that is divided falls evenly.
    low and high, and whether the turned features are scaled as well, are what a
    checkpoint was adapted with: the defaults, 1 and 4, go with no scale; 1 and 32
    with rotary_scale(factor)."""
    if d_rot < 2 or d_rot % 2 or not base > 1 or not factor >= 1 or original_len < 0 or not 0 <= low < high:
        raise ValueError("rotary_freqs: need an even d_rot >= 2, base > 1, factor >= 1, original_len >= 0, 0 <= low < high")
    turns = []
    for i in range(d_rot // 2):
        f = float(base) ** (-2 * i / d_rot) / (2 * math.pi)
        kept = min(1.0, max(0.0, (original_len * f - low) / (high - low))) if original_len else 0.0
        turns.append(round((f * kept + f / factor * (1 - kept)) * 2.0 ** 64))
    return torch.tensor(turns, dtype=torch.int64, device=device or "cuda")


def rotary_scale(factor: float) -> float:
    """The scale of the turned features that goes with rotary_freqs(.., factor=factor, low=1, high=32): 1 + 0.1 ln factor.
    Not for checkpoints of the default ramp, whose logits it would make (1 + 0.1 ln factor)^2 times as large."""
    return 1.0 + 0.1 * math.log(factor) if factor > 1 else 1.0


def _rotary(shape: RotaryShape, back: bool, q, k, freqs, positions, q_out, k_out, stream):
    if stream is not None:
        dev = freqs.device
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        with torch.cuda.stream(stream):
            return _rotary(shape, back, q, k, freqs, positions, q_out, k_out, None)
    r = (_binding or binding()).rotary(shape._call, back, q, k, positions, freqs, q_out, k_out)
    if type(r) is int:
        _check(r)
    return r


def rotary_fwd(shape: RotaryShape, q, k, freqs, *, positions=None, q_out=None, k_out=None, stream=None):
    """msa_rotary_fwd: (q_out, k_out) of q [.., Hq, d] and k [.., Hkv, d] bf16, T tokens
    each, evenly spaced (slices of one projection's output, say); one may be
    None.  freqs: rotary_freqs'.  positions [T] int32.  q_out may be q, k_out k.
    Outputs that are not given are zeros for tokens with a negative position, those
    given are left as they were."""
    return _rotary(shape, False, q, k, freqs, positions, q_out, k_out, stream)


def rotary_bwd(shape: RotaryShape, dq_out, dk_out, freqs, *, positions=None, dq=None, dk=None, stream=None):
    """msa_rotary_bwd: (dq, dk), the gradients of rotary_fwd's inputs from those of its outputs."""
    return _rotary(shape, True, dq_out, dk_out, freqs, positions, dq, dk, stream)


def check_device_status(workspace, stream=None) -> None:
    """msa_check_device_status: raises MsaError on a recorded device-side error."""
    _check(lib().msa_check_device_status(_ptr(workspace), _stream(stream)))


def kernel_timing(enable: bool) -> bool:
    """msa_kernel_timing: bracket each library kernel with CUDA events on its
    stream while enabled (clears earlier records); returns the previous setting."""
    return bool(lib().msa_kernel_timing(1 if enable else 0))


def kernel_times() -> dict:
    """msa_kernel_timing_report: {kernel name: (launches, total ms)} of the
    launches recorded since timing was last switched."""
    L = lib()
    need = int(L.msa_kernel_timing_report(None, 0))
    buf = ctypes.create_string_buffer(need)
    L.msa_kernel_timing_report(buf, need)
    out = {}
    for line in buf.value.decode().splitlines():
        name, n, ms = line.split()
        out[name] = (int(n), float(ms))
    return out


def launch_count() -> int:
    """Kernels launched through the library by this process so far."""
    return int(lib().msa_launch_count())


def version() -> str:
    return lib().msa_version().decode()


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def warmup_kl(shape: Shape, q, k, v, q_idx, k_idx, kl_coef: float = 1.0, *, out=None, workspace=None, stream=None):
    """msa_warmup_kl: the dense indexer warm-up loss and its gradient in the
    index inputs.  Returns a dict with lse [B,Hq,Nq], lse_idx, kl_rows
    [B,Hkv,Nq], kl_loss (scalar), dq_idx, dk_idx (bf16)."""
    s = shape
    for t, n, shp in ((q, "q", (s.B, s.Nq, s.Hq, s.d)), (k, "k", (s.B, s.Nk, s.Hkv, s.d)),
                      (v, "v", (s.B, s.Nk, s.Hkv, s.d)), (q_idx, "q_idx", (s.B, s.Nq, s.Hkv, s.d_idx)),
                      (k_idx, "k_idx", (s.B, s.Nk, s.d_idx))):
        _need(t, n, shp, torch.bfloat16)
    dev = q.device
    if out is None:
        f32 = dict(dtype=torch.float32, device=dev)
        out = {"lse": torch.empty((s.B, s.Hq, s.Nq), **f32), "lse_idx": torch.empty((s.B, s.Hkv, s.Nq), **f32),
               "kl_rows": torch.empty((s.B, s.Hkv, s.Nq), **f32), "kl_loss": torch.empty((), **f32),
               "dq_idx": torch.empty_like(q_idx), "dk_idx": torch.empty_like(k_idx)}
    ws = _ws(workspace, s, OP_WARMUP_KL, dev)
    _check(lib().msa_warmup_kl(ctypes.byref(s.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx),
                               ctypes.c_float(kl_coef), _ptr(out["lse"]), _ptr(out["lse_idx"]), _ptr(out["kl_rows"]),
                               _ptr(out["kl_loss"]), _ptr(out["dq_idx"]), _ptr(out["dk_idx"]), _ptr(ws), ws.numel(),
                               _stream(stream)))
    return out


def proj_workspace(shape: ProjShape, device=None) -> torch.Tensor:
    n = lib().msa_index_proj_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        _check(1)
    ws = torch.empty(int(n), dtype=torch.uint8, device=device or "cuda")
    ws[:256].zero_()
    return ws


def index_proj_fwd(shape: ProjShape, x, wq_idx, wk_idx, *, q_idx=None, k_idx=None, workspace=None, stream=None):
    """msa_index_proj_fwd: q_idx [T, Hkv, d_idx], k_idx [T, d_idx] (bf16) of x [T, Dm]."""
    s = shape
    _need(x, "x", (s.T, s.Dm), torch.bfloat16)
    _need(wq_idx, "wq_idx", (s.Dm, s.Hkv * s.d_idx), torch.bfloat16)
    _need(wk_idx, "wk_idx", (s.Dm, s.d_idx), torch.bfloat16)
    dev = x.device
    q_idx = torch.empty((s.T, s.Hkv, s.d_idx), dtype=torch.bfloat16, device=dev) if q_idx is None else q_idx
    k_idx = torch.empty((s.T, s.d_idx), dtype=torch.bfloat16, device=dev) if k_idx is None else k_idx
    ws = proj_workspace(s, dev) if workspace is None else workspace
    _check(lib().msa_index_proj_fwd(ctypes.byref(s.c()), _ptr(x), _ptr(wq_idx), _ptr(wk_idx), _ptr(q_idx),
                                    _ptr(k_idx), _ptr(ws), ws.numel(), _stream(stream)))
    return q_idx, k_idx


def index_proj_bwd(shape: ProjShape, x, dq_idx, dk_idx, *, dwq=None, dwk=None, workspace=None, stream=None):
    """msa_index_proj_bwd: dwq [Dm, Hkv*d_idx], dwk [Dm, d_idx] (fp32); x gets no gradient."""
    s = shape
    _need(x, "x", (s.T, s.Dm), torch.bfloat16)
    _need(dq_idx, "dq_idx", (s.T, s.Hkv, s.d_idx), torch.bfloat16)
    _need(dk_idx, "dk_idx", (s.T, s.d_idx), torch.bfloat16)
    dev = x.device
    dwq = torch.empty((s.Dm, s.Hkv * s.d_idx), dtype=torch.float32, device=dev) if dwq is None else dwq
    dwk = torch.empty((s.Dm, s.d_idx), dtype=torch.float32, device=dev) if dwk is None else dwk
    ws = proj_workspace(s, dev) if workspace is None else workspace
    _check(lib().msa_index_proj_bwd(ctypes.byref(s.c()), _ptr(x), _ptr(dq_idx), _ptr(dk_idx), _ptr(dwq), _ptr(dwk),
                                    _ptr(ws), ws.numel(), _stream(stream)))
    return dwq, dwk


def selftest_wait_timeout(workspace, spin_limit: int = 4096, stream=None) -> None:
    """msa_selftest_wait_timeout: one thread's bounded wait on a barrier that
    nothing arrives on runs out and is recorded in the workspace's status word."""
    _check(lib().msa_selftest_wait_timeout(_ptr(workspace), int(spin_limit), _stream(stream)))
