"""MiniMax Sparse Attention (MSA) hot path for NVIDIA GB300 (sm_103a).

A thin ctypes binding over libmsa.so (C ABI in include/msa.h).  Every function
here only marshals arguments: it checks dtypes, shapes and devices, allocates
outputs with torch when the caller passes none, and calls the C entry point of
the same name on torch's current CUDA stream.  All arithmetic runs in the CUDA
kernels; there is no CPU path.  Importing this package without the built
library raises immediately.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmsa.so")

MSA_PHASE_DECODE = 0
MSA_PHASE_PREFILL = 1
MSA_PHASE_DECODE_MULTI = 2
MSA_OP_INVERT = 0
MSA_OP_DECODE = 1
MSA_OP_PREFILL = 2
MSA_OP_SELECT_PREFILL = 3
MSA_OP_SELECT_INVERT_PREFILL = 4
MSA_OP_TREE = 5
MSA_TREE_MAX_NODES = 64

STATUS = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_CUDA",
          4: "MSA_ERR_DEVICE_BOUNDS", 5: "MSA_ERR_TIMEOUT", 6: "MSA_ERR_WORKSPACE",
          7: "MSA_ERR_DEVICE_UNSUPPORTED"}


class MsaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")
        self.status = status


class msa_dims_t(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("G", ctypes.c_int32), ("D", ctypes.c_int32),
                ("Di", ctypes.c_int32), ("page_size", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("sm_scale", ctypes.c_float)]


@dataclass(frozen=True)
class Dims:
    Hq: int
    G: int
    D: int
    Di: int
    topk: int
    max_blocks: int
    sm_scale: Optional[float] = None
    page_size: int = 128

    def c(self) -> msa_dims_t:
        sc = self.sm_scale if self.sm_scale is not None else 1.0 / math.sqrt(self.D)
        return msa_dims_t(self.Hq, self.G, self.D, self.Di, self.page_size, self.topk, self.max_blocks, sc)

    def ref(self):
        """A ctypes reference to c(), made once (the fields are frozen and the library only reads them)."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = ctypes.byref(self.c())
            object.__setattr__(self, "_ref", r)
        return r

    def __getstate__(self):   # copies and pickles make their own
        return {k: v for k, v in self.__dict__.items() if k != "_ref"}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmsa.so is not built ({LIB_PATH}); run __graft_entry__.build() "
                          "or python -m block_sparse_attention_06_gb300._build")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, S, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.POINTER(msa_dims_t)
    sigs = {
        "msa_index_score": [P, P, P, P, P, I, I, I, D, I, P, P, P],
        "msa_topk_blocks": [P, P, I, D, P, P, P],
        "msa_build_page_table": [P, P, P, I, I, D, P, P, P, P],
        "msa_invert_selection": [P, P, I, I, D, P, P, P, P, S, P, P],
        "msa_sparse_attn_prefill": [P, P, P, P, P, P, P, P, I, I, I, D, P, P, P, S, P, P],
        "msa_lse_merge": [P, P, P, P, I, D, P, P, P, P],
        "msa_sparse_attn_decode": [P, P, P, P, P, I, I, D, P, P, P, S, P, P],
        "msa_decode_step": [P, P, P, P, P, P, P, I, I, D, P, P, P, P, P, P, P, S, P, P],
        "msa_offload_gather": [P, P, I, P, I, D, P, P, P, P, P],
        "msa_stage_from_host": [P, P, S, P],
        "msa_select_prefill": [P, P, P, P, P, I, I, I, D, P, P, S, P, P],
        "msa_tree_rows": [P, P, P, I, I, D, P, P, P, P, P],
        "msa_tree_index_score": [P, P, P, P, P, P, P, I, I, I, D, P, P, P],
        "msa_sparse_attn_tree": [P, P, P, P, P, P, P, P, P, P, I, I, I, D, P, P, P, S, P, P],
        "msa_verify_tree": [P, P, I, P, P, P, P, P, I, I, P, P, P, P, P],
        "msa_commit_tree": [P, P, P, I, P, P, P, P, P, P, P, P, I, I, I, D, P, P, P],
        "msa_check": [P, P],
    }
    for name, argt in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argt
        fn.restype = ctypes.c_int
    lib.msa_workspace_bytes.argtypes = [I, I, I, D]
    lib.msa_workspace_bytes.restype = ctypes.c_size_t
    lib.msa_last_error.restype = ctypes.c_char_p
    lib.msa_last_error.argtypes = []
    lib.msa_status_str.restype = ctypes.c_char_p
    lib.msa_status_str.argtypes = [ctypes.c_int]
    lib.msa_version.restype = ctypes.c_int32
    lib.msa_version.argtypes = []
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _call(name: str, *args):
    rc = getattr(_lib, name)(*args)
    if rc != 0:
        raise MsaError(rc, name, _lib.msa_last_error().decode(errors="replace"))


def _req_result(t: torch.Tensor, dtype, name: str, shape=None):
    """A decode result buffer: a CUDA tensor, or a page-locked CPU tensor that the attention
    kernel writes directly over the host link."""
    if isinstance(t, torch.Tensor) and not t.is_cuda:
        if not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or page-locked (pinned) host memory")
        if t.dtype != dtype or not t.is_contiguous() or (shape is not None and tuple(t.shape) != tuple(shape)):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
        return t
    return _req(t, dtype, name, shape)


def _req(t: torch.Tensor, dtype, name: str, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def new_err_word(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def msa_check(err_word: torch.Tensor) -> None:
    """Synchronise the current stream, raise MsaError if a kernel flagged an error, clear the word."""
    _req(err_word, torch.int32, "err_word")
    _call("msa_check", _ptr(err_word), _stream(err_word.device))


def msa_selftest_timeout(err_word: torch.Tensor) -> None:
    """Queue the device self-test of the bounded-wait timeout: a wait that nothing
    completes gives up after its limit (2 s) and raises MSA_FLAG_TIMEOUT in err_word,
    which the next msa_check reports as MSA_ERR_TIMEOUT."""
    _req(err_word, torch.int32, "err_word")
    _call("msa_selftest_timeout", _ptr(err_word), _stream(err_word.device))


def msa_workspace_bytes(op: int, n_rows: int, n_req: int, dims: Dims) -> int:
    d = dims.c()
    return int(_lib.msa_workspace_bytes(op, n_rows, n_req, ctypes.byref(d)))


def msa_index_score(q_idx, kidx_cache, block_table, q_req, q_pos, dims: Dims, phase: int,
                    scores=None, err_word=None):
    n_rows = q_idx.shape[0]
    _req(q_idx, torch.bfloat16, "q_idx", (n_rows, dims.G, dims.Di))
    _req(kidx_cache, torch.bfloat16, "kidx_cache")
    if kidx_cache.dim() != 4 or tuple(kidx_cache.shape[1:]) != (dims.page_size, dims.G, dims.Di):
        raise ValueError("kidx_cache must be [n_pages][128][G][Di]")
    _req(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[1] != dims.max_blocks:
        raise ValueError("block_table must be [n_req][max_blocks]")
    _req(q_req, torch.int32, "q_req", (n_rows,))
    _req(q_pos, torch.int32, "q_pos", (n_rows,))
    dev = q_idx.device
    if scores is None:
        scores = torch.empty((n_rows, dims.G, dims.max_blocks), dtype=torch.float32, device=dev)
    _req(scores, torch.float32, "scores", (n_rows, dims.G, dims.max_blocks))
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_index_score", _ptr(q_idx), _ptr(kidx_cache), _ptr(block_table), _ptr(q_req), _ptr(q_pos),
          n_rows, block_table.shape[0], kidx_cache.shape[0], ctypes.byref(d), phase, _ptr(scores),
          _ptr(err_word), _stream(dev))
    return scores


def msa_select_prefill(q_idx, kidx_cache, block_table, q_req, q_pos, dims: Dims, sel=None, workspace=None,
                       err_word=None):
    """Prefill scoring and top-k in one pass (the selection of msa_index_score +
    msa_topk_blocks, without the scores); topk <= 16."""
    n_rows = q_idx.shape[0]
    _req(q_idx, torch.bfloat16, "q_idx", (n_rows, dims.G, dims.Di))
    _req(kidx_cache, torch.bfloat16, "kidx_cache")
    if kidx_cache.dim() != 4 or tuple(kidx_cache.shape[1:]) != (dims.page_size, dims.G, dims.Di):
        raise ValueError("kidx_cache must be [n_pages][128][G][Di]")
    _req(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[1] != dims.max_blocks:
        raise ValueError("block_table must be [n_req][max_blocks]")
    _req(q_req, torch.int32, "q_req", (n_rows,))
    _req(q_pos, torch.int32, "q_pos", (n_rows,))
    dev = q_idx.device
    n_req = block_table.shape[0]
    if sel is None:
        sel = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, device=dev)
    _req(sel, torch.int32, "sel", (n_rows, dims.G, dims.topk))
    need = msa_workspace_bytes(MSA_OP_SELECT_PREFILL, n_rows, n_req, dims)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    _req(workspace, torch.uint8, "workspace")
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_select_prefill", _ptr(q_idx), _ptr(kidx_cache), _ptr(block_table), _ptr(q_req), _ptr(q_pos), n_rows,
          n_req, kidx_cache.shape[0], ctypes.byref(d), _ptr(sel), _ptr(workspace), workspace.numel(), _ptr(err_word),
          _stream(dev))
    return sel


def msa_topk_blocks(scores, q_pos, dims: Dims, sel=None, err_word=None):
    n_rows = scores.shape[0]
    _req(scores, torch.float32, "scores", (n_rows, dims.G, dims.max_blocks))
    _req(q_pos, torch.int32, "q_pos", (n_rows,))
    dev = scores.device
    if sel is None:
        sel = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, device=dev)
    _req(sel, torch.int32, "sel", (n_rows, dims.G, dims.topk))
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_topk_blocks", _ptr(scores), _ptr(q_pos), n_rows, ctypes.byref(d), _ptr(sel), _ptr(err_word),
          _stream(dev))
    return sel


def msa_build_page_table(sel, block_table, seq_lens, n_pages: int, dims: Dims, page_table=None, row_len=None,
                         err_word=None):
    B = sel.shape[0]
    _req(sel, torch.int32, "sel", (B, dims.G, dims.topk))
    _req(block_table, torch.int32, "block_table", (B, dims.max_blocks))
    _req(seq_lens, torch.int32, "seq_lens", (B,))
    dev = sel.device
    if page_table is None:
        page_table = torch.empty((B * dims.G, dims.topk), dtype=torch.int32, device=dev)
    if row_len is None:
        row_len = torch.empty((B * dims.G,), dtype=torch.int32, device=dev)
    _req(page_table, torch.int32, "page_table", (B * dims.G, dims.topk))
    _req(row_len, torch.int32, "row_len", (B * dims.G,))
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_build_page_table", _ptr(sel), _ptr(block_table), _ptr(seq_lens), B, n_pages, ctypes.byref(d),
          _ptr(page_table), _ptr(row_len), _ptr(err_word), _stream(dev))
    return page_table, row_len


def msa_select_invert_prefill(q_idx, kidx_cache, block_table, q_req, q_pos, dims: Dims, sel=None, blk_off=None,
                              blk_ent=None, ent_pos=None, workspace=None, err_word=None):
    """msa_select_prefill then msa_invert_selection in one call, the inversion's
    marking pass done by the list merge -> (sel, blk_off, blk_ent, ent_pos); the
    requests are the rows of block_table; topk <= 16."""
    n_rows = q_idx.shape[0]
    _req(q_idx, torch.bfloat16, "q_idx", (n_rows, dims.G, dims.Di))
    _req(kidx_cache, torch.bfloat16, "kidx_cache")
    if kidx_cache.dim() != 4 or tuple(kidx_cache.shape[1:]) != (dims.page_size, dims.G, dims.Di):
        raise ValueError("kidx_cache must be [n_pages][128][G][Di]")
    _req(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[1] != dims.max_blocks:
        raise ValueError("block_table must be [n_req][max_blocks]")
    _req(q_req, torch.int32, "q_req", (n_rows,))
    _req(q_pos, torch.int32, "q_pos", (n_rows,))
    dev = q_idx.device
    n_req = block_table.shape[0]
    n_keys = dims.G * n_req * dims.max_blocks
    if sel is None:
        sel = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, device=dev)
    if blk_off is None:
        blk_off = torch.empty((n_keys + 1,), dtype=torch.int32, device=dev)
    if blk_ent is None:
        blk_ent = torch.empty((max(1, n_rows * dims.G * dims.topk),), dtype=torch.int32, device=dev)
    if ent_pos is None:
        ent_pos = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, device=dev)
    _req(sel, torch.int32, "sel", (n_rows, dims.G, dims.topk))
    _req(blk_off, torch.int32, "blk_off", (n_keys + 1,))
    _req(blk_ent, torch.int32, "blk_ent")
    if blk_ent.numel() < n_rows * dims.G * dims.topk:
        raise ValueError("blk_ent too small")
    _req(ent_pos, torch.int32, "ent_pos", (n_rows, dims.G, dims.topk))
    need = msa_workspace_bytes(MSA_OP_SELECT_INVERT_PREFILL, n_rows, n_req, dims)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    _req(workspace, torch.uint8, "workspace")
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_select_invert_prefill", _ptr(q_idx), _ptr(kidx_cache), _ptr(block_table), _ptr(q_req), _ptr(q_pos),
          n_rows, n_req, kidx_cache.shape[0], ctypes.byref(d), _ptr(sel), _ptr(blk_off), _ptr(blk_ent),
          _ptr(ent_pos), _ptr(workspace), workspace.numel(), _ptr(err_word), _stream(dev))
    return sel, blk_off, blk_ent, ent_pos


def msa_invert_selection(sel, q_req, n_req: int, dims: Dims, blk_off=None, blk_ent=None, ent_pos=None,
                         workspace=None, err_word=None):
    """-> (blk_off, blk_ent, ent_pos): the {block -> queries} CSR and each selected
    (row, group, slot)'s position in it."""
    n_rows = sel.shape[0]
    _req(sel, torch.int32, "sel", (n_rows, dims.G, dims.topk))
    _req(q_req, torch.int32, "q_req", (n_rows,))
    dev = sel.device
    n_keys = dims.G * n_req * dims.max_blocks
    if blk_off is None:
        blk_off = torch.empty((n_keys + 1,), dtype=torch.int32, device=dev)
    if blk_ent is None:
        blk_ent = torch.empty((max(1, n_rows * dims.G * dims.topk),), dtype=torch.int32, device=dev)
    _req(blk_off, torch.int32, "blk_off", (n_keys + 1,))
    _req(blk_ent, torch.int32, "blk_ent")
    if blk_ent.numel() < n_rows * dims.G * dims.topk:
        raise ValueError("blk_ent too small")
    if ent_pos is None:
        ent_pos = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, device=dev)
    _req(ent_pos, torch.int32, "ent_pos", (n_rows, dims.G, dims.topk))
    need = msa_workspace_bytes(MSA_OP_INVERT, n_rows, n_req, dims)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    _req(workspace, torch.uint8, "workspace")
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_invert_selection", _ptr(sel), _ptr(q_req), n_rows, n_req, ctypes.byref(d), _ptr(blk_off),
          _ptr(blk_ent), _ptr(ent_pos), _ptr(workspace), workspace.numel(), _ptr(err_word), _stream(dev))
    return blk_off, blk_ent, ent_pos


def partials_shape(n_ent: int, hpg: int, D: int):
    """Shape of the prefill partials buffer: per entry, D // 8 column chunks x hpg heads x 8 bf16
    (the layout msa.h documents)."""
    return (n_ent, D // 8, hpg, 8)


def partials_entry_major(o_part, n_ent: int, hpg: int, D: int):
    """The partials rearranged as [n_ent][hpg][D] (a permute; for inspection and tests)."""
    return o_part[:n_ent].permute(0, 2, 1, 3).reshape(n_ent, hpg, D)


def partials_from_entry_major(o_ent, hpg: int, D: int):
    """[n_ent][hpg][D] partials rearranged into the prefill partials layout (the inverse of
    partials_entry_major)."""
    n_ent = o_ent.shape[0]
    return o_ent.reshape(n_ent, hpg, D // 8, 8).permute(0, 2, 1, 3).contiguous()


def msa_sparse_attn_prefill(q, k_cache, v_cache, block_table, q_req, q_pos, blk_off, blk_ent, dims: Dims,
                            o_part=None, lse_part=None, workspace=None, err_word=None):
    n_rows = q.shape[0]
    _req(q, torch.bfloat16, "q", (n_rows, dims.Hq, dims.D))
    _req(k_cache, torch.bfloat16, "k_cache")
    _req(v_cache, torch.bfloat16, "v_cache", tuple(k_cache.shape))
    if k_cache.dim() != 4 or tuple(k_cache.shape[1:]) != (dims.page_size, dims.G, dims.D):
        raise ValueError("k_cache must be [n_pages][128][G][D]")
    _req(block_table, torch.int32, "block_table")
    n_req = block_table.shape[0]
    _req(q_req, torch.int32, "q_req", (n_rows,))
    _req(q_pos, torch.int32, "q_pos", (n_rows,))
    _req(blk_off, torch.int32, "blk_off", (dims.G * n_req * dims.max_blocks + 1,))
    _req(blk_ent, torch.int32, "blk_ent")
    dev = q.device
    n_ent, hpg = n_rows * dims.G * dims.topk, dims.Hq // dims.G
    if o_part is None:
        o_part = torch.empty(partials_shape(n_ent, hpg, dims.D), dtype=torch.bfloat16, device=dev)
    if lse_part is None:
        lse_part = torch.empty((n_ent, hpg), dtype=torch.float32, device=dev)
    _req(o_part, torch.bfloat16, "o_part", partials_shape(n_ent, hpg, dims.D))
    _req(lse_part, torch.float32, "lse_part", (n_ent, hpg))
    need = msa_workspace_bytes(MSA_OP_PREFILL, n_rows, n_req, dims)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    _req(workspace, torch.uint8, "workspace")
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_sparse_attn_prefill", _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(q_req),
          _ptr(q_pos), _ptr(blk_off), _ptr(blk_ent), n_rows, n_req, k_cache.shape[0], ctypes.byref(d),
          _ptr(o_part), _ptr(lse_part), _ptr(workspace), workspace.numel(), _ptr(err_word), _stream(dev))
    return o_part, lse_part


def msa_lse_merge(o_part, lse_part, sel, ent_pos, dims: Dims, out=None, lse=None, err_word=None):
    n_rows = sel.shape[0]
    n_ent, hpg = n_rows * dims.G * dims.topk, dims.Hq // dims.G
    _req(o_part, torch.bfloat16, "o_part", partials_shape(n_ent, hpg, dims.D))
    _req(lse_part, torch.float32, "lse_part", (n_ent, hpg))
    _req(sel, torch.int32, "sel", (n_rows, dims.G, dims.topk))
    _req(ent_pos, torch.int32, "ent_pos", (n_rows, dims.G, dims.topk))
    dev = o_part.device
    if out is None:
        out = torch.empty((n_rows, dims.Hq, dims.D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((n_rows, dims.Hq), dtype=torch.float32, device=dev)
    _req(out, torch.bfloat16, "out", (n_rows, dims.Hq, dims.D))
    _req(lse, torch.float32, "lse", (n_rows, dims.Hq))
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_lse_merge", _ptr(o_part), _ptr(lse_part), _ptr(sel), _ptr(ent_pos), n_rows, ctypes.byref(d),
          _ptr(out), _ptr(lse), _ptr(err_word), _stream(dev))
    return out, lse


def msa_sparse_attn_decode(q, k_cache, v_cache, page_table, row_len, dims: Dims, out=None, lse=None,
                           workspace=None, err_word=None):
    B = q.shape[0]
    _req(q, torch.bfloat16, "q", (B, dims.Hq, dims.D))
    _req(k_cache, torch.bfloat16, "k_cache")
    _req(v_cache, torch.bfloat16, "v_cache", tuple(k_cache.shape))
    if k_cache.dim() != 4 or tuple(k_cache.shape[1:]) != (dims.page_size, dims.G, dims.D):
        raise ValueError("k_cache must be [n_pages][128][G][D]")
    _req(page_table, torch.int32, "page_table", (B * dims.G, dims.topk))
    _req(row_len, torch.int32, "row_len", (B * dims.G,))
    dev = q.device
    if out is None:
        out = torch.empty((B, dims.Hq, dims.D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, dims.Hq), dtype=torch.float32, device=dev)
    _req_result(out, torch.bfloat16, "out", (B, dims.Hq, dims.D))
    _req_result(lse, torch.float32, "lse", (B, dims.Hq))
    need = msa_workspace_bytes(MSA_OP_DECODE, B, 0, dims)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    _req(workspace, torch.uint8, "workspace")
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_sparse_attn_decode", _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(row_len), B,
          k_cache.shape[0], ctypes.byref(d), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
          _ptr(err_word), _stream(dev))
    return out, lse


def msa_offload_gather(host_k_cache, host_v_cache, page_table, dims: Dims, pool_k=None, pool_v=None,
                       pool_page_table=None, err_word=None):
    """Gather the selected group slices of host-resident K/V pages into a device pool;
    returns (pool_k, pool_v, pool_page_table) for msa_sparse_attn_decode."""
    for t, name in ((host_k_cache, "host_k_cache"), (host_v_cache, "host_v_cache")):
        if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 CPU tensor")
        if not t.is_pinned():
            raise ValueError(f"{name} must be page-locked (pin_memory)")
        if t.dim() != 4 or tuple(t.shape[1:]) != (dims.page_size, dims.G, dims.D):
            raise ValueError(f"{name} must be [n_pages][128][G][D]")
    if tuple(host_v_cache.shape) != tuple(host_k_cache.shape):
        raise ValueError("host_v_cache must match host_k_cache")
    rows = page_table.shape[0]
    _req(page_table, torch.int32, "page_table", (rows, dims.topk))
    if rows % dims.G:
        raise ValueError("page_table rows must be B*G")
    B = rows // dims.G
    dev = page_table.device
    shape = (B * dims.topk, dims.page_size, dims.G, dims.D)
    pool_k = torch.empty(shape, dtype=torch.bfloat16, device=dev) if pool_k is None else pool_k
    pool_v = torch.empty(shape, dtype=torch.bfloat16, device=dev) if pool_v is None else pool_v
    _req(pool_k, torch.bfloat16, "pool_k", shape)
    _req(pool_v, torch.bfloat16, "pool_v", shape)
    if pool_page_table is None:
        pool_page_table = torch.empty_like(page_table)
    _req(pool_page_table, torch.int32, "pool_page_table", tuple(page_table.shape))
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_offload_gather", _ptr(host_k_cache), _ptr(host_v_cache), host_k_cache.shape[0], _ptr(page_table), B,
          ctypes.byref(d), _ptr(pool_k), _ptr(pool_v), _ptr(pool_page_table), _ptr(err_word), _stream(dev))
    return pool_k, pool_v, pool_page_table


def msa_decode_step(q, q_idx, k_cache, v_cache, kidx_cache, block_table, seq_lens, dims: Dims, scores=None,
                    sel=None, page_table=None, row_len=None, out=None, lse=None, workspace=None, err_word=None):
    """One whole decode step (index scan, top-k, page tables, sparse attention) in one
    call; returns (out, lse, sel, page_table, row_len, scores)."""
    B = q.shape[0]
    _req(q, torch.bfloat16, "q", (B, dims.Hq, dims.D))
    _req(q_idx, torch.bfloat16, "q_idx", (B, dims.G, dims.Di))
    _req(k_cache, torch.bfloat16, "k_cache")
    _req(v_cache, torch.bfloat16, "v_cache", tuple(k_cache.shape))
    if k_cache.dim() != 4 or tuple(k_cache.shape[1:]) != (dims.page_size, dims.G, dims.D):
        raise ValueError("k_cache must be [n_pages][128][G][D]")
    _req(kidx_cache, torch.bfloat16, "kidx_cache", (k_cache.shape[0], dims.page_size, dims.G, dims.Di))
    _req(block_table, torch.int32, "block_table", (B, dims.max_blocks))
    _req(seq_lens, torch.int32, "seq_lens", (B,))
    dev = q.device
    f = dict(device=dev)
    scores = torch.empty((B, dims.G, dims.max_blocks), dtype=torch.float32, **f) if scores is None else scores
    sel = torch.empty((B, dims.G, dims.topk), dtype=torch.int32, **f) if sel is None else sel
    if page_table is None:
        page_table = torch.empty((B * dims.G, dims.topk), dtype=torch.int32, **f)
    row_len = torch.empty((B * dims.G,), dtype=torch.int32, **f) if row_len is None else row_len
    out = torch.empty((B, dims.Hq, dims.D), dtype=torch.bfloat16, **f) if out is None else out
    lse = torch.empty((B, dims.Hq), dtype=torch.float32, **f) if lse is None else lse
    _req(scores, torch.float32, "scores", (B, dims.G, dims.max_blocks))
    _req(sel, torch.int32, "sel", (B, dims.G, dims.topk))
    _req(page_table, torch.int32, "page_table", (B * dims.G, dims.topk))
    _req(row_len, torch.int32, "row_len", (B * dims.G,))
    _req_result(out, torch.bfloat16, "out", (B, dims.Hq, dims.D))
    _req_result(lse, torch.float32, "lse", (B, dims.Hq))
    need = msa_workspace_bytes(MSA_OP_DECODE, B, 0, dims)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, **f)
    _req(workspace, torch.uint8, "workspace")
    err_word = new_err_word(dev) if err_word is None else err_word
    d = dims.c()
    _call("msa_decode_step", _ptr(q), _ptr(q_idx), _ptr(k_cache), _ptr(v_cache), _ptr(kidx_cache), _ptr(block_table),
          _ptr(seq_lens), B, k_cache.shape[0], ctypes.byref(d), _ptr(scores), _ptr(sel), _ptr(page_table),
          _ptr(row_len), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(err_word), _stream(dev))
    return out, lse, sel, page_table, row_len, scores


# ------------------------------------------------------------------ drafted trees (speculative decode)

def _arg(t, dtype, shape, index: int, name: str) -> int:
    """The address of a tensor argument on device `index`, checked as _req does (which words the
    refusal).  A decode step makes these calls per layer, so the checks that pass are kept short."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _req(t, dtype, name, shape)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _lead(t, name: str) -> int:
    """The device index of the argument that decides where a call runs."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _ndim(t, n: int, name: str, what: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must be {what}")
    return t.shape


def _n_req(node_off) -> int:
    n = _ndim(node_off, 1, "node_off", "[n_req + 1]")[0] - 1
    if n < 1:
        raise ValueError("node_off must be [n_req + 1]")
    return n


def _launch(index: int, name: str, *args):
    """_call on the current stream of device `index`, with that device current."""
    if index == torch._C._cuda_getDevice():
        _call(name, *args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            _call(name, *args, torch._C._cuda_getCurrentRawStream(index))


_I32, _I64, _F32, _BF16, _U8 = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.uint8


def msa_tree_rows(node_off, parents, ctx_lens, dims: Dims, q_req=None, q_pos=None, anc=None, err_word=None):
    """Positions and ancestors of the rows of drafted trees -> (q_req, q_pos, anc); anc is int64,
    bit m of a row's word set where node m is the row's ancestor or the row itself."""
    dev = _lead(parents, "parents")
    n_req = _n_req(node_off)
    rows = _ndim(parents, 1, "parents", "[n_rows]")
    q_req = torch.empty_like(parents) if q_req is None else q_req
    q_pos = torch.empty_like(parents) if q_pos is None else q_pos
    anc = torch.empty_like(parents, dtype=_I64) if anc is None else anc
    err_word = new_err_word(parents.device) if err_word is None else err_word
    _launch(dev, "msa_tree_rows", _arg(node_off, _I32, (n_req + 1,), dev, "node_off"),
            _arg(parents, _I32, rows, dev, "parents"), _arg(ctx_lens, _I32, (n_req,), dev, "ctx_lens"), rows[0], n_req,
            dims.ref(), _arg(q_req, _I32, rows, dev, "q_req"), _arg(q_pos, _I32, rows, dev, "q_pos"),
            _arg(anc, _I64, rows, dev, "anc"), _arg(err_word, _I32, (1,), dev, "err_word"))
    return q_req, q_pos, anc


def msa_tree_index_score(q_idx, kidx_cache, kidx_new, block_table, ctx_lens, node_off, anc, dims: Dims, scores=None,
                         err_word=None):
    """Block scores of the nodes of drafted trees: msa_index_score over the cached tokens and each
    node's drafted ancestors (anc from msa_tree_rows)."""
    dev = _lead(q_idx, "q_idx")
    n_req, n_rows = _n_req(node_off), _ndim(q_idx, 3, "q_idx", "[n_rows][G][Di]")[0]
    n_pages = _ndim(kidx_cache, 4, "kidx_cache", "[n_pages][128][G][Di]")[0]
    index = (n_rows, dims.G, dims.Di)
    if scores is None:
        scores = torch.empty((n_rows, dims.G, dims.max_blocks), dtype=_F32, device=q_idx.device)
    err_word = new_err_word(q_idx.device) if err_word is None else err_word
    _launch(dev, "msa_tree_index_score", _arg(q_idx, _BF16, index, dev, "q_idx"),
            _arg(kidx_cache, _BF16, (n_pages, dims.page_size, dims.G, dims.Di), dev, "kidx_cache"),
            _arg(kidx_new, _BF16, index, dev, "kidx_new"),
            _arg(block_table, _I32, (n_req, dims.max_blocks), dev, "block_table"),
            _arg(ctx_lens, _I32, (n_req,), dev, "ctx_lens"), _arg(node_off, _I32, (n_req + 1,), dev, "node_off"),
            _arg(anc, _I64, (n_rows,), dev, "anc"), n_rows, n_req, n_pages, dims.ref(),
            _arg(scores, _F32, (n_rows, dims.G, dims.max_blocks), dev, "scores"),
            _arg(err_word, _I32, (1,), dev, "err_word"))
    return scores


def msa_sparse_attn_tree(q, k_cache, v_cache, k_new, v_new, block_table, ctx_lens, node_off, anc, sel, dims: Dims,
                         out=None, lse=None, workspace=None, err_word=None):
    """Sparse attention of the nodes of drafted trees: the cached tokens of each row's selected
    blocks and the row's drafted ancestors whose block is selected -> (out, lse)."""
    dev = _lead(q, "q")
    n_req, n_rows = _n_req(node_off), _ndim(q, 3, "q", "[n_rows][Hq][D]")[0]
    n_pages = _ndim(k_cache, 4, "k_cache", "[n_pages][128][G][D]")[0]
    heads, cache = (n_rows, dims.Hq, dims.D), (n_pages, dims.page_size, dims.G, dims.D)
    rows = (n_rows, dims.G, dims.D)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(heads[:2], dtype=_F32, device=q.device) if lse is None else lse
    if workspace is None:
        workspace = torch.empty(max(msa_workspace_bytes(MSA_OP_TREE, n_rows, n_req, dims), 1), dtype=_U8, device=q.device)
    err_word = new_err_word(q.device) if err_word is None else err_word
    ws_bytes = _ndim(workspace, 1, "workspace", "a uint8 vector")
    _launch(dev, "msa_sparse_attn_tree", _arg(q, _BF16, heads, dev, "q"), _arg(k_cache, _BF16, cache, dev, "k_cache"),
            _arg(v_cache, _BF16, cache, dev, "v_cache"), _arg(k_new, _BF16, rows, dev, "k_new"),
            _arg(v_new, _BF16, rows, dev, "v_new"),
            _arg(block_table, _I32, (n_req, dims.max_blocks), dev, "block_table"),
            _arg(ctx_lens, _I32, (n_req,), dev, "ctx_lens"), _arg(node_off, _I32, (n_req + 1,), dev, "node_off"),
            _arg(anc, _I64, (n_rows,), dev, "anc"), _arg(sel, _I32, (n_rows, dims.G, dims.topk), dev, "sel"), n_rows,
            n_req, n_pages, dims.ref(), _arg(out, _BF16, heads, dev, "out"), _arg(lse, _F32, heads[:2], dev, "lse"),
            _arg(workspace, _U8, ws_bytes, dev, "workspace"), ws_bytes[0], _arg(err_word, _I32, (1,), dev, "err_word"))
    return out, lse


def msa_verify_tree(target_probs, draft_probs, tokens, node_off, parents, u_accept, u_next, path=None,
                    n_accepted=None, next_token=None, err_word=None):
    """Accept drafted tokens against the target's probabilities from given random numbers ->
    (path, n_accepted, next_token); draft_probs None: drafts chosen without chance."""
    dev = _lead(target_probs, "target_probs")
    n_req, probs = _n_req(node_off), _ndim(target_probs, 2, "target_probs", "[n_rows][vocab]")
    n_rows, vocab = probs
    if vocab < 1:
        raise ValueError("target_probs must be [n_rows][vocab]")
    new = dict(dtype=_I32, device=target_probs.device)
    path = torch.empty(n_rows, **new) if path is None else path
    n_accepted = torch.empty(n_req, **new) if n_accepted is None else n_accepted
    next_token = torch.empty(n_req, **new) if next_token is None else next_token
    err_word = new_err_word(target_probs.device) if err_word is None else err_word
    _launch(dev, "msa_verify_tree", _arg(target_probs, _F32, probs, dev, "target_probs"),
            None if draft_probs is None else _arg(draft_probs, _F32, probs, dev, "draft_probs"), vocab,
            _arg(tokens, _I32, (n_rows,), dev, "tokens"), _arg(node_off, _I32, (n_req + 1,), dev, "node_off"),
            _arg(parents, _I32, (n_rows,), dev, "parents"), _arg(u_accept, _F32, (n_rows,), dev, "u_accept"),
            _arg(u_next, _F32, (n_req,), dev, "u_next"), n_rows, n_req, _arg(path, _I32, (n_rows,), dev, "path"),
            _arg(n_accepted, _I32, (n_req,), dev, "n_accepted"), _arg(next_token, _I32, (n_req,), dev, "next_token"),
            _arg(err_word, _I32, (1,), dev, "err_word"))
    return path, n_accepted, next_token


def _layers(t, lead: int):
    """A tensor of all layers; one layer's tensor may come without the layer dimension."""
    return t if not isinstance(t, torch.Tensor) or t.dim() == lead + 1 else t.unsqueeze(0)


def msa_commit_tree(k_new, v_new, kidx_new, k_cache, v_cache, kidx_cache, block_table, ctx_lens, node_off, path,
                    n_accepted, dims: Dims, new_lens=None, err_word=None):
    """Append the accepted paths to the caches of all layers (in place) -> new_lens.  Rows are
    [n_layers][n_rows][G][D], caches [n_layers][n_pages][128][G][D] (the k-index with Di); for one
    layer the leading dimension may be left out."""
    dev = _lead(k_new, "k_new")
    n_req = _n_req(node_off)
    k_new, v_new, kidx_new = _layers(k_new, 3), _layers(v_new, 3), _layers(kidx_new, 3)
    k_cache, v_cache, kidx_cache = _layers(k_cache, 4), _layers(v_cache, 4), _layers(kidx_cache, 4)
    L, n_rows = _ndim(k_new, 4, "k_new", "[n_layers][n_rows][G][D]")[:2]
    n_pages = _ndim(k_cache, 5, "k_cache", "[n_layers][n_pages][128][G][D]")[1]
    rows, cache = (L, n_rows, dims.G, dims.D), (L, n_pages, dims.page_size, dims.G, dims.D)
    new_lens = torch.empty(n_req, dtype=_I32, device=k_new.device) if new_lens is None else new_lens
    err_word = new_err_word(k_new.device) if err_word is None else err_word
    _launch(dev, "msa_commit_tree", _arg(k_new, _BF16, rows, dev, "k_new"), _arg(v_new, _BF16, rows, dev, "v_new"),
            _arg(kidx_new, _BF16, (L, n_rows, dims.G, dims.Di), dev, "kidx_new"), L,
            _arg(k_cache, _BF16, cache, dev, "k_cache"), _arg(v_cache, _BF16, cache, dev, "v_cache"),
            _arg(kidx_cache, _BF16, (L, n_pages, dims.page_size, dims.G, dims.Di), dev, "kidx_cache"),
            _arg(block_table, _I32, (n_req, dims.max_blocks), dev, "block_table"),
            _arg(ctx_lens, _I32, (n_req,), dev, "ctx_lens"), _arg(node_off, _I32, (n_req + 1,), dev, "node_off"),
            _arg(path, _I32, (n_rows,), dev, "path"), _arg(n_accepted, _I32, (n_req,), dev, "n_accepted"), n_rows,
            n_req, n_pages, dims.ref(), _arg(new_lens, _I32, (n_req,), dev, "new_lens"),
            _arg(err_word, _I32, (1,), dev, "err_word"))
    return new_lens


# ------------------------------------------------------------------ whole-path helpers

def dims_of(case) -> Dims:
    """Dims of a workload from the seeded generator (msa_inputs.Case)."""
    d = case.dims
    return Dims(d.Hq, d.G, d.D, d.Di, d.topk, case.max_blocks, d.sm_scale, d.page)


class DecodeStep:
    """One MSA decode step with preallocated buffers: index scoring -> top-k ->
    page table -> paged sparse attention.  Buffers are reused across calls so the
    step can be replayed (and captured in a CUDA graph).

    Calling the object runs the fused entry point msa_decode_step (three kernels);
    composed() runs the same step through the four separate entry points."""

    def __init__(self, dims: Dims, B: int, n_req: int, n_pages: int, device):
        self.dims, self.B, self.n_req, self.n_pages = dims, B, n_req, n_pages
        f = dict(device=device)
        self.scores = torch.empty((B, dims.G, dims.max_blocks), dtype=torch.float32, **f)
        self.sel = torch.empty((B, dims.G, dims.topk), dtype=torch.int32, **f)
        self.page_table = torch.empty((B * dims.G, dims.topk), dtype=torch.int32, **f)
        self.row_len = torch.empty((B * dims.G,), dtype=torch.int32, **f)
        # out and lse share one device buffer, so a step's results come back in one copy
        self._out_buf, (self.out, self.lse) = _packed(
            [((B, dims.Hq, dims.D), torch.bfloat16), ((B, dims.Hq), torch.float32)], device)
        self.workspace = torch.empty((max(1, msa_workspace_bytes(MSA_OP_DECODE, B, 0, dims)),),
                                     dtype=torch.uint8, **f)
        self.err = new_err_word(device)
        self.q_req = torch.arange(B, dtype=torch.int32, **f)
        self.kernel_launches = 3   # index scan, selection (top-k + page table), attention with merge

    def scores_only(self, q_idx, kidx_cache, block_table, q_pos):
        return msa_index_score(q_idx, kidx_cache, block_table, self.q_req, q_pos, self.dims, MSA_PHASE_DECODE,
                               scores=self.scores, err_word=self.err)

    def rest(self, q, k_cache, v_cache, block_table, q_pos, seq_lens):
        msa_topk_blocks(self.scores, q_pos, self.dims, sel=self.sel, err_word=self.err)
        msa_build_page_table(self.sel, block_table, seq_lens, self.n_pages, self.dims, self.page_table,
                             self.row_len, err_word=self.err)
        return msa_sparse_attn_decode(q, k_cache, v_cache, self.page_table, self.row_len, self.dims, self.out,
                                      self.lse, self.workspace, err_word=self.err)

    def composed(self, q, q_idx, k_cache, v_cache, kidx_cache, block_table, seq_lens, q_pos):
        self.scores_only(q_idx, kidx_cache, block_table, q_pos)
        return self.rest(q, k_cache, v_cache, block_table, q_pos, seq_lens)

    def offloaded(self, q, q_idx, host_k_cache, host_v_cache, kidx_cache, block_table, seq_lens, q_pos):
        """The step with K/V in page-locked host memory and the k-index on the GPU: scan,
        top-k and page tables on the GPU, then only the selected pages are gathered into a
        device pool (msa_offload_gather) and attended there."""
        self.scores_only(q_idx, kidx_cache, block_table, q_pos)
        msa_topk_blocks(self.scores, q_pos, self.dims, sel=self.sel, err_word=self.err)
        msa_build_page_table(self.sel, block_table, seq_lens, self.n_pages, self.dims, self.page_table,
                             self.row_len, err_word=self.err)
        if getattr(self, "_pool", None) is None:
            self._pool = (None, None, None)
        pk, pv, ppt = msa_offload_gather(host_k_cache, host_v_cache, self.page_table, self.dims, *self._pool,
                                         err_word=self.err)
        self._pool = (pk, pv, ppt)
        return msa_sparse_attn_decode(q, pk, pv, ppt, self.row_len, self.dims, self.out, self.lse, self.workspace,
                                      err_word=self.err)

    def __call__(self, q, q_idx, k_cache, v_cache, kidx_cache, block_table, seq_lens, q_pos=None, out=None,
                 lse=None):
        """The step through msa_decode_step; out and lse default to the step's device buffers
        and may be page-locked host views (host_results()), which the step then writes directly."""
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        msa_decode_step(q, q_idx, k_cache, v_cache, kidx_cache, block_table, seq_lens, self.dims, self.scores,
                        self.sel, self.page_table, self.row_len, out, lse, self.workspace, self.err)
        return out, lse

    def capture(self, q, q_idx, k_cache, v_cache, kidx_cache, block_table, seq_lens, inputs=None,
                host_results=None):
        """Record one whole step on these tensors into a CUDA graph and keep it for replay():
        a serving engine replays the decode step instead of launching its kernels one by
        one.  With `inputs` (a DecodeInputs whose device views are the tensors passed here)
        the graph also holds that step's upload, and with `host_results` (the buffer from
        host_results()) the attention kernel writes out and lse straight into that
        page-locked buffer, so they need no copy of their own.  The tensors are baked into
        the graph: write new values into them, then replay().  One eager call runs first,
        so every kernel's attributes are set before capture."""
        args = (q, q_idx, k_cache, v_cache, kidx_cache, block_table, seq_lens)
        res = {}
        if host_results is not None:
            _, (h_out, h_lse) = self._host_views(host_results)
            res = dict(out=h_out, lse=h_lse)
        if inputs is not None:
            inputs.upload()
        self._graph_results = self(*args, **res)
        torch.cuda.synchronize(q.device)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if inputs is not None:
                inputs.upload()
            self(*args, **res)
        self._graph = graph
        return graph

    def replay(self):
        """Replay the step recorded by capture() on the current stream; returns the (out,
        lse) it writes (the host views when it was captured with host_results)."""
        self._graph.replay()
        return self._graph_results

    def host_results(self):
        """Page-locked host buffer laid out like the device (out, lse) buffer, with its
        (out, lse) views: download() fills it from the device buffer, and a step given the
        views (or captured with the buffer) writes them directly."""
        buf = torch.empty(self._out_buf.shape, dtype=torch.uint8).pin_memory()
        return self._host_views(buf)

    def _host_views(self, buf):
        return buf, _views(buf, [(tuple(self.out.shape), self.out.dtype), (tuple(self.lse.shape), self.lse.dtype)])

    def download(self, host_buf):
        """Queue one device-to-host copy of out and lse into host_buf (from host_results)."""
        host_buf.copy_(self._out_buf, non_blocking=True)


def _layout(specs):
    """Byte offsets of tensors packed back to back, each on a 256-byte boundary."""
    offs, n = [], 0
    for shape, dtype in specs:
        offs.append(n)
        nbytes = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        n += (nbytes + 255) // 256 * 256
    return offs, max(n, 1)


def _views(buf, specs):
    offs, _ = _layout(specs)
    out = []
    for (shape, dtype), o in zip(specs, offs):
        nbytes = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        out.append(buf[o:o + nbytes].view(dtype).view(shape))
    return out


def _packed(specs, device):
    _, n = _layout(specs)
    buf = torch.empty((n,), dtype=torch.uint8, device=device)
    return buf, _views(buf, specs)


def msa_stage_from_host(host: torch.Tensor, dev: torch.Tensor) -> torch.Tensor:
    """Copy the bytes of a page-locked host tensor into a device tensor of the same byte
    size with the staging kernel of msa_stage_from_host (16-byte loads reading the host
    buffer in place), queued on the current stream."""
    if host.is_cuda or not host.is_pinned():
        raise ValueError("host must be a page-locked CPU tensor")
    if not host.is_contiguous():
        raise ValueError("host must be contiguous")
    _req(dev, dev.dtype, "dev")
    n = host.numel() * host.element_size()
    if dev.numel() * dev.element_size() != n:
        raise ValueError(f"dev holds {dev.numel() * dev.element_size()} bytes, host {n}")
    _call("msa_stage_from_host", _ptr(host), _ptr(dev), n, _stream(dev.device))
    return dev


class DecodeInputs:
    """The per-step inputs of a decode step for B requests -- q, q_idx, seq_lens,
    q_pos and block_table -- packed in one page-locked host buffer and one device
    buffer of the same layout, so a step's host-to-device traffic is one staging kernel
    (upload, msa_stage_from_host) instead of one copy per tensor.  Fill the host views
    (h_q, ...), call upload(), then pass the device views (q, ...) to DecodeStep."""

    def __init__(self, dims: Dims, B: int, device):
        specs = [((B, dims.Hq, dims.D), torch.bfloat16), ((B, dims.G, dims.Di), torch.bfloat16),
                 ((B,), torch.int32), ((B,), torch.int32), ((B, dims.max_blocks), torch.int32)]
        _, n = _layout(specs)
        self.host = torch.empty((n,), dtype=torch.uint8).pin_memory()
        self.h_q, self.h_q_idx, self.h_seq_lens, self.h_q_pos, self.h_block_table = _views(self.host, specs)
        self.dev, (self.q, self.q_idx, self.seq_lens, self.q_pos, self.block_table) = _packed(specs, device)

    @property
    def nbytes(self) -> int:
        return self.host.numel()

    def upload(self):
        """Queue the host-to-device copy of all inputs on the current stream: one staging
        kernel reads the page-locked buffer over the host link (a copy-engine transfer of
        these few hundred KB costs about 10 us more per step on a Grace-Blackwell node)."""
        msa_stage_from_host(self.host, self.dev)


class PrefillStep:
    """One MSA prefill chunk: tensor-core index scoring -> top-k -> {q,blk}->{blk,q}
    inversion -> KV-block-major sparse attention -> LSE merge.

    With fuse_topk (the default where topk <= 16 and max_blocks <= 8704) scoring,
    top-k and the inversion run as msa_select_invert_prefill and no scores are kept;
    otherwise msa_index_score writes `scores`, msa_topk_blocks selects from them and
    msa_invert_selection inverts."""

    def __init__(self, dims: Dims, n_rows: int, n_req: int, device, fuse_topk=None):
        self.dims, self.n_rows, self.n_req = dims, n_rows, n_req
        f = dict(device=device)
        n_chunks = (dims.max_blocks + 127) // 128
        if fuse_topk is None:
            fuse_topk = dims.topk <= 16 and n_chunks * 15 <= 1024
        self.fuse_topk = bool(fuse_topk)
        if self.fuse_topk:
            self.scores = None
            self.sel_ws = torch.empty(
                (max(1, msa_workspace_bytes(MSA_OP_SELECT_INVERT_PREFILL, n_rows, n_req, dims)),),
                dtype=torch.uint8, **f)
        else:
            self.scores = torch.empty((n_rows, dims.G, dims.max_blocks), dtype=torch.float32, **f)
        self.sel = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, **f)
        n_keys = dims.G * n_req * dims.max_blocks
        self.blk_off = torch.empty((n_keys + 1,), dtype=torch.int32, **f)
        self.blk_ent = torch.empty((max(1, n_rows * dims.G * dims.topk),), dtype=torch.int32, **f)
        self.ent_pos = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, **f)
        self.inv_ws = None if self.fuse_topk else torch.empty(
            (max(1, msa_workspace_bytes(MSA_OP_INVERT, n_rows, n_req, dims)),), dtype=torch.uint8, **f)
        self.attn_ws = torch.empty((max(1, msa_workspace_bytes(MSA_OP_PREFILL, n_rows, n_req, dims)),),
                                   dtype=torch.uint8, **f)
        n_ent, hpg = n_rows * dims.G * dims.topk, dims.Hq // dims.G
        self.o_part = torch.empty(partials_shape(n_ent, hpg, dims.D), dtype=torch.bfloat16, **f)
        self.lse_part = torch.empty((n_ent, hpg), dtype=torch.float32, **f)
        self.out = torch.empty((n_rows, dims.Hq, dims.D), dtype=torch.bfloat16, **f)
        self.lse = torch.empty((n_rows, dims.Hq), dtype=torch.float32, **f)
        self.err = new_err_word(device)
        # fused: scoring, list merge (+ the inversion's marks), 3 inversion kernels, plan, attention, merge;
        # otherwise scoring, top-k and 4 inversion kernels
        self.kernel_launches = 8 if self.fuse_topk else 9

    def select(self, q_idx, kidx_cache, block_table, q_req, q_pos):
        if self.fuse_topk:
            msa_select_invert_prefill(q_idx, kidx_cache, block_table, q_req, q_pos, self.dims, self.sel,
                                      self.blk_off, self.blk_ent, self.ent_pos, self.sel_ws, err_word=self.err)
            return
        msa_index_score(q_idx, kidx_cache, block_table, q_req, q_pos, self.dims, MSA_PHASE_PREFILL,
                        scores=self.scores, err_word=self.err)
        msa_topk_blocks(self.scores, q_pos, self.dims, sel=self.sel, err_word=self.err)
        msa_invert_selection(self.sel, q_req, self.n_req, self.dims, self.blk_off, self.blk_ent, self.ent_pos,
                             self.inv_ws, err_word=self.err)

    def attend(self, q, k_cache, v_cache, block_table, q_req, q_pos):
        msa_sparse_attn_prefill(q, k_cache, v_cache, block_table, q_req, q_pos, self.blk_off, self.blk_ent,
                                self.dims, self.o_part, self.lse_part, self.attn_ws, err_word=self.err)
        return msa_lse_merge(self.o_part, self.lse_part, self.sel, self.ent_pos, self.dims, self.out, self.lse,
                             err_word=self.err)

    def partials_by_slot(self):
        """The partials rearranged as [rows][topk][Hq][D] / [rows][topk][Hq] (host copies;
        slots with sel < 0 hold zeros / -inf).  For inspection and tests."""
        sel, pos = self.sel.cpu(), self.ent_pos.cpu()
        n_rows, G, k = sel.shape
        hpg = self.dims.Hq // G
        op = partials_entry_major(self.o_part.cpu(), n_rows * G * k, hpg, self.dims.D)
        lp = self.lse_part.cpu()
        valid = sel >= 0
        p = torch.where(valid, pos, torch.zeros_like(pos)).long()
        o = op[p]                                  # [rows][G][k][hpg][D]
        lse = lp[p]                                # [rows][G][k][hpg]
        o = torch.where(valid[..., None, None], o, torch.zeros_like(o))
        lse = torch.where(valid[..., None], lse, torch.full_like(lse, float("-inf")))
        o = o.permute(0, 2, 1, 3, 4).reshape(n_rows, k, G * hpg, -1)
        lse = lse.permute(0, 2, 1, 3).reshape(n_rows, k, G * hpg)
        return o, lse

    def __call__(self, q, q_idx, k_cache, v_cache, kidx_cache, block_table, q_req, q_pos):
        self.select(q_idx, kidx_cache, block_table, q_req, q_pos)
        return self.attend(q, k_cache, v_cache, block_table, q_req, q_pos)


class MixedStep:
    """One step of a chunked-prefill engine over ONE shared page pool: a batch of decode
    requests (one new token each) and a prefill chunk of one or more requests.  Decode
    rows take the decode path (index scan, top-k + page tables, paged attention:
    msa_decode_step); chunk rows take the block-major path (tensor-core scoring with the
    top-k fused, inversion, block-major attention, LSE merge: PrefillStep).  The two
    halves share the K, V and k-index caches and read disjoint block-table rows.

    With overlap=True the decode half runs on a side stream that forks from the caller's
    current stream and joins it again before the call returns, so the HBM-bound decode
    scan can run beside the prefill kernels where SM resources allow; otherwise both run
    in order on the current stream.  Either way every result is produced by the same
    kernels as the separate steps, so the outputs are bit-identical to them."""

    def __init__(self, dims: Dims, n_decode: int, n_prefill_rows: int, n_prefill_req: int, n_pages: int, device,
                 overlap: bool = True):
        self.decode = DecodeStep(dims, n_decode, n_decode, n_pages, device)
        self.prefill = PrefillStep(dims, n_prefill_rows, n_prefill_req, device)
        self.overlap = bool(overlap)
        self.device = torch.device(device)
        self._side = torch.cuda.Stream(device=self.device) if self.overlap else None
        self.kernel_launches = self.decode.kernel_launches + self.prefill.kernel_launches

    @property
    def err_words(self):
        return (self.decode.err, self.prefill.err)

    def __call__(self, k_cache, v_cache, kidx_cache, dec_q, dec_q_idx, dec_block_table, dec_seq_lens, pre_q,
                 pre_q_idx, pre_block_table, pre_q_req, pre_q_pos):
        """-> (decode out, decode lse, prefill out, prefill lse)"""
        if not self.overlap:
            self.decode(dec_q, dec_q_idx, k_cache, v_cache, kidx_cache, dec_block_table, dec_seq_lens)
            self.prefill(pre_q, pre_q_idx, k_cache, v_cache, kidx_cache, pre_block_table, pre_q_req, pre_q_pos)
            return self.decode.out, self.decode.lse, self.prefill.out, self.prefill.lse
        main = torch.cuda.current_stream(self.device)
        self._side.wait_stream(main)                 # inputs written on the caller's stream are visible
        with torch.cuda.stream(self._side):
            self.decode(dec_q, dec_q_idx, k_cache, v_cache, kidx_cache, dec_block_table, dec_seq_lens)
        self.prefill(pre_q, pre_q_idx, k_cache, v_cache, kidx_cache, pre_block_table, pre_q_req, pre_q_pos)
        main.wait_stream(self._side)                 # the decode results are complete on the caller's stream
        return self.decode.out, self.decode.lse, self.prefill.out, self.prefill.lse


class TreeStep:
    """One speculative decode step over drafted trees, with preallocated buffers: layout() once per
    step, attend() once per layer, then verify() and commit().

    n_rows is the largest number of drafted tokens of a step, over all requests; node_off (int32
    [n_req + 1]) and parents (int32 [n_rows]) say which rows are in use, so one captured step serves
    trees of any shape: rows at or past node_off[n_req] are padding.  Every node sees what it would
    see in a sequential decode along its path, block selection included.  Steps that may run at once
    need a TreeStep each."""

    def __init__(self, dims: Dims, n_rows: int, n_req: int, device):
        self.dims, self.n_rows, self.n_req = dims, n_rows, n_req
        f = dict(device=device)
        self.q_req = torch.empty((n_rows,), dtype=torch.int32, **f)
        self.q_pos = torch.empty((n_rows,), dtype=torch.int32, **f)
        self.anc = torch.empty((n_rows,), dtype=torch.int64, **f)
        self.scores = torch.empty((n_rows, dims.G, dims.max_blocks), dtype=torch.float32, **f)
        self.sel = torch.empty((n_rows, dims.G, dims.topk), dtype=torch.int32, **f)
        self.out = torch.zeros((n_rows, dims.Hq, dims.D), dtype=torch.bfloat16, **f)
        self.lse = torch.zeros((n_rows, dims.Hq), dtype=torch.float32, **f)
        self.workspace = torch.empty((max(1, msa_workspace_bytes(MSA_OP_TREE, n_rows, n_req, dims)),),
                                     dtype=torch.uint8, **f)
        self.path = torch.full((n_rows,), -1, dtype=torch.int32, **f)
        self.n_accepted = torch.zeros((n_req,), dtype=torch.int32, **f)
        self.next_token = torch.zeros((n_req,), dtype=torch.int32, **f)
        self.new_lens = torch.zeros((n_req,), dtype=torch.int32, **f)
        self.err = new_err_word(device)
        self.node_off = self.parents = self.ctx_lens = None   # of the step in hand, from layout()

    def layout(self, node_off, parents, ctx_lens):
        """Positions and ancestors of this step's rows, shared by every layer."""
        self.node_off, self.parents, self.ctx_lens = node_off, parents, ctx_lens
        return msa_tree_rows(node_off, parents, ctx_lens, self.dims, self.q_req, self.q_pos, self.anc,
                             err_word=self.err)

    def attend(self, q, q_idx, k_new, v_new, kidx_new, k_cache, v_cache, kidx_cache, block_table, out=None, lse=None):
        """One layer: block scores, top-k, attention -> (out, lse); the step's buffers unless given."""
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        msa_tree_index_score(q_idx, kidx_cache, kidx_new, block_table, self.ctx_lens, self.node_off, self.anc,
                             self.dims, self.scores, err_word=self.err)
        msa_topk_blocks(self.scores, self.q_pos, self.dims, sel=self.sel, err_word=self.err)
        return msa_sparse_attn_tree(q, k_cache, v_cache, k_new, v_new, block_table, self.ctx_lens, self.node_off,
                                    self.anc, self.sel, self.dims, out, lse, self.workspace, err_word=self.err)

    def verify(self, target_probs, draft_probs, tokens, u_accept, u_next):
        """-> (path, n_accepted, next_token) of this step's trees."""
        return msa_verify_tree(target_probs, draft_probs, tokens, self.node_off, self.parents, u_accept, u_next,
                               self.path, self.n_accepted, self.next_token, err_word=self.err)

    def commit(self, k_new, v_new, kidx_new, k_cache, v_cache, kidx_cache, block_table):
        """Append the accepted paths to all layers' caches; -> new context lengths (the next step's
        ctx_lens, after a copy: the buffer is written again by the next commit)."""
        return msa_commit_tree(k_new, v_new, kidx_new, k_cache, v_cache, kidx_cache, block_table, self.ctx_lens,
                               self.node_off, self.path, self.n_accepted, self.dims, self.new_lens,
                               err_word=self.err)
