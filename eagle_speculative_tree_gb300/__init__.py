"""Python binding of libtreespec (tree-attention verify + accept walk on GB300).

Argument marshalling only: every step runs in the CUDA library.  torch tensors
carry device memory and streams; nothing here computes any part of the method.
Importing the package fails if the compiled library is missing -- build it with
`python -m eagle_speculative_tree_gb300.build` (or `__graft_entry__.build()`).
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import re
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtreespec.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "treespec.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libtreespec.so is not built ({LIB_PATH}); run eagle_speculative_tree_gb300/build.py")

_lib = ctypes.CDLL(LIB_PATH)

DTYPE_F32, DTYPE_BF16, DTYPE_E4M3 = 0, 1, 2
KERNEL_AUTO, KERNEL_SIMT, KERNEL_TC, KERNEL_TC_PAIR, KERNEL_TC_2SM, KERNEL_TC_STREAM = 0, 1, 2, 3, 4, 5
ACCEPT_AUTO, ACCEPT_ALL_ROWS, ACCEPT_PATH_ONLY = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ABSENT = -2                     # parent entry of a padding slot after a smaller tree
STATUS_BITS = {1: "BAD_PARENT", 2: "BAD_PAGE", 4: "BAD_LENGTH", 8: "BAD_TOKEN", 16: "TIMEOUT", 32: "INTERNAL",
               64: "BAD_PATH"}


class AttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_nodes", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_pages_per_seq", "num_pool_pages", "dtype", "kernel", "num_splits")]


class AttnPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "kernel", "num_splits", "split_tokens", "rows_per_block", "row_blocks", "merge")]


class ChunkShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_tokens", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_pages_per_seq", "num_pool_pages", "dtype", "kv_dtype", "kernel")]


class AppendOptions(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_norm", "k_norm", "inv_freq", "positions")] + \
        [(n, ctypes.c_float) for n in ("norm_eps", "rope_scale")] + \
        [(n, ctypes.c_int32) for n in ("rot_dim", "layout")]


_vp, _i32p, _f32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_lib.treespec_attn_workspace_bytes.argtypes = [ctypes.POINTER(AttnShape)]
_lib.treespec_attn_workspace_bytes.restype = ctypes.c_size_t
_lib.treespec_attn_plan_for.argtypes = [ctypes.POINTER(AttnShape), ctypes.POINTER(AttnPlan)]
_lib.treespec_attn_plan_for.restype = ctypes.c_int
_lib.tree_attn_verify.argtypes = [_vp] * 7 + [ctypes.POINTER(AttnShape), _vp, ctypes.c_size_t, _vp]
_lib.tree_attn_verify.restype = ctypes.c_int
_lib.treespec_accept_workspace_bytes.argtypes = [ctypes.c_int32] * 3
_lib.treespec_accept_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_accept.argtypes = [_vp] * 5 + [ctypes.c_float] + [_vp] * 3 + [ctypes.c_int32] * 3 + \
    [_vp, ctypes.c_size_t, _vp]
_lib.tree_accept.restype = ctypes.c_int
_lib.tree_accept_with_mode.argtypes = [_vp] * 5 + [ctypes.c_float] + [_vp] * 3 + [ctypes.c_int32] * 4 + \
    [_vp, ctypes.c_size_t, _vp]
_lib.tree_accept_with_mode.restype = ctypes.c_int
_lib.treespec_commit_workspace_bytes.argtypes = []
_lib.treespec_commit_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_kv_commit.argtypes = [_vp] * 7 + [ctypes.POINTER(AttnShape), _vp, ctypes.c_size_t, _vp]
_lib.tree_kv_commit.restype = ctypes.c_int
_lib.treespec_draft_workspace_bytes.argtypes = [ctypes.c_int32] * 3
_lib.treespec_draft_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_draft_step.argtypes = [_vp] + [ctypes.c_int32] * 5 + [_vp] * 4 + [ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp]
_lib.tree_draft_step.restype = ctypes.c_int
_lib.tree_rerank.argtypes = [_vp] * 3 + [ctypes.c_int32] * 3 + [_vp] * 3 + [ctypes.c_size_t, _vp]
_lib.tree_rerank.restype = ctypes.c_int
_lib.tree_rerank_pool.argtypes = [_vp] * 4 + [ctypes.c_int32] * 4 + [_vp] * 3 + [ctypes.c_size_t, _vp]
_lib.tree_rerank_pool.restype = ctypes.c_int
_lib.treespec_append_workspace_bytes.argtypes = []
_lib.treespec_append_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_chunk_append.argtypes = [_vp, ctypes.c_int64] * 3 + [_vp] * 8 + \
    [ctypes.POINTER(ChunkShape), ctypes.POINTER(AppendOptions), _vp, ctypes.c_size_t, _vp]
_lib.tree_chunk_append.restype = ctypes.c_int
_lib.treespec_chunk_attn_workspace_bytes.argtypes = [ctypes.POINTER(ChunkShape)]
_lib.treespec_chunk_attn_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_chunk_attn.argtypes = [_vp] * 9 + [ctypes.POINTER(ChunkShape), _vp, ctypes.c_size_t, _vp]
_lib.tree_chunk_attn.restype = ctypes.c_int
_lib.treespec_attn_e4m3_workspace_bytes.argtypes = [ctypes.POINTER(AttnShape)]
_lib.treespec_attn_e4m3_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_attn_verify_e4m3.argtypes = [_vp] * 9 + [ctypes.POINTER(AttnShape), _vp, ctypes.c_size_t, _vp]
_lib.tree_attn_verify_e4m3.restype = ctypes.c_int
_lib.tree_kv_commit_e4m3.argtypes = [_vp] * 9 + [ctypes.POINTER(AttnShape), _vp, ctypes.c_size_t, _vp]
_lib.tree_kv_commit_e4m3.restype = ctypes.c_int
_lib.treespec_chunk_window_workspace_bytes.argtypes = [ctypes.POINTER(ChunkShape)] + [ctypes.c_int32] * 2
_lib.treespec_chunk_window_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_chunk_attn_window.argtypes = [_vp] * 9 + [ctypes.POINTER(ChunkShape)] + [ctypes.c_int32] * 2 + \
    [_vp, ctypes.c_size_t, _vp]
_lib.tree_chunk_attn_window.restype = ctypes.c_int
_lib.treespec_attn_window_workspace_bytes.argtypes = [ctypes.POINTER(AttnShape)] + [ctypes.c_int32] * 3
_lib.treespec_attn_window_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_attn_verify_window.argtypes = [_vp] * 9 + [ctypes.POINTER(AttnShape)] + [ctypes.c_int32] * 3 + \
    [_vp, ctypes.c_size_t, _vp]
_lib.tree_attn_verify_window.restype = ctypes.c_int
_lib.treespec_chunk_shared_workspace_bytes.argtypes = [ctypes.POINTER(ChunkShape), ctypes.c_int32]
_lib.treespec_chunk_shared_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_chunk_attn_shared.argtypes = [_vp] * 11 + [ctypes.POINTER(ChunkShape), ctypes.c_int32, _vp, ctypes.c_size_t, _vp]
_lib.tree_chunk_attn_shared.restype = ctypes.c_int
_lib.treespec_attn_shared_workspace_bytes.argtypes = [ctypes.POINTER(AttnShape)] + [ctypes.c_int32] * 2
_lib.treespec_attn_shared_workspace_bytes.restype = ctypes.c_size_t
_lib.tree_attn_verify_shared.argtypes = [_vp] * 11 + [ctypes.POINTER(AttnShape)] + [ctypes.c_int32] * 2 + \
    [_vp, ctypes.c_size_t, _vp]
_lib.tree_attn_verify_shared.restype = ctypes.c_int
_lib.treespec_read_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32), _vp]
_lib.treespec_read_status.restype = ctypes.c_int
_lib.treespec_error_string.argtypes = [ctypes.c_int]
_lib.treespec_error_string.restype = ctypes.c_char_p
_lib.treespec_version.restype = ctypes.c_int
_lib.treespec_launch_count.restype = ctypes.c_uint64
_lib.treespec_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
_lib.treespec_set_wait_limit_ns.restype = None
_lib.treespec_last_launch_error.argtypes = [ctypes.POINTER(ctypes.c_char_p)]
_lib.treespec_last_launch_error.restype = ctypes.c_int


class TreespecError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(f"treespec error {code}: {_lib.treespec_error_string(code).decode()}")


def _check(code: int) -> None:
    if code != 0:
        raise TreespecError(code)


def exported_symbols() -> list[str]:
    """Function names declared in include/treespec.h."""
    text = open(HEADER_PATH).read()
    # declarations start in column 0 with a C return type; comment lines never do
    return sorted(set(re.findall(r"^(?:const\s+)?(?:int|size_t|void|uint64_t|uint32_t|char)\s*\*?\s*([a-z_0-9]+)\s*\(",
                                 text, re.M)))


def version() -> int:
    return _lib.treespec_version()


def launch_count() -> int:
    return int(_lib.treespec_launch_count())


def last_launch_error() -> tuple:
    """(cudaError_t code, its name) behind the last launch the CUDA runtime rejected."""
    name = ctypes.c_char_p()
    code = _lib.treespec_last_launch_error(ctypes.byref(name))
    return code, (name.value or b"").decode()


def set_wait_limit_ns(ns: int) -> None:
    """Bound (ns) of the tensor-core kernels' internal waits for later calls; 0 = the default
    2 s.  For tests of the timeout path (see include/treespec.h)."""
    _lib.treespec_set_wait_limit_ns(int(ns))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream: Optional[torch.cuda.Stream], device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _need_rows(t: torch.Tensor, name: str, device) -> None:
    """float32 rows on `device`, or in pinned host memory (read in place by the kernel)."""
    if not ((t.is_cuda and t.device == device) or (t.device.type == "cpu" and t.is_pinned())):
        raise ValueError(f"{name} must be on {device} or in pinned host memory")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be torch.float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, device) -> None:
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@dataclass
class AttnProblem:
    batch: int
    num_nodes: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    page_size: int
    max_pages_per_seq: int
    num_pool_pages: int
    dtype: int
    kernel: int = KERNEL_AUTO
    num_splits: int = 0

    def c_shape(self) -> AttnShape:
        return AttnShape(self.batch, self.num_nodes, self.num_q_heads, self.num_kv_heads, self.head_dim,
                         self.page_size, self.max_pages_per_seq, self.num_pool_pages, self.dtype,
                         self.kernel, self.num_splits)


def attn_problem(q: torch.Tensor, k_pages: torch.Tensor, page_table: torch.Tensor, *,
                 kernel: int = KERNEL_AUTO, num_splits: int = 0) -> AttnProblem:
    B, N, Hq, D = q.shape
    P, ps, Hkv, D2 = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and k_pages differ")
    dt = DTYPE_BF16 if q.dtype == torch.bfloat16 else DTYPE_F32
    return AttnProblem(B, N, Hq, Hkv, D, ps, page_table.shape[1], P, dt, kernel, num_splits)


def attn_workspace_bytes(prob: AttnProblem) -> int:
    n = _lib.treespec_attn_workspace_bytes(ctypes.byref(prob.c_shape()))
    if n == 0:
        raise ValueError(f"unsupported attention shape {prob}")
    return int(n)


def attn_plan(prob: AttnProblem) -> AttnPlan:
    plan = AttnPlan()
    _check(_lib.treespec_attn_plan_for(ctypes.byref(prob.c_shape()), ctypes.byref(plan)))
    return plan


def tree_attn_verify(q, k_pages, v_pages, page_table, prefix_lens, tree_parents, out=None, *,
                     kernel: int = KERNEL_AUTO, num_splits: int = 0,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Tree-attention verification pass; see include/treespec.h for the operation.

    q [B][N][Hq][D], k_pages / v_pages [P][16][Hkv][D] (float32 or bfloat16),
    page_table [B][max_pages] int32, prefix_lens [B] int32, tree_parents [B][N] int32.
    Returns out [B][N][Hq][D] in q's dtype.
    """
    dev = q.device
    dt = q.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("q must be float32 or bfloat16")
    _need(q, "q", dt, dev)
    _need(k_pages, "k_pages", dt, dev)
    _need(v_pages, "v_pages", dt, dev)
    _need(page_table, "page_table", torch.int32, dev)
    _need(prefix_lens, "prefix_lens", torch.int32, dev)
    _need(tree_parents, "tree_parents", torch.int32, dev)
    prob = attn_problem(q, k_pages, page_table, kernel=kernel, num_splits=num_splits)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", dt, dev)
    need = attn_workspace_bytes(prob)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(_lib.tree_attn_verify(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(prefix_lens), _ptr(tree_parents),
        _ptr(out), ctypes.byref(prob.c_shape()), _ptr(workspace), workspace.numel(),
        _stream_handle(stream, dev)))
    return out


def accept_workspace_bytes(batch: int, num_nodes: int, vocab: int) -> int:
    n = _lib.treespec_accept_workspace_bytes(batch, num_nodes, vocab)
    if n == 0:
        raise ValueError("unsupported accept sizes")
    return int(n)


def tree_accept(target_logits, draft_tokens, draft_probs, tree_parents, uniforms, temperature: float, *,
                accept_path=None, accept_len=None, bonus_token=None, mode: int = ACCEPT_AUTO,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Accept walk; see include/treespec.h.  Returns (accept_path, accept_len, bonus_token).

    mode: ACCEPT_AUTO, ACCEPT_ALL_ROWS or ACCEPT_PATH_ONLY (tree_accept_with_mode).
    target_logits and draft_probs may be device tensors or pinned host tensors: the
    kernel reads host rows in place over the CPU-GPU link, and the path-only schedule
    reads only the rows on each sequence's walk."""
    dev = draft_tokens.device
    B, N, V = target_logits.shape
    _need_rows(target_logits, "target_logits", dev)
    _need(draft_tokens, "draft_tokens", torch.int32, dev)
    _need(tree_parents, "tree_parents", torch.int32, dev)
    if temperature > 0:
        _need_rows(draft_probs, "draft_probs", dev)
        _need(uniforms, "uniforms", torch.float32, dev)
    if accept_path is None:
        accept_path = torch.empty((B, N), dtype=torch.int32, device=dev)
    if accept_len is None:
        accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    if bonus_token is None:
        bonus_token = torch.empty((B,), dtype=torch.int32, device=dev)
    need = accept_workspace_bytes(B, N, V)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(_lib.tree_accept_with_mode(
        _ptr(target_logits), _ptr(draft_tokens), _ptr(draft_probs) if temperature > 0 else None,
        _ptr(tree_parents), _ptr(uniforms) if temperature > 0 else None, float(temperature),
        _ptr(accept_path), _ptr(accept_len), _ptr(bonus_token), B, N, V, int(mode),
        _ptr(workspace), workspace.numel(), _stream_handle(stream, dev)))
    return accept_path, accept_len, bonus_token


def commit_workspace_bytes() -> int:
    return int(_lib.treespec_commit_workspace_bytes())


def tree_kv_commit(k_pages, v_pages, page_table, prefix_lens, accept_path, accept_len, new_prefix_lens=None, *,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Move the accepted path's K/V next to each prefix, in place; see include/treespec.h.

    k_pages / v_pages [P][16][Hkv][D] (float32 or bfloat16), page_table [B][max_pages],
    prefix_lens [B], accept_path [B][N], accept_len [B] (int32).  Returns new_prefix_lens
    [B] int32 (prefix + 1 + accept_len, or -1 for a sequence left unchanged)."""
    dev = k_pages.device
    dt = k_pages.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("k_pages must be float32 or bfloat16")
    _need(k_pages, "k_pages", dt, dev)
    _need(v_pages, "v_pages", dt, dev)
    for name, t in (("page_table", page_table), ("prefix_lens", prefix_lens), ("accept_path", accept_path),
                    ("accept_len", accept_len)):
        _need(t, name, torch.int32, dev)
    B, N = accept_path.shape
    P, ps, Hkv, D = k_pages.shape
    shape = AttnShape(B, N, Hkv, Hkv, D, ps, page_table.shape[1], P,
                      DTYPE_BF16 if dt == torch.bfloat16 else DTYPE_F32, KERNEL_AUTO, 0)
    if new_prefix_lens is None:
        new_prefix_lens = torch.empty((B,), dtype=torch.int32, device=dev)
    _need(new_prefix_lens, "new_prefix_lens", torch.int32, dev)
    need = commit_workspace_bytes()
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(_lib.tree_kv_commit(_ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(prefix_lens), _ptr(accept_path),
                               _ptr(accept_len), _ptr(new_prefix_lens), ctypes.byref(shape), _ptr(workspace),
                               workspace.numel(), _stream_handle(stream, dev)))
    return new_prefix_lens


def draft_workspace_bytes(batch: int, frontier: int, topk: int) -> int:
    n = _lib.treespec_draft_workspace_bytes(batch, frontier, topk)
    if n == 0:
        raise ValueError("unsupported draft-step sizes")
    return int(n)


def tree_draft_step(logprobs, step: int, topk: int, frontier_in, node_parent, node_token, node_score,
                    frontier_out=None, *, workspace: Optional[torch.Tensor] = None, stream=None):
    """One beam-expansion step of the draft tree, in place on the node arrays; see
    include/treespec.h.  logprobs [B][F][V] float32 (F = 1 at step 0, else topk);
    frontier_in [B][F] int32 (the previous step's result; None at step 0); node_parent /
    node_token [B][M] int32, node_score [B][M] float32.  Returns (frontier_out [B][topk],
    workspace)."""
    dev = logprobs.device
    _need(logprobs, "logprobs", torch.float32, dev)
    _need(node_parent, "node_parent", torch.int32, dev)
    _need(node_token, "node_token", torch.int32, dev)
    _need(node_score, "node_score", torch.float32, dev)
    if frontier_in is not None:
        _need(frontier_in, "frontier_in", torch.int32, dev)
    B, F, V = logprobs.shape
    M = node_parent.shape[1]
    if frontier_out is None:
        frontier_out = torch.empty((B, topk), dtype=torch.int32, device=dev)
    _need(frontier_out, "frontier_out", torch.int32, dev)
    need = draft_workspace_bytes(B, F, topk)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(_lib.tree_draft_step(_ptr(logprobs), B, F, V, topk, step, _ptr(frontier_in), _ptr(node_parent),
                                _ptr(node_token), _ptr(node_score), M, _ptr(frontier_out), _ptr(workspace),
                                workspace.numel(), _stream_handle(stream, dev)))
    return frontier_out, workspace


def tree_rerank(node_parent, node_token, node_score, num_nodes: int, tree_parents=None, draft_tokens=None, *,
                pool=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Keep the root and the num_nodes - 1 best nodes (of all, or of `pool` [B][P] int32
    node ids: tree_rerank_pool); returns (tree_parents, draft_tokens) [B][num_nodes] int32.
    See include/treespec.h."""
    dev = node_parent.device
    _need(node_parent, "node_parent", torch.int32, dev)
    _need(node_token, "node_token", torch.int32, dev)
    _need(node_score, "node_score", torch.float32, dev)
    B, M = node_parent.shape
    if tree_parents is None:
        tree_parents = torch.empty((B, num_nodes), dtype=torch.int32, device=dev)
    if draft_tokens is None:
        draft_tokens = torch.empty((B, num_nodes), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=dev)
    if pool is None:
        _check(_lib.tree_rerank(_ptr(node_parent), _ptr(node_token), _ptr(node_score), B, M, num_nodes,
                                _ptr(tree_parents), _ptr(draft_tokens), _ptr(workspace), workspace.numel(),
                                _stream_handle(stream, dev)))
    else:
        _need(pool, "pool", torch.int32, dev)
        _check(_lib.tree_rerank_pool(_ptr(node_parent), _ptr(node_token), _ptr(node_score), _ptr(pool),
                                     pool.shape[1], B, M, num_nodes, _ptr(tree_parents), _ptr(draft_tokens),
                                     _ptr(workspace), workspace.numel(), _stream_handle(stream, dev)))
    return tree_parents, draft_tokens


# ------------------------------------------------- chunks of new tokens, 8-bit cache
#
# These calls are as short as a decoding step's launches, so their checks are one pass over
# the tensors' attributes, and the C structs of a problem's sizes are made once per size.

_I32, _F32, _BF16, _E4M3 = torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _need_tensors(**named) -> None:
    for name, t in named.items():
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")


def _need_all(index: int, *wants) -> None:
    """Each want is (tensor, name, dtype, shape): contiguous, on cuda:`index`."""
    try:
        for t, name, dtype, shape in wants:
            if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
                continue
            _need_tensors(**{name: t})
            if not t.is_cuda or t.get_device() != index:
                raise ValueError(f"{name} must be on cuda:{max(index, 0)}")
            if t.dtype is not dtype:
                raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
            raise ValueError(f"{name} must be contiguous")
    except AttributeError:                                     # no cost to the calls that are right
        _need_tensors(**{want[1]: want[0] for want in wants})
        raise


def _float_type_error(q) -> ValueError:
    _need_tensors(q=q)
    return ValueError("q must be float32 or bfloat16")


def _code_type_error(k_pages) -> ValueError:
    _need_tensors(k_pages=k_pages)
    return ValueError(f"k_pages must be {_E4M3}, got {k_pages.dtype}")


def _index_of(q: torch.Tensor, name: str) -> int:
    if not q.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return q.get_device()


def _pool_wants(q_dtype, k_pages, v_pages, k_scales, v_scales) -> tuple:
    """What _need_all has to see of a pair of page pools."""
    if k_pages.dim() != 4:
        raise ValueError("k_pages must have shape [pages][16][kv heads][head_dim]")
    shape = k_pages.shape
    if k_pages.dtype is not _E4M3:
        if k_scales is not None or v_scales is not None:
            raise ValueError("scales belong to float8_e4m3fn pools only")
        return (k_pages, "k_pages", q_dtype, shape), (v_pages, "v_pages", q_dtype, shape)
    if k_scales is None or v_scales is None:
        raise ValueError("k_scales and v_scales are needed with float8_e4m3fn pools")
    scales = (shape[0], shape[2], shape[1])
    return ((k_pages, "k_pages", _E4M3, shape), (v_pages, "v_pages", _E4M3, shape),
            (k_scales, "k_scales", _F32, scales), (v_scales, "v_scales", _F32, scales))


def _fresh(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor that a call makes for itself, out of the memory of the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace_for(workspace, need: int, index: int, device, stream) -> torch.Tensor:
    if workspace is None:
        return _fresh((need,), torch.uint8, device, stream)
    _need_tensors(workspace=workspace)
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{index}")
    return workspace


def _launch(index: int, stream, fn, *args) -> None:
    """The library launches on the current device: make it the tensors' own for the call."""
    handle = stream.cuda_stream if stream is not None else _raw_stream(index)
    if _current_device() == index:
        code = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            code = fn(*args, handle)
    if code != 0:
        raise TreespecError(code)


@dataclass(frozen=True)
class ChunkProblem:
    batch: int
    num_tokens: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    page_size: int
    max_pages_per_seq: int
    num_pool_pages: int
    dtype: int
    kv_dtype: int
    kernel: int = KERNEL_AUTO

    def c_shape(self) -> ChunkShape:
        return ChunkShape(self.batch, self.num_tokens, self.num_q_heads, self.num_kv_heads, self.head_dim,
                          self.page_size, self.max_pages_per_seq, self.num_pool_pages, self.dtype, self.kv_dtype,
                          self.kernel)


@functools.lru_cache(maxsize=1024)
def _chunk_struct(*sizes):
    return ctypes.pointer(ChunkShape(*sizes))


@functools.lru_cache(maxsize=1024)
def _attn_struct(*sizes):
    return ctypes.pointer(AttnShape(*sizes))


def _chunk_sizes(q, k_pages, page_table, chunk_offsets, kernel) -> tuple:
    """The sizes of a call in the order of ChunkProblem's fields."""
    try:
        if q.dim() != 3 or k_pages.dim() != 4 or page_table.dim() != 2 or chunk_offsets.dim() != 1:
            raise ValueError("q is [tokens][heads][head_dim], k_pages [pages][16][kv heads][head_dim], "
                             "page_table [batch][pages], chunk_offsets [batch + 1]")
    except AttributeError:
        _need_tensors(q=q, k_pages=k_pages, page_table=page_table, chunk_offsets=chunk_offsets)
        raise
    T, Hq, D = q.shape
    P, ps, Hkv, D2 = k_pages.shape
    B, pages = page_table.shape
    if D2 != D:
        raise ValueError("head_dim of q and k_pages differ")
    if chunk_offsets.shape[0] != B + 1:
        raise ValueError(f"chunk_offsets must have shape {(B + 1,)}, got {tuple(chunk_offsets.shape)}")
    dt = DTYPE_BF16 if q.dtype is _BF16 else DTYPE_F32
    return B, T, Hq, Hkv, D, ps, pages, P, dt, DTYPE_E4M3 if k_pages.dtype is _E4M3 else dt, kernel


def chunk_problem(q: torch.Tensor, k_pages: torch.Tensor, page_table: torch.Tensor, chunk_offsets: torch.Tensor, *,
                  kernel: int = KERNEL_AUTO) -> ChunkProblem:
    """Sizes of a tree_chunk_attn / tree_chunk_append call: q [T][Hq][D], page_table [B][max_pages]."""
    return ChunkProblem(*_chunk_sizes(q, k_pages, page_table, chunk_offsets, kernel))


def append_workspace_bytes() -> int:
    return int(_lib.treespec_append_workspace_bytes())


def tree_chunk_append(q, k, v, k_pages, v_pages, page_table, prefix_lens, chunk_offsets, q_out=None, *,
                      positions=None, q_norm=None, k_norm=None, norm_eps: float = 1e-6, inv_freq=None,
                      rope: int = ROPE_HALF, rope_scale: float = 1.0, k_scales=None, v_scales=None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Norm, rotary positions and the write of new tokens into the page pools; see
    include/treespec.h for the operation.

    q [T][Hq][D], k / v [T][Hkv][D] (float32 or bfloat16; views whose heads are contiguous,
    such as slices of one projection's output), k_pages / v_pages [P][16][Hkv][D] in the
    same type or float8_e4m3fn with k_scales / v_scales [P][Hkv][16] float32, page_table
    [B][max_pages], prefix_lens [B], chunk_offsets [B + 1], positions [T] (int32),
    q_norm / k_norm [D] and inv_freq [rot_dim / 2] float32 (None: no norm, no rotation).
    Returns q_out [T][Hq][D] (q itself may be given); the pools are written in place.  Rows
    that are left out stay as they are in `q_out` (and hold nothing of use in a new one)."""
    dt = getattr(q, "dtype", None)
    if dt is not _BF16 and dt is not _F32:
        raise _float_type_error(q)
    index = _index_of(q, "q")
    sizes = _chunk_sizes(q, k_pages, page_table, chunk_offsets, KERNEL_AUTO)
    B, T, Hq, Hkv, D = sizes[:5]
    strides = []
    for name, t, H in (("q", q, Hq), ("k", k, Hkv), ("v", v, Hkv)):
        if getattr(t, "dtype", None) is not dt or t.get_device() != index or t.shape != (T, H, D):
            _need_tensors(**{name: t})
            raise ValueError(f"{name} must be {dt} on cuda:{index} with shape {(T, H, D)}")
        to_token, to_head, to_element = t.stride()
        if to_element != 1 or (H > 1 and to_head != D):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        # one token has no distance to the next: its row counts as packed
        strides.append(to_token if T > 1 else H * D)
    wants = [*_pool_wants(dt, k_pages, v_pages, k_scales, v_scales), (page_table, "page_table", _I32, (B, sizes[6])),
             (prefix_lens, "prefix_lens", _I32, (B,)), (chunk_offsets, "chunk_offsets", _I32, (B + 1,))]
    if positions is not None:
        wants.append((positions, "positions", _I32, (T,)))
    if q_norm is not None:
        wants.append((q_norm, "q_norm", _F32, (D,)))
    if k_norm is not None:
        wants.append((k_norm, "k_norm", _F32, (D,)))
    rot = 0
    if inv_freq is not None:
        _need_tensors(inv_freq=inv_freq)
        rot = 2 * inv_freq.numel()
        wants.append((inv_freq, "inv_freq", _F32, (rot // 2,)))
    if q_out is None:
        q_out = _fresh((T, Hq, D), dt, q.device, stream)
    else:
        wants.append((q_out, "q_out", dt, (T, Hq, D)))
    _need_all(index, *wants)
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        workspace = _workspace_for(workspace, append_workspace_bytes(), index, q.device, stream)
    opt = AppendOptions(_ptr(q_norm), _ptr(k_norm), _ptr(inv_freq), _ptr(positions), norm_eps, rope_scale, rot, rope)
    _launch(index, stream, _lib.tree_chunk_append, q.data_ptr(), strides[0], k.data_ptr(), strides[1], v.data_ptr(),
            strides[2], q_out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales),
            page_table.data_ptr(), prefix_lens.data_ptr(), chunk_offsets.data_ptr(), _chunk_struct(*sizes), opt,
            workspace.data_ptr(), workspace.nbytes)
    return q_out


def chunk_attn_workspace_bytes(prob: ChunkProblem) -> int:
    n = _lib.treespec_chunk_attn_workspace_bytes(prob.c_shape())
    if n == 0:
        raise ValueError(f"unsupported chunk attention shape {prob}")
    return int(n)


def _attend_chunks(fn, need, q, k_pages, v_pages, page_table, prefix_lens, chunk_offsets, out, k_scales, v_scales,
                   kernel, workspace, stream, need_args=(), more=(), groups=()) -> torch.Tensor:
    """An attention call over packed chunks: need(problem, *need_args) gives its workspace bytes, `more`
    are the call's whole numbers behind the shape, `groups` (group_offsets, shared_lens)."""
    dt = getattr(q, "dtype", None)
    if dt is not _BF16 and dt is not _F32:
        raise _float_type_error(q)
    index = _index_of(q, "q")
    sizes = _chunk_sizes(q, k_pages, page_table, chunk_offsets, kernel)
    B = sizes[0]
    wants = [(q, "q", dt, q.shape), *_pool_wants(dt, k_pages, v_pages, k_scales, v_scales),
             (page_table, "page_table", _I32, (B, sizes[6])), (prefix_lens, "prefix_lens", _I32, (B,)),
             (chunk_offsets, "chunk_offsets", _I32, (B + 1,))]
    if groups:
        wants += _group_wants(*groups)
    if out is None:
        out = torch.empty_like(q) if stream is None else _fresh(q.shape, dt, q.device, stream)   # q is contiguous
    else:
        wants.append((out, "out", dt, q.shape))
    _need_all(index, *wants)
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        workspace = _workspace_for(workspace, need(ChunkProblem(*sizes), *need_args), index, q.device, stream)
    _launch(index, stream, fn, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales),
            _ptr(v_scales), page_table.data_ptr(), prefix_lens.data_ptr(), chunk_offsets.data_ptr(),
            *[t.data_ptr() for t in groups], out.data_ptr(), _chunk_struct(*sizes), *more, workspace.data_ptr(),
            workspace.nbytes)
    return out


def tree_chunk_attn(q, k_pages, v_pages, page_table, prefix_lens, chunk_offsets, out=None, *, k_scales=None,
                    v_scales=None, kernel: int = KERNEL_AUTO, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Causal attention of packed new tokens over the paged cache that holds them already;
    see include/treespec.h for the operation.

    q [T][Hq][D] (float32 or bfloat16), k_pages / v_pages [P][16][Hkv][D] in the same type
    or float8_e4m3fn with k_scales / v_scales [P][Hkv][16] float32, page_table [B][max_pages],
    prefix_lens [B], chunk_offsets [B + 1] int32.  Returns out [T][Hq][D] in q's dtype; rows
    that belong to no sequence are left as they are in `out` (and hold nothing of use in a
    new one)."""
    return _attend_chunks(_lib.tree_chunk_attn, chunk_attn_workspace_bytes, q, k_pages, v_pages, page_table, prefix_lens,
                          chunk_offsets, out, k_scales, v_scales, kernel, workspace, stream)


def attn_e4m3_workspace_bytes(prob: AttnProblem) -> int:
    n = _lib.treespec_attn_e4m3_workspace_bytes(ctypes.byref(prob.c_shape()))
    if n == 0:
        raise ValueError(f"unsupported attention shape {prob}")
    return int(n)


def _attend_trees(fn, need, q, k_pages, v_pages, k_scales, v_scales, page_table, prefix_lens, tree_parents, out, kernel,
                  workspace, stream, need_args=(), more=(), groups=()) -> torch.Tensor:
    """A verification call over any pools; arguments as for _attend_chunks."""
    dt = getattr(q, "dtype", None)
    if dt is not _BF16 and dt is not _F32:
        raise _float_type_error(q)
    index = _index_of(q, "q")
    if not isinstance(k_pages, torch.Tensor) or not isinstance(page_table, torch.Tensor) or q.dim() != 4 or \
            page_table.dim() != 2:
        _need_tensors(k_pages=k_pages, page_table=page_table)
        raise ValueError("q is [batch][nodes][heads][head_dim], page_table [batch][pages]")
    B, N, Hq, D = q.shape
    wants = [(q, "q", dt, q.shape), *_pool_wants(dt, k_pages, v_pages, k_scales, v_scales),
             (page_table, "page_table", _I32, (B, page_table.shape[1])), (prefix_lens, "prefix_lens", _I32, (B,)),
             (tree_parents, "tree_parents", _I32, (B, N))]
    if groups:
        wants += _group_wants(*groups)
    if out is None:
        out = torch.empty_like(q) if stream is None else _fresh(q.shape, dt, q.device, stream)   # q is contiguous
    else:
        wants.append((out, "out", dt, q.shape))
    _need_all(index, *wants)
    P, ps, Hkv, D2 = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and k_pages differ")
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        workspace = _workspace_for(workspace, need(attn_problem(q, k_pages, page_table, kernel=kernel), *need_args), index, q.device,
                                   stream)
    _launch(index, stream, fn, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales),
            page_table.data_ptr(), prefix_lens.data_ptr(), tree_parents.data_ptr(), *[t.data_ptr() for t in groups],
            out.data_ptr(), _attn_struct(B, N, Hq, Hkv, D, ps, page_table.shape[1], P,
                                         DTYPE_BF16 if dt is _BF16 else DTYPE_F32, kernel, 0),
            *more, workspace.data_ptr(), workspace.nbytes)
    return out


def tree_attn_verify_e4m3(q, k_pages, v_pages, k_scales, v_scales, page_table, prefix_lens, tree_parents, out=None, *,
                          kernel: int = KERNEL_AUTO, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Tree-attention verification over float8_e4m3fn pools; see include/treespec.h.

    q [B][N][Hq][D] (float32 or bfloat16), k_pages / v_pages [P][16][Hkv][D] float8_e4m3fn,
    k_scales / v_scales [P][Hkv][16] float32, page_table [B][max_pages], prefix_lens [B],
    tree_parents [B][N] int32.  Returns out [B][N][Hq][D] in q's dtype."""
    dt = getattr(q, "dtype", None)
    if dt is not _BF16 and dt is not _F32:
        raise _float_type_error(q)
    _index_of(q, "q")
    if getattr(k_pages, "dtype", None) is not _E4M3:
        raise _code_type_error(k_pages)
    return _attend_trees(_lib.tree_attn_verify_e4m3, attn_e4m3_workspace_bytes, q, k_pages, v_pages, k_scales, v_scales,
                         page_table, prefix_lens, tree_parents, out, kernel, workspace, stream)


def tree_kv_commit_e4m3(k_pages, v_pages, k_scales, v_scales, page_table, prefix_lens, accept_path, accept_len,
                        new_prefix_lens=None, *, workspace: Optional[torch.Tensor] = None, stream=None):
    """Move the accepted path's codes and scales next to each prefix, in place; see
    include/treespec.h.  Pools and scales as for tree_attn_verify_e4m3, the rest as for
    tree_kv_commit.  Returns new_prefix_lens [B] int32."""
    if getattr(k_pages, "dtype", None) is not _E4M3:
        raise _code_type_error(k_pages)
    index = _index_of(k_pages, "k_pages")
    if not isinstance(accept_path, torch.Tensor) or not isinstance(page_table, torch.Tensor) or \
            accept_path.dim() != 2 or page_table.dim() != 2:
        _need_tensors(accept_path=accept_path, page_table=page_table)
        raise ValueError("accept_path is [batch][nodes], page_table [batch][pages]")
    B, N = accept_path.shape
    wants = [*_pool_wants(None, k_pages, v_pages, k_scales, v_scales),
             (page_table, "page_table", _I32, (B, page_table.shape[1])), (prefix_lens, "prefix_lens", _I32, (B,)),
             (accept_path, "accept_path", _I32, (B, N)), (accept_len, "accept_len", _I32, (B,))]
    if new_prefix_lens is None:
        new_prefix_lens = _fresh((B,), _I32, k_pages.device, stream)
    else:
        wants.append((new_prefix_lens, "new_prefix_lens", _I32, (B,)))
    _need_all(index, *wants)
    P, ps, Hkv, D = k_pages.shape
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        workspace = _workspace_for(workspace, commit_workspace_bytes(), index, k_pages.device, stream)
    _launch(index, stream, _lib.tree_kv_commit_e4m3, k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
            v_scales.data_ptr(), page_table.data_ptr(), prefix_lens.data_ptr(), accept_path.data_ptr(),
            accept_len.data_ptr(), new_prefix_lens.data_ptr(),
            _attn_struct(B, N, Hkv, Hkv, D, ps, page_table.shape[1], P, DTYPE_BF16, KERNEL_AUTO, 0),
            workspace.data_ptr(), workspace.nbytes)
    return new_prefix_lens


# --------------------------------------------- sliding windows and shared prefixes

def _groups_of(group_offsets, shared_lens) -> int:
    _need_tensors(group_offsets=group_offsets, shared_lens=shared_lens)
    if shared_lens.dim() != 1 or shared_lens.numel() < 1:
        raise ValueError("shared_lens must have shape [groups], with one group at least")
    return shared_lens.numel()


def _group_wants(group_offsets, shared_lens) -> tuple:
    n = shared_lens.numel()
    return (group_offsets, "group_offsets", _I32, (n + 1,)), (shared_lens, "shared_lens", _I32, (n,))


def _window_of(window, sinks) -> tuple:
    """window >= 1 and sinks >= 0 as the C calls take them: 2^30 reaches every token."""
    window, sinks = operator.index(window), operator.index(sinks)
    if window < 1:
        raise ValueError(f"window must be at least 1, got {window}")
    if sinks < 0:
        raise ValueError(f"sinks must not be negative, got {sinks}")
    return min(window, 1 << 30), min(sinks, 1 << 30)


def _kv_dtype(q, k_pages) -> int:
    return DTYPE_E4M3 if getattr(k_pages, "dtype", None) is _E4M3 else DTYPE_BF16 if getattr(q, "dtype", None) is _BF16 \
        else DTYPE_F32


def _bytes_or_error(n: int, prob, *more) -> int:
    if n == 0:
        raise ValueError(f"unsupported attention shape {prob} {more}")
    return int(n)


def chunk_window_workspace_bytes(prob: ChunkProblem, window: int, sinks: int = 0) -> int:
    w = _window_of(window, sinks)
    return _bytes_or_error(_lib.treespec_chunk_window_workspace_bytes(prob.c_shape(), *w), prob, *w)


def attn_window_workspace_bytes(prob: AttnProblem, kv_dtype: int, window: int, sinks: int = 0) -> int:
    w = _window_of(window, sinks)
    return _bytes_or_error(_lib.treespec_attn_window_workspace_bytes(prob.c_shape(), kv_dtype, *w), prob, kv_dtype, *w)


def chunk_shared_workspace_bytes(prob: ChunkProblem, num_groups: int) -> int:
    return _bytes_or_error(_lib.treespec_chunk_shared_workspace_bytes(prob.c_shape(), num_groups), prob, num_groups)


def attn_shared_workspace_bytes(prob: AttnProblem, kv_dtype: int, num_groups: int) -> int:
    return _bytes_or_error(_lib.treespec_attn_shared_workspace_bytes(prob.c_shape(), kv_dtype, num_groups), prob, kv_dtype,
                           num_groups)


def tree_chunk_attn_window(q, k_pages, v_pages, page_table, prefix_lens, chunk_offsets, window: int, sinks: int = 0,
                           out=None, *, k_scales=None, v_scales=None, kernel: int = KERNEL_AUTO,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tree_chunk_attn where a row sees itself, the window - 1 tokens before it and the sequence's
    first `sinks` tokens; see include/treespec.h.  Pages that no row sees are not read, and their
    entries in page_table may hold anything."""
    w = _window_of(window, sinks)
    return _attend_chunks(_lib.tree_chunk_attn_window, chunk_window_workspace_bytes, q, k_pages, v_pages, page_table,
                          prefix_lens, chunk_offsets, out, k_scales, v_scales, kernel, workspace, stream, w, w)


def tree_attn_verify_window(q, k_pages, v_pages, page_table, prefix_lens, tree_parents, window: int, sinks: int = 0,
                            out=None, *, k_scales=None, v_scales=None, kernel: int = KERNEL_AUTO,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Tree verification where a node sees, of its prefix and its ancestors, those fewer than
    `window` positions before it and those at the first `sinks` positions; a node's position is
    the prefix length plus its depth.  See include/treespec.h.

    q [B][N][Hq][D], k_pages / v_pages in the same type or float8_e4m3fn with k_scales /
    v_scales, the rest as for tree_attn_verify."""
    w = _window_of(window, sinks)
    more = (_kv_dtype(q, k_pages), *w)
    return _attend_trees(_lib.tree_attn_verify_window, attn_window_workspace_bytes, q, k_pages, v_pages, k_scales, v_scales,
                         page_table, prefix_lens, tree_parents, out, kernel, workspace, stream, more, more)


def tree_chunk_attn_shared(q, k_pages, v_pages, page_table, prefix_lens, chunk_offsets, group_offsets, shared_lens,
                           out=None, *, k_scales=None, v_scales=None, kernel: int = KERNEL_AUTO,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tree_chunk_attn of a batch whose sequences share prefixes, each read and multiplied once: the
    sequences group_offsets[g] .. group_offsets[g + 1] - 1 have their first shared_lens[g] tokens
    in common.  group_offsets [groups + 1] and shared_lens [groups] int32 on the device; see
    include/treespec.h."""
    n = _groups_of(group_offsets, shared_lens)
    return _attend_chunks(_lib.tree_chunk_attn_shared, chunk_shared_workspace_bytes, q, k_pages, v_pages, page_table,
                          prefix_lens, chunk_offsets, out, k_scales, v_scales, kernel, workspace, stream, (n,), (n,),
                          (group_offsets, shared_lens))


def tree_attn_verify_shared(q, k_pages, v_pages, page_table, prefix_lens, tree_parents, group_offsets, shared_lens,
                            out=None, *, k_scales=None, v_scales=None, kernel: int = KERNEL_AUTO,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Tree verification of a batch whose sequences share prefixes; groups as for
    tree_chunk_attn_shared, pools as for tree_attn_verify_window.  See include/treespec.h."""
    more = (_kv_dtype(q, k_pages), _groups_of(group_offsets, shared_lens))
    return _attend_trees(_lib.tree_attn_verify_shared, attn_shared_workspace_bytes, q, k_pages, v_pages, k_scales, v_scales,
                         page_table, prefix_lens, tree_parents, out, kernel, workspace, stream, more, more,
                         (group_offsets, shared_lens))


def read_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and return the device status word of the last call that used `workspace`."""
    st = ctypes.c_uint32(0)
    _check(_lib.treespec_read_status(_ptr(workspace), ctypes.byref(st),
                                     _stream_handle(stream, workspace.device)))
    return int(st.value)


def raw_library() -> ctypes.CDLL:
    """The loaded C library (for callers that pass raw pointers)."""
    return _lib
