"""Python binding of libtlsp (include/tlsp.h): argument marshalling only.

Every step of the path runs in the CUDA library; this module only turns
torch tensors into device pointers, allocates outputs and the workspace with
PyTorch, and passes the current CUDA stream. It fails loudly when the library
is missing: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import operator
import os
import struct
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtlsp.so")

TLSP_OK = 0
TLSP_ERR_INVALID_ARG = -1
TLSP_ERR_UNSUPPORTED = -2
TLSP_ERR_WORKSPACE = -3
TLSP_ERR_CUDA = -4
TLSP_ERR_TIMEOUT = -5
TLSP_ERR_DEVICE_ASSERT = -6

TLSP_F32 = 0
TLSP_BF16 = 1

EXPORTED = [
    "tlsp_num_groups", "tlsp_num_levels", "tlsp_workspace_bytes", "tlsp_group_queries",
    "tlsp_group_queries_trace", "tlsp_split_from_projections", "tlsp_anchor_attention",
    "tlsp_reuse_attention", "tlsp_dense_attention", "tlsp_dense_attention_noalloc",
    "tlsp_topk_from_scores", "tlsp_get_device_status",
    "tlsp_reset_device_status", "tlsp_debug_bounded_wait", "tlsp_status_string",
    "tlsp_last_cuda_error", "tlsp_launch_count", "tlsp_group_raster",
    "tlsp_block_topk_from_scores", "tlsp_pooled_block_select",
    "tlsp_rotary_make_plan", "tlsp_rotary", "tlsp_packed_make_plan", "tlsp_packed_attention",
    "tlsp_prefix_attention",
]


class TlspError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("n_q", ctypes.c_int32),
                ("n_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int), ("axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * 4), ("scaling", ctypes.c_int),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("fast", ctypes.c_double),
                ("slow", ctypes.c_double), ("amplitude", ctypes.c_double)]


class RotaryPlanData(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("axis", ctypes.c_uint8 * 128), ("turns", ctypes.c_uint64 * 128)]


class PackedDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("causal", ctypes.c_int32),
                ("prefix_len", ctypes.c_int32)]


class PackedPlanData(ctypes.Structure):
    _fields_ = [("desc", PackedDesc), ("tile_items", ctypes.c_int32),
                ("token_items", ctypes.c_int32), ("token_segments", ctypes.c_int32),
                ("merge_items", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("merge_parts", ctypes.c_int32), ("q_rows", ctypes.c_int64),
                ("kv_rows", ctypes.c_int64), ("part_rows", ctypes.c_int64),
                ("items_bytes", ctypes.c_uint64), ("ws_bytes", ctypes.c_uint64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads the in-tree libtlsp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m token_level_sparse_pddp_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        dp = ctypes.POINTER(Dims)
        sig = {
            "tlsp_num_groups": (i32, [i32, i32]),
            "tlsp_num_levels": (i32, [i32, i32]),
            "tlsp_workspace_bytes": (sz, [dp, i32, i32]),
            "tlsp_group_queries": (ctypes.c_int, [dp, vp, i32, vp, vp, sz, vp]),
            "tlsp_group_queries_trace": (ctypes.c_int, [dp, vp, i32, vp, vp, vp, sz, vp]),
            "tlsp_split_from_projections": (ctypes.c_int, [vp, vp, i32, i32, vp, vp, vp, sz, vp]),
            "tlsp_anchor_attention": (ctypes.c_int,
                                      [dp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "tlsp_reuse_attention": (ctypes.c_int,
                                     [dp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, sz, vp]),
            "tlsp_dense_attention": (ctypes.c_int, [dp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "tlsp_dense_attention_noalloc": (ctypes.c_int, [dp, vp, vp, vp, vp, vp]),
            "tlsp_topk_from_scores": (ctypes.c_int, [vp, i32, i32, i32, vp, vp, sz, vp]),
            "tlsp_get_device_status": (ctypes.c_int, [vp]),
            "tlsp_reset_device_status": (ctypes.c_int, [vp, vp]),
            "tlsp_debug_bounded_wait": (ctypes.c_int, [vp, sz, i64, vp]),
            "tlsp_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "tlsp_last_cuda_error": (ctypes.c_int, []),
            "tlsp_launch_count": (i64, []),
            "tlsp_group_raster": (ctypes.c_int, [dp, i32, vp, vp]),
            "tlsp_block_topk_from_scores": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, vp]),
            "tlsp_pooled_block_select": (ctypes.c_int,
                                         [dp, vp, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]),
            "tlsp_rotary_make_plan": (ctypes.c_int, [vp, vp]),
            "tlsp_rotary": (ctypes.c_int, [vp, vp, vp, vp, i32, vp]),
            "tlsp_packed_make_plan": (ctypes.c_int, [vp, vp, vp, vp, vp, sz, vp]),
            "tlsp_packed_attention": (ctypes.c_int,
                                      [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, sz, vp]),
            "tlsp_prefix_attention": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                     ctypes.c_float, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().tlsp_status_string(code).decode()


def _check(code: int, what: str):
    if code != TLSP_OK:
        if code == TLSP_ERR_CUDA:
            what += f" (cudaError {lib().tlsp_last_cuda_error()})"
        raise TlspError(code, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return TLSP_F32
    if dt == torch.bfloat16:
        return TLSP_BF16
    raise ValueError(f"unsupported dtype {dt}")


def _fits(value, what: str, bits: int = 32) -> int:
    """A whole number that the library's type holds (ctypes would keep its low bits only)."""
    n = operator.index(value)
    if not -(1 << bits - 1) <= n < 1 << bits - 1:
        raise ValueError(f"{what} is out of range: {n}")
    return n


def dims_of(Q: torch.Tensor, K: Optional[torch.Tensor] = None) -> Dims:
    B, H, n_q, d = Q.shape
    n_kv = K.shape[2] if K is not None else n_q
    return Dims(B, H, n_q, n_kv, d, _dtype_code(Q.dtype))


def num_groups(n_q: int, group_size: int) -> int:
    return lib().tlsp_num_groups(n_q, group_size)


def num_levels(n_q: int, group_size: int) -> int:
    return lib().tlsp_num_levels(n_q, group_size)


def launch_count() -> int:
    return lib().tlsp_launch_count()


class Workspace:
    """Caller-owned scratch for the library calls (a zeroed torch byte tensor)."""

    def __init__(self, dims: Optional[Dims], group_size: int = 1, k: int = 1, device=None,
                 nbytes: Optional[int] = None):
        n = nbytes if nbytes is not None else lib().tlsp_workspace_bytes(
            ctypes.byref(dims), group_size, k)
        if n == 0:
            raise TlspError(TLSP_ERR_INVALID_ARG, "tlsp_workspace_bytes")
        self.nbytes = n
        self.buf = torch.zeros(n, dtype=torch.uint8, device=device or "cuda")
        self.made_on = torch.cuda.current_stream(self.buf.device).cuda_stream

    @classmethod
    def status_only(cls, device=None) -> "Workspace":
        """The 256-byte workspace that the reuse step needs (its status word only)."""
        return cls(None, nbytes=256, device=device)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    def status(self) -> int:
        return lib().tlsp_get_device_status(self.ptr)

    def reset(self):
        _check(lib().tlsp_reset_device_status(self.ptr, _stream()), "tlsp_reset_device_status")


def group_queries(Q: torch.Tensor, group_size: int, ws: Workspace, trace: bool = False,
                  out: Optional[torch.Tensor] = None):
    """PDDP grouping -> groups int32 [B, H, G*group_size] (and per-level projections)."""
    d = dims_of(Q)
    G = num_groups(d.n_q, group_size)
    groups = (torch.empty((d.batch, d.heads, G * group_size), dtype=torch.int32, device=Q.device)
              if out is None else out)
    if trace:
        L = num_levels(d.n_q, group_size)
        proj = torch.empty((max(L, 0), d.batch, d.heads, d.n_q), dtype=torch.float32,
                           device=Q.device)
        _check(lib().tlsp_group_queries_trace(ctypes.byref(d), _ptr(Q), group_size, _ptr(groups),
                                              _ptr(proj) if L > 0 else ctypes.c_void_p(
                                                  groups.data_ptr()),
                                              ws.ptr, ws.nbytes, _stream()),
               "tlsp_group_queries_trace")
        return groups, proj
    _check(lib().tlsp_group_queries(ctypes.byref(d), _ptr(Q), group_size, _ptr(groups), ws.ptr,
                                    ws.nbytes, _stream()), "tlsp_group_queries")
    return groups


def anchor_attention(Q, K, V, groups, group_size: int, k: int, ws: Workspace,
                     return_scores: bool = False, out=None):
    """Anchor step -> (O_full, indices, R[, scores])."""
    d = dims_of(Q, K)
    G = num_groups(d.n_q, group_size)
    if out is None:
        O = torch.empty_like(Q)
        idx = torch.empty((d.batch, d.heads, G, k), dtype=torch.int32, device=Q.device)
        R = torch.empty(Q.shape, dtype=torch.float32, device=Q.device)
    else:
        O, idx, R = out
    S = (torch.empty((d.batch, d.heads, G, d.n_kv), dtype=torch.float32, device=Q.device)
         if return_scores else None)
    _check(lib().tlsp_anchor_attention(ctypes.byref(d), _ptr(Q), _ptr(K), _ptr(V), _ptr(groups),
                                       group_size, k, _ptr(O), _ptr(idx), _ptr(R), _ptr(S),
                                       ws.ptr, ws.nbytes, _stream()), "tlsp_anchor_attention")
    return (O, idx, R, S) if return_scores else (O, idx, R)


def reuse_attention(Q, K, V, groups, group_size: int, k: int, indices, R, ws: Workspace,
                    out: Optional[torch.Tensor] = None):
    """Reuse step -> O = sparse attention over the anchor's selection + R."""
    d = dims_of(Q, K)
    O = torch.empty_like(Q) if out is None else out
    _check(lib().tlsp_reuse_attention(ctypes.byref(d), _ptr(Q), _ptr(K), _ptr(V), _ptr(groups),
                                      group_size, k, _ptr(indices), _ptr(R), _ptr(O), ws.ptr,
                                      ws.nbytes, _stream()), "tlsp_reuse_attention")
    return O


def dense_attention(Q, K, V, ws: Workspace, out=None, lse=None):
    """Dense attention alone -> O (and fills lse [B, H, n_q] if given)."""
    d = dims_of(Q, K)
    O = torch.empty_like(Q) if out is None else out
    _check(lib().tlsp_dense_attention(ctypes.byref(d), _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                      _ptr(lse), ws.ptr, ws.nbytes, _stream()),
           "tlsp_dense_attention")
    return O


def dense_attention_noalloc(Q, K, V, out=None):
    """Dense attention through the entry point that allocates nothing (fixed library scratch)."""
    d = dims_of(Q, K)
    O = torch.empty_like(Q) if out is None else out
    _check(lib().tlsp_dense_attention_noalloc(ctypes.byref(d), _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                              _stream()), "tlsp_dense_attention_noalloc")
    return O


def topk_from_scores(scores: torch.Tensor, k: int, ws: Optional[Workspace] = None) -> torch.Tensor:
    """Per row of fp32 scores [..., n_kv]: ascending indices of the k largest (ties: lower index).

    With a workspace, a timed-out wait inside the kernel is recorded in its status word."""
    n_kv = scores.shape[-1]
    rows = scores.numel() // n_kv
    idx = torch.empty(scores.shape[:-1] + (k,), dtype=torch.int32, device=scores.device)
    wsp, wsn = (ws.ptr, ws.nbytes) if ws is not None else (None, 0)
    _check(lib().tlsp_topk_from_scores(_ptr(scores), rows, n_kv, k, _ptr(idx), wsp, wsn,
                                       _stream()),
           "tlsp_topk_from_scores")
    return idx


def split_from_projections(proj: torch.Tensor, members: torch.Tensor,
                           n_left: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """One PDDP cut of ascending `members` on proj[token] -> (left, right)."""
    n = members.numel()
    left = torch.empty(max(n_left, 1), dtype=torch.int32, device=members.device)
    right = torch.empty(max(n - n_left, 1), dtype=torch.int32, device=members.device)
    _check(lib().tlsp_split_from_projections(_ptr(proj), _ptr(members), n, n_left, _ptr(left),
                                             _ptr(right), None, 0, _stream()),
           "tlsp_split_from_projections")
    return left[:n_left], right[:n - n_left]


def debug_bounded_wait(ws: Workspace, spin_limit: int):
    _check(lib().tlsp_debug_bounded_wait(ws.ptr, ws.nbytes, spin_limit, _stream()),
           "tlsp_debug_bounded_wait")


# ----------------------------------------------------------------- ablation

def group_raster(Q: torch.Tensor, group_size: int, out: Optional[torch.Tensor] = None):
    """Raster query groups (consecutive tokens, no PDDP) -> int32 [B, H, G*group_size]."""
    d = dims_of(Q)
    G = num_groups(d.n_q, group_size)
    groups = (torch.empty((d.batch, d.heads, G * group_size), dtype=torch.int32, device=Q.device)
              if out is None else out)
    _check(lib().tlsp_group_raster(ctypes.byref(d), group_size, _ptr(groups), _stream()),
           "tlsp_group_raster")
    return groups


def block_topk_from_scores(scores: torch.Tensor, k: int, block: int,
                           return_block_scores: bool = False):
    """Block-granular selection from per-key scores [..., n_kv] -> indices [..., k]
    (and the block scores [..., n_kv / block] when asked)."""
    n_kv = scores.shape[-1]
    rows = scores.numel() // n_kv
    idx = torch.empty(scores.shape[:-1] + (k,), dtype=torch.int32, device=scores.device)
    bs = (torch.empty(scores.shape[:-1] + (n_kv // block,), dtype=torch.float32,
                      device=scores.device) if return_block_scores else None)
    _check(lib().tlsp_block_topk_from_scores(_ptr(scores), rows, n_kv, k, block, _ptr(idx),
                                             _ptr(bs), _stream()),
           "tlsp_block_topk_from_scores")
    return (idx, bs) if return_block_scores else idx


def pooled_block_select(Q: torch.Tensor, K: torch.Tensor, groups: torch.Tensor, group_size: int,
                        k: int, block: int, ws: Workspace, return_block_scores: bool = False):
    """Block-sparse baseline selection (mean-pooled block scores) -> indices [B, H, G, k]."""
    d = dims_of(Q, K)
    G = num_groups(d.n_q, group_size)
    idx = torch.empty((d.batch, d.heads, G, k), dtype=torch.int32, device=Q.device)
    bs = (torch.empty((d.batch, d.heads, G, d.n_kv // block), dtype=torch.float32,
                      device=Q.device) if return_block_scores else None)
    _check(lib().tlsp_pooled_block_select(ctypes.byref(d), _ptr(Q), _ptr(K), _ptr(groups),
                                          group_size, k, block, _ptr(idx), _ptr(bs), ws.ptr,
                                          ws.nbytes, _stream()),
           "tlsp_pooled_block_select")
    return (idx, bs) if return_block_scores else idx


# ----------------------------------------------------------------- rotary positions

_ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
_ROTARY_SCALINGS = {None: 0, "none": 0, "linear": 1, "base": 2, "ramp": 3}


class RotaryPlan:
    """Frequencies of a rotary embedding, made once and passed to every call (host memory only).

    head_dim     channels of a head (a multiple of 8, at most 256)
    rotary_dim   leading channels that are turned (default: all)
    layout       "half": channel i pairs with i + rotary_dim / 2; "interleaved": 2i with 2i + 1
    base         pair i of a section of s pairs turns by base^(-i / s) per position
    scaling      None, "linear" (frequencies / factor), "base" (base * factor^(D / (D - 2))),
                 "ramp" (pairs that turn fewer than `slow` times over original_len positions are
                 divided by factor, those that turn more than `fast` times are kept, linear in
                 between; amplitude 1 + 0.1 ln(factor) unless given)
    sections     pairs of each position axis, e.g. (22, 21, 21) for (frame, row, column);
                 default: one axis
    """

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, base: float = 10000.0,
                 layout: str = "half", scaling: Optional[str] = None, factor: float = 1.0,
                 original_len: float = 0.0, fast: float = 32.0, slow: float = 1.0,
                 amplitude: Optional[float] = None, sections=None):
        if layout not in _ROTARY_LAYOUTS:
            raise ValueError(f"layout must be one of {list(_ROTARY_LAYOUTS)}")
        if scaling not in _ROTARY_SCALINGS:
            raise ValueError(f"scaling must be one of {list(_ROTARY_SCALINGS)}")
        if amplitude is not None and not amplitude > 0:
            raise ValueError("amplitude must be positive")
        head_dim = _fits(head_dim, "head_dim")
        r = head_dim if rotary_dim is None else _fits(rotary_dim, "rotary_dim")
        sec = [r // 2] if sections is None else [_fits(x, "a section") for x in sections]
        if not 1 <= len(sec) <= 4:
            raise ValueError("1 to 4 sections")
        desc = RotaryDesc(head_dim, r, _ROTARY_LAYOUTS[layout], len(sec),
                          (ctypes.c_int32 * 4)(*sec), _ROTARY_SCALINGS[scaling], base, factor,
                          original_len, fast, slow, 0.0 if amplitude is None else amplitude)
        self.data = RotaryPlanData()
        _check(lib().tlsp_rotary_make_plan(ctypes.byref(desc), ctypes.byref(self.data)),
               "tlsp_rotary_make_plan")
        self._at = ctypes.addressof(self.data)
        self.head_dim, self.rotary_dim, self.axes = head_dim, r, len(sec)


# C structs that are filled anew for every call, as bytes: tlsp_rotary_tensor, tlsp_rotary_call,
# tlsp_rows (a call's host time is mostly the marshalling of its arguments)
_ROTARY_TENSOR = struct.Struct("PPqqqqqqi4x")
_ROTARY_CALL = struct.Struct("iiiiPqq")
_ROWS = struct.Struct("Pqq")
_DTYPE_CODES = {torch.float32: TLSP_F32, torch.bfloat16: TLSP_BF16}


def _launch(device: int, fn, *args):
    """fn(*args, stream) on `device`'s current stream (`device` need not be the current one)."""
    stream = torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        return fn(*args, stream)
    with torch.cuda.device(device):
        return fn(*args, stream)


def _like(x: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype,
                                                                     device=x.device)


def _rotary_tensor(x: torch.Tensor, out: torch.Tensor, rank: int, heads: int) -> bytes:
    st, so = x.stride(), out.stride()
    if st[-1] != 1 or so[-1] != 1:
        raise ValueError("channels must be contiguous")
    if rank == 3:
        return _ROTARY_TENSOR.pack(x.data_ptr(), out.data_ptr(), 0, st[0], st[1], 0, so[0], so[1],
                                   heads)
    return _ROTARY_TENSOR.pack(x.data_ptr(), out.data_ptr(), st[0], st[2], st[1], so[0], so[2],
                               so[1], heads)


def _rotary_out(x: torch.Tensor, o: torch.Tensor, dev: int):
    if o.shape != x.shape or o.dtype != x.dtype or o.get_device() != dev:
        raise ValueError("out must match the input's shape, type and device")
    if 0 in o.stride() and any(s == 0 and n > 1 for s, n in zip(o.stride(), o.shape)):
        raise ValueError("out must not be a broadcast tensor")


def _rotary(Q, K, positions, plan: RotaryPlan, out, backward: int):
    shape = Q.shape
    rank = len(shape)
    if rank == 3:
        batch, (tokens, heads, d) = 1, shape
    elif rank == 4:
        batch, heads, tokens, d = shape
    else:
        raise ValueError("tensors are [tokens, heads, head_dim] or [batch, heads, tokens, head_dim]")
    dev, dtype = Q.get_device(), Q.dtype
    if dev < 0:
        raise ValueError("tensors must live on the CUDA device")
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    if d != plan.head_dim or heads < 1:
        raise ValueError(f"expected heads of {plan.head_dim} channels, got {tuple(shape)}")
    if K is not None:
        if K.dtype != dtype or K.get_device() != dev or K.dim() != rank:
            raise ValueError("queries and keys must have the same rank, type and device")
        k_heads = K.shape[1]
        if K.shape != ((tokens, k_heads, d) if rank == 3 else (batch, k_heads, tokens, d)) or \
                k_heads < 1:
            raise ValueError(f"queries and keys must have the same tokens and channels, got "
                             f"{tuple(shape)} and {tuple(K.shape)}")
    p_type, p_shape, p_stride = positions.dtype, positions.shape, positions.stride()
    if (p_type != torch.int32 and p_type != torch.int64) or positions.get_device() != dev:
        raise ValueError("positions must be int32 or int64 on the tensors' device")
    lead = () if plan.axes == 1 else (plan.axes,)
    if p_shape == lead + (tokens,):
        p_batch = 0
    elif rank == 4 and p_shape == lead + (batch, tokens):
        p_batch = p_stride[-2]
    else:
        raise ValueError(f"positions must be {lead + (tokens,)} (or with the batch before the "
                         f"tokens), got {tuple(p_shape)}")
    if tokens > 1 and p_stride[-1] != 1:
        raise ValueError("positions must be contiguous along the tokens")
    if out is None:
        q_out, k_out = _like(Q), None if K is None else _like(K)
    elif K is None:
        q_out, k_out = out, None
        _rotary_out(Q, q_out, dev)
    else:
        if len(out) != 2:
            raise ValueError("out must be one tensor per input")
        q_out, k_out = out
        _rotary_out(Q, q_out, dev)
        _rotary_out(K, k_out, dev)
    rc = _launch(dev, lib().tlsp_rotary, plan._at,
                 _ROTARY_CALL.pack(batch, tokens, code, p_type == torch.int64,
                                   positions.data_ptr(), p_stride[0] if lead else 0, p_batch),
                 _rotary_tensor(Q, q_out, rank, heads),
                 None if K is None else _rotary_tensor(K, k_out, rank, k_heads), backward)
    _check(rc, "tlsp_rotary")
    return q_out if K is None else (q_out, k_out)


class _RotaryGrad(torch.autograd.Function):
    """_rotary with its gradient, which is the transposed map (and whose own is the map again)."""

    @staticmethod
    def forward(ctx, Q, K, positions, plan, backward):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.plan, ctx.turned = plan, backward
        return _rotary(Q, K, positions, plan, None, backward)

    @staticmethod
    def backward(ctx, *grads):
        positions, = ctx.saved_tensors
        g = [None if x is None or not need else x if x.stride(-1) == 1 else x.contiguous()
             for x, need in zip(grads, ctx.needs_input_grad)]
        there = [x for x in g if x is not None]
        if there:
            d = _turn(there[0], there[1] if len(there) > 1 else None, positions, ctx.plan, None,
                      1 - ctx.turned)
            d = iter(d if len(there) > 1 else (d,))
            g = [None if x is None else next(d) for x in g]
        return (*g, *[None] * (5 - len(g)))


def _turn(Q, K, positions, plan: RotaryPlan, out, backward: int):
    wanted = Q.requires_grad or (K is not None and K.requires_grad)
    if out is not None:
        for x in (out,) if K is None else out:
            wanted = wanted or x.requires_grad
    if wanted and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("a given `out` carries no gradient: call without it, or under "
                             "torch.no_grad()")
        return _RotaryGrad.apply(Q, K, positions, plan, backward)
    return _rotary(Q, K, positions, plan, out, backward)


def rotary(Q: torch.Tensor, K: Optional[torch.Tensor], positions: torch.Tensor, plan: RotaryPlan,
           out=None):
    """Rotates queries and keys of the same tokens in one launch -> (Q', K') (Q' if K is None).

    Q, K       [tokens, heads, head_dim] or [batch, heads, tokens, head_dim], any strides with
               contiguous channels (slices of a fused projection, for instance)
    positions  int32 or int64 [tokens] or [batch, tokens]; with several sections [axes, tokens]
               or [axes, batch, tokens]
    out        tensors to write: each its own input (in place), or memory that no input or other
               output lies in (other parts of one wider tensor may be used)

    Carries gradients to Q and K (not with `out`).
    """
    return _turn(Q, K, positions, plan, out, 0)


def rotary_backward(dQ: torch.Tensor, dK: Optional[torch.Tensor], positions: torch.Tensor,
                    plan: RotaryPlan, out=None):
    """Gradients of rotary()'s inputs from those of its outputs (the transposed map)."""
    return _turn(dQ, dK, positions, plan, out, 1)


# ----------------------------------------------------------------- packed attention

def _host_ints(values, ctype, what: str):
    if isinstance(values, torch.Tensor):
        if values.is_cuda:
            raise ValueError("lengths are planned on the host: pass a list or a CPU tensor")
        values = values.tolist()
    values = list(values)
    made = (ctype * len(values))(*values)
    for x in (min(values), max(values)) if values else ():
        _fits(x, what, 8 * ctypes.sizeof(ctype))
    return made, len(values)


class PackedPlan:
    """The work of a batch of packed sequences, laid out once and used by every layer.

    q_lens, kv_lens  queries and keys of each sequence (host integers, each >= 0)
    causal           query i of n sees keys j <= i + m - n of its sequence's m keys; else all m
    prefix_len       keys of a prefix that every query of every sequence sees
    kv_starts        first key row of each sequence (default: end to end), e.g. [0, cap, 2 * cap]
                     for a cache of fixed capacity per sequence

    The plan's table lives in device memory: keep the plan until the calls (and replays of
    captured graphs) that use it have finished. Made outside of stream capture.
    """

    def __init__(self, q_lens, kv_lens, heads: int, kv_heads: int, head_dim: int,
                 dtype: torch.dtype = torch.bfloat16, causal: bool = True, prefix_len: int = 0,
                 kv_starts=None, device=None):
        device = torch.device(device or "cuda")
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        heads, kv_heads = _fits(heads, "heads"), _fits(kv_heads, "kv_heads")
        head_dim, prefix_len = _fits(head_dim, "head_dim"), _fits(prefix_len, "prefix_len")
        q, n = _host_ints(q_lens, ctypes.c_int32, "a length")
        kv, n_kv = _host_ints(kv_lens, ctypes.c_int32, "a length")
        starts, n_st = (None, n) if kv_starts is None else _host_ints(kv_starts, ctypes.c_int64,
                                                                      "a start")
        if n != n_kv or n != n_st:
            raise ValueError("q_lens, kv_lens and kv_starts must have one entry per sequence")
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a plan is made outside of stream capture")
        desc = PackedDesc(n, heads, kv_heads, head_dim, _dtype_code(dtype), bool(causal),
                          prefix_len)
        self.data = PackedPlanData()
        table = bytearray(1 << 16)
        while True:
            buf = (ctypes.c_char * len(table)).from_buffer(table)
            code = lib().tlsp_packed_make_plan(ctypes.byref(desc), q, kv, starts, buf, len(table),
                                               ctypes.byref(self.data))
            if code != TLSP_ERR_WORKSPACE:
                break
            table = bytearray(self.data.items_bytes)
        _check(code, "tlsp_packed_make_plan")
        self.heads, self.kv_heads, self.head_dim, self.dtype = heads, kv_heads, head_dim, dtype
        self.prefix_len, self.device = prefix_len, device
        self.q_rows, self.kv_rows = self.data.q_rows, self.data.kv_rows
        used = max(self.data.items_bytes, 16)
        # a blocking copy: the table is in place for every stream when this returns
        self.items = torch.frombuffer(table, dtype=torch.uint8)[:used].to(device)
        self._at, self._dev = ctypes.addressof(self.data), device.index
        self._made_on = torch.cuda.current_stream(device).cuda_stream

    def workspace(self) -> "Workspace":
        """A workspace for calls with this plan (calls that overlap in time need one each), zeroed
        on the current stream. Like the plan, kept until replays of graphs that use it are done."""
        return Workspace(None, nbytes=self.data.ws_bytes, device=self.device)


def _packed_rows(t: Optional[torch.Tensor], what: str, rows: int, heads: int, plan: PackedPlan):
    if t is None:
        if rows:
            raise ValueError(f"{what} is missing")
        return None
    shape = t.shape
    if len(shape) != 3 or shape[0] < rows or shape[1] != heads or shape[2] != plan.head_dim:
        raise ValueError(f"{what} must be [>= {rows}, {heads}, {plan.head_dim}], "
                         f"got {tuple(shape)}")
    if t.dtype != plan.dtype or t.get_device() != plan._dev:
        raise ValueError(f"{what} must be {plan.dtype} on {plan.device}")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{what}: channels must be contiguous")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, and packed attention has no backward pass: "
                         "call it under torch.no_grad()")
    return _ROWS.pack(t.data_ptr(), s0, s1)


def _packed(Q, Kp, Vp, K, V, plan: PackedPlan, ws: Workspace, scale, out, lse):
    q_rows, kv_rows, h, hk, dev = plan.q_rows, plan.kv_rows, plan.heads, plan.kv_heads, plan._dev
    q = _packed_rows(Q, "Q", q_rows, h, plan)
    k = _packed_rows(K, "K", kv_rows, hk, plan)
    v = _packed_rows(V, "V", kv_rows, hk, plan)
    if out is None:
        out = _like(Q)
        if Q.shape[0] > q_rows:
            out[q_rows:].zero_()
    o = _packed_rows(out, "out", q_rows, h, plan)
    lse_ptr = None
    if lse is not None:
        if lse.dtype != torch.float32 or lse.get_device() != dev or lse.dim() != 2 or \
                lse.shape[0] < q_rows or lse.shape[1] != h or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous fp32 [>= {q_rows}, {h}] on {plan.device}")
        lse_ptr = lse.data_ptr()
    if ws.buf.get_device() != dev:
        raise ValueError(f"the workspace must live on {plan.device}")
    if scale is None:
        scale = 0.0
    elif abs(scale) < 2.0 ** -149:  # 0 for the library: 1/sqrt(d)
        raise ValueError("scale must not be 0 in 32 bits")
    here = torch._C._cuda_getCurrentRawStream(dev)
    if (here != plan._made_on or here != ws.made_on) and \
            not torch.cuda.is_current_stream_capturing():
        # what was made on another stream is not reused before this call is done
        stream = torch.cuda.current_stream(dev)
        if here != plan._made_on:
            plan.items.record_stream(stream)
        if here != ws.made_on:
            ws.buf.record_stream(stream)
    items, at = plan.items.data_ptr(), plan._at
    if plan.prefix_len:
        kp = _packed_rows(Kp, "K_prefix", plan.prefix_len, hk, plan)
        vp = _packed_rows(Vp, "V_prefix", plan.prefix_len, hk, plan)
        rc = _launch(dev, lib().tlsp_prefix_attention, at, items, q, kp, vp, k, v, o, lse_ptr,
                     scale, ws.buf.data_ptr(), ws.nbytes)
        _check(rc, "tlsp_prefix_attention")
    else:
        rc = _launch(dev, lib().tlsp_packed_attention, at, items, q, k, v, o, lse_ptr, scale,
                     ws.buf.data_ptr(), ws.nbytes)
        _check(rc, "tlsp_packed_attention")
    return out


def packed_attention(Q, K, V, plan: PackedPlan, ws: Workspace, scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Attention over packed sequences (causal, grouped heads) -> O [tokens, heads, head_dim].

    Q [tokens, heads, d], K, V [tokens, kv_heads, d]: sequences end to end (keys: at the plan's
    kv_starts), any strides that are multiples of 16 bytes with contiguous channels. lse, if
    given (fp32 [tokens, heads]), receives each row's log partition; rows that see no key get
    O = 0 and lse = -inf. Rows of a given `out` (and lse) behind the last sequence are left as
    they are; without `out` they are zero. `out` and lse may share no memory with an input or
    each other (not out=Q): other parts of one wider tensor may be used. No backward pass: tensors
    that require gradients are refused unless gradients are switched off.
    """
    if plan.prefix_len:
        raise ValueError("the plan has a prefix: call prefix_attention")
    return _packed(Q, None, None, K, V, plan, ws, scale, out, lse)


def prefix_attention(Q, K_prefix, V_prefix, K, V, plan: PackedPlan, ws: Workspace,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None):
    """packed_attention in which every query also sees all keys of one shared prefix
    (K_prefix, V_prefix [prefix_len, kv_heads, d]), which is read once for all short sequences.
    K and V may be None when no sequence has keys of its own."""
    if not plan.prefix_len:
        raise ValueError("the plan has no prefix: call packed_attention")
    return _packed(Q, K_prefix, V_prefix, K, V, plan, ws, scale, out, lse)
