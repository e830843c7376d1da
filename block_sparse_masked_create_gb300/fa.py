"""Python binding of libfa.so: argument marshalling only. Every step of the computation runs in the
library's CUDA kernels; PyTorch provides device memory and the current stream.

Names follow the C ABI (include/fa.h): create_block_mask, flex_forward, flex_decode, ...
The library must have been built (``__graft_entry__.build()`` or ``python -m
block_sparse_masked_create_gb300.build``); a missing library is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass, field
from typing import Optional, Sequence

import torch

from . import build as _build

MAX_OPS = 16
MAX_TERMS = 8

OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE_CHECK, ERR_BUFFER = range(8)
_OPS = {"true": 0, "causal": 1, "window": 2, "prefix": 3, "doc": 4, "and": 5, "or": 6}


class FaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


class MaskRule(ctypes.Structure):
    _fields_ = [("n_ops", ctypes.c_int32), ("op", ctypes.c_int32 * MAX_OPS), ("arg", ctypes.c_int64 * MAX_OPS),
                ("doc_ids", ctypes.c_void_p), ("doc_batch", ctypes.c_int32), ("doc_len", ctypes.c_int32),
                ("q_offset", ctypes.c_void_p), ("batch_dependent", ctypes.c_int32),
                ("head_dependent", ctypes.c_int32)]


class ScoreRule(ctypes.Structure):
    _fields_ = [("alibi_slopes", ctypes.c_void_p), ("rel_bias", ctypes.c_void_p), ("softcap", ctypes.c_float)]


class RowsC(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_n", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


class QkRule(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class BlockMaskC(ctypes.Structure):
    _fields_ = [("Bm", ctypes.c_int32), ("Hm", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("kv_len", ctypes.c_int32), ("bq", ctypes.c_int32), ("bk", ctypes.c_int32),
                ("nq", ctypes.c_int32), ("nk", ctypes.c_int32),
                ("kv_num", ctypes.c_void_p), ("kv_idx", ctypes.c_void_p), ("full_kv_num", ctypes.c_void_p),
                ("full_kv_idx", ctypes.c_void_p), ("q_num", ctypes.c_void_p), ("q_idx", ctypes.c_void_p),
                ("full_q_num", ctypes.c_void_p), ("full_q_idx", ctypes.c_void_p),
                ("block_class", ctypes.c_void_p), ("doc_run", ctypes.c_void_p), ("doc_sorted", ctypes.c_void_p),
                ("row_order", ctypes.c_void_p), ("rule", MaskRule)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libfa.so (raises if it has not been built: there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libfa.so not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    P = ctypes.POINTER
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_status_string.argtypes = [ctypes.c_int]
    lib.fa_version.restype = ctypes.c_char_p
    lib.fa_block_mask_bytes.restype = sz
    lib.fa_block_mask_bytes.argtypes = [P(MaskRule), i32, i32, i32, i32, i32, i32]
    lib.fa_create_block_mask.restype = ctypes.c_int
    lib.fa_create_block_mask.argtypes = [P(MaskRule), i32, i32, i32, i32, i32, i32, vp, sz, P(BlockMaskC), vp]
    fwd_args = [vp, vp, vp, P(BlockMaskC), P(ScoreRule), f32, vp, i32, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.fa_flex_forward.restype = ctypes.c_int
    lib.fa_flex_forward.argtypes = fwd_args
    lib.fa_flex_forward_mma.restype = ctypes.c_int
    lib.fa_flex_forward_mma.argtypes = fwd_args
    lib.fa_block_mask_select_bytes.restype = sz
    lib.fa_block_mask_select_bytes.argtypes = [P(BlockMaskC), i32]
    lib.fa_block_mask_select_rows.restype = ctypes.c_int
    lib.fa_block_mask_select_rows.argtypes = [P(BlockMaskC), vp, i32, vp, sz, P(BlockMaskC), vp, vp]
    lib.fa_forward_split_workspace_bytes.restype = sz
    lib.fa_forward_split_workspace_bytes.argtypes = [P(BlockMaskC), i32, i32, i32, i32]
    lib.fa_flex_forward_split.restype = ctypes.c_int
    lib.fa_flex_forward_split.argtypes = [vp, vp, vp, P(BlockMaskC), P(ScoreRule), f32, vp, i32, vp, i32, i32, i32, i32,
                                          i32, i32, i32, vp, sz, vp, vp]
    lib.fa_forward_host_workspace_bytes.restype = sz
    lib.fa_forward_host_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.fa_flex_forward_host.restype = ctypes.c_int
    lib.fa_flex_forward_host.argtypes = [vp, vp, vp, P(BlockMaskC), P(ScoreRule), f32, vp, i32, vp, i32, i32, i32, i32,
                                         i32, i32, vp, sz, vp, vp]
    lib.fa_flex_forward_paged.restype = ctypes.c_int
    lib.fa_flex_forward_paged.argtypes = [vp, vp, vp, vp, i32, i32, i32, P(BlockMaskC), P(ScoreRule), f32, vp, i32, vp,
                                          i32, i32, i32, i32, i32, i32, vp, vp]
    lib.fa_flex_backward.restype = ctypes.c_int
    lib.fa_flex_backward.argtypes = [vp, vp, vp, vp, i32, vp, vp, P(BlockMaskC), P(ScoreRule), f32, vp, vp, vp, vp,
                                     i32, i32, i32, i32, i32, i32, vp, vp]
    lib.fa_decode_workspace_bytes.restype = sz
    lib.fa_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.fa_flex_decode.restype = ctypes.c_int
    lib.fa_flex_decode.argtypes = [vp, vp, vp, vp, i32, P(BlockMaskC), P(ScoreRule), f32, vp, i32, vp, i32, i32, i32, i32,
                                   i32, i32, vp, sz, vp, vp, vp]
    lib.fa_flex_decode_noalloc.restype = ctypes.c_int
    lib.fa_flex_decode_noalloc.argtypes = [vp, vp, vp, vp, i32, P(BlockMaskC), P(ScoreRule), f32, vp, i32, vp, i32,
                                           i32, i32, i32, i32, i32, vp, vp, vp]
    lib.fa_decode_noalloc_scratch_bytes.restype = sz
    lib.fa_decode_noalloc_scratch_bytes.argtypes = []
    R, K = P(RowsC), P(QkRule)
    lib.fa_qk_norm_rope.restype = ctypes.c_int
    lib.fa_qk_norm_rope.argtypes = [R, R, R, K, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
    lib.fa_qk_norm_rope_backward_workspace_bytes.restype = sz
    lib.fa_qk_norm_rope_backward_workspace_bytes.argtypes = [i32, i32, i32]
    lib.fa_qk_norm_rope_backward.restype = ctypes.c_int
    lib.fa_qk_norm_rope_backward.argtypes = [R, R, vp, vp, vp, K, vp, R, R, R, i32, vp, vp, i32, i32, i32, i32, i32, vp,
                                             sz, vp]
    lib.fa_kv_append.restype = ctypes.c_int
    lib.fa_kv_append.argtypes = [R, R, R, K, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.fa_kv_append_fp8.restype = ctypes.c_int
    lib.fa_kv_append_fp8.argtypes = [R, R, R, K, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                     vp, vp]
    lib.fa_decode_fp8_workspace_bytes.restype = sz
    lib.fa_decode_fp8_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.fa_flex_decode_fp8.restype = ctypes.c_int
    lib.fa_flex_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, P(BlockMaskC), P(ScoreRule), f32, vp, i32, vp, i32,
                                       i32, i32, i32, i32, i32, vp, sz, vp, vp, vp]
    lib.fa_forward_paged_fp8_workspace_bytes.restype = sz
    lib.fa_forward_paged_fp8_workspace_bytes.argtypes = [P(BlockMaskC), P(ScoreRule), i32, i32, i32, i32, i32]
    lib.fa_flex_forward_paged_fp8.restype = ctypes.c_int
    lib.fa_flex_forward_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, P(BlockMaskC), P(ScoreRule), f32, vp,
                                              i32, vp, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp, vp]
    lib.fa_block_mask_stats.restype = ctypes.c_int
    lib.fa_block_mask_stats.argtypes = [P(BlockMaskC), vp, vp]
    lib.fa_check_status.restype = ctypes.c_int
    lib.fa_check_status.argtypes = [vp, vp]
    lib.fa_set_wait_timeout_ns.restype = None
    lib.fa_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.fa_get_wait_timeout_ns.restype = ctypes.c_uint64
    lib.fa_get_wait_timeout_ns.argtypes = []
    lib.fa_debug_wait_timeout.restype = ctypes.c_int
    lib.fa_debug_wait_timeout.argtypes = [vp, ctypes.c_uint64, vp]
    lib.fa_debug_softcap.restype = ctypes.c_int
    lib.fa_debug_softcap.argtypes = [vp, vp, i32, ctypes.c_float, vp]
    lib.fa_debug_tc5_gemm.restype = ctypes.c_int
    lib.fa_debug_tc5_gemm.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
    _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return load().fa_status_string(code).decode()
    except Exception:  # library not loadable
        return f"status {code}"


def _check(code: int, what: str):
    if code != OK:
        raise FaError(code, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


# ----------------------------------------------------------------------------------------------
# rules
# ----------------------------------------------------------------------------------------------
def make_mask_rule(spec: Sequence[tuple], doc_ids: Optional[torch.Tensor] = None,
                   q_offset: Optional[torch.Tensor] = None, batch_dependent: Optional[bool] = None,
                   head_dependent: bool = False) -> MaskRule:
    """Rule spec (postfix tuples, see workloads.py) -> fa_mask_rule. doc_ids int32 [doc_batch, doc_len] and
    q_offset int32 [B] must be device tensors and stay alive while the rule is used."""
    if not 1 <= len(spec) <= MAX_OPS:
        raise ValueError("rule must have 1..16 ops")
    r = MaskRule()
    r.n_ops = len(spec)
    for i, op in enumerate(spec):
        r.op[i] = _OPS[op[0]]
        r.arg[i] = int(op[1]) if len(op) > 1 else 0
    if doc_ids is not None:
        if doc_ids.dtype != torch.int32 or doc_ids.dim() != 2 or not doc_ids.is_contiguous():
            raise ValueError("doc_ids must be contiguous int32 [doc_batch, doc_len]")
        r.doc_ids = doc_ids.data_ptr()
        r.doc_batch, r.doc_len = doc_ids.shape
    if q_offset is not None:
        if q_offset.dtype != torch.int32 or not q_offset.is_contiguous():
            raise ValueError("q_offset must be contiguous int32 [B]")
        r.q_offset = q_offset.data_ptr()
    if batch_dependent is None:
        batch_dependent = q_offset is not None or (doc_ids is not None and doc_ids.shape[0] > 1)
    r.batch_dependent = int(bool(batch_dependent))
    r.head_dependent = int(bool(head_dependent))
    r._tensors = (doc_ids, q_offset)  # the raw pointers above stay valid while the rule lives
    return r


def make_score_rule(alibi_slopes: Optional[torch.Tensor] = None, rel_bias: Optional[torch.Tensor] = None,
                    softcap: float = 0.0) -> ScoreRule:
    s = ScoreRule()
    for t in (alibi_slopes, rel_bias):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError("score tables must be contiguous fp32 device tensors")
    s.alibi_slopes = None if alibi_slopes is None else alibi_slopes.data_ptr()
    s.rel_bias = None if rel_bias is None else rel_bias.data_ptr()
    s.softcap = float(softcap or 0.0)
    s._tensors = (alibi_slopes, rel_bias)  # the raw pointers above stay valid while the rule lives
    return s


# ----------------------------------------------------------------------------------------------
# BlockMask
# ----------------------------------------------------------------------------------------------
@dataclass
class BlockMask:
    c: BlockMaskC
    buf: torch.Tensor
    keep: list = field(default_factory=list)   # tensors the rule points into

    @property
    def shape(self):
        return (self.c.Bm, self.c.Hm, self.c.nq, self.c.nk)

    def _view(self, addr: int, n: int, dtype) -> torch.Tensor:
        off = addr - self.buf.data_ptr()
        nbytes = n * (4 if dtype == torch.int32 else 1)
        return self.buf[off:off + nbytes].view(dtype)

    def tables(self) -> dict:
        """Device views of the tables: kv_num [Bm,Hm,nq], kv_idx [Bm,Hm,nq,nk], ..., block_class."""
        Bm, Hm, nq, nk = self.shape
        c = self.c
        out = {}
        for name, n, shp in (("kv_num", Bm * Hm * nq, (Bm, Hm, nq)), ("full_kv_num", Bm * Hm * nq, (Bm, Hm, nq)),
                             ("q_num", Bm * Hm * nk, (Bm, Hm, nk)), ("full_q_num", Bm * Hm * nk, (Bm, Hm, nk)),
                             ("kv_idx", Bm * Hm * nq * nk, (Bm, Hm, nq, nk)),
                             ("full_kv_idx", Bm * Hm * nq * nk, (Bm, Hm, nq, nk)),
                             ("q_idx", Bm * Hm * nk * nq, (Bm, Hm, nk, nq)),
                             ("full_q_idx", Bm * Hm * nk * nq, (Bm, Hm, nk, nq))):
            out[name] = self._view(getattr(c, name), n, torch.int32).view(shp)
        out["block_class"] = self._view(c.block_class, Bm * Hm * nq * nk, torch.uint8).view(Bm, Hm, nq, nk)
        if c.row_order:
            out["row_order"] = self._view(c.row_order, Bm * Hm * nq, torch.int32).view(Bm, Hm, nq)
        return out


def block_mask_bytes(rule: MaskRule, B: int, H: int, Q_LEN: int, KV_LEN: int, Bq: int, Bk: int) -> int:
    return int(load().fa_block_mask_bytes(ctypes.byref(rule), B, H, Q_LEN, KV_LEN, Bq, Bk))


def create_block_mask(rule: MaskRule, B: int, H: int, Q_LEN: int, KV_LEN: int, Bq: int = 128, Bk: int = 128,
                      device="cuda", keep: Optional[list] = None, buf: Optional[torch.Tensor] = None) -> BlockMask:
    """fa_create_block_mask: classify every block, compact the lists, build the transpose (on `device`)."""
    lib = load()
    n = block_mask_bytes(rule, B, H, Q_LEN, KV_LEN, Bq, Bk)
    if n == 0:
        raise FaError(ERR_SHAPE, "fa_block_mask_bytes")
    if buf is None or buf.numel() < n:
        buf = torch.empty(n, dtype=torch.uint8, device=device)
    c = BlockMaskC()
    _check(lib.fa_create_block_mask(ctypes.byref(rule), B, H, Q_LEN, KV_LEN, Bq, Bk, _ptr(buf), buf.numel(),
                                    ctypes.byref(c), _stream(buf.device)), "fa_create_block_mask")
    return BlockMask(c, buf, list(keep or []))


def recreate_block_mask(bm: BlockMask, rule: MaskRule, B: int, H: int, Q_LEN: int, KV_LEN: int, Bq: int,
                        Bk: int) -> None:
    """Rebuild into an existing BlockMask's buffer (same sizes; no allocation)."""
    _check(load().fa_create_block_mask(ctypes.byref(rule), B, H, Q_LEN, KV_LEN, Bq, Bk, _ptr(bm.buf), bm.buf.numel(),
                                       ctypes.byref(bm.c), _stream(bm.buf.device)), "fa_create_block_mask")


def select_rows(src: BlockMask, q_pos: torch.Tensor, out: Optional[BlockMask] = None,
                status: Optional[torch.Tensor] = None) -> BlockMask:
    """fa_block_mask_select_rows: from a table prebuilt for the longest context (global positions), the row
    block holding each request's query position q_pos[b] (device int32 [Bz]), as a one-row-per-request
    mask (Bm = Bz, q_len = 1, Bq = 1) whose rule sees q_pos as the query offset. Reuses `out`'s buffer."""
    if q_pos.dtype != torch.int32 or not q_pos.is_contiguous() or q_pos.dim() != 1:
        raise ValueError("q_pos must be contiguous int32 [Bz]")
    lib = load()
    Bz = q_pos.shape[0]
    n = int(lib.fa_block_mask_select_bytes(ctypes.byref(src.c), Bz))
    if n == 0:
        raise FaError(ERR_SHAPE, "fa_block_mask_select_bytes")
    if out is None or out.buf.numel() < n:
        out = BlockMask(BlockMaskC(), torch.empty(n, dtype=torch.uint8, device=src.buf.device), [])
    out.keep = list(src.keep) + [src, q_pos]
    _check(lib.fa_block_mask_select_rows(ctypes.byref(src.c), _ptr(q_pos), Bz, _ptr(out.buf), out.buf.numel(),
                                         ctypes.byref(out.c), _ptr(status), _stream(out.buf.device)),
           "fa_block_mask_select_rows")
    return out


def block_mask_stats(bm: BlockMask, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int64[6] on the device: full, partial, empty, max row length, sum of row lengths, rows."""
    if out is None:
        out = torch.empty(6, dtype=torch.int64, device=bm.buf.device)
    _check(load().fa_block_mask_stats(ctypes.byref(bm.c), _ptr(out), _stream(out.device)), "fa_block_mask_stats")
    return out


# ----------------------------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------------------------
def _out_code(out: torch.Tensor) -> int:
    if out.dtype == torch.bfloat16:
        return 0
    if out.dtype == torch.float32:
        return 1
    raise ValueError("out must be bf16 or fp32")


def flex_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask,
                 score: Optional[ScoreRule] = None, scale: Optional[float] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, counters: Optional[torch.Tensor] = None,
                 force_mma: bool = False, out_dtype=torch.bfloat16):
    """fa_flex_forward: q [B,Hq,Q_LEN,d], k/v [B,Hkv,KV_LEN,d] bf16 contiguous on the GPU.
    Returns (out [B,Hq,Q_LEN,d] in bf16 or fp32 (the dtype of `out`, else out_dtype), lse fp32 [B,Hq,Q_LEN])."""
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    B, Hq, Q_LEN, d = q.shape
    Hkv, KV_LEN = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Q_LEN), dtype=torch.float32, device=q.device)
    fn = load().fa_flex_forward_mma if force_mma else load().fa_flex_forward
    _check(fn(_ptr(q), _ptr(k), _ptr(v), ctypes.byref(block_mask.c), ctypes.byref(score) if score else None,
              float(scale) if scale else 0.0, _ptr(out), _out_code(out), _ptr(lse), B, Hq, Hkv, Q_LEN, KV_LEN, d,
              _ptr(status), _ptr(counters), _stream(q.device)), "fa_flex_forward")
    return out, lse


def forward_split_workspace_bytes(block_mask: BlockMask, B: int, Hq: int, d: int, chunk_blocks: int) -> int:
    return int(load().fa_forward_split_workspace_bytes(ctypes.byref(block_mask.c), B, Hq, d, chunk_blocks))


def flex_forward_split(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask,
                       score: Optional[ScoreRule] = None, scale: Optional[float] = None, chunk_blocks: int = 16,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       out_dtype=torch.bfloat16):
    """fa_flex_forward_split: the forward with each query block row cut into chunks of at most chunk_blocks
    key blocks, run as separate tiles and merged. Same inputs and outputs as flex_forward."""
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    B, Hq, Q_LEN, d = q.shape
    Hkv, KV_LEN = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Q_LEN), dtype=torch.float32, device=q.device)
    n = forward_split_workspace_bytes(block_mask, B, Hq, d, chunk_blocks)
    if n == 0:
        raise FaError(ERR_SHAPE, "fa_forward_split_workspace_bytes")
    if workspace is None or workspace.numel() < n:
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _check(load().fa_flex_forward_split(_ptr(q), _ptr(k), _ptr(v), ctypes.byref(block_mask.c),
                                        ctypes.byref(score) if score else None, float(scale) if scale else 0.0,
                                        _ptr(out), _out_code(out), _ptr(lse), B, Hq, Hkv, Q_LEN, KV_LEN, d,
                                        chunk_blocks, _ptr(workspace), workspace.numel(), _ptr(status),
                                        _stream(q.device)), "fa_flex_forward_split")
    return out, lse


def forward_host_workspace_bytes(B: int, Hq: int, Hkv: int, Q_LEN: int, KV_LEN: int, d: int,
                                 out_dtype=torch.bfloat16) -> int:
    return int(load().fa_forward_host_workspace_bytes(B, Hq, Hkv, Q_LEN, KV_LEN, d,
                                                      1 if out_dtype == torch.float32 else 0))


def flex_forward_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask,
                      score: Optional[ScoreRule] = None, scale: Optional[float] = None,
                      out: torch.Tensor = None, lse: torch.Tensor = None, workspace: torch.Tensor = None,
                      status: Optional[torch.Tensor] = None, device=None):
    """fa_flex_forward_host: q/k/v (bf16), out (bf16 or fp32) and lse (fp32) are host tensors (pin them for
    full copy speed); the chunks stream through `workspace` on `device`. Returns (out, lse) once the
    current stream of `device` has been synchronised by the caller."""
    for t in (q, k, v, out, lse):
        if t is None or t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v, out, lse must be contiguous host tensors")
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise ValueError("q, k, v must be bf16")
    B, Hq, Q_LEN, d = q.shape
    Hkv, KV_LEN = k.shape[1], k.shape[2]
    dev = torch.device(device) if device is not None else block_mask.buf.device
    if workspace is None:
        workspace = torch.empty(forward_host_workspace_bytes(B, Hq, Hkv, Q_LEN, KV_LEN, d, out.dtype),
                                dtype=torch.uint8, device=dev)
    _check(load().fa_flex_forward_host(_ptr(q), _ptr(k), _ptr(v), ctypes.byref(block_mask.c),
                                       ctypes.byref(score) if score else None, float(scale) if scale else 0.0,
                                       _ptr(out), _out_code(out), _ptr(lse), B, Hq, Hkv, Q_LEN, KV_LEN, d,
                                       _ptr(workspace), workspace.numel(), _ptr(status), _stream(dev)),
           "fa_flex_forward_host")
    return out, lse


def flex_forward_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                       block_mask: BlockMask, KV_LEN: int, score: Optional[ScoreRule] = None,
                       scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       out_dtype=torch.bfloat16):
    """fa_flex_forward_paged: q [B,Hq,Q_LEN,d]; k/v pages [P,Hkv,page,d] bf16 with page == the mask's Bk;
    page_table int32 [B,max_pages] (logical key block -> physical page)."""
    for t in (q, k_pages, v_pages):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("q, k_pages, v_pages must be contiguous bf16 CUDA tensors")
    if page_table.dtype != torch.int32 or not page_table.is_contiguous() or page_table.dim() != 2:
        raise ValueError("page_table must be contiguous int32 [B, max_pages]")
    B, Hq, Q_LEN, d = q.shape
    P, Hkv, page, _ = k_pages.shape
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Q_LEN), dtype=torch.float32, device=q.device)
    _check(load().fa_flex_forward_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), P, page,
                                        page_table.shape[1], ctypes.byref(block_mask.c),
                                        ctypes.byref(score) if score else None, float(scale) if scale else 0.0,
                                        _ptr(out), _out_code(out), _ptr(lse), B, Hq, Hkv, Q_LEN, KV_LEN, d,
                                        _ptr(status), _stream(q.device)), "fa_flex_forward_paged")
    return out, lse


def flex_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                  dout: torch.Tensor, block_mask: BlockMask, score: Optional[ScoreRule] = None,
                  scale: Optional[float] = None, dq: Optional[torch.Tensor] = None,
                  dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                  delta: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """fa_flex_backward: gradients (dq, dk, dv) in fp32 of fa_flex_forward's out for the upstream gradient
    dout (bf16, layout of q); out and lse are that forward's outputs."""
    for t in (q, k, v, dout):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("q, k, v, dout must be contiguous bf16 CUDA tensors")
    B, Hq, Q_LEN, d = q.shape
    Hkv, KV_LEN = k.shape[1], k.shape[2]
    dev = q.device
    dq = torch.empty(q.shape, dtype=torch.float32, device=dev) if dq is None else dq
    dk = torch.empty(k.shape, dtype=torch.float32, device=dev) if dk is None else dk
    dv = torch.empty(v.shape, dtype=torch.float32, device=dev) if dv is None else dv
    delta = torch.empty((B, Hq, Q_LEN), dtype=torch.float32, device=dev) if delta is None else delta
    _check(load().fa_flex_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _out_code(out), _ptr(dout), _ptr(lse),
                                   ctypes.byref(block_mask.c), ctypes.byref(score) if score else None,
                                   float(scale) if scale else 0.0, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(delta),
                                   B, Hq, Hkv, Q_LEN, KV_LEN, d, _ptr(status), _stream(dev)), "fa_flex_backward")
    return dq, dk, dv


def decode_workspace_bytes(Bz: int, Hq: int, d: int, max_pages: int, page: int) -> int:
    return int(load().fa_decode_workspace_bytes(Bz, Hq, d, max_pages, page))


def flex_decode(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                block_mask: BlockMask, score: Optional[ScoreRule] = None, scale: Optional[float] = None,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                counters: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16):
    """fa_flex_decode: q [Bz,Hq,d], k/v pages [P,Hkv,page,d] bf16, page_table int32 [Bz,max_pages]."""
    Bz, Hq, d = q.shape
    P, Hkv, page, _ = k_pages.shape
    max_pages = page_table.shape[1]
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((Bz, Hq), dtype=torch.float32, device=q.device)
    need = decode_workspace_bytes(Bz, Hq, d, max_pages, page)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(load().fa_flex_decode(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), P,
                                 ctypes.byref(block_mask.c), ctypes.byref(score) if score else None,
                                 float(scale) if scale else 0.0, _ptr(out), _out_code(out), _ptr(lse), Bz, Hq, Hkv,
                                 d, page, max_pages, _ptr(workspace), workspace.numel(), _ptr(status),
                                 _ptr(counters), _stream(q.device)), "fa_flex_decode")
    return out, lse


def decode_noalloc_scratch_bytes() -> int:
    return int(load().fa_decode_noalloc_scratch_bytes())


def flex_decode_noalloc(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                        block_mask: BlockMask, score: Optional[ScoreRule] = None, scale: Optional[float] = None,
                        out: torch.Tensor = None, lse: torch.Tensor = None, status: Optional[torch.Tensor] = None,
                        counters: Optional[torch.Tensor] = None) -> int:
    """fa_flex_decode_noalloc: the paged decode with its split workspace in the library's fixed device
    array, for callers that cannot allocate. `out` and `lse` must be provided (nothing is allocated here).
    Returns the fa_status code (FA_ERR_BUFFER_TOO_SMALL when the problem exceeds the fixed array)."""
    if out is None or lse is None:
        raise ValueError("out and lse must be provided")
    Bz, Hq, d = q.shape
    P, Hkv, page, _ = k_pages.shape
    return int(load().fa_flex_decode_noalloc(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), P, ctypes.byref(block_mask.c),
        ctypes.byref(score) if score else None, float(scale) if scale else 0.0, _ptr(out), _out_code(out), _ptr(lse),
        Bz, Hq, Hkv, d, page, page_table.shape[1], _ptr(status), _ptr(counters), _stream(q.device)))


# ----------------------------------------------------------------------------------------------
# the attention's inputs: norms, rotation, paged-cache append
# ----------------------------------------------------------------------------------------------
KV_SCALE_TOKENS = 32  # tokens of a page that share a scale in the 8-bit cache


def make_qk_rule(q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False) -> QkRule:
    """fa_qk_rule: norm weights fp32 [d] (None: no norm), rotation frequencies fp32 [rot_dim / 2] (None: no rotation;
    the first rot_dim = 2 * len(inv_freq) elements of a row are rotated), pairs (i, i + rot_dim / 2) or, interleaved,
    (2 i, 2 i + 1)."""
    r = QkRule()
    for t in (q_weight, k_weight, inv_freq):
        if t is not None and (t.dtype != torch.float32 or t.dim() != 1 or not t.is_contiguous()):
            raise ValueError("norm weights and inv_freq must be contiguous 1-D fp32 device tensors")
    r.q_weight = None if q_weight is None else q_weight.data_ptr()
    r.k_weight = None if k_weight is None else k_weight.data_ptr()
    r.eps = float(eps)
    r.inv_freq = None if inv_freq is None else inv_freq.data_ptr()
    r.rot_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
    r.interleaved = int(bool(interleaved))
    r._tensors = (q_weight, k_weight, inv_freq)  # the raw pointers above stay valid while the rule lives
    return r


def _rows(t: Optional[torch.Tensor], shape, dtype, device, what: str, written: bool = False):
    """fa_rows of a [B, N, H, d] tensor of any b / n / h strides."""
    if t is None:
        return None
    sb, sn, sh, sd = t.stride() if t.dim() == 4 else (0, 0, 0, 0)
    if sd != 1 or t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)} on {device} with contiguous rows")
    if written and not (sb and sn and sh) and any(st == 0 and n > 1 for st, n in zip((sb, sn, sh), shape)):
        raise ValueError(f"{what} is written: its elements must not share memory")
    return RowsC(t.data_ptr(), sb, sn, sh)


def _same(t: Optional[torch.Tensor], shape, dtype, device, what: str):
    if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _scratch(t: Optional[torch.Tensor], device) -> int:
    """Bytes of a caller's workspace (0: none given)."""
    if t is None:
        return 0
    if not t.is_contiguous() or t.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return t.numel() * t.element_size()


def _check_qk_rule(rule: Optional[QkRule], d: int, device):
    if rule is None:
        return
    wq, wk, f = rule._tensors
    if ((wq is not None and (wq.device != device or wq.shape != (d,))) or
            (wk is not None and (wk.device != device or wk.shape != (d,))) or (f is not None and f.device != device)):
        raise ValueError(f"the rule's tensors must be on {device}, its weights of {d} elements")


def _ref(s):
    return None if s is None else ctypes.byref(s)


def _at(t: Optional[torch.Tensor]):
    """Address for an argument declared as a pointer."""
    return None if t is None else t.data_ptr()


def _call(device, fn, *args) -> int:
    """fn(*args, stream) on `device`'s current stream, with that device current. (The stream's handle is taken without the
    torch.cuda.Stream object around it, which costs as much as half the launch.)"""
    i = device.index
    if i == torch.cuda.current_device():
        return fn(*args, torch._C._cuda_getCurrentRawStream(i))
    with torch.cuda.device(device):
        return fn(*args, torch._C._cuda_getCurrentRawStream(i))


def _qkv_shape(q, k, v):
    """(B, Hq, Hkv, N, d, device) of the rows that are there; without query (key) rows Hq = Hkv."""
    any_ = q if q is not None else k if k is not None else v
    if any_ is None or any_.dim() != 4 or not any_.is_cuda:
        raise ValueError("q, k, v must be CUDA tensors [B, N, H, d]")
    B, N, H, d = any_.shape
    kv = k if k is not None else v
    Hq = q.shape[2] if q is not None else H
    return B, Hq, kv.shape[2] if kv is not None else Hq, N, d, any_.device


def qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor], rule: QkRule,
                 q_offset: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None):
    """fa_qk_norm_rope: rows q [B,N,Hq,d], k, v [B,N,Hkv,d] bf16 (views of a packed projection are fine; None: left out)
    -> (q_out [B,Hq,N,d], k_out, v_out [B,Hkv,N,d]), normalised and rotated, as fa_flex_forward reads them."""
    B, Hq, Hkv, N, d, dev = _qkv_shape(q, k, v)
    bf = torch.bfloat16
    rq, rk, rv = (_rows(q, (B, N, Hq, d), bf, dev, "q"), _rows(k, (B, N, Hkv, d), bf, dev, "k"),
                  _rows(v, (B, N, Hkv, d), bf, dev, "v"))

    def out(t, o, h, name):
        if t is None:
            return None
        if o is None:
            return torch.empty((B, h, N, d), dtype=bf, device=dev)
        return _same(o, (B, h, N, d), bf, dev, name)

    q_out, k_out, v_out = out(q, q_out, Hq, "q_out"), out(k, k_out, Hkv, "k_out"), out(v, v_out, Hkv, "v_out")
    _check_qk_rule(rule, d, dev)
    _same(q_offset, (B,), torch.int32, dev, "q_offset")
    _check(_call(dev, load().fa_qk_norm_rope, _ref(rq), _ref(rk), _ref(rv), ctypes.byref(rule), _at(q_offset), _at(q_out),
                 _at(k_out), _at(v_out), B, Hq, Hkv, N, d), "fa_qk_norm_rope")
    return q_out, k_out, v_out


def qk_norm_rope_backward_workspace_bytes(B: int, N: int, d: int) -> int:
    return int(load().fa_qk_norm_rope_backward_workspace_bytes(B, N, d))


def qk_norm_rope_backward(q: Optional[torch.Tensor], k: Optional[torch.Tensor], dq: Optional[torch.Tensor],
                          dk: Optional[torch.Tensor], dv: Optional[torch.Tensor], rule: QkRule,
                          q_offset: Optional[torch.Tensor] = None, grad_dtype=torch.bfloat16,
                          dq_in: Optional[torch.Tensor] = None, dk_in: Optional[torch.Tensor] = None,
                          dv_in: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """fa_qk_norm_rope_backward: gradients dq [B,Hq,N,d], dk, dv [B,Hkv,N,d] fp32 (as flex_backward returns them; None:
    left out) -> (dq_in [B,N,Hq,d], dk_in, dv_in [B,N,Hkv,d] in the type of the tensors given, else grad_dtype; dq_weight,
    dk_weight fp32 [d] or None). q, k are the forward's rows."""
    given = dq if dq is not None else dk if dk is not None else dv
    if given is not None:
        size = _scratch(workspace, given.device)
    if given is None or given.dim() != 4 or not given.is_cuda:
        raise ValueError("dq, dk, dv must be CUDA tensors [B, H, N, d]")
    B, H, N, d = given.shape
    dev = given.device
    kv = dk if dk is not None else dv
    Hq = dq.shape[1] if dq is not None else kv.shape[1]
    Hkv = kv.shape[1] if kv is not None else Hq
    f32, bf = torch.float32, torch.bfloat16
    _same(dq, (B, Hq, N, d), f32, dev, "dq")
    _same(dk, (B, Hkv, N, d), f32, dev, "dk")
    _same(dv, (B, Hkv, N, d), f32, dev, "dv")
    first = dq_in if dq_in is not None else dk_in if dk_in is not None else dv_in
    kind = first.dtype if first is not None else grad_dtype
    if kind != bf and kind != f32:
        raise ValueError("gradients are bf16 or fp32")
    rows_q, rows_kv = (B, N, Hq, d), (B, N, Hkv, d)
    rq = _rows(q, rows_q, bf, dev, "q") if dq is not None else None
    rk = _rows(k, rows_kv, bf, dev, "k") if dk is not None else None

    def out(t, o, shape):
        return None if t is None else torch.empty(shape, dtype=kind, device=dev) if o is None else o

    dq_in, dk_in, dv_in = out(dq, dq_in, rows_q), out(dk, dk_in, rows_kv), out(dv, dv_in, rows_kv)
    gq = _rows(dq_in, rows_q, kind, dev, "dq_in", written=True)
    gk = _rows(dk_in, rows_kv, kind, dev, "dk_in", written=True)
    gv = _rows(dv_in, rows_kv, kind, dev, "dv_in", written=True)
    _check_qk_rule(rule, d, dev)
    _same(q_offset, (B,), torch.int32, dev, "q_offset")
    dwq = torch.empty(d, dtype=f32, device=dev) if rule.q_weight and dq is not None else None
    dwk = torch.empty(d, dtype=f32, device=dev) if rule.k_weight and dk is not None else None
    lib = load()
    if workspace is None and (dwq is not None or dwk is not None):
        size = lib.fa_qk_norm_rope_backward_workspace_bytes(B, N, d)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(_call(dev, lib.fa_qk_norm_rope_backward, _ref(rq), _ref(rk), _at(dq), _at(dk), _at(dv), ctypes.byref(rule),
                 _at(q_offset), _ref(gq), _ref(gk), _ref(gv), 1 if kind == f32 else 0, _at(dwq), _at(dwk), B, Hq, Hkv, N, d,
                 _at(workspace), size), "fa_qk_norm_rope_backward")
    return dq_in, dk_in, dv_in, dwq, dwk


def _append(q, k, v, k_pages, v_pages, k_scale, v_scale, page_table, rule, q_offset, n_new, q_out, status):
    if k is None or v is None:
        raise ValueError("k and v are required")
    B, Hq, Hkv, N, d, dev = _qkv_shape(q, k, v)
    bf, i32 = torch.bfloat16, torch.int32
    fp8 = k_scale is not None
    rq, rk, rv = (_rows(q, (B, N, Hq, d), bf, dev, "q"), _rows(k, (B, N, Hkv, d), bf, dev, "k"),
                  _rows(v, (B, N, Hkv, d), bf, dev, "v"))
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("pages must be [P, Hkv, page, d] and page_table [B, max_pages]")
    P, _, page, _ = k_pages.shape
    max_pages, pages, kind = page_table.shape[1], (P, Hkv, page, d), torch.float8_e4m3fn if fp8 else bf
    _same(k_pages, pages, kind, dev, "k_pages")
    _same(v_pages, pages, kind, dev, "v_pages")
    if fp8:
        scales = (P, Hkv, page // KV_SCALE_TOKENS)
        _same(k_scale, scales, torch.float32, dev, "k_scale")
        _same(v_scale, scales, torch.float32, dev, "v_scale")
    _same(page_table, (B, max_pages), i32, dev, "page_table")
    _same(q_offset, (B,), i32, dev, "q_offset")
    _same(n_new, (B,), i32, dev, "n_new")
    _same(status, (1,), i32, dev, "status")
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = torch.empty((B, Hq, N, d), dtype=bf, device=dev)
    else:
        _same(q_out, (B, Hq, N, d), bf, dev, "q_out")
    _check_qk_rule(rule, d, dev)
    lib = load()
    if fp8:
        _check(_call(dev, lib.fa_kv_append_fp8, _ref(rq), _ref(rk), _ref(rv), _ref(rule), _at(q_offset), _at(n_new),
                     _at(q_out), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                     page_table.data_ptr(), P, page, max_pages, B, Hq, Hkv, N, d, _at(status)), "fa_kv_append_fp8")
    else:
        _check(_call(dev, lib.fa_kv_append, _ref(rq), _ref(rk), _ref(rv), _ref(rule), _at(q_offset), _at(n_new), _at(q_out),
                     k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), P, page, max_pages, B, Hq, Hkv, N, d,
                     _at(status)), "fa_kv_append")
    return q_out


def kv_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
              page_table: torch.Tensor, rule: Optional[QkRule] = None, q_offset: Optional[torch.Tensor] = None,
              n_new: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """fa_kv_append: normalise and rotate the rows q [B,N,Hq,d] (or None), k, v [B,N,Hkv,d] and put the first n_new[b] keys
    and values of request b at positions q_offset[b] .. of its pages [P,Hkv,page,d] bf16. Returns q_out [B,Hq,N,d] (for
    N = 1, q_out[:, :, 0] is flex_decode's q); rows past n_new[b] are left as they were."""
    return _append(q, k, v, k_pages, v_pages, None, None, page_table, rule, q_offset, n_new, q_out, status)


def kv_append_fp8(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                  v_pages: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, page_table: torch.Tensor,
                  rule: Optional[QkRule] = None, q_offset: Optional[torch.Tensor] = None,
                  n_new: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """fa_kv_append_fp8: kv_append into float8_e4m3fn pages with a power-of-two fp32 scale for each 32 tokens of a page and
    head (k_scale, v_scale [P, Hkv, page / 32]); the cached value is scale * page value."""
    if k_scale is None or v_scale is None:
        raise ValueError("k_scale and v_scale are required")
    return _append(q, k, v, k_pages, v_pages, k_scale, v_scale, page_table, rule, q_offset, n_new, q_out, status)


# ----------------------------------------------------------------------------------------------
# attention over an 8-bit paged cache
# ----------------------------------------------------------------------------------------------
def _check_fp8_cache(q, k_pages, v_pages, k_scale, v_scale, page_table, B, d):
    if q.dtype != torch.bfloat16 or not q.is_contiguous() or not q.is_cuda:
        raise ValueError("q must be a contiguous bf16 CUDA tensor")
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("pages must be [P, Hkv, page, d] and page_table [B, max_pages]")
    dev = q.device
    P, Hkv, page, _ = shape = k_pages.shape
    f8, f32 = torch.float8_e4m3fn, torch.float32
    _same(k_pages, (P, Hkv, page, d), f8, dev, "k_pages")
    _same(v_pages, shape, f8, dev, "v_pages")
    scales = (P, Hkv, page // KV_SCALE_TOKENS)
    _same(k_scale, scales, f32, dev, "k_scale")
    _same(v_scale, scales, f32, dev, "v_scale")
    max_pages = page_table.shape[1]
    _same(page_table, (B, max_pages), torch.int32, dev, "page_table")
    return P, Hkv, page, max_pages, dev


def _outputs(shape, dev, out, lse, out_dtype):
    out = torch.empty(shape, dtype=out_dtype, device=dev) if out is None else _same(out, shape, out.dtype, dev, "out")
    rows = shape[:-1]
    lse = torch.empty(rows, dtype=torch.float32, device=dev) if lse is None else _same(lse, rows, torch.float32, dev, "lse")
    return out, lse


def decode_fp8_workspace_bytes(Bz: int, Hq: int, Hkv: int, d: int, max_pages: int, page: int) -> int:
    return int(load().fa_decode_fp8_workspace_bytes(Bz, Hq, Hkv, d, max_pages, page))


def flex_decode_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, page_table: torch.Tensor, block_mask: BlockMask,
                    score: Optional[ScoreRule] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, counters: Optional[torch.Tensor] = None,
                    out_dtype=torch.bfloat16):
    """fa_flex_decode_fp8: flex_decode over float8_e4m3fn pages [P,Hkv,page,d] with scales fp32 [P,Hkv,page/32]."""
    if q.dim() != 3:
        raise ValueError("q must be [Bz, Hq, d]")
    Bz, Hq, d = q.shape
    q = q.contiguous()
    _same(status, (1,), torch.int32, q.device, "status")
    _same(counters, (4,), torch.int64, q.device, "counters")
    size = _scratch(workspace, q.device)
    P, Hkv, page, max_pages, dev = _check_fp8_cache(q, k_pages, v_pages, k_scale, v_scale, page_table, Bz, d)
    out, lse = _outputs((Bz, Hq, d), dev, out, lse, out_dtype)
    if workspace is None:
        size = max(decode_fp8_workspace_bytes(Bz, Hq, Hkv, d, max_pages, page), 16)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(_call(dev, load().fa_flex_decode_fp8, _at(q), _at(k_pages), _at(v_pages), _at(k_scale), _at(v_scale),
                 _at(page_table), P, ctypes.byref(block_mask.c), _ref(score), float(scale) if scale else 0.0, _at(out),
                 _out_code(out), _at(lse), Bz, Hq, Hkv, d, page, max_pages, _at(workspace), size, _at(status),
                 _at(counters)), "fa_flex_decode_fp8")
    return out, lse


def forward_paged_fp8_workspace_bytes(block_mask: BlockMask, B: int, Hq: int, Hkv: int, d: int, chunk_blocks: int = 0,
                                      score: Optional[ScoreRule] = None) -> int:
    return int(load().fa_forward_paged_fp8_workspace_bytes(ctypes.byref(block_mask.c), _ref(score), B, Hq, Hkv, d,
                                                           chunk_blocks))


def flex_forward_paged_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                           v_scale: torch.Tensor, page_table: torch.Tensor, block_mask: BlockMask, KV_LEN: int,
                           score: Optional[ScoreRule] = None, scale: Optional[float] = None, chunk_blocks: int = 0,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                           out_dtype=torch.bfloat16):
    """fa_flex_forward_paged_fp8: q [B,Hq,Q_LEN,d] over float8_e4m3fn pages [P,Hkv,page,d] with scales fp32 [P,Hkv,page/32];
    the page size is independent of the mask's Bk. chunk_blocks: key blocks per chunk of a long row (0: chosen, -1: rows
    are not cut). A batch may be padded in front (rows at negative positions see nothing) or behind (those rows see slots that
    nobody wrote, which must hold no NaN bytes; the other rows are right)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, Q_LEN, d]")
    B, Hq, Q_LEN, d = q.shape
    _same(status, (1,), torch.int32, q.device, "status")
    size = _scratch(workspace, q.device)
    P, Hkv, page, max_pages, dev = _check_fp8_cache(q, k_pages, v_pages, k_scale, v_scale, page_table, B, d)
    out, lse = _outputs((B, Hq, Q_LEN, d), dev, out, lse, out_dtype)
    if workspace is None:
        size = max(forward_paged_fp8_workspace_bytes(block_mask, B, Hq, Hkv, d, chunk_blocks, score), 256)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(_call(dev, load().fa_flex_forward_paged_fp8, _at(q), _at(k_pages), _at(v_pages), _at(k_scale),
                 _at(v_scale), _at(page_table), P, page, max_pages, ctypes.byref(block_mask.c), _ref(score),
                 float(scale) if scale else 0.0, _at(out), _out_code(out), _at(lse), B, Hq, Hkv, Q_LEN, KV_LEN, d,
                 chunk_blocks, _at(workspace), size, _at(status)), "fa_flex_forward_paged_fp8")
    return out, lse


def check_status(status: torch.Tensor) -> int:
    return int(load().fa_check_status(_ptr(status), _stream(status.device)))


def set_wait_timeout_ns(ns: int) -> None:
    load().fa_set_wait_timeout_ns(int(ns))


def get_wait_timeout_ns() -> int:
    return int(load().fa_get_wait_timeout_ns())


def debug_wait_timeout(status: torch.Tensor, timeout_ns: int) -> int:
    return int(load().fa_debug_wait_timeout(_ptr(status), int(timeout_ns), _stream(status.device)))


def debug_softcap(x: torch.Tensor, c: float) -> torch.Tensor:
    """c * tanh(x / c) as the kernels compute it, for a contiguous fp32 CUDA tensor."""
    y = torch.empty_like(x)
    _check(load().fa_debug_softcap(_ptr(x), _ptr(y), x.numel(), float(c), _stream(x.device)), "fa_debug_softcap")
    return y


def debug_tc5_gemm(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, K: int, b_mn_major: bool, use_tma: bool,
                   status: Optional[torch.Tensor] = None) -> int:
    return int(load().fa_debug_tc5_gemm(_ptr(A), _ptr(B), _ptr(C), K, int(b_mn_major), int(use_tma), _ptr(status),
                                        _stream(A.device)))
