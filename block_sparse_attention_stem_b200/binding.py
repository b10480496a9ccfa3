"""ctypes binding of ``libstem.so`` (the C ABI declared in include/stem.h).

Argument marshalling only: every step of the path runs inside the CUDA
library.  PyTorch supplies device memory and the current stream.  If the
shared library is missing, importing this module raises; there is no fallback.

Entry points mirror the C names: ``stem_plan``, ``stem_score``,
``stem_select``, ``stem_bsa_fwd``, ``stem_prefill``, for the paged cache
``stem_cache_extend``, ``stem_rope`` and ``stem_tree_attn``, and
``stem_read_device_status``, ``stem_status_string``.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libstem.so")

STEM_OK = 0
STATUS_NAMES = {0: "STEM_OK", 1: "STEM_ERR_INVALID_ARG", 2: "STEM_ERR_UNSUPPORTED",
                3: "STEM_ERR_WORKSPACE_TOO_SMALL", 4: "STEM_ERR_MISALIGNED", 5: "STEM_ERR_CUDA",
                6: "STEM_ERR_TIMEOUT", 7: "STEM_ERR_BAD_BLOCKLIST", 8: "STEM_ERR_BAD_INPUT",
                9: "STEM_ERR_OUT_OF_PAGES"}
STEM_BF16, STEM_FP8_E4M3 = 0, 1
FP8_DTYPES = (torch.uint8, torch.float8_e4m3fn)
EXPORTED = ("stem_plan", "stem_score", "stem_select", "stem_score_select", "stem_bsa_fwd", "stem_bsa_fwd_paged",
            "stem_prefill",
            "stem_prefill_host",
            "stem_prefill_noalloc", "stem_noalloc_read_device_status",
            "stem_cache_extend", "stem_rope", "stem_tree_plan", "stem_tree_attn",
            "stem_selftest_wait_timeout", "stem_read_device_status", "stem_status_string", "stem_version")


class StemParams(ctypes.Structure):
    _fields_ = [("block_size", ctypes.c_int32), ("stride", ctypes.c_int32), ("chunk_size", ctypes.c_int32),
                ("norm", ctypes.c_double), ("beta", ctypes.c_double), ("keep_ratio", ctypes.c_double),
                ("mu", ctypes.c_double), ("sink_blocks", ctypes.c_int32), ("window_blocks", ctypes.c_int32),
                ("softmax_scale", ctypes.c_double), ("budget_mode", ctypes.c_int32), ("bonus_mode", ctypes.c_int32),
                ("list_mode", ctypes.c_int32), ("select_mode", ctypes.c_int32)]


class StemQKV(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int32)),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_scale", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class StemPagedKV(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p)]


class StemCacheStep(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32), ("num_free", ctypes.c_int32),
                ("mask_words", ctypes.c_int32), ("cache_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
                ("held_pages", ctypes.c_void_p), ("free_pages", ctypes.c_void_p), ("cursor", ctypes.c_void_p),
                ("parents", ctypes.c_void_p)]


class StemRope(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_len", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("amplitude", ctypes.c_double)]


class StemRopeIO(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("positions", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_scale", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p)]


class StemTree(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("max_seq_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("mask_words", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p),
                ("kv_lens", ctypes.c_void_p), ("mask", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("q_scale", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("softmax_scale", ctypes.c_double)]


class StemPlan(ctypes.Structure):
    _fields_ = [("nb_total", ctypes.c_int64), ("nb_max", ctypes.c_int64), ("num_rows", ctypes.c_int64),
                ("nnz", ctypes.c_int64), ("nnz_per_head", ctypes.c_int64), ("scores_bytes", ctypes.c_size_t),
                ("vbonus_bytes", ctypes.c_size_t), ("ws_bytes", ctypes.c_size_t),
                ("ws_prefill_bytes", ctypes.c_size_t), ("attn_flops", ctypes.c_double),
                ("dense_attn_flops", ctypes.c_double), ("score_flops", ctypes.c_double),
                ("vwide_bytes", ctypes.c_size_t)]


class StemError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({stem_status_string(code)})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with `python -m block_sparse_attention_stem_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER
    lib.stem_plan.argtypes = [P(StemQKV), P(StemParams), P(StemPlan)]
    lib.stem_score.argtypes = [P(StemQKV), P(StemParams), vp, vp, vp, sz, vp]
    lib.stem_select.argtypes = [P(StemQKV), P(StemParams), vp, vp, vp, vp, vp, sz, vp]
    lib.stem_score_select.argtypes = [P(StemQKV), P(StemParams), vp, vp, vp, vp, vp, vp, sz, vp]
    lib.stem_bsa_fwd.argtypes = [P(StemQKV), P(StemParams), vp, vp, vp, vp, vp, sz, vp]
    lib.stem_bsa_fwd_paged.argtypes = [P(StemQKV), P(StemPagedKV), P(StemParams), vp, vp, vp, vp, vp, sz, vp]
    lib.stem_prefill.argtypes = [P(StemQKV), P(StemParams), vp, vp, vp, vp, vp, sz, vp]
    lib.stem_prefill_noalloc.argtypes = [P(StemQKV), P(StemParams), vp, vp, vp, vp, vp]
    lib.stem_noalloc_read_device_status.argtypes = [vp, P(ctypes.c_int)]
    lib.stem_prefill_host.argtypes = [P(StemQKV), P(StemParams), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.stem_cache_extend.argtypes = [P(StemCacheStep)] + [vp] * 9 + [sz, vp]
    lib.stem_rope.argtypes = [P(StemRope), P(StemRopeIO), P(StemPagedKV), vp]
    lib.stem_tree_plan.argtypes = [P(StemTree), P(sz)]
    lib.stem_tree_attn.argtypes = [P(StemTree), P(StemPagedKV), vp, vp, vp, sz, vp]
    lib.stem_selftest_wait_timeout.argtypes = [vp, vp]
    lib.stem_read_device_status.argtypes = [vp, vp, P(ctypes.c_int)]
    lib.stem_status_string.argtypes = [ctypes.c_int]
    lib.stem_status_string.restype = ctypes.c_char_p
    lib.stem_version.restype = ctypes.c_int32
    for name in ("stem_plan", "stem_score", "stem_select", "stem_bsa_fwd", "stem_prefill",
                 "stem_prefill_noalloc", "stem_noalloc_read_device_status", "stem_selftest_wait_timeout",
                 "stem_cache_extend", "stem_rope", "stem_tree_plan", "stem_tree_attn", "stem_read_device_status"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


LIB = _load()


def stem_status_string(code: int) -> str:
    return LIB.stem_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != STEM_OK:
        raise StemError(code, where)


def make_params(block_size=128, stride=8, chunk_size=2048, norm=1.0, beta=0.2, keep_ratio=0.25, mu=0.7,
                sink_blocks=4, window_blocks=4, softmax_scale=0.0, budget_mode=0, bonus_mode=0,
                list_mode=0, select_mode=0) -> StemParams:
    return StemParams(block_size, stride, chunk_size, float(norm), float(beta), float(keep_ratio), float(mu),
                      sink_blocks, window_blocks, float(softmax_scale), budget_mode, bonus_mode, list_mode,
                      select_mode)


def _ptr(t):
    return None if t is None else t.data_ptr()


@dataclass
class QKV:
    """Tensors of one call plus the ctypes descriptor that points at them.
    Keeps references so the memory stays alive while the descriptor is used."""
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    cu_dev: torch.Tensor
    cu_host: torch.Tensor
    q_scale: torch.Tensor | None
    k_scale: torch.Tensor | None
    v_scale: torch.Tensor | None
    desc: StemQKV

    @property
    def total_tokens(self) -> int:
        return int(self.cu_host[-1])


def make_qkv(q, k, v, cu_seqlens, q_scale=None, k_scale=None, v_scale=None, cu_seqlens_dev=None) -> QKV:
    """q [T,Hq,128], k/v [T,Hkv,128]: bf16, or uint8 / float8_e4m3fn bytes with
    fp32 per-head scales.  cu_seqlens: host int32 offsets (list or tensor)."""
    cu_host = torch.as_tensor(cu_seqlens, dtype=torch.int32).cpu().contiguous()
    if cu_seqlens_dev is None:
        cu_seqlens_dev = cu_host.to(q.device)
    if q.dtype == torch.bfloat16:
        dtype = STEM_BF16
    elif q.dtype in (torch.uint8, torch.float8_e4m3fn):
        dtype = STEM_FP8_E4M3
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k and v must be contiguous [T, H, d]")
    desc = StemQKV(dtype, cu_host.numel() - 1, int(cu_host[-1]), _ptr(cu_seqlens_dev),
                   ctypes.cast(cu_host.data_ptr(), ctypes.POINTER(ctypes.c_int32)),
                   q.shape[1], k.shape[1], q.shape[2], _ptr(q), _ptr(k), _ptr(v),
                   _ptr(q_scale), _ptr(k_scale), _ptr(v_scale))
    return QKV(q, k, v, cu_seqlens_dev, cu_host, q_scale, k_scale, v_scale, desc)


def stem_plan(qkv: QKV, params: StemParams) -> StemPlan:
    out = StemPlan()
    _check(LIB.stem_plan(ctypes.byref(qkv.desc), ctypes.byref(params), ctypes.byref(out)), "stem_plan")
    return out


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _elsewhere(stream, device, fn, *args):
    """fn(*args) with `stream` current, as every call with stream= runs.  What it
    makes then belongs to that stream: the allocator does not hand it to work on
    another one, and does not take it from work that another one still has to do.
    Results may be used on the caller's current stream too."""
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        made = fn(*args)
    if here != stream:
        for t in made if isinstance(made, tuple) else vars(made).values():
            if t is not None:
                t.record_stream(here)
    return made


def _ws(nbytes: int, device, ws):
    if ws is None:
        ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    return ws


def stem_score(qkv: QKV, params: StemParams, scores=None, vbonus=None, ws=None, stream=None):
    if stream is not None:
        return _elsewhere(stream, qkv.q.device, stem_score, qkv, params, scores, vbonus, ws)
    pl = stem_plan(qkv, params)
    dev = qkv.q.device
    hq, hkv = qkv.q.shape[1], qkv.k.shape[1]
    if scores is None:
        scores = torch.empty(hq, pl.nb_total, pl.nb_max, dtype=torch.float32, device=dev)
    if vbonus is None:
        vbonus = torch.empty(hkv, pl.nb_total, dtype=torch.float32, device=dev)
    ws = _ws(pl.ws_bytes, dev, ws)
    _check(LIB.stem_score(ctypes.byref(qkv.desc), ctypes.byref(params), _ptr(scores), _ptr(vbonus),
                          _ptr(ws), ws.numel(), _stream(None)), "stem_score")
    return scores, vbonus, ws


def stem_select(qkv: QKV, params: StemParams, scores, budgets=None, row_ptr=None, col_idx=None, ws=None,
                stream=None):
    if stream is not None:
        return _elsewhere(stream, scores.device, stem_select, qkv, params, scores, budgets, row_ptr, col_idx, ws)
    pl = stem_plan(qkv, params)
    dev = scores.device
    if budgets is None:
        budgets = torch.empty(pl.num_rows, dtype=torch.int32, device=dev)
    if row_ptr is None:
        row_ptr = torch.empty(pl.num_rows + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        col_idx = torch.empty(max(pl.nnz, 1), dtype=torch.int32, device=dev)
    ws = _ws(pl.ws_bytes, dev, ws)
    _check(LIB.stem_select(ctypes.byref(qkv.desc), ctypes.byref(params), _ptr(scores), _ptr(budgets),
                           _ptr(row_ptr), _ptr(col_idx), _ptr(ws), ws.numel(), _stream(None)), "stem_select")
    return budgets, row_ptr, col_idx[:pl.nnz], ws


def stem_score_select(qkv: QKV, params: StemParams, scores=None, vbonus=None, budgets=None, row_ptr=None,
                      col_idx=None, ws=None, stream=None):
    """stem_score then stem_select in one call (in one pass when params.select_mode is 1)."""
    if stream is not None:
        return _elsewhere(stream, qkv.q.device, stem_score_select, qkv, params, scores, vbonus, budgets, row_ptr, col_idx, ws)
    pl = stem_plan(qkv, params)
    dev = qkv.q.device
    hq, hkv = qkv.q.shape[1], qkv.k.shape[1]
    if scores is None:
        scores = torch.empty(hq, pl.nb_total, pl.nb_max, dtype=torch.float32, device=dev)
    if budgets is None:
        budgets = torch.empty(pl.num_rows, dtype=torch.int32, device=dev)
    if row_ptr is None:
        row_ptr = torch.empty(pl.num_rows + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        col_idx = torch.empty(max(pl.nnz, 1), dtype=torch.int32, device=dev)
    ws = _ws(pl.ws_bytes, dev, ws)
    _check(LIB.stem_score_select(ctypes.byref(qkv.desc), ctypes.byref(params), _ptr(scores), _ptr(vbonus),
                                 _ptr(budgets), _ptr(row_ptr), _ptr(col_idx), _ptr(ws), ws.numel(),
                                 _stream(None)), "stem_score_select")
    return scores, budgets, row_ptr, col_idx[:pl.nnz], ws


@dataclass
class PagedKV:
    """A paged K/V pool and the descriptor that points at it; keeps the
    tensors alive while the descriptor is used."""
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    page_table: torch.Tensor
    desc: StemPagedKV

    def __post_init__(self):
        # (device, e4m3, KV heads, head dim) of the pages; None when the two differ or are not contiguous
        k, v = self.k_pages, self.v_pages
        fp8 = k.dtype in FP8_DTYPES
        same = (k.dtype == v.dtype and k.shape == v.shape and k.device == v.device == self.page_table.device
                and k.dim() == 4 and k.is_contiguous() and v.is_contiguous() and (fp8 or k.dtype == torch.bfloat16))
        self.kind = (k.device, fp8, k.shape[2], k.shape[3]) if same else None


def paged_kv(k_pages, v_pages, page_table, page_size: int) -> PagedKV:
    """k_pages/v_pages [P, page_size, Hkv, d] device tensors, page_table int32
    [num_seqs, max_pages] on the device."""
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 [num_seqs, max_pages] tensor")
    if k_pages.shape != v_pages.shape or k_pages.shape[1] != page_size:
        raise ValueError("k_pages and v_pages must both be [P, page_size, Hkv, d]")
    desc = StemPagedKV(page_size, k_pages.shape[0], page_table.shape[1], _ptr(page_table), _ptr(k_pages),
                       _ptr(v_pages))
    return PagedKV(k_pages, v_pages, page_table, desc)


def stem_bsa_fwd_paged(qkv: QKV, kv: PagedKV, params: StemParams, row_ptr, col_idx, out=None, lse=None,
                       ws=None, stream=None):
    if stream is not None:
        return _elsewhere(stream, qkv.q.device, stem_bsa_fwd_paged, qkv, kv, params, row_ptr, col_idx, out, lse, ws)
    pl = stem_plan(qkv, params)
    dev = qkv.q.device
    T, hq = qkv.total_tokens, qkv.q.shape[1]
    if out is None:
        out = torch.empty(T, hq, 128, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(hq, T, dtype=torch.float32, device=dev)
    ws = _ws(pl.ws_bytes, dev, ws)
    _check(LIB.stem_bsa_fwd_paged(ctypes.byref(qkv.desc), ctypes.byref(kv.desc), ctypes.byref(params), _ptr(row_ptr),
                                  _ptr(col_idx), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(None)),
           "stem_bsa_fwd_paged")
    return out, lse, ws


def stem_bsa_fwd(qkv: QKV, params: StemParams, row_ptr, col_idx, out=None, lse=None, ws=None, stream=None):
    if stream is not None:
        return _elsewhere(stream, qkv.q.device, stem_bsa_fwd, qkv, params, row_ptr, col_idx, out, lse, ws)
    pl = stem_plan(qkv, params)
    dev = qkv.q.device
    T, hq = qkv.total_tokens, qkv.q.shape[1]
    if out is None:
        out = torch.empty(T, hq, 128, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(hq, T, dtype=torch.float32, device=dev)
    ws = _ws(pl.ws_bytes, dev, ws)
    _check(LIB.stem_bsa_fwd(ctypes.byref(qkv.desc), ctypes.byref(params), _ptr(row_ptr), _ptr(col_idx),
                            _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(None)), "stem_bsa_fwd")
    return out, lse, ws


def stem_prefill(qkv: QKV, params: StemParams, out=None, lse=None, row_ptr=None, col_idx=None, ws=None,
                 stream=None, return_lists=True):
    if stream is not None:
        return _elsewhere(stream, qkv.q.device, stem_prefill, qkv, params, out, lse, row_ptr, col_idx, ws, None, return_lists)
    pl = stem_plan(qkv, params)
    dev = qkv.q.device
    T, hq = qkv.total_tokens, qkv.q.shape[1]
    if out is None:
        out = torch.empty(T, hq, 128, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(hq, T, dtype=torch.float32, device=dev)
    if return_lists and row_ptr is None:
        row_ptr = torch.empty(pl.num_rows + 1, dtype=torch.int32, device=dev)
    if return_lists and col_idx is None:
        col_idx = torch.empty(max(pl.nnz, 1), dtype=torch.int32, device=dev)
    ws = _ws(pl.ws_prefill_bytes, dev, ws)
    _check(LIB.stem_prefill(ctypes.byref(qkv.desc), ctypes.byref(params), _ptr(out), _ptr(lse), _ptr(row_ptr),
                            _ptr(col_idx), _ptr(ws), ws.numel(), _stream(None)), "stem_prefill")
    return out, lse, row_ptr, (None if col_idx is None else col_idx[:pl.nnz]), ws


def stem_prefill_host(qkv: QKV, params: StemParams, q_host, k_host, v_host, out_host, lse_host, out=None, lse=None,
                      ws=None, stream=None):
    """stem_prefill with inputs and outputs in (page-locked) host tensors; the
    device tensors of `qkv` are filled by the call, transfers overlap compute.
    Only enqueues: synchronize `stream` before reading out_host / lse_host."""
    if stream is not None:
        return _elsewhere(stream, qkv.q.device, stem_prefill_host, qkv, params, q_host, k_host, v_host, out_host, lse_host,
                          out, lse, ws)
    pl = stem_plan(qkv, params)
    dev = qkv.q.device
    T, hq = qkv.total_tokens, qkv.q.shape[1]
    for name, t, like in (("q_host", q_host, qkv.q), ("k_host", k_host, qkv.k), ("v_host", v_host, qkv.v)):
        if t.device.type != "cpu" or t.shape != like.shape or t.dtype != like.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor shaped like the device one")
    if out_host.device.type != "cpu" or tuple(out_host.shape) != (T, hq, 128) or out_host.dtype != torch.bfloat16:
        raise ValueError("out_host must be a host bf16 tensor [T, Hq, 128]")
    if lse_host.device.type != "cpu" or tuple(lse_host.shape) != (hq, T) or lse_host.dtype != torch.float32:
        raise ValueError("lse_host must be a host fp32 tensor [Hq, T]")
    if out is None:
        out = torch.empty(T, hq, 128, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(hq, T, dtype=torch.float32, device=dev)
    ws = _ws(pl.ws_prefill_bytes, dev, ws)
    _check(LIB.stem_prefill_host(ctypes.byref(qkv.desc), ctypes.byref(params), _ptr(q_host), _ptr(k_host),
                                 _ptr(v_host), _ptr(out), _ptr(lse), _ptr(out_host), _ptr(lse_host), _ptr(ws),
                                 ws.numel(), _stream(None)), "stem_prefill_host")
    return out, lse, ws


def stem_prefill_noalloc(qkv: QKV, params: StemParams, out=None, lse=None, row_ptr=None, col_idx=None,
                         stream=None, return_lists=True):
    """stem_prefill on the library's built-in 32 MiB workspace (for callers that
    cannot allocate one); the outputs are still the caller's."""
    if stream is not None:
        return _elsewhere(stream, qkv.q.device, stem_prefill_noalloc, qkv, params, out, lse, row_ptr, col_idx, None, return_lists)
    pl = stem_plan(qkv, params)
    dev = qkv.q.device
    T, hq = qkv.total_tokens, qkv.q.shape[1]
    if out is None:
        out = torch.empty(T, hq, 128, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(hq, T, dtype=torch.float32, device=dev)
    if return_lists and row_ptr is None:
        row_ptr = torch.empty(pl.num_rows + 1, dtype=torch.int32, device=dev)
    if return_lists and col_idx is None:
        col_idx = torch.empty(max(pl.nnz, 1), dtype=torch.int32, device=dev)
    _check(LIB.stem_prefill_noalloc(ctypes.byref(qkv.desc), ctypes.byref(params), _ptr(out), _ptr(lse),
                                    _ptr(row_ptr), _ptr(col_idx), _stream(None)), "stem_prefill_noalloc")
    return out, lse, row_ptr, (None if col_idx is None else col_idx[:pl.nnz])


def stem_noalloc_read_device_status(stream=None) -> int:
    """Status word of stem_prefill_noalloc's built-in workspace on the current
    device (synchronises the stream)."""
    out = ctypes.c_int(0)
    _check(LIB.stem_noalloc_read_device_status(_stream(stream), ctypes.byref(out)),
           "stem_noalloc_read_device_status")
    return out.value


# ------------------------------------------------------------------ the paged cache
# These run once per layer and token: the checks are kept to a few comparisons
# of attributes, and nothing is looked up that the descriptors already hold.
def _run(device, where, fn, *args):
    """fn(*args, current stream of the tensors' device) with that device current."""
    if device.type != "cuda":
        raise ValueError(f"{where}: the tensors must be on a GPU, not on {device}")
    on = torch._C._cuda_getCurrentRawStream(device.index)
    if torch._C._cuda_getDevice() == device.index:
        code = fn(*args, on)
    else:
        with torch.cuda.device(device):
            code = fn(*args, on)
    if code != STEM_OK:
        raise StemError(code, where)


def _need(name, t, dtype, shape, device):
    """A contiguous tensor of the documented type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _need_ws(ws, device):
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {device}, got strides {ws.stride()} on {ws.device}")


@dataclass
class CacheStep:
    """Outputs of stem_cache_extend (int32; the mask's words as int32 bit patterns)."""
    held: torch.Tensor        # [S] pages held now
    cursor: torch.Tensor      # [1] position in the free list
    cu_seqlens: torch.Tensor  # [S + 1]
    kv_lens: torch.Tensor     # [S]
    slots: torch.Tensor       # [max_tokens]
    positions: torch.Tensor   # [max_tokens]
    mask: torch.Tensor | None  # [max_tokens, mask_words]
    ws: torch.Tensor


def stem_cache_extend(page_table, page_size: int, num_pages: int, cache_lens, new_lens, held_pages, free_pages, cursor,
                      max_tokens: int, parents=None, mask_words: int = 0, out: CacheStep | None = None, ws=None,
                      stream=None) -> CacheStep:
    """Extends `page_table` [S, max_pages] in place by the pages that the step's
    tokens need and returns the step's maps.  All tensors are int32 on the
    device.  `out`: the buffers to write (its held, cursor and kv_lens may be
    the input tensors, so that a captured step advances its own state).
    Out-of-range values and an exhausted free list are reported in the
    workspace's status word."""
    dev = page_table.device
    if stream is not None:
        return _elsewhere(stream, dev, stem_cache_extend, page_table, page_size, num_pages, cache_lens, new_lens, held_pages,
                          free_pages, cursor, max_tokens, parents, mask_words, out, ws)
    i32 = torch.int32
    if page_table.dim() != 2:
        raise ValueError("page_table must be [num_seqs, max_pages]")
    _need("page_table", page_table, i32, page_table.shape, dev)
    S = page_table.shape[0]
    per_seq = (S,)
    _need("cache_lens", cache_lens, i32, per_seq, dev)
    _need("new_lens", new_lens, i32, per_seq, dev)
    _need("held_pages", held_pages, i32, per_seq, dev)
    _need("free_pages", free_pages, i32, (free_pages.numel(),), dev)
    _need("cursor", cursor, i32, (1,), dev)
    tree = parents is not None
    if tree:
        _need("parents", parents, i32, (max_tokens,), dev)
    words = mask_words if tree else 0
    if out is None:
        if max_tokens < 0 or words < 0:
            raise ValueError("max_tokens and mask_words must not be negative")
        sizes = (S, 1, S + 1, S, max_tokens, max_tokens, max_tokens * words)  # one allocation
        parts = torch.empty(sum(sizes), dtype=i32, device=dev).split_with_sizes(sizes)
        out = CacheStep(*parts[:6], parts[6].view(max_tokens, words) if tree else None, None)
    else:
        for name, t, shape in (("held", out.held, per_seq), ("cursor", out.cursor, (1,)),
                               ("cu_seqlens", out.cu_seqlens, (S + 1,)), ("kv_lens", out.kv_lens, per_seq),
                               ("slots", out.slots, (max_tokens,)), ("positions", out.positions, (max_tokens,))):
            _need("out." + name, t, i32, shape, dev)
        if tree:
            if out.mask is None:
                raise ValueError("out.mask is needed with parents")
            _need("out.mask", out.mask, i32, (max_tokens, words), dev)
    if ws is None:
        ws = out.ws if out.ws is not None else _ws(256, dev, None)
    _need_ws(ws, dev)
    out.ws = ws
    desc = StemCacheStep(S, max_tokens, page_size, num_pages, page_table.shape[1], free_pages.shape[0], words,
                         cache_lens.data_ptr(), new_lens.data_ptr(), held_pages.data_ptr(), free_pages.data_ptr(),
                         cursor.data_ptr(), parents.data_ptr() if tree else None)
    _run(dev, "stem_cache_extend", LIB.stem_cache_extend, ctypes.byref(desc), page_table.data_ptr(),
         out.held.data_ptr(), out.cursor.data_ptr(), out.cu_seqlens.data_ptr(), out.kv_lens.data_ptr(),
         out.slots.data_ptr(), out.positions.data_ptr(), out.mask.data_ptr() if tree else None, ws.data_ptr(), ws.nbytes)
    return out


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


def make_rope(rotary_dim=128, layout="half", base=1e6, scaling="plain", factor=1.0, original_len=1, beta_fast=32.0,
              beta_slow=1.0, amplitude=0.0) -> StemRope:
    """layout: a name of ROPE_LAYOUTS; scaling: one of ROPE_SCALINGS."""
    return StemRope(ROPE_LAYOUTS[layout], rotary_dim, ROPE_SCALINGS[scaling], original_len, float(base), float(factor),
                    float(beta_fast), float(beta_slow), float(amplitude))


def _token_rows(name, t, T, device):
    """(heads, head dim, stride between tokens) of a bf16 [T, H, d] tensor whose heads are contiguous."""
    shape, strides = t.shape, t.stride()
    if t.dtype is not torch.bfloat16 or len(shape) != 3 or shape[0] != T:
        raise ValueError(f"{name} must be a bf16 [{T}, H, d] tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors are on {device}")
    _, H, d = shape
    if strides[2] != 1 or (H > 1 and strides[1] != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return H, d, strides[0] if T > 1 else H * d


def stem_rope(rope: StemRope, q, k, v, positions, cache: PagedKV | None = None, slots=None, q_scale=None, k_scale=None,
              v_scale=None, q_out=None, k_out=None, v_out=None, fp8: bool | None = None, stream=None):
    """Rotates q [T, Hq, 128] and k [T, Hkv, 128] (bf16; slices of a fused
    projection are fine) and stores k and v in the cache's pages at `slots`.
    Returns (q_out, k_out, v_out): q_out is made when not given (unless q is
    None), k_out and v_out are made only without a cache.  Outputs are bf16, or
    e4m3 bytes (uint8) when the scales, fp32 [H], are given (or `fp8` says so).
    v may be None without a cache; so may q or k."""
    dev = positions.device
    if stream is not None:
        return _elsewhere(stream, dev, stem_rope, rope, q, k, v, positions, cache, slots, q_scale, k_scale, v_scale, q_out,
                          k_out, v_out, fp8)
    T = positions.shape[0] if positions.dim() else 1
    _need("positions", positions, torch.int32, (T,), dev)
    if fp8 is None:
        fp8 = q_scale is not None or k_scale is not None or v_scale is not None
    hq = hkv = sq = sk = sv = 0
    d = None
    pq = pk = pv = pqo = pko = pvo = pslots = None
    if q is not None:
        hq, d, sq = _token_rows("q", q, T, dev)
        pq = q.data_ptr()
    if k is not None:
        hkv, dk, sk = _token_rows("k", k, T, dev)
        pk = k.data_ptr()
        if d is None:
            d = dk
        elif d != dk:
            raise ValueError("q and k must have the same head dimension")
    if v is not None:
        hv, dv, sv = _token_rows("v", v, T, dev)
        pv = v.data_ptr()
        if (k is not None and hv != hkv) or (d is not None and dv != d):
            raise ValueError("k and v must have the same heads, q, k and v the same head dimension")
        hkv, d = hv, dv
    made = torch.uint8 if fp8 else torch.bfloat16
    pcache = None
    if cache is not None:
        if slots is None or k is None or v is None:
            raise ValueError("a cache needs k, v and slots")
        _need("slots", slots, torch.int32, (T,), dev)
        pslots = slots.data_ptr()
        if cache.kind != (dev, fp8, hkv, d):
            raise ValueError(f"the pages must be contiguous [P, page_size, {hkv}, {d}] on {dev} in "
                             f"{'e4m3' if fp8 else 'bf16'}, got (device, e4m3, heads, dim) {cache.kind}")
        pcache = ctypes.byref(cache.desc)
    else:
        k_out = torch.empty((T, hkv, d), dtype=made, device=dev) if k_out is None and k is not None else k_out
        v_out = torch.empty((T, hkv, d), dtype=made, device=dev) if v_out is None and v is not None else v_out
    if q_out is None:
        if q is not None:
            q_out = torch.empty((T, hq, d), dtype=made, device=dev)
            pqo = q_out.data_ptr()
    else:
        _need("q_out", q_out, q_out.dtype if fp8 and q_out.dtype in FP8_DTYPES else made, (T, hq, d), dev)
        pqo = q_out.data_ptr()
    if k_out is not None:
        _need("k_out", k_out, k_out.dtype if fp8 and k_out.dtype in FP8_DTYPES else made, (T, hkv, d), dev)
        pko = k_out.data_ptr()
    if v_out is not None:
        _need("v_out", v_out, v_out.dtype if fp8 and v_out.dtype in FP8_DTYPES else made, (T, hkv, d), dev)
        pvo = v_out.data_ptr()
    pqs = pks = pvs = None
    if fp8:
        if q_scale is not None:
            _need("q_scale", q_scale, torch.float32, (hq,), dev)
            pqs = q_scale.data_ptr()
        if k_scale is not None:
            _need("k_scale", k_scale, torch.float32, (hkv,), dev)
            pks = k_scale.data_ptr()
        if v_scale is not None:
            _need("v_scale", v_scale, torch.float32, (hkv,), dev)
            pvs = v_scale.data_ptr()
    elif q_scale is not None or k_scale is not None or v_scale is not None:
        raise ValueError("scales are for e4m3 outputs")
    io = StemRopeIO(T, hq, hkv, 128 if d is None else d, STEM_FP8_E4M3 if fp8 else STEM_BF16, positions.data_ptr(),
                    pslots, pq, pk, pv, sq, sk, sv, pqs, pks, pvs, pqo, pko, pvo)
    _run(dev, "stem_rope", LIB.stem_rope, ctypes.byref(rope), ctypes.byref(io), pcache)
    return q_out, k_out, v_out


@dataclass
class TreeQ:
    """The queries of one step and the descriptor that points at them; keeps
    the tensors alive while the descriptor is used."""
    q: torch.Tensor
    cu_seqlens: torch.Tensor
    kv_lens: torch.Tensor
    mask: torch.Tensor | None
    q_scale: torch.Tensor | None
    k_scale: torch.Tensor | None
    v_scale: torch.Tensor | None
    desc: StemTree

    def __post_init__(self):
        # (device, e4m3, KV heads, head dim): what the pages have to be
        self.kind = (self.q.device, self.desc.dtype == STEM_FP8_E4M3, self.desc.num_kv_heads, self.desc.head_dim)


def make_tree(q, cu_seqlens, kv_lens, num_kv_heads: int, mask=None, max_seq_tokens: int = 0, q_scale=None, k_scale=None,
              v_scale=None, softmax_scale: float = 0.0) -> TreeQ:
    """q [T, Hq, 128] bf16, or e4m3 bytes with fp32 per-head scales; cu_seqlens
    [S + 1], kv_lens [S] and mask [T, words] int32 on q's device.  Give
    max_seq_tokens (the most queries of one sequence) where it is known: with 0
    the launch is sized for T of them."""
    dev = q.device
    fp8 = q.dtype in FP8_DTYPES
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, d]")
    _need("q", q, q.dtype if fp8 else torch.bfloat16, q.shape, dev)
    S = kv_lens.numel()
    _need("kv_lens", kv_lens, torch.int32, (S,), dev)
    _need("cu_seqlens", cu_seqlens, torch.int32, (S + 1,), dev)
    if mask is not None:
        _need("mask", mask, torch.int32, (q.shape[0], mask.shape[-1]), dev)
    if fp8:
        for name, t, h in (("q_scale", q_scale, q.shape[1]), ("k_scale", k_scale, num_kv_heads),
                           ("v_scale", v_scale, num_kv_heads)):
            if t is None:
                raise ValueError(f"{name} is needed with e4m3 inputs")
            _need(name, t, torch.float32, (h,), dev)
    desc = StemTree(STEM_FP8_E4M3 if fp8 else STEM_BF16, S, q.shape[0], max_seq_tokens, q.shape[1], num_kv_heads,
                    q.shape[2], 0 if mask is None else mask.shape[1], _ptr(cu_seqlens), _ptr(kv_lens), _ptr(mask),
                    _ptr(q), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), float(softmax_scale))
    return TreeQ(q, cu_seqlens, kv_lens, mask, q_scale, k_scale, v_scale, desc)


def stem_tree_ws_bytes(tree: TreeQ) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.stem_tree_plan(ctypes.byref(tree.desc), ctypes.byref(out)), "stem_tree_plan")
    return out.value


def stem_tree_attn(tree: TreeQ, kv: PagedKV, out=None, lse=None, ws=None, stream=None):
    """Attention of a step's queries over the paged cache: out bf16 [T, Hq, 128],
    lse fp32 [Hq, T], and the workspace (whose status word tells of bad lengths)."""
    q = tree.q
    if stream is not None:
        return _elsewhere(stream, q.device, stem_tree_attn, tree, kv, out, lse, ws)
    desc = tree.desc
    T, hq, d = q.shape
    if kv.kind != tree.kind:
        raise ValueError(f"the pages must be contiguous and of the queries' kind: (device, e4m3, KV heads, head dim) "
                         f"{tree.kind}, got {kv.kind}")
    if kv.page_table.shape[0] < tree.kv_lens.shape[0]:
        raise ValueError("page_table must have a row per sequence")
    dev = tree.kind[0]
    if out is None:
        out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _need("out", out, torch.bfloat16, (T, hq, d), dev)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=dev)
    else:
        _need("lse", lse, torch.float32, (hq, T), dev)
    if ws is None:
        ws = _ws(stem_tree_ws_bytes(tree), dev, None)
    else:
        _need_ws(ws, dev)
    _run(dev, "stem_tree_attn", LIB.stem_tree_attn, ctypes.byref(desc), ctypes.byref(kv.desc), out.data_ptr(),
         lse.data_ptr(), ws.data_ptr(), ws.nbytes)
    return out, lse, ws


def stem_selftest_wait_timeout(ws, stream=None):
    """Run the bounded-wait self-test; read the result with stem_read_device_status."""
    _check(LIB.stem_selftest_wait_timeout(_ptr(ws), _stream(stream)), "stem_selftest_wait_timeout")


def stem_read_device_status(ws, stream=None) -> int:
    out = ctypes.c_int(0)
    _check(LIB.stem_read_device_status(_ptr(ws), _stream(stream), ctypes.byref(out)), "stem_read_device_status")
    return out.value
