"""Python binding of the paged-cache entry points: argument marshalling only.

A PagedKV and a PagedBatch check and describe the tensors of a cache and of a
step once; kv_append_paged and paged_attn then pass them on with the step's
rows. The tensors are read on the device by every call, so a program updates
lengths, tables and pages in place and keeps the descriptors.
"""
import ctypes

import torch

from . import _abi
from ._abi import FR_KV_E4M3, FR_KV_F16, FR_ROWS_F16, FR_ROWS_F32, FrError
from .ops import _as_rope, _check_dev

_ROWS = {torch.float32: FR_ROWS_F32, torch.float16: FR_ROWS_F16}
_KV = {torch.float16: FR_KV_F16, torch.float8_e4m3fn: FR_KV_E4M3}


def _stream_of(stream, index):
    """Handle of the stream to launch on: the given one, else the current one of GPU `index`."""
    return _current(index) if stream is None else stream.cuda_stream


# the handle alone, where torch offers it: a Stream object costs a decode call microseconds
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class PagedKV:
    """fr_paged_kv: a paged K/V cache.

    k_pages, v_pages: f16 or float8_e4m3fn [n_pages, n_kv_head, page_size, hd]
    with unit inner stride; the other strides are free (a [n_pages, page_size,
    n_kv_head, hd] pool is passed as its transpose(1, 2)). k_scale, v_scale: f32
    [n_pages, n_kv_head], contiguous, for e4m3 pages (value = scale * code)."""

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None):
        _check_dev(k_pages, v_pages, k_scale, v_scale)
        if k_pages.dtype not in _KV or v_pages.dtype != k_pages.dtype:
            raise TypeError("k_pages and v_pages must both be float16 or both float8_e4m3fn")
        if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
            raise ValueError("k_pages and v_pages must be [n_pages, n_kv_head, page_size, hd]")
        if k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
            raise ValueError("k_pages and v_pages need unit inner stride")
        n_pages, n_kv_head, page_size, hd = k_pages.shape
        e4m3 = k_pages.dtype == torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if (t is not None) != e4m3:
                raise ValueError(f"{name}: scales go with float8_e4m3fn pages, and only with them")
            if t is None:
                continue
            if t.dtype != torch.float32:
                raise TypeError(f"{name} must be float32")
            if tuple(t.shape) != (n_pages, n_kv_head) or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous [n_pages, n_kv_head]")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.n_pages, self.n_kv_head, self.page_size, self.hd = n_pages, n_kv_head, page_size, hd
        self.device = k_pages.device
        self._index = self.device.index
        for t in (v_pages, k_scale, v_scale):
            if t is not None and t.device != self.device:
                raise ValueError("tensors of a cache must be on one GPU")
        self._lib = _abi.load()
        self._desc = _abi.FrPagedKV()
        self._p = ctypes.c_void_p(ctypes.addressof(self._desc))
        st = [(ctypes.c_int64 * 3)(*t.stride()[:3]) for t in (k_pages, v_pages)]
        with torch.cuda.device(self.device):
            _abi.check(self._lib.fr_paged_kv_init(
                self._p, _KV[k_pages.dtype], k_pages.data_ptr(), st[0], v_pages.data_ptr(), st[1],
                k_scale.data_ptr() if e4m3 else None, v_scale.data_ptr() if e4m3 else None, n_pages, page_size,
                n_kv_head, hd), "fr_paged_kv_init")


class PagedBatch:
    """fr_paged_batch: the sequences of a step.

    tok_start: int32 [n_seq + 1], sequence b's new tokens are rows tok_start[b]
    .. tok_start[b+1] - 1 of the step's rows; kv_len: int32 [n_seq], keys of each
    sequence, its new tokens included; page_table: int32 [n_seq, max_pages]
    (row stride free). n_tok, the rows that a step's tensors have, is taken from
    each call's tensors."""

    def __init__(self, tok_start, kv_len, page_table):
        _check_dev(tok_start, kv_len, page_table)
        for name, t in (("tok_start", tok_start), ("kv_len", kv_len), ("page_table", page_table)):
            if t.dtype != torch.int32:
                raise TypeError(f"{name} must be int32")
        if kv_len.dim() != 1 or tok_start.dim() != 1 or tok_start.shape[0] != kv_len.shape[0] + 1:
            raise ValueError("tok_start must be [n_seq + 1] and kv_len [n_seq]")
        if page_table.dim() != 2 or page_table.shape[0] != kv_len.shape[0]:
            raise ValueError("page_table must be [n_seq, max_pages]")
        if not tok_start.is_contiguous() or not kv_len.is_contiguous():
            raise ValueError("tok_start and kv_len must be contiguous")
        if page_table.shape[1] > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table needs unit inner stride")
        if len({t.device for t in (tok_start, kv_len, page_table)}) != 1:
            raise ValueError("tensors of a batch must be on one GPU")
        self.tok_start, self.kv_len, self.page_table = tok_start, kv_len, page_table
        self.device = kv_len.device
        self._by_rows = {}

    def _desc(self, n_tok):
        """The descriptor for steps of n_tok rows, as (pointer, struct). The caller
        holds the pair until its library call returns: the library runs without
        the interpreter's lock, and another thread may replace what is kept here."""
        d = self._by_rows.get(n_tok)
        if d is None:
            d = _abi.FrPagedBatch()
            n_seq, max_pages = self.page_table.shape
            stride = max(self.page_table.stride(0), max_pages) if n_seq == 1 else self.page_table.stride(0)
            with torch.cuda.device(self.device):
                _abi.check(_abi.load().fr_paged_batch_init(
                    ctypes.addressof(d), self.tok_start.data_ptr(), self.kv_len.data_ptr(), self.page_table.data_ptr(),
                    stride, n_seq, n_tok, max_pages), "fr_paged_batch_init")
            if len(self._by_rows) >= 64:
                self._by_rows.clear()
            d = self._by_rows.setdefault(n_tok, (ctypes.addressof(d), d))
        return d


def _rows(t, name, cache):
    """k_new / v_new: [n_tok, n_kv_head, hd] with contiguous heads, or [n_tok, n_kv_head * hd]; returns (n_tok, token stride)."""
    shape, stride, heads, hd = t.shape, t.stride(), cache.n_kv_head, cache.hd
    if len(shape) == 3:
        ok = shape[1] == heads and shape[2] == hd and stride[2] == 1 and (heads == 1 or stride[1] == hd)
    else:
        ok = len(shape) == 2 and shape[1] == heads * hd and stride[1] == 1
    if not ok:
        raise ValueError(f"{name} must be [n_tok, n_kv_head, hd] with contiguous heads")
    return shape[0], stride[0] if shape[0] > 1 else heads * hd


def kv_append_paged(cache, batch, k_new, v_new, pos, rope, workspace=None, stream=None):
    """fr_kv_append_paged: rotate the step's K rows, and write K and V into the
    pages of their sequences (f16, or e4m3 with a power-of-two scale for each
    page and head). k_new, v_new: f32 or f16 [n_tok, n_kv_head, hd] (the token
    stride may be larger, e.g. columns of a fused QKV buffer); pos: int32
    [n_tok]. workspace: optional, its status word reports bad pages and lengths
    (workspace_check)."""
    if not (k_new.is_cuda and v_new.is_cuda and pos.is_cuda and (workspace is None or workspace.is_cuda)):
        raise ValueError("tensors must be CUDA tensors")
    dtype = k_new.dtype
    if dtype not in _ROWS or v_new.dtype != dtype:
        raise TypeError("k_new and v_new must both be float32 or both float16")
    if pos.dtype != torch.int32:
        raise TypeError("pos must be int32")
    n_tok, k_stride = _rows(k_new, "k_new", cache)
    if v_new.shape == k_new.shape and v_new.stride() == k_new.stride():
        n_v, v_stride = n_tok, k_stride
    else:
        n_v, v_stride = _rows(v_new, "v_new", cache)
    if n_v != n_tok or pos.shape != (n_tok,) or not pos.is_contiguous():
        raise ValueError("k_new, v_new and pos must have one row a token")
    rope, desc = _as_rope(rope), batch._desc(n_tok)
    st = cache._lib.fr_kv_append_paged(
        cache._p, desc[0], _ROWS[dtype], k_new.data_ptr(), k_stride, v_new.data_ptr(), v_stride,
        pos.data_ptr(), ctypes.addressof(rope), None if workspace is None else workspace.data_ptr(),
        _stream_of(stream, cache._index))
    if st:
        _abi.check(st, "fr_kv_append_paged")


def paged_attn_workspace_size(n_head, n_kv_head, hd):
    return int(_abi.load().fr_paged_attn_workspace_size(n_head, n_kv_head, hd))


def make_paged_workspace(n_head, n_kv_head, hd, device="cuda", stream=None):
    """Allocate (torch) and zero (library) a workspace for paged_attn calls of these heads, any batch."""
    n = paged_attn_workspace_size(n_head, n_kv_head, hd)
    if n == 0:
        raise FrError(2, "fr_paged_attn_workspace_size")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        _abi.check(_abi.load().fr_workspace_init(ws.data_ptr(), n, _stream_of(stream, ws.device.index)), "fr_workspace_init")
    return ws


def paged_attn(cache, batch, q16, n_head, *, causal=True, window=0, kq_scale=1.0, out=None, workspace=None, stream=None):
    """fr_paged_attn: attention of the step's query rows over the paged cache.
    q16: f16 [n_tok, n_head, hd] (the token stride may be larger) or [n_tok *
    n_head, hd] contiguous, as qkv_post returns it. causal: token i of a
    sequence sees the keys up to its own; window > 0: only the last `window` of
    them. Returns out [n_tok, n_head, hd] f32; rows behind the last sequence are
    left as they were."""
    if not (q16.is_cuda and (out is None or out.is_cuda) and (workspace is None or workspace.is_cuda)):
        raise ValueError("tensors must be CUDA tensors")
    hd, shape, strides = cache.hd, q16.shape, q16.stride()
    if q16.dtype != torch.float16:
        raise TypeError("q16 must be float16")
    if len(shape) == 3 and shape[1] == n_head and shape[2] == hd and strides[2] == 1 and (
            n_head == 1 or strides[1] == hd):
        n_tok = shape[0]
        stride = strides[0] if n_tok > 1 else n_head * hd
    elif len(shape) == 2 and shape[1] == hd and n_head > 0 and shape[0] % n_head == 0 and q16.is_contiguous():
        n_tok, stride = shape[0] // n_head, n_head * hd
    else:
        raise ValueError("q16 must be [n_tok, n_head, hd] with contiguous heads, or [n_tok * n_head, hd] contiguous")
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.empty((n_tok, n_head, hd), dtype=torch.float32, device=q16.device)
    elif out.dtype != torch.float32 or out.shape != (n_tok, n_head, hd) or not out.is_contiguous():
        raise ValueError("out must be contiguous float32 [n_tok, n_head, hd]")
    if workspace is None:
        workspace = make_paged_workspace(n_head, cache.n_kv_head, hd, cache.device, stream)
    # (a C int would keep the low 32 bits of what does not fit it)
    window = -1 if window < 0 else 2 ** 31 - 1 if window > 2 ** 31 - 1 else window
    desc = batch._desc(n_tok)
    st = cache._lib.fr_paged_attn(
        cache._p, desc[0], q16.data_ptr(), stride, n_head, 1 if causal else 0, window, kq_scale,
        out.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_of(stream, cache._index))
    if st:
        _abi.check(st, "fr_paged_attn")
    return out
