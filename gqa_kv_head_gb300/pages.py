"""Python binding of the page-pool entry points: argument marshalling only.

A PagePool checks and describes the tensors of a pool once; the calls pass it on.
The tensors are read and changed on the device by every call.
"""
import ctypes

import torch

from . import _abi
from ._abi import FrError
from .ops import _check_dev
from .paged import _stream_of

_INT_MAX = 2 ** 31 - 1


def _int(n):
    """n, or -1 or the largest C int in its place (a C int would keep the low 32 bits of what does not fit it)."""
    return max(-1, min(n, _INT_MAX))


def pages_workspace_size(n_pages, n_seq):
    return int(_abi.load().fr_pages_workspace_size(_int(n_pages), _int(n_seq)))


class PagePool:
    """fr_page_pool: which pages of a cache belong to whom.

    refs: int32 [n_pages], holders of each page; kv_len: int32 [n_seq]; page_table:
    int32 [n_seq, max_pages] (row stride free): the tensors that a PagedBatch of
    the same slots has. One pool serves the caches of all layers. Its workspace
    is allocated (torch) and zeroed (library) here.

    After pages_reserve or pages_compact, n_moves (int32, one element) and moves
    (int32 [., 4]: from, to, rows, 0) say what pages_copy is to copy; after
    pages_compact page_map (int32 [n_pages]) says where each page went."""

    def __init__(self, refs, kv_len, page_table, page_size, stream=None):
        _check_dev(refs, kv_len, page_table)
        for name, t in (("refs", refs), ("kv_len", kv_len), ("page_table", page_table)):
            if t.dtype != torch.int32:
                raise TypeError(f"{name} must be int32")
        if refs.dim() != 1 or kv_len.dim() != 1 or not refs.is_contiguous() or not kv_len.is_contiguous():
            raise ValueError("refs must be contiguous [n_pages] and kv_len contiguous [n_seq]")
        if page_table.dim() != 2 or page_table.shape[0] != kv_len.shape[0]:
            raise ValueError("page_table must be [n_seq, max_pages]")
        if page_table.shape[1] > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table needs unit inner stride")
        if len({t.device for t in (refs, kv_len, page_table)}) != 1:
            raise ValueError("tensors of a pool must be on one GPU")
        self.refs, self.kv_len, self.page_table, self.page_size = refs, kv_len, page_table, page_size
        self.device, self._index = refs.device, refs.device.index
        n_pages, (n_seq, max_pages) = refs.shape[0], page_table.shape
        self._lib = _abi.load()
        n = pages_workspace_size(n_pages, n_seq)
        if n == 0:
            raise FrError(2, "fr_pages_workspace_size")
        self._desc = _abi.FrPagePool()
        self._p = ctypes.c_void_p(ctypes.addressof(self._desc))
        row = max(page_table.stride(0), max_pages) if n_seq == 1 else page_table.stride(0)
        with torch.cuda.device(self.device), torch.cuda.stream(stream):
            self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)
            _abi.check(self._lib.fr_page_pool_init(
                self._p, refs.data_ptr(), n_pages, _int(page_size), kv_len.data_ptr(), page_table.data_ptr(), row, n_seq, max_pages,
                self.workspace.data_ptr(), n), "fr_page_pool_init")
            _abi.check(self._lib.fr_workspace_init(self.workspace.data_ptr(), n, _stream_of(stream, self._index)),
                       "fr_workspace_init")
        most, end = max(n_seq, n_pages // 2 + 1), 1024 + 16 * max(n_seq, n_pages // 2 + 1)
        self.n_moves = self.workspace[64:68].view(torch.int32)
        self.moves = self.workspace[1024:end].view(torch.int32).view(most, 4)
        self.page_map = self.workspace[end:end + 4 * n_pages].view(torch.int32)


def _slots(pool, name, t, n=None):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.get_device() != pool._index:                   # (-1: not on a GPU)
        raise ValueError(f"{name} must be on the pool's GPU")
    shape = t.shape
    if len(shape) != 1 or not t.is_contiguous() or (n is not None and shape[0] != n):
        raise ValueError(f"{name} must be contiguous, one number a slot" if n is None else f"{name} must be contiguous [{n}]")
    return t.data_ptr()


def _done(status, where):
    if status:
        _abi.check(status, where)


def pages_reserve(pool, tok_start, stream=None):
    """fr_pages_reserve: pages for a step's new rows (int32 tok_start [n_seq + 1];
    kv_len counts them already), shared last pages replaced by copies of the
    slot's own. Run pages_copy for each layer's cache after it."""
    ts = _slots(pool, "tok_start", tok_start, pool.kv_len.shape[0] + 1)
    _done(pool._lib.fr_pages_reserve(pool._p, ts, _stream_of(stream, pool._index)), "fr_pages_reserve")


def pages_fork(pool, parent, child, length=None, stream=None):
    """fr_pages_fork: slot child[i], empty so far, shares the pages of the first
    length[i] keys (None: all) of slot parent[i]. int32 tensors; -1: no pair."""
    p = _slots(pool, "parent", parent)
    n = parent.shape[0]
    c = _slots(pool, "child", child, n)
    m = None if length is None else _slots(pool, "length", length, n)
    if n:
        _done(pool._lib.fr_pages_fork(pool._p, p, c, m, n, _stream_of(stream, pool._index)), "fr_pages_fork")


def pages_free(pool, seq, keep=None, stream=None):
    """fr_pages_free: slots seq (int32, -1: none) keep their first keep[i] keys (None:
    none) and give back the pages behind."""
    s = _slots(pool, "seq", seq)
    n = seq.shape[0]
    k = None if keep is None else _slots(pool, "keep", keep, n)
    if n:
        _done(pool._lib.fr_pages_free(pool._p, s, k, n, _stream_of(stream, pool._index)), "fr_pages_free")


def pages_trim(pool, window, sinks=0, tok_start=None, stream=None):
    """fr_pages_trim: every slot gives back the pages that paged_attn(window=,
    sinks=) does not look up any more, from the step of tok_start on (None: from
    the next key on)."""
    ts = None if tok_start is None else _slots(pool, "tok_start", tok_start, pool.kv_len.shape[0] + 1)
    _done(pool._lib.fr_pages_trim(pool._p, ts, _int(window), _int(sinks), _stream_of(stream, pool._index)), "fr_pages_trim")


def pages_compact(pool, stream=None):
    """fr_pages_compact: held pages move to the front of the pool; tables and refs
    follow. Run pages_copy for each layer's cache after it."""
    _done(pool._lib.fr_pages_compact(pool._p, _stream_of(stream, pool._index)), "fr_pages_compact")


def pages_copy(cache, pool, stream=None):
    """fr_pages_copy: the copies that the pool's last pages_reserve or pages_compact
    asks for, in one cache (a PagedKV of the pool's pages)."""
    _done(pool._lib.fr_pages_copy(cache._p, pool._p, _stream_of(stream, pool._index)), "fr_pages_copy")


def pages_check(pool, stream=None):
    """fr_pages_check: raise FrError if an earlier call on the pool ran out of pages
    (FR_ERR_DEVICE_PAGES) or met bad numbers (FR_ERR_DEVICE_INPUT); of both the first
    now, the second by the next check."""
    _done(pool._lib.fr_pages_check(pool._p, _stream_of(stream, pool._index)), "fr_pages_check")
