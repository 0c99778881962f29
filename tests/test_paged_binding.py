"""The Python side of the paged calls without a GPU, over a stand-in for the
library: what it is handed, and that it stays valid while a call runs."""
import ctypes
import threading

import pytest
import torch

import gqa_kv_head_gb300 as fr
from gqa_kv_head_gb300 import _abi


class Fake:
    """As much of a CUDA tensor as the binding looks at."""
    is_cuda = True

    def __init__(self, shape, dtype):
        self.t = torch.zeros(shape, dtype=dtype)
        self.shape, self.dtype, self.device = self.t.shape, dtype, None

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    cuda_stream = 0


class Library:
    """Records what a call was handed; `during` runs inside it."""

    def __init__(self):
        self.calls, self.during, self.in_init = [], lambda: None, lambda: None

    def fr_paged_batch_init(self, d, *args):
        self.in_init()
        return 0

    def fr_paged_attn(self, kv, batch, *args):
        self.during()
        self.calls.append(("attn", batch, args))
        return 0

    def fr_kv_append_paged(self, kv, batch, *args):
        self.during()
        self.calls.append(("append", batch, args))
        return 0


@pytest.fixture
def lib(monkeypatch):
    x = Library()
    monkeypatch.setattr(_abi, "load", lambda: x)
    return x


@pytest.fixture
def freed(monkeypatch):
    """Addresses of the batch descriptors that are gone."""
    gone = set()

    class Counted(_abi.FrPagedBatch):
        def __del__(self):
            gone.add(ctypes.addressof(self))
    monkeypatch.setattr(_abi, "FrPagedBatch", Counted)
    return gone


def make_cache(lib):
    c = object.__new__(fr.PagedKV)
    c._lib, c._p, c._index, c.hd, c.n_kv_head, c.device = lib, ctypes.c_void_p(16), 0, 64, 1, None
    return c


def make_batch():
    b = object.__new__(fr.PagedBatch)
    i = torch.zeros((1, 1), dtype=torch.int32)
    b.tok_start, b.kv_len, b.page_table, b.device, b._by_rows = i, i, i, -1, {}
    return b


def attend(cache, batch, n_tok=1, **kw):
    return fr.paged_attn(cache, batch, Fake((n_tok, 2, 64), torch.float16), 2, out=Fake((n_tok, 2, 64), torch.float32),
                         workspace=Fake((64,), torch.uint8), stream=Stream(), **kw)


def append(cache, batch, n_tok=1):
    x = Fake((n_tok, 1, 64), torch.float32)
    fr.kv_append_paged(cache, batch, x, x, Fake((n_tok,), torch.int32), fr.rope_params(64), stream=Stream())


@pytest.mark.parametrize("call", [attend, append])
def test_descriptor_lives_while_two_threads_make_their_first_call(lib, freed, call):
    """Both find no descriptor for their rows and make one each, since the
    library runs without the interpreter's lock; one of the two is kept for later
    calls, and neither may go while its thread's call runs."""
    cache, batch = make_cache(lib), make_batch()
    made, called = threading.Barrier(2), threading.Barrier(2)
    lib.in_init = lambda: made.wait(30)
    seen = []

    def during():
        called.wait(30)              # both descriptors are made, and one has been put aside
        seen.append(set(freed))
        called.wait(30)
    lib.during = during
    threads = [threading.Thread(target=call, args=(cache, batch)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert len(lib.calls) == 2 and len(seen) == 2
    for (_, address, _), gone in zip(lib.calls, seen):
        assert int(getattr(address, "value", address)) not in gone


@pytest.mark.parametrize("call", [attend, append])
def test_descriptor_lives_while_others_replace_it(lib, freed, call):
    """Another thread's calls with many numbers of rows empty the kept descriptors during a call."""
    cache, batch = make_cache(lib), make_batch()
    gone = []

    def during():
        for n in range(100, 300):
            batch._desc(n)
        gone.append(set(freed))
    lib.during = during
    call(cache, batch)
    (_, address, _), = lib.calls
    assert int(getattr(address, "value", address)) not in gone[0]
    assert len(batch._by_rows) <= 64


def test_descriptor_is_kept_between_calls(lib, freed):
    cache, batch = make_cache(lib), make_batch()
    for _ in range(3):
        attend(cache, batch)
        append(cache, batch)
    assert len({int(getattr(a, "value", a)) for _, a, _ in lib.calls}) == 1 and not freed


@pytest.mark.parametrize("window,handed", [(0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                           (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1)])
def test_windows_beyond_32_bits_stay_wide(lib, window, handed):
    attend(make_cache(lib), make_batch(), window=window)
    (_, _, args), = lib.calls
    assert ctypes.c_int(args[4]).value == handed


def test_negative_windows_stay_negative(lib):
    """(so that the library refuses them)"""
    for window in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 5):
        attend(make_cache(lib), make_batch(), window=window)
        assert ctypes.c_int(lib.calls[-1][2][4]).value < 0
