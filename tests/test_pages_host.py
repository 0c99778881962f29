"""The page pool without a GPU: refusals that the host makes before any CUDA call,
the binding's checks, and the sequential form that the GPU tests compare with."""
import ctypes
import random

import pytest
import torch

from pages_ref import Pool

FAKE = 0x10000            # aligned, never dereferenced: validation fails first
OK_BUT_NO_GPU = (1, 4)    # past the host's checks: no GPU here (4), or not device memory (1)


@pytest.fixture(scope="module")
def lib():
    from gqa_kv_head_gb300 import build
    build.build()
    import gqa_kv_head_gb300 as fr
    return fr.load()


def test_pool_descriptor_refusals(lib):
    from gqa_kv_head_gb300._abi import FrPagePool
    need = lib.fr_pages_workspace_size(100, 8)
    assert need >= 1024 + 16 * 51 + 2 * 400 + 16 * 8

    def call(refs=FAKE, n_pages=100, ps=64, kl=FAKE, tab=FAKE, stride=16, n_seq=8, max_pages=16, ws=FAKE, n=need, desc=True):
        d = FrPagePool()
        return lib.fr_page_pool_init(ctypes.addressof(d) if desc else None, refs, n_pages, ps, kl, tab, stride, n_seq, max_pages, ws, n)
    assert call() in OK_BUT_NO_GPU
    assert call(desc=False) == 1 and call(refs=None) == 1 and call(kl=None) == 1 and call(tab=None) == 1 and call(ws=None) == 1
    assert call(n_pages=0) == 1 and call(n_seq=0) == 1 and call(max_pages=0) == 1 and call(ps=0) == 1 and call(ps=-64) == 1
    assert call(stride=15) == 1 and call(refs=FAKE + 2) == 1 and call(kl=FAKE + 1) == 1 and call(tab=FAKE + 3) == 1
    assert call(ws=FAKE + 4) == 1
    for ps in (1, 8, 24, 100, 512):
        assert call(ps=ps) == 2
    assert call(n_pages=(1 << 28) + 1) == 2 and call(n_seq=65537) == 2 and call(max_pages=(1 << 22) + 1, stride=1 << 23) == 2
    assert call(n=need - 1) == 3


def test_workspace_size(lib):
    ws = lib.fr_pages_workspace_size
    assert ws(0, 1) == 0 and ws(1, 0) == 0 and ws(-1, 4) == 0 and ws((1 << 28) + 1, 1) == 0 and ws(1, 65537) == 0
    assert ws(1, 1) > 0 and ws(1 << 28, 65536) > 2 * 4 * (1 << 28)
    assert lib.fr_status_string(7).startswith(b"FR_ERR_DEVICE_PAGES")


def test_calls_want_filled_descriptors(lib):
    from gqa_kv_head_gb300._abi import FrPagedKV, FrPagePool
    d, kv = FrPagePool(), FrPagedKV()
    for p in (None, ctypes.addressof(d)):
        assert lib.fr_pages_reserve(p, FAKE, None) == 1
        assert lib.fr_pages_fork(p, FAKE, FAKE, None, 1, None) == 1
        assert lib.fr_pages_free(p, FAKE, None, 1, None) == 1
        assert lib.fr_pages_trim(p, None, 1, 0, None) == 1
        assert lib.fr_pages_compact(p, None) == 1
        assert lib.fr_pages_copy(ctypes.addressof(kv), p, None) == 1
        assert lib.fr_pages_check(p, None) == 1
    # a refused fill leaves a descriptor that no call takes
    d.opaque[3] = 5
    assert lib.fr_page_pool_init(ctypes.addressof(d), FAKE, 10, 64, FAKE, FAKE, 1, 4, 4, FAKE, 1 << 20) == 1
    assert not any(d.opaque)


def test_rows_call_refusals(lib):
    """fr_qkv_post_paged and fr_paged_attn_sinks without filled descriptors."""
    from gqa_kv_head_gb300 import rope_params
    from gqa_kv_head_gb300._abi import FrPagedBatch, FrPagedKV
    kv, bt, rp = FrPagedKV(), FrPagedBatch(), rope_params(64)
    for a, b in ((None, ctypes.addressof(bt)), (ctypes.addressof(kv), None), (ctypes.addressof(kv), ctypes.addressof(bt))):
        assert lib.fr_qkv_post_paged(a, b, 0, FAKE, 256, FAKE, 64, FAKE, 64, FAKE, 4, None, None, 0.0, ctypes.addressof(rp), 0, 0.0,
                                     FAKE, None, None) == 1
        assert lib.fr_paged_attn_sinks(a, b, FAKE, 256, 4, 1, 16, 4, 1.0, FAKE, FAKE, 1 << 30, None) == 1


def test_binding_refuses_cpu_tensors():
    import gqa_kv_head_gb300 as fr
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        fr.PagePool(i, i, i[None].expand(4, 4), 16)


# ---- the sequential form itself ------------------------------------------------

def holds(pool, extra=()):
    """Every page counts the entries that hold it."""
    n = [0] * len(pool.refs)
    for b, length in enumerate(pool.kv_len):
        for e in range(pool.pages(length)):
            if pool.table[b][e] >= 0:
                n[pool.table[b][e]] += 1
    for p in extra:
        n[p] += 1
    return n == pool.refs


def random_steps(rng, pool, turns, most_new=40):
    """Yields the calls of a host that never asks for more than there is: (name, arguments), applied to the pool."""
    n_seq = len(pool.kv_len)
    for _ in range(turns):
        what = rng.choice(["step", "step", "step", "fork", "free", "keep", "trim", "compact"])
        live = [b for b in range(n_seq) if pool.kv_len[b]]
        empty = [b for b in range(n_seq) if not pool.kv_len[b]]
        if what == "step":
            new = [0] * n_seq
            left = sum(r == 0 for r in pool.refs)
            for b in rng.sample(range(n_seq), n_seq):
                a = rng.choice([0, 1, 1, 2, rng.randint(0, most_new)])
                cost = a // pool.ps + 2
                if a and cost <= left and pool.kv_len[b] + a <= pool.most:
                    new[b], left = a, left - cost
            starts = [sum(new[:i]) for i in range(n_seq + 1)]
            for b in range(n_seq):
                pool.kv_len[b] += new[b]
            lens = list(pool.kv_len)
            pool.reserve(starts)
            yield "reserve", (lens, starts)
        elif what == "fork" and live and empty:
            k = rng.randint(1, len(empty))
            child = rng.sample(empty, k)
            parent = [rng.choice(live) for _ in child]
            length = None if rng.random() < 0.5 else [rng.randint(0, pool.kv_len[p]) for p in parent]
            if rng.random() < 0.3:
                parent, child = parent + [-1], child + [rng.choice(empty)]
                length = length and length + [5]
            if len(child) > n_seq:
                continue
            pool.fork(parent, child, length)
            yield "fork", (parent, child, length)
        elif what in ("free", "keep") and live:
            seq = rng.sample(live, rng.randint(1, max(1, len(live) // 2))) + [-1] * rng.randint(0, 2)
            keep = None if what == "free" else [rng.randint(0, pool.kv_len[b]) if b >= 0 else 3 for b in seq]
            pool.free(seq, keep)
            yield "free", (seq, keep)
        elif what == "trim" and rng.random() < 0.3:
            window, sinks = rng.randint(20, 400), rng.randint(0, 70)
            pool.trim(window, sinks)
            yield "trim", (window, sinks)
        elif what == "compact":
            pool.compact()
            yield "compact", ()


@pytest.mark.parametrize("seed", range(8))
def test_sequential_form_keeps_count(seed):
    rng = random.Random(seed)
    pool = Pool(60, 16, 9, 40)
    done = set()
    for name, _ in random_steps(rng, pool, 150):
        done.add(name)
        assert holds(pool), name
        assert not pool.bad and not pool.short
        if name == "compact":
            used = [r > 0 for r in pool.refs]
            assert used == sorted(used, reverse=True)
        if name == "reserve":
            # rows to be written are in pages of their slot's own
            assert len({m[1] for m in pool.moves}) == len(pool.moves)
    assert done == {"reserve", "fork", "free", "trim", "compact"}
