"""The page pool on the GPU against its sequential form (pages_ref.py): tables, counts,
lengths and moves exactly, pages bit by bit, over random histories, many slots, large
pools, shared and last pages, pools that run out, bad numbers, repeated slots, two
layers, strides, streams and captured graphs; and a serving history as it is used."""
import random

import pytest
import torch

import gqa_kv_head_gb300 as fr
import paged_ref as ref
from pages_ref import Pool
from test_gpu_paged import make_cache
from test_pages_host import holds, random_steps

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A pool on the GPU and its sequential form."""

    def __init__(self, n_pages, ps, n_seq, max_pages, pad=0, plain=None):
        self.ref = plain or Pool(n_pages, ps, n_seq, max_pages)
        self.table = torch.full((n_seq, max_pages + pad), -1, dtype=torch.int32, device="cuda")[:, :max_pages]
        self.table.copy_(ints(self.ref.table))
        self.pool = fr.PagePool(ints(self.ref.refs), ints(self.ref.kv_len), self.table, ps)

    def compare(self, what="", moves=False):
        r = self.ref
        assert self.pool.refs.tolist() == r.refs, what
        assert self.pool.kv_len.tolist() == r.kv_len, what
        assert self.table.tolist() == r.table, what
        if moves:
            n = int(self.pool.n_moves)
            assert n == len(r.moves), what
            got = [tuple(m) for m in self.pool.moves[:n, :3].tolist()]
            assert got == r.moves, what

    def call(self, name, args):
        if name == "reserve":
            lens, starts = args
            self.pool.kv_len.copy_(ints(lens))
            fr.pages_reserve(self.pool, ints(starts))
        elif name == "fork":
            fr.pages_fork(self.pool, ints(args[0]), ints(args[1]), None if args[2] is None else ints(args[2]))
        elif name == "free":
            fr.pages_free(self.pool, ints(args[0]), None if args[1] is None else ints(args[1]))
        elif name == "trim":
            fr.pages_trim(self.pool, *args)
        else:
            fr.pages_compact(self.pool)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("n_pages,ps,n_seq,max_pages", [(60, 16, 9, 40), (300, 32, 40, 70), (40, 256, 5, 9)])
def test_random_histories(seed, n_pages, ps, n_seq, max_pages):
    two = Both(n_pages, ps, n_seq, max_pages, pad=3)
    for name, args in random_steps(random.Random(seed), two.ref, 60, most_new=3 * ps):
        two.call(name, args)
        two.compare(name, moves=name in ("reserve", "compact"))
        if name == "compact":
            assert two.pool.page_map.tolist() == two.ref.map
    # (a slot cut back into its trimmed pages goes on in no page: both say so)
    assert two_status(two.pool) == (6 if two.ref.bad else 0)


@pytest.mark.parametrize("n_seq,n_pages,c", [(1, 1, 1), (1, 5, 3), (3000, 16385, 5), (9000, 40000, 3), (20000, 70001, 2), (65536, 200000, 2)])
def test_sizes_of_the_cluster(n_seq, n_pages, c):
    """One CTA to eight, one sequence of a thread to several; every third slot without tokens."""
    rng = random.Random(n_seq)
    two = Both(n_pages, 16, n_seq, c)
    r = two.ref
    for turn in range(3):
        new = [0 if (b + turn) % 3 == 0 else rng.randint(1, 16 * c // 3 if c > 2 else 12) for b in range(n_seq)]
        new = [min(a, r.most - n) for a, n in zip(new, r.kv_len)]
        starts = [0]
        for a in new:
            starts.append(starts[-1] + a)
        r.kv_len = [n + a for n, a in zip(r.kv_len, new)]
        lens = list(r.kv_len)
        r.reserve(starts)
        two.call("reserve", (lens, starts))
        two.compare(f"turn {turn}", moves=True)
        gone = [b for b in range(n_seq) if rng.random() < 0.3] or [0]
        r.free(gone)
        two.call("free", (gone, None))
        pairs = [(b, b + 1) for b in range(0, n_seq - 1) if r.kv_len[b] and not r.kv_len[b + 1]]
        if pairs:
            p, k = [x for x, _ in pairs], [y for _, y in pairs]
            r.fork(p, k)
            two.call("fork", (p, k, None))
        two.compare(f"turn {turn}, freed and forked")
    r.compact()
    two.call("compact", ())
    two.compare("compact", moves=True)
    assert r.short == (two_status(two.pool) == 7)


def two_status(pool):
    try:
        fr.pages_check(pool)
    except fr.FrError as e:
        return e.status
    return 0


def test_long_sequences():
    """Thousands of entries of one slot; the fork's pieces and the free's steps."""
    two = Both(40000, 16, 6, 30000)
    r = two.ref
    for lens in ([300000, 0, 0, 7, 0, 0], [300013, 160000, 0, 1000, 0, 0]):
        new = [a - b for a, b in zip(lens, r.kv_len)]
        starts = [sum(new[:i]) for i in range(7)]
        r.kv_len = list(lens)
        r.reserve(starts)
        two.call("reserve", (lens, starts))
        two.compare("reserve", moves=True)
    for name, args in (("fork", ([0, 0, 1], [2, 4, 5], [300000, 12345, 160000])), ("trim", (1000, 40)), ("free", ([0, 5], [100000, 0])),
                       ("free", ([2], None)), ("compact", ())):
        getattr(r, name)(*args)
        two.call(name, args)
        two.compare(name)
    fr.pages_check(two.pool)


def test_shared_last_pages():
    """All holders go on: the last keeps the page. Some go on: they copy. A page's first row needs no copy."""
    for ps, length in ((16, 21), (16, 32), (64, 1), (64, 63)):
        for who in ([0, 1, 2, 3], [0, 1], [3], [1, 2, 3]):
            two = Both(30, ps, 5, 4)
            r = two.ref
            r.kv_len[0] = length
            two.pool.kv_len[0] = length
            starts = [0] + [length] * 5
            r.reserve(starts)
            fr.pages_reserve(two.pool, ints(starts))
            r.fork([0, 0, 0], [1, 2, 3])
            two.call("fork", ([0, 0, 0], [1, 2, 3], None))
            new = [1 if b in who else 0 for b in range(5)]
            starts = [sum(new[:i]) for i in range(6)]
            r.kv_len = [n + a for n, a in zip(r.kv_len, new)]
            lens = list(r.kv_len)
            r.reserve(starts)
            two.call("reserve", (lens, starts))
            two.compare(f"{ps} {length} {who}", moves=True)
            assert holds(r)
            if length % ps and len(who) == 4:
                assert len(r.moves) == 3 and all(m[2] == length % ps for m in r.moves)


def test_pool_runs_out():
    """The lowest slots get the pages that are left; the others' entries become -1; the next step goes on."""
    two = Both(10, 16, 4, 8)
    r = two.ref
    for lens, starts in (([40, 33, 0, 0], [0, 40, 73, 73, 73]), ([57, 65, 20, 100], [0, 17, 49, 69, 169])):
        r.kv_len = list(lens)
        r.reserve(starts)
        two.call("reserve", (lens, starts))
        two.compare("reserve", moves=True)
    assert r.short and two_status(two.pool) == 7 and two_status(two.pool) == 0
    r.free([3, 1])
    two.call("free", ([3, 1], None))
    two.compare("freed")
    # a shared page that can not be copied: its rows are lost to the slot
    two = Both(2, 16, 3, 2)
    r = two.ref
    for step in range(3):
        lens, starts = ([20, 0, 0], [0, 20, 20, 20]) if step == 0 else ([20, 21, 0], [0, 0, 1, 1])
        if step == 1:
            r.fork([0], [1])
            two.call("fork", ([0], [1], None))
            continue
        r.kv_len = list(lens)
        r.reserve(starts)
        two.call("reserve", (lens, starts))
        two.compare("", moves=True)
    assert r.moves == [(1, -1, 4)] and two_status(two.pool) == 7
    _, cache = make_cache("f16", 2, 1, 16, 64)
    before = cache.k_pages.clone()
    fr.pages_copy(cache, two.pool)                       # (a move to nowhere is none)
    assert torch.equal(before, cache.k_pages)


def test_bad_numbers():
    """Skipped and reported; what fits is done; counts below one are never taken."""
    two = Both(50, 16, 8, 6)
    r = two.ref
    lens, starts = [20, 50, 96, 5, 0, 0, 0, 0], [0, 20, 70, 166, 171, 171, 171, 171, 171]
    r.kv_len = list(lens)
    r.reserve(starts)
    two.call("reserve", (lens, starts))
    two.compare()
    assert two_status(two.pool) == 0

    def both(name, args, edit=None):
        if edit:
            edit()
        getattr(r, name)(*args) if name != "reserve" else r.reserve(args[1])
        two.call(name, args)
        two.compare(name)
        assert r.bad == (two_status(two.pool) == 6), name
        r.bad = False
    both("fork", ([0, 0, 9, 1, -3, 2, 3, 0], [4, 4, 5, -2, 5, 2, 0, 8], None))       # twice one child, out of range, itself, not empty
    both("fork", ([1, 1, 2], [5, 6, 7], [51, -1, 96]))                               # longer than the parent, negative
    both("free", ([8, -2, 100000, 4], None))
    both("free", ([0, 1], [-1, 60]))
    two.ref.kv_len[3] = 97                                                          # longer than a table row
    both("reserve", (list(r.kv_len), [0] * 9))
    both("trim", (1, 0))
    two.ref.kv_len[3] = -4
    two.pool.kv_len[3] = -4
    both("free", ([3], None))
    both("trim", (10, 0))
    two.ref.kv_len[3] = 0
    two.pool.kv_len[3] = 0
    both("reserve", (list(r.kv_len), [0, 0, 5, 3, 3, 3, 3, 3, 2]))                   # not in order
    both("reserve", (list(r.kv_len), [-5, 0, 0, 0, 0, 0, 0, 0, 0]))
    # entries that hold no page, or one that counts no holder
    two.ref.table[2][0], two.ref.table[2][5] = 50, -9
    two.table[2, 0], two.table[2, 5] = 50, -9
    both("free", ([2], None))
    two.ref.refs = [0] * 50
    two.pool.refs.zero_()
    both("free", ([1], None))
    assert all(x == 0 for x in two.pool.refs.tolist())


@pytest.mark.parametrize("entry", [-1, 7, 50, 2 ** 31 - 1])
def test_going_on_in_no_page(entry):
    """The page of a slot's last rows is none, or counts no holder: the entry is filled anew, and reported."""
    two = Both(50, 16, 2, 6)
    r = two.ref
    for p in (r.table[0], two.table[0]):
        p[0] = entry
    r.reserve([0, 0, 0])
    r.kv_len = [6, 0]
    r.reserve([0, 3, 3])
    two.call("reserve", ([6, 0], [0, 3, 3]))
    two.compare("", moves=True)
    assert r.bad and two_status(two.pool) == 6


def test_slots_named_more_than_once():
    two = Both(60, 16, 6, 8)
    r = two.ref
    lens, starts = [100, 60, 30, 0, 0, 0], [0, 100, 160, 190, 190, 190, 190]
    r.kv_len = list(lens)
    r.reserve(starts)
    two.call("reserve", (lens, starts))
    for args in (([0, 0, 0], [90, 20, 50]), ([1, 2, 1], None), ([0] * 6, [20, 3, 3, 90, 3, 20])):
        r.free(*args)
        two.call("free", args)
        two.compare(str(args))
    assert two_status(two.pool) == 0


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("H,ps,hd,nhd", [(1, 16, 64, False), (3, 64, 128, False), (2, 32, 256, True), (5, 128, 64, True), (8, 256, 128, False)])
def test_copies(kind, H, ps, hd, nhd):
    """The moves of a reserve (part of the rows) and of a compact, in the caches of two layers."""
    n_pages = 24
    layers = [make_cache(kind, n_pages, H, ps, hd, s, nhd) for s in (1, 2)]
    two = Both(n_pages, ps, 6, 6)
    r = two.ref
    first = 2 * ps + 5
    lens, starts = [first, ps, 3 * ps, 0, 0, 0], [0, first, first + ps, first + 4 * ps] + [first + 4 * ps] * 3
    r.kv_len = list(lens)
    r.reserve(starts)
    two.call("reserve", (lens, starts))
    for name, args in (("fork", ([0, 0, 0], [3, 4, 5], None)), ("free", ([1], None))):
        getattr(r, name)(*args)
        two.call(name, args)
    now = [[t.clone() for t in (c.k_pages, c.v_pages)] + [None if s is None else s.clone() for s in (c.k_scale, c.v_scale)] for _, c in layers]

    def copied():
        for (_, cache), old in zip(layers, now):
            fr.pages_copy(cache, two.pool)
            for i, t in enumerate((cache.k_pages, cache.v_pages)):
                want = old[i].clone()
                w8, o8 = (x.view(torch.uint8) if kind == "e4m3" else x for x in (want, old[i]))
                for a, b, rows in r.moves:
                    w8[b, :, :rows] = o8[a, :, :rows]
                assert ref.same_bits(t.cpu(), want.cpu())
                old[i] = want
            if kind == "e4m3":
                for i, s in enumerate((cache.k_scale, cache.v_scale)):
                    want = old[2 + i].clone()
                    for a, b, _ in r.moves:
                        want[b] = old[2 + i][a]
                    assert torch.equal(s, want)
                    old[2 + i] = want
    lens = [first, 0, 3 * ps, first + 1, first + ps, first + 2]
    r.kv_len = list(lens)
    starts = [0, 0, 0, 0, 1, 1 + ps, 3 + ps]
    r.reserve(starts)
    two.call("reserve", (lens, starts))
    two.compare("reserve", moves=True)
    assert [m[2] for m in r.moves] == [5, 5, 5]
    copied()
    r.free([0])
    two.call("free", ([0], None))
    r.compact()
    two.call("compact", ())
    two.compare("compact", moves=True)
    assert r.moves
    copied()


def test_copy_wants_the_pools_cache():
    two = Both(24, 16, 3, 4)
    for n_pages, ps in ((23, 16), (24, 32)):
        _, cache = make_cache("f16", n_pages, 1, ps, 64)
        with pytest.raises(fr.FrError):
            fr.pages_copy(cache, two.pool)


def test_refusals():
    refs, lens, table = ints([0] * 8), ints([0] * 3), torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    pool = fr.PagePool(refs, lens, table, 16)
    for bad in (lambda: fr.PagePool(refs.long(), lens, table, 16), lambda: fr.PagePool(refs, lens.float(), table, 16),
                lambda: fr.PagePool(refs, lens, table.long(), 16), lambda: fr.pages_reserve(pool, ints([0] * 4).long()),
                lambda: fr.pages_free(pool, ints([0]).long()), lambda: fr.pages_fork(pool, ints([0]), ints([1]), ints([1]).float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fr.PagePool(refs[None], lens, table, 16), lambda: fr.PagePool(refs, lens[:2], table, 16),
                lambda: fr.PagePool(refs[::2], lens, table, 16), lambda: fr.PagePool(refs, lens, table.T, 16),
                lambda: fr.PagePool(refs, lens, torch.zeros((3, 8), dtype=torch.int32, device="cuda")[:, ::2], 16),
                lambda: fr.pages_reserve(pool, ints([0] * 3)), lambda: fr.pages_fork(pool, ints([0]), ints([1, 2])),
                lambda: fr.pages_fork(pool, ints([0]), ints([1]), ints([1, 2])), lambda: fr.pages_free(pool, ints([0, 1]), ints([0])),
                lambda: fr.pages_free(pool, torch.zeros(1, dtype=torch.int32)), lambda: fr.pages_reserve(pool, ints([0] * 8)[::2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fr.PagePool(refs, lens, table, 24), lambda: fr.PagePool(refs, lens, table, 0),
                lambda: fr.PagePool(refs, lens, torch.zeros((1, 4), dtype=torch.int32, device="cuda").expand(3, 4), 16),
                lambda: fr.pages_trim(pool, 0), lambda: fr.pages_trim(pool, 5, -1), lambda: fr.pages_trim(pool, -2 ** 40),
                lambda: fr.pages_fork(pool, ints([0] * 4), ints([1] * 4))):
        with pytest.raises(fr.FrError):
            bad()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    fr.pages_free(pool, none)
    fr.pages_fork(pool, none, none)
    fr.pages_trim(pool, 2 ** 40, 2 ** 40)
    fr.pages_check(pool)
    assert refs.tolist() == [0] * 8


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_serving_history(kind):
    """Prompts, samples that branch off, decode steps with a window and sinks, trimming and
    compacting, as a host runs them: each step captured once and replayed. What the slots
    hold is the same as in caches of their own, and so is what the attention makes of it."""
    hd, H, G, ps, n_seq, max_pages, window, sinks = 64, 2, 2, 16, 6, 20, 60, 5
    n_pages, n_own = 48, n_seq * max_pages
    two = Both(n_pages, ps, n_seq, max_pages)
    r, pool = two.ref, two.pool
    _, cache = make_cache(kind, n_pages, H, ps, hd, 1)
    _, plain = make_cache(kind, n_own, H, ps, hd, 2)            # every slot has its own pages, for good
    own_table = torch.arange(n_own, dtype=torch.int32).view(n_seq, max_pages).cuda()
    most = 256
    g = torch.Generator().manual_seed(3)
    q = torch.zeros((most, G * H, hd), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((most, H, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos, tok_start = torch.zeros(most, dtype=torch.int32, device="cuda"), ints([0] * (n_seq + 1))
    batch, own_batch = fr.PagedBatch(tok_start, pool.kv_len, two.table), fr.PagedBatch(tok_start, pool.kv_len, own_table)
    rope, w = fr.rope_params(hd), torch.rand(hd, generator=g).cuda() + 0.5
    ws, ws2 = (fr.make_paged_workspace(G * H, H, hd) for _ in range(2))
    q16, q16b = (torch.zeros((most * G * H, hd), dtype=torch.float16, device="cuda") for _ in range(2))
    out, out2 = (torch.zeros((most, G * H, hd), device="cuda") for _ in range(2))

    def step():
        fr.pages_trim(pool, window, sinks, tok_start)
        fr.pages_reserve(pool, tok_start)
        fr.pages_copy(cache, pool)
        fr.qkv_post_paged(cache, batch, q, k, v, pos, rope, q_norm=w, k_norm=w, q16_out=q16, workspace=ws)
        fr.paged_attn(cache, batch, q16, G * H, window=window, sinks=sinks, out=out, workspace=ws)
        fr.qkv_post_paged(plain, own_batch, q, k, v, pos, rope, q_norm=w, k_norm=w, q16_out=q16b, workspace=ws2)
        fr.paged_attn(plain, own_batch, q16b, G * H, window=window, sinks=sinks, out=out2, workspace=ws2)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rng = random.Random(5)
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(graph, stream=s):
            step()
        for turn in range(30):
            if turn in (4, 12, 20):
                empty = [b for b in range(n_seq) if not r.kv_len[b]]
                live = [b for b in range(n_seq) if r.kv_len[b]]
                child = empty[:3]
                parent = [rng.choice(live) for _ in child]
                length = [r.kv_len[p] for p in parent]
                r.fork(parent, child, length)
                fr.pages_fork(pool, ints(parent), ints(child), ints(length))
                for p, c in zip(parent, child):              # (copied in full beside it)
                    a, b = own_table[p].long(), own_table[c].long()
                    for t in (plain.k_pages, plain.v_pages, plain.k_scale, plain.v_scale):
                        if t is not None:
                            t[b] = t[a]
            if turn in (10, 18, 25):
                gone = [b for b in range(n_seq) if r.kv_len[b]][::2]
                r.free(gone)
                fr.pages_free(pool, ints(gone))
            if turn in (11, 22):
                r.compact()
                fr.pages_compact(pool)
                fr.pages_copy(cache, pool)
            new = [0] * n_seq
            for b in range(n_seq):
                if turn == 0 and b < 2 or turn == 15 and not r.kv_len[b]:
                    new[b] = 40 + 13 * b
                elif r.kv_len[b]:
                    new[b] = rng.choice([1, 1, 1, 0, 5])
            starts = [sum(new[:i]) for i in range(n_seq + 1)]
            r.kv_len = [n + a for n, a in zip(r.kv_len, new)]
            at = [p for a, n in zip(new, r.kv_len) for p in range(n - a, n)]
            for t in (q, k, v):
                t.copy_(torch.randn(t.shape, generator=g))
            pos[:len(at)] = ints(at)
            tok_start.copy_(ints(starts))
            pool.kv_len.copy_(ints(r.kv_len))
            graph.replay()
            s.synchronize()
            r.trim(window, sinks, starts)
            r.reserve(starts)
            two.compare(f"turn {turn}", moves=True)
            n = starts[-1]
            assert torch.equal(q16[:n * G * H], q16b[:n * G * H])
            # same keys in other pages: the same sums, in f16 bit by bit; e4m3 scales and the work's
            # cuts are the same too, since lengths and pages' contents are
            assert torch.equal(out[:n], out2[:n]), f"turn {turn}"
    assert holds(r)
    fr.pages_check(pool)
    fr.workspace_check(ws)
    fr.workspace_check(ws2)
