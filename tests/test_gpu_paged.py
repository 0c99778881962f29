"""The paged cache on the GPU: fr_kv_append_paged and fr_paged_attn against plain
64-bit forms (paged_ref.py), with tolerances from the arithmetic, over types,
head dims, groups, page sizes, uneven lengths (none, one, page and tile edges),
windows, strides, masked and unused places that hold infinities or NaN, bad
page tables, streams, captured graphs, and both operators as a step runs them."""
import numpy as np
import pytest
import torch

import gqa_kv_head_gb300 as fr
import paged_ref as ref

pytestmark = pytest.mark.gpu

TYPES = ["f16", "e4m3"]


def make_cache(kind, n_pages, H, ps, hd, seed=0, nhd=False):
    """Random pages (CPU) and their device copies: (cpu pages/scales, PagedKV)."""
    g = torch.Generator().manual_seed(seed)
    cpu, dev = [], []
    for which in range(2):
        x = torch.randn((n_pages, H, ps, hd), generator=g)
        if which == 0:
            x[..., ::31] *= 4.0
        if kind == "f16":
            p, s = x.half(), None
        else:
            x *= torch.exp2(torch.randint(-3, 4, (n_pages, H, 1, 1), generator=g).float())
            amax = x.abs().amax(dim=(2, 3))
            s = torch.tensor([[ref.pow2_scale(float(a)) for a in r] for r in amax])
            p = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        d = p.cuda()
        if nhd:                                       # [n_pages, page_size, n_kv_head, hd] pool
            d = d.transpose(1, 2).contiguous().transpose(1, 2)
        cpu += [p, s]
        dev += [d, None if s is None else s.cuda()]
    return tuple(cpu), fr.PagedKV(dev[0], dev[2], dev[1], dev[3])


def make_tables(kv_len, ps, n_pages, seed=0, fill=-1):
    need = [-(-n // ps) for n in kv_len]
    assert sum(need) <= n_pages
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).int()
    t = torch.full((len(kv_len), max(1, max(need))), fill, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def starts(new):
    return [0] + list(np.cumsum(new))


def make_batch(new, kv_len, table):
    return fr.PagedBatch(torch.tensor(starts(new), dtype=torch.int32).cuda(),
                         torch.tensor(kv_len, dtype=torch.int32).cuda(), table.cuda())


def rand_q(n_tok, n_head, hd, seed=1, scale=None):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n_tok, n_head, hd), generator=g) * (hd ** -0.5 if scale is None else scale)).half()


def check(got, want, tol, what=""):
    d = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = float((d / tol.clamp(min=1e-30)).max()) if d.numel() else 0.0
    assert bool((d <= tol + 1e-37).all()), f"{what}: {worst:.2f} times the tolerance, max {float(d.max()):.3e}"


def run_case(kind, hd, H, G, ps, new, kv_len, seed=0, nhd=False, **kw):
    n_pages = sum(-(-n // ps) for n in kv_len) + 2
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, seed, nhd)
    table = make_tables(kv_len, ps, n_pages, seed)
    q = rand_q(sum(new), H * G, hd, seed + 1)
    out = fr.paged_attn(cache, make_batch(new, kv_len, table), q.cuda(), H * G, **kw)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), starts(new), kv_len, table, H * G,
                              v_scale=vs, **kw)
    check(out, want, tol, f"{kind} hd{hd} H{H} G{G} ps{ps} {kw}")
    return out


# ---- attention --------------------------------------------------------------

LENS = [1, 2, 15, 16, 17, 31, 63, 64, 65, 100, 129, 300]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(1, 1), (4, 1), (8, 1), (7, 2), (5, 3), (4, 8), (16, 3)])
def test_attention_head_layouts(kind, hd, G, n):
    """Every row-tile width (8, 16, 32 rows; more rows than one tile) at every head dim."""
    run_case(kind, hd, 2, G, 32, [n] * len(LENS), [max(n, x) for x in LENS], seed=hd + G)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps", [16, 64, 128, 256])
@pytest.mark.parametrize("nhd", [False, True])
def test_attention_page_sizes_and_layouts(kind, ps, nhd):
    run_case(kind, 128, 3, 2, ps, [1] * len(LENS), LENS, seed=ps, nhd=nhd)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=5), dict(window=16), dict(window=100),
                                dict(window=100000), dict(window=2 ** 31 - 1), dict(kq_scale=0.37), dict(causal=False, kq_scale=-2.0)],
                         ids=lambda k: "_".join(f"{a}{b}" for a, b in k.items()))
@pytest.mark.parametrize("n", [1, 4])
def test_attention_masks(kind, kw, n):
    run_case(kind, 128, 2, 3, 16, [n] * len(LENS), [max(n, x) for x in LENS], seed=3, **kw)


@pytest.mark.parametrize("kind", TYPES)
def test_uneven_tokens_and_empty_sequences(kind):
    """Sequences without new tokens, without keys, with more tokens than keys
    (their first rows see nothing and are 0), and one token beside forty."""
    new = [0, 3, 1, 0, 40, 2, 1, 5]
    kv = [0, 3, 0, 50, 75, 1, 200, 2]
    run_case(kind, 128, 2, 4, 16, new, kv, seed=6, window=2 ** 31 - 1)
    run_case(kind, 128, 2, 4, 16, new, kv, seed=7, window=3)
    out = run_case(kind, 128, 2, 4, 16, new, kv, seed=5)
    s = starts(new)
    assert not out[s[2]].any()                       # no keys
    assert not out[s[5]].any() and out[s[5] + 1].any()
    assert not out[s[7]:s[7] + 3].any() and out[s[7] + 3:].any()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd,G,n,kv", [(128, 4, 1, 30000), (256, 8, 4, 9000), (64, 3, 2, 20011)])
def test_one_long_sequence(kind, hd, G, n, kv):
    """One segment split over every CTA, merged from many states."""
    run_case(kind, hd, 1, G, 64, [n], [kv], seed=7)


@pytest.mark.parametrize("kind", TYPES)
def test_many_sequences(kind):
    """More sequences than threads of a block: the list of units is found in several steps."""
    rng = np.random.default_rng(11)
    kv = [int(x) for x in rng.integers(1, 90, 400)]
    new = [int(min(a, b)) for a, b in zip(rng.integers(0, 3, 400), kv)]
    run_case(kind, 64, 2, 2, 16, new, kv, seed=11)


@pytest.mark.parametrize("kind", TYPES)
def test_long_beside_short(kind):
    run_case(kind, 128, 2, 4, 64, [1] * 40, [17] * 39 + [12000], seed=13)


def test_strided_q_padding_rows_and_given_buffers():
    """q16 as columns of a wider buffer; rows behind the last sequence keep what
    the output held; a page table with a wider row stride."""
    hd, H, G, ps, new, kv = 128, 2, 4, 16, [1, 2], [40, 33]
    (k, ks, v, vs), cache = make_cache("f16", 8, H, ps, hd)
    table = make_tables(kv, ps, 8)
    wide = torch.full((2, 7), -5, dtype=torch.int32)
    wide[:, :3] = table
    qw = torch.full((5, H * G * hd + 64), 7.0, dtype=torch.float16)
    q = rand_q(5, H * G, hd)
    qw[:, :H * G * hd] = q.reshape(5, -1)
    qd = qw.cuda()[:, :H * G * hd].unflatten(1, (H * G, hd))
    out = torch.full((5, H * G, hd), -3.0, device="cuda")
    batch = fr.PagedBatch(torch.tensor(starts(new), dtype=torch.int32).cuda(), torch.tensor(kv, dtype=torch.int32).cuda(),
                          wide.cuda()[:, :3])
    ws = fr.make_paged_workspace(H * G, H, hd)
    got = fr.paged_attn(cache, batch, qd, H * G, out=out, workspace=ws)
    assert got is out
    want, tol = ref.attention(q, k.double(), v.double(), starts(new), kv, table, H * G, out=torch.full_like(out.cpu(), -3.0))
    check(out, want, tol)
    assert (out[3:] == -3.0).all()
    fr.workspace_check(ws)


@pytest.mark.parametrize("kind", TYPES)
def test_places_out_of_view_do_not_reach_the_result(kind):
    """Rows of a page behind the sequence's end, pages of nobody, and keys that
    a query row's mask leaves out hold NaN and infinities."""
    hd, H, G, ps = 128, 2, 3, 32
    new, kv = [4, 1, 2], [50, 33, 64]
    n_pages = 8
    (k, ks, v, vs), _ = make_cache(kind, n_pages, H, ps, hd, 17)
    table = make_tables(kv, ps, n_pages, 17)
    clean = (k.clone(), v.clone())
    junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 448.0])
    dirty = [k.clone(), v.clone()]
    used = torch.zeros((n_pages, ps), dtype=torch.bool)
    for b, n in enumerate(kv):
        for j in range(n):
            used[table[b, j // ps], j % ps] = True
    for d in dirty:
        raw = torch.int16 if kind == "f16" else torch.uint8
        bits = junk.to(d.dtype).view(raw)[torch.arange(int((~used).sum())) % 4]
        for h in range(H):
            d.view(raw)[:, h][~used] = bits[:, None].expand(-1, hd)
    # the last new token of sequence 0: seen by its own row only
    page, row = int(table[0, 49 // ps]), 49 % ps
    dirty[1].view(raw)[page, :, row] = junk.to(dirty[1].dtype).view(raw)[0]
    sc = [None, None] if ks is None else [ks.cuda(), vs.cuda()]
    cache = fr.PagedKV(dirty[0].cuda(), dirty[1].cuda(), *sc)
    q = rand_q(sum(new), H * G, hd, 18)
    out = fr.paged_attn(cache, make_batch(new, kv, table), q.cuda(), H * G)
    want, tol = ref.attention(q, ref.values(clean[0], ks), ref.values(clean[1], vs), starts(new), kv, table, H * G)
    assert torch.isnan(out[3]).all()
    keep = [0, 1, 2, 4, 5, 6]
    check(out[keep], want[keep], tol[keep])


def test_visible_nan_reaches_its_rows_only():
    hd, H, G, ps = 64, 1, 2, 16
    (k, _, v, _), _ = make_cache("f16", 4, H, ps, hd, 3)
    table = torch.tensor([[0, 1, 2], [3, 0, 0]], dtype=torch.int32)
    k[0, 0, 5, 7] = float("nan")
    cache = fr.PagedKV(k.cuda(), v.cuda())
    q = rand_q(2, G, hd)
    out = fr.paged_attn(cache, make_batch([1, 1], [40, 12], table), q.cuda(), G)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    k[0, 0, 5, 7] = 1.0
    cache = fr.PagedKV(torch.full_like(k, float("nan")).cuda(), v.cuda())
    out = fr.paged_attn(cache, make_batch([1, 1], [40, 12], table), q.cuda(), G)
    assert torch.isnan(out).all()                     # every score NaN


def test_large_scores_and_ties():
    """Scores far apart (the weights of all but one key vanish) and all equal."""
    hd, H, G, ps, kv = 128, 1, 4, 16, [100]
    (k, _, v, _), cache = make_cache("f16", 8, H, ps, hd, 23)
    table = make_tables(kv, ps, 8, 23)
    q = rand_q(1, G, hd, 24, scale=8.0)
    out = fr.paged_attn(cache, make_batch([1], kv, table), q.cuda(), G)
    want, tol = ref.attention(q, k.double(), v.double(), [0, 1], kv, table, G)
    check(out, want, tol)
    z = torch.zeros_like(q)
    out = fr.paged_attn(cache, make_batch([1], kv, table), z.cuda(), G)
    want, tol = ref.attention(z, k.double(), v.double(), [0, 1], kv, table, G)
    check(out, want, tol)


def test_e4m3_scales_of_any_size():
    """V scales from 2^-60 to 2^60 in one sequence, zero scales, negative and
    other than powers of two: the definition holds for any finite scale."""
    hd, H, G, ps, kv = 128, 2, 4, 16, [160, 37]
    (k, ks, v, vs), _ = make_cache("e4m3", 16, H, ps, hd, 29)
    table = make_tables(kv, ps, 16, 29)
    g = torch.Generator().manual_seed(30)
    vs = torch.exp2(torch.randint(-60, 61, vs.shape, generator=g).float()) * 1.3
    vs[:, 1] = -vs[:, 1]
    vs[table[0, 1].long()] = 0.0
    ks = ks * 0.7
    cache = fr.PagedKV(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    q = rand_q(2, H * G, hd, 31)
    out = fr.paged_attn(cache, make_batch([1, 1], kv, table), q.cuda(), H * G)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), [0, 1, 2], kv, table, H * G)
    check(out, want, tol)
    zero = fr.PagedKV(k.cuda(), v.cuda(), ks.cuda(), torch.zeros_like(vs).cuda())
    assert not fr.paged_attn(zero, make_batch([1, 1], kv, table), q.cuda(), H * G).any()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps,n,window", [(16, 1, 40), (16, 3, 16), (32, 2, 50), (64, 1, 1)])
def test_pages_behind_the_window_may_be_gone(kind, ps, n, window):
    """Table entries of pages that no row sees are not used: nothing is
    reported, and what other sequences keep in such pages does not matter."""
    hd, H, G = 128, 2, 4
    kv = [1000, 77, 16, 300 + n]
    n_pages = sum(-(-x // ps) for x in kv) + 2
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 83)
    table = make_tables(kv, ps, n_pages, 83)
    q = rand_q(n * len(kv), H * G, hd, 84)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), starts([n] * len(kv)), kv, table, H * G, window=window)
    gone = table.clone()
    for b, x in enumerate(kv):
        first = max(0, x - n + 1 - window)
        gone[b, :first // ps] = torch.tensor([-1, n_pages, 2 ** 31 - 1], dtype=torch.int32)[torch.arange(first // ps) % 3]
    ws = fr.make_paged_workspace(H * G, H, hd)
    out = fr.paged_attn(cache, make_batch([n] * len(kv), kv, gone), q.cuda(), H * G, window=window, workspace=ws)
    check(out, want, tol)
    fr.workspace_check(ws)


@pytest.mark.parametrize("kind", TYPES)
def test_shared_prefix_pages(kind):
    hd, H, G, ps, kv = 128, 2, 4, 16, [40, 45, 33]
    (k, ks, v, vs), cache = make_cache(kind, 8, H, ps, hd, 37)
    table = torch.tensor([[0, 1, 2], [0, 1, 3], [0, 1, 4]], dtype=torch.int32)
    q = rand_q(3, H * G, hd, 38)
    out = fr.paged_attn(cache, make_batch([1] * 3, kv, table), q.cuda(), H * G)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), [0, 1, 2, 3], kv, table, H * G)
    check(out, want, tol)


@pytest.mark.parametrize("kind", TYPES)
def test_bad_tables_and_lengths_are_reported(kind):
    """A page outside the pool masks its keys, a length beyond the table or a
    token range outside the rows skips its sequence; the others are right, and
    the status word tells."""
    hd, H, G, ps = 128, 2, 2, 16
    n_pages = 12
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 41)
    kv = [40, 40, 40]
    table = make_tables(kv, ps, n_pages, 41)
    q = rand_q(3, H * G, hd, 42)
    ws = fr.make_paged_workspace(H * G, H, hd)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), [0, 1, 2, 3], kv, table, H * G)
    for bad_page in (-1, n_pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 1] = bad_page
        out = fr.paged_attn(cache, make_batch([1] * 3, kv, t), q.cuda(), H * G, workspace=ws)
        with pytest.raises(fr.FrError) as e:
            fr.workspace_check(ws)
        assert e.value.status == 6
        fr.workspace_check(ws)
        check(out[[0, 2]], want[[0, 2]], tol[[0, 2]])
        # keys 16..31 masked: the same as a sequence that holds the others only
        kk, vv = ref.values(k, ks), ref.values(v, vs)
        two = torch.tensor([[table[1, 0], table[1, 2]]])
        w1, t1 = ref.attention(q[1:2], kk, vv, [0, 1], [24], two, H * G)
        check(out[1:2], w1, t1)
    for lens in ([40, -1, 40], [40, 49, 40], [40, 2 ** 31 - 1, 40]):
        out = torch.full((3, H * G, hd), 9.0, device="cuda")
        fr.paged_attn(cache, make_batch([1] * 3, lens, table), q.cuda(), H * G, out=out, workspace=ws)
        with pytest.raises(fr.FrError):
            fr.workspace_check(ws)
        check(out[[0, 2]], want[[0, 2]], tol[[0, 2]])
        assert (out[1] == 9.0).all()
    out = torch.full((3, H * G, hd), 9.0, device="cuda")
    b = fr.PagedBatch(torch.tensor([0, 1, -7, 3], dtype=torch.int32).cuda(), torch.tensor(kv, dtype=torch.int32).cuda(),
                      table.cuda())
    fr.paged_attn(cache, b, q.cuda(), H * G, out=out, workspace=ws)
    with pytest.raises(fr.FrError):
        fr.workspace_check(ws)
    check(out[:1], want[:1], tol[:1])


def test_same_inputs_same_bits_and_two_streams():
    hd, H, G, ps = 128, 4, 4, 64
    kv = [3000, 5, 700, 1800]
    n_pages = 100
    _, cache = make_cache("f16", n_pages, H, ps, hd, 43)
    batch = make_batch([1] * 4, kv, make_tables(kv, ps, n_pages, 43))
    q = rand_q(4, H * G, hd, 44).cuda()
    first = fr.paged_attn(cache, batch, q, H * G)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [fr.make_paged_workspace(H * G, H, hd) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for st, ws in zip(streams, spaces):
            outs.append(fr.paged_attn(cache, batch, q, H * G, workspace=ws, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("kind", TYPES)
def test_graph_follows_the_lengths(kind):
    """One captured append + attention step, replayed as the lengths, tables and
    rows in its buffers change."""
    hd, H, G, ps, n_pages = 128, 2, 4, 16, 24
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 47)
    kv_steps = [[20, 1, 47], [21, 2, 48], [22, 3, 49], [90, 80, 140]]
    table = make_tables([96, 96, 144], ps, n_pages, 47)
    kv_d = torch.tensor(kv_steps[0], dtype=torch.int32).cuda()
    batch = fr.PagedBatch(torch.tensor([0, 1, 2, 3], dtype=torch.int32).cuda(), kv_d, table.cuda())
    rope = fr.rope_params(hd)
    q_d = rand_q(3, H * G, hd, 48).cuda()
    kn, vn = torch.randn(3, H, hd).cuda(), torch.randn(3, H, hd).cuda()
    pos = torch.zeros(3, dtype=torch.int32).cuda()
    out = torch.empty((3, H * G, hd), device="cuda")
    ws = fr.make_paged_workspace(H * G, H, hd)

    def step():
        fr.kv_append_paged(cache, batch, kn, vn, pos, rope, workspace=ws)
        fr.paged_attn(cache, batch, q_d, H * G, out=out, workspace=ws)
    save = [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8))]
    sc = None if ks is None else [cache.k_scale.clone(), cache.v_scale.clone()]
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
    torch.cuda.synchronize()
    cache.k_pages.view(torch.uint8).copy_(save[0])
    cache.v_pages.view(torch.uint8).copy_(save[1])
    if sc:
        cache.k_scale.copy_(sc[0])
        cache.v_scale.copy_(sc[1])
    for i, kv in enumerate(kv_steps):
        g = torch.Generator().manual_seed(100 + i)
        q = rand_q(3, H * G, hd, 200 + i)
        a, b = torch.randn((3, H, hd), generator=g), torch.randn((3, H, hd), generator=g)
        kv_d.copy_(torch.tensor(kv, dtype=torch.int32))
        q_d.copy_(q)
        kn.copy_(a)
        vn.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        k, v, ks, vs = ref.append(a, b, [0, 1, 2, 3], kv, table, k, v, ks, vs)      # position 0: no rotation
        assert ref.same_bits(cache.k_pages.cpu(), k) and ref.same_bits(cache.v_pages.cpu(), v)
        want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), [0, 1, 2, 3], kv, table, H * G)
        check(out, want, tol, f"replay {i}")
    fr.workspace_check(ws)


def test_pages_beyond_32_bit_offsets():
    """A pool of more than 2^32 elements, its last pages in use."""
    hd, H, ps, G = 256, 8, 256, 2
    n_pages = 2 ** 32 // (hd * H * ps) + 9
    k = torch.empty((n_pages, H, ps, hd), dtype=torch.float16, device="cuda")
    v = torch.empty((n_pages, H, ps, hd), dtype=torch.float16, device="cuda")
    (ks, _, vs, _), _ = make_cache("f16", 4, H, ps, hd, 53)
    last = torch.tensor([n_pages - 1, 0, n_pages - 4, n_pages - 7])
    k[last.cuda()] = ks.cuda()
    v[last.cuda()] = vs.cuda()
    cache = fr.PagedKV(k, v)
    kv, new = [500, 300], [1, 1]
    table = last.view(2, 2).int()
    batch = make_batch(new, kv, table)
    rows = torch.randn((2, H, hd), generator=torch.Generator().manual_seed(54))
    fr.kv_append_paged(cache, batch, rows.cuda(), rows.cuda(), torch.zeros(2, dtype=torch.int32).cuda(), fr.rope_params(hd))
    small = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    ek, ev, _, _ = ref.append(rows, rows, [0, 1, 2], kv, small, ks, vs)
    assert torch.equal(k[last.cuda()].cpu(), ek) and torch.equal(v[last.cuda()].cpu(), ev)
    q = rand_q(2, H * G, hd, 55)
    out = fr.paged_attn(cache, batch, q.cuda(), H * G)
    want, tol = ref.attention(q, ek.double(), ev.double(), [0, 1, 2], kv, small, H * G)
    check(out, want, tol)


def test_agrees_with_the_contiguous_operators():
    """One sequence, one KV head, pages in order: fr_decode_attn on the same keys."""
    hd, G, ps, n = 256, 8, 64, 4
    kv = 1000
    (k, _, v, _), cache = make_cache("f16", 16, 1, ps, hd, 59)
    table = torch.arange(16, dtype=torch.int32)[None]
    q = rand_q(n, G, hd, 60)
    mask = torch.zeros((n, 1024), dtype=torch.float16)
    for i in range(n):
        mask[i, kv - n + i + 1:] = float("-inf")
    a = fr.paged_attn(cache, make_batch([n], [kv], table), q.cuda(), G)
    b = fr.decode_attn(k.reshape(-1, hd).cuda(), v.reshape(-1, hd).cuda(), n, G, q16=q.reshape(-1, hd).cuda(), mask=mask.cuda())
    _, tol = ref.attention(q, k.double(), v.double(), [0, n], [kv], table, G)
    check(a, b.double().cpu(), 2 * tol)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd,H,G,n", [(256, 1, 8, 300), (128, 2, 4, 200), (64, 1, 16, 130)])
def test_many_query_rows(kind, hd, H, G, n):
    """A prompt's rows: many row tiles, each over its own keys."""
    run_case(kind, hd, H, G, 64, [n, 1, n // 3], [n + 50, 20, n // 3], seed=hd, window=0)
    run_case(kind, hd, H, G, 16, [n], [n + 7], seed=hd + 1, window=33)


def test_more_sequences_than_threads_of_large_blocks():
    rng = np.random.default_rng(19)
    kv = [int(x) for x in rng.integers(0, 40, 700)]
    new = [int(min(a, b)) for a, b in zip(rng.integers(0, 4, 700), kv)]
    run_case("f16", 256, 1, 8, 16, new, kv, seed=19)


@pytest.mark.parametrize("kind", TYPES)
def test_nothing_else_is_written(kind):
    """Margins around the output and the workspace, and the cache itself, stay as they were."""
    hd, H, G, ps = 128, 2, 4, 16
    kv, new = [300, 7, 1000], [2, 1, 1]
    n_pages = 90
    _, cache = make_cache(kind, n_pages, H, ps, hd, 73)
    before = [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8))]
    n = 4 * H * G * hd
    out = torch.full((n + 4096,), 5.0, device="cuda")
    size = fr.paged_attn_workspace_size(H * G, H, hd)
    ws = torch.full((size + 8192,), 171, dtype=torch.uint8, device="cuda")
    ws[4096:4096 + size] = 0
    fr.paged_attn(cache, make_batch(new, kv, make_tables(kv, ps, n_pages, 73)), rand_q(4, H * G, hd, 74).cuda(), H * G,
                  out=out[2048:2048 + n].view(4, H * G, hd), workspace=ws[4096:4096 + size])
    torch.cuda.synchronize()
    assert (out[:2048] == 5.0).all() and (out[2048 + n:] == 5.0).all()
    assert (ws[:4096] == 171).all() and (ws[4096 + size:] == 171).all()
    assert torch.equal(cache.k_pages.view(torch.uint8), before[0]) and torch.equal(cache.v_pages.view(torch.uint8), before[1])


def test_two_graphs_share_a_workspace():
    """Captured with one workspace and replayed in turn on one stream."""
    hd, H, G, ps, n_pages = 128, 2, 8, 64, 60
    (k, _, v, _), cache = make_cache("f16", n_pages, H, ps, hd, 79)
    ws = fr.make_paged_workspace(H * G, H, hd)
    cases = []
    for i, (new, kv) in enumerate((([1], [3500]), ([2, 1, 1], [100, 900, 40]))):
        table = make_tables(kv, ps, n_pages, 80 + i)
        q = rand_q(sum(new), H * G, hd, 82 + i)
        want, tol = ref.attention(q, k.double(), v.double(), starts(new), kv, table, H * G)
        qd, batch = q.cuda(), make_batch(new, kv, table)
        out = fr.paged_attn(cache, batch, qd, H * G, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fr.paged_attn(cache, batch, qd, H * G, out=out, workspace=ws)
        cases.append((graph, out, want, tol, qd, batch))
    for _ in range(3):
        for graph, out, *_ in cases:
            out.fill_(float("nan"))
            graph.replay()
    torch.cuda.synchronize()
    for _, out, want, tol, *_ in cases:
        check(out, want, tol)


def test_refusals():
    """What the calls refuse, before anything is launched."""
    hd, H, G, ps = 128, 2, 4, 16
    _, cache = make_cache("f16", 4, H, ps, hd)
    _, cache8 = make_cache("e4m3", 4, H, ps, hd)
    table = make_tables([20, 20], ps, 4)
    batch = make_batch([1, 1], [20, 20], table)
    q = rand_q(2, H * G, hd).cuda()
    ws = fr.make_paged_workspace(H * G, H, hd)

    def status(f, want):
        with pytest.raises(fr.FrError) as e:
            f()
        assert e.value.status == want
    for bad in (dict(window=-1), dict(window=4, causal=False), dict(kq_scale=float("nan")), dict(kq_scale=float("inf")),
                dict(kq_scale=3e38)):
        status(lambda: fr.paged_attn(cache, batch, q, H * G, workspace=ws, **bad), 1)
    status(lambda: fr.paged_attn(cache, batch, q, H * G, workspace=ws[:1024]), 3)
    status(lambda: fr.paged_attn(cache, batch, q[:, :7].contiguous(), 7, workspace=ws), 1)       # 7 heads on 2
    for bad in (q.float(), q.bfloat16()):
        with pytest.raises(TypeError):
            fr.paged_attn(cache, batch, bad, H * G)
    for bad in (q[..., :64], q.transpose(0, 1), q.view(2, -1)[:, :-8]):
        with pytest.raises(ValueError):
            fr.paged_attn(cache, batch, bad, H * G)
    with pytest.raises(ValueError):
        fr.paged_attn(cache, batch, q, H * G, out=torch.empty((2, H * G, hd + 1), device="cuda"))
    with pytest.raises(ValueError):
        fr.paged_attn(cache, batch, q, H * G, out=torch.empty((2, H * G, hd), dtype=torch.float16, device="cuda"))
    wide = torch.zeros(2, H * G * hd + 4, dtype=torch.float16, device="cuda")[:, :H * G * hd].unflatten(1, (H * G, hd))
    status(lambda: fr.paged_attn(cache, batch, wide, H * G, workspace=ws), 1)                    # token stride of 8 bytes more

    rows = torch.zeros((2, H, hd), device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    rope = fr.rope_params(hd)
    fr.kv_append_paged(cache8, batch, rows, rows, pos, rope)
    for bad in (fr.rope_params(127), fr.rope_params(256), fr.rope_params(128, freq_base=-1.0)):
        status(lambda: fr.kv_append_paged(cache, batch, rows, rows, pos, bad), 1)
    for a, b in ((rows.half(), rows), (rows.double(), rows.double()), (rows.bfloat16(), rows.bfloat16())):
        with pytest.raises(TypeError):
            fr.kv_append_paged(cache, batch, a, b, pos, rope)
    with pytest.raises(TypeError):
        fr.kv_append_paged(cache, batch, rows, rows, pos.long(), rope)
    for a, p in ((rows[:, :1], pos), (rows[..., :64], pos), (rows, pos[:1]), (rows.transpose(0, 1), pos)):
        with pytest.raises(ValueError):
            fr.kv_append_paged(cache, batch, a, a, p, rope)
    k = cache.k_pages
    with pytest.raises(TypeError):
        fr.PagedKV(k.float(), k.float())
    with pytest.raises(TypeError):
        fr.PagedKV(k, cache8.k_pages)
    with pytest.raises(ValueError):
        fr.PagedKV(k, k[:2])
    with pytest.raises(ValueError):
        fr.PagedKV(k, k, cache8.k_scale, cache8.v_scale)
    with pytest.raises(ValueError):
        fr.PagedKV(cache8.k_pages, cache8.v_pages)
    with pytest.raises(ValueError):
        fr.PagedKV(cache8.k_pages, cache8.v_pages, cache8.k_scale[:2], cache8.v_scale)
    status(lambda: fr.PagedKV(k[:, :, :12], k[:, :, :12]), 2)
    status(lambda: fr.PagedKV(k[:1].expand(4, -1, -1, -1), k), 1)                                # one page four times
    with pytest.raises(TypeError):
        fr.PagedBatch(batch.tok_start.long(), batch.kv_len, batch.page_table)
    with pytest.raises(ValueError):
        fr.PagedBatch(batch.tok_start[:2], batch.kv_len, batch.page_table)
    with pytest.raises(ValueError):
        fr.PagedBatch(batch.tok_start, batch.kv_len, batch.page_table.t().contiguous().t())
    torch.cuda.synchronize()


# ---- append -----------------------------------------------------------------

def rotated_rows(k_new, pos, rope):
    """The f32 rows fr_kv_append rounds from, one call a head (bit-exact arithmetic shared by both)."""
    n_tok, H, hd = k_new.shape
    out = torch.empty((n_tok, H, hd), dtype=torch.float32)
    for h in range(H):
        kc = torch.zeros((n_tok, hd), dtype=torch.float16, device="cuda")
        k32 = torch.empty((n_tok, hd), dtype=torch.float32, device="cuda")
        v32 = torch.empty_like(k32)
        x = k_new[:, h].float().contiguous().cuda()
        fr.kv_append(x, x, pos.cuda(), rope, kc, torch.zeros_like(kc), 0, k32_out=k32, v32_out=v32)
        out[:, h] = k32.cpu()
    return out


APPEND_NEW = [1, 0, 3, 16, 17, 40, 70, 1]
APPEND_KV = [1, 5, 3, 33, 17, 75, 70, 48]


def run_append(kind, hd, H, ps, new, kv, rope, rows="f32", seed=0, nhd=False, fused=False, k_rows=None, v_rows=None):
    n_pages = sum(-(-n // ps) for n in kv) + 3
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, seed, nhd)
    table = make_tables(kv, ps, n_pages, seed)
    g = torch.Generator().manual_seed(seed + 1)
    n_tok = sum(new)
    dt = torch.float32 if rows == "f32" else torch.float16
    a = torch.randn((n_tok, H, hd), generator=g).to(dt) if k_rows is None else k_rows
    b = (3 * torch.randn((n_tok, H, hd), generator=g)).to(dt) if v_rows is None else v_rows
    pos = torch.randint(0, 100000, (n_tok,), generator=g).int()
    if fused:
        qkv = torch.zeros((n_tok, 4 * H * hd), dtype=dt)
        qkv[:, 2 * H * hd:3 * H * hd], qkv[:, 3 * H * hd:] = a.reshape(n_tok, -1), b.reshape(n_tok, -1)
        d = qkv.cuda()
        da, db = (d[:, i * H * hd:(i + 1) * H * hd].unflatten(1, (H, hd)) for i in (2, 3))
    else:
        da, db = a.cuda(), b.cuda()
    fr.kv_append_paged(cache, make_batch(new, kv, table), da, db, pos.cuda(), rope)
    torch.cuda.synchronize()
    ek, ev, eks, evs = ref.append(rotated_rows(a, pos, rope), b.float(), starts(new), kv, table, k, v, ks, vs)
    assert ref.same_bits(cache.k_pages.cpu(), ek), "K pages"
    assert ref.same_bits(cache.v_pages.cpu(), ev), "V pages"
    if kind == "e4m3":
        assert torch.equal(cache.k_scale.cpu(), eks) and torch.equal(cache.v_scale.cpu(), evs), "scales"


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("rows", ["f32", "f16"])
def test_append(kind, hd, rows):
    """Pages start, go on, end and grow their scales; every other byte of the pool is untouched."""
    run_append(kind, hd, 3, 16, APPEND_NEW, APPEND_KV, fr.rope_params(hd), rows, seed=hd)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps,H", [(32, 1), (64, 8), (128, 5), (256, 2)])
def test_append_page_sizes(kind, ps, H):
    """Up to pages whose rows a block does not keep in registers; fused QKV rows; head pairs and a head left over."""
    run_append(kind, 128, H, ps, APPEND_NEW + [600], APPEND_KV + [700], fr.rope_params(128), seed=ps, nhd=ps == 64, fused=True)


@pytest.mark.parametrize("kind", TYPES)
def test_append_many_heads_share_angles(kind):
    run_append(kind, 256, 5, 128, [300, 500, 900], [400, 500, 1500], fr.rope_params(256), seed=2, fused=True)
    run_append(kind, 64, 8, 16, [700, 300], [700, 800], fr.rope_params(64), "f16", seed=3)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rope", [dict(n_dims=64), dict(n_dims=20), dict(n_dims=2), dict(n_dims=126),
                                  dict(n_dims=128, mode=1), dict(n_dims=128, ext_factor=1.0, freq_scale=0.25),
                                  dict(n_dims=128, freq_factors=[1.0 + i / 64 for i in range(64)], mode=1)],
                         ids=["half", "20", "2", "126", "ggml", "yarn", "factors"])
def test_append_rotations(kind, rope):
    """Partial rotation (also of dims that no vector covers), ggml's angles, YaRN, frequency factors."""
    run_append(kind, 128, 2, 16, APPEND_NEW, APPEND_KV, fr.rope_params(**rope), seed=4)


@pytest.mark.parametrize("kind", TYPES)
def test_append_many_sequences(kind):
    rng = np.random.default_rng(5)
    kv = [int(x) for x in rng.integers(1, 60, 300)]
    new = [int(min(a, b)) for a, b in zip(rng.integers(0, 4, 300), kv)]
    run_append(kind, 64, 2, 16, new, kv, fr.rope_params(64), seed=5)


def test_append_e4m3_values_and_scales_at_the_edges():
    """Zeros, subnormals, exact 448 * 2^k maxima and the value above, values
    beyond the range, infinities and NaN."""
    H, hd, ps = 1, 64, 16
    up = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9))
    tops = [0.0, 448.0, float(up), 447.0, 224.0, 1e-38, 1e-44, 3e38, 1.0, 2.0 ** -100, 1e-31]
    new = [1] * len(tops)
    kv = [1] * len(tops)
    rows = torch.zeros((len(tops), H, hd))
    for i, t in enumerate(tops):
        rows[i, 0, 0] = t
        rows[i, 0, 1:9] = t * torch.tensor([-1.0, 0.5, 0.3, 2.0 ** -7, -2.0 ** -15, 2.0 ** -17, 2.0 ** -18, 0.999])
    odd = rows.clone()
    odd[3, 0, 20], odd[4, 0, 21], odd[4, 0, 22] = float("nan"), float("inf"), -float("inf")
    rope = fr.rope_params(2)
    n_pages = 16
    (k, ks, v, vs), cache = make_cache("e4m3", n_pages, H, ps, hd, 6)
    table = make_tables(kv, ps, n_pages, 6)
    pos = torch.zeros(len(tops), dtype=torch.int32)
    fr.kv_append_paged(cache, make_batch(new, kv, table), rows.cuda(), odd.cuda(), pos.cuda(), rope)
    # (the rotation by 0 turns a -0 into +0)
    ek, ev, eks, evs = ref.append(rotated_rows(rows, pos, rope), odd, starts(new), kv, table, k, v, ks, vs)
    assert torch.equal(cache.k_scale.cpu(), eks) and torch.equal(cache.v_scale.cpu(), evs)
    for got, want in ((cache.k_pages.cpu(), ek), (cache.v_pages.cpu(), ev)):
        at = [(i, d) for i in range(len(tops)) for d in range(hd)
              if not ref.same_bits(got[table[i, 0], 0, 0, d:d + 1], want[table[i, 0], 0, 0, d:d + 1])]
        assert not at, at[:8]
        assert ref.same_bits(got, want)


def test_append_token_by_token_keeps_e4m3_precision():
    """A page filled token by token with growing values: the codes stay within
    one rounding at the final scale of the values (half a step of e4m3, 2^-4, or
    half its smallest step, plus the same for each growth below e4m3's
    normal range)."""
    H, hd, ps, n = 2, 128, 32, 32
    g = torch.Generator().manual_seed(8)
    rows = torch.randn((n, H, hd), generator=g) * torch.exp2(torch.linspace(-4, 6, n))[:, None, None]
    k = torch.zeros((1, H, ps, hd), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    sc = [torch.full((1, H), float("nan"), device="cuda") for _ in range(2)]
    cache = fr.PagedKV(k, v, *sc)
    kv_d = torch.zeros(1, dtype=torch.int32).cuda()
    batch = fr.PagedBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(), kv_d, torch.zeros((1, 1), dtype=torch.int32).cuda())
    for i in range(n):
        kv_d.fill_(i + 1)
        fr.kv_append_paged(cache, batch, rows[i:i + 1].cuda(), rows[i:i + 1].cuda(), torch.zeros(1, dtype=torch.int32).cuda(), fr.rope_params(hd))
    torch.cuda.synchronize()
    for pages, s in ((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale)):
        s = s.cpu()
        want = rows.permute(1, 0, 2)[None].double()
        for h in range(H):
            assert float(s[0, h]) == ref.pow2_scale(float(rows[:, h].abs().max()))
        got = ref.values(pages.cpu(), s)
        step = 2.0 ** -9 * s.double()[:, :, None, None]
        # at most 11 growths, each rounding to at most half the smallest step of its scale: their sum is below a whole one of the last
        assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 1.0 * step).all())


@pytest.mark.parametrize("kind", TYPES)
def test_append_bad_input_is_reported_and_writes_nothing(kind):
    hd, H, ps, n_pages = 128, 2, 16, 6
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 61)
    ws = fr.make_paged_workspace(H, H, hd)
    rows = torch.randn((3, H, hd), generator=torch.Generator().manual_seed(1))
    d = rows.cuda()
    pos = torch.zeros(3, dtype=torch.int32).cuda()
    good = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32)
    for table, kv in ((torch.tensor([[0, 1], [2, 77], [4, 5]], dtype=torch.int32), [20, 20, 20]),
                      (torch.tensor([[0, 1], [2, -1], [4, 5]], dtype=torch.int32), [20, 20, 20]),
                      (good, [20, 0, 20]), (good, [20, 33, 20]), (good, [20, -4, 20])):
        fr.kv_append_paged(cache, make_batch([1] * 3, kv, table), d, d, pos, fr.rope_params(hd), workspace=ws)
        with pytest.raises(fr.FrError) as e:
            fr.workspace_check(ws)
        assert e.value.status == 6
        k, v, ks, vs = ref.append(rows[[0, 2]], rows[[0, 2]], [0, 1, 2], [20, 20], good[[0, 2]], k, v, ks, vs)
        assert ref.same_bits(cache.k_pages.cpu(), k) and ref.same_bits(cache.v_pages.cpu(), v)
        fr.workspace_check(ws)
    fr.kv_append_paged(cache, make_batch([1] * 3, [20, 40, 20], good), d, d, pos, fr.rope_params(hd))      # without a workspace
    assert ref.same_bits(cache.k_pages.cpu(), k)


# ---- a run of steps -----------------------------------------------------------

@pytest.mark.parametrize("kind", TYPES)
def test_a_serving_run(kind):
    """Prompts, then decode steps of several sequences, one of them joining
    late and one leaving: append, qkv_post and attention on a side stream,
    every step against the 64-bit form over the cache as the reference fills it."""
    hd, H, G, ps, n_pages = 128, 2, 4, 16, 40
    n_head = H * G
    rope = fr.rope_params(hd, freq_base=500000.0)
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 71)
    table = make_tables([96, 160, 64], ps, n_pages, 71)
    steps = [([40, 100, 0], [40, 100, 0]), ([1, 1, 0], [41, 101, 0]), ([1, 2, 30], [42, 103, 30]), ([1, 1, 1], [43, 104, 31]),
             ([0, 1, 3], [43, 105, 34])]
    st = torch.cuda.Stream()
    ws = fr.make_paged_workspace(n_head, H, hd)
    torch.cuda.synchronize()
    for i, (new, kv) in enumerate(steps):
        n_tok = sum(new)
        g = torch.Generator().manual_seed(300 + i)
        qkv = torch.randn((n_tok, (n_head + 2 * H) * hd), generator=g)
        pos = torch.cat([torch.arange(b - a, b) for a, b in zip(new, kv)]).int()
        with torch.cuda.stream(st):
            d, p = qkv.cuda(), pos.cuda()
            batch = make_batch(new, kv, table)
            kn = d[:, n_head * hd:(n_head + H) * hd].unflatten(1, (H, hd))
            vn = d[:, (n_head + H) * hd:].unflatten(1, (H, hd))
            fr.kv_append_paged(cache, batch, kn, vn, p, rope, stream=st)
            q16, _ = fr.qkv_post(d, p, n_head, hd, rope)
            out = fr.paged_attn(cache, batch, q16, n_head, workspace=ws, stream=st)
        st.synchronize()
        kr = rotated_rows(qkv[:, n_head * hd:(n_head + H) * hd].unflatten(1, (H, hd)), pos, rope)
        vr = qkv[:, (n_head + H) * hd:].unflatten(1, (H, hd))
        k, v, ks, vs = ref.append(kr, vr, starts(new), kv, table, k, v, ks, vs)
        want, tol = ref.attention(q16.cpu().view(n_tok, n_head, hd), ref.values(k, ks), ref.values(v, vs), starts(new), kv, table, n_head)
        check(out, want, tol, f"step {i}")
    fr.workspace_check(ws)


# ---- many query rows (prompts, wide windows): the 128-row tiles --------------------

PROMPTS = ([70, 1, 129, 0, 300, 64, 33, 5], [70, 65, 129, 40, 300, 1000, 33, 3])     # (the last: more tokens than keys)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("H,G", [(2, 1), (2, 3), (1, 8), (1, 16), (1, 100)])
def test_prompt_head_layouts(kind, hd, H, G):
    new, kv = PROMPTS if G < 16 else ([x // 4 for x in PROMPTS[0]], PROMPTS[1])
    run_case(kind, hd, H, G, 32, new, kv, seed=hd + G)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps", [16, 64, 128, 256])
@pytest.mark.parametrize("nhd", [False, True])
def test_prompt_page_sizes_and_layouts(kind, ps, nhd):
    run_case(kind, 128, 2, 4, ps, *PROMPTS, seed=ps, nhd=nhd)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps", [16, 32, 256])
@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=50), dict(window=130),
                                dict(window=2 ** 31 - 1), dict(kq_scale=-1.5)],
                         ids=lambda k: "_".join(f"{a}{b}" for a, b in k.items()))
def test_prompt_masks(kind, ps, kw):
    run_case(kind, 128, 1, 5, ps, *PROMPTS, seed=3, **kw)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd,G,n,kv", [(128, 8, 16, 20000), (256, 4, 40, 9000), (64, 16, 9, 30011)])
def test_prompt_behind_a_long_cache(kind, hd, G, n, kv):
    """Few row tiles, split over every CTA."""
    run_case(kind, hd, 1, G, 64, [n], [kv], seed=7)


@pytest.mark.parametrize("kind", TYPES)
def test_prompts_of_many_sequences(kind):
    """More sequences than threads of a block; many segments to a CTA."""
    rng = np.random.default_rng(12)
    kv = [int(x) for x in rng.integers(1, 130, 400)]
    new = [int(min(a, b)) for a, b in zip(rng.integers(0, 30, 400), kv)]
    run_case(kind, 64, 2, 4, 16, new, kv, seed=12)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prompt_places_out_of_view(kind, hd):
    """Junk behind the sequences' ends, in V rows that only later tokens see (one
    row NaN, one infinite, in two places of a tile), and in pages of nobody: each
    row of the result has what its own view holds."""
    H, G, ps = 2, 4, 32
    new, kv = [100, 40], [150, 40]
    n_pages = 9
    (k, ks, v, vs), _ = make_cache(kind, n_pages, H, ps, hd, 17)
    table = make_tables(kv, ps, n_pages, 17)
    want, tol = ref.attention(rand_q(sum(new), H * G, hd, 18), ref.values(k, ks), ref.values(v, vs), starts(new), kv, table, H * G,
                              v_scale=vs)
    used = torch.zeros((n_pages, ps), dtype=torch.bool)
    for b, n in enumerate(kv):
        for j in range(n):
            used[table[b, j // ps], j % ps] = True
    sc = [None, None] if ks is None else [ks.cuda(), vs.cuda()]
    nan, inf = (0x7e00, 0x7c00) if kind == "f16" else (0x7f, 0x7f)       # (e4m3 has no infinity)
    kb, vb = (x.view(torch.int16 if kind == "f16" else torch.uint8) for x in (k, v))
    for d in (kb, vb):
        d.transpose(1, 2)[~used] = nan
    at = lambda b, j: (int(table[b, j // ps]), j % ps)
    p, r = at(0, 149)
    vb[p, :, r] = nan                           # seen by the last token only
    p, r = at(0, 130)
    vb[p, 1, r, 5] = inf                        # tokens from 80 on, head 1, one dim
    out = fr.paged_attn(fr.PagedKV(k.cuda(), v.cuda(), *sc), make_batch(new, kv, table), rand_q(sum(new), H * G, hd, 18).cuda(),
                        H * G)
    assert torch.isnan(out[99]).all()
    # (a weight is the sum of two f16 terms, the second of either sign or 0: infinity
    # times them is infinity or NaN)
    assert not torch.isfinite(out[80:99, G:, 5]).any()
    keep = torch.ones(out.shape, dtype=torch.bool)
    keep[99] = False
    keep[80:99, G:, 5] = False
    got = torch.where(keep, out.cpu().double(), want)
    check(got.float().where(keep, torch.zeros(())), want.where(keep, torch.zeros((), dtype=torch.float64)), tol)


@pytest.mark.parametrize("kind", TYPES)
def test_prompt_visible_nan_keys(kind):
    """A NaN key makes NaN of the rows that see it, and of no others."""
    hd, G, ps, n, kv = 128, 4, 16, 100, 120
    (k, ks, v, vs), _ = make_cache(kind, 8, 1, ps, hd, 3)
    table = make_tables([kv], ps, 8, 3)
    q = rand_q(n, G, hd)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), [0, n], [kv], table, G, v_scale=vs)
    sc = [None, None] if ks is None else [ks.cuda(), vs.cuda()]
    kb = k.view(torch.int16 if kind == "f16" else torch.uint8)
    kb[int(table[0, 90 // ps]), 0, 90 % ps, 7] = 0x7e00 if kind == "f16" else 0x7f
    out = fr.paged_attn(fr.PagedKV(k.cuda(), v.cuda(), *sc), make_batch([n], [kv], table), q.cuda(), G)
    assert torch.isnan(out[70:]).all()
    check(out[:70], want[:70], tol[:70])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps", [16, 32, 128])
def test_prompt_pages_behind_the_window_and_bad_pages(kind, ps):
    hd, H, G, window = 128, 1, 4, 70
    new, kv = [40, 30], [500, 300]
    n_pages = sum(-(-x // ps) for x in kv) + 2
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 83)
    table = make_tables(kv, ps, n_pages, 83)
    q = rand_q(sum(new), H * G, hd, 84)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), starts(new), kv, table, H * G, window=window,
                              v_scale=vs)
    gone = table.clone()
    for b in range(2):
        gone[b, :max(0, kv[b] - new[b] + 1 - window) // ps] = -1
    ws = fr.make_paged_workspace(H * G, H, hd)
    out = fr.paged_attn(cache, make_batch(new, kv, gone), q.cuda(), H * G, window=window, workspace=ws)
    check(out, want, tol)
    fr.workspace_check(ws)
    # a page that is in view and outside the pool: its keys are masked, and the status word tells
    first = kv[1] - 10                                   # (within the last page, or its tile)
    bad = table.clone()
    bad[1, first // ps] = n_pages
    out = fr.paged_attn(cache, make_batch(new, kv, bad), q.cuda(), H * G, workspace=ws)
    with pytest.raises(fr.FrError):
        fr.workspace_check(ws)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), starts(new), kv, table, H * G,
                              v_scale=vs)
    check(out[:40], want[:40], tol[:40])
    cut = first // ps * ps                               # tokens that see nothing of that page
    before = max(0, cut - (kv[1] - new[1]))
    check(out[40:40 + before], want[40:40 + before], tol[40:40 + before])
    assert torch.isfinite(out).all()


def test_prompt_strided_q_rows_behind_and_repeats():
    """q16 as columns of a wider buffer; rows behind the last sequence keep what
    the output held; the same call twice gives the same bits; a captured graph
    follows the lengths."""
    hd, H, G, ps, new, kv = 128, 2, 4, 16, [50, 21], [400, 33]
    n_pages, n_tok = 30, 80
    (k, _, v, _), cache = make_cache("f16", n_pages, H, ps, hd)
    table = make_tables(kv, ps, n_pages)
    q = rand_q(n_tok, H * G, hd)
    qw = torch.full((n_tok, H * G * hd + 64), float("nan"), dtype=torch.float16)
    qw[:, :H * G * hd] = q.reshape(n_tok, -1)
    qd = qw.cuda()[:, :H * G * hd].unflatten(1, (H * G, hd))
    out = torch.full((n_tok, H * G, hd), -3.0, device="cuda")
    batch = make_batch(new, kv, table)
    ws = fr.make_paged_workspace(H * G, H, hd)
    keep = torch.full(out.shape, -3.0)
    fr.paged_attn(cache, batch, qd, H * G, out=out, workspace=ws)
    want, tol = ref.attention(q, k.double(), v.double(), starts(new), kv, table, H * G, out=keep)
    check(out, want, tol)
    assert (out[sum(new):] == -3.0).all()
    again = torch.full_like(out, -3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fr.paged_attn(cache, batch, qd, H * G, out=again, workspace=ws, stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    kv2, new2 = [300, 100], [10, 60]
    t2 = make_tables(kv2, ps, n_pages, 9)
    batch.kv_len.copy_(torch.tensor(kv2, dtype=torch.int32))
    batch.tok_start.copy_(torch.tensor(starts(new2), dtype=torch.int32))
    batch.page_table[:, :t2.shape[1]].copy_(t2)
    again.fill_(-3.0)
    graph.replay()
    torch.cuda.synchronize()
    want, tol = ref.attention(q, k.double(), v.double(), starts(new2), kv2, t2, H * G, out=keep)
    check(again, want, tol)
    fr.workspace_check(ws)


@pytest.mark.parametrize("kind", TYPES)
def test_prompt_as_its_tokens_one_by_one(kind):
    """A prompt's rows are those that each token gives by itself over the keys before it."""
    hd, H, G, ps, n = 128, 2, 4, 16, 64
    (k, ks, v, vs), cache = make_cache(kind, 8, H, ps, hd, 5)
    table = make_tables([n], ps, 8, 5)
    q = rand_q(n, H * G, hd, 6)
    out = fr.paged_attn(cache, make_batch([n], [n], table), q.cuda(), H * G)
    one = torch.cat([fr.paged_attn(cache, make_batch([1], [i + 1], table), q[i:i + 1].cuda(), H * G) for i in range(n)])
    _, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), [0, n], [n], table, H * G, v_scale=vs)
    check(out, one.double().cpu(), 2 * tol)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prompt_e4m3_scales_of_any_size(hd):
    """V scales from 2^-60 to 2^60, zero, negative, other than powers of two; a
    row's result does not depend on the scales of pages behind it."""
    H, G, ps, new, kv = 2, 4, 16, [60, 37], [160, 37]
    (k, ks, v, vs), _ = make_cache("e4m3", 16, H, ps, hd, 29)
    table = make_tables(kv, ps, 16, 29)
    vs = torch.exp2(torch.randint(-60, 61, vs.shape, generator=torch.Generator().manual_seed(30)).float()) * 1.3
    vs[:, 1] = -vs[:, 1]
    vs[table[0, 1].long()] = 0.0
    ks = ks * 0.7
    q = rand_q(sum(new), H * G, hd, 31)
    out = fr.paged_attn(fr.PagedKV(k.cuda(), v.cuda(), ks.cuda(), vs.cuda()), make_batch(new, kv, table), q.cuda(), H * G)
    want, tol = ref.attention(q, ref.values(k, ks), ref.values(v, vs), starts(new), kv, table, H * G,
                              v_scale=vs)
    check(out, want, tol)
    zero = fr.PagedKV(k.cuda(), v.cuda(), ks.cuda(), torch.zeros_like(vs).cuda())
    assert not fr.paged_attn(zero, make_batch(new, kv, table), q.cuda(), H * G).any()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("G,n", [(128, 3), (129, 1), (160, 4)])
def test_prompt_groups_as_large_as_a_tile(kind, G, n):
    """A token's heads fill a 128-row tile, or do not fit one."""
    run_case(kind, 64, 1, G, 16, [n, 1, n], [50, 17, 129], seed=G)


def test_prompt_graphs_share_a_workspace():
    """Two captured prompts, one workspace, replayed in turn on one stream."""
    hd, H, G, ps = 128, 2, 4, 16
    ws = fr.make_paged_workspace(H * G, H, hd)
    runs = []
    for seed, kind, new, kv in ((1, "f16", [60, 20], [500, 20]), (2, "e4m3", [33, 90], [64, 700])):
        n_pages = sum(-(-x // ps) for x in kv) + 2
        (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, seed)
        table = make_tables(kv, ps, n_pages, seed)
        q = rand_q(sum(new), H * G, hd, seed)
        batch, qd, out = make_batch(new, kv, table), q.cuda(), torch.zeros((sum(new), H * G, hd), device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            fr.paged_attn(cache, batch, qd, H * G, out=out, workspace=ws, stream=st)
        want = ref.attention(q, ref.values(k, ks), ref.values(v, vs), starts(new), kv, table, H * G, v_scale=vs)
        runs.append((graph, out, want, cache, batch, qd))
    for _ in range(3):
        for r in runs:
            r[1].zero_()
            r[0].replay()
    torch.cuda.synchronize()
    for _, out, (want, tol), *_ in runs:
        check(out, want, tol)
    fr.workspace_check(ws)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H,G,n", [(3, 5, 4), (3, 7, 7), (1, 5, 4), (1, 3, 17)])
def test_either_side_of_the_large_tiles(kind, H, G, n):
    """hd 256: the row tile goes by the rows and, in f16, by the number of segments."""
    run_case(kind, 256, H, G, 16, [n] * len(LENS), [max(n, x) for x in LENS], seed=G)
