"""paged_attn with a window and first tokens that stay visible, on the GPU, against
the plain 64-bit form: head layouts and row tiles of both kernels, sinks that end
inside tiles and pages, sinks that meet the window, pages between the two that are
gone or hold anything, infinities, scales far apart, streams and graphs."""
import pytest
import torch

import gqa_kv_head_gb300 as fr
import paged_ref as ref
import paged_sinks
from test_gpu_paged import check, make_batch, make_cache, make_tables, rand_q, starts

pytestmark = pytest.mark.gpu

TYPES = ["f16", "e4m3"]
LENS = [1, 2, 17, 64, 65, 100, 129, 300, 523]


def run_case(kind, hd, H, G, ps, new, kv_len, window, sinks, seed=0, nhd=False, kq_scale=1.0):
    n_pages = sum(-(-n // ps) for n in kv_len) + 2
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, seed, nhd)
    table = make_tables(kv_len, ps, n_pages, seed)
    q = rand_q(sum(new), H * G, hd, seed + 1)
    out = fr.paged_attn(cache, make_batch(new, kv_len, table), q.cuda(), H * G, window=window, sinks=sinks, kq_scale=kq_scale)
    want, tol = paged_sinks.attention(q, ref.values(k, ks), ref.values(v, vs), starts(new), kv_len, table, H * G,
                                      window, sinks, kq_scale, vs)
    check(out, want, tol, f"{kind} hd{hd} H{H} G{G} ps{ps} w{window} s{sinks}")
    return out


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(1, 1), (8, 1), (5, 3), (4, 8), (16, 4), (3, 40)])
def test_head_layouts(kind, hd, G, n):
    """Every row-tile width of the small tiles, and 128-row tiles, at every head dim."""
    run_case(kind, hd, 2, G, 32, [n] * len(LENS), [max(n, x) for x in LENS], 70, 5, seed=hd + G)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 16), (5, 33), (16, 64), (63, 65), (64, 130), (100, 15), (200, 1), (520, 3),
                                          (2 ** 31 - 1, 4), (50, 2 ** 31 - 1), (3, 100)])
@pytest.mark.parametrize("G,n", [(3, 1), (2, 6), (4, 33)])
def test_windows_and_sinks(kind, window, sinks, G, n):
    """Sinks that end at, before and behind tile edges, that meet the window, that outgrow the sequence."""
    run_case(kind, 128, 2, G, 16, [n] * len(LENS), [max(n, x) for x in LENS], window, sinks, seed=window % 97 + sinks % 89)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps", [16, 64, 128, 256])
@pytest.mark.parametrize("G,n", [(2, 1), (4, 20)])
def test_page_sizes_and_layouts(kind, ps, G, n):
    run_case(kind, 64, 3, G, ps, [n] * len(LENS), [max(n, x) for x in LENS], 90, 20, seed=ps, nhd=ps == 64)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("G,n,kv,window,sinks", [(4, 1, 9000, 6000, 40), (8, 2, 20011, 3000, 7), (4, 70, 5000, 1500, 100)])
def test_one_long_sequence(kind, G, n, kv, window, sinks):
    """One segment split over every CTA: the sinks' tiles are in the first share, the window's in all."""
    run_case(kind, 128, 1, G, 64, [n], [kv], window, sinks, seed=7)


@pytest.mark.parametrize("kind", TYPES)
def test_uneven_tokens_and_empty_sequences(kind):
    new = [0, 3, 1, 0, 40, 2, 1, 5]
    kv = [0, 3, 0, 50, 75, 1, 200, 2]
    out = run_case(kind, 128, 2, 4, 16, new, kv, 9, 4, seed=5)
    s = starts(new)
    assert not out[s[2]].any()                       # no keys
    assert not out[s[7]:s[7] + 3].any() and out[s[7] + 3:].any()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(2, 1), (4, 3), (5, 30)])
@pytest.mark.parametrize("ps", [16, 64])
def test_pages_between_are_gone(kind, hd, G, n, ps):
    """Pages without a sink or a key of some row's window: their table entries are -1 or
    out of range, and no status is set; what the other pages hold in unseen rows is NaN."""
    kv, window, sinks, H = [700, 333, 260 + n], 60, 18, 2
    n_pages = sum(-(-x // ps) for x in kv) + 2
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 3)
    table = make_tables(kv, ps, n_pages, 3)
    odd = table.clone()
    q = rand_q(n * len(kv), H * G, hd, 4)
    for b, m in enumerate(kv):
        low = m - n + 1 - window
        for p in range(sinks // ps + 1, low // ps):
            odd[b, p] = (-1, n_pages + 5, 2 ** 31 - 1, -7)[p % 4]
        for j in list(range(sinks, low)) + list(range(m, -(-m // ps) * ps)):
            for t in (cache.k_pages, cache.v_pages):
                t[table[b, j // ps], :, j % ps] = float("nan")
    ws = fr.make_paged_workspace(H * G, H, hd)
    out = fr.paged_attn(cache, make_batch([n] * len(kv), kv, odd), q.cuda(), H * G, window=window, sinks=sinks, workspace=ws)
    fr.workspace_check(ws)
    want, tol = paged_sinks.attention(q, ref.values(k, ks), ref.values(v, vs), starts([n] * len(kv)), kv, table, H * G,
                                      window, sinks, 1.0, vs)
    check(out, want, tol, f"{kind} hd{hd}")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("G,n", [(2, 1), (4, 3), (4, 40)])
def test_bad_page_in_view(kind, G, n):
    """A sink's page that is none: its keys are masked, and the status says so."""
    kv, window, sinks, H, ps, hd = 400, 50, 20, 1, 16, 128
    (k, ks, v, vs), cache = make_cache(kind, 30, H, ps, hd, 3)
    table = make_tables([kv], ps, 30, 3)
    bad = table.clone()
    bad[0, 0] = 30
    q = rand_q(n, H * G, hd, 4)
    ws = fr.make_paged_workspace(H * G, H, hd)
    out = fr.paged_attn(cache, make_batch([n], [kv], bad), q.cuda(), H * G, window=window, sinks=sinks, workspace=ws)
    with pytest.raises(fr.FrError):
        fr.workspace_check(ws)
    # keys 16 .. 19 and the window: the first page's sinks moved out by a huge negative score would be the same
    kk = ref.values(k, ks)
    want = torch.zeros((n, H * G, hd), dtype=torch.float64)
    tol = torch.zeros_like(want)
    for i in range(n):
        see = [j for j in paged_sinks.seen_keys(kv - n + i, kv, window, sinks) if j >= 16]
        see = torch.tensor(see)
        page, row = table[0, see // ps].long(), see % ps
        kx, vx = kk[page, 0, row], ref.values(v, vs)[page, 0, row]
        w = torch.softmax(q[i].double() @ kx.T, dim=1)
        want[i] = w @ vx
        ds = (hd + 4) * 2.0 ** -23 * (q[i].double().abs() @ kx.abs().T).amax(dim=1)
        tol[i] = (w @ vx.abs()) * (2 * (2 * ds + 2.0 ** -20 + 500 * 2.0 ** -23))[:, None] + 2.0 ** -24 * vx.abs().sum(dim=0)
    check(out, want, tol)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("G,n", [(1, 1), (4, 6), (4, 40)])
def test_infinite_values_reach_only_rows_that_see_them(kind, G, n):
    """NaN in V: at a sink (every row), and at a key that left some rows' windows."""
    kv, window, sinks, H, ps, hd = 300, 100, 10, 1, 16, 64
    (k, ks, v, vs), cache = make_cache(kind, 30, H, ps, hd, 8)
    table = make_tables([kv], ps, 30, 8)
    q = rand_q(n, H * G, hd, 9)
    clean, tol = paged_sinks.attention(q, ref.values(k, ks), ref.values(v, vs), [0, n], [kv], table, H * G, window, sinks, 1.0, vs)
    leaving = kv - n + 1 - window + n // 2               # rows 0 .. n // 2 see it
    cache.v_pages[table[0, leaving // ps], 0, leaving % ps, 5] = float("nan")
    out = fr.paged_attn(cache, make_batch([n], [kv], table), q.cuda(), H * G, window=window, sinks=sinks).cpu()
    sees = torch.arange(n) <= n // 2
    assert torch.isnan(out[sees][..., 5]).all()
    assert not torch.isnan(out[~sees]).any()
    rest = [d for d in range(hd) if d != 5]
    assert bool(((out.double() - clean).abs() <= tol)[:, :, rest].all())
    assert bool(((out.double() - clean).abs() <= tol)[~sees].all())
    cache.v_pages[table[0, 0], 0, 3, 7] = float("nan")
    out = fr.paged_attn(cache, make_batch([n], [kv], table), q.cuda(), H * G, window=window, sinks=sinks).cpu()
    assert torch.isnan(out[..., 7]).all()


@pytest.mark.parametrize("G,n", [(1, 1), (4, 6), (8, 2), (4, 40)])
@pytest.mark.parametrize("where", ["between", "sink", "window"])
def test_scales_far_apart(G, n, where):
    """V scales of pages that no row sees cost nothing; those of the sinks and of the
    window may be far apart."""
    kv, window, sinks, H, ps, hd = 420, 100, 20, 2, 16, 128
    (k, ks, v, vs), cache = make_cache("e4m3", 60, H, ps, hd, 11)
    table = make_tables([kv], ps, 60, 11)
    p = {"between": [2, 3, 10], "sink": [0], "window": [24, 26]}[where]
    vs = vs.clone()
    vs[table[0, p].long()] *= 2.0 ** 30
    cache.v_scale.copy_(vs)
    q = rand_q(n, H * G, hd, 12)
    out = fr.paged_attn(cache, make_batch([n], [kv], table), q.cuda(), H * G, window=window, sinks=sinks)
    seen = vs.clone()
    if where == "between":                               # (the tolerance must not grant it either)
        seen[table[0, p].long()] = 1e-30
    want, tol = paged_sinks.attention(q, ref.values(k, ks), ref.values(v, vs), [0, n], [kv], table, H * G, window, sinks, 1.0, seen)
    check(out, want, tol, where)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("n", [1, 5, 40])
def test_no_sinks_is_the_plain_call(kind, n):
    kv = [max(n, x) for x in LENS]
    _, cache = make_cache(kind, 120, 2, 16, 128, 1)
    batch = make_batch([n] * len(kv), kv, make_tables(kv, 16, 120, 1))
    q = rand_q(n * len(kv), 8, 128).cuda()
    a = fr.paged_attn(cache, batch, q, 8, window=40)
    b = fr.paged_attn(cache, batch, q, 8, window=40, sinks=0)
    assert torch.equal(a, b)
    # sinks that the window holds anyway
    c = fr.paged_attn(cache, batch, q, 8, window=600, sinks=9)
    assert torch.equal(c, fr.paged_attn(cache, batch, q, 8))


@pytest.mark.parametrize("kind", TYPES)
def test_graph_follows_lengths_on_another_stream(kind):
    """Captured with sequences inside their window, replayed when they have outgrown it."""
    kv, ps, H, G, hd, window, sinks = [30, 90, 17], 16, 2, 4, 128, 40, 6
    most = [400, 300, 517]
    n_pages = sum(-(-x // ps) for x in most)
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, 2)
    table = make_tables(most, ps, n_pages, 2)
    q = rand_q(3, H * G, hd, 2)
    qd, out = q.cuda(), torch.zeros((3, H * G, hd), device="cuda")
    batch = make_batch([1, 1, 1], kv, table)
    ws = fr.make_paged_workspace(H * G, H, hd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        fr.paged_attn(cache, batch, qd, H * G, window=window, sinks=sinks, out=out, workspace=ws, stream=s)
        with torch.cuda.graph(graph, stream=s):
            fr.paged_attn(cache, batch, qd, H * G, window=window, sinks=sinks, out=out, workspace=ws, stream=s)
        for now in (kv, most, [41, 47, 46]):
            batch.kv_len.copy_(torch.tensor(now, dtype=torch.int32))
            graph.replay()
            s.synchronize()
            want, tol = paged_sinks.attention(q, ref.values(k, ks), ref.values(v, vs), [0, 1, 2, 3], now, table, H * G,
                                              window, sinks, 1.0, vs)
            check(out, want, tol, str(now))
    fr.workspace_check(ws)


def test_refusals():
    _, cache = make_cache("f16", 8, 1, 16, 64)
    batch = make_batch([1], [20], make_tables([20], 16, 8))
    q = rand_q(1, 1, 64).cuda()
    for kw in (dict(sinks=1), dict(sinks=-1), dict(sinks=-1, window=4), dict(sinks=2, causal=False), dict(sinks=2, window=-1),
               dict(sinks=2, window=4, causal=False), dict(sinks=-2 ** 40, window=4)):
        with pytest.raises(fr.FrError):
            fr.paged_attn(cache, batch, q, 1, **kw)
    assert torch.equal(fr.paged_attn(cache, batch, q, 1, window=4, sinks=2 ** 40), fr.paged_attn(cache, batch, q, 1))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("sinks", [0, 9])
@pytest.mark.parametrize("off", [4, 8, 12])
def test_output_begins_anywhere_on_16_bytes(kind, hd, sinks, off):
    """Whole and split pieces of 128-row tiles, stored 32 or 16 bytes at a time: the same bits, and nothing beside them."""
    new, kv, H, G = [40, 70], [3000, 170], 2, 4
    n_pages = sum(-(-n // 32) for n in kv) + 2
    cache = make_cache(kind, n_pages, H, 32, hd, 3)[1]
    batch, q = make_batch(new, kv, make_tables(kv, 32, n_pages, 3)), rand_q(sum(new), H * G, hd, 4).cuda()
    want = fr.paged_attn(cache, batch, q, H * G, window=1500, sinks=sinks)
    buf = torch.full((want.numel() + 24,), 7.0, device="cuda")
    out = buf[off:off + want.numel()].view(want.shape)
    fr.paged_attn(cache, batch, q, H * G, window=1500, sinks=sinks, out=out)
    assert torch.equal(out, want)
    assert bool((buf[:off] == 7).all()) and bool((buf[off + want.numel():] == 7).all())
