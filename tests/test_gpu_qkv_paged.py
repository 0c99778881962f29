"""qkv_post_paged on the GPU: normed and rotated rows against the plain 64-bit form
(paged_qkv_ref.py), pages against it too, the calls that it joins where it has their
arithmetic, over row types, page types, head dims and layouts, rotated parts, norms,
strides, uneven and empty sequences, bad input, streams and captured graphs."""
import pytest
import torch

import gqa_kv_head_gb300 as fr
import paged_qkv_ref as qref
import paged_ref as ref
from test_gpu_paged import make_batch, make_cache, make_tables, starts

pytestmark = pytest.mark.gpu

ROWS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPES = ["f16", "e4m3"]


def make_rows(rows, n_tok, H, G, hd, seed, pad=0, size=2.0):
    """q, k, v as columns of one buffer."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((n_tok, (G + 2) * H * hd + pad), generator=g) * size).to(ROWS[rows])
    d = x.cuda()
    cut = [0, G * H * hd, (G + 1) * H * hd, (G + 2) * H * hd]
    return [[t[:, a:b].view(n_tok, -1, hd) for a, b in zip(cut, cut[1:])] for t in (x, d)]


def make_weights(hd, seed):
    g = torch.Generator().manual_seed(seed)
    return [1.0 + 0.3 * torch.randn(hd, generator=g) for _ in range(2)]


def positions(new, kv, seed=0):
    return [p for a, n in zip(new, kv) for p in range(n - a, n)]


def check_f16(got, want, tol, what):
    """want +- tol, rounded to f16: half a step of f16 more (2^-11 of the value, or 2^-25)."""
    d = (got.double().cpu() - want).abs()
    t = tol + want.abs() * 2.0 ** -11 + 2.0 ** -25
    assert bool((d <= t).all()), f"{what}: {float((d / t).max()):.2f} times the tolerance"


def check_pages(kind, new_rows, tol, new, kv, table, old, old_scale, got, got_scale, what):
    """Pages after the step: new rows within their tolerance and a rounding, all else untouched."""
    ps, H = old.shape[2], old.shape[1]
    want_touched = torch.zeros(old.shape[0], ps, dtype=torch.bool)
    got, was = got.cpu(), old
    got_scale = None if got_scale is None else got_scale.cpu()
    first_rows = {}
    t = 0
    for b, (a, n) in enumerate(zip(new, kv)):
        for i in range(a):
            slot = n - a + i
            page, r = int(table[b, slot // ps]), slot % ps
            want_touched[page, r] = True
            first_rows.setdefault(page, (r, []))[1].append(t + i)
            if kind == "f16":
                check_f16(got[page, :, r], new_rows[t + i], tol[t + i], what)
        t += a
    if kind == "f16":
        same = ref.same_bits(got.permute(0, 2, 1, 3)[~want_touched], was.permute(0, 2, 1, 3)[~want_touched])
        assert same, what
        return
    for page in range(old.shape[0]):
        if page not in first_rows:
            assert ref.same_bits(got[page], was[page]) and torch.equal(got_scale[page], old_scale[page]), what
            continue
        r0, toks = first_rows[page]
        x, e = new_rows[toks].transpose(0, 1), tol[toks].transpose(0, 1)
        for h in range(H):
            s, top = float(got_scale[page, h]), float(x[h].abs().max())
            off = float(e[h].max())
            prior = float(old_scale[page, h]) if r0 else 0.0
            # (a largest value within its tolerance of a border may have the scale of either side)
            assert s in {max(ref.pow2_scale(max(0.0, top + d)), prior) for d in (-off, 0.0, off)}, what
            y = got[page, h].double() * s
            d = (y[r0:r0 + len(toks)] - x[h]).abs()
            # half a step of e4m3: 2^-4 of the value, or of the smallest normal value's 2^-6 s
            t = e[h] + x[h].abs().clamp(min=2.0 ** -6 * s) * 2.0 ** -4
            # (values at a border may pass 448 s by their tolerance, and are held to it)
            assert bool((d <= t).all()), f"{what}: {float((d / t).max()):.2f}"
            if s == prior or not r0:
                assert ref.same_bits(got[page, h, :r0], was[page, h, :r0]), what
            else:
                w = was[page, h, :r0].double() * (prior / s)
                assert ref.same_bits(got[page, h, :r0], w.float().to(torch.float8_e4m3fn)), what
            assert ref.same_bits(got[page, h, r0 + len(toks):], was[page, h, r0 + len(toks):]), what


def run_case(kind, rows, hd, H, G, ps, new, kv, rope=None, norm=True, interleaved=False, seed=0, nhd=False, pad=0, eps=1e-6,
             q_scale=None, size=2.0, pos=None):
    n_pages, n_tok = sum(-(-n // ps) for n in kv) + 2, sum(new)
    (k, ks, v, vs), cache = make_cache(kind, n_pages, H, ps, hd, seed, nhd)
    table = make_tables(kv, ps, n_pages, seed)
    (q, kn, vn), (dq, dk, dv) = make_rows(rows, n_tok, H, G, hd, seed + 1, pad, size)
    wq, wk = make_weights(hd, seed) if norm else (None, None)
    rope = {"n_dims": hd, "freq_base": 10000.0, **(rope or {})}
    pos = positions(new, kv) if pos is None else pos
    ws = fr.make_paged_workspace(G * H, H, hd)
    out = fr.qkv_post_paged(cache, make_batch(new, kv, table), dq, dk, dv, torch.tensor(pos, dtype=torch.int32).cuda(),
                            fr.rope_params(**rope), q_norm=None if wq is None else wq.cuda(), k_norm=None if wk is None else wk.cuda(),
                            eps=eps, interleaved=interleaved, q_scale=q_scale, workspace=ws)
    fr.workspace_check(ws)
    what = f"{kind} {rows} hd{hd} H{H} G{G} ps{ps} {rope} norm {norm} il {interleaved}"
    y, tol = qref.rows(q, pos, rope, wq, eps, interleaved, hd ** -0.5 if q_scale is None else q_scale)
    check_f16(out.view(n_tok, G * H, hd), y, tol, what)
    y, tol = qref.rows(kn, pos, rope, wk, eps, interleaved)
    check_pages(kind, y, tol, new, kv, table, k, ks, cache.k_pages, cache.k_scale, what + " K")
    check_pages(kind, vn.double(), vn.double().abs() * 2.0 ** -24, new, kv, table, v, vs, cache.v_pages, cache.v_scale, what + " V")


# one token beside others, none, a page's last and first rows, several pages
NEW = [1, 0, 2, 37, 1, 16, 70]
KV = [1, 9, 65, 100, 64, 16, 200]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_prompts(kind, rows, hd, interleaved):
    run_case(kind, rows, hd, 2, 3, 32, NEW, KV, interleaved=interleaved, seed=hd)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_decode(kind, rows, hd, interleaved):
    kv = [1, 2, 16, 17, 33, 64, 65, 300]
    run_case(kind, rows, hd, 3, 5, 16, [1] * len(kv), kv, interleaved=interleaved, seed=hd + 1)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hd,n_dims", [(64, 2), (64, 32), (64, 48), (64, 62), (128, 96), (128, 70), (128, 12), (256, 64), (256, 250)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [5, 64, 300]), ([40, 3], [64, 99])])
def test_part_of_the_head(kind, hd, n_dims, interleaved, new, kv):
    """Rotated dims that vectors of eight divide, and others; odd numbers of pairs."""
    run_case(kind, "f16", hd, 2, 2, 32, new, kv, rope={"n_dims": n_dims}, interleaved=interleaved, seed=n_dims)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rope", [dict(freq_scale=0.25), dict(freq_scale=0.25, ext_factor=1.0, n_ctx_orig=512), dict(freq_base=5e5, attn_factor=0.8),
                                  dict(freq_factors=[1.0 + 0.1 * i for i in range(64)])], ids=["linear", "yarn", "base", "factors"])
@pytest.mark.parametrize("norm", [False, True])
def test_scaled_rotations(rope, interleaved, norm):
    run_case("f16", "f32", 128, 2, 2, 64, [3, 1, 20], [300, 64, 1000], rope=rope, interleaved=interleaved, norm=norm)


@pytest.mark.parametrize("kind", TYPES)
def test_far_positions(kind):
    """Positions up to 2^31 - 1 and negative ones keep exact angles."""
    run_case(kind, "f32", 128, 1, 2, 16, [5], [40], pos=[2 ** 31 - 1, 0, 1_000_003, 131_071, -70_001])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps,nhd", [(16, True), (64, True), (128, False), (256, False)])
@pytest.mark.parametrize("hd", [128, 256])
def test_page_sizes_and_layouts(kind, ps, nhd, hd):
    run_case(kind, "bf16", hd, 2, 2, ps, [90, 1, 300], [200, 33, 310], seed=ps, nhd=nhd, pad=64)


# 8, 16 and 32 rows of a page to a thread of 256, pages begun by earlier rows, odd numbers of heads
@pytest.mark.parametrize("rows", ["f32", "f16"])
@pytest.mark.parametrize("hd,ps", [(64, 256), (128, 128), (128, 256), (256, 64), (256, 128), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_large_pages(rows, hd, ps, interleaved):
    run_case("e4m3", rows, hd, 3, 3, ps, [5, 0, 290, 77], [ps + 8, 40, 290 + ps // 2, 77], {"n_dims": hd // 2}, seed=hd + ps,
             interleaved=interleaved, pad=8)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H,G", [(1, 1), (1, 7), (5, 1), (8, 4), (1, 64)])
def test_head_counts(kind, H, G):
    run_case(kind, "f16", 64, H, G, 16, [1, 1], [20, 33], seed=H)
    run_case(kind, "f16", 64, H, G, 16, [30, 5], [60, 33], seed=H)


@pytest.mark.parametrize("n_seq", [33, 130, 300])
def test_many_sequences(n_seq):
    run_case("f16", "f16", 64, 1, 2, 16, [1] * n_seq, [1 + i % 40 for i in range(n_seq)])


def test_long_prompt():
    """More tokens than one qkv_post call takes, more tiles than blocks run at a time."""
    run_case("f16", "bf16", 64, 1, 2, 64, [9001], [9100])


@pytest.mark.parametrize("size", [1e-12, 1e18, 3e37])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("new,kv", [([1, 1], [3, 17]), ([40], [55])])
def test_rows_whose_squares_leave_the_range(size, kind, new, kv):
    """fp32 squares overflow, or vanish beside eps."""
    n_tok, hd, H, G, ps = sum(new), 128, 1, 2, 16
    (k, ks, v, vs), cache = make_cache(kind, 12, H, ps, hd, 1)
    table = make_tables(kv, ps, 12, 1)
    (q, kn, vn), (dq, dk, dv) = make_rows("f32", n_tok, H, G, hd, 2, size=size)
    dv.copy_(torch.ones_like(dv))
    wq, wk = make_weights(hd, 3)
    pos, rope = positions(new, kv), {"n_dims": hd}
    out = fr.qkv_post_paged(cache, make_batch(new, kv, table), dq, dk, dv, torch.tensor(pos, dtype=torch.int32).cuda(), fr.rope_params(**rope),
                            q_norm=wq.cuda(), k_norm=wk.cuda(), eps=1e-5)
    y, tol = qref.rows(q, pos, rope, wq, 1e-5, False, hd ** -0.5)
    check_f16(out.view(n_tok, G * H, hd), y, tol, "q")
    y, tol = qref.rows(kn, pos, rope, wk, 1e-5)
    check_pages(kind, y, tol, new, kv, table, k, ks, cache.k_pages, cache.k_scale, "K")


@pytest.mark.parametrize("new,kv", [([1, 1, 0, 1], [9, 64, 5, 100]), ([50, 0, 3], [64, 7, 40])])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("mode", [fr.FR_ROPE_EXACT, fr.FR_ROPE_GGML_F32])
@pytest.mark.parametrize("n_dims", [128, 100, 44])
def test_bits_of_the_calls_that_it_joins(new, kv, kind, mode, n_dims):
    """Without norms and with pairs of halves: qkv_post and kv_append_paged, bit by bit."""
    hd, H, G, ps, n_tok = 128, 2, 4, 32, sum(new)
    table = make_tables(kv, ps, 20, 4)
    (q, kn, vn), (dq, dk, dv) = make_rows("f32", n_tok, H, G, hd, 5)
    pos = torch.tensor(positions(new, kv), dtype=torch.int32).cuda()
    rope = fr.rope_params(n_dims, freq_scale=0.5, ext_factor=1.0, n_ctx_orig=256, mode=mode)
    caches = [make_cache(kind, 20, H, ps, hd, 6)[1] for _ in range(2)]
    batch = make_batch(new, kv, table)
    a, _ = fr.qkv_post(dq, pos, G * H, hd, rope)
    fr.kv_append_paged(caches[0], batch, dk, dv, pos, rope)
    b = fr.qkv_post_paged(caches[1], batch, dq, dk, dv, pos, rope)
    assert torch.equal(a, b)
    assert ref.same_bits(caches[0].k_pages, caches[1].k_pages) and ref.same_bits(caches[0].v_pages, caches[1].v_pages)
    if kind == "e4m3":
        assert torch.equal(caches[0].k_scale, caches[1].k_scale) and torch.equal(caches[0].v_scale, caches[1].v_scale)
    # one norm alone: the other rows keep their bits
    w = torch.ones(hd, device="cuda")
    c = fr.qkv_post_paged(caches[1], batch, dq, dk, dv, pos, rope, k_norm=w)
    assert torch.equal(a, c)
    d = fr.qkv_post_paged(caches[1], batch, dq, dk, dv, pos, rope, q_norm=w)
    assert not torch.equal(a, d)
    fr.kv_append_paged(caches[0], batch, dk, dv, pos, rope)
    if kind == "f16":
        assert ref.same_bits(caches[0].k_pages, caches[1].k_pages)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("new,kv,pad", [([1, 1], [9, 40], 3), ([20, 9], [30, 40], 60)])
def test_padding_rows_and_bad_sequences(kind, new, kv, pad):
    """Rows behind the last sequence hold NaN and are left alone; a sequence whose numbers do
    not fit is skipped and reported, its neighbours are not."""
    hd, H, G, ps, n_tok = 64, 2, 2, 16, sum(new) + pad
    (k, ks, v, vs), cache = make_cache(kind, 12, H, ps, hd, 1)
    table = make_tables(kv, ps, 12, 1)
    (q, kn, vn), (dq, dk, dv) = make_rows("f16", n_tok, H, G, hd, 2)
    for t in (dq, dk, dv):
        t[sum(new):] = float("nan")
    pos = torch.tensor(positions(new, kv) + [0] * pad, dtype=torch.int32).cuda()
    wq, wk = make_weights(hd, 1)
    ws = fr.make_paged_workspace(G * H, H, hd)
    batch = make_batch(new, kv, table)
    out = torch.full((n_tok * G * H, hd), 7.0, dtype=torch.float16, device="cuda")
    fr.qkv_post_paged(cache, batch, dq, dk, dv, pos, fr.rope_params(hd), q_norm=wq.cuda(), k_norm=wk.cuda(), q16_out=out, workspace=ws)
    fr.workspace_check(ws)
    assert bool((out[sum(new) * G * H:] == 7.0).all())
    y, tol = qref.rows(q[:sum(new)], positions(new, kv), {"n_dims": hd}, wq, 1e-6, False, hd ** -0.5)
    check_f16(out[:sum(new) * G * H].view(sum(new), G * H, hd), y, tol, "q")
    y, tol = qref.rows(kn[:sum(new)], positions(new, kv), {"n_dims": hd}, wk)
    check_pages(kind, y, tol, new, kv, table, k, ks, cache.k_pages, cache.k_scale, "K")
    # the second sequence has fewer keys than tokens
    before = [t.clone() for t in (cache.k_pages, cache.v_pages)]
    batch.kv_len[1] = new[1] - 1
    fr.qkv_post_paged(cache, batch, dq, dk, dv, pos, fr.rope_params(hd), q_norm=wq.cuda(), k_norm=wk.cuda(), q16_out=out, workspace=ws)
    with pytest.raises(fr.FrError):
        fr.workspace_check(ws)
    page = int(table[1, 0])
    assert ref.same_bits(before[0][page].cpu(), cache.k_pages[page].cpu())
    assert ref.same_bits(before[0][int(table[0, 0])].cpu(), cache.k_pages[int(table[0, 0])].cpu())


@pytest.mark.parametrize("kind", TYPES)
def test_bad_page_is_not_written(kind):
    new, kv, hd, H, ps = [3], [18], 64, 1, 16
    (k, ks, v, vs), cache = make_cache(kind, 4, H, ps, hd, 1)
    (q, kn, vn), (dq, dk, dv) = make_rows("f32", 3, H, 1, hd, 2)
    for bad in (-1, 4, 2 ** 31 - 1):
        ws = fr.make_paged_workspace(1, 1, hd)
        table = torch.tensor([[2, bad]], dtype=torch.int32)
        fr.qkv_post_paged(cache, make_batch(new, kv, table), dq, dk, dv, torch.zeros(3, dtype=torch.int32).cuda(), fr.rope_params(hd), workspace=ws)
        with pytest.raises(fr.FrError):
            fr.workspace_check(ws)
        for p in (0, 1, 3):
            assert ref.same_bits(cache.k_pages[p].cpu(), k[p])
            assert ref.same_bits(cache.v_pages[p].cpu(), v[p])


@pytest.mark.parametrize("kind", TYPES)
def test_non_finite_rows(kind):
    """NaN and infinities reach their own head alone."""
    hd, H, G, ps = 128, 2, 2, 16
    (k, ks, v, vs), cache = make_cache(kind, 6, H, ps, hd, 1)
    table = make_tables([20], ps, 6, 1)
    (q, kn, vn), (dq, dk, dv) = make_rows("f16", 20, H, G, hd, 2)
    dq[3, 1, 5], dq[4, 0, 7] = float("nan"), float("inf")
    dk[3, 1, 5], dk[17, 0, 7] = float("nan"), float("inf")
    w = torch.ones(hd, device="cuda")
    out = fr.qkv_post_paged(cache, make_batch([20], [20], table), dq, dk, dv, torch.arange(20, dtype=torch.int32).cuda(),
                            fr.rope_params(hd), q_norm=w, k_norm=w).view(20, H * G, hd)
    bad = torch.isnan(out).any(dim=2)
    want = torch.zeros_like(bad)
    want[3, 1] = want[4, 0] = True
    assert torch.equal(bad, want)
    assert torch.isnan(out[3, 1]).all()
    got = cache.k_pages[table[0, :2].long().cuda()].float().permute(0, 2, 1, 3).reshape(-1, H, hd)[:20]
    bad = torch.isnan(got).any(dim=2)
    want = torch.zeros_like(bad)
    want[3, 1] = want[17, 0] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("n", [1, 30])
def test_graph_on_another_stream_with_the_attention(kind, n):
    """A step as it is used: rows, then attention with sinks, captured together; replayed as
    the sequences grow; against the 64-bit attention over what the pages hold."""
    import paged_sinks
    hd, H, G, ps, window, sinks = 64, 2, 3, 16, 40, 5
    kv = [n, 33 + n, 90 + n]
    n_pages, n_tok = 40, 3 * n
    _, cache = make_cache(kind, n_pages, H, ps, hd, 2)
    table = make_tables([200, 200, 200], ps, n_pages, 2)
    (q, kn, vn), (dq, dk, dv) = make_rows("bf16", n_tok, H, G, hd, 3)
    wq, wk = make_weights(hd, 4)
    rope, batch = fr.rope_params(hd), make_batch([n] * 3, kv, table)
    pos = torch.zeros(n_tok, dtype=torch.int32, device="cuda")
    ws, wqd, wkd = fr.make_paged_workspace(H * G, H, hd), wq.cuda(), wk.cuda()
    q16 = torch.empty((n_tok * H * G, hd), dtype=torch.float16, device="cuda")
    out = torch.empty((n_tok, H * G, hd), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        fr.qkv_post_paged(cache, batch, dq, dk, dv, pos, rope, q_norm=wqd, k_norm=wkd, q16_out=q16, workspace=ws, stream=s)
        fr.paged_attn(cache, batch, q16, H * G, window=window, sinks=sinks, out=out, workspace=ws, stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(graph, stream=s):
            step()
        for turn in range(3):
            at = positions([n] * 3, kv)
            pos.copy_(torch.tensor(at, dtype=torch.int32))
            batch.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
            graph.replay()
            s.synchronize()
            y, tol = qref.rows(q, at, {"n_dims": hd}, wq, 1e-6, False, hd ** -0.5)
            check_f16(q16.view(n_tok, H * G, hd), y, tol, "q")
            ks = None if cache.k_scale is None else cache.k_scale.cpu()
            vs = None if cache.v_scale is None else cache.v_scale.cpu()
            want, tol = paged_sinks.attention(q16.view(n_tok, H * G, hd).cpu(), ref.values(cache.k_pages.cpu(), ks),
                                              ref.values(cache.v_pages.cpu(), vs), starts([n] * 3), kv, table, H * G, window, sinks, 1.0, vs)
            d = (out.double().cpu() - want).abs()
            assert bool((d <= tol + 1e-37).all())
            kv = [x + n for x in kv]
    fr.workspace_check(ws)


def test_refusals():
    hd, H, G, ps = 64, 2, 2, 16
    _, cache = make_cache("f16", 8, H, ps, hd)
    batch = make_batch([2], [20], make_tables([20], ps, 8))
    _, (q, k, v) = make_rows("f16", 2, H, G, hd, 1, pad=8)
    pos, rope, w = torch.zeros(2, dtype=torch.int32).cuda(), fr.rope_params(hd), torch.ones(hd, device="cuda")
    ok = dict(q=q, k_new=k, v_new=v, pos=pos, rope=rope)

    def call(**kw):
        a = {**ok, **kw}
        return fr.qkv_post_paged(cache, batch, a.pop("q"), a.pop("k_new"), a.pop("v_new"), a.pop("pos"), a.pop("rope"), **a)
    call()
    for kw in (dict(q=q.float()), dict(q=q.double(), k_new=k.double(), v_new=v.double()), dict(pos=pos.long()), dict(q_norm=w.half()),
               dict(k_norm=w.double())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=q[:1]), dict(k_new=k[:, :1]), dict(v_new=v[..., :32]), dict(pos=pos[:1]), dict(q_norm=w[:32]), dict(k_norm=w[None]),
               dict(q=q.cpu()), dict(q_norm=w.cpu()), dict(q=q.transpose(1, 2)), dict(q=q[..., ::2]),
               dict(q16_out=torch.empty((8, hd), device="cuda")), dict(q16_out=torch.empty((7, hd), dtype=torch.float16, device="cuda")),
               dict(pos=torch.zeros(4, dtype=torch.int32).cuda()[::2])):
        with pytest.raises(ValueError):
            call(**kw)
    odd = torch.zeros(hd + 1, device="cuda")[1:]
    _, (q2, k2, v2) = make_rows("f16", 2, H, G, hd, 1, pad=4)           # token stride no multiple of 16 bytes
    for kw in (dict(eps=-1e-6, q_norm=w), dict(eps=float("nan"), k_norm=w), dict(eps=float("inf"), k_norm=w), dict(q_norm=odd),
               dict(rope=fr.rope_params(hd + 2)), dict(rope=fr.rope_params(63)), dict(q=q2, k_new=k2, v_new=v2)):
        with pytest.raises(fr.FrError):
            call(**kw)
