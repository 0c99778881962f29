"""Paged attention where the tokens of a sequence see different pages: what a
row does not see does not reach it, the scales of e4m3 pages among that."""
import pytest
import torch

import gqa_kv_head_gb300 as fr
import paged_ref as ref
import paged_views
from test_gpu_paged import check, make_batch, make_cache, make_tables, rand_q, starts


def scale_case(hd, H, G, ps, new, kv, kw, seed, scales):
    """An e4m3 cache whose V scales are scales(page shape, table): inputs, the
    64-bit result and its tolerance, all on the CPU."""
    n_pages = sum(-(-n // ps) for n in kv) + 2
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn((n_pages, H, ps, hd), generator=g).to(torch.float8_e4m3fn) for _ in range(2))
    table = make_tables(kv, ps, n_pages, seed)
    ks = torch.exp2(torch.randint(-2, 3, (n_pages, H), generator=g).float()) * 0.02      # (small scores: little error in them)
    vs = scales((n_pages, H), table, g)
    q = rand_q(sum(new), H * G, hd, seed + 1)
    want, tol = paged_views.attention(q, ref.values(k, ks), ref.values(v, vs), starts(new), kv, table, H * G, v_scale=vs, **kw)
    return k, ks, v, vs, table, q, want, tol


def run(case, new, kv, H, G, kw):
    k, ks, v, vs, table, q, want, tol = case
    cache = fr.PagedKV(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    check(fr.paged_attn(cache, make_batch(new, kv, table), q.cuda(), H * G, **kw), want, tol)


def any_size(shape, table, g):
    vs = torch.exp2(torch.randint(-60, 61, shape, generator=g).float()) * 1.3
    vs[:, 1] = -vs[:, 1]
    return vs


NEW = {2: [2, 2, 2, 2, 2], 4: [4, 4, 4, 4, 4], 8: [8, 8, 8, 8, 8], 0: [1, 6, 3, 8, 2], 40: [40, 17, 33, 60, 50]}
KV = [33, 49, 66, 133, 500]                # the new tokens lie on both sides of a page's first row
VIEWS = [dict(), dict(window=17), dict(window=40), dict(causal=False)]


def view_id(kw):
    return "_".join(f"{a}{b}" for a, b in kw.items()) or "causal"


@pytest.mark.parametrize("n", sorted(NEW))
@pytest.mark.parametrize("kw", VIEWS, ids=view_id)
def test_the_tolerance_can_fail_a_result(n, kw):
    """On the CPU: it lies far below the result for nearly every element."""
    kv = [max(a, b) for a, b in zip(NEW[n], KV)]
    *_, want, tol = scale_case(128, 2, 2, 16, NEW[n], kv, kw, n, any_size)
    assert float((tol > 2.0 ** -6 * want.abs()).double().mean()) < 0.03


@pytest.mark.gpu
@pytest.mark.parametrize("n", sorted(NEW))
@pytest.mark.parametrize("hd,G", [(64, 2), (128, 2), (128, 1), (256, 2), (128, 4)])
@pytest.mark.parametrize("kw", VIEWS, ids=view_id)
@pytest.mark.parametrize("ps", [16, 64])
def test_e4m3_scales_of_other_tokens_pages(n, hd, G, kw, ps):
    """V scales from 2^-60 to 2^60 on both signs: small tiles of 8, 16 and 32 rows, and the 128-row tiles."""
    kv = [max(a, b) for a, b in zip(NEW[n], KV)]
    run(scale_case(hd, 2, G, ps, NEW[n], kv, kw, n + hd, any_size), NEW[n], kv, 2, G, kw)


@pytest.mark.gpu
@pytest.mark.parametrize("ratio", [20, 24, 40, 100, 200])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("side", ["ahead", "behind", "both"])
def test_e4m3_one_unseen_page_outweighs_the_rest(ratio, hd, side):
    """The page that only the last token sees, the one that only the first
    token's window holds, or both, have V scales 2^ratio times the others'."""
    H, G, ps, new = 2, 2, 16, [2, 2, 2, 2]
    kv = [33, 49, 65, 145]                     # the second new token opens a page
    kw = {} if side == "ahead" else dict(window=17 if side == "both" else 16)
    if side == "behind":
        kv = [32, 48, 64, 144]                 # the second new token's window begins with a page, the first's one row before

    def scales(shape, table, g):
        low = -100 if ratio > 100 else 0
        vs = torch.full(shape, 2.0 ** low)
        for b, n in enumerate(kv):
            if side != "behind":
                vs[table[b, (n - 1) // ps].long()] = 2.0 ** (low + ratio)
            if side != "ahead":
                first = max(0, n - 1 - kw["window"])           # the first new token sees this key, the second does not
                vs[table[b, first // ps].long()] = 2.0 ** (low + ratio)
        assert torch.isfinite(vs).all()
        return vs
    case = scale_case(hd, H, G, ps, new, kv, kw, ratio + hd, scales)
    run(case, new, kv, H, G, kw)
