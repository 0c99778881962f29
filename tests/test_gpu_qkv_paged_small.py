"""Norms of rows whose squares vanish in fp32, with eps 0 or so small that it does not
hide them: against the plain 64-bit form, in every form of the call (decode steps, the
ring of prompts into f16 pages, pieces of e4m3 pages, rotated parts that vectors do not
divide)."""
import pytest
import torch

import gqa_kv_head_gb300 as fr
import paged_qkv_ref as qref
from test_gpu_paged import make_batch, make_cache, make_tables
from test_gpu_qkv_paged import check_f16, check_pages, make_rows, make_weights, positions

pytestmark = pytest.mark.gpu

# 2^-52: squares about 2^-104; 1e-24: below the normal range; 1e-30 and 1e-39: none left (1e-39: subnormal rows)
SIZES = [2.0 ** -52, 1e-24, 1e-30, 1e-39]
FORMS = {"decode": ([1, 1], [3, 17], 16, 128), "prompt": ([40], [55], 16, 128), "large pages": ([300], [310], 128, 128),
         "odd decode": ([1, 1], [3, 17], 16, 100), "odd prompt": ([40], [55], 16, 100)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("rows", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -120, 2.0 ** -100])
def test_small_rows(form, kind, rows, size, eps):
    new, kv, ps, n_dims = FORMS[form]
    n_tok, hd, H, G = sum(new), 128, 2, 2
    (k, ks, v, vs), cache = make_cache(kind, 12, H, ps, hd, 1)
    table = make_tables(kv, ps, 12, 1)
    (q, kn, vn), (dq, dk, dv) = make_rows(rows, n_tok, H, G, hd, 2, size=size)
    # rows of other sizes beside them in one launch
    for t, d in ((q, dq), (kn, dk)):
        t[0, 0] *= 2.0 ** 60
        d[0, 0] *= 2.0 ** 60
        assert torch.equal(t, d.cpu())
    dv.copy_(torch.ones_like(dv))
    wq, wk = make_weights(hd, 3)
    pos, rope = positions(new, kv), {"n_dims": n_dims}
    out = fr.qkv_post_paged(cache, make_batch(new, kv, table), dq, dk, dv, torch.tensor(pos, dtype=torch.int32).cuda(), fr.rope_params(**rope),
                            q_norm=wq.cuda(), k_norm=wk.cuda(), eps=eps)
    y, tol = qref.rows(q, pos, rope, wq, eps, False, hd ** -0.5)
    check_f16(out.view(n_tok, G * H, hd), y, tol, "q")
    y, tol = qref.rows(kn, pos, rope, wk, eps)
    check_pages(kind, y, tol, new, kv, table, k, ks, cache.k_pages, cache.k_scale, "K")


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("new,kv", [([1, 1], [3, 17]), ([40], [55])])
def test_zeros(kind, new, kv):
    """Rows of zeros: zeros beside any eps > 0, NaN with eps 0 as the formula says; their neighbours are not touched."""
    n_tok, hd, H, G, ps = sum(new), 128, 2, 2, 16
    for eps in (0.0, 1e-38, 1e-6):
        (k, ks, v, vs), cache = make_cache(kind, 12, H, ps, hd, 1)
        (q, kn, vn), (dq, dk, dv) = make_rows("f32", n_tok, H, G, hd, 2)
        dq[0, 1], dq[1, 0] = 0.0, 0.0
        dk.zero_()
        w = torch.ones(hd, device="cuda")
        pos = positions(new, kv)
        table = make_tables(kv, ps, 12, 1)
        out = fr.qkv_post_paged(cache, make_batch(new, kv, table), dq, dk, dv, torch.tensor(pos, dtype=torch.int32).cuda(),
                                fr.rope_params(hd), q_norm=w, k_norm=w, eps=eps).view(n_tok, G * H, hd)
        nan = torch.isnan(out)
        want = torch.zeros_like(nan)
        want[0, 1] = want[1, 0] = eps == 0.0
        assert torch.equal(nan, want)
        assert eps == 0.0 or not out[0, 1].any()
        if kind == "f16":
            first = cache.k_pages[int(table[0, (kv[0] - new[0]) // ps]), :, (kv[0] - new[0]) % ps]
            assert bool(torch.isnan(first).all()) if eps == 0.0 else not bool(first.any())


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("new,kv", [([1, 1], [3, 17]), ([40], [55])])
@pytest.mark.parametrize("size,eps", [(1.0e19, 1.0e37), (2.0 ** 64, 2.0 ** 124)])
def test_large_rows_beside_a_large_eps(kind, new, kv, size, eps):
    """Squares past fp32's range, and an eps that counts beside their mean."""
    n_tok, hd, H, G, ps = sum(new), 128, 2, 2, 16
    (k, ks, v, vs), cache = make_cache(kind, 12, H, ps, hd, 1)
    table = make_tables(kv, ps, 12, 1)
    (q, kn, vn), (dq, dk, dv) = make_rows("f32", n_tok, H, G, hd, 2, size=size)
    dv.copy_(torch.ones_like(dv))
    wq, wk = make_weights(hd, 3)
    pos, rope = positions(new, kv), {"n_dims": hd}
    out = fr.qkv_post_paged(cache, make_batch(new, kv, table), dq, dk, dv, torch.tensor(pos, dtype=torch.int32).cuda(), fr.rope_params(**rope),
                            q_norm=wq.cuda(), k_norm=wk.cuda(), eps=eps)
    y, tol = qref.rows(q, pos, rope, wq, float(torch.tensor(eps)), False, hd ** -0.5)
    check_f16(out.view(n_tok, G * H, hd), y, tol, "q")
    y, tol = qref.rows(kn, pos, rope, wk, float(torch.tensor(eps)))
    check_pages(kind, y, tol, new, kv, table, k, ks, cache.k_pages, cache.k_scale, "K")
