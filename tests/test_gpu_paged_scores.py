"""Paged attention where scores are so large that their last place is worth
more than the softmax's range: equal scores weigh the same, the largest takes all,
and scores a few places apart weigh as their differences say.

The data make every score exact in fp32 (one or two products of few bits), and
kq_scale = ln 2 makes the exponent of 2 the score itself, so a weight's
only errors are those of 2^x, of its two f16 terms and of the fp32 sums."""
import math

import pytest
import torch

import gqa_kv_head_gb300 as fr
from test_gpu_paged import check, make_batch, make_tables, starts

LN2 = torch.tensor(math.log(2.0)).float().item()       # (times log2 e: 1 in fp32)

CASES = {"small": ([1, 2, 1], [40, 300, 17], 4), "wide": ([8, 5, 8], [40, 300, 70], 4), "prompt": ([70, 64, 90], [100, 300, 90], 4)}


def scores_case(kind, hd, case, exps, parts):
    """Pages and queries whose scores are 2^exps + parts[i] 2^(exps - 23), i drawn
    for each key: q = (2^14, ...), k = (2^(exps - 14), parts[i])."""
    new, kv, G = CASES[case]
    n_pages, ps = sum(-(-n // 16) for n in kv) + 1, 16
    g = torch.Generator().manual_seed(hd + exps)
    scale = 0 if kind == "f16" else max(0, exps - 22)              # e4m3: K = 2^scale * code
    part = torch.tensor(parts, dtype=torch.float64)[torch.randint(0, len(parts), (n_pages, 1, ps), generator=g)]
    k = torch.zeros((n_pages, 1, ps, hd), dtype=torch.float64)
    k[..., 0], k[..., 1] = 2.0 ** (exps - 14 - scale), part
    v = torch.randn((n_pages, 1, ps, hd), generator=g)
    q = torch.zeros((sum(new), G, hd), dtype=torch.float16)
    q[..., 0], q[..., 1] = 2.0 ** 14, 2.0 ** (exps - 23 - scale)
    dt = torch.float16 if kind == "f16" else torch.float8_e4m3fn
    kp, vp = k.float().to(dt), v.to(dt)
    assert torch.equal(kp.double(), k)
    s = (float(q[0, 0, 0]) * k[..., 0] + float(q[0, 0, 1]) * part) * 2.0 ** scale
    assert torch.equal(s.float().double(), s) and torch.equal(s, 2.0 ** exps + part * 2.0 ** (exps - 23))
    return q, kp, vp, s, make_tables(kv, ps, n_pages, 5), 2.0 ** scale


def weighted(new, kv, table, G, s, v):
    """softmax in base 2 of exact scores s [n_pages, 1, ps], and its tolerance: 2^x
    and the f16 terms within 2^-21 each, in numerator and denominator; sums as in
    paged_ref.py; the reference may be the maximum itself (from 2^27 on, where 7
    less is no other number), so that f16's fixed step is 2^-25 of the largest weight."""
    hd = v.shape[-1]
    want = torch.zeros((sum(new), G, hd), dtype=torch.float64)
    tol = torch.zeros_like(want)
    at = starts(new)
    for b, n in enumerate(kv):
        ids = table[b, :-(-n // 16)].long()
        sb, vb = s[ids, 0].reshape(-1), v.double()[ids, 0].reshape(-1, hd)
        for i in range(new[b]):
            end = n - new[b] + i + 1
            w = torch.exp2(sb[:end] - sb[:end].max())
            w /= w.sum()
            want[at[b] + i] = w @ vb[:end]
            share = 4 * 2.0 ** -21 + 2 * (end / 16 + 400) * 2.0 ** -23
            tol[at[b] + i] = share * (w @ vb[:end].abs()) + 2.0 ** -25 * float(w.max()) * vb[:end].abs().sum(dim=0)
    return want, tol


def run(kind, hd, case, exps, parts):
    new, kv, G = CASES[case]
    q, k, v, s, table, scale = scores_case(kind, hd, case, exps, parts)
    sc = [None, None] if kind == "f16" else [torch.full(k.shape[:2], x).cuda() for x in (scale, 1.0)]
    out = fr.paged_attn(fr.PagedKV(k.cuda(), v.cuda(), *sc), make_batch(new, kv, table), q.cuda(), G, kq_scale=LN2)
    check(out, *weighted(new, kv, table, G, s, v), f"2^{exps}")


def test_inputs_are_exact():
    """On the CPU: the scores are what they are meant to be, in fp32 and in the cache's types."""
    for kind in ("f16", "e4m3"):
        for exps in (20, 24, 25, 26, 27, 28, 29):
            scores_case(kind, 64, "wide", exps, list(range(8)))
    assert torch.tensor(LN2 * 1.4426950408889634, dtype=torch.float64).float().item() == 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("exps", [20, 24, 25, 26, 27])
def test_scores_a_few_places_apart(kind, hd, case, exps):
    """The last place is 2^(exps - 23): 1/8 to 16. Differences of 0 to 7 of them."""
    run(kind, hd, case, exps, list(range(8)))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("exps", [28, 29])
def test_largest_scores_take_all(kind, hd, case, exps):
    """Ties at the maximum share the weight, whatever the last place is worth."""
    run(kind, hd, case, exps, [0, 1, 2, 3])


@pytest.mark.gpu
@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("kq", [1.0, -1.0, 0.37, 3.7])
@pytest.mark.parametrize("exps", [24, 28, 30, 40, 60, 100])
def test_e4m3_k_scales_of_any_size(case, hd, kq, exps):
    """Scores c * 2^exps, c = 1..15, through K scales up to 2^100: the keys with the
    largest (smallest) c share the weight."""
    new, kv, G = CASES[case]
    n_pages = sum(-(-n // 16) for n in kv) + 1
    g = torch.Generator().manual_seed(exps)
    table = make_tables(kv, 16, n_pages, 5)
    c = torch.randint(1, 16, (n_pages, 1, 16), generator=g).double()
    k = torch.zeros((n_pages, 1, 16, hd), dtype=torch.float64)
    k[..., 3] = c
    v = torch.randn((n_pages, 1, 16, hd), generator=g).to(torch.float8_e4m3fn)
    q = torch.zeros((sum(new), G, hd), dtype=torch.float16)
    q[..., 3] = 1.0
    sc = [torch.full((n_pages, 1), x).cuda() for x in (2.0 ** exps, 1.0)]
    cache = fr.PagedKV(k.to(torch.float8_e4m3fn).cuda(), v.cuda(), *sc)
    out = fr.paged_attn(cache, make_batch(new, kv, table), q.cuda(), G, kq_scale=kq)
    # (two scores lie 2^exps |kq| log2 e apart, more than 8 million: nothing but ties is left of the weights)
    check(out, *weighted(new, kv, table, G, c * (2.0 ** 20 if kq > 0 else -2.0 ** 20), v), f"{case} 2^{exps}")
