"""Paged attention over token ranges that are not in order."""
import pytest
import torch

import gqa_kv_head_gb300 as fr
from test_gpu_paged import check, make_cache, make_tables, rand_q
import paged_ref as ref


def units(n_seq, n_tok, row_tile, keys, unit, ends):
    """Units of work that the ranges 0..n_tok of every other sequence count, as the kernels count them."""
    return -(-n_seq // 2) * -(-n_tok // row_tile) * (ends + -(-keys // unit))


def test_the_overlapping_cases_pass_31_bits_and_wrap_to_positive_numbers():
    for args in ((65534, 1 << 20, 32, 1024, 256, 2), (8192, 1 << 20, 128, 9984, 64, 4)):
        n = units(*args)
        assert n >= 1 << 31 and 0 < n % (1 << 32) < 1 << 31


@pytest.mark.gpu
@pytest.mark.parametrize("n_seq,keys", [(65534, 1024), (8192, 9984)], ids=["32-row tiles", "128-row tiles"])
def test_overlapping_ranges_of_more_work_than_an_int_counts(n_seq, keys):
    """tok_start 0, n, 0, n, ...: every other range is backwards, and skipped; the
    others are all of the tokens each, 2^33 rows and more. Nothing is written, the
    status word tells, and the workspace serves the next call."""
    hd, ps, n_tok = 64, 16, 1 << 20
    (k, _, v, _), cache = make_cache("f16", 4, 1, ps, hd)
    ts = torch.zeros(n_seq + 1, dtype=torch.int32)
    ts[1::2] = n_tok
    table = torch.zeros((n_seq, keys // ps), dtype=torch.int32, device="cuda")
    batch = fr.PagedBatch(ts.cuda(), torch.full((n_seq,), keys, dtype=torch.int32, device="cuda"), table)
    q = torch.zeros((n_tok, 1, hd), dtype=torch.float16, device="cuda")
    out = torch.full((n_tok, 1, hd), 9.0, device="cuda")
    ws = fr.make_paged_workspace(1, 1, hd)
    fr.paged_attn(cache, batch, q, 1, causal=False, out=out, workspace=ws)
    with pytest.raises(fr.FrError) as e:
        fr.workspace_check(ws)
    assert e.value.status == 6
    assert bool((out == 9.0).all())
    kv, table = [40, 17], make_tables([40, 17], ps, 5)
    (k, _, v, _), cache = make_cache("f16", 5, 1, ps, hd)
    q = rand_q(2, 1, hd)
    batch = fr.PagedBatch(torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), torch.tensor(kv, dtype=torch.int32).cuda(), table.cuda())
    got = fr.paged_attn(cache, batch, q.cuda(), 1, workspace=ws)
    check(got, *ref.attention(q, k.double(), v.double(), [0, 1, 2], kv, table, 1))
    fr.workspace_check(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("start,skipped", [([1, 3, 2, 4], False), ([0, 3, 1, 4], True), ([0, 4, 0, 4], True), ([0, 4, -1, 3], False), ([2, 4, 3, 4], False)])
def test_ranges_out_of_order(start, skipped):
    """The backward range is skipped; the others are served as long as they have no
    more tokens than the step together, and else nothing is."""
    hd, G, ps, kv = 64, 2, 16, [40, 30, 21]
    (k, _, v, _), cache = make_cache("f16", 8, 1, ps, hd)
    table = make_tables(kv, ps, 8)
    q = rand_q(4, G, hd)
    batch = fr.PagedBatch(torch.tensor(start, dtype=torch.int32).cuda(), torch.tensor(kv, dtype=torch.int32).cuda(), table.cuda())
    out = torch.full((4, G, hd), 9.0, device="cuda")
    ws = fr.make_paged_workspace(G, 1, hd)
    fr.paged_attn(cache, batch, q.cuda(), G, out=out, workspace=ws)
    with pytest.raises(fr.FrError) as e:
        fr.workspace_check(ws)
    assert e.value.status == 6
    served = torch.zeros(4, dtype=torch.bool)
    for b in range(3):
        t0, t1 = start[b], start[b + 1]
        if skipped or t0 < 0 or t1 < t0:
            continue
        served[t0:t1] = True
        want, tol = ref.attention(q[t0:t1], k.double(), v.double(), [0, t1 - t0], kv[b:b + 1], table[b:b + 1], G)
        only = [t for t in range(t0, t1) if not any(start[c] <= t < start[c + 1] for c in range(3) if c != b)]    # (one sequence's row)
        rows = [t - t0 for t in only]
        check(out[only], want[rows], tol[rows])
    assert bool((out[~served] == 9.0).all())
