"""Sums over many keys: what the matrix units' accumulators drop at each step is always
towards zero, so with values of one sign it would grow with the length; the mean error
of many results is held to a bound that does not. And long sums whose reference moves
late, against the 64-bit form, computed with torch in 64 bits on the GPU."""
import pytest
import torch

import gqa_kv_head_gb300 as fr

pytestmark = pytest.mark.gpu

PS = 64
# Keys that one accumulator takes at most, in 16-key steps of two products (P_hi V and P_lo V): each
# step drops less than 2^-23 of what it holds, which is less than the final sum.
STEPS = {("wide", "f16"): 2 * 16 * 4, ("wide", "e4m3"): 2 * 48 * 4, ("few", "f16"): 2 * 64, ("few", "e4m3"): 2 * 64}


def long_case(kind, hd, H, G, n, n_seq, kv, window, sinks, k, v, v_scale=1.0, q=None, seed=0):
    """Sequences of kv keys that share their pages (k, v: [kv, H, hd] f32; v_scale: [n_pages] or a number);
    yields (out, w, V, ds) for some of the sequences and heads, in 64 bits."""
    n_pages = -(-kv // PS)

    def pages(x):
        x = torch.cat([x, x.new_zeros(n_pages * PS - kv, H, hd)])
        return x.view(n_pages, PS, H, hd).permute(0, 2, 1, 3).contiguous()
    vs = (torch.ones(n_pages, device="cuda") * v_scale)[:, None].expand(n_pages, H).contiguous()
    if kind == "f16":
        kp, vp = pages(k).half(), pages(v).half()
        cache, kd, vd = fr.PagedKV(kp, vp), kp.double(), vp.double()
    else:
        ks = torch.full_like(vs, 2.0 ** -6)
        kp, vp = (pages(k) / 2.0 ** -6).to(torch.float8_e4m3fn), (pages(v) * 256.0).to(torch.float8_e4m3fn)
        vs = vs / 256.0
        cache, kd, vd = fr.PagedKV(kp, vp, ks, vs), kp.double() * 2.0 ** -6, vp.double() * vs.double()[:, :, None, None]
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    order = torch.argsort(table)                 # page p holds rows order[p] * PS ..
    cache.k_pages.view(torch.uint8).copy_(cache.k_pages.view(torch.uint8)[order.cuda()].clone())
    cache.v_pages.view(torch.uint8).copy_(cache.v_pages.view(torch.uint8)[order.cuda()].clone())
    if cache.v_scale is not None:
        cache.v_scale.copy_(cache.v_scale[order.cuda()].clone())
    ts = torch.arange(n_seq + 1, dtype=torch.int32, device="cuda") * n
    lens = torch.full((n_seq,), kv, dtype=torch.int32, device="cuda")
    ws = fr.make_paged_workspace(H * G, H, hd)
    out = fr.paged_attn(cache, fr.PagedBatch(ts, lens, table.cuda().repeat(n_seq, 1)), q, H * G, window=window, sinks=sinks, workspace=ws)
    fr.workspace_check(ws)
    j = torch.arange(kv, device="cuda")
    for b in range(0, n_seq, max(1, n_seq // 3)):
        for h in range(H):
            K, V = kd[:, h].reshape(-1, hd)[:kv], vd[:, h].reshape(-1, hd)[:kv]
            Q = q[b * n:(b + 1) * n, h * G:(h + 1) * G].double().reshape(-1, hd)
            p = (kv - n + torch.arange(n, device="cuda")).repeat_interleave(G)[:, None]
            see = (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p
            w = torch.softmax((Q @ K.T).masked_fill(~see, -float("inf")), dim=1)
            ds = (hd + 4) * 2.0 ** -23 * (Q.abs() @ K.abs().T).amax(dim=1)
            got = out[b * n:(b + 1) * n, h * G:(h + 1) * G].double().reshape(-1, hd)
            yield got, w, V, ds


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (32900, 4)])
@pytest.mark.parametrize("form,G,n,n_seq", [("wide", 8, 16, 40), ("few", 4, 1, 160), ("few", 4, 3, 160)])
def test_values_of_one_sign(form, G, n, n_seq, kind, hd, window, sinks):
    """Weights about equal, values in 0.5 .. 1.5. Beside the drops (see STEPS) a result errs in its weights,
    by 2^-21 each at most, and in roundings to nearest, neither to one side: 2^-20 for their mean."""
    H, kv = 4, 33000
    g = torch.Generator(device="cuda").manual_seed(hd)
    k = torch.randn((kv, H, hd), generator=g, device="cuda") * 0.5
    v = torch.rand((kv, H, hd), generator=g, device="cuda") + 0.5
    q = (torch.randn((n_seq * n, H * G, hd), generator=g, device="cuda") * 0.02).half()
    errs = []
    for got, w, V, _ in long_case(kind, hd, H, G, n, n_seq, kv, window, sinks, k, v, q=q):
        want = w @ V
        errs.append(((got - want) / want).flatten())
    mean = float(torch.cat(errs).mean())
    assert abs(mean) <= STEPS[form, kind] * 2.0 ** -23 + 2.0 ** -20, mean


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5900, 70)])
@pytest.mark.parametrize("G,n,n_seq,kv", [(8, 16, 40, 6001), (8, 16, 3, 30011), (5, 20, 50, 4100), (4, 1, 170, 9001), (4, 7, 120, 5003),
                                            (3, 4, 2, 30011)])
def test_references_that_move_late(kind, hd, window, sinks, G, n, n_seq, kv):
    """Scores grow along the keys, and with them the scales of V's pages, so that what was summed
    up is scaled again and again. The tolerance is that of paged_ref.attention, with one dim that makes
    the scores (exact products, the rounding of scale and exponent left: ds)."""
    H = 4 if n_seq > 3 else 1
    g = torch.Generator(device="cuda").manual_seed(hd + kv)
    k = torch.zeros((kv, H, hd), device="cuda")
    k[..., 0] = (torch.arange(kv, device="cuda") // 100 * (100 * 40.0 / kv))[:, None]
    k[..., 1] = torch.randn((kv, H), generator=g, device="cuda")
    k[..., 0].clamp_(max=6.9 if kind == "e4m3" else 40.0)
    v = torch.randn((kv, H, hd), generator=g, device="cuda").clamp(-1.7, 1.7)
    q = torch.zeros((n_seq * n, H * G, hd), device="cuda")
    q[..., 0] = 6.0 if kind == "e4m3" else 1.0
    q[..., 1] = torch.rand(q.shape[:2], generator=g, device="cuda")
    n_pages = -(-kv // PS)
    steps = 2.0 ** (torch.arange(n_pages, device="cuda") * 12 // n_pages).float() if kind == "e4m3" else 1.0
    for got, w, V, ds in long_case(kind, hd, H, G, n, n_seq, kv, window, sinks, k, v, steps, q.half()):
        share = 2 * ds + 2 * 2.0 ** -21 + (kv / 16 + 400) * 2.0 ** -23
        top = float(steps.max()) / 256 if kind == "e4m3" else 1.0
        code = V.abs()
        if kind == "e4m3":
            code = code / (steps / 256.0).double().repeat_interleave(PS)[:kv, None]
        tol = (w @ V.abs()) * (2 * share)[:, None] + 2.0 ** -32 * w.amax(dim=1)[:, None] * top * code.sum(dim=0)
        d = (got - w @ V).abs()
        assert bool((d <= tol).all()), float((d / tol).max())
