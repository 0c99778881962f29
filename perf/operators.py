"""Cases for timing and comparing the paged-cache operators.

Three operators of a serving step over a paged K/V cache:

  append   the step's new K and V rows: K rotated (NEOX RoPE), both written into
           the pages of their sequences, as f16 or as e4m3 with one power-of-two
           scale for each page and head
  attend   attention of the step's query rows over an f16 paged cache
  attend   the same over an e4m3 paged cache with a scale for each page and head

listed() names fixed cases, draw() one more from the same ranges; prepare()
makes a case's inputs, run() makes one pass (plain torch operations, or the
library's calls where `own` is true), exact() is the result in 64 bits and
work() the bytes and operations of one pass.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------

def _append(name, kv, rows, n_seq, max_len, new, hd, heads, page):
    return {"name": name, "op": "append", "kv": kv, "rows": rows, "n_seq": n_seq, "max_len": max_len, "new": new,
            "hd": hd, "kv_heads": heads, "page": page}


def _attend(name, kv, n_seq, max_len, new, hd, heads, group, page, window=0, causal=True):
    return {"name": name, "op": "attend", "kv": kv, "n_seq": n_seq, "max_len": max_len, "new": new, "hd": hd,
            "kv_heads": heads, "group": group, "page": page, "window": window, "causal": causal}


def listed():
    return [
        # one robot-policy decode token, one shared KV head: pure latency
        _append("append f16 1x1", "f16", "f32", 1, 968, 1, 256, 1, 64),
        # a batch of chats, one new token each, rows out of a half-precision projection
        _append("append f16 64x1", "f16", "f16", 64, 1024, 1, 128, 8, 16),
        # prompts of uneven lengths joining a running batch
        _append("append f16 prompts", "f16", "f32", 8, 2048, 2000, 128, 8, 64),
        # the batch of chats on an 8-bit cache
        _append("append e4m3 64x1", "e4m3", "f32", 64, 1024, 1, 128, 8, 64),
        # prompts into an 8-bit cache; the first page of each is partly full
        _append("append e4m3 prompts", "e4m3", "f16", 7, 2500, 2000, 128, 8, 64),
        # one token of one short sequence, 8 query heads on one KV head: latency
        _attend("attend f16 1x968", "f16", 1, 968, 1, 256, 1, 8, 64),
        # a batch of chats of uneven lengths, grouped heads, one token each
        _attend("attend f16 64x8192", "f16", 64, 8192, 1, 128, 8, 4, 64),
        # one long document, four tokens verified at once, hd 256
        _attend("attend f16 1x65536", "f16", 1, 65536, 4, 256, 1, 8, 128),
        # long chats through a layer with a sliding window; pages of 16 tokens
        _attend("attend f16 window", "f16", 16, 32768, 2, 128, 4, 7, 16, window=4096),
        # four short chats on an 8-bit cache
        _attend("attend e4m3 4x1000", "e4m3", 4, 1000, 1, 128, 8, 4, 32),
        # the uneven batch of chats on an 8-bit cache
        _attend("attend e4m3 64x8192", "e4m3", 64, 8192, 1, 128, 8, 4, 64),
        # one very long document on an 8-bit cache, two tokens
        _attend("attend e4m3 1x131072", "e4m3", 1, 131072, 2, 128, 8, 8, 64),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hd = rng.choice([64, 128, 256])
    kv = rng.choice(["f16", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 2, 4, 5, 8])
    if rng.random() < 0.4:
        n_seq = _between(rng, 1, 64)
        new = _between(rng, 1, max(1, 8000 // n_seq)) if rng.random() < 0.6 else 1
        return {"op": "append", "kv": kv, "rows": rng.choice(["f32", "f16"]), "n_seq": n_seq,
                "max_len": new + _between(rng, 1, 1200), "new": new, "hd": hd, "kv_heads": heads, "page": page}
    n_seq = _between(rng, 1, 64)
    new = rng.choice([1, 1, 1, 2, 3, 4, 8])
    longest = min(131072, 64 * 8192 * 8 * 128 // (n_seq * heads * hd))
    max_len = _between(rng, 64, max(65, longest))
    window = _between(rng, 16, max_len) if rng.random() < 0.25 else 0
    group = rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    while n_seq * heads * max_len * hd * group * new > 64 * 8 * 8192 * 128 * 16:
        max_len = max(64, max_len // 2)
    return {"op": "attend", "kv": kv, "n_seq": n_seq, "max_len": max_len, "new": new, "hd": hd, "kv_heads": heads,
            "group": group, "page": page, "window": min(window, max_len), "causal": window > 0 or rng.random() < 0.8}


def _lengths(case):
    """New tokens and keys of each sequence: uneven, the last ones the longest; from the case alone."""
    n, new, longest = case["n_seq"], case["new"], case["max_len"]
    if n == 1:
        return [new], [longest]
    frac = [((i * 0.6180339887498949) % 1.0) for i in range(n - 1)] + [1.0]
    if case["op"] == "append" and new > 16:
        q = [max(1, int(round(new * (0.02 + 0.98 * f * f)))) for f in frac]
    else:
        q = [new] * n
    kv = [max(qi, int(round(longest * max(f, 1.0 / longest)))) for qi, f in zip(q, frac)]
    return q, kv


def _rows_in_view(case, q, kv):
    """Keys that some query row of a sequence sees."""
    w = case.get("window", 0)
    return kv if not w else min(kv, w + q - 1)


def work(case):
    q, kv = _lengths(case)
    H, hd = case["kv_heads"], case["hd"]
    elem = 2 if case["kv"] == "f16" else 1
    tables = 4 * sum(-(-k // case["page"]) for k in kv) + 8 * len(q)
    if case["op"] == "append":
        n = sum(q)
        rows = 4 if case["rows"] == "f32" else 2
        touched = sum(-(-k // case["page"]) - (k - a) // case["page"] for a, k in zip(q, kv))
        tables = 4 * touched + 8 * len(q) + 4 * n
        scales = 0 if case["kv"] == "f16" else 2 * 2 * 4 * touched * H
        return {"bytes": 2 * n * H * hd * (rows + elem) + scales + tables, "flops": 3.0 * n * H * hd}
    G = case["group"]
    keys = sum(_rows_in_view(case, a, k) for a, k in zip(q, kv))
    scales = 0 if case["kv"] == "f16" else 2 * 4 * H * sum(
        -(-_rows_in_view(case, a, k) // case["page"]) for a, k in zip(q, kv))
    scored = 0
    for a, k in zip(q, kv):
        if case["causal"]:
            w = case["window"] or k
            scored += sum(min(w, k - a + i + 1) for i in range(a))
        else:
            scored += a * k
    return {"bytes": 2 * keys * H * hd * elem + sum(q) * H * G * hd * (2 + 4) + scales + tables,
            "flops": 4.0 * scored * G * H * hd}


# ---- inputs -----------------------------------------------------------------

def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s; at least 2^-100."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1)
    k = torch.where(m <= 0.875, e - 9, e - 8)      # 448 = 0.875 * 2^9
    k = torch.where(amax > 0, k, torch.full_like(k, -100)).clamp(min=-100)
    return torch.exp2(k.double()).float()


def _to_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    q, kv = _lengths(case)
    n_seq, H, hd, ps = case["n_seq"], case["kv_heads"], case["hd"], case["page"]
    n_tok = sum(q)
    need = [-(-k // ps) for k in kv]
    max_pages = max(need)
    n_pages = sum(need) + 3                        # a few pages belong to nobody
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device=dev)   # entries behind a sequence's pages: unused
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st = {
        "case": dict(case), "table": table,
        "tok_start": torch.tensor([0] + [sum(q[:i + 1]) for i in range(n_seq)], dtype=torch.int32, device=dev),
        "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev),
    }
    pages = []
    for which in range(2):
        x = torch.randn((n_pages, H, ps, hd), generator=g, device=dev)
        if which == 0:                             # a few K channels run hot, as they do in trained models
            x *= 1.0 + 3.0 * (torch.rand((1, H, 1, hd), generator=g, device=dev) < 0.03)
        if case["kv"] == "f16":
            pages.append((x.half(), None))
        else:
            x *= torch.exp2(torch.randn((n_pages, H, 1, 1), generator=g, device=dev))
            s = _pow2_scale(x.abs().amax(dim=(2, 3)))
            pages.append((_to_e4m3(x / s[:, :, None, None]), s))
        del x
    (st["k"], st["k_scale"]), (st["v"], st["v_scale"]) = pages
    if case["op"] == "append":
        rows = torch.float32 if case["rows"] == "f32" else torch.float16
        qkv = torch.randn((n_tok, 4 * H * hd), generator=g, device=dev).to(rows)   # Q columns, then K, then V
        st["k_new"] = qkv[:, 2 * H * hd:3 * H * hd].view(n_tok, H, hd)
        st["v_new"] = qkv[:, 3 * H * hd:].view(n_tok, H, hd)
        st["pos"] = torch.cat([torch.arange(k - a, k, dtype=torch.int32) for a, k in zip(q, kv)]).to(dev)
        st["rope"] = {"n_dims": hd, "freq_base": 10000.0}
    else:
        G = case["group"]
        x = torch.randn((n_tok, H * G, hd), generator=g, device=dev) * (1.0 / math.sqrt(hd))
        st["q16"] = x.half()                       # what qkv_post leaves: rotated and scaled rows
        st["out"] = torch.empty((n_tok, H * G, hd), dtype=torch.float32, device=dev)
    if own:
        import gqa_kv_head_gb300 as fr
        st["cache"] = fr.PagedKV(st["k"], st["v"], st["k_scale"], st["v_scale"])
        st["batch"] = fr.PagedBatch(st["tok_start"], st["kv_len"], st["table"])
        if case["op"] == "append":
            st["rope_params"] = fr.rope_params(**st["rope"])
        else:
            st["workspace"] = fr.make_paged_workspace(H * case["group"], H, hd)
    return st


# ---- one pass -----------------------------------------------------------------

def run(st):
    case = st["case"]
    if case["op"] == "append":
        if own:
            import gqa_kv_head_gb300 as fr
            fr.kv_append_paged(st["cache"], st["batch"], st["k_new"], st["v_new"], st["pos"], st["rope_params"])
        else:
            _append_plain(st)
        if case["kv"] == "f16":
            return {"k": st["k"], "v": st["v"]}
        return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if own:
        import gqa_kv_head_gb300 as fr
        return fr.paged_attn(st["cache"], st["batch"], st["q16"], case["kv_heads"] * case["group"],
                             causal=case["causal"], window=case["window"], out=st["out"], workspace=st["workspace"])
    return _attend_plain(st)


def _slots(st):
    """Sequence, page and row in the page of every new token."""
    tok_start, kv_len = st["tok_start"].long(), st["kv_len"].long()
    n_tok = st["pos"].shape[0]
    t = torch.arange(n_tok, device=kv_len.device)
    b = torch.searchsorted(tok_start[1:].contiguous(), t, right=True)
    slot = kv_len[b] - tok_start[b + 1] + t
    ps = st["k"].shape[2]
    return st["table"].long()[b, slot // ps], slot % ps


def _rotate_plain(st):
    x = st["k_new"].float()
    half = x.shape[2] // 2
    w = st["rope"]["freq_base"] ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / x.shape[2])
    a = st["pos"].double()[:, None] * w                          # far positions: angles in 64 bits
    c, s = torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]
    lo, hi = x[..., :half], x[..., half:]
    return torch.cat([lo * c - hi * s, lo * s + hi * c], dim=2)


def _append_plain(st):
    page, row = _slots(st)
    rows = {"k": _rotate_plain(st), "v": st["v_new"].float()}
    _put_plain(st, "k", rows["k"], page, row)
    _put_plain(st, "v", rows["v"], page, row)


def _put_plain(st, name, rows, page, row):
    cache, scale = st[name], st[name + "_scale"]
    n_pages, H, ps, hd = cache.shape
    if scale is None:
        cache[page, :, row] = rows.half()
        return
    first = torch.full((n_pages,), ps, device=cache.device).scatter_reduce(0, page, row, "amin")
    amax = torch.zeros((n_pages, H), device=cache.device).scatter_reduce(
        0, page[:, None].expand(-1, H), rows.abs().amax(dim=2), "amax")
    touched = (first < ps)[:, None]
    wanted = torch.maximum(_pow2_scale(amax), torch.where(first[:, None] > 0, scale, torch.zeros_like(scale)))
    new = torch.where(touched, wanted, scale)
    # rows already in a page whose scale grew are stored again at the new scale
    grown = (new != scale)[:, :, None] & (torch.arange(ps, device=cache.device) < first[:, None])[:, None, :]
    ratio = torch.where(grown, (scale / new)[:, :, None], torch.ones((), device=cache.device))
    stored = (cache.float() * ratio[..., None]).to(torch.float8_e4m3fn)
    codes = cache.view(torch.uint8)
    codes.copy_(torch.where(grown[..., None], stored.view(torch.uint8), codes))
    codes[page, :, row] = _to_e4m3(rows / new[page][:, :, None]).view(torch.uint8)
    scale.copy_(new)


def _attend_plain(st):
    case = st["case"]
    k, v, table = st["k"], st["v"], st["table"].long().clamp(min=0)
    n_pages, H, ps, hd = k.shape
    n_seq, max_pages = table.shape
    L, G, n = max_pages * ps, case["group"], case["new"]        # every sequence brings n query tokens
    kf = k.float() if st["k_scale"] is None else k.float() * st["k_scale"][:, :, None, None]
    vf = v.float() if st["v_scale"] is None else v.float() * st["v_scale"][:, :, None, None]
    kf = kf[table].permute(0, 2, 1, 3, 4).reshape(n_seq, H, L, hd)
    vf = vf[table].permute(0, 2, 1, 3, 4).reshape(n_seq, H, L, hd)
    q = st["q16"].float().view(n_seq, n, H, G, hd).permute(0, 2, 1, 3, 4).reshape(n_seq, H, n * G, hd)
    j = torch.arange(L, device=k.device)
    kv_len = st["kv_len"].long()[:, None, None]
    here = kv_len - n + torch.arange(n, device=k.device)[None, :, None]     # the key of each query token itself
    seen = (j < kv_len).expand(n_seq, n, L)
    if case["causal"]:
        seen = seen & (j <= here)
        if case["window"]:
            seen = seen & (j > here - case["window"])
    seen = seen[:, None, :, None, :].expand(n_seq, 1, n, G, L).reshape(n_seq, 1, n * G, L)
    s = torch.matmul(q, kf.transpose(2, 3)).masked_fill(~seen, float("-inf"))
    m = s.amax(dim=3, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s - m)
    l = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, vf) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(n_seq, H, n, G, hd).permute(0, 2, 1, 3, 4).reshape(n_seq * n, H * G, hd)


# ---- 64 bits --------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    q, kv = _lengths(case)
    starts = [sum(q[:i]) for i in range(len(q))]
    return _append_exact(st, q, kv, starts) if case["op"] == "append" else _attend_exact(st, q, kv, starts)


def _append_exact(st, q, kv, starts):
    case = st["case"]
    ps, hd, H = case["page"], case["hd"], case["kv_heads"]
    half = hd // 2
    d = torch.arange(half, dtype=torch.float64, device="cuda")
    angle = st["pos"].double()[:, None, None] / st["rope"]["freq_base"] ** (d / half)
    z = torch.complex(st["k_new"][..., :half].double(), st["k_new"][..., half:].double())
    z = z * torch.polar(torch.ones_like(angle), angle)
    new = {"k": torch.cat([z.real, z.imag], dim=2), "v": st["v_new"].double()}
    res = {}
    for name in ("k", "v"):
        pool = st[name].double()
        scale = None if st[name + "_scale"] is None else st[name + "_scale"].double()
        for b in range(case["n_seq"]):
            for p in range((kv[b] - q[b]) // ps, -(-kv[b] // ps)):
                lo, hi = max(kv[b] - q[b], p * ps), min(kv[b], (p + 1) * ps)   # cache rows written in this page
                page = int(st["table"][b, p])
                x = new[name][starts[b] + lo - (kv[b] - q[b]):starts[b] + hi - (kv[b] - q[b])].transpose(0, 1)
                if scale is not None:
                    top = x.abs().amax(dim=(1, 2)) / E4M3_MAX
                    s = torch.exp2(torch.ceil(torch.log2(top)))
                    s = torch.where(s < top, 2 * s, torch.where(s / 2 >= top, s / 2, s))
                    if lo > p * ps:
                        s = torch.maximum(s, scale[page])
                        pool[page, :, :lo - p * ps] *= (scale[page] / s)[:, None, None]
                    scale[page] = s
                    x = x / s[:, None, None]
                pool[page, :, lo - p * ps:hi - p * ps] = x
        res[name] = pool
        if scale is not None:
            res[name + "_scale"] = scale
    return res


def _attend_exact(st, q, kv, starts):
    case = st["case"]
    H, G, hd, ps = case["kv_heads"], case["group"], case["hd"], case["page"]
    out = torch.zeros((sum(q), H * G, hd), dtype=torch.float64, device="cuda")
    for b, (a, n_kv) in enumerate(zip(q, kv)):
        if not a:
            continue
        ids = st["table"][b, :-(-n_kv // ps)].long()
        k, v = st["k"][ids].double(), st["v"][ids].double()
        if st["k_scale"] is not None:
            k = k * st["k_scale"][ids].double()[:, :, None, None]
            v = v * st["v_scale"][ids].double()[:, :, None, None]
        for t in range(a):
            pos = n_kv - a + t
            end = pos + 1 if case["causal"] else n_kv
            begin = max(0, pos + 1 - case["window"]) if case["causal"] and case["window"] else 0
            for h in range(H):
                kh = k[:, h].reshape(-1, hd)[begin:end]
                vh = v[:, h].reshape(-1, hd)[begin:end]
                if end <= begin:
                    continue
                x = st["q16"][starts[b] + t, h * G:(h + 1) * G].double()
                out[starts[b] + t, h * G:(h + 1) * G] = torch.softmax(x @ kh.T, dim=1) @ vh
    return out
