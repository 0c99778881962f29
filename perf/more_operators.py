"""Cases for timing and comparing the operators of a serving step around the paged cache.

  qkv      a step's query, key and value rows: queries and keys normed for each
           head (RMS, with weights), rotated (half or interleaved pairs, part of
           the head, YaRN), queries scaled to f16 rows, keys and values written
           into the pages of their sequences (f16, or e4m3 with a power-of-two
           scale for each page and head)
  attend   attention over the paged cache with a sliding window and a few first
           tokens that stay visible
  pages    the pages' own bookkeeping: sequences that share the pages of a prefix
           (fork), pages for a step's new rows (reserve, with a copy of a shared
           last page), pages given back (free, trim), and a pool moved together
           (compact)

listed() names fixed cases, draw() one more from the same ranges; prepare()
makes a case's inputs, run() makes one pass (plain torch operations, or the
library's calls where `own` is true), exact() is the result in 64 bits and
work() the bytes and operations of one pass.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
ROWS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------

def _qkv(name, rows, kv, n_seq, max_len, new, hd, heads, group, page, norm=True, interleaved=False, n_dims=0, yarn=False):
    return {"name": name, "op": "qkv", "rows": rows, "kv": kv, "n_seq": n_seq, "max_len": max_len, "new": new, "hd": hd,
            "kv_heads": heads, "group": group, "page": page, "norm": norm, "interleaved": interleaved,
            "n_dims": n_dims or hd, "yarn": yarn}


def _attend(name, kv, n_seq, max_len, new, hd, heads, group, page, window, sinks):
    return {"name": name, "op": "attend", "kv": kv, "n_seq": n_seq, "max_len": max_len, "new": new, "hd": hd,
            "kv_heads": heads, "group": group, "page": page, "window": window, "sinks": sinks}


def _pages(name, what, kv, n_seq, max_len, new, hd, heads, page, width=0, prefix=0, window=0, sinks=0):
    return {"name": name, "op": "pages", "what": what, "kv": kv, "n_seq": n_seq, "max_len": max_len, "new": new, "hd": hd,
            "kv_heads": heads, "page": page, "width": width, "prefix": prefix, "window": window, "sinks": sinks}


def listed():
    return [
        # one token of one chat, rows out of a half-precision projection: pure latency
        _qkv("qkv f16 1x1", "f16", "f16", 1, 968, 1, 128, 8, 4, 64),
        # a batch of chats, one token each, on an 8-bit cache
        _qkv("qkv bf16 to e4m3 64x1", "bf16", "e4m3", 64, 1024, 1, 128, 8, 4, 64),
        # prompts of uneven lengths joining a running batch
        _qkv("qkv bf16 prompts", "bf16", "f16", 8, 2048, 2000, 128, 8, 4, 64),
        # prompts of a model with interleaved pairs, half of the head rotated, scaled for a longer context, 8-bit cache
        _qkv("qkv f32 to e4m3 prompts", "f32", "e4m3", 7, 2500, 2000, 64, 5, 3, 32, interleaved=True, n_dims=32, yarn=True),
        # one endless chat, one token: latency
        _attend("sinks f16 1x65536", "f16", 1, 65536, 1, 128, 8, 4, 64, 1024, 4),
        # a batch of long chats of uneven lengths on an 8-bit cache
        _attend("sinks e4m3 64x16384", "e4m3", 64, 16384, 1, 128, 8, 4, 64, 4096, 64),
        # four tokens verified at once, hd 256, small pages
        _attend("sinks f16 16x20000 verified", "f16", 16, 20000, 4, 256, 2, 8, 16, 2048, 5),
        # chunks of four long prompts
        _attend("sinks f16 chunks", "f16", 4, 16384, 512, 128, 8, 4, 64, 2048, 16),
        # several samples of each of sixteen chats: children share the pages, and copy the last one to go on
        _pages("pages branch f16", "branch", "f16", 16, 4000, 1, 128, 8, 64, width=4),
        # requests that start from one system prompt, on an 8-bit cache
        _pages("pages prefix e4m3", "branch", "e4m3", 1, 4500, 1500, 128, 8, 64, width=32, prefix=4100),
        # endless chats one token on: pages that left the window go, and come back for new rows
        _pages("pages stream", "stream", "f16", 64, 16384, 1, 64, 1, 16, window=4096, sinks=4),
        # a pool with a third of its sequences gone, moved together
        _pages("pages compact f16", "compact", "f16", 24, 8000, 0, 128, 8, 64),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hd = rng.choice([64, 128, 256])
    kv = rng.choice(["f16", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    op = rng.choice(["qkv", "attend", "pages"])
    n_seq = _between(rng, 1, 64)
    if op == "qkv":
        most = min(2000, 8000 * 6 * 8 * 128 // (n_seq * heads * (group + 2) * hd))
        new = _between(rng, 1, max(1, most)) if rng.random() < 0.6 else 1
        return {"op": "qkv", "rows": rng.choice(["f32", "f16", "bf16"]), "kv": kv, "n_seq": n_seq,
                "max_len": new + _between(rng, 1, 1200), "new": new, "hd": hd, "kv_heads": heads, "group": group,
                "page": page, "norm": rng.random() < 0.8, "interleaved": rng.random() < 0.5,
                "n_dims": rng.choice([hd, hd, hd // 2, hd // 4 * 3]), "yarn": rng.random() < 0.4}
    if op == "attend":
        new = rng.choice([1, 1, 1, 2, 4, 8, 64, 300])
        window = _between(rng, 64, 8192)
        while (n_seq * heads * group * new * (window + new) * hd > 4 * 32 * 512 * 2560 * 128 or
               n_seq * heads * (window + new + 256) * hd > 64 * 8 * 4200 * 128 // (2 if kv == "f16" else 1)):
            n_seq, new, window = max(1, n_seq // 2), max(1, new // 2), max(64, window * 3 // 4)
        longest = min(65536, 64 * 16384 * 8 * 128 // (n_seq * heads * hd))
        max_len = max(new, _between(rng, window // 2, max(window, longest)))
        return {"op": "attend", "kv": kv, "n_seq": n_seq, "max_len": max_len, "new": new, "hd": hd, "kv_heads": heads,
                "group": group, "page": page, "window": window, "sinks": _between(rng, 1, 256)}
    what = rng.choice(["branch", "prefix", "stream", "compact"])
    if what == "stream":
        window = _between(rng, 64, 8192)
        return {"op": "pages", "what": what, "kv": kv, "n_seq": n_seq, "max_len": window + _between(rng, 300, 8192),
                "new": rng.choice([1, 1, 4]), "hd": 64, "kv_heads": 1, "page": page, "width": 0, "prefix": 0,
                "window": window, "sinks": _between(rng, 1, 256)}
    room = 16 * 8192 * 8 * 128 // (heads * hd)                                   # tokens that the pool may hold
    if what == "compact":
        n_seq = max(3, n_seq)
        return {"op": "pages", "what": what, "kv": kv, "n_seq": n_seq, "max_len": _between(rng, 2, max(3, min(16000, room // n_seq))),
                "new": 0, "hd": hd, "kv_heads": heads, "page": page, "width": 0, "prefix": 0, "window": 0, "sinks": 0}
    n_seq = min(n_seq, 16) if what == "branch" else 1
    width = _between(rng, 1, 8 if what == "branch" else 48)
    new = rng.choice([1, 1, 3, 40]) if what == "branch" else _between(rng, 1, max(1, min(1500, room // (2 * width))))
    max_len = _between(rng, 2, max(3, min(8000, room // (2 * n_seq))))
    return {"op": "pages", "what": "branch", "kv": kv, "n_seq": n_seq, "max_len": max_len, "new": new, "hd": hd,
            "kv_heads": heads, "page": page, "width": width,
            "prefix": 0 if what == "branch" else rng.randint(max(1, max_len // 2), max_len), "window": 0, "sinks": 0}


def _uneven(n, longest, least=1):
    """n lengths up to `longest`, the last the longest."""
    if n == 1:
        return [max(least, longest)]
    frac = [((i * 0.6180339887498949) % 1.0) for i in range(n - 1)] + [1.0]
    return [max(least, int(round(longest * f))) for f in frac]


def _lengths(case):
    """New tokens and keys (new ones included) of each sequence of a qkv or attend case; from the case alone."""
    n, new, longest = case["n_seq"], case["new"], case["max_len"]
    if case["op"] == "qkv" and new > 16 and n > 1:
        q = [max(1, int(round(new * (0.02 + 0.98 * f * f)))) for f in [((i * 0.6180339887498949) % 1.0) for i in range(n - 1)] + [1.0]]
    else:
        q = [new] * n
    return q, [max(a, k) for a, k in zip(q, _uneven(n, longest))]


def _slots(case):
    """A pages case: keys of every slot before the pass, and of a branch case the parents, the children and their new tokens."""
    kv = _uneven(case["n_seq"], case["max_len"], case["prefix"] or 1)
    if case["what"] != "branch":
        return kv, [], [], []
    parents = [p for p in range(case["n_seq"]) for _ in range(case["width"])]
    children = [case["n_seq"] + i for i in range(len(parents))]
    new = [case["new"]] * len(parents) if case["new"] <= 64 else _uneven(len(parents), case["new"])
    return kv + [0] * len(parents), parents, children, new


def _need(case):
    """Pages that a pages case's pool needs in all: the sequences' own, those of the children, and a few more."""
    kv, parents, _, new = _slots(case)
    ps = case["page"]
    own_pages = sum(-(-n // ps) for n in kv)
    return own_pages + sum(-(-(n + ps - 1) // ps) + 1 for n in new) + (case["n_seq"] if case["what"] == "stream" else 0) + 3


def _is_gone(case):
    """The sequences of a compact case that have ended."""
    return [i % 3 == 1 for i in range(case["n_seq"])]


def work(case):
    elem = 2 if case["kv"] == "f16" else 1
    H, hd, ps = case["kv_heads"], case["hd"], case["page"]
    e4 = case["kv"] == "e4m3"
    if case["op"] == "qkv":
        q, kv = _lengths(case)
        n, G = sum(q), case["group"]
        rows = 4 if case["rows"] == "f32" else 2
        touched = sum(-(-k // ps) - (k - a) // ps for a, k in zip(q, kv))
        small = 4 * touched + 8 * len(q) + 4 * n + (16 * touched * H if e4 else 0) + (8 * hd if case["norm"] else 0)
        return {"bytes": n * H * hd * ((G + 2) * rows + 2 * G + 2 * elem) + small,
                "flops": float(n * H * hd * ((G + 1) * (4 + (4 if case["norm"] else 0))))}
    if case["op"] == "attend":
        q, kv = _lengths(case)
        W, S, G = case["window"], case["sinks"], case["group"]
        keys = scored = 0
        for a, k in zip(q, kv):
            keys += k - max(0, k - a - W + 1) + min(S, max(0, k - a - W + 1))
            lows = [max(0, k - a + i + 1 - W) for i in range(a)]
            scored += sum(k - a + i + 1 - lo + min(S, lo) for i, lo in enumerate(lows))
        pages = sum(-(-k // ps) for k in kv) if W + S >= max(kv) else len(kv) * (-(-(W + q[0]) // ps) + -(-S // ps))
        return {"bytes": 2 * keys * H * hd * elem + sum(q) * H * G * hd * 6 + 4 * pages + 8 * len(q) +
                (8 * H * pages if e4 else 0), "flops": 4.0 * scored * G * H * hd}
    kv, parents, children, new = _slots(case)
    row = 2 * H * hd * elem                                                # K and V of a token
    if case["what"] == "branch":
        length = [case["prefix"] or kv[p] for p in parents]
        shared = sum(-(-n // ps) for n in length)
        fresh = sum(-(-(n + a) // ps) - -(-n // ps) for n, a in zip(length, new))
        copied = sum(n % ps for n in length)
        copies = sum(1 for n in length if n % ps)
        # a table entry read and written and a count raised for each shared page, both undone by the free; copied rows twice
        return {"bytes": shared * (8 + 8 + 8 + 8) + 20 * (fresh + copies) + 2 * copied * row + (16 * H * copies if e4 else 0) +
                4 * _need(case), "flops": float(shared)}
    if case["what"] == "stream":
        return {"bytes": sum(4 * (-(-n // ps)) for n in kv) + 4 * _need(case) + 20 * len(kv), "flops": float(len(kv))}
    live = sum(-(-n // ps) for n, g in zip(kv, _is_gone(case)) if not g)
    gone = sum(-(-n // ps) for n, g in zip(kv, _is_gone(case)) if g)
    moved = live * (gone + 3) / (live + gone + 3)                        # pages are in no order
    return {"bytes": int(2 * moved * (ps * row + (8 * H if e4 else 0))) + 8 * live + 4 * _need(case), "flops": float(moved)}


# ---- inputs -----------------------------------------------------------------

def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s; at least 2^-100."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1)
    k = torch.where(m <= 0.875, e - 9, e - 8)      # 448 = 0.875 * 2^9
    k = torch.where(amax > 0, k, torch.full_like(k, -100)).clamp(min=-100)
    return torch.exp2(k.double()).float()


def _to_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn)


def _pool(st, case, n_pages, g):
    """Random pages: K with a few hot channels, as trained models have them."""
    dev, H, ps, hd = g.device, case["kv_heads"], case["page"], case["hd"]
    for name in ("k", "v"):
        x = torch.randn((n_pages, H, ps, hd), generator=g, device=dev)
        if name == "k":
            x *= 1.0 + 3.0 * (torch.rand((1, H, 1, hd), generator=g, device=dev) < 0.03)
        if case["kv"] == "f16":
            st[name], st[name + "_scale"] = x.half(), None
        else:
            x *= torch.exp2(torch.randn((n_pages, H, 1, 1), generator=g, device=dev))
            s = _pow2_scale(x.abs().amax(dim=(2, 3)))
            st[name], st[name + "_scale"] = _to_e4m3(x / s[:, :, None, None]), s


def _tables(need, max_pages, n_pages, g):
    """Page tables of pages in no order; entries behind a sequence's pages are -1."""
    order = torch.randperm(n_pages, generator=g, device=g.device).to(torch.int32)
    n = torch.tensor(need, device=g.device)
    j = torch.arange(max_pages, device=g.device)
    at = (torch.cumsum(n, 0) - n)[:, None] + j
    return torch.where(j < n[:, None], order[at.clamp(max=n_pages - 1)], torch.full_like(order[:1], -1))


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": dict(case)}
    if case["op"] == "pages":
        _prepare_pages(st, case, g)
    else:
        _prepare_rows(st, case, g)
    if own:
        import gqa_kv_head_gb300 as fr
        st["cache"] = fr.PagedKV(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if case["op"] == "pages":
            st["pool"] = fr.PagePool(st["refs"], st["kv_len"], st["table"], case["page"])
        else:
            st["batch"] = fr.PagedBatch(st["tok_start"], st["kv_len"], st["table"])
        if case["op"] == "qkv":
            st["rope_params"] = fr.rope_params(**st["rope"])
        if case["op"] == "attend":
            st["workspace"] = fr.make_paged_workspace(case["kv_heads"] * case["group"], case["kv_heads"], case["hd"])
    return st


def _prepare_rows(st, case, g):
    dev = g.device
    q, kv = _lengths(case)
    H, G, hd, ps = case["kv_heads"], case["group"], case["hd"], case["page"]
    n_tok, need = sum(q), [-(-k // ps) for k in kv]
    n_pages = sum(need) + 3                        # a few pages belong to nobody
    st["table"] = _tables(need, max(need), n_pages, g)
    st["tok_start"] = _ints([sum(q[:i]) for i in range(len(q) + 1)])
    st["kv_len"] = _ints(kv)
    _pool(st, case, n_pages, g)
    if case["op"] == "attend":
        st["q16"] = (torch.randn((n_tok, H * G, hd), generator=g, device=dev) / math.sqrt(hd)).half()
        st["out"] = torch.empty((n_tok, H * G, hd), dtype=torch.float32, device=dev)
        return
    # the rows of one fused projection: queries, keys, values
    qkv = (torch.randn((n_tok, (G + 2) * H * hd), generator=g, device=dev) * 2.0).to(ROWS[case["rows"]])
    st["q"] = qkv[:, :G * H * hd].view(n_tok, G * H, hd)
    st["k_new"] = qkv[:, G * H * hd:(G + 1) * H * hd].view(n_tok, H, hd)
    st["v_new"] = qkv[:, (G + 1) * H * hd:].view(n_tok, H, hd)
    st["pos"] = torch.cat([torch.arange(k - a, k, dtype=torch.int32) for a, k in zip(q, kv)]).to(dev)
    st["rope"] = {"n_dims": case["n_dims"], "freq_base": 10000.0}
    if case["yarn"]:
        st["rope"].update(freq_scale=0.25, ext_factor=1.0, n_ctx_orig=4096)
    st["q_norm"] = st["k_norm"] = None
    if case["norm"]:
        st["q_norm"] = 1.0 + 0.2 * torch.randn(hd, generator=g, device=dev)
        st["k_norm"] = 1.0 + 0.2 * torch.randn(hd, generator=g, device=dev)
    st["q16"] = torch.empty((n_tok * H * G, hd), dtype=torch.float16, device=dev)


def _prepare_pages(st, case, g):
    kv, parents, children, new = _slots(case)
    ps, n_pages = case["page"], _need(case)
    need = [-(-n // ps) for n in kv]
    length = [case["prefix"] or kv[p] for p in parents]
    max_pages = max(need + [-(-(n + a) // ps) for n, a in zip(length, new)])
    table = _tables(need, max_pages, n_pages, g)
    st["kv_len"] = _ints(kv)
    st["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=g.device)
    if case["what"] == "branch":
        st["parent"], st["child"] = _ints(parents), _ints(children)
        st["length"] = _ints(length) if case["prefix"] else None
        starts = [0] * (case["n_seq"] + 1) + [sum(new[:i + 1]) for i in range(len(new))]
        st["tok_start"], st["new"] = _ints(starts), _ints(new)
    elif case["what"] == "stream":
        # trimmed the last time at most 256 tokens ago; the step's new tokens are counted, and have no pages so far
        j = torch.arange(max_pages, device=g.device)
        n = st["kv_len"][:, None]
        start = (n - case["new"]).clamp(min=0)
        gone = (j * ps >= case["sinks"]) & ((j + 1) * ps <= n - n % 256 - 256 - case["window"] + 1)
        table = torch.where(gone | (j >= -(-start // ps)), torch.full_like(table, -1), table)
        st["tok_start"] = torch.cat([_ints([0]), torch.cumsum(n[:, 0] - start[:, 0], 0).to(torch.int32)])
    else:
        ended = torch.tensor(_is_gone(case), device=g.device)
        table = torch.where(ended[:, None], torch.full_like(table, -1), table)
        st["kv_len"] = torch.where(ended, torch.zeros_like(st["kv_len"]), st["kv_len"])
    st["table"] = table
    st["refs"][table[table >= 0].long()] = 1
    if case["what"] != "branch":                   # the pass starts from these again
        st["table_was"], st["refs_was"] = table.clone(), st["refs"].clone()
    _pool(st, case, n_pages, g)


# ---- one pass -----------------------------------------------------------------

def run(st):
    case = st["case"]
    if case["op"] == "attend":
        if own:
            import gqa_kv_head_gb300 as fr
            return fr.paged_attn(st["cache"], st["batch"], st["q16"], case["kv_heads"] * case["group"], window=case["window"],
                                 sinks=case["sinks"], out=st["out"], workspace=st["workspace"])
        return _attend_plain(st)
    if case["op"] == "qkv":
        if own:
            import gqa_kv_head_gb300 as fr
            q16 = fr.qkv_post_paged(st["cache"], st["batch"], st["q"], st["k_new"], st["v_new"], st["pos"],
                                    st["rope_params"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS,
                                    interleaved=case["interleaved"], q16_out=st["q16"])
        else:
            q16 = _qkv_plain(st)
        return {"q16": q16, **_pages_of(st)}
    if case["what"] != "branch":
        # (moved and dropped pages keep what they held: with the tables as they were, the pass finds the same work)
        st["table"].copy_(st["table_was"])
        st["refs"].copy_(st["refs_was"])
    if own:
        import gqa_kv_head_gb300 as fr
        pool = st["pool"]
        if case["what"] == "branch":
            fr.pages_free(pool, st["child"])
            fr.pages_fork(pool, st["parent"], st["child"], st["length"])
            st["kv_len"][case["n_seq"]:] += st["new"]
            fr.pages_reserve(pool, st["tok_start"])
        elif case["what"] == "stream":
            fr.pages_trim(pool, case["window"], case["sinks"], st["tok_start"])
            fr.pages_reserve(pool, st["tok_start"])
        else:
            fr.pages_compact(pool)
        fr.pages_copy(st["cache"], pool)
    elif case["what"] == "branch":
        _free_plain(st, st["child"].long())
        _fork_plain(st)
        st["kv_len"][case["n_seq"]:] += st["new"]
        _copy_plain(st, *_reserve_plain(st, st["child"].long(), st["new"].long()))
    elif case["what"] == "stream":
        _trim_plain(st)
        new = (st["tok_start"][1:] - st["tok_start"][:-1]).long()
        _copy_plain(st, *_reserve_plain(st, torch.arange(case["n_seq"], device="cuda"), new))
    else:
        _compact_plain(st)
    return {"table": st["table"], "refs": st["refs"], "kv_len": st["kv_len"], **_pages_of(st)}


def _pages_of(st):
    names = ("k", "v") if st["k_scale"] is None else ("k", "v", "k_scale", "v_scale")
    return {n: st[n] for n in names}


def _angles(st):
    """Angle of every pair at every token, and the factor of the magnitude; in 64 bits."""
    r, n = st["rope"], st["rope"]["n_dims"]
    i = torch.arange(n // 2, device="cuda", dtype=torch.float64)
    w = r["freq_base"] ** (-2.0 * i / n)
    if "ext_factor" not in r:
        return st["pos"].double()[:, None] * w, 1.0
    # YaRN: pairs that turn often in the original context stay, those that turn seldom are interpolated
    low, high = [n * math.log(r["n_ctx_orig"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(r["freq_base"])) for turns in (32.0, 1.0)]
    low, high = max(0.0, math.floor(low)), min(n - 1.0, math.ceil(high))
    mix = r["ext_factor"] * (1.0 - ((i - low) / max(0.001, high - low)).clamp(0.0, 1.0))
    return st["pos"].double()[:, None] * (w * (r["freq_scale"] * (1.0 - mix) + mix)), 1.0 + 0.1 * math.log(1.0 / r["freq_scale"])


def _norm_rotate(st, x, weight):
    case, n = st["case"], st["case"]["n_dims"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS) * weight.to(x.dtype)
    a, size = _angles(st)
    c, s = (torch.cos(a) * size).to(x.dtype)[:, None, :], (torch.sin(a) * size).to(x.dtype)[:, None, :]
    if case["interleaved"]:
        lo, hi = x[..., 0:n:2], x[..., 1:n:2]
        y = torch.stack([lo * c - hi * s, lo * s + hi * c], dim=3).flatten(2)
    else:
        lo, hi = x[..., :n // 2], x[..., n // 2:n]
        y = torch.cat([lo * c - hi * s, lo * s + hi * c], dim=2)
    return torch.cat([y, x[..., n:]], dim=2)


def _qkv_plain(st):
    case = st["case"]
    q = _norm_rotate(st, st["q"].float(), st["q_norm"]) * (1.0 / math.sqrt(case["hd"]))
    tok_start, kv_len, ps = st["tok_start"].long(), st["kv_len"].long(), case["page"]
    t = torch.arange(st["pos"].shape[0], device="cuda")
    b = torch.searchsorted(tok_start[1:].contiguous(), t, right=True)
    slot = kv_len[b] - tok_start[b + 1] + t
    page, row = st["table"].long()[b, slot // ps], slot % ps
    # (a page's scale hangs on its largest value, which may lie next to a border)
    wide = torch.float32 if st["k_scale"] is None else torch.float64
    _put_plain(st, "k", _norm_rotate(st, st["k_new"].to(wide), st["k_norm"]), page, row)
    _put_plain(st, "v", st["v_new"].to(wide), page, row)
    return q.half().flatten(0, 1)


def _put_plain(st, name, rows, page, row):
    cache, scale = st[name], st[name + "_scale"]
    n_pages, H, ps, hd = cache.shape
    if scale is None:
        cache[page, :, row] = rows.half()
        return
    first = torch.full((n_pages,), ps, device=cache.device).scatter_reduce(0, page, row, "amin")
    amax = torch.zeros((n_pages, H), dtype=rows.dtype, device=cache.device).scatter_reduce(
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
    H, hd, ps, G, n = case["kv_heads"], case["hd"], case["page"], case["group"], case["new"]
    W, S, n_seq = case["window"], case["sinks"], case["n_seq"]
    kv_len, dev = st["kv_len"].long(), st["kv_len"].device
    # the keys that some row sees: the first S, and those from the first row's window on
    begin = (kv_len - n + 1 - W).clamp(min=0)
    cols = min(W + n, case["max_len"])
    j = torch.cat([torch.arange(S, device=dev).expand(n_seq, S), begin[:, None] + torch.arange(cols, device=dev)], dim=1)
    there = torch.cat([j[:, :S] < begin[:, None], j[:, S:] < kv_len[:, None]], dim=1)        # each key once
    at = j.clamp(max=case["max_len"] - 1)
    page = st["table"].long().gather(1, at // ps).clamp(min=0)
    kf, vf = st["k"][page, :, at % ps].float(), st["v"][page, :, at % ps].float()              # [n_seq, columns, H, hd]
    if st["k_scale"] is not None:
        kf, vf = kf * st["k_scale"][page][..., None], vf * st["v_scale"][page][..., None]
    kf, vf = kf.transpose(1, 2), vf.transpose(1, 2)
    q = st["q16"].float().view(n_seq, n, H, G, hd).permute(0, 2, 1, 3, 4).reshape(n_seq, H, n * G, hd)
    here = kv_len[:, None, None] - n + torch.arange(n, device=dev)[None, :, None]
    seen = there[:, None, :] & (j[:, None, :] <= here) & ((j[:, None, :] > here - W) | (j[:, None, :] < S))
    seen = seen[:, None, :, None, :].expand(-1, 1, n, G, -1).reshape(n_seq, 1, n * G, -1)
    s = torch.matmul(q, kf.transpose(2, 3)).masked_fill(~seen, float("-inf"))
    m = s.amax(dim=3, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s - m)
    o = torch.matmul(p, vf) / p.sum(dim=3, keepdim=True)
    return o.view(n_seq, H, n, G, hd).permute(0, 2, 1, 3, 4).reshape(n_seq * n, H * G, hd)


def _count(refs, pages, live, by):
    refs.index_add_(0, pages.clamp(min=0).flatten().long(), (live & (pages >= 0)).flatten().to(torch.int32) * by)


def _drop(st, slots, drop):
    """The entries of the slots' table rows where drop is true are given back."""
    rows = st["table"][slots]
    _count(st["refs"], rows, drop, -1)
    st["table"][slots] = torch.where(drop, torch.full_like(rows, -1), rows)


def _free_plain(st, slots):
    ps, j = st["case"]["page"], torch.arange(st["table"].shape[1], device="cuda")
    _drop(st, slots, j * ps < st["kv_len"][slots][:, None])
    st["kv_len"][slots] = 0


def _trim_plain(st):
    case, ps = st["case"], st["case"]["page"]
    j = torch.arange(st["table"].shape[1], device="cuda")
    drop = (j * ps >= case["sinks"]) & ((j + 1) * ps <= st["kv_len"][:, None] - case["new"] - case["window"] + 1)
    _drop(st, torch.arange(case["n_seq"], device="cuda"), drop)


def _fork_plain(st):
    parent, child = st["parent"].long(), st["child"].long()
    n = st["kv_len"][parent] if st["length"] is None else st["length"]
    rows = st["table"][parent]
    live = torch.arange(rows.shape[1], device="cuda") * st["case"]["page"] < n[:, None]
    st["table"][child] = torch.where(live, rows, st["table"][child])
    _count(st["refs"], rows, live, 1)
    st["kv_len"][child] = n


def _reserve_plain(st, slots, new):
    """Pages for the last `new` tokens of the slots, the lowest free ones in order; (source, destination, rows) of every slot's copy."""
    refs, ps, dev = st["refs"], st["case"]["page"], st["refs"].device
    n_pages, n_kv = refs.shape[0], st["kv_len"][slots].long()
    first, i = n_kv - new, torch.arange(slots.shape[0], device=dev)
    i0, r0 = first // ps, first % ps
    rows = st["table"][slots].long()
    last_page = rows.gather(1, i0[:, None])[:, 0].clamp(min=0)
    part = (r0 > 0) & (new > 0)
    # of a shared page that all its holders go on in, the last of these keeps it
    writers = torch.zeros_like(refs).index_add_(0, last_page, part.to(torch.int32))
    latest = torch.full((n_pages,), -1, device=dev).scatter_reduce(0, last_page, torch.where(part, i, -1), "amax")
    keep = part & (refs[last_page] == writers[last_page]) & (latest[last_page] == i)
    copy = part & ~keep
    j = torch.arange(rows.shape[1], device=dev)
    want = (j >= (i0 + keep)[:, None]) & (j * ps < n_kv[:, None]) & (new > 0)[:, None]
    free = refs == 0
    place = torch.where(free, torch.cumsum(free, 0) - 1, n_pages)
    lowest = torch.full((n_pages + 1,), -1, device=dev).scatter(0, place, torch.where(free, torch.arange(n_pages, device=dev), -1))
    fresh = lowest[(torch.cumsum(want.flatten(), 0) - 1).clamp(0, n_pages)].view_as(want)
    rows = torch.where(want, fresh, rows)
    st["table"][slots] = rows.to(torch.int32)
    refs.index_add_(0, last_page, -copy.to(torch.int32))
    _count(refs, rows, want, 1)
    dst = rows.gather(1, i0[:, None])[:, 0]              # (a page of the slot's own, so that no two are alike)
    return torch.where(copy, last_page, dst), dst, torch.where(copy, r0, 0)


def _copy_plain(st, src, dst, n_rows):
    here = (torch.arange(st["case"]["page"], device="cuda") < n_rows[:, None])[:, None, :, None]
    for name, x in _pages_of(st).items():
        if name.endswith("scale"):
            x[dst] = torch.where(n_rows[:, None] > 0, x[src], x[dst])
        else:
            x = x if x.dtype == torch.float16 else x.view(torch.uint8)
            x[dst] = torch.where(here, x[src], x[dst])


def _compact_plain(st):
    refs, n_pages = st["refs"], st["refs"].shape[0]
    used, j = refs > 0, torch.arange(n_pages, device="cuda")
    inside = j < used.sum()
    src, dst = torch.nonzero(used & ~inside)[:, 0].flip(0), torch.nonzero(~used & inside)[:, 0]    # highest page to lowest hole
    to = j.clone()
    to[src] = dst
    st["table"].copy_(torch.where(st["table"] >= 0, to[st["table"].clamp(min=0).long()], -1))
    refs[dst] = refs[src]
    refs[src] = 0
    for name, x in _pages_of(st).items():
        x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        x[dst] = x[src]


# ---- 64 bits --------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pages":
        return _pages_exact(st, case)
    q, kv = _lengths(case)
    starts = [sum(q[:i]) for i in range(len(q))]
    return _qkv_exact(st, q, kv, starts) if case["op"] == "qkv" else _attend_exact(st, q, kv, starts)


def _turned(x, weight, turn, n, interleaved):
    """Rows [tokens, heads, hd] in 64 bits: normed, and their pairs turned as complex numbers."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=2, keepdim=True) ** 2 / x.shape[2] + EPS) * weight.double()
    a, b = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    z = torch.complex(x[..., a], x[..., b]) * turn[:, None, :]
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _qkv_exact(st, q, kv, starts):
    case, r = st["case"], st["rope"]
    n, ps = case["n_dims"], case["page"]
    speed, size = [], 1.0
    for i in range(n // 2):
        w = math.exp(-2.0 * i / n * math.log(r["freq_base"]))
        if case["yarn"]:
            c = [n * math.log(r["n_ctx_orig"] / (t * 2.0 * math.pi)) / (2.0 * math.log(r["freq_base"])) for t in (32.0, 1.0)]
            c = max(0.0, math.floor(c[0])), min(n - 1.0, math.ceil(c[1]))
            stay = 1.0 - min(1.0, max(0.0, (i - c[0]) / max(0.001, c[1] - c[0])))
            w = r["freq_scale"] * w * (1.0 - stay) + w * stay
            size = 1.0 - 0.1 * math.log(r["freq_scale"])
        speed.append(w)
    angle = st["pos"].double()[:, None] * torch.tensor(speed, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, size), angle)
    out = {"q16": (_turned(st["q"], st["q_norm"], turn, n, case["interleaved"]) / math.sqrt(case["hd"])).flatten(0, 1)}
    new = {"k": _turned(st["k_new"], st["k_norm"], turn, n, case["interleaved"]), "v": st["v_new"].double()}
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
        out[name] = pool
        if scale is not None:
            out[name + "_scale"] = scale
    return out


def _attend_exact(st, q, kv, starts):
    case = st["case"]
    H, G, hd, ps, W, S = (case[x] for x in ("kv_heads", "group", "hd", "page", "window", "sinks"))
    if sum(q) * H > 20000:
        return None
    out = torch.zeros((sum(q), H * G, hd), dtype=torch.float64, device="cuda")
    for b, (a, n_kv) in enumerate(zip(q, kv)):
        ids = st["table"][b, :-(-n_kv // ps)].long()
        k, v = st["k"][ids].double(), st["v"][ids].double()
        if st["k_scale"] is not None:
            k = k * st["k_scale"][ids].double()[:, :, None, None]
            v = v * st["v_scale"][ids].double()[:, :, None, None]
        k, v = k.transpose(0, 1).reshape(H, -1, hd), v.transpose(0, 1).reshape(H, -1, hd)
        for t in range(a):
            end = n_kv - a + t + 1
            low = max(0, end - W)
            see = list(range(min(S, low))) + list(range(low, end))
            see = slice(0, end) if len(see) == end else torch.tensor(see, device="cuda")
            x = st["q16"][starts[b] + t].double().view(H, G, hd)
            out[starts[b] + t] = (torch.softmax(x @ k[:, see].transpose(1, 2), dim=2) @ v[:, see]).view(H * G, hd)
    return out


def _pages_exact(st, case):
    """The definition, one sequence and one page after the other, on the host."""
    ps = case["page"]
    table, refs, n = st["table"].tolist(), st["refs"].tolist(), st["kv_len"].tolist()
    moves = []

    def reserve(b, new):
        if not new:
            return
        for p in range((n[b] - new) // ps, -(-n[b] // ps)):
            rows = (n[b] - new) % ps if p == (n[b] - new) // ps else 0
            old = table[b][p]
            if rows and refs[old] == 1:
                continue
            table[b][p] = free.pop(0) if free else -1
            if rows:
                refs[old] -= 1
                moves.append((old, table[b][p], rows))
            refs[table[b][p]] += 1

    if case["what"] == "branch":
        _, parents, children, new = _slots(case)
        for a, c in zip(parents, children):
            n[c] = case["prefix"] or n[a]
            for p in range(-(-n[c] // ps)):
                table[c][p] = table[a][p]
                refs[table[a][p]] += 1
        free = [p for p, r in enumerate(refs) if r == 0]
        for c, a in zip(children, new):
            n[c] += a
            reserve(c, a)
    elif case["what"] == "stream":
        for b, length in enumerate(n):
            for p, page in enumerate(table[b]):
                if page >= 0 and p * ps >= case["sinks"] and (p + 1) * ps <= length - case["new"] - case["window"] + 1:
                    table[b][p] = -1
                    refs[page] -= 1
        free = [p for p, r in enumerate(refs) if r == 0]
        starts = st["tok_start"].tolist()
        for b in range(case["n_seq"]):
            reserve(b, starts[b + 1] - starts[b])
    else:
        hole, top = 0, len(refs) - 1
        while hole < top:
            if refs[hole]:
                hole += 1
            elif not refs[top]:
                top -= 1
            else:
                refs[hole], refs[top] = refs[top], 0
                moves.append((top, hole, ps))
        to = {a: b for a, b, _ in moves}
        table = [[to.get(p, p) for p in row] for row in table]
    out = {"table": _ints(table), "refs": _ints(refs), "kv_len": _ints(n)}
    for name, x in _pages_of(st).items():
        y = x.double()
        for a, b, rows in moves:
            y[b] = torch.cat([y[a][:, :rows], y[b][:, rows:]], dim=1) if y.dim() == 4 else y[a]
        out[name] = y
    return out
