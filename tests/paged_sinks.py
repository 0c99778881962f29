"""Plain 64-bit attention with a sliding window and first tokens that stay visible,
row by row, with the tolerances of paged_ref.attention and paged_views.attention
(derived there) taken over the keys that each row sees."""
import torch


def seen_keys(p, n_kv, window, sinks):
    """Keys that the token at position p sees, in order."""
    low = max(0, p + 1 - window) if window else 0
    end = max(0, min(n_kv, p + 1))
    return list(range(min(sinks, low, end))) + list(range(low, end))


def attention(q16, k, v, tok_start, kv_len, table, n_head, window=0, sinks=0, kq_scale=1.0, v_scale=None):
    """(out, tol); k, v: float64 pages [n_pages, n_kv_head, page_size, hd]."""
    n_tok, hd = q16.shape[0], q16.shape[2]
    H, ps = k.shape[1], k.shape[2]
    G, eps = n_head // H, 2.0 ** -23
    out = torch.zeros((n_tok, n_head, hd), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(len(kv_len)):
        n_q, n = tok_start[b + 1] - tok_start[b], kv_len[b]
        for i in range(n_q):
            see = torch.tensor(seen_keys(n - n_q + i, n, window, sinks), dtype=torch.long)
            if not len(see):
                continue
            t, page, row = tok_start[b] + i, table[b, see // ps].long(), see % ps
            for h in range(H):
                rows = slice(h * G, (h + 1) * G)
                kk, vv, q = k[page, h, row], v[page, h, row], q16[t, rows].double()
                w = torch.softmax(kq_scale * (q @ kk.T), dim=1)
                out[t, rows] = w @ vv
                ds = (hd + 4) * eps * (abs(kq_scale) * (q.abs() @ kk.abs().T)).amax(dim=1)
                share = 2 * ds + 2 * 2.0 ** -21 + (len(see) / 16 + 400) * eps
                scale = torch.ones(len(see), dtype=torch.float64) if v_scale is None else v_scale[page, h].double().abs()
                every = torch.ones(1, dtype=torch.float64) if v_scale is None else v_scale[:, h].double().abs()
                code = torch.where(scale[:, None] > 0, vv.abs() / scale[:, None], 0.0)
                top = torch.minimum(256.0 * scale.max(), every.max())
                floor = 2.0 ** -32 * w.amax(dim=1)[:, None] * (top * code.sum(dim=0))
                tol[t, rows] = (w @ vv.abs()) * (2 * share)[:, None] + floor
    return out, tol
