"""The plain 64-bit attention of paged_ref.py with tolerances that go by what
each row sees: the V scales of pages out of a row's view grant it nothing."""
import torch

import paged_ref as ref


def attention(q16, k, v, tok_start, kv_len, table, n_head, causal=True, window=0, kq_scale=1.0, v_scale=None):
    """(out, tol). out is paged_ref.attention's; tol has its terms (share and floor,
    derived there), with the largest V scale taken over the pages of the row's
    own keys. Pages that other rows see may raise the reference that the floor goes
    by 256 times above that (twice 16, at either end of the views), no further."""
    out, _ = ref.attention(q16, k, v, tok_start, kv_len, table, n_head, causal=causal, window=window, kq_scale=kq_scale,
                           v_scale=v_scale)
    tol = torch.zeros_like(out)
    hd, H, ps = q16.shape[2], k.shape[1], k.shape[2]
    G = n_head // H
    eps = 2.0 ** -23
    for b in range(len(kv_len)):
        n_q, n = tok_start[b + 1] - tok_start[b], kv_len[b]
        ids = table[b, :-(-n // ps)].long()
        for h in range(H):
            scale = torch.ones(len(ids), dtype=torch.float64) if v_scale is None else v_scale[ids, h].double().abs()
            scale = scale.repeat_interleave(ps)[:n]
            kh, vh = k[ids, h].reshape(-1, hd)[:n], v[ids, h].reshape(-1, hd)[:n].abs()
            code = torch.where(scale[:, None] > 0, vh / scale[:, None], 0.0)
            for i in range(n_q):
                p = n - n_q + i
                end = max(0, min(n, p + 1)) if causal else n
                begin = max(0, p + 1 - window) if window else 0
                if end <= begin:
                    continue
                t, rows = tok_start[b] + i, slice(h * G, (h + 1) * G)
                q, see = q16[t, rows].double(), slice(begin, end)
                w = torch.softmax(kq_scale * (q @ kh[see].T), dim=1)
                ds = (hd + 4) * eps * (abs(kq_scale) * (q.abs() @ kh[see].abs().T)).amax(dim=1)
                share = 2 * ds + 2 * 2.0 ** -21 + ((end - begin) / 16 + 400) * eps
                top = torch.minimum(256.0 * scale[see].max(), scale.max())
                floor = 2.0 ** -32 * w.amax(dim=1)[:, None] * (top * code[see].sum(dim=0))
                tol[t, rows] = (w @ vh[see]) * (2 * share)[:, None] + floor
    return out, tol
