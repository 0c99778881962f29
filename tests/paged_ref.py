"""Plain 64-bit forms of the paged-cache operators on the CPU, for the tests:
written from the definitions, sequence by sequence, sharing no code with the
library. Tensors are torch CPU tensors."""
import torch

E4M3_MAX = 448.0


def pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s, not below 2^-100 (exact, by comparison)."""
    s = 2.0 ** -100
    while s * E4M3_MAX < amax:
        s *= 2.0
    return s


def attention(q16, k, v, tok_start, kv_len, table, n_head, causal=True, window=0, kq_scale=1.0, out=None,
              v_scale=None):
    """k, v: float64 [n_pages, n_kv_head, page_size, hd]. Returns (out, tol): the
    rows in 64 bits, and for each element the error a kernel may have that

      * accumulates each score's hd products in fp32, one rounding (2^-23, as an
        accumulator that truncates makes) for each addition and two for the scale
        and the exponent's argument: |ds| <= (hd + 4) 2^-23 sum_i |q_i k_i|,
        doubled because the reference maximum carries the same error;
      * takes 2^x within 2^-21 and holds a weight within 2^-21;
      * sums weights and weighted values in fp32, a rounding of 2^-23 for each
        16-key step and for each of at most 400 joins of states.

    Both the numerator and the denominator err by that share.

    A weight times its V scale (over the largest V scale in view) is held as two
    f16 terms, with the row's largest weight at 2^7 or more. The second term is
    rounded to f16's grid, which below 2^-14 has the fixed step 2^-24: it is off by
    2^-25 at most there, 2^-25 / 2^7 = 2^-32 of the largest weight, and a share of
    the weight (counted above) elsewhere. With codes c_j = v_j / v_scale_j the
    numerator errs by another 2^-32 max_j w_j max v_scale sum_j |c_j| (for f16
    pages the scales are 1). It matters where the keys that carry the weight have
    zeros in a dim. v_scale: [n_pages, n_kv_head], or None."""
    n_tok, hd = q16.shape[0], q16.shape[2]
    H, ps = k.shape[1], k.shape[2]
    G = n_head // H
    out = torch.zeros((n_tok, n_head, hd), dtype=torch.float64) if out is None else out.double().clone()
    tol = torch.zeros_like(out)
    eps = 2.0 ** -23
    for b in range(len(kv_len)):
        t0, t1, n = tok_start[b], tok_start[b + 1], kv_len[b]
        if t1 <= t0:
            continue
        ids = table[b, :-(-n // ps)].long()
        for h in range(H):
            vs = torch.ones(len(ids), dtype=torch.float64) if v_scale is None else v_scale[ids, h].double().abs()
            per_key = vs.repeat_interleave(ps)[:n, None]
            kh, vh = k[ids, h].reshape(-1, hd)[:n], v[ids, h].reshape(-1, hd)[:n]
            for t in range(t0, t1):
                p = n - (t1 - t0) + (t - t0)
                end = max(0, min(n, p + 1)) if causal else n
                begin = max(0, p + 1 - window) if causal and window else 0
                if end <= begin:
                    out[t, h * G:(h + 1) * G] = 0.0
                    continue
                q = q16[t, h * G:(h + 1) * G].double()
                kk, vv = kh[begin:end], vh[begin:end]
                s = kq_scale * (q @ kk.T)
                w = torch.softmax(s, dim=1)
                out[t, h * G:(h + 1) * G] = w @ vv
                ds = (hd + 4) * eps * (abs(kq_scale) * (q.abs() @ kk.abs().T)).amax(dim=1)
                share = 2 * ds + 2 * 2.0 ** -21 + ((end - begin) / 16 + 400) * eps
                code = torch.where(per_key[begin:end] > 0, vv.abs() / per_key[begin:end], 0.0).sum(dim=0)
                floor = 2.0 ** -32 * w.amax(dim=1)[:, None] * (vs.max() * code)
                tol[t, h * G:(h + 1) * G] = (w @ vv.abs()) * (2 * share)[:, None] + floor
    return out, tol


def append(k_new, v_new, tok_start, kv_len, table, k, v, k_scale=None, v_scale=None):
    """New rows (k_new already rotated; float32 values) into copies of the pages.
    f16 pages: k, v float16. e4m3: k, v float8_e4m3fn with scales."""
    res = []
    ps = k.shape[2]
    for new, pages, scale in ((k_new, k, k_scale), (v_new, v, v_scale)):
        pages = pages.clone()
        scale = None if scale is None else scale.clone()
        for b in range(len(kv_len)):
            n_q = tok_start[b + 1] - tok_start[b]
            first = kv_len[b] - n_q
            if n_q <= 0 or first < 0:
                continue
            for pi in range(first // ps, (kv_len[b] - 1) // ps + 1):
                page = int(table[b, pi])
                r0, r1 = max(first - pi * ps, 0), min(kv_len[b] - pi * ps, ps)
                t = tok_start[b] + pi * ps + r0 - first
                rows = new[t:t + r1 - r0]
                for h in range(pages.shape[1]):
                    x = rows[:, h]
                    if scale is None:
                        pages[page, h, r0:r1] = x.half()
                        continue
                    fin = x[torch.isfinite(x)].abs()
                    s = pow2_scale(float(fin.max()) if fin.numel() else 0.0)
                    old = float(scale[page, h]) if r0 else 0.0
                    s = max(s, old)
                    if r0 and s > old:
                        # exact products, one rounding
                        was = pages[page, h, :r0].double() * (old / s)
                        pages[page, h, :r0] = was.float().to(torch.float8_e4m3fn)
                    y = (x.double() / s).clamp(-E4M3_MAX, E4M3_MAX).float()      # NaN stays NaN
                    pages[page, h, r0:r1] = y.to(torch.float8_e4m3fn)
                    scale[page, h] = s
        res.append((pages, scale))
    return res[0][0], res[1][0], res[0][1], res[1][1]


def values(pages, scale=None):
    """The numbers that pages stand for, in 64 bits."""
    x = pages.double()
    return x if scale is None else x * scale.double()[:, :, None, None]


def same_bits(a, b):
    """Bitwise equality, any NaN code equal to any other."""
    a, b = a.contiguous(), b.contiguous()
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    eq = (a.view(kind) == b.view(kind)) | (torch.isnan(a.float()) & torch.isnan(b.float()))
    return bool(eq.all())

