"""Plain 64-bit form of a step's query and key rows: RMS norm of each head, rotation
of pairs of either layout, and a bound on what fp32 arithmetic may add."""
import math

import numpy as np
import torch


def angles(pos, rope):
    """float64 [n_tok, n_dims / 2] angles and the magnitude (YaRN as ggml's rope_ext defines it)."""
    n = rope["n_dims"]
    # (the parameters are f32 numbers in the interface)
    rope = {k: [float(np.float32(x)) for x in v] if k == "freq_factors" else float(np.float32(v)) for k, v in rope.items()}
    base, fs = rope.get("freq_base", 10000.0), rope.get("freq_scale", 1.0)
    ext = rope.get("ext_factor", 0.0)
    w, mag = [], rope.get("attn_factor", 1.0)
    for i in range(n // 2):
        theta = base ** (-2.0 * i / n) / (rope["freq_factors"][i] if rope.get("freq_factors") else 1.0)
        if ext:
            def dim(turns):
                return n * math.log(rope["n_ctx_orig"] / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(0.0, math.floor(dim(rope.get("beta_fast", 32.0)))), min(n - 1.0, math.ceil(dim(rope.get("beta_slow", 1.0))))
            ramp = 1.0 - min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
            theta = fs * theta * (1 - ramp * ext) + theta * ramp * ext
        else:
            theta = fs * theta
        w.append(theta)
    if ext:
        mag *= 1.0 + 0.1 * math.log(1.0 / fs)
    # (positions times frequencies modulo a turn in more than 64 bits, so that far positions are exact)
    turn = np.longdouble(2) * np.arctan2(np.longdouble(0), np.longdouble(-1))
    a = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(w, dtype=np.longdouble)
    return torch.from_numpy(np.remainder(a, turn).astype(np.float64)), mag


def rows(x, pos, rope, weight=None, eps=1e-6, interleaved=False, scale=1.0):
    """x: [n_tok, heads, hd] of any type. Returns (y, tol) in 64 bits: y = scale R(pos) n(x),
    and for each element what fp32 arithmetic (before the rounding to the output's type) may be off by:

      * the norm: hd squares and additions, each off by 2^-24 of the (positive) sum at most, so
        (hd + 1) 2^-24 of the mean, half of that in its root, and 4 roundings for the root, the
        weight and the two products: (hd / 2 + 5) 2^-24 of the element;
      * the rotation: cos and sin within 2^-21 (sincospi of an angle rounded to fp32: 2^-24 pi of
        a turn, and its own 2 units) times the pair's size, 4 roundings, 1 for the scale."""
    x = x.double()
    hd, n = x.shape[2], rope["n_dims"]
    share = 0.0
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + eps) * weight.double()
        share = (hd / 2 + 5) * 2.0 ** -24
    a, mag = angles(pos, rope)
    c, s = mag * torch.cos(a)[:, None, :], mag * torch.sin(a)[:, None, :]
    first, second = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    lo, hi = x[..., first], x[..., second]
    y, tol = x.clone(), x.abs() * (share + 2.0 ** -24)
    y[..., first], y[..., second] = lo * c - hi * s, lo * s + hi * c
    size = abs(mag) * (lo.abs() + hi.abs()) * (share + 2.0 ** -21 + 5 * 2.0 ** -24)
    tol[..., first], tol[..., second] = size, size
    return y * scale, tol * abs(scale)
