"""The paged cache and its attention in 64 bits, from their definitions (tests only), with the bound
on what a kernel may differ by."""
import numpy as np

import oracle as O


def quantize(x):
    """[..., d] -> E4M3 codes and UE8M0 bytes [...]: a scale of its own for each row."""
    x = np.asarray(x, np.float64)
    nan = np.isnan(x).any(-1)
    y = np.where(nan[..., None], 0, x)
    top = np.where(np.isinf(y), 2.0 ** 128, np.abs(y)).max(-1)
    e = O.roundup_exponent(top)
    with np.errstate(over="ignore"):
        codes = O.e4m3_encode(y / np.exp2(e.astype(np.float64))[..., None])
    return codes, np.where(nan, 255, e + 127).astype(np.uint8)


def dequantize(codes, scales):
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return O.e4m3_decode(codes) * s[..., None]


def attend(q, keys, values, group, scale=None, left=-1, softcap=0.0):
    """One sequence: q [c, hq, d] at the last c of the positions of keys, values [L, hkv, d].  o, lse [hq, c] and
    tol_*, elementwise bounds on a kernel's difference."""
    c, hq, d = q.shape
    L = keys.shape[0]
    scale = 1 / np.sqrt(d) if scale is None else scale
    h16, u24 = 2.0 ** -8, 2.0 ** -24            # half a step of bf16, of fp32
    # relative bounds end where a format's do.  fp32 and bf16: values below 2^-126 may be flushed.  Products in
    # fp16 take a row of queries at 2^14 or more for its largest value and the largest weight times scale at
    # 2^13 or more: half a subnormal step, 2^-25, is 2^-39 and 2^-38 of those
    tiny = 2.0 ** -126
    r = {"o": np.zeros((c, hq, d)), "tol_o": np.zeros((c, hq, d)), "lse": np.zeros((hq, c)), "tol_lse": np.zeros((hq, c))}
    i, j = np.arange(L - c, L)[:, None], np.arange(L)[None, :]
    hide = (j > i) | ((j < i - left) if left >= 0 else False)
    for h in range(hq):
        Q, K, V = q[:, h], keys[:, h // group], values[:, h // group]
        u = scale * Q @ K.T
        # the product's d terms (queries flushed beside their row's largest), then cap, scaling and maximum
        eu = scale * (u24 * (d + 8) * (np.abs(Q) @ np.abs(K.T)) + 2.0 ** -39 * np.outer(np.abs(Q).max(1), np.abs(K).sum(1)))
        if softcap:
            u = softcap * np.tanh(u / softcap)
            eu = eu + 16 * u24 * softcap
        eu = np.where(hide, 0, eu + 8 * u24 * (1 + np.abs(u))).max(1)
        u = np.where(hide, -np.inf, u)
        m = u.max(1)
        e = np.exp(u - m[:, None])
        l = e.sum(1)
        P = e / l[:, None]
        A = P @ np.abs(V)
        # a code's row of values is at most 2 of its scale's 448: weight times scale in units of its values
        flushed = L * 2.0 ** -38 * (P * 2 * np.abs(V).max(1)).max(1)
        r["o"][:, h] = P @ V
        r["lse"][h] = m + np.log(l)
        r["tol_o"][:, h] = ((h16 + 2 * eu[:, None] + 2 * L * u24) * A + h16 * np.abs(P @ V) + flushed[:, None]
                            + tiny * (1 + np.abs(V).sum(0)))
        r["tol_lse"][h] = eu + (L + 8) * u24 * (1 + np.abs(r["lse"][h]))
    return r
