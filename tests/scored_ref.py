"""Scored attention in 64 bits, from its definition (tests only), with the bound on what a
kernel with bf16 products may differ by."""
import numpy as np

NEG = -2.0 ** 100


def bucket(r, num_buckets, max_distance, bidirectional):
    """Bucket of distance r = key - query, by whole numbers: far bucket x starts at the first n with
    (n / e)^c >= (max_distance / e)^x."""
    base, b = 0, num_buckets
    if bidirectional:
        b //= 2
        base, n = (b if r > 0 else 0), abs(r)
    else:
        n = max(-r, 0)
    e = b // 2
    if n < e:
        return base + n
    c = b - e
    x = 0
    while x + 1 < c and n ** c * e ** (x + 1) >= max_distance ** (x + 1) * e ** c:
        x += 1
    return base + e + x


def bucket_bias(table, max_distance, bidirectional, R):
    """[hq, 2R + 1] bias by clipped distance."""
    ids = [bucket(r, table.shape[0], max_distance, bidirectional) for r in range(-R, R + 1)]
    return np.ascontiguousarray(table[ids].T), np.array(ids)


def visible(n, window, pre):
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    see = np.ones((n, n), bool)
    if window[0] >= 0:
        see &= j >= i - window[0]
    if window[1] >= 0:
        see &= j <= i + window[1]
    return see | (j < pre)


def run(q, k, v, lengths, scale=None, window=(-1, 0), softcap=0.0, slopes=None, rel=None, prefix=None, dout=None,
        out=None, lse=None):
    """float64 arrays [T, H, d].  Forward, and with dout the gradients from the given out and lse
    (default: the forward's own).  tol_*: elementwise bounds on a kernel's difference."""
    T, hq, d = q.shape
    hkv = k.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    h16, u24 = 2.0 ** -8, 2.0 ** -24            # half a step of bf16, of fp32
    # relative bounds end at the smallest normal number: a value below 2^-126 may be flushed, so a
    # probability, a score gradient and an output are each off by up to 2^-126 beside them
    tiny = 2.0 ** -126
    R = (rel.shape[1] - 1) // 2 if rel is not None else 0
    res = {"o": np.zeros((T, hq, d)), "lse": np.full((hq, T), np.inf)}
    res["tol_o"], res["tol_lse"] = np.zeros((T, hq, d)), np.zeros((hq, T))
    if dout is not None:
        for n, h in (("dq", hq), ("dk", hkv), ("dv", hkv)):
            res[n], res["tol_" + n] = np.zeros((T, h, d)), np.zeros((T, h, d))
        res["drel"] = np.zeros((hq, 2 * R + 1))
        res["tol_drel"] = np.zeros((hq, 2 * R + 1))
    base = 0
    for doc, n in enumerate(lengths):
        rows = slice(base, base + n)
        base += n
        if n == 0:
            continue
        see = visible(n, window, min(max(prefix[doc], 0), n) if prefix is not None else 0)
        gap = np.arange(n)[None, :] - np.arange(n)[:, None]
        for h in range(hq):
            hk = h // (hq // hkv)
            Q, K, V = q[rows, h], k[rows, hk], v[rows, hk]
            u = scale * Q @ K.T
            # fp32: the product's d terms, then the cap (its 32-bit value), biases and base-2 scaling
            eu = u24 * (d + 8) * scale * (np.abs(Q) @ np.abs(K.T))
            g = np.ones_like(u)
            if softcap:
                th = np.tanh(u / softcap)
                u, g = softcap * th, 1 - th ** 2
                eu = eu + 16 * u24 * softcap
            if slopes is not None:
                u = u - slopes[h] * np.abs(gap)
                eu = eu + 4 * u24 * slopes[h] * np.abs(gap)
            hide = ~see
            if rel is not None:
                b = rel[h][np.clip(gap, -R, R) + R]
                hide = hide | (b < NEG)
                u = u + np.where(b < NEG, 0, b)
                eu = eu + 4 * u24 * np.abs(np.where(b < NEG, 0, b))
            eu = eu + 8 * u24 * (1 + np.abs(u))
            u = np.where(hide, -np.inf, u)
            some = ~hide.all(1)
            m = np.where(some, u.max(1), 0)
            e = np.where(hide, 0, np.exp(u - m[:, None]))
            l = np.where(some, e.sum(1), 1)
            P = e / l[:, None]
            res["o"][rows, h] = P @ V
            res["lse"][h, rows] = np.where(some, m + np.log(l), np.inf)
            eus = np.where(hide, 0, eu).max(1)
            A = P @ np.abs(V)
            res["tol_o"][rows, h] = (h16 + 2 * eus[:, None] + 2 * n * u24) * A + h16 * np.abs(P @ V) + tiny * (1 + np.abs(V).sum(0))
            res["tol_lse"][h, rows] = np.where(some, eus + (n + 8) * u24 * (1 + np.abs(m + np.log(l))), 0)
            if dout is None:
                continue
            dO = dout[rows, h]
            L = res["lse"][h, rows] if lse is None else lse[h, rows]
            O = res["o"][rows, h] if out is None else out[rows, h]
            P = np.where(hide | ~some[:, None], 0, np.exp(np.where(hide, 0, u) - np.where(some, L, 0)[:, None]))
            D = (dO * O).sum(1)
            dP = dO @ V.T
            dU = P * (dP - D[:, None])
            dS = dU * g
            ep = eu + 8 * u24 * (1 + np.abs(np.where(some, L, 0)))[:, None]
            ed = u24 * (d + 8) * (np.abs(dO) @ np.abs(V.T) + (np.abs(dO) * np.abs(O)).sum(1)[:, None])
            eU = np.where(hide, 0, np.abs(dU) * 2 * ep + P * ed + tiny * (np.abs(dP) + np.abs(D[:, None])))
            eS = eU + np.abs(dS) * (h16 + 16 * u24) + np.abs(dU) * 32 * u24 + np.where(hide, 0, tiny)
            sum32 = 2 * n * u24
            res["dq"][rows, h] = scale * dS @ K
            res["tol_dq"][rows, h] = scale * ((eS + sum32 * np.abs(dS)) @ np.abs(K)) + h16 * np.abs(scale * dS @ K)
            res["dk"][rows, hk] += scale * dS.T @ Q
            res["tol_dk"][rows, hk] += scale * ((eS + sum32 * np.abs(dS)).T @ np.abs(Q))
            res["dv"][rows, hk] += P.T @ dO
            res["tol_dv"][rows, hk] += (P * (h16 + 2 * ep + sum32) + 2 * tiny).T @ np.abs(dO)
            if rel is not None:
                ids = np.clip(gap, -R, R) + R
                np.add.at(res["drel"][h], ids, dU)
                np.add.at(res["tol_drel"][h], ids, eU + np.abs(dU) * u24 * 4 * (n + 64))
    if dout is not None:
        for n in ("dq", "dk", "dv"):
            res["tol_" + n] += tiny
        res["tol_dk"] += h16 * np.abs(res["dk"])
        res["tol_dv"] += h16 * np.abs(res["dv"])
    return res
