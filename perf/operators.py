"""Scored attention and the bucketed relative position bias: the measured cases.

Scored attention is softmax attention over packed documents whose scores are changed before the
softmax and whose mask is more than causal.  For a document's query i and key j (local positions):

    s_ij = softmax_scale * q_i . k_j
    t_ij = softcap * tanh(s_ij / softcap)                     (softcap 0: t = s)
    u_ij = t_ij - slope[h] * |j - i| + table[bucket(j - i), h]
    seen = i - left <= j <= i + right  or  j < prefix_len     (-1: no limit; causal: right = 0)
    O_i  = sum_j exp(u_ij - LSE_i) v_j,   LSE_i = log sum_j exp(u_ij)

The backward pass takes the saved O (bf16) and LSE (fp32) and gives dq, dk, dv (bf16) and, with a
table, its gradient (fp32).  Rows after the last document: O and gradients 0, LSE +inf.

``own = False`` runs elementary torch operations in 32 bits; ``own = True`` calls the library.
"""
import math

import torch

own = False

LN_BORDER = 2.0 ** -30     # a distance on a bucket's border belongs to the upper bucket


# ------------------------------------------------------------------------------------ cases

def _packed(total, lo, hi, seed):
    """Document lengths in [lo, hi] that add up to total (a plain congruential sequence)."""
    out, left, x = [], total, seed
    while left > 0:
        x = (x * 1103515245 + 12345) % (1 << 31)
        n = min(left, lo + x % (hi - lo + 1))
        out.append(n)
        left -= n
    return out


def _case(name, op, lengths, hq, hkv, d, causal=True, left=-1, right=-1, cap=0.0, slopes=False, prefix="", buckets=0,
          max_distance=0, pad=0, q_gain=2.0):
    return {"name": name, "op": op, "lengths": ",".join(str(n) for n in lengths), "hq": hq, "hkv": hkv, "d": d,
            "causal": causal, "left": left, "right": right, "cap": cap, "slopes": slopes, "prefix": prefix,
            "buckets": buckets, "max_distance": max_distance, "pad": pad, "q_gain": q_gain}


_ODD = [4097, 1, 1283, 2999, 640, 77]
_ODD_PREFIX = "1500,1,0,2999,129,5"


def listed():
    packed = _packed(16384, 128, 4096, 1)
    return [
        # one short document, two heads: a call whose time is its latency (a small model's layer, a smoke run)
        _case("cap_fwd_1x256_h2_d64", "fwd", [256], 2, 2, 64, cap=50.0),
        # a packed microbatch of a capped-score model: the framework's headline layout of documents
        _case("cap_fwd_packed_16k_h16_d128", "fwd", packed, 16, 16, 128, cap=50.0, q_gain=4.0),
        # long documents, grouped heads, linear distance bias: the largest forward
        _case("slopes_fwd_4x8192_h32_kv8_d128", "fwd", [8192] * 4, 32, 8, 128, slopes=True),
        # ragged documents with bidirectional prefixes (prompt and answer) and rows of padding behind the last one
        _case("prefix_cap_fwd_odd_h8_kv2_d128", "fwd", _ODD, 8, 2, 128, cap=30.0, prefix=_ODD_PREFIX, pad=119, q_gain=3.0),
        # an encoder's packed batch with a bucketed relative bias, both directions
        _case("buckets_fwd_noncausal_2x8192_h16_d64", "fwd", [8192] * 2, 16, 16, 64, causal=False, buckets=32,
              max_distance=128),
        # a decoder's layer with a sliding window and a bucketed bias over one long document
        _case("buckets_fwd_window_16k_h8_d128", "fwd", [16384], 8, 8, 128, left=2047, buckets=32, max_distance=256),
        # the same uses, backward
        _case("cap_bwd_1x256_h2_d64", "bwd", [256], 2, 2, 64, cap=50.0),
        _case("cap_bwd_packed_16k_h16_d128", "bwd", packed, 16, 16, 128, cap=50.0, q_gain=4.0),
        _case("slopes_bwd_4x8192_h32_kv8_d128", "bwd", [8192] * 4, 32, 8, 128, slopes=True),
        _case("prefix_cap_bwd_odd_h8_kv2_d128", "bwd", _ODD, 8, 2, 128, cap=30.0, prefix=_ODD_PREFIX, pad=119, q_gain=3.0),
        _case("buckets_bwd_noncausal_2x8192_h16_d64", "bwd", [8192] * 2, 16, 16, 64, causal=False, buckets=32,
              max_distance=128),
        _case("buckets_bwd_packed_16k_h16_d128", "bwd", packed, 16, 16, 128, buckets=32, max_distance=128),
    ]


def draw(rng):
    most = 4 * 8192 * 8193 // 2 * 32 * 128
    while True:
        total = int(2 ** rng.uniform(6, 15))
        n = rng.randint(1, max(1, min(24, total // 8)))
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        hkv = rng.choice([1, 2, 4, 8, 16])
        hq = hkv * rng.choice([1, 1, 2, 4])
        d = rng.choice([64, 128])
        causal = rng.random() < 0.7
        kind = rng.choice(["cap", "slopes", "prefix", "buckets", "cap_slopes", "cap_buckets"])
        left, right = -1, -1
        if rng.random() < 0.35:
            left = rng.randint(0, 3000)
            right = -1 if causal else rng.randint(0, 3000)
        c = _case("", rng.choice(["fwd", "bwd"]), lengths, hq, hkv, d, causal=causal, left=left, right=right,
                  cap=rng.choice([20.0, 30.0, 50.0]) if "cap" in kind or kind == "prefix" else 0.0,
                  slopes="slopes" in kind,
                  prefix=",".join(str(rng.randint(0, x)) for x in lengths) if kind == "prefix" else "",
                  buckets=rng.choice([16, 32, 64]) if "buckets" in kind else 0,
                  max_distance=rng.choice([96, 128, 200, 512]) if "buckets" in kind else 0,
                  pad=rng.choice([0, 0, rng.randint(1, 300)]), q_gain=rng.choice([1.0, 2.0, 4.0]))
        if _pairs(c) * hq * d <= most // 2 and total * hq * d <= 32768 * 32 * 128:
            del c["name"]
            return c


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def _prefix(case):
    return [int(x) for x in case["prefix"].split(",")] if case["prefix"] else [0] * len(_lengths(case))


def _window(case):
    return case["left"], 0 if case["causal"] else case["right"]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    left, right = _window(case)
    total = 0
    for n, pre in zip(_lengths(case), _prefix(case)):
        if n == 0:
            continue
        i = torch.arange(n, dtype=torch.int64)
        lo = (i - left).clamp(min=0) if left >= 0 else torch.zeros_like(i)
        hi = (i + right).clamp(max=n - 1) if right >= 0 else torch.full_like(i, n - 1)
        total += int((hi - lo + 1).sum() + torch.minimum(lo, torch.full_like(i, pre)).sum()
                     + (pre - 1 - torch.maximum(hi, lo - 1)).clamp(min=0).sum())
    return total


def work(case):
    T, hq, hkv, d = sum(_lengths(case)), case["hq"], case["hkv"], case["d"]
    q, kv, lse = T * hq * d * 2, T * hkv * d * 2, T * hq * 4
    pairs = _pairs(case) * hq
    if case["op"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * pairs}
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * d * pairs}


# ------------------------------------------------------------------------------------ inputs

def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lengths = _lengths(case)
    T = sum(lengths) + case["pad"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rnd = lambda h, gain=1.0: (torch.randn(T, h, d, generator=g, device=dev) * gain).to(torch.bfloat16)
    st = {"case": case, "lengths": lengths, "T": T, "scale": 1.0 / math.sqrt(d), "q": rnd(hq, case["q_gain"]), "k": rnd(hkv),
          "v": rnd(hkv), "table": None, "slopes": None, "prefix": None}
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["prefix"]:
        st["prefix"] = torch.tensor(_prefix(case), dtype=torch.int32, device=dev)
    if case["slopes"]:
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=dev)
    if case["buckets"]:
        st["table"] = torch.randn(case["buckets"], hq, generator=g, device=dev)
    if case["op"] == "bwd":
        st["do"] = rnd(hq)
        out, lse = _plain_fwd(st)
        st["out"], st["lse"] = out, lse
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import microscaled_precision_causal_gb300 as F
        st["att"] = F.FlamiaScoredAttention(
            st["T"], len(st["lengths"]), case["hq"], case["hkv"], case["d"], causal=case["causal"],
            window=(case["left"], case["right"]), softcap=case["cap"],
            buckets=(case["buckets"], case["max_distance"], not case["causal"]) if case["buckets"] else None)
        st["att"].plan_build(st["cu"])
    return st


def run(state):
    if own:
        att, st = state["att"], state
        extra = {"slopes": st["slopes"], "prefix_lens": st["prefix"], "table": st["table"]}
        if state["case"]["op"] == "fwd":
            out, lse = att.forward(st["q"], st["k"], st["v"], st["cu"], **extra)
            return {"out": out, "lse": lse}
        got = att.backward(st["q"], st["k"], st["v"], st["out"], st["lse"], st["do"], st["cu"], **extra)
        return dict(zip(("dq", "dk", "dv", "dtable"), got))
    if state["case"]["op"] == "fwd":
        out, lse = _plain_fwd(state)
        return {"out": out, "lse": lse}
    return _plain_bwd(state)


# ------------------------------------------------------------------------------------ plain form

def _bucket(rel, buckets, max_distance, both):
    """Bucket of key position minus query position: half the buckets for distances up to a border, the
    rest spread over the distance's logarithm up to max_distance; both: later keys have buckets of their own."""
    base = torch.zeros_like(rel)
    if both:
        buckets //= 2
        base = (rel > 0).to(rel.dtype) * buckets
        dist = rel.abs()
    else:
        dist = (-rel).clamp(min=0)
    exact_to = buckets // 2
    far = torch.log(dist.clamp(min=1).double() / exact_to) / math.log(max_distance / exact_to) * (buckets - exact_to)
    far = (exact_to + torch.floor(far + LN_BORDER).to(rel.dtype)).clamp(max=buckets - 1)
    return base + torch.where(dist < exact_to, dist, far)


def _chunks(state):
    """(first token, rows, first row, keys) of pieces of the documents small enough to keep whole scores."""
    left, right = _window(state["case"])
    pre = _prefix(state["case"])
    base = 0
    for n, p in zip(state["lengths"], pre):
        r0 = 0
        while r0 < n:
            rows = max(64, min(n - r0, (1 << 28) // (state["case"]["hq"] * n)))
            rows = min(rows, n - r0)
            keys = n if right < 0 else min(n, max(r0 + rows + right, p))
            yield base, n, p, r0, rows, keys
            r0 += rows
        base += n


def _piece(state, base, n, p, r0, rows, keys):
    """Scores before the softmax [hq, rows, keys], tanh factor or None, the hidden pairs and the piece's q, k."""
    case = state["case"]
    group = case["hq"] // case["hkv"]
    left, right = _window(case)
    q = state["q"][base + r0:base + r0 + rows].float().transpose(0, 1)
    k = state["k"][base:base + keys].float().transpose(0, 1).repeat_interleave(group, 0)
    s = torch.matmul(q, k.transpose(1, 2)) * state["scale"]
    th = None
    if case["cap"]:
        th = torch.tanh(s / case["cap"])
        s = th * case["cap"]
    i = torch.arange(r0, r0 + rows, device=q.device)[:, None]
    j = torch.arange(keys, device=q.device)[None, :]
    if state["slopes"] is not None:
        s = s - state["slopes"][:, None, None] * (j - i).abs()
    if state["table"] is not None:
        rel = torch.arange(-(r0 + rows - 1), keys - r0, device=q.device)      # every distance of the piece
        bias = state["table"][_bucket(rel, case["buckets"], case["max_distance"], not case["causal"])].t()
        s = s + bias[:, (j - i) + (r0 + rows - 1)]
    seen = torch.ones(rows, keys, dtype=torch.bool, device=q.device)
    if left >= 0:
        seen &= j >= i - left
    if right >= 0:
        seen &= j <= i + right
    seen |= j < p
    return s, th, ~seen, q, k


def _plain_fwd(state):
    case, T, hq, d = state["case"], state["T"], state["case"]["hq"], state["case"]["d"]
    group = hq // case["hkv"]
    out = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=state["q"].device)
    lse = torch.full((hq, T), math.inf, device=state["q"].device)
    for base, n, p, r0, rows, keys in _chunks(state):
        s, _, hidden, _, _ = _piece(state, base, n, p, r0, rows, keys)
        s = s.masked_fill(hidden, -math.inf)
        m = s.amax(2, keepdim=True)
        e = torch.exp(s - m)
        l = e.sum(2, keepdim=True)
        v = state["v"][base:base + keys].float().transpose(0, 1).repeat_interleave(group, 0)
        o = torch.matmul(e, v) / l
        out[base + r0:base + r0 + rows] = o.transpose(0, 1).to(torch.bfloat16)
        lse[:, base + r0:base + r0 + rows] = (m + torch.log(l))[:, :, 0]
    return out, lse


def _plain_bwd(state):
    case, T, hq, hkv, d = state["case"], state["T"], state["case"]["hq"], state["case"]["hkv"], state["case"]["d"]
    group = hq // hkv
    dev = state["q"].device
    dq = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=dev)
    dk = torch.zeros(hkv, T, d, device=dev)
    dv = torch.zeros(hkv, T, d, device=dev)
    dtable = torch.zeros_like(state["table"]) if state["table"] is not None else None
    for base, n, p, r0, rows, keys in _chunks(state):
        s, th, hidden, q, k = _piece(state, base, n, p, r0, rows, keys)
        at = slice(base + r0, base + r0 + rows)
        v = state["v"][base:base + keys].float().transpose(0, 1).repeat_interleave(group, 0)
        do = state["do"][at].float().transpose(0, 1)
        o = state["out"][at].float().transpose(0, 1)
        e = torch.exp(s - state["lse"][:, at, None]).masked_fill(hidden, 0.0)
        dv[:, base:base + keys] += torch.matmul(e.transpose(1, 2), do).view(hkv, group, keys, d).sum(1)
        du = e * (torch.matmul(do, v.transpose(1, 2)) - (do * o).sum(2, keepdim=True))
        if dtable is not None:
            # rows padded by their own count and read back one shorter: equal distances in one column
            w = torch.nn.functional.pad(du.flip(1), (0, rows)).view(hq, rows * (keys + rows))
            by_rel = w[:, :rows * (keys + rows - 1)].view(hq, rows, keys + rows - 1).sum(1)
            rel = torch.arange(-(r0 + rows - 1), keys - r0, device=dev)
            ids = _bucket(rel, case["buckets"], case["max_distance"], not case["causal"])
            one = (ids[None, :] == torch.arange(case["buckets"], device=dev)[:, None]).float()
            dtable += torch.matmul(one, by_rel.t())
        ds = du if th is None else du * (1.0 - th * th)
        ds = ds * state["scale"]
        dq[at] = torch.matmul(ds, k).transpose(0, 1).to(torch.bfloat16)
        dk[:, base:base + keys] += torch.matmul(ds.transpose(1, 2), q).view(hkv, group, keys, d).sum(1)
    got = {"dq": dq, "dk": dk.transpose(0, 1).to(torch.bfloat16).contiguous(),
           "dv": dv.transpose(0, 1).to(torch.bfloat16).contiguous()}
    if dtable is not None:
        got["dtable"] = dtable
    return got


# ------------------------------------------------------------------------------------ in 64 bits

def _first_distances(buckets, max_distance):
    """The first distance of each far bucket, by whole numbers: n with (n/e)^c >= (m/e)^b, e the border."""
    e = buckets // 2
    c = buckets - e
    out = []
    for b in range(1, c):
        n = e
        while n ** c * e ** b < max_distance ** b * e ** c:
            n += 1
        out.append(n)
    return e, out


def exact(case, seed):
    pairs = _pairs(case) * case["hq"] * case["d"]
    if pairs > 2.5e12:
        return None
    st = _inputs(case, seed)
    T, hq, hkv, d, dev = st["T"], case["hq"], case["hkv"], case["d"], st["q"].device
    left, right = _window(case)
    f64 = torch.float64
    bwd = case["op"] == "bwd"
    out = torch.zeros(T, hq, d, dtype=f64, device=dev)
    lse = torch.full((hq, T), math.inf, dtype=f64, device=dev)
    dk, dv = (torch.zeros(T, hkv, d, dtype=f64, device=dev) for _ in range(2))
    dtable = torch.zeros(case["buckets"], hq, dtype=f64, device=dev)
    if case["buckets"]:
        half = case["buckets"] // (1 if case["causal"] else 2)
        border, firsts = _first_distances(half, case["max_distance"])
        firsts = torch.tensor(firsts, dtype=torch.int64, device=dev)
        longest = max(st["lengths"])
        dist = torch.arange(longest, device=dev)
        by_dist = torch.where(dist < border, dist, border + torch.searchsorted(firsts, dist, right=True))
    for h in range(hq):
        hk = h * hkv // hq
        at0 = 0
        for n, pre in zip(st["lengths"], _prefix(case)):
            key = st["k"][at0:at0 + n, hk].to(f64)
            val = st["v"][at0:at0 + n, hk].to(f64)
            step = max(1, min(n, (1 << 26) // max(n, 1)))
            for a in range(0, n, step):
                b = min(n, a + step)
                last = n if right < 0 else min(n, max(b + right, pre))
                pos = torch.arange(a, b, device=dev).unsqueeze(1)
                gap = torch.arange(last, device=dev).unsqueeze(0) - pos           # j - i
                query = st["q"][at0 + a:at0 + b, h].to(f64)
                u = query @ key[:last].T / math.sqrt(d)
                slope = None
                if case["cap"]:
                    w = torch.tanh(u / case["cap"])
                    u, slope = case["cap"] * w, 1 - w ** 2
                if st["slopes"] is not None:
                    u = u - float(st["slopes"][h]) * gap.abs().to(f64)
                if case["buckets"]:
                    if case["causal"]:
                        ids = by_dist[(-gap).clamp(min=0)]
                    else:
                        ids = by_dist[gap.abs()] + half * (gap > 0)
                    u = u + st["table"][:, h].to(f64)[ids]
                no = torch.zeros_like(gap, dtype=torch.bool)
                if left >= 0:
                    no |= gap < -left
                if right >= 0:
                    no |= gap > right
                no &= gap + pos >= pre
                u = torch.where(no, -math.inf, u)
                rows = slice(at0 + a, at0 + b)
                if not bwd:
                    top = u.max(1).values
                    e = torch.exp(u - top[:, None])
                    total = e.sum(1)
                    out[rows, h] = (e @ val[:last]) / total[:, None]
                    lse[h, rows] = top + torch.log(total)
                    continue
                e = torch.exp(u - st["lse"][h, rows].to(f64)[:, None])
                grad = st["do"][rows, h].to(f64)
                mean = (grad * st["out"][rows, h].to(f64)).sum(1, keepdim=True)
                du = e * (grad @ val[:last].T - mean)
                dv[at0:at0 + last, hk] += e.T @ grad
                if case["buckets"]:
                    for x in range(case["buckets"]):
                        dtable[x, h] += torch.where(ids == x, du, 0.0).sum()
                if slope is not None:
                    du = du * slope
                out[rows, h] = du @ key[:last] / math.sqrt(d)
                dk[at0:at0 + last, hk] += du.T @ query / math.sqrt(d)
            at0 += n
    if not bwd:
        return {"out": out, "lse": lse}
    got = {"dq": out, "dk": dk, "dv": dv}
    if case["buckets"]:
        got["dtable"] = dtable
    return got
