"""A paged cache of keys and values: writing it, reading it back, attention over it: the measured cases.

Sequence n of a call brings c_n = cu[n + 1] - cu[n] new tokens, packed as the framework packs documents, and
has L_n = kv_lens[n] keys with them: its new token t stands at position L_n - c_n + t.  Position j of a sequence
lives in page table[n][j / P], slot j % P, of pools [pages, hkv, P, d].

    write   e4m3: per token and head e = least integer with max |x| <= 448 2^e (0 for a row of zeros),
                  codes E4M3(x 2^-e) and scale byte e + 127; bf16: the values
    read    the new tokens' rows back from the cache, packed: bf16(code 2^e); rows behind the last sequence 0
    attend  s = softmax_scale q.k, t = softcap tanh(s / softcap) (softcap 0: t = s), key j seen by position i iff
            i - left <= j <= i (left -1: no limit), O = sum_j exp(t - LSE) v_j, LSE = log sum_j exp(t);
            rows behind the last sequence: O 0, LSE +inf

``own = False`` runs elementary torch operations in 32 bits; ``own = True`` calls the library.
"""
import math

import torch

own = False


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


def _case(name, op, chunks, before, hq, hkv, d, fmt, page, left=-1, cap=0.0, pad=0):
    """chunks: new tokens of each sequence; before: its tokens in the cache already."""
    return {"name": name, "op": op, "chunks": ",".join(map(str, chunks)), "before": ",".join(map(str, before)), "hq": hq,
            "hkv": hkv, "d": d, "fmt": fmt, "page": page, "left": left, "cap": cap, "pad": pad}


_ODD = [4097, 1, 1283, 2999, 640, 77]


def listed():
    packed = _packed(16384, 128, 4096, 1)
    served = _packed(1 << 18, 1, 8191, 7)[:64]        # context lengths of a batch that is being served
    return [
        # one generation step of a batch: each sequence's new token goes into its page
        _case("write_step_64_hkv8_d128_e4m3", "write", [1] * 64, [n % 1000 for n in served], 8, 8, 128, "e4m3", 16),
        # the framework's headline layout of documents as prompts
        _case("write_prompts_16k_hkv16_d128_e4m3", "write", packed, [0] * len(packed), 16, 16, 128, "e4m3", 64),
        # ragged sequences read back for a training call, rows of padding behind the last one
        _case("read_odd_hkv2_d64_e4m3", "read", _ODD, [0] * len(_ODD), 2, 2, 64, "e4m3", 32, pad=119),
        # long sequences read back whole
        _case("read_4x8192_hkv8_d128_e4m3", "read", [8192] * 4, [0] * 4, 8, 8, 128, "e4m3", 128),
        # a step of one short sequence: a call whose time is its latency
        _case("step_1x256_h2_d64_e4m3", "attend", [1], [255], 2, 2, 64, "e4m3", 16),
        # a step of a served batch, ragged contexts, grouped heads
        _case("step_64_ragged_h32_kv8_d128_e4m3", "attend", [1] * 64, served, 32, 8, 128, "e4m3", 16),
        # a step over two of the longest documents that the framework's tests run
        _case("step_2x131972_h32_kv8_d128_e4m3", "attend", [1, 1], [131971, 131971], 32, 8, 128, "e4m3", 64),
        # a sliding-window layer with capped scores, a cache that is not quantized
        _case("step_window_cap_32_h16_d128_bf16", "attend", [1] * 32, [2 * n + 1 for n in served[:32]], 16, 16, 128,
              "bf16", 64, left=2047, cap=50.0),
        # four drafted tokens a sequence, checked in one call
        _case("draft_16x4_h32_kv4_d128_e4m3", "attend", [4] * 16, served[:16], 32, 4, 128, "e4m3", 16),
        # a long prompt, the chunk that ends it
        _case("chunk_2048_of_16384_h32_kv8_d128_e4m3", "attend", [2048], [14336], 32, 8, 128, "e4m3", 64),
        # prompts' chunks and single steps in one call, ragged, capped, padding behind the last sequence
        _case("mixed_odd_h8_kv2_d64_bf16", "attend", [1283, 1, 77, 640, 1, 5], [2999, 4097, 0, 1500, 1, 640], 8, 2, 64,
              "bf16", 32, cap=30.0, pad=57),
        # chunks of four prompts in a sliding-window layer
        _case("chunk_4x1024_window_h16_d64_e4m3", "attend", [1024] * 4, [7168, 3000, 0, 5121], 16, 16, 64, "e4m3", 128,
              left=2047),
    ]


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "attend", "attend", "attend"])
        d = rng.choice([64, 128])
        fmt = rng.choice(["e4m3", "e4m3", "bf16"])
        page = rng.choice([16, 32, 64, 128])
        pad = rng.choice([0, 0, rng.randint(1, 200)])
        if op != "attend":
            total = int(2 ** rng.uniform(4, 14.5))
            n = rng.randint(1, max(1, min(64, total // 4)))
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            chunks = [b - a for a, b in zip([0] + cuts, cuts + [total])]
            before = [rng.choice([0, 0, rng.randint(0, 500)]) for _ in chunks]
            hkv = rng.choice([1, 2, 4, 8, 16])
            c = _case("", op, chunks, before, hkv, hkv, d, fmt, page, pad=pad)
        else:
            kind = rng.choice(["step", "step", "draft", "chunk", "mixed"])
            n = int(2 ** rng.uniform(0, 6)) if kind == "step" else rng.randint(1, 16)
            top = {"step": 1, "draft": rng.randint(2, 8), "chunk": int(2 ** rng.uniform(4, 11)), "mixed": int(2 ** rng.uniform(3, 10))}[kind]
            longest = int(2 ** rng.uniform(4, 16))
            chunks = [1 if kind == "mixed" and rng.random() < 0.5 else (top if kind != "mixed" else rng.randint(1, top)) for _ in range(n)]
            before = [rng.randint(0, longest) for _ in range(n)]
            hkv = rng.choice([1, 2, 4, 8])
            hq = hkv * rng.choice([1, 2, 4, 7, 8])
            c = _case("", op, chunks, before, hq, hkv, d, fmt, page, left=rng.choice([-1, -1, rng.randint(0, 4095)]),
                      cap=rng.choice([0.0, 0.0, 30.0, 50.0]), pad=pad)
            most = max(a + b for a, b in zip(chunks, before))
            if len(chunks) * max(chunks) * most * hq > 1 << 30 or len(chunks) * most * hkv * d > 1 << 29:
                continue
        del c["name"]
        return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _spans(case):
    """(new tokens, keys) of each sequence."""
    return [(c, c + b) for c, b in zip(_ints(case["chunks"]), _ints(case["before"]))]


def work(case):
    T, hq, hkv, d = sum(_ints(case["chunks"])), case["hq"], case["hkv"], case["d"]
    kept = d + 1 if case["fmt"] == "e4m3" else 2 * d           # bytes of a key or value in the cache
    if case["op"] != "attend":
        return {"bytes": 2 * T * hkv * (kept + 2 * d), "flops": 0}
    pairs = seen = 0
    for c, L in _spans(case):
        if c == 0:
            continue
        first = L - c if case["left"] < 0 else min(L - c, case["left"])          # keys before a token, at most
        if case["left"] < 0:
            pairs += c * (L - c) + c * (c + 1) // 2
        else:
            pairs += sum(min(i, case["left"]) + 1 for i in range(L - c, L))
        seen += c + first
    return {"bytes": 2 * seen * hkv * kept + 4 * T * hq * d + 4 * T * hq, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------ inputs

def _bits(e):
    """2^e for whole numbers e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _quantize(x):
    """fp32 [..., d] -> E4M3 codes and UE8M0 bytes [...]."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, 0, e - 9 + (m > 0.875).to(e.dtype)).clamp(-126, 127)
    return (x * _bits(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
    spans = _spans(case)
    T = sum(c for c, _ in spans) + case["pad"]
    used = [-(-L // P) for _, L in spans]
    width, pages = max(max(used), 1), sum(used) + 3
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev)
    st = {"case": case, "T": T, "N": len(spans), "scale": 1.0 / math.sqrt(d), "longest": max(L for _, L in spans)}
    # tokens differ in size, as a trained model's keys and values do
    for name in ("k", "v"):
        x = (rnd(pages, hkv, P, d) * torch.exp2(rnd(pages, hkv, P, 1))).to(torch.bfloat16)
        if case["fmt"] == "e4m3":
            st["pool_" + name], st["scales_" + name] = _quantize(x.float())
        else:
            st["pool_" + name], st["scales_" + name] = x, None
        del x
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(spans), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for n, u in enumerate(used):
        table[n, :u] = order[at:at + u]
        at += u
    cu = [0]
    for c, _ in spans:
        cu.append(cu[-1] + c)
    st["table"] = table
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["kv_lens"] = torch.tensor([L for _, L in spans], dtype=torch.int32, device=dev)
    if case["op"] == "write":
        st["k"], st["v"] = ((rnd(T, hkv, d) * torch.exp2(rnd(T, hkv, 1))).to(torch.bfloat16) for _ in range(2))
    elif case["op"] == "read":
        st["k"], st["v"] = (torch.empty(T, hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    else:
        st["q"] = (rnd(T, hq, d) * 2).to(torch.bfloat16)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import microscaled_precision_causal_gb300 as F
        pages = st["pool_k"].shape[0]
        st["cache"] = F.FlamiaPagedCache(pages, case["page"], case["hkv"], case["d"], fmt=case["fmt"])
        for name in ("k", "v"):
            getattr(st["cache"], name).copy_(st.pop("pool_" + name))
            scales = st.pop("scales_" + name)
            if scales is not None:
                getattr(st["cache"], name + "_scales").copy_(scales)
        st["att"] = F.FlamiaCachedAttention(st["T"], st["N"], case["hq"], case["hkv"], case["d"],
                                            max_chunk=max(_ints(case["chunks"])), max_pages=st["table"].shape[1],
                                            page_size=case["page"], window=case["left"], softcap=case["cap"])
        st["att"].plan_build(st["cu"], st["kv_lens"])
    return st


def _pools(k, v, k_scales, v_scales):
    if k_scales is None:
        return {"k": k, "v": v}
    f8 = torch.float8_e4m3fn
    return {"k": k.view(f8), "v": v.view(f8), "k_scales": k_scales, "v_scales": v_scales}


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        att, cache = st["att"], st["cache"]
        if op == "write":
            att.write(cache, st["k"], st["v"], st["table"])
            return _pools(cache.k, cache.v, cache.k_scales, cache.v_scales)
        if op == "read":
            att.read(cache, st["table"], st["k"], st["v"])
            return {"k": st["k"], "v": st["v"]}
        out, lse = att.forward(cache, st["q"], st["table"])
        return {"out": out, "lse": lse}
    if op == "write":
        return _plain_write(st)
    return _plain_read(st) if op == "read" else _plain_attend(st)


# ------------------------------------------------------------------------------------ plain form

def _rows(st):
    """(sequence, position) of every packed row; sequence N for the rows behind the last one."""
    row = torch.arange(st["T"], device=st["cu"].device)
    n = torch.searchsorted(st["cu"][1:].contiguous(), row, right=True)
    m = n.clamp(max=st["N"] - 1)
    return n, (st["kv_lens"][m] - st["cu"][m + 1] + row).long()


def _plain_write(st):
    n, pos = _rows(st)
    row = torch.nonzero(n < st["N"])[:, 0] if st["case"]["pad"] else slice(None)
    n, pos, P = n[row], pos[row], st["case"]["page"]
    page, slot = st["table"][n, pos // P].long(), pos % P
    for name in ("k", "v"):
        x = st[name][row]
        if st["scales_" + name] is not None:
            x, scale = _quantize(x.float())
            st["scales_" + name][page, :, slot] = scale
        st["pool_" + name][page, :, slot] = x
    return _pools(st["pool_k"], st["pool_v"], st["scales_k"], st["scales_v"])


def _values(st, name, n, pos):
    """fp32 rows [..., hkv, d] of the cache at positions pos of sequences n."""
    P = st["case"]["page"]
    page, slot = st["table"][n, pos // P].long().clamp(min=0), pos % P
    x = st["pool_" + name][page, :, slot]
    if st["scales_" + name] is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * _bits(st["scales_" + name][page, :, slot].int() - 127)[..., None]


def _plain_read(st):
    n, pos = _rows(st)
    m = n.clamp(max=st["N"] - 1)
    for name in ("k", "v"):
        x = _values(st, name, m, pos.clamp(min=0, max=st["longest"] - 1))
        st[name].copy_(torch.where((n < st["N"])[:, None, None], x, 0.0))
    return {"k": st["k"], "v": st["v"]}


def _plain_attend(st):
    case, T, N, dev = st["case"], st["T"], st["N"], st["cu"].device
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group, most, L = hq // hkv, max(_ints(case["chunks"])), st["longest"]
    # sequences side by side: [N, hkv, group * most, d] queries, [N, hkv, L, d] keys
    first = st["cu"][:-1].long()
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    t = torch.arange(most, device=dev)
    row = (first[:, None] + t).clamp(max=T - 1)
    q = st["q"][row].float().view(N, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(N, hkv, group * most, d)
    j = torch.arange(L, device=dev)
    n = torch.arange(N, device=dev)[:, None]
    s = torch.matmul(q, _values(st, "k", n, j[None, :]).permute(0, 2, 3, 1)) * st["scale"]
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    at = (st["kv_lens"].long() - new)[:, None] + t                                # positions [N, most]
    hidden = j > at[..., None]
    if case["left"] >= 0:
        hidden |= j < at[..., None] - case["left"]
    s = s.view(N, hkv, group, most, L).masked_fill_(hidden[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    del s
    l = e.sum(-1, keepdim=True)
    # keys behind a sequence's last one are anything, and weight 0 does not silence an infinity
    v = torch.where((j < st["kv_lens"][:, None])[..., None, None], _values(st, "v", n, j[None, :]), 0.0)
    o = torch.matmul(e.view(N, hkv, group * most, L), v.permute(0, 2, 1, 3)).view(N, hkv, group, most, d) / l
    lse = (m + torch.log(l))[..., 0]
    out_all = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=dev)
    lse_all = torch.full((hq, T), math.inf, device=dev)
    use = t < new[:, None]
    rows = row[use]
    out_all[rows] = o.permute(0, 3, 1, 2, 4).reshape(N, most, hq, d)[use].to(torch.bfloat16)
    lse_all[:, rows] = lse.permute(0, 3, 1, 2).reshape(N, most, hq)[use].t()
    return {"out": out_all, "lse": lse_all}


# ------------------------------------------------------------------------------------ in 64 bits

def _e4m3(y):
    """Nearest E4M3 value (ties to even) of fp64 |y| <= 448."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _decoded(st, name):
    x = st["pool_" + name]
    return x.view(torch.float8_e4m3fn).double() if x.dtype == torch.uint8 else x.double()


def exact(case, seed):
    st = _inputs(case, seed)
    P, hq, hkv, d, dev = case["page"], case["hq"], case["hkv"], case["d"], st["cu"].device
    table = st["table"].tolist()
    got, at = {}, 0
    if case["op"] == "write":
        for name in ("k", "v"):
            got[name], at = _decoded(st, name), 0
            for n, (c, L) in enumerate(_spans(case)):
                for p in range((L - c) // P, -(-L // P) if c else 0):
                    a, b = max(p * P, L - c), min(p * P + P, L)
                    x = st[name][at:at + b - a].double()
                    if case["fmt"] == "e4m3":
                        top = x.abs().amax(2, keepdim=True)
                        e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -300)))
                        e += (top > 448 * torch.exp2(e)).double()
                        e -= (top <= 448 * torch.exp2(e - 1)).double()
                        x = _e4m3(x / torch.exp2(torch.where(top == 0, 0.0, e)))
                    got[name][table[n][p], :, a - p * P:b - p * P] = x.transpose(0, 1)
                    at += b - a
        if case["fmt"] == "e4m3":
            got["k_scales"] = got["v_scales"] = None
        return got
    whole = {}
    for name in ("k", "v"):
        x = _decoded(st, name)
        if case["fmt"] == "e4m3":
            x = x * torch.exp2(st["scales_" + name].double() - 127)[..., None]
        whole[name] = [x[torch.tensor(table[n][:-(-L // P)], dtype=torch.long, device=dev)].transpose(0, 1).reshape(hkv, -1, d)[:, :L]
                       for n, (_, L) in enumerate(_spans(case))]
        del x
    if case["op"] == "read":
        for name in ("k", "v"):
            got[name] = torch.zeros(st["T"], hkv, d, dtype=torch.float64, device=dev)
            at = 0
            for n, (c, L) in enumerate(_spans(case)):
                got[name][at:at + c] = whole[name][n][:, L - c:].transpose(0, 1)
                at += c
        return got
    out = torch.zeros(st["T"], hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((hq, st["T"]), math.inf, dtype=torch.float64, device=dev)
    for n, (c, L) in enumerate(_spans(case)):
        for h in range(hq):
            key, val = whole["k"][n][h * hkv // hq], whole["v"][n][h * hkv // hq]
            step = max(1, (1 << 26) // max(L, 1))
            for a in range(0, c, step):
                b = min(c, a + step)
                u = st["q"][at + a:at + b, h].double() @ key.T / math.sqrt(d)
                if case["cap"]:
                    u = case["cap"] * torch.tanh(u / case["cap"])
                i = torch.arange(L - c + a, L - c + b, device=dev).unsqueeze(1)
                gap = i - torch.arange(L, device=dev).unsqueeze(0)
                no = gap < 0 if case["left"] < 0 else (gap < 0) | (gap > case["left"])
                u = torch.where(no, -math.inf, u)
                lse[h, at + a:at + b] = torch.logsumexp(u, 1)
                out[at + a:at + b, h] = torch.softmax(u, 1) @ val
        at += c
    return {"out": out, "lse": lse}
