"""The paged cache and its attention on the GPU: codes bit for bit, attention against the 64-bit
definition over the cache's own values (elementwise bounds that count roundings)."""
import numpy as np
import pytest

import cached_ref as C
import oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from microscaled_precision_causal_gb300 import build
    build.build()
    import microscaled_precision_causal_gb300 as F
    return F


def f64(t):
    return t.double().cpu().numpy()


def dev(x, dtype):
    import torch
    return torch.tensor(np.asarray(x), dtype=dtype).cuda()


def bf16(rng, *shape, gain=1.0):
    import torch
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(gain)).to(torch.bfloat16).cuda()


def same(a, b):
    import torch
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


class Batch:
    """Sequences with `before` tokens in the cache already and `chunks` new ones; pages in a random order."""

    def __init__(self, F, chunks, before, hq=4, hkv=2, d=64, fmt="e4m3", page=16, pad=0, seed=0, window=-1, softcap=0.0,
                 gain=2.0, scale=0.0, spare=2, sizes=1.0, max_chunk=None):
        import torch
        rng = np.random.default_rng(seed)
        self.F, self.chunks, self.keys = F, list(chunks), [a + b for a, b in zip(chunks, before)]
        self.hq, self.hkv, self.d, self.fmt, self.P = hq, hkv, d, fmt, page
        self.N, self.T = len(chunks), sum(chunks) + pad
        self.window, self.softcap, self.scale = window, softcap, scale
        used = [-(-n // page) for n in self.keys]
        width = max(used + [1])
        self.pages = sum(used) + spare
        order = rng.permutation(self.pages)
        table = np.full((self.N, width), -1)                     # (entries behind a sequence are not looked at)
        at = 0
        for n, u in enumerate(used):
            table[n, :u] = order[at:at + u]
            at += u
        self.table_np, self.table = table, dev(table.reshape(self.N, width), torch.int32)
        self.cu = dev(np.concatenate([[0], np.cumsum(chunks)]), torch.int32)
        self.kv_lens = dev(self.keys, torch.int32)
        self.cache = F.FlamiaPagedCache(self.pages, page, hkv, d, fmt)
        for name in ("k", "v"):
            x = bf16(rng, self.pages, hkv, page, d) * torch.from_numpy(
                np.exp2(sizes * rng.standard_normal((self.pages, hkv, page, 1))).astype(np.float32)).to(torch.bfloat16).cuda()
            self.fill(name, x)
        self.q = bf16(rng, self.T, hq, d, gain=gain)
        self.k, self.v = bf16(rng, self.T, hkv, d), bf16(rng, self.T, hkv, d, gain=3.0)
        self.att = F.FlamiaCachedAttention(self.T, self.N, hq, hkv, d, max_chunk or max(list(chunks) + [1]), width, page,
                                           window=window, softcap=softcap)
        self.att.plan_build(self.cu, self.kv_lens)

    def fill(self, name, x):
        import torch
        if self.fmt == "e4m3":
            codes, scales = C.quantize(f64(x))
            getattr(self.cache, name).copy_(torch.from_numpy(codes))
            getattr(self.cache, name + "_scales").copy_(torch.from_numpy(scales))
        else:
            getattr(self.cache, name).copy_(x)

    def pool(self, name):
        x = getattr(self.cache, name)
        return C.dequantize(x.cpu().numpy(), getattr(self.cache, name + "_scales").cpu().numpy()) if self.fmt == "e4m3" else f64(x)

    def rows(self, name):
        """Every sequence's [L, hkv, d] values in the cache."""
        pool = self.pool(name)
        return [pool[self.table_np[n, :-(-L // self.P)]].transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.d)[:L]
                for n, L in enumerate(self.keys)]

    def places(self):
        """(page, slot) of every packed row of the sequences."""
        pos = [(n, L - c + t) for n, (c, L) in enumerate(zip(self.chunks, self.keys)) for t in range(c)]
        return np.array([(self.table_np[n, p // self.P], p % self.P) for n, p in pos]).reshape(-1, 2)

    def forward(self, **kw):
        return self.att.forward(self.cache, self.q, self.table, softmax_scale=self.scale, **kw)

    def check(self):
        import torch
        self.att.out.fill_(float("nan"))
        self.att.lse.fill_(float("nan"))
        self.att.workspace.fill_(255)
        out, lse = self.forward()
        torch.cuda.synchronize()
        assert self.att.device_status() == 0
        self.within(f64(out), f64(lse))
        return out, lse

    def within(self, out, lse, skip=()):
        keys, values, q, at = self.rows("k"), self.rows("v"), f64(self.q), 0
        for n, c in enumerate(self.chunks):
            rows = slice(at, at + c)
            at += c
            if c == 0 or n in skip:
                continue
            ref = C.attend(q[rows], keys[n], values[n], self.hq // self.hkv, scale=self.scale or None, left=self.window,
                           softcap=self.softcap)
            for name, got in (("o", out[rows]), ("lse", lse[:, rows])):
                assert np.isfinite(got).all(), f"{name} of sequence {n}"
                over = np.abs(got - ref[name]) - ref["tol_" + name]
                assert (over <= 0).all(), f"{name} of sequence {n}: {over.max():.3e} over its bound at {np.argmax(over)} of {over.size}"
        assert (out[at:] == 0).all() and np.isposinf(lse[:, at:]).all()


BOTH = pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
DIMS = pytest.mark.parametrize("d", [64, 128])


# ------------------------------------------------------------------ write, read

@BOTH
@DIMS
@pytest.mark.parametrize("page,hkv", [(16, 2), (32, 1), (64, 5), (128, 16)])
def test_write_and_read(F, fmt, d, page, hkv):
    """New rows bit for bit, every other slot as it was; read back: the code times its scale, rows behind 0."""
    import torch
    b = Batch(F, [5, 0, 1, 200, 17], [11, 40, 16, 0, 3], hkv, hkv, d, fmt, page, pad=9, seed=page + d)
    b.k *= torch.exp2(torch.randint(-30, 30, (b.T, hkv, 1), device="cuda")).to(torch.bfloat16)
    b.k[3], b.k[4, 0, :] = 0, 0.0
    b.k[7, 0, 5], b.k[8, 0, :3] = 3.3e38, 1e-39                                  # the type's ends
    b.v[9, 0, 2], b.v[10, 0, :2] = float("inf"), torch.tensor([float("-inf"), 1.0])
    b.v[11, 0, 1] = float("nan")
    names = ["k", "v"] + (["k_scales", "v_scales"] if fmt == "e4m3" else [])
    old = {n: getattr(b.cache, n).cpu() for n in names}
    b.att.write(b.cache, b.k, b.v, b.table)
    torch.cuda.synchronize()
    assert b.att.device_status() == 0
    at, n = b.places(), sum(b.chunks)
    for name in ("k", "v"):
        x = f64(getattr(b, name))[:n]
        want = {name: old[name].clone()}
        if fmt == "e4m3":
            codes, scales = C.quantize(x)
            want[name + "_scales"] = old[name + "_scales"].clone()
            want[name][at[:, 0], :, at[:, 1]] = torch.from_numpy(codes)
            want[name + "_scales"][at[:, 0], :, at[:, 1]] = torch.from_numpy(scales)
        else:
            want[name][at[:, 0], :, at[:, 1]] = getattr(b, name)[:n].cpu()
        for part, w in want.items():
            assert same(getattr(b.cache, part).cpu(), w), part
    k, v = (torch.full_like(b.k, float("nan")) for _ in range(2))
    assert b.att.read(b.cache, b.table, k, v) == (k, v)
    torch.cuda.synchronize()
    assert b.att.device_status() == 0
    for name, got in (("k", k), ("v", v)):
        want = torch.from_numpy(b.pool(name)[at[:, 0], :, at[:, 1]]).to(torch.bfloat16)
        assert torch.equal(got[:n].cpu().nan_to_num(nan=7.0, posinf=5.0, neginf=-5.0),
                           want.nan_to_num(nan=7.0, posinf=5.0, neginf=-5.0)), name
        assert (got[n:] == 0).all()


@BOTH
def test_read_of_whole_sequences(F, fmt):
    import torch
    b = Batch(F, [300, 1, 0, 129], [0, 0, 0, 0], 3, 3, 128, fmt, 32, pad=70, seed=4)
    k, v = torch.full_like(b.k, float("nan")), torch.full_like(b.v, float("nan"))
    b.att.read(b.cache, b.table, k, v)
    for name, got in (("k", k), ("v", v)):
        assert np.array_equal(f64(got)[:430], np.concatenate(b.rows(name))) and (got[430:] == 0).all()


def test_codes_are_the_operand_quantizers_per_token_form(F):
    """A sequence's codes in the cache equal flamia_quantize_tokenblock's with per_token."""
    import torch
    b = Batch(F, [77, 40], [0, 0], 2, 2, 128, "e4m3", 16, seed=5)
    b.att.write(b.cache, b.k, b.v, b.table)
    plan = torch.zeros(F.flamia_plan_bytes(b.T, 2), dtype=torch.uint8, device="cuda")
    codes, scales = torch.empty_like(b.k, dtype=torch.uint8), torch.empty(b.T, 2, dtype=torch.uint8, device="cuda")
    F.flamia_plan_build(b.cu, 2, b.T, plan)
    F.flamia_quantize_tokenblock(b.v, b.cu, 2, plan, codes, scales, per_token=True)
    at = b.places()
    assert torch.equal(b.cache.v[at[:, 0], :, at[:, 1]], codes) and torch.equal(b.cache.v_scales[at[:, 0], :, at[:, 1]], scales)


# ------------------------------------------------------------------ attention

STEPS = {
    "one": ([1], [0]), "short": ([1, 1, 1], [1, 15, 16]), "ragged": ([1] * 7, [0, 63, 64, 65, 500, 127, 1300]),
    "drafts": ([4, 2, 3, 1], [200, 0, 61, 700]), "gaps": ([1, 0, 1, 0, 0, 1], [30, 0, 90, 7, 0, 260]),
}
CHUNKS = {
    "whole": ([300], [0]), "later": ([130], [401]), "odd": ([129, 1, 0, 257, 33, 5], [100, 64, 3, 0, 1000, 640]),
    "longer": ([700, 64], [900, 2000]),
}
HEADS = pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (3, 1), (16, 1), (20, 2)])


@BOTH
@DIMS
@HEADS
@pytest.mark.parametrize("layout", STEPS)
def test_steps(F, layout, hq, hkv, d, fmt):
    Batch(F, *STEPS[layout], hq, hkv, d, fmt, 16, pad=3, seed=1).check()


@BOTH
@DIMS
@HEADS
@pytest.mark.parametrize("layout", CHUNKS)
def test_chunks(F, layout, hq, hkv, d, fmt):
    Batch(F, *CHUNKS[layout], hq, hkv, d, fmt, 32, pad=5, seed=2).check()


@BOTH
@DIMS
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_page_sizes(F, page, d, fmt):
    Batch(F, [1, 200, 2], [777, 150, 129], 4, 2, d, fmt, page, seed=3).check()


@BOTH
@DIMS
@pytest.mark.parametrize("window", [0, 1, 63, 64, 100, 1000, 2**31 - 1])
def test_windows(F, window, d, fmt):
    Batch(F, [1, 4, 300, 1], [900, 500, 300, 20], 4, 2, d, fmt, 16, seed=4, window=window, pad=1).check()


@BOTH
@DIMS
@pytest.mark.parametrize("softcap", [1e-3, 0.5, 5.0, 50.0, 1e4])
def test_caps(F, softcap, d, fmt):
    Batch(F, [1, 3, 200], [300, 64, 90], 4, 2, d, fmt, 16, seed=5, softcap=softcap, gain=4.0).check()


@DIMS
def test_window_and_cap_together(F, d):
    Batch(F, [1, 1, 150], [1000, 3, 700], 2, 1, d, "e4m3", 64, seed=6, softcap=8.0, window=200).check()


@BOTH
@pytest.mark.parametrize("scale", [1e-6, 0.02, 3.0])
def test_scales(F, scale, fmt):
    Batch(F, [1, 140], [300, 60], 4, 2, 128, fmt, 16, seed=7, scale=scale).check()


@BOTH
@DIMS
@pytest.mark.parametrize("sizes", [8.0, 25.0])
def test_tokens_of_very_different_size(F, sizes, d, fmt):
    """Scales 2^(25 x) apart: a large value that is not attended to must not cost the others their digits."""
    Batch(F, [1, 4, 150], [600, 300, 200], 4, 2, d, fmt, 16, seed=8, sizes=sizes, scale=2.0 ** -12, gain=0.01).check()


@BOTH
@DIMS
@pytest.mark.parametrize("exponent", [-114, 100])
def test_values_near_the_ends_of_their_range(F, exponent, d, fmt):
    """Value scales down to a byte of some 6, and up to 2^95: steps of one and two row tiles, a chunk."""
    for chunks in ([1, 4, 150], [1, 4, 8]):
        b = Batch(F, chunks, [600, 300, 200], 8, 2, d, fmt, 16, seed=33)
        b.fill("v", bf16(np.random.default_rng(34), *b.cache.v.shape, gain=2.0 ** exponent))
        b.check()


@pytest.mark.parametrize("shape", [([1], [16000]), ([1, 1], [9000, 20000]), ([2], [6000]), ([40], [12000]), ([300], [5000])])
@DIMS
def test_long_contexts_are_split_and_joined(F, shape, d):
    Batch(F, *shape, 4, 1, d, "e4m3", 64, seed=9).check()


@BOTH
@DIMS
@pytest.mark.parametrize("hq,hkv,chunks", [(32, 1, [1, 1, 0, 1]), (24, 1, [1, 1]), (4, 1, [8, 5, 7]), (12, 4, [10, 9, 1]), (40, 1, [1, 1, 2]),
                                           (160, 1, [1, 2, 0])])
def test_rows_around_the_tiles(F, hq, hkv, chunks, d, fmt):
    """One and two row tiles of a step, the least chunks, groups above both tiles' rows; many pieces to a unit."""
    for before in (7000, 90):
        Batch(F, chunks, [before + 100 * n for n in range(len(chunks))], hq, hkv, d, fmt, 64, seed=27, pad=2).check()


@BOTH
@DIMS
def test_steps_beside_chunks(F, d, fmt):
    """A few steps among chunks, and a few chunks among steps: either kind gets its SMs, and each result its definition."""
    Batch(F, [300, 1, 200, 2, 1], [100, 3000, 700, 64, 5000], 4, 2, d, fmt, 16, seed=28, window=4000).check()
    Batch(F, [1] * 30 + [40], [3000 + 50 * n for n in range(31)], 8, 4, d, fmt, 64, seed=29).check()


@BOTH
@DIMS
@pytest.mark.parametrize("chunk,count", [(1, 200), (26, 60)])
@pytest.mark.parametrize("longest", [200, 30000])
def test_short_sequences_and_a_long_one(F, longest, chunk, count, d, fmt):
    """Many short units, some of them a CTA's, and the same ones beside one that has to be split."""
    before = [7 * n % 190 for n in range(count - 1)] + [longest]
    Batch(F, [chunk] * count, before, 16, 4, d, fmt, 64, seed=32, pad=1).check()


@pytest.mark.parametrize("window,gone", [(100, [900 - 1 - 100, 2000 - 4 - 100, 700 - 300 - 100]), (0, [899, 1996, 400])])
def test_pages_before_a_window_may_be_given_back(F, window, gone):
    import torch
    b = Batch(F, [1, 4, 300], [899, 1996, 400], 4, 2, 64, "e4m3", 16, seed=30, window=window)
    want = [t.clone() for t in b.check()]
    for n, first in enumerate(gone):
        b.table[n, :first // 16] = -7
    out = b.forward()
    assert b.att.device_status() == 0 and all(torch.equal(x, y) for x, y in zip(out, want))


def test_one_plan_serves_many_calls(F):
    """Layers of a step on one plan, split units in all of them, one after the other without a wait between."""
    import torch
    layers = [Batch(F, [1, 200, 1], [9000, 3000, 64], 4, 1, 128, fmt, 64, seed=31 + i) for i, fmt in enumerate(("e4m3", "bf16", "e4m3"))]
    att = layers[0].att
    want = [[t.clone() for t in b.check()] for b in layers]
    got = []
    for _ in range(4):
        for b in layers:
            got.append([t.clone() for t in att.forward(b.cache, b.q, b.table)])
    torch.cuda.synchronize()
    assert att.device_status() == 0
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 3]))


def test_many_sequences(F):
    rng = np.random.default_rng(10)
    chunks = rng.choice([0, 1, 1, 1, 2, 30], 1500)
    Batch(F, [int(x) for x in chunks], [int(x) for x in rng.integers(0, 90, 1500)], 4, 2, 64, "e4m3", 16, seed=10, pad=4).check()


def test_a_bound_on_chunks_above_the_chunks(F):
    """Steps alone in a call that could bring chunks, and the same bits as in one that could not."""
    import torch
    a = Batch(F, [1, 1], [500, 300], 4, 2, 64, seed=11)
    b = Batch(F, [1, 1], [500, 300], 4, 2, 64, seed=11, max_chunk=600)
    assert all(torch.equal(x, y) for x, y in zip(a.check(), b.check()))


def test_no_sequences_and_no_tokens(F):
    import torch
    Batch(F, [0, 0], [5, 0], pad=40).check()
    Batch(F, [0, 0], [5, 0], pad=0).check()
    att = F.FlamiaCachedAttention(7, 0, 4, 2, 64, 1, 1, 16)
    att.plan_build(dev([0], torch.int32), dev([], torch.int32))
    cache = F.FlamiaPagedCache(1, 16, 2, 64)
    out, lse = att.forward(cache, torch.ones(7, 4, 64, dtype=torch.bfloat16, device="cuda"),
                           torch.empty(0, 1, dtype=torch.int32, device="cuda"))
    assert (out == 0).all() and torch.isposinf(lse).all() and att.device_status() == 0


# ------------------------------------------------------------------ garbage, bad arguments

@BOTH
@DIMS
def test_pages_may_hold_anything_behind_the_last_position(F, d, fmt):
    import torch
    b = Batch(F, [1, 4, 150, 1], [600, 300, 205, 0], 4, 2, d, fmt, 64, seed=12, pad=50)
    want = [t.clone() for t in b.check()]
    keep = torch.zeros(b.pages, b.P, dtype=torch.bool)
    for n, L in enumerate(b.keys):
        for j in range(L):
            keep[b.table_np[n, j // b.P], j % b.P] = True
    keep = keep.cuda()[:, None, :, None]
    for fill, byte in ((float("nan"), 255), (float("inf"), 0x7e), (float("-inf"), 254)):
        for name in ("k", "v"):
            x = getattr(b.cache, name)
            x.copy_(torch.where(keep, x, torch.full_like(x, byte if fmt == "e4m3" else fill)))
            if fmt == "e4m3":
                s = getattr(b.cache, name + "_scales")
                s.copy_(torch.where(keep[..., 0], s, torch.full_like(s, 255 if byte == 255 else 254)))
        b.q[sum(b.chunks):] = fill
        assert all(torch.equal(x, y) for x, y in zip(b.forward(), want))


@BOTH
@DIMS
def test_a_sequence_of_infinities_stays_alone(F, d, fmt):
    import torch
    b = Batch(F, [1, 4, 150, 1, 129], [600, 300, 205, 0, 300], 4, 2, d, fmt, 16, seed=13)
    want = [t.clone() for t in b.check()]
    rows = torch.ones(b.T, dtype=torch.bool, device="cuda")
    rows[1:155] = False
    for n in (1, 2):
        for p in b.table_np[n]:
            if p >= 0:
                if fmt == "e4m3":
                    b.cache.k_scales[p], b.cache.v_scales[p] = 255, 255
                else:
                    b.cache.k[p], b.cache.v[p] = float("nan"), float("inf")
    b.q[1:5] = float("inf")
    out, lse = b.forward()
    assert torch.equal(out[rows], want[0][rows]) and torch.equal(lse[:, rows], want[1][:, rows])
    assert not torch.isfinite(out[5:155].float()).any()


@BOTH
def test_a_nan_shows(F, fmt):
    """A NaN key or value is written as one and shows in the rows that see it."""
    import torch
    for name in ("k", "v"):
        b = Batch(F, [1, 4, 200], [70, 0, 300], 4, 2, 64, fmt, 16, seed=14)
        getattr(b, name)[0, 1, 3] = float("nan")
        getattr(b, name)[5, 0, 3] = float("nan")
        b.att.write(b.cache, b.k, b.v, b.table)
        out, lse = b.forward()
        d = slice(None) if name == "k" or fmt == "e4m3" else 3
        assert torch.isnan(out[0, 2:, d].float()).all() and torch.isfinite(out[0, :2].float()).all()
        assert torch.isnan(out[5:, :2, d].float()).all() and torch.isfinite(out[1:5].float()).all()
        assert torch.isfinite(out[5:, 2:].float()).all()


def _untouched(b, run):
    """run() between guards: the pools keep their bits."""
    import torch
    names = ["k", "v"] + (["k_scales", "v_scales"] if b.fmt == "e4m3" else [])
    old = [getattr(b.cache, n).clone() for n in names]
    got = run()
    torch.cuda.synchronize()
    assert all(same(getattr(b.cache, n), o) for n, o in zip(names, old))
    return got


@pytest.mark.parametrize("chunks", [[1, 1, 1], [1, 150, 3]])
@pytest.mark.parametrize("what", ["kv_short", "kv_long", "kv_negative", "cu_decreasing", "cu_long", "cu_first", "chunk"])
def test_bad_lengths(F, what, chunks):
    import torch
    b = Batch(F, chunks, [40, 200, 8], 4, 2, 64, seed=15, pad=6)
    cu, kv = b.cu.clone(), b.kv_lens.clone()
    want = F.DEV_BAD_KV_LENS
    if what.startswith("kv"):
        kv[1] = {"kv_short": chunks[1] - 1, "kv_long": b.table.shape[1] * b.P + 1, "kv_negative": -1}[what]
    elif what == "chunk":
        cu[1:], want = cu[1:] + 6, F.DEV_CAPACITY
        kv += 200
        if chunks[1] == 150:
            cu[2] += 0
            cu[1] = 1
    else:
        cu[{"cu_decreasing": 1, "cu_long": 3, "cu_first": 0}[what]] = {"cu_decreasing": 500, "cu_long": b.T + 1, "cu_first": 1}[what]
        want = F.DEV_BAD_CU_SEQLENS
    b.att.plan_build(cu, kv)
    k, v = torch.ones_like(b.k), torch.ones_like(b.v)

    def run():
        b.att.write(b.cache, b.k, b.v, b.table)
        b.att.read(b.cache, b.table, k, v)
        return b.forward()
    out, lse = _untouched(b, run)
    assert b.att.device_status() & want
    assert (out == 0).all() and torch.isposinf(lse).all() and (k == 0).all() and (v == 0).all()
    b.att.plan_build(b.cu, b.kv_lens)                       # a good plan clears the status
    b.check()


@BOTH
@pytest.mark.parametrize("page", [-1, -2**31, 2**31 - 1, "one more"])
def test_bad_pages(F, page, fmt):
    """A page outside the cache: nothing is read or written there, the other sequences keep their results."""
    import torch
    b = Batch(F, [1, 40, 2, 300], [40, 200, 8, 100], 4, 2, 64, fmt, 16, seed=16, pad=6)
    want = [t.clone() for t in b.check()]
    good = b.table.clone()
    page = b.pages if page == "one more" else page
    b.table[0, 2], b.table[1, 3], b.table[1, 14] = page, page, page          # of the new token; an old one; new ones
    k, v = torch.ones_like(b.k), torch.ones_like(b.v)
    b.att.read(b.cache, b.table, k, v)
    assert b.att.device_status() == F.DEV_BAD_PAGE
    b.att.plan_build(b.cu, b.kv_lens)
    out, lse = _untouched(b, b.forward)
    assert b.att.device_status() == F.DEV_BAD_PAGE
    rows = torch.ones(b.T, dtype=torch.bool, device="cuda")
    rows[:41] = False
    assert torch.equal(out[rows], want[0][rows]) and torch.equal(lse[:, rows], want[1][:, rows])
    lost = [0] + [1 + t for t in range(40) if (200 + t) // 16 == 14]
    assert (k[lost] == 0).all() and (v[lost] == 0).all() and (k[41] != 0).any()
    b.att.plan_build(b.cu, b.kv_lens)
    old = b.cache.k.clone()
    b.att.write(b.cache, b.k, b.v, b.table)
    assert b.att.device_status() == F.DEV_BAD_PAGE
    at = b.places()
    some = np.setdiff1d(np.arange(len(at)), lost)
    touched = torch.zeros(b.pages, b.P, dtype=torch.bool)
    touched[at[some, 0], at[some, 1]] = True
    changed = (b.cache.k != old).any(3).any(1).cpu()
    assert torch.equal(changed, touched)
    b.table.copy_(good)


@pytest.mark.parametrize("other", [dict(T=1), dict(N=1), dict(hq=4), dict(chunk=1), dict(left=1)])
def test_a_plan_of_another_call(F, other):
    import torch
    b = Batch(F, [1, 40], [40, 200], 8, 2, 64, seed=17)
    T, N, hq = b.T + other.get("T", 0), 2 + other.get("N", 0), 8 - other.get("hq", 0)
    plan = torch.zeros(F.flamia_cache_plan_bytes(100, 10, 8, 2), dtype=torch.uint8, device="cuda")
    F.flamia_cache_plan_build(b.cu, b.kv_lens, 2, b.T, 8, 2, 40, b.table.shape[1] * 16, -1, plan)
    q = torch.ones(T, hq, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.ones_like(q), torch.zeros(hq, T, device="cuda")
    table = torch.zeros(N, b.table.shape[1], dtype=torch.int32, device="cuda")
    F.flamia_cached_fwd(q, b.cache.view, table, N, plan, out, lse, b.att.workspace, 40 + other.get("chunk", 0),
                        window_left=-1 + other.get("left", 0))
    assert F.flamia_get_device_status(plan) == F.DEV_PLAN_MISMATCH
    assert (out == 0).all() and torch.isposinf(lse).all()


# ------------------------------------------------------------------ as a program uses it

@BOTH
def test_equal_inputs_give_equal_bits(F, fmt):
    import torch
    b = Batch(F, [1, 300, 4, 1], [5000, 800, 64, 200], 8, 2, 128, fmt, 16, seed=18)
    want = [t.clone() for t in b.check()]
    for _ in range(5):
        b.att.workspace.fill_(255)
        assert all(torch.equal(x, y) for x, y in zip(b.forward(), want))


@BOTH
def test_captured_and_replayed_with_other_lengths(F, fmt):
    """A captured step (plan, write, attention) replayed for other lengths, tables and values."""
    import torch
    b = Batch(F, [1, 3, 40], [100, 64, 0], 4, 2, 64, fmt, 16, seed=19, spare=3)
    c = Batch(F, [2, 40, 1], [60, 25, 103], 4, 2, 64, fmt, 16, seed=20, pad=1)
    assert b.T == c.T and b.table.shape == c.table.shape and b.pages == c.pages
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.att.plan_build(b.cu, b.kv_lens)
        b.att.write(b.cache, b.k, b.v, b.table)
        b.forward()
    for s in (b, c, b):
        s.att.plan_build(s.cu, s.kv_lens)
        s.att.write(s.cache, s.k, s.v, s.table)
        want = [t.clone() for t in s.check()]
        names = ["q", "k", "v", "cu", "kv_lens", "table"]
        old = [getattr(b, n).clone() for n in names]
        parts = ["k", "v"] + (["k_scales", "v_scales"] if fmt == "e4m3" else [])
        pools = [getattr(b.cache, n).clone() for n in parts]
        for n in names:
            getattr(b, n).copy_(getattr(s, n))
        for n in parts:
            getattr(b.cache, n).copy_(getattr(s.cache, n))
        b.att.workspace.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert b.att.device_status() == 0
        assert all(torch.equal(x, y) for x, y in zip((b.att.out, b.att.lse), want))
        for n, o in zip(names, old):
            getattr(b, n).copy_(o)
        for n, o in zip(parts, pools):
            getattr(b.cache, n).copy_(o)


def test_captured_twice_in_a_row(F):
    import torch
    b = Batch(F, [1, 1, 200], [3000, 64, 700], 4, 2, 128, seed=21)
    want = [t.clone() for t in b.check()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            b.forward()
    for _ in range(3):
        b.att.out.fill_(float("nan"))
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((b.att.out, b.att.lse), want))


def test_two_streams_and_one_cache(F):
    """Two objects' calls on one cache overlap; a call on another stream than the current one."""
    import torch
    b = Batch(F, [1, 1, 200], [3000, 64, 700], 4, 2, 128, seed=22)
    c = Batch(F, [1] * 9, [700] * 9, 8, 8, 64, "bf16", seed=23)
    want = [[t.clone() for t in x.check()] for x in (b, c)]
    other = F.FlamiaCachedAttention(b.T, b.N, 4, 2, 128, b.att.max_chunk, b.table.shape[1], 16)
    other.plan_build(b.cu, b.kv_lens)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        b.forward(stream=streams[0])
        c.forward(stream=streams[1])
        other.forward(b.cache, b.q, b.table, stream=streams[2])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((b.att.out, b.att.lse), want[0]))
    assert all(torch.equal(x, y) for x, y in zip((other.out, other.lse), want[0]))
    assert all(torch.equal(x, y) for x, y in zip((c.att.out, c.att.lse), want[1]))


def test_tensors_at_the_smallest_alignment(F):
    import torch
    b = Batch(F, [1, 200, 3], [300, 64, 70], 4, 2, 64, seed=24)
    b.att.write(b.cache, b.k, b.v, b.table)
    want = [t.clone() for t in b.check()]
    pool = b.cache.k.clone()

    def moved(t):
        n = 16 // t.element_size()
        v = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")[n:].view(t.shape)
        v.copy_(t)
        return v
    for x, names in ((b, ("q", "k", "v")), (b.att, ("out", "lse")), (b.cache, ("k", "v", "k_scales", "v_scales"))):
        for n in names:
            setattr(x, n, moved(getattr(x, n)))
    for n in ("k", "v", "k_scales", "v_scales"):
        setattr(b.cache.view, n, getattr(b.cache, n).data_ptr())
    assert all(torch.equal(x, y) for x, y in zip(b.forward(), want))
    at = b.places()
    b.cache.k[at[:, 0], :, at[:, 1]] = 0
    b.att.write(b.cache, b.k, b.v, b.table)
    assert torch.equal(b.cache.k, pool)
    k, v = moved(b.k), moved(b.v)
    b.att.read(b.cache, b.table, k, v)
    assert torch.equal(k.double().cpu(), torch.from_numpy(b.pool("k")[at[:, 0], :, at[:, 1]]))


@BOTH
def test_offsets_past_32_bits(F, fmt):
    """A cache of more than 4 GB whose last pages are used."""
    import torch
    hkv, P, d = 16, 128, 128
    pages = (1 << 32) // (hkv * P * d * (1 if fmt == "e4m3" else 2)) + 40
    b = Batch(F, [1, 300, 1], [900, 250, 0], 16, hkv, d, fmt, P, seed=25, spare=0)
    big = F.FlamiaPagedCache(pages, P, hkv, d, fmt)
    for n in ["k", "v"] + (["k_scales", "v_scales"] if fmt == "e4m3" else []):
        getattr(big, n)[pages - b.pages:] = getattr(b.cache, n)
    want = [t.clone() for t in b.check()]
    b.table[b.table >= 0] += pages - b.pages
    b.cache = big
    assert all(torch.equal(x, y) for x, y in zip(b.forward(), want))
    b.att.write(big, b.k, b.v, b.table)
    k, v = torch.empty_like(b.k), torch.empty_like(b.v)
    b.att.read(big, b.table, k, v)
    assert b.att.device_status() == 0
    step = 2.0 ** -4 if fmt == "e4m3" else 0.0
    top = b.k.float().abs().amax(2, keepdim=True) * 2.0 ** -17          # (half a subnormal step)
    assert ((k.float() - b.k.float()).abs() <= step * b.k.float().abs() + step * 16 * top).all()


@BOTH
def test_generation_over_two_layers(F, fmt):
    """Prompts in chunks, then drafts and single tokens: every step's rows against the whole sequences' attention
    over what the caches hold in the end (a later token changes no earlier code)."""
    import torch
    rng = np.random.default_rng(26)
    hq, hkv, d, P, layers = 8, 2, 64, 16, 2
    plan = [[150, 40, 0], [77, 1, 33], [1, 1, 1], [4, 2, 1], [1, 0, 1], [1, 1, 1]]
    total = np.sum(plan, 0)
    width = -(-int(total.max()) // P)
    table_np = rng.permutation(3 * width + 1)[:3 * width].reshape(3, width)
    table = dev(table_np, torch.int32)
    caches = [F.FlamiaPagedCache(3 * width + 1, P, hkv, d, fmt) for _ in range(layers)]
    x = {n: [bf16(rng, 3, int(total.max()), h, d, gain=g) for _ in range(layers)] for n, h, g in (("q", hq, 2.0), ("k", hkv, 1.0), ("v", hkv, 1.0))}
    outs = [[np.zeros((L, hq, d)) for L in total] for _ in range(layers)]
    lses = [[np.zeros((hq, L)) for L in total] for _ in range(layers)]
    done = np.zeros(3, int)
    for chunks in plan:
        new = np.array(chunks)
        att = F.FlamiaCachedAttention(int(new.sum()), 3, hq, hkv, d, int(new.max()), width, P)
        cu = np.concatenate([[0], np.cumsum(new)])
        att.plan_build(dev(cu, torch.int32), dev(done + new, torch.int32))
        for i in range(layers):
            q, k, v = (torch.cat([x[n][i][s, done[s]:done[s] + new[s]] for s in range(3)]).contiguous() for n in ("q", "k", "v"))
            att.write(caches[i], k, v, table)
            out, lse = att.forward(caches[i], q, table)
            assert att.device_status() == 0
            for s in range(3):
                outs[i][s][done[s]:done[s] + new[s]] = f64(out[cu[s]:cu[s + 1]])
                lses[i][s][:, done[s]:done[s] + new[s]] = f64(lse[:, cu[s]:cu[s + 1]])
        done += new
    for i in range(layers):
        back = F.FlamiaCachedAttention(int(total.sum()), 3, hq, hkv, d, int(total.max()), width, P)
        back.plan_build(dev(np.concatenate([[0], np.cumsum(total)]), torch.int32), dev(total, torch.int32))
        k, v = (torch.empty(int(total.sum()), hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        back.read(caches[i], table, k, v)
        at = 0
        for s, L in enumerate(total):
            ref = C.attend(f64(x["q"][i][s, :L]), f64(k[at:at + L]), f64(v[at:at + L]), hq // hkv)
            at += L
            assert (np.abs(outs[i][s] - ref["o"]) <= ref["tol_o"]).all() and (np.abs(lses[i][s] - ref["lse"]) <= ref["tol_lse"]).all()


# ------------------------------------------------------------------ infinities of an E4M3 cache

def _as_read(pool):
    """The cache's values as reading gives them: a code times its scale past bf16's range is an infinity."""
    import torch
    return f64(torch.from_numpy(pool).to(torch.bfloat16))


ROWS = {"steps": [1, 4, 1], "two_row_tiles": [1, 8, 1], "chunks": [1, 60, 1]}        # (of four heads on one)
ENDS = [(fmt, x) for x in (float("inf"), float("-inf")) for fmt in ("e4m3", "bf16")] + [("e4m3", 3.35e38)]


@DIMS
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("fmt,value", ENDS)
def test_an_infinite_key(F, value, softcap, rows, d, fmt):
    """Scores +inf: nothing finite in the row.  Scores -inf: the key has no weight.  Capped: the cap."""
    import torch
    chunks = ROWS[rows]
    b = Batch(F, chunks, [70, 200, 300], 8, 2, d, fmt, 16, seed=35, softcap=softcap)
    a, big = 5, 40 * softcap * np.sqrt(d)       # (in its place: scores beyond 20 caps, tanh 1 in any precision)
    sign = torch.from_numpy(np.random.default_rng(36).choice([-1.0, 1.0], (b.T, 8))).cuda()
    b.q[:, :, a] = (sign * (0.5 + b.q[:, :, a].double().abs().clamp(max=1.5))).to(torch.bfloat16)
    row = 1                                     # the second sequence's first new token, kv head 1
    b.k[row, 1, a] = value
    b.att.write(b.cache, b.k, b.v, b.table)
    out, lse = b.forward()
    assert b.att.device_status() == 0
    keys, vals, q, at = [_as_read(x) for x in b.rows("k")], b.rows("v"), f64(b.q), 0
    assert np.isinf(keys[1][200, 1, a]) and np.isfinite(keys[1]).sum() == keys[1].size - 1
    up = f64(sign)[1:1 + chunks[1]] * np.sign(value) > 0
    for n, c in enumerate(chunks):
        o, l = f64(out[at:at + c]), f64(lse[:, at:at + c])
        for h in range(8):
            g, one = h // 4, q[at:at + c, h:h + 1]
            K, V = keys[n][:, g:g + 1], vals[n][:, g:g + 1]
            if n == 1 and g == 1:
                K = np.where(np.isinf(K), np.sign(K) * big, K)
            full = C.attend(one, K, V, 1, softcap=softcap)
            if n == 1 and g == 1 and not softcap:
                bad = up[:, h]
                assert not np.isfinite(o[bad, h]).any() and not np.isfinite(l[h, bad]).any(), h
                # the others: as without the key
                keep = np.arange(len(K)) != 200
                for t in np.nonzero(~bad)[0]:
                    if t == 0 and keep[:201].sum() == 0:
                        continue
                    x = C.attend(one[t:t + 1], K[keep][:200 + t], V[keep][:200 + t], 1)
                    assert (np.abs(o[t, h] - x["o"][0, 0]) <= x["tol_o"][0, 0]).all() and abs(l[h, t] - x["lse"][0, 0]) <= x["tol_lse"][0, 0]
            else:
                assert (np.abs(o[:, h] - full["o"][:, 0]) <= full["tol_o"][:, 0]).all(), (n, h)
                assert (np.abs(l[h] - full["lse"][0]) <= full["tol_lse"][0]).all(), (n, h)
        at += c


@DIMS
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("fmt,value", ENDS + [("e4m3", 3.1e38)])
def test_an_infinite_value(F, value, softcap, rows, d, fmt):
    """It shows in its head dimension of every row that sees it, however small its weight; the largest finite code does not."""
    import torch
    chunks = ROWS[rows]
    b = Batch(F, chunks, [70, 200, 300], 8, 2, d, fmt, 16, seed=37, softcap=softcap, gain=0.5)
    a, row = 9, 1
    b.k[row, 1] = -b.q[row, 4:8].float().mean(0).sign().to(torch.bfloat16)      # a small weight for its own token's heads
    b.v[row, 1, a] = value
    b.att.write(b.cache, b.k, b.v, b.table)
    out, lse = b.forward()
    assert b.att.device_status() == 0
    keys, vals, q, at = b.rows("k"), [_as_read(x) for x in b.rows("v")], f64(b.q), 0
    shows = value != 3.1e38
    assert np.isinf(vals[1]).sum() == shows
    some = shows
    for n, c in enumerate(chunks):
        o, l = f64(out[at:at + c]), f64(lse[:, at:at + c])
        for h in range(8):
            g = h // 4
            V = vals[n][:, g:g + 1]
            ref = C.attend(q[at:at + c, h:h + 1], keys[n][:, g:g + 1], np.where(np.isinf(V), 0.0, V), 1, softcap=softcap)
            sure = np.ones((c, d), bool)
            if n == 1 and g == 1 and shows:
                assert not np.isfinite(o[:, h, a]).any(), h
                sure[:, a] = False
            elif n == 1 and g == 1:
                # finite where sums with weights of up to 2^8 times exp(t - the row's largest t) are (the header)
                u = q[at:at + c, h] @ keys[n][:, g].T / np.sqrt(d)
                u = softcap * np.tanh(u / softcap) if softcap else u
                u = np.where(np.arange(len(V)) > np.arange(200, 200 + c)[:, None], -np.inf, u)
                sure[:, a] = 2.0 ** 8 * np.exp(u - u.max(1, keepdims=True)) @ np.abs(V[:, 0, a]) < 2.0 ** 128
                some |= sure[:, a].any()
            assert ((np.abs(o[:, h] - ref["o"][:, 0]) <= ref["tol_o"][:, 0]) | ~sure).all(), (n, h)
            assert (np.abs(l[h] - ref["lse"][0]) <= ref["tol_lse"][0]).all(), (n, h)
        at += c
    assert some or softcap                      # (capped at 5, every row's weights are too near one another)


@DIMS
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("exponent", [-123, -121, -119, -117])
@pytest.mark.parametrize("gain", [0.2, 4.0])
def test_values_of_the_least_scales(F, gain, exponent, rows, d):
    """Scale bytes 0 to some 5, with maxima that rise by less and by more than the slack of the weights' reference."""
    b = Batch(F, ROWS[rows], [600, 300, 200], 8, 2, d, "e4m3", 16, seed=38, gain=gain)
    b.fill("v", bf16(np.random.default_rng(39), *b.cache.v.shape, gain=2.0 ** exponent))
    assert max(0, exponent + 119) <= b.cache.v_scales.min() <= max(0, exponent + 120)
    b.check()


@DIMS
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("queries,keys", [(118, -122), (119, -118), (110, -110), (-110, 110), (-118, 118)])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_queries_and_keys_of_opposite_size(F, softcap, queries, keys, rows, d):
    """Scores of some units from queries and keys at either end of their type's range, a key's scale byte of 0 among them."""
    b = Batch(F, ROWS[rows], [600, 300, 200], 8, 2, d, "e4m3", 16, seed=40, softcap=softcap, scale=2.0 ** -(queries + keys) / np.sqrt(d))
    rng = np.random.default_rng(41)
    b.q.copy_(bf16(rng, *b.q.shape, gain=2.0 ** queries))
    b.fill("k", bf16(rng, *b.cache.k.shape, gain=2.0 ** keys))
    assert (b.cache.k_scales == 0).any() or keys != -122
    b.check()


# ------------------------------------------------------------------ tensors that take another's place

@BOTH
def test_restored_pages(F, fmt):
    """Pages assigned anew are what the calls read and write from then on, and the old ones' memory is left alone."""
    import torch
    b = Batch(F, [1, 40], [60, 100], 4, 2, 64, fmt, 16, seed=42)
    want = [t.clone() for t in b.check()]
    names = ["k", "v"] + (["k_scales", "v_scales"] if fmt == "e4m3" else [])
    old = {n: getattr(b.cache, n) for n in names}
    for n in names:
        setattr(b.cache, n, old[n].clone())
        old[n].fill_(7)
    assert all(torch.equal(x, y) for x, y in zip(b.forward(), want))
    b.att.write(b.cache, b.k, b.v, b.table)
    torch.cuda.synchronize()
    assert all((old[n] == 7).all() for n in names)
    k, v = b.att.read(b.cache, b.table, torch.empty_like(b.k), torch.empty_like(b.v))
    at = b.places()
    for name, got in (("k", k), ("v", v)):
        assert np.array_equal(f64(got), b.pool(name)[at[:, 0], :, at[:, 1]])
    with pytest.raises(F.FlamiaError, match="k: want"):
        b.cache.k = b.cache.k.cpu()


def test_plans_and_outputs_take_turns(F):
    """A plan kept for later and outputs of their own for each layer, by assignment."""
    import torch
    b = Batch(F, [1, 40], [900, 100], 4, 2, 64, page=16, seed=43)
    want = [t.clone() for t in b.check()]
    mine, first = b.att.plan, b.att.out
    other = torch.zeros_like(mine)
    b.att.plan = other
    b.att.plan_build(b.cu, torch.ones_like(b.kv_lens))                # bad: O 0
    assert (b.forward()[0] == 0).all() and b.att.device_status() == F.DEV_BAD_KV_LENS
    b.att.plan, b.att.out, b.att.lse = mine, torch.empty_like(b.att.out), torch.empty_like(b.att.lse)
    b.att.workspace = torch.full_like(b.att.workspace, 255)
    out, lse = b.forward()
    assert out is b.att.out and torch.equal(out, want[0]) and torch.equal(lse, want[1]) and (first == 0).all()
    assert b.att.device_status() == 0
    with pytest.raises(F.FlamiaError, match="workspace: want"):
        b.att.workspace = b.att.workspace[:-256]
