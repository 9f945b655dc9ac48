"""Scored attention and the bucketed relative bias on the GPU against the 64-bit definition.

Every bound is elementwise and counts roundings: half a step of bf16 (2^-8 of the value) for each
probability or score gradient that enters a product and for each output, fp32 roundings (2^-24)
for the products' terms and the sums."""
import numpy as np
import pytest

import scored_ref as S

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


def bf16(rng, *shape, gain=1.0):
    import torch
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * gain).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def dev(x, dtype):
    import torch
    return None if x is None else torch.tensor(np.asarray(x), dtype=dtype).cuda()


class Problem:
    def __init__(self, F, lengths, hq=2, hkv=1, d=64, pad=0, seed=0, causal=True, window=(-1, -1), softcap=0.0, slopes=None,
                 prefix=None, buckets=None, rel=None, gain=2.0, scale=0.0):
        import torch
        rng = np.random.default_rng(seed)
        self.F, self.lengths, self.hq, self.hkv, self.d = F, list(lengths), hq, hkv, d
        self.T = sum(lengths) + pad
        self.q, self.k, self.v = bf16(rng, self.T, hq, d, gain=gain), bf16(rng, self.T, hkv, d), bf16(rng, self.T, hkv, d)
        self.do = bf16(rng, self.T, hq, d)
        self.cu = dev(np.concatenate([[0], np.cumsum(lengths)]), torch.int32)
        slopes = np.linspace(0.5, 0.01, hq) if slopes is True else slopes
        self.slopes = dev(slopes, torch.float32)
        self.prefix = dev(prefix, torch.int32)
        self.table = None
        if buckets:
            self.table = dev(rng.standard_normal((buckets[0], hq)) * 2, torch.float32)
            rel, self.ids = S.bucket_bias(f64(self.table), buckets[1], buckets[2], buckets[1])
        self.buckets, self.rel, self.scale = buckets, rel, scale
        self.ref_kw = dict(lengths=lengths, window=(window[0], 0 if causal else window[1]), softcap=softcap,
                           slopes=None if slopes is None else f64(self.slopes), prefix=prefix, rel=rel,
                           scale=scale if scale > 0 else None)
        self.att = F.FlamiaScoredAttention(self.T, len(lengths), hq, hkv, d, causal=causal, window=window, softcap=softcap,
                                           buckets=buckets)
        self.att.plan_build(self.cu)
        self.extra = dict(softmax_scale=scale, slopes=self.slopes, prefix_lens=self.prefix, table=self.table)

    def forward(self):
        return self.att.forward(self.q, self.k, self.v, self.cu, **self.extra)

    def backward(self, out, lse):
        return self.att.backward(self.q, self.k, self.v, out, lse, self.do, self.cu, **self.extra)

    def check(self, q=None):
        import torch
        for t in (self.att.out, self.att.lse, self.att.dq, self.att.dk, self.att.dv):
            t.fill_(float("nan"))
        out, lse = self.forward()
        got = self.backward(out, lse)
        torch.cuda.synchronize()
        assert self.att.device_status() == 0
        n = sum(self.lengths)
        z = lambda t: np.where(np.arange(self.T)[:, None, None] < n, f64(t), 0)
        ref = S.run(z(self.q), z(self.k), z(self.v), dout=z(self.do), out=f64(out), lse=f64(lse), **self.ref_kw)
        pairs = [("o", out), ("lse", lse)] + list(zip(("dq", "dk", "dv"), got))
        for name, t in pairs:
            within(name, f64(t), ref[name], ref["tol_" + name])
        if self.table is not None:
            one = (self.ids[None, :] == np.arange(self.buckets[0])[:, None]).astype(float)
            want, tol = one @ ref["drel"].T, one @ ref["tol_drel"].T
            within("dtable", f64(got[3]), want, tol + 2.0 ** -24 * len(self.ids) * (one @ np.abs(ref["drel"]).T))
        return out, lse, got


def within(name, got, want, tol):
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine]), name
    assert np.isfinite(got[fine]).all(), name
    over = np.abs(got[fine] - want[fine]) - tol[fine]
    assert (over <= 0).all(), f"{name}: {over.max():.3e} over its bound at {np.argmax(over)} of {over.size}"


LAYOUTS = {
    "one": [1], "tiny": [5, 1, 2], "tile": [128], "tile+1": [129], "two": [256, 255], "odd": [300, 77, 0, 129, 1, 513],
    "empty_docs": [0, 0, 70, 0],
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_layouts_causal_cap(F, layout, d):
    Problem(F, LAYOUTS[layout], 4, 2, d, pad=3, softcap=5.0, seed=1).check()


MODS = {
    "plain": {}, "cap": dict(softcap=10.0), "cap_saturated": dict(softcap=0.5), "cap_large": dict(softcap=1e4),
    "slopes": dict(slopes=True), "slopes_steep": dict(slopes=[8.0, 0.0, 2.0, 0.001]),
    "prefix": dict(prefix=[200, 0, 129]), "prefix_over": dict(prefix=[1000, -4, 1]),
    "buckets": dict(buckets=(32, 128, False)), "buckets_far": dict(buckets=(16, 400, False)),
    "buckets_few": dict(buckets=(4, 3, False)), "cap_slopes": dict(softcap=8.0, slopes=True),
    "all": dict(softcap=8.0, slopes=True, buckets=(16, 60, False), prefix=[10, 64, 129]),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mod", MODS)
def test_scores_causal(F, mod, d):
    Problem(F, [300, 64, 129], 4, 4, d, seed=2, **MODS[mod]).check()


@pytest.mark.parametrize("window", [(-1, -1), (100, -1), (0, 0), (17, 40), (-1, 130), (200, 0)])
@pytest.mark.parametrize("mod", ["cap", "slopes", "prefix", "buckets"])
def test_scores_windows(F, mod, window):
    kw = dict(MODS[mod])
    if mod == "buckets":
        kw["buckets"] = (32, 90, True)
    Problem(F, [390, 1, 131], 2, 1, 64, seed=3, causal=False, window=window, pad=5,
            **dict(kw, prefix=[5, 0, 131] if mod == "prefix" else None)).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (8, 2), (6, 6)])
def test_shared_heads(F, hq, hkv):
    Problem(F, [200, 130], hq, hkv, 128, seed=4, softcap=20.0, slopes=True, buckets=(8, 40, False)).check()


@pytest.mark.parametrize("d", [64, 128])
def test_longer_documents(F, d):
    Problem(F, [1500, 700], 2, 1, d, seed=5, softcap=30.0, prefix=[333, 0], buckets=(32, 512, False), gain=4.0).check()


@pytest.mark.parametrize("causal", [True, False])
def test_sliding_window_skips_tiles(F, causal):
    Problem(F, [1700], 2, 2, 128, seed=6, causal=causal, window=(150, 60), softcap=30.0, prefix=[140]).check()


def test_given_scale_and_large_scores(F):
    Problem(F, [260], 2, 2, 64, seed=7, scale=1.0, gain=4.0).check()


# ------------------------------------------------------------------ masks, garbage, edges of the range

def bits(*ts):
    import torch
    return [t.clone().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32) for t in ts]


def same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


def run_all(p):
    import torch
    out, lse = p.forward()
    got = p.backward(out, lse)
    torch.cuda.synchronize()
    assert p.att.device_status() == 0
    return bits(out, lse, *got)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(softcap=9.0, prefix=[30, 100]), dict(slopes=True, causal=False),
                                dict(buckets=(16, 40, False))], ids=["cap", "slopes", "buckets"])
def test_rows_behind_the_last_document_may_hold_anything(F, d, kw):
    import torch
    p = Problem(F, [150, 131], 4, 2, d, pad=200, seed=11, **kw)
    want = run_all(p)
    for fill in (float("nan"), float("inf")):
        for t in (p.q, p.k, p.v, p.do):
            t[281:] = fill
        p.att.out.fill_(float("nan"))
        p.att.dk.fill_(float("nan"))
        assert same(run_all(p), want)
    assert (p.att.out[281:] == 0).all() and torch.isinf(p.att.lse[:, 281:]).all() and (p.att.dv[281:] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_document_of_infinities_stays_alone(F, d):
    kw = dict(softcap=9.0, buckets=(16, 40, True), causal=False)
    p = Problem(F, [100, 77, 259], 2, 1, d, seed=12, **kw)
    want = run_all(p)
    for t, x in ((p.q, float("nan")), (p.k, float("inf")), (p.v, float("-inf")), (p.do, float("nan"))):
        t[100:177] = x
    out, lse = p.forward()
    got = bits(out, lse.t(), *p.backward(out, lse)[:3])
    want = [want[0], want[1].t()] + want[2:5]
    for rows in (slice(0, 100), slice(177, 436)):
        assert same([t[rows].contiguous() for t in got], [t[rows].contiguous() for t in want])


@pytest.mark.parametrize("value", [float("-inf"), -3.4028234663852886e38, -2.0 ** 101])
@pytest.mark.parametrize("far", [False, True])
def test_a_bias_that_hides(F, value, far):
    """Hidden buckets: near ones (the row's own key among them) leave a document's first rows empty."""
    p = Problem(F, [200, 3, 140], 2, 2, 64, seed=13, buckets=(8, 20, False))
    p.table[(slice(6, 8) if far else slice(0, 3)), 1] = value
    p.ref_kw["rel"] = S.bucket_bias(f64(p.table), 20, False, 20)[0]
    out, lse, got = p.check()
    if not far:
        empty = [0, 1, 2, 200, 201, 202, 203, 204, 205]
        assert (out[empty, 1] == 0).all() and (got[0][empty, 1] == 0).all() and np.isinf(f64(lse)[1, empty]).all()
    assert (got[3][6 if far else 0, 1] == 0).all()


@pytest.mark.parametrize("nb,md,both", [(73, 905, False), (146, 905, True), (21, 1006, False), (32, 128, True), (24, 96, False),
                                        (64, 1024, True), (1024, 1024, True), (1023, 1023, False), (2, 2, False)])
def test_buckets_at_their_borders(F, nb, md, both):
    """Every distance of the table's range: on a border, just below one (73, 905: 347 by 3.7e-10), just above."""
    import torch
    R = min(md + 3, 1024)
    want = np.array([S.bucket(r, nb, md, both) for r in range(-R, R + 1)])
    table = torch.arange(nb, dtype=torch.float32, device="cuda")[:, None].repeat(1, 3) * torch.tensor([1.0, 2.0, 0.0], device="cuda")
    rel = torch.full((3, 2 * R + 1), float("nan"), device="cuda")
    F.flamia_relbias_expand(table.contiguous(), md, both, rel)
    assert np.array_equal(f64(rel), np.stack([want, 2 * want, 0 * want]))
    dtable = torch.full((nb, 3), float("nan"), device="cuda")
    counts = torch.ones_like(rel) * torch.tensor([[1.0], [3.0], [0.0]], device="cuda")
    F.flamia_relbias_reduce(counts, md, both, dtable)
    n = np.bincount(want, minlength=nb)
    assert np.array_equal(f64(dtable), np.stack([n, 3 * n, 0 * n], 1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["table", "slopes"])
def test_nan_parameters_show(F, what, d):
    """A NaN in a head's table or slope is not a number that counts: its rows are NaN, other heads keep their bits."""
    import torch
    p = Problem(F, [200, 140], 4, 4, d, seed=36, buckets=(8, 20, False), slopes=True)
    out, lse = (t.clone() for t in p.forward())
    want = [t.clone() for t in p.backward(out, lse)]
    if what == "table":
        p.table[5, 1] = float("nan")                       # distances 6 to 8
    else:
        p.slopes[1] = float("nan")
    far = np.concatenate([np.arange(n) >= 8 for n in (200, 140)])
    o, l = p.forward()
    got = p.backward(o, l)
    torch.cuda.synchronize()
    assert p.att.device_status() == 0
    assert np.isnan(f64(o)[far, 1]).all() and np.isnan(f64(l)[1, far]).all() and np.isnan(f64(got[0])[far, 1]).all()
    others = [0, 2, 3]
    assert torch.equal(o[:, others], out[:, others]) and torch.equal(l[others], lse[others])
    assert all(torch.equal(a[:, others], b[:, others]) for a, b in zip(got, want))


def test_largest_relative_range(F):
    Problem(F, [2300], 1, 1, 64, seed=14, buckets=(64, 1024, True), causal=False).check()


@pytest.mark.parametrize("scale", [1e-6, 0.02, 3.0])
def test_scales(F, scale):
    Problem(F, [140, 60], 2, 1, 128, seed=15, scale=scale, softcap=4.0, slopes=True).check()


@pytest.mark.parametrize("cap", [1e-3, 0.05, 700.0, 1e6])
def test_caps_of_every_size(F, cap):
    Problem(F, [140, 60], 2, 1, 128, seed=16, softcap=cap, gain=4.0).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,scale", [(1e-8, 0.0), (2e-7, 0.0), (1e-30, 0.0), (5.0, 0.0), (1.0, 1e30), (1e-8, 1e22)])
def test_caps_that_dwarf_the_scores_and_products_of_zero(F, cap, scale, d):
    """A cap far below the scores (folded coefficients past the fp32 range), with blocks of hidden pairs on the
    diagonal, a head whose queries are zero and a document whose keys are."""
    p = Problem(F, [140, 64, 60], 4, 2, d, seed=16, softcap=cap, scale=scale)
    p.q[:, 1] = 0
    p.k[140:204] = 0
    p.check()


def forward_within(p, u):
    """The forward of causal documents against the softmax of u(head, rows, queries, keys), where the scores are so
    large that a row is its largest key's alone."""
    import torch
    out, lse = p.forward()
    torch.cuda.synchronize()
    assert p.att.device_status() == 0
    base = 0
    for n in p.lengths:
        rows = slice(base, base + n)
        base += n
        for h in range(p.hq):
            hk = h // (p.hq // p.hkv)
            s = u(h, rows, f64(p.q[rows, h]) @ f64(p.k[rows, hk]).T)
            s = np.where(np.tri(n, dtype=bool), s, -np.inf)
            top, two = s.max(1), np.sort(s, 1)[:, -2] if n > 1 else np.full(n, -np.inf)
            # decided whatever the roundings: (d + 8) 2^-24 of a product's terms, which add up to some 30 times it
            sure = top - two > 2.0 ** -12 * np.abs(top) + 200
            assert sure.mean() > 0.9
            v = f64(p.v[rows, hk])[s.argmax(1)]
            assert np.isfinite(f64(out[rows, h])).all()
            assert (np.abs(f64(out[rows, h]) - v)[sure] <= 2.1 * 2.0 ** -8 * np.abs(v[sure])).all()
            assert (np.abs(f64(lse[h, rows]) - top) <= 2.0 ** -12 * np.abs(top) + 64).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,scale", [(0.0, 1e30), (0.0, 1e10), (0.0, 1e7), (1e28, 1e30), (1e13, 1e10)])
def test_scores_beyond_any_use(F, cap, scale, d):
    """x - m is taken of rounded values: an exact product less a rounded maximum would reach 2^128."""
    p = Problem(F, [300, 129, 1], 2, 1, d, seed=33, softcap=cap, scale=scale)
    if cap == 1e28:
        p.q[:, 1] = 0                          # folded coefficients past the range meet products of 0
        p.forward()
        assert np.isfinite(f64(p.att.out)).all()
        p.q[:, 1] = p.q[:, 0]
        p.q /= 8192                            # capped, but not all to the same
    forward_within(p, lambda h, rows, x: cap * np.tanh(scale * x / cap) if cap else scale * x)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slopes", [None, [0.5, 0.01]])
@pytest.mark.parametrize("offset", [1e12, -1e12, -1e30, 1e30, 3e38])
def test_a_bias_beyond_any_use(F, offset, slopes, d):
    """Large scores under a bias that leaves them no digits: finite, and a mean of the document's values."""
    import torch
    p = Problem(F, [500, 1], 2, 1, d, seed=34, gain=40.0, buckets=(32, 64, False), slopes=slopes, pad=2)
    p.table += offset
    p.v.copy_(p.v.abs())
    out, lse = p.forward()
    torch.cuda.synchronize()
    o, v = f64(out), f64(p.v)
    assert np.isfinite(o).all() and (o[:500] <= 1.01 * v[:500].max(0)).all() and (o[:500] >= 0.99 * v[:500].min(0)).all()
    limit = min(abs(offset), 2.0 ** 100)
    assert (np.abs(np.abs(f64(lse)[:, :501]) - limit) <= 1e-6 * limit + 1e4).all()
    assert np.array_equal(o[500], np.repeat(v[500], 2, 0))
    for t in p.backward(out, lse):                         # no LSE says what P was
        assert (t == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_rows_without_a_usable_lse_give_no_gradient(F, d, cap):
    """A bias of -1e9 for the nearest keys, as masks are often written: a document's first rows see nothing else, and
    the others weigh those keys 0.  The gradients are those of the other rows."""
    import torch
    p = Problem(F, [300, 3, 140], 4, 2, d, seed=35, softcap=cap, buckets=(8, 20, False))
    p.table[:4, 1] = -1e9
    out, lse = p.forward()
    got = [f64(t) for t in p.backward(out, lse)]
    few = np.concatenate([np.arange(n) < 4 for n in p.lengths])          # buckets 0 .. 3 are the distances 0 .. 3
    assert np.array_equal(np.abs(f64(lse[1])) > 2.0 ** 23, few)
    assert (np.abs(f64(lse[[0, 2, 3]])) < 1e4).all()
    rel, _ = S.bucket_bias(f64(p.table), 20, False, 20)
    rel = np.where(rel < -1e8, -np.inf, rel)                             # what it amounts to for every other row
    keep = np.where(few, np.inf, f64(lse[1]))
    ref_lse = f64(lse)
    ref_lse[1] = keep
    ref = S.run(f64(p.q), f64(p.k), f64(p.v), dout=f64(p.do), out=f64(out), lse=ref_lse, **dict(p.ref_kw, rel=rel))
    for name, t in zip(("dq", "dk", "dv"), got):
        within(name, t, ref[name], ref["tol_" + name])
    assert (got[0][few][:, 1] == 0).all() and (got[3][:4, 1] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 9.0])
@pytest.mark.parametrize("scale", [0.0, 1e-30])
@pytest.mark.parametrize("causal", [True, False])
def test_slopes_of_every_size(F, d, cap, scale, causal):
    """Finite slopes up to the type's largest: a key a step farther weighs e^-slope less, here 0, so a row is its own
    key's alone."""
    import torch
    p = Problem(F, [300, 1, 129], 4, 4, d, pad=3, seed=19, causal=causal, softcap=cap, scale=scale,
                slopes=[3.4e38, 2.0 ** 100, 1e30, 3e9])
    out, lse = p.forward()
    dq, dk, dv = p.backward(out, lse)
    torch.cuda.synchronize()
    assert torch.equal(out[:430], p.v[:430]) and torch.equal(dv[:430], p.do[:430])
    q, k, v, do = (f64(t[:430]) for t in (p.q, p.k, p.v, p.do))
    u = (scale or d ** -0.5) * (q * k).sum(2)
    u = cap * np.tanh(u / cap) if cap else u
    # the product's d terms and some roundings of the value itself
    tol = 2.0 ** -24 * ((d + 8) * (scale or d ** -0.5) * np.abs(q * k).sum(2) + 16 * np.abs(u) + 16 * cap) + 2.0 ** -120
    assert (np.abs(f64(lse)[:, :430] - u.T) <= tol.T).all()
    # dP - D of equal sums: their roundings, times P = 1 (1 + 8 roundings of 1 + |LSE|)
    ds = 2.0 ** -24 * 2 * (d + 8) * np.abs(do * v).sum(2, keepdims=True) * (scale or d ** -0.5) + 2.0 ** -126
    assert (np.abs(f64(dq[:430])) <= 2 * ds * np.abs(k) + 2.0 ** -126).all()
    assert (np.abs(f64(dk[:430])) <= 2 * ds * np.abs(q) + 2.0 ** -126).all()


@pytest.mark.parametrize("d", [64, 128])
def test_steep_negative_slopes(F, d):
    """The farthest key takes all: a causal row is its document's first."""
    p = Problem(F, [300, 129], 3, 3, d, seed=20, slopes=[-3.4e38, -1e30, -3e6])
    out, lse = p.forward()
    first = np.repeat([0, 300], [300, 129])
    # P and O are rounded, half a step each; P need not be 1 where the bias leaves the scores no digits
    assert (np.abs(f64(out) - f64(p.v)[first]) <= 2.1 * 2.0 ** -8 * np.abs(f64(p.v)[first])).all()
    assert np.isfinite(f64(lse)).all()


def test_negative_slopes_and_many_documents(F):
    Problem(F, [1] * 40 + [7] * 20 + [129] * 3, 3, 3, 64, seed=17, slopes=[-0.4, 0.0, 1.0], pad=1).check()


@pytest.mark.parametrize("d", [64, 128])
def test_units_dealt_out_and_taken_over(F, d):
    """Many units are dealt out in rounds, fewer are taken over by whoever is free: a document's bits are the same."""
    import torch
    lengths = [300] + [40 + i % 50 for i in range(75)]
    many, few = (Problem(F, ls, 64, 8, d, pad=9, softcap=6.0) for ls in (lengths, lengths[:1]))
    for a in ("q", "k", "v"):
        getattr(few, a).copy_(getattr(many, a)[:309])
    out, lse, _ = many.check()
    o, l = few.forward()
    torch.cuda.synchronize()
    assert torch.equal(o[:300], out[:300]) and torch.equal(l[:, :300], lse[:, :300])
    assert torch.count_nonzero(o[300:]) == 0 and torch.isposinf(l[:, 300:]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (16, 8)])
def test_runs_of_one_tile_units(F, hq, hkv, d):
    """Documents of up to 128 rows: the second query tile's warps have nothing to do for many units on end, until
    the one document of two tiles.  4 heads: units taken over; 16: dealt out."""
    rng = np.random.default_rng(7)
    lengths = [int(x) for x in rng.integers(1, 129, 300)]
    lengths[250] = 200
    Problem(F, lengths, hq, hkv, d, pad=7, seed=18, slopes=True, buckets=(16, 40, False)).check()


def test_no_valid_tokens(F):
    Problem(F, [0, 0, 0], 4, 2, 64, pad=300, slopes=True, causal=False).check()


def test_no_tokens(F):
    import torch
    att = F.FlamiaScoredAttention(0, 2, 2, 1, 64, buckets=(8, 20, False))
    cu = dev([0, 0, 0], torch.int32)
    att.plan_build(cu)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    out, lse = att.forward(z(0, 2, 64), z(0, 1, 64), z(0, 1, 64), cu, table=z(8, 2, dtype=torch.float32))
    att.drel_bias.fill_(3.0)
    got = att.backward(z(0, 2, 64), z(0, 1, 64), z(0, 1, 64), out, lse, out, cu, table=z(8, 2, dtype=torch.float32))
    assert out.numel() == 0 and (got[3] == 0).all()
    Problem(F, [0, 0], 2, 1, 64, pad=5, softcap=3.0).check()


def test_calls_before_the_plan(F):
    """Refused before a launch; a plan whose building is captured but not replayed holds no documents."""
    import torch
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    q, k, lse, cu = z(40, 2, 64), z(40, 1, 64), z(2, 40, dtype=torch.float32), dev([0, 30, 40], torch.int32)
    att = F.FlamiaScoredAttention(40, 2, 2, 1, 64)
    assert torch.count_nonzero(att.plan) == 0
    for call in (lambda: att.forward(q, k, k, cu), lambda: att.backward(q, k, k, q, lse, q, cu)):
        with pytest.raises(F.FlamiaError, match="plan_build"):
            call()
    att.plan_build(cu)
    torch.cuda.synchronize()
    att.plan.zero_()
    out, lse = att.forward(q, k, k, cu)
    got = att.backward(q, k, k, out, lse, q, cu)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isposinf(lse).all() and all((g == 0).all() for g in got)


def test_bad_cu_seqlens(F):
    import torch
    p = Problem(F, [100, 28], 2, 1, 64, seed=18, softcap=3.0)
    p.cu.copy_(dev([0, 90, 40], torch.int32))
    p.att.plan_build(p.cu)
    out, lse = p.forward()
    got = p.backward(out, lse)
    assert p.att.device_status() == F.DEV_BAD_CU_SEQLENS
    assert (out == 0).all() and torch.isinf(lse).all() and all((g == 0).all() for g in got)


# ------------------------------------------------------------------ how the calls are made

KW = dict(softcap=20.0, slopes=True, buckets=(16, 100, False), prefix=[50, 0])


def test_equal_inputs_give_equal_bits(F):
    p = Problem(F, [900, 333], 6, 2, 128, seed=21, **KW)
    want = run_all(p)
    for _ in range(3):
        assert same(run_all(p), want)


FORMS = {
    "plain": dict(hkv=16), "cap": dict(hkv=16, softcap=50.0), "slopes": dict(hkv=8, slopes=True),
    "prefix": dict(hkv=8, softcap=30.0, prefix=[1500, 0, 2999, 1, 129, 700, 64, 0, 33, 200, 4]),
    "buckets": dict(hkv=16, buckets=(32, 128, False)),
    "cap_buckets": dict(hkv=8, softcap=50.0, slopes=True, buckets=(32, 100, False)),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_bits_do_not_depend_on_when_a_load_lands(F, form, d):
    """Many units per SM, operands from memory (L2 is overwritten and another problem runs in between): a product
    that does not wait for its tile multiplies by what its stage held before."""
    import torch
    lengths = [4000, 129, 2886, 84, 1500, 3000, 700, 513, 2048, 1024, 500]
    p = Problem(F, lengths, 16, d=d, seed=41, **FORMS[form])
    other = Problem(F, [3000, 1000], 16, 16, d, seed=42, causal=False)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    o_out, o_lse = other.forward()
    out, lse = (t.clone() for t in p.forward())
    want = bits(out, lse, *p.backward(out, lse))
    wrong = torch.zeros(len(want), dtype=torch.int64, device="cuda")
    for i in range(100):
        other.backward(o_out, o_lse)
        flush.fill_(i)
        p.forward()
        flush.fill_(i)
        got = p.backward(out, lse)
        wrong += torch.stack([(a != b).sum() for a, b in zip(bits(p.att.out, p.att.lse, *got), want)])
    assert wrong.tolist() == [0] * len(want)
    assert p.att.device_status() == 0


# Each with more units than SMs, several per CTA, and documents longer than the rings of tiles: what one unit or
# head leaves behind for the next (tables, sums, tensor memory, barriers' phases).
UNITS = {
    "slopes_128": dict(hq=8, hkv=8, d=128, slopes=True),
    "plain_128": dict(hq=8, hkv=8, d=128),
    "plain_64": dict(hq=8, hkv=8, d=64),
    "cap_64": dict(hq=8, hkv=8, d=64, softcap=12.0),
    "slopes_noncausal_128": dict(hq=6, hkv=6, d=128, slopes=True, causal=False),
    "buckets_128": dict(hq=12, hkv=12, d=128, buckets=(16, 90, False)),
    "buckets_shared_128": dict(hq=16, hkv=8, d=128, buckets=(16, 90, False)),
    "buckets_shared_64": dict(hq=16, hkv=8, d=64, buckets=(16, 200, True), causal=False),
    "all_shared_128": dict(hq=16, hkv=8, d=128, softcap=9.0, slopes=True, buckets=(16, 90, False), window=(300, -1),
                           prefix=[100, 0, 650, 7, 33, 129, 1]),
    "all_shared_64": dict(hq=16, hkv=8, d=64, softcap=9.0, slopes=True, buckets=(16, 200, True), causal=False,
                          prefix=[100, 0, 650, 7, 33, 129, 1]),
}


@pytest.mark.parametrize("form", UNITS)
def test_many_units_against_the_definition(F, form):
    kw = dict(UNITS[form])
    lengths = [1300, 700, 900, 129, 513, 1100, 650]
    if kw["hq"] > kw["hkv"]:                               # enough of them that query heads share a dK/dV unit
        lengths, kw["prefix"] = lengths + [830, 470, 600, 700, 500], kw["prefix"] + [0, 300, 2, 700, 0] if "prefix" in kw else None
        assert (sum(lengths) // 128 + len(lengths) + 1) * kw["hkv"] >= 608
    Problem(F, lengths, pad=6, seed=43, **kw).check()


def test_any_plan_of_the_same_documents(F):
    p = Problem(F, [700, 333], 2, 1, 64, seed=22, window=(200, -1), softcap=20.0)
    want = run_all(p)
    F.flamia_plan_build(p.cu, 2, p.T, p.att.plan)          # a plan of the plain causal call
    assert same(run_all(p), want)


def test_captured_and_replayed(F):
    import torch
    p = Problem(F, [700, 333], 4, 2, 128, seed=23, **KW)
    want = run_all(p)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        p.att.plan_build(p.cu)
        out, lse = p.forward()
    with torch.cuda.graph(g2):
        p.backward(out, lse)
    outs = (p.att.out, p.att.lse, p.att.dq, p.att.dk, p.att.dv, p.att.dtable)
    for _ in range(2):
        for t in outs:
            t.fill_(float("nan"))
        p.att.workspace.fill_(255)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert same(bits(*outs), want)


def test_other_streams_and_two_calls_at_once(F):
    import torch
    p1 = Problem(F, [1500, 333], 4, 2, 128, seed=24, **KW)
    p2 = Problem(F, [64, 2000], 8, 8, 64, seed=25, softcap=5.0, causal=False)
    want = run_all(p1), run_all(p2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in ((p1, s1), (p2, s2)):
            p.extra["stream"] = s
            out, lse = p.forward()
            p.backward(out, lse)
    torch.cuda.synchronize()
    for p, w in ((p1, want[0]), (p2, want[1])):
        a = p.att
        assert same(bits(a.out, a.lse, a.dq, a.dk, a.dv, *([a.dtable] if p.table is not None else [])), w)


def test_two_calls_on_one_plan(F):
    """The plan is only read: two forwards on it overlap."""
    import torch
    p = Problem(F, [1500, 700], 4, 4, 128, seed=26, softcap=20.0)
    want = bits(*p.forward())
    o = F.default_score_options()
    o.softcap = 20.0
    outs = [(torch.empty_like(p.att.out), torch.empty_like(p.att.lse)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for (out, lse), s in zip(outs, streams):
        F.flamia_scored_fwd(p.q, p.k, p.v, p.cu, 2, p.att.plan, out, lse, opts=o, stream=s)
    torch.cuda.synchronize()
    for x in outs:
        assert same(bits(*x), want)


def test_outputs_at_the_smallest_alignment(F):
    """16-byte aligned tensors (views that start eight elements into an allocation)."""
    import torch
    p = Problem(F, [300, 77], 2, 1, 64, seed=27, softcap=20.0)
    want = run_all(p)

    def moved(t):
        n = 16 // t.element_size()
        buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        v = buf[n:].view(t.shape)
        v.copy_(t)
        return v
    for n in ("q", "k", "v", "do"):
        setattr(p, n, moved(getattr(p, n)))
    for n in ("out", "dq", "dk", "dv", "lse"):
        setattr(p.att, n, moved(getattr(p.att, n)))
    assert same(run_all(p), want)


def test_offsets_past_32_bits(F):
    """2.3e9 query elements: the last documents' rows against the definition."""
    import torch
    n, hq, d = 18000, 1000, 128
    lengths = [120] * (n // 120)
    T = n
    att = F.FlamiaScoredAttention(T, len(lengths), hq, 1, d, softcap=20.0)
    cu = dev(np.concatenate([[0], np.cumsum(lengths)]), torch.int32)
    att.plan_build(cu)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    do = torch.empty_like(q).normal_(generator=g)
    k, v = (torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    assert q.numel() > 1 << 31
    out, lse = att.forward(q, k, v, cu)
    dq, dk, dv = att.backward(q, k, v, out, lse, do, cu)
    torch.cuda.synchronize()
    assert att.device_status() == 0
    rows = slice(T - 120, T)
    heads = [0, 1, 499, 998, 999]
    ref = S.run(f64(q[rows][:, heads]), f64(k[rows].expand(-1, 5, -1)), f64(v[rows].expand(-1, 5, -1)), [120],
                dout=f64(do[rows][:, heads]), out=f64(out[rows][:, heads]), lse=f64(lse[heads][:, rows]), softcap=20.0)
    within("o", f64(out[rows][:, heads]), ref["o"], ref["tol_o"])
    within("dq", f64(dq[rows][:, heads]), ref["dq"], ref["tol_dq"])
    assert (out[:5].float().abs().sum((1, 2)) > 0).all() and torch.isfinite(dk.float()).all() and torch.isfinite(dv.float()).all()


def test_layers_of_a_training_step(F):
    """Two layers as a model uses them: capped scores with a prefix, then a bucketed bias; the second's
    gradient with respect to its queries is the first's dO.  Against the definition on the same bf16 values."""
    import torch
    lengths = [400, 57, 130]
    a = Problem(F, lengths, 4, 2, 64, seed=31, softcap=15.0, prefix=[100, 0, 9], gain=3.0)
    b = Problem(F, lengths, 4, 2, 64, seed=32, buckets=(32, 128, False))
    o1, l1 = a.forward()
    b.q = o1.clone()
    o2, l2 = b.forward()
    dq2 = b.backward(o2, l2)
    a.do = dq2[0].clone()
    dq1 = a.backward(o1, l1)
    torch.cuda.synchronize()
    r2 = S.run(f64(b.q), f64(b.k), f64(b.v), dout=f64(b.do), out=f64(o2), lse=f64(l2), **b.ref_kw)
    r1 = S.run(f64(a.q), f64(a.k), f64(a.v), dout=f64(a.do), out=f64(o1), lse=f64(l1), **a.ref_kw)
    for got, ref in ((dq2, r2), (dq1, r1)):
        for name, t in zip(("dq", "dk", "dv"), got):
            within(name, f64(t), ref[name], ref["tol_" + name])
    # a step along the whole chain's gradient lowers <o2, do> by its own size (differences of the bf16 chain)
    eps = 0.02
    dirn = f64(dq1[0]) / np.linalg.norm(f64(dq1[0]))
    q0 = f64(a.q)

    def loss(s):
        a.q = torch.from_numpy(q0 + s * dirn * np.sqrt(dirn.size)).to(torch.bfloat16).cuda()
        b.q = a.forward()[0].clone()
        x = f64(a.q)
        return float((f64(b.forward()[0]) * f64(b.do)).sum()), x
    (hi, xh), (lo, xl) = loss(eps), loss(-eps)
    want = float((f64(dq1[0]) * (xh - xl)).sum())
    # o2 is rounded to bf16 once and o1 in between: 2^-8 of each of the 150,000 terms, random in sign
    noise = 4 * 2.0 ** -8 * np.sqrt(2 * (f64(b.att.out) ** 2 * f64(b.do) ** 2).sum()) + 4 * 2.0 ** -8 * np.sqrt(
        2 * (f64(o1) ** 2 * f64(dq2[0]) ** 2).sum())
    assert abs((hi - lo) - want) <= noise + 0.1 * abs(want)


@pytest.mark.parametrize("docs", [20, 128, 129])
def test_prefix_documents_ranked_or_not(F, docs):
    """Up to 128 work items and more than 152 units the forward ranks the items by their work itself."""
    rng = np.random.default_rng(docs)
    lengths = [int(x) for x in rng.integers(1, 120, docs)]
    lengths[3], lengths[7] = (700, 0) if docs == 20 else (121, 119)
    Problem(F, lengths, 16, 4, 64, pad=5, softcap=8.0, prefix=[int(x) for x in rng.integers(0, 130, docs)], seed=3).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("offset", [300.0, -4000.0])
def test_a_bias_far_from_zero(F, d, offset):
    """A constant added to the whole table changes no probability; only u's own roundings grow."""
    p = Problem(F, [300, 129, 40], 4, 2, d, pad=3, causal=False, buckets=(32, 64, True), seed=5)
    p.table += offset
    p.rel, _ = S.bucket_bias(f64(p.table), p.buckets[1], p.buckets[2], p.buckets[1])
    p.ref_kw["rel"] = p.rel
    p.check()


@pytest.mark.parametrize("d", [64, 128])
def test_captured_twice_in_a_row(F, d):
    """Two whole calls in one graph, one workspace: launches that start early still come behind the call before."""
    import torch
    p = Problem(F, [1500, 333, 700], 4, 4, d, seed=31, causal=False, buckets=(32, 100, True))
    want = run_all(p)
    outs = (p.att.out, p.att.lse, p.att.dq, p.att.dk, p.att.dv, p.att.dtable)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            p.backward(*p.forward())
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert same(bits(*outs), want)
