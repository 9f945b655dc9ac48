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
